"""A decode loop that drafts, verifies and commits, with the target's side on the GPU.

A small random-weight model (one attention layer over a paged cache, an output head)
answers a batch of requests whose histories repeat themselves, as text being copied
does.  Every step, for the whole batch:

    draft          lookup_draft_ex: what followed the last occurrence of the suffix
    block          the last committed token, then the drafted ones
    kv append      lookup_kv_append: the block's queries and keys rotated, cached
    attention      lookup_paged_attention over the cache
    verification   lookup_verify_logits against the head's logits, greedy or sampled
    commit         lookup_append: the next step's histories; kv_len grows by the
                   committed count, so the next block overwrites what was refused

Greedy output equals plain decoding, one token a step (checked at the end, up to
logits that tie within the rounding of their 16-bit inputs).

    python examples/verify_step.py [--steps 32] [--sampled]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import prompt_lookup_speculative_gb300 as pld  # noqa: E402


class Model:
    """Embedding, one attention layer with rotary positions and grouped heads, output head."""

    def __init__(self, vocab: int, hq: int, hkv: int, d: int, max_pos: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n, self.hq, self.hkv, self.d, self.vocab = hq * d, hq, hkv, d, vocab

        def make(*shape, std):
            return (torch.randn(shape, device="cuda", generator=g) * std).to(torch.bfloat16)

        self.embed = make(vocab, n, std=1.0)
        self.qkv = make(n, (hq + 2 * hkv) * d, std=n ** -0.5)
        self.out = make(n, n, std=n ** -0.5)
        # the head sees the token itself besides what attention gathers: copying pays
        self.head = make(n, vocab, std=2.0 * n ** -0.5)
        self.rotary = pld.rotary_table(max_pos, d)

    def logits(self, block, cache, table, kv_len, q_len):
        """The block's tokens [B, N] through the model: logits [B, N, vocab]."""
        B, N = block.shape
        x = self.embed[block.clamp(min=0).long()]
        qkv = (x @ self.qkv).view(B, N, self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], 2)
        q, status = cache.append(q, k, v, kv_len, table, rotary=self.rotary, q_len=q_len)
        a, _ = cache.attention(q, table, kv_len, q_len=q_len)
        h = x + a.reshape(B, N, -1) @ self.out
        return h @ self.head, status


class Batch:
    """Requests with their histories (CSR), their pages and their cached counts."""

    def __init__(self, model: Model, histories, room: int, page: int = 16):
        self.model, B = model, len(histories)
        self.tokens = torch.cat([torch.tensor(h, dtype=torch.int32) for h in histories]).cuda()
        ends = torch.tensor([0] + [len(h) for h in histories]).cumsum(0)
        self.offsets = ends.to(torch.int64).cuda()
        self.lens = torch.tensor([len(h) for h in histories], dtype=torch.int32, device="cuda")
        width = -(-(max(len(h) for h in histories) + room) // page)
        self.table = torch.randperm(B * width, dtype=torch.int32).view(B, width).cuda()
        self.cache = pld.PagedKVCache(B * width, page, model.hkv, model.d)
        # the prompt, all but its last token, which opens the first block
        longest = max(len(h) for h in histories) - 1
        prompt = torch.zeros((B, longest), dtype=torch.int32)
        for r, h in enumerate(histories):
            prompt[r, :len(h) - 1] = torch.tensor(h[:-1])
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.model.logits(prompt.cuda(), self.cache, self.table, self.kv_len, self.lens - 1)
        self.kv_len = self.lens - 1

    def step(self, K: int, sampling=None):
        """One verify step with K drafted tokens (K = 0: plain decoding); returns the commits."""
        B = self.lens.shape[0]
        draft, length, _, _ = pld.lookup_draft_ex(self.tokens, self.offsets, 2, 8, K)
        last = self.tokens[self.offsets[1:] - 1]
        block = torch.cat([last[:, None], draft], 1)
        logits, status = self.model.logits(block, self.cache, self.table, self.kv_len, length + 1)
        out = pld.lookup_verify_logits(draft, length, logits, **(sampling(B, K) if sampling else {}))
        accepted, commit, ncommit, _ = out
        self.tokens, self.offsets = pld.lookup_append(self.tokens, self.offsets, commit, ncommit)
        self.lens = self.lens + ncommit
        self.kv_len = self.kv_len + ncommit
        return commit, ncommit, status


def histories(B: int, vocab: int, seed: int):
    """Requests that end inside a repeated passage."""
    g = torch.Generator()
    g.manual_seed(seed)
    out = []
    for r in range(B):
        passage = torch.randint(vocab, (24 + r % 7,), generator=g).tolist()
        out.append(passage * 3 + passage[:5 + r % 11])
    return out


def generate(model, hist, steps: int, K: int, sampling=None):
    """Every request's committed tokens after `steps` steps."""
    batch = Batch(model, hist, room=steps * (K + 1) + K + 2)
    got = [[] for _ in hist]
    for _ in range(steps):
        commit, ncommit, status = batch.step(K, sampling)
        if int(status.sum()):
            raise RuntimeError("a request ran out of pages")
        for r, n in enumerate(ncommit.tolist()):
            got[r] += commit[r, :n].tolist()
    return got


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--sampled", action="store_true")
    a = ap.parse_args()
    model = Model(a.vocab, hq=8, hkv=2, d=64, max_pos=4096)
    hist = histories(a.requests, a.vocab, 3)
    if a.sampled:
        g = torch.Generator(device="cuda")
        g.manual_seed(1)

        def sampling(B, K):
            return dict(u=torch.rand((B, K), device="cuda", generator=g),
                        noise=torch.empty((B, a.vocab), device="cuda").exponential_(generator=g),
                        temperature=torch.full((B,), 0.8, device="cuda"))

        got = generate(model, hist, a.steps, 15, sampling)
        print(f"sampled: {sum(map(len, got)) / a.steps / a.requests:.2f} tokens per step and request")
        return
    got = generate(model, hist, a.steps, 15)
    plain = generate(model, hist, min(map(len, got)), 0)
    same = sum(p == q for g, w in zip(got, plain) for p, q in zip(g, w))
    total = sum(len(w) for w in plain)
    first = [next((i for i, (p, q) in enumerate(zip(g, w)) if p != q), None) for g, w in zip(got, plain)]
    print(f"greedy: {sum(map(len, got)) / a.steps / a.requests:.2f} tokens per step and request; "
          f"{same} of {total} tokens equal plain decoding's, first differences at {first}")


if __name__ == "__main__":
    main()
