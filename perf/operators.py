"""The target model's side of a verify step, as measured cases.

Three operators: the block's keys and values rotated and written to the paged
cache (``kv_append``), the block's attention over that cache (``attention``), and
the block's verification against the target's logits (``verify``).  ``run`` computes
each in its plain form (elementary torch operations in 32 bits, rounded once), or,
with ``own`` set, through this package's entry points.  ``exact`` restates the
definitions in 64 bits.
"""
import math

import torch

own = False

VOCAB_SMALL, VOCAB = 32000, 151936      # the two vocabularies of the generators
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one chat, a short greedy block (7 proposals), a small vocabulary: the launch itself counts
        dict(name="verify_one", op="verify", B=1, P=7, V=VOCAB_SMALL, type="f32", mode="greedy", pad=0),
        # eight short requests, lookup drafts (point masses), sampled
        dict(name="verify_tiny", op="verify", B=8, P=15, V=VOCAB_SMALL, type="bf16", mode="point", pad=0),
        # 64 requests reciting a document, long blocks (7 head + 8 tail) for half of them
        dict(name="verify_recite", op="verify", B=64, P=15, V=VOCAB, type="bf16", mode="point", pad=0),
        # 64 requests with a draft model's own distribution; a vocabulary padded in the logits' rows
        dict(name="verify_drafted", op="verify", B=64, P=7, V=VOCAB - 1, type="f32", mode="draft", pad=129),
        # one new token of one request
        dict(name="append_one", op="kv_append", B=1, N=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=16,
             lmin=4096, lmax=4096, type="bf16"),
        # the verify blocks of 64 requests of 25000 tokens
        dict(name="append_block", op="kv_append", B=64, N=16, Hq=32, Hkv=4, D=128, rot=128, inter=False, page=64,
             lmin=1000, lmax=25000, type="bf16"),
        # 4096 chats' blocks, a part of the head rotated, neighbours paired
        dict(name="append_chats", op="kv_append", B=4096, N=8, Hq=16, Hkv=2, D=64, rot=32, inter=True, page=32,
             lmin=100, lmax=2048, type="f16"),
        # a prompt of 8191 tokens for each of four requests
        dict(name="append_prompt", op="kv_append", B=4, N=8191, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=64,
             lmin=0, lmax=5, type="bf16"),
        # one new token of one request over 4096 cached ones: latency
        dict(name="attend_one", op="attention", B=1, N=1, Hq=32, Hkv=8, D=128, page=16, lmin=4096, lmax=4096,
             window=0, type="bf16"),
        # plain decoding of 64 requests of up to 25000 tokens
        dict(name="attend_decode", op="attention", B=64, N=1, Hq=32, Hkv=8, D=128, page=64, lmin=12000, lmax=25000,
             window=0, type="bf16"),
        # the verify blocks (last committed token + 15 proposals) of 64 requests of 25000 tokens
        dict(name="attend_block", op="attention", B=64, N=16, Hq=32, Hkv=4, D=128, page=64, lmin=25000, lmax=25000,
             window=0, type="bf16"),
        # ragged long contexts, short blocks, an odd group of heads
        dict(name="attend_ragged", op="attention", B=16, N=8, Hq=14, Hkv=2, D=64, page=32, lmin=512, lmax=262144,
             window=0, type="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "kv_append", "attention"])
    if op == "verify":
        P = rng.choice([0, 1, 2, 3, 5, 7, 7, 11, 15, 15])
        V = _log(rng, 500, VOCAB)
        B = _log(rng, 1, max(1, min(512, 64 * 16 * VOCAB // ((P + 1) * V))))
        return dict(op=op, B=B, P=P, V=V, type=rng.choice(["f32", "bf16", "f16"]) if B * (P + 1) * V < 64 * 8 * VOCAB
                    else rng.choice(["bf16", "f16"]), mode=rng.choice(["greedy", "point", "draft"]),
                    pad=rng.choice([0, 0, 1, 8, 128]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    kind = rng.choice(["bf16", "f16"])
    if op == "kv_append":
        N = rng.choice([1, 1, 2, 7, 8, 16, _log(rng, 17, 4096)])
        B = _log(rng, 1, max(1, min(4096, 4 * 8191 * 48 * 128 // (N * (Hq + 2 * Hkv) * D))))
        lmax = max(1, min(_log(rng, 16, 32768), 400000000 // (B * Hkv * D)))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    inter=rng.random() < 0.4, page=page, lmin=lmax // 3, lmax=lmax, type=kind)
    N = rng.choice([1, 1, 1, 2, 4, 7, 8, 11, 16])
    L = _log(rng, 64, 131072)
    most = min(64 * 25000 * 4 * 128 // (L * Hkv * D), 64 * 25000 * 16 * 32 * 128 // (L * N * Hq * D))
    B = _log(rng, 1, max(1, min(256, most)))
    return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, lmin=max(1, L // rng.choice([1, 3, 20])), lmax=L,
                window=rng.choice([0, 0, 0, 2048, 500]), type=kind)


# ------------------------------------------------------------------ inputs ----
def _lengths(case):
    """Cached tokens of each request, spread over the logarithm from lmin to lmax, the
    same for every seed (what a pass reads depends on them); the last one is lmax."""
    B, lo, hi = case["B"], case["lmin"], case["lmax"]
    out = []
    for r in range(B):
        f = (0.6180339887498949 * (r + 1)) % 1.0 if r + 1 < B else 1.0
        out.append(int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** f)) - 1)
    return out


def _block_lengths(case):
    """Proposals of each request: every second one's block is the short one."""
    P = case["P"]
    return [P if r % 2 == 0 else P // 2 for r in range(case["B"])]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(case, tokens, g):
    """A page table over a shuffled pool with room for `tokens` tokens per request;
    entries past a request's last page are -1."""
    page = case["page"]
    need = [-(-t // page) for t in tokens]
    width = max(1, max(need))
    total = max(1, sum(need))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    start = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(width, device="cuda")
    at = start[:, None] + col
    table = torch.where(col < need_t[:, None], perm[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    return table, total


def prepare(case, seed):
    g = _gen(seed)
    dev, f32 = "cuda", torch.float32
    s = dict(case=case)
    if case["op"] == "verify":
        B, P, V, mode = case["B"], case["P"], case["V"], case["mode"]
        dt = TYPES[case["type"]]
        z = torch.randn((B, P + 1, V), device=dev, generator=g) * 2.5
        lse = math.log(V) + 2.5 * 2.5 / 2
        if mode == "draft":        # the draft model's distribution, near the target's; proposals drawn from it
            top = torch.randint(V, (B, P + 1, 3), device=dev, generator=g)
            z.scatter_(2, top, lse + torch.randn((B, P + 1, 3), device=dev, generator=g))
            dz = z[:, :P] + 0.6 * torch.randn((B, P, V), device=dev, generator=g)
            qprobs = torch.softmax(dz, -1)
            noise = torch.empty((B, P, V), device=dev).exponential_(generator=g)
            block = (qprobs / noise).argmax(-1).to(torch.int32)
        else:                      # lookup drafts: the target mostly agrees
            qprobs = None
            block = torch.randint(V, (B, P), device=dev, generator=g).to(torch.int32)
            z[:, :P].scatter_(2, block.long()[..., None],
                              lse + 1.5 + 1.5 * torch.randn((B, P, 1), device=dev, generator=g))
        banned = torch.randint(V, (B, 1, max(1, V // 64)), device=dev, generator=g).expand(B, P + 1, -1)
        z.scatter_(2, banned, -math.inf)
        store = torch.zeros((B, P + 1, V + case["pad"]), device=dev, dtype=dt)
        store[:, :, :V] = z
        length = torch.tensor(_block_lengths(case), device=dev, dtype=torch.int32)
        s |= dict(block=block, length=length, logits=store[:, :, :V], qprobs=qprobs, point=None, u=None,
                  temperature=None, noise=None)
        if mode != "greedy":
            s["u"] = torch.rand((B, P), device=dev, generator=g)
            s["noise"] = torch.empty((B, V), device=dev).exponential_(generator=g).clamp_(min=1e-30)
            t = 0.6 + 0.6 * torch.rand(B, device=dev, generator=g)
            t[7::8] = 0.0          # greedy requests in the same batch
            s["temperature"] = t
        if mode == "draft":        # the first positions of some blocks were filled by the lookup
            s["point"] = (torch.rand((B, P), device=dev, generator=g) < 0.25).to(torch.int32)
        return s
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    dt = TYPES[case["type"]]
    lens = _lengths(case)
    table, pages = _pool(case, [n + N for n in lens], g)
    s |= dict(table=table, kv_len=torch.tensor(lens, device=dev, dtype=torch.int32))
    shape = (pages, Hkv, case["page"], D)
    s["kc"] = torch.randn(shape, device=dev, dtype=dt, generator=g)
    s["vc"] = torch.randn(shape, device=dev, dtype=dt, generator=g)
    qn = [N if r % 3 != 1 else max(1, N - N // 3) for r in range(B)]
    s["q_len"] = torch.tensor(qn, device=dev, dtype=torch.int32)
    if case["op"] == "attention":
        s["q"] = (torch.randn((B, N, Hq, D), device=dev, generator=g) * 2).to(dt)
        return s
    # q, k and v as one projection writes them: heads side by side in a token's row
    qkv = torch.randn((B, N, Hq + 2 * Hkv, D), device=dev, dtype=dt, generator=g)
    s |= dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:])
    # cos and sin of every position, formed in 64 bits; positions stretched four times
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half) / 4.0
    ang = torch.arange(max(lens) + N, device=dev, dtype=torch.float64)[:, None] * freq
    s["rotary"] = torch.cat([ang.cos(), ang.sin()], 1).to(f32).contiguous()
    return s


def run(s):
    case = s["case"]
    if own:
        import prompt_lookup_speculative_gb300 as pld
        if case["op"] == "verify":
            return pld.lookup_verify_logits(s["block"], s["length"], s["logits"], noise=s["noise"], u=s["u"],
                                            temperature=s["temperature"], qprobs=s["qprobs"], point_mass=s["point"])
        if case["op"] == "kv_append":
            q, status = pld.lookup_kv_append(s["q"], s["k"], s["v"], s["kv_len"], s["table"], s["kc"], s["vc"],
                                             rotary=s["rotary"], q_len=s["q_len"], interleaved=case["inter"])
            return q, s["kc"], s["vc"], status
        return pld.lookup_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["kv_len"], q_len=s["q_len"],
                                          window=case["window"])
    return {"verify": _verify, "kv_append": _kv_append, "attention": _attention}[case["op"]](s)


# ------------------------------------------------------------- plain forms ----
def _first_max(key):
    """The lowest index of the largest value, along the last axis."""
    idx = torch.arange(key.shape[-1], device=key.device)
    return torch.where(key == key.amax(-1, keepdim=True), idx, key.shape[-1]).amin(-1)


def _verify(s):
    z = s["logits"].float()
    B, P1, V = z.shape
    P, dev, inf = P1 - 1, z.device, math.inf
    greedy = torch.ones(B, dtype=torch.bool, device=dev) if s["noise"] is None else ~(s["temperature"] > 0)
    inv = torch.ones(B, device=dev) if s["noise"] is None else torch.where(greedy, 1.0, 1.0 / s["temperature"])
    z = torch.where(torch.isnan(z), -inf, z)
    m = z.amax(-1, keepdim=True)
    w = torch.where(z == m, 1.0, torch.exp((z - m) * inv[:, None, None])) * (z > -inf)
    total = w.sum(-1, keepdim=True)
    p = w / total.clamp(min=1e-30)
    idx = s["block"].long()
    fits = (idx >= 0) & (idx < V)
    pd = torch.where(fits, p[:, :P].gather(2, idx.clamp(0, V - 1)[..., None])[..., 0], 0.0)
    best = torch.where(m[..., 0] > -inf, _first_max(z), -1)
    point = torch.ones((B, P), dtype=torch.bool, device=dev)
    if s["qprobs"] is not None:
        point = s["point"] != 0
    if s["noise"] is None:
        ok = idx == best[:, :P]
    else:
        qd = torch.ones((B, P), device=dev)
        if s["qprobs"] is not None:
            qd = torch.where(point, 1.0, s["qprobs"].gather(2, idx.clamp(0, V - 1)[..., None])[..., 0])
        ok = torch.where(greedy[:, None], idx == best[:, :P], s["u"] * qd < pd)
    pos = torch.arange(P1, device=dev)
    ok = torch.cat([ok & (pos[:P] < s["length"][:, None]), torch.zeros((B, 1), dtype=torch.bool, device=dev)], 1)
    a = torch.where(ok, P1, pos).amin(1)
    # the token at the first position not accepted (or past the block)
    row = a[:, None, None]
    pa = p.gather(1, row.expand(B, 1, V))[:, 0]
    token = best.gather(1, a[:, None])[:, 0]
    if s["noise"] is not None:
        left = a < s["length"]
        ca = a.clamp(max=max(P - 1, 0))
        if P:
            da, pt = idx.gather(1, ca[:, None]), point.gather(1, ca[:, None])
            qa = torch.zeros_like(pa)
            if s["qprobs"] is not None:
                qa = s["qprobs"].gather(1, ca[:, None, None].expand(B, 1, V))[:, 0]
            one = (torch.arange(V, device=dev) == da).float()
            qa = torch.where(pt, one, qa) * left[:, None]
            res = (pa - qa).clamp(min=0)
            res = torch.where((res > 0).any(-1, keepdim=True), res, pa)
        else:
            res = pa
        drawn = torch.where((res > 0).any(-1), _first_max(res / s["noise"]), -1)
        token = torch.where(greedy, token, drawn)
    accepted = a.to(torch.int32)
    ncommit = (a + (token >= 0)).to(torch.int32)
    full = torch.cat([idx, torch.zeros((B, 1), dtype=torch.long, device=dev)], 1)
    commit = torch.where(pos < a[:, None], full, torch.where(pos == a[:, None], token[:, None], -1))
    at = commit.clamp(0, V - 1)[..., None]
    lp = (z.gather(2, at) - m)[..., 0] * inv[:, None] - torch.log(total[..., 0])
    lp = torch.where(pos < ncommit[:, None], lp, 0.0)
    return accepted, commit.to(torch.int32), ncommit, lp


def _slots(s):
    """Positions [B, N], page and row in it of each new token."""
    page = s["case"]["page"]
    pos = s["kv_len"].long()[:, None] + torch.arange(s["q"].shape[1], device="cuda")
    at = s["table"].long().gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1))
    return pos, at, pos % page


def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, :, None], sin[:, :, None]
    if inter:
        a, b = part[..., 0::2], part[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, rest], -1)


def _kv_append(s):
    case, dt = s["case"], s["q"].dtype
    pos, at, row = _slots(s)
    tab = s["rotary"][pos.clamp(max=s["rotary"].shape[0] - 1)]
    half = case["rot"] // 2
    cos, sin = tab[..., :half], tab[..., half:]
    valid = torch.arange(case["N"], device="cuda") < s["q_len"][:, None]
    q = torch.where(valid[..., None, None], _rotate(s["q"], cos, sin, case["rot"], case["inter"]), 0.0).to(dt)
    k = _rotate(s["k"], cos, sin, case["rot"], case["inter"]).to(dt)
    for cache, new in ((s["kc"], k), (s["vc"], s["v"])):     # slots past q_len keep what they hold
        cache[at, :, row] = torch.where(valid[..., None, None], new, cache[at, :, row])
    return q, s["kc"], s["vc"], torch.zeros(case["B"], dtype=torch.int32, device="cuda")


def _attention(s):
    case, q = s["case"], s["q"]
    B, N, Hq, D = q.shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * case["page"]
    k = s["kc"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    v = s["vc"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    kv_len, q_len = s["kv_len"].long(), s["q_len"].long()
    j, i = torch.arange(L, device="cuda"), torch.arange(N, device="cuda")
    v = torch.where((j < (kv_len + q_len)[:, None])[:, None, :, None], v, 0.0)
    pos = kv_len[:, None] + i
    see = (j <= pos[..., None]) & (i < q_len[:, None])[..., None]
    if case["window"]:
        see &= j > pos[..., None] - case["window"]
    qh = q.float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    sc = torch.matmul(qh, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    sc = torch.where(see[:, None, :, None].expand(B, Hkv, N, G, L).reshape(B, Hkv, N * G, L), sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    w = torch.exp(sc - torch.where(m > -math.inf, m, 0.0))
    t = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v) / torch.where(t > 0, t, 1.0)
    lse = m + torch.log(t)
    back = lambda x: x.reshape(B, Hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, -1)  # noqa: E731
    return back(o).to(q.dtype).contiguous(), back(lse)[..., 0].contiguous()


# -------------------------------------------------------------------- work ----
def work(case):
    if case["op"] == "verify":
        B, V, size = case["B"], case["V"], 4 if case["type"] == "f32" else 2
        rows = sum(n + 1 for n in _block_lengths(case))        # every row with a proposal to test, and the bonus row
        sampled = case["mode"] != "greedy"
        byte = rows * V * size + (B * V * 4 if sampled else 0) + (B * V * 4 if case["mode"] == "draft" else 0)
        return {"bytes": byte + B * (case["P"] + 1) * 20, "flops": 4 * rows * V}
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    lens = _lengths(case)
    qn = [N if r % 3 != 1 else max(1, N - N // 3) for r in range(B)]
    if case["op"] == "kv_append":
        t = sum(qn)
        # read and written once each; a token's row of the table once; the padded rows of q are written
        return {"bytes": 2 * t * (Hq + 2 * Hkv) * D * 2 + (B * N - t) * Hq * D * 2 + t * case["rot"] * 4,
                "flops": 3 * t * (Hq + Hkv) * case["rot"]}
    keys = pairs = 0
    for n, c in zip(lens, qn):
        w = case["window"] or n + c
        keys += min(n + c, w + c - 1)
        pairs += sum(min(n + i + 1, w) for i in range(c))
    return {"bytes": 2 * keys * Hkv * D * 2 + (sum(qn) + B * N) * Hq * D * 2 + B * N * Hq * 4,
            "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------- exact ----
def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "kv_append": _exact_append, "attention": _exact_attention}[case["op"]](s)


def _exact_verify(s):
    """Request by request, as the definition reads."""
    B, P1, V = s["logits"].shape
    acc, commit, nc, lps = [], [], [], []
    lens = s["length"].tolist()
    temp = s["temperature"].double().tolist() if s["temperature"] is not None else [0.0] * B
    block = s["block"].tolist()
    point = s["point"].tolist() if s["point"] is not None else None
    u = s["u"].double().tolist() if s["u"] is not None else None
    for b in range(B):
        T = temp[b] if temp[b] > 0 else 1.0
        z = s["logits"][b, :lens[b] + 1].double().nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf) / T
        lp = torch.log_softmax(z, -1)
        row, out, a = [-1] * P1, [0.0] * P1, 0
        heads = z.argmax(-1).tolist()
        while a < lens[b]:
            d = block[b][a]
            if temp[b] > 0:
                is_point = s["qprobs"] is None or point[b][a] != 0
                q = 1.0 if is_point else float(s["qprobs"][b, a, d])
                take = u[b][a] * q < math.exp(float(lp[a, d]))
            else:
                take = heads[a] == d
            if not take:
                break
            row[a], out[a] = d, float(lp[a, d])
            a += 1
        if temp[b] > 0:
            left = lp[a].exp()
            if a < lens[b]:
                if s["qprobs"] is None or point[b][a] != 0:
                    left[block[b][a]] = 0.0
                else:
                    left = torch.relu(left - s["qprobs"][b, a].double())
                if not bool((left > 0).any()):
                    left = lp[a].exp()
            t = int((left / s["noise"][b].double()).argmax())
        else:
            t = heads[a]
        row[a], out[a] = t, float(lp[a, t])
        acc.append(a)
        commit.append(row)
        nc.append(a + 1)
        lps.append(out)
    i32 = dict(dtype=torch.int32, device="cuda")
    return (torch.tensor(acc, **i32), torch.tensor(commit, **i32), torch.tensor(nc, **i32),
            torch.tensor(lps, dtype=torch.float64, device="cuda"))


def _exact_append(s):
    """Pairs as complex numbers, each turned by its angle's unit."""
    case = s["case"]
    half, f64 = case["rot"] // 2, torch.float64
    q_len, kv_len = s["q_len"].tolist(), s["kv_len"].tolist()
    turned = {}
    for name in ("q", "k"):
        x = s[name].to(f64).clone()
        for b in range(case["B"]) if case["B"] <= 64 else [slice(None)]:
            start = torch.as_tensor(kv_len[b], device="cuda").reshape(-1, 1)
            at = (start + torch.arange(case["N"], device="cuda")).clamp(max=s["rotary"].shape[0] - 1)
            tab = s["rotary"][at].to(f64)
            unit = torch.complex(tab[..., :half], tab[..., half:])[:, :, None]
            part = x[b][..., :case["rot"]].reshape(-1, case["N"], x.shape[2], case["rot"])
            if case["inter"]:
                pair = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous())
                back = torch.view_as_real(pair * unit).flatten(-2)
            else:
                pair = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * unit
                back = torch.cat([pair.real, pair.imag], -1)
            x[b][..., :case["rot"]] = back if isinstance(b, slice) else back[0]
        turned[name] = x
    kc, vc = s["kc"].to(f64), s["vc"].to(f64)
    b = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), s["q_len"].long())
    first = torch.cumsum(s["q_len"].long(), 0) - s["q_len"].long()
    i = torch.arange(b.numel(), device="cuda") - first[b]
    pos = s["kv_len"].long()[b] + i
    page = s["table"].long()[b, torch.div(pos, case["page"], rounding_mode="floor")]
    kc[page, :, pos.remainder(case["page"])] = turned["k"][b, i]
    vc[page, :, pos.remainder(case["page"])] = s["v"].to(f64)[b, i]
    q = torch.zeros_like(turned["q"])
    q[b, i] = turned["q"][b, i]
    return q, kc, vc, torch.zeros(case["B"], dtype=torch.int32, device="cuda")


def _exact_attention(s):
    """One request at a time over its own positions; softmax through its logarithm."""
    case, q = s["case"], s["q"]
    B, N, Hq, D = q.shape
    if work(case)["flops"] > 6e12:
        return None
    G = Hq // case["Hkv"]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, c) in enumerate(zip(s["kv_len"].tolist(), s["q_len"].tolist())):
        pages = s["table"][b, :-(-(n + c) // case["page"])].long()
        k = s["kc"][pages].transpose(0, 1).flatten(1, 2)[:, :n + c].double()
        v = s["vc"][pages].transpose(0, 1).flatten(1, 2)[:, :n + c].double()
        gap = (n + torch.arange(c, device="cuda"))[:, None] - torch.arange(n + c, device="cuda")
        hide = gap < 0
        if case["window"]:
            hide |= gap >= case["window"]
        for h in range(case["Hkv"]):
            qs = q[b, :c, h * G:(h + 1) * G].double()
            sc = torch.einsum("igd,jd->gij", qs, k[h]) / math.sqrt(D)
            sc.masked_fill_(hide, -math.inf)
            one = torch.logsumexp(sc, -1)
            out[b, :c, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", (sc - one[..., None]).exp(), v[h])
            lse[b, :c, h * G:(h + 1) * G] = one.T
    return out, lse
