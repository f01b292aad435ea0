"""The target's operators (include/lookup_target.h) in 64 bits, element by element as the
header states them, with the bounds the kernels' roundings stay within.

Nothing here shares code with the package.  Inputs and outputs are CPU tensors.
"""
from __future__ import annotations

import math

import torch

# half a unit in the last place, relative: 8, 11 and 24 significant bits
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def slot(table, pos, page, pages):
    """(page, row) of cached position pos in a request's table row, or None."""
    at = pos // page
    if at >= len(table):
        return None
    pg = int(table[at])
    return (pg, pos % page) if 0 <= pg < pages else None


def kv_append(q, k, v, kv_len, q_len, table, kc, vc, rotary, interleaved):
    """Returns (out_q, kc, vc, status) in 64 bits and the bound of each rounded element
    (relative to the larger product of the pair)."""
    B, N, Hq, D = q.shape
    pages, _, page, _ = kc.shape
    out_q = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    kc, vc = kc.double().clone(), vc.double().clone()
    bq, bk = torch.zeros_like(out_q), torch.zeros_like(kc)
    status = torch.zeros(B, dtype=torch.int32)
    u = UNIT[q.dtype]

    def turn(x, pos):
        x = x.double()
        if rotary is None:
            return x, torch.zeros_like(x)
        half = rotary.shape[1] // 2
        out, size = x.clone(), torch.zeros_like(x)
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = float(rotary[pos, j]), float(rotary[pos, half + j])
            out[:, a], out[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
            size[:, a] = (x[:, a] * c).abs() + (x[:, b] * s).abs()
            size[:, b] = (x[:, b] * c).abs() + (x[:, a] * s).abs()
        # two products and a sum in float32, then one rounding to the type
        return out, out.abs() * u + size * 2.0 ** -22 + (size > 0) * TINY[q.dtype]

    for b in range(B):
        n = min(max(int(q_len[b]), 0), N)
        for i in range(n):
            pos = max(int(kv_len[b]), 0) + i
            sl = slot(table[b], pos, page, pages)
            if sl is None or (rotary is not None and pos >= rotary.shape[0]):
                status[b] = 1
                continue
            out_q[b, i], bq[b, i] = turn(q[b, i], pos)
            kc[sl[0], :, sl[1]], bk[sl[0], :, sl[1]] = turn(k[b, i], pos)
            vc[sl[0], :, sl[1]] = v[b, i].double()
    return out_q, kc, vc, status, bq, bk


def attention(q, kc, vc, table, kv_len, q_len, scale, window):
    """Returns (out, lse, bound of out, bound of lse) in 64 bits."""
    B, N, Hq, D = q.shape
    pages, Hkv, page, _ = kc.shape
    G, u = Hq // Hkv, UNIT[q.dtype]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    bout, blse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = min(max(int(q_len[b]), 0), N)
        kv = max(int(kv_len[b]), 0)
        end = min(kv + n, len(table[b]) * page)
        if end <= 0 or n == 0:
            continue
        k = torch.zeros((end, Hkv, D), dtype=torch.float64)
        v = torch.zeros((end, Hkv, D), dtype=torch.float64)
        for at in range(-(-end // page)):
            pg = int(table[b][at])
            if 0 <= pg < pages:
                m = min(page, end - at * page)
                k[at * page:at * page + m] = kc[pg, :, :m].double().transpose(0, 1)
                v[at * page:at * page + m] = vc[pg, :, :m].double().transpose(0, 1)
        for i in range(n):
            pos = kv + i
            lo, hi = (max(0, pos - window + 1) if window else 0), min(pos + 1, end)
            if hi <= lo:
                continue
            kk, vv = k[lo:hi].repeat_interleave(G, 1), v[lo:hi].repeat_interleave(G, 1)     # [S, Hq, D]
            qq = q[b, i].double()
            s = (qq[None] * kk).sum(-1) * scale
            one = torch.logsumexp(s, 0)
            p = (s - one).exp()
            o = (p[..., None] * vv).sum(0)
            out[b, i], lse[b, i] = o, one
            # a score: D products summed in float32 and scaled; its error moves p and lse by as much.
            # p relative to the running maximum: the exponent's argument rounds, relative 2^-23 of its size
            ds = ((qq[None] * kk).abs().sum(-1) * abs(scale) * (D + 4) * 2.0 ** -24).amax(0)
            ds = ds + (s.amax(0) - s.amin(0)).clamp(max=100.0) * 2.0 ** -23 + 2.0 ** -20
            # p rounded to the type for the product (u), then the result (u); sums in float32
            mass = (p[..., None] * vv.abs()).sum(0)
            bout[b, i] = mass * (1.02 * u + 2 * ds[:, None] + (hi - lo + 64) * 2.0 ** -24) + o.abs() * u + TINY[q.dtype] \
                + (2.0 ** -24 * vv.abs().sum(0) if q.dtype == torch.float16 else 0.0)   # p below f16's normal range
            blse[b, i] = 2 * ds + one.abs() * 2.0 ** -22 + (hi - lo + 64) * 2.0 ** -24
    return out, lse, bout, blse


def verify(block, length, logits, noise, u, temperature, qprobs, point_mass):
    """Returns (accepted, commit, ncommit, logprobs, bound of logprobs, sure): `sure`
    marks requests none of whose decisions is nearer to a tie than float32 can tell."""
    B, P = block.shape
    V = logits.shape[2]
    acc, nc = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    commit = torch.full((B, P + 1), -1, dtype=torch.int32)
    lps, bound = torch.zeros((B, P + 1), dtype=torch.float64), torch.zeros((B, P + 1), dtype=torch.float64)
    sure = torch.ones(B, dtype=torch.bool)
    # relative error of a probability: each weight's exponent and the sum of V of them
    near = 2.0 ** -18 + (V / 256 + 32) * 2.0 ** -24
    for b in range(B):
        n = int(length[b])
        if n < 0 or n > P:
            acc[b] = -1
            continue
        T = 0.0
        if noise is not None:
            T = 1.0 if temperature is None else float(temperature[b])
            if not (T > 0 and T <= 3.4028234663852886e38):
                T = 0.0
        inv = 1.0 / T if T else 1.0

        def row_of(i):
            x = logits[b, i].double()
            x = torch.where(torch.isnan(x), -math.inf, x)
            m = x.max()
            if m == -math.inf:
                return x, m, None
            w = torch.where(x == m, torch.ones_like(x), ((x - m) * inv).exp())
            w = torch.where(x == -math.inf, torch.zeros_like(w), w)
            return x, m, w

        def logprob(x, m, w, t):
            z = 0.0 if x[t] == m else float((x[t] - m) * inv)
            return z - math.log(float(w.sum())), near + abs(z) * 2.0 ** -22

        a = n
        for i in range(n):
            x, m, w = row_of(i)
            d = int(block[b, i])
            fits = 0 <= d < V and w is not None
            if T == 0.0:
                ok = fits and d == int((x == m).nonzero()[0])
            else:
                pd = float(w[d] / w.sum()) if fits else 0.0
                point = qprobs is None or (point_mass is not None and int(point_mass[b, i]) != 0)
                t = float(u[b, i]) * (1.0 if point or not fits else float(qprobs[b, i, d]))
                ok = t < pd
                if abs(t - pd) <= 4 * near * max(pd, 1e-30) + 1e-38 and fits and w is not None:
                    sure[b] = False
            if not ok:
                a = i
                break
            commit[b, i] = d
            lps[b, i], bound[b, i] = logprob(x, m, w, d)
        x, m, w = row_of(a)
        tok = -1
        if w is not None:
            if T == 0.0:
                tok = int((x == m).nonzero()[0])
            else:
                p = w / w.sum()
                left, q = p.clone(), None
                if a < n:
                    if qprobs is None or (point_mass is not None and int(point_mass[b, a]) != 0):
                        if 0 <= int(block[b, a]) < V:
                            left[int(block[b, a])] = 0.0
                    else:
                        q = qprobs[b, a].double()
                        left = (p - q).clamp(min=0)
                if not bool((left > 0).any()):
                    left = p
                key = left / noise[b].double()
                best = key.max()
                tok = int((key == best).nonzero()[0])
                # p - q rounds by p's error over what is left
                slack = (p * near + (q * 2.0 ** -23 if q is not None else 0.0)) / noise[b].double()
                rivals = key + slack >= best - slack[tok]
                rivals[tok] = False
                if bool(rivals.any()):
                    sure[b] = False
        acc[b] = a
        if tok >= 0:
            commit[b, a] = tok
            lps[b, a], bound[b, a] = logprob(x, m, w, tok)
        nc[b] = a + (tok >= 0)
    return acc, commit, nc, lps, bound, sure
