"""The target's operators (include/lookup_target.h) against their definition in 64 bits.

Every bound is derived in target_reference.py from the roundings the header allows:
one rounding to the type of each probability and of each result, float32 sums.
Whole numbers are compared exactly, for every request whose decisions are further
from a tie than float32's rounding.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("prompt_lookup_speculative_gb300")

import target_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def tables(tokens, page, g, spare=0, pad=1):
    """A shuffled page table with room for tokens[r] tokens, -1 past the last page."""
    need = [-(-t // page) for t in tokens]
    total = max(1, sum(need) + spare)
    perm = torch.randperm(total, generator=g).tolist()
    width = max(1, max(need, default=1)) + pad
    out = torch.full((len(tokens), width), -1, dtype=torch.int32)
    for r, n in enumerate(need):
        for j in range(n):
            out[r, j] = perm.pop()
    return out, total


def close(got, want, bound, what):
    got = got.double().cpu()
    same = (got == want) | ((got - want).abs() <= bound)
    assert bool(same.all()), (what, float(((got - want).abs() / (bound + 1e-300))[~same].max()),
                              (~same).nonzero()[:4].tolist())


# ------------------------------------------------------------------ append ----
def append_case(B, N, Hq, Hkv, D, rot, inter, page, lens, qn, dt, seed, fused=True, max_pos=None, with_rotary=True):
    g = gen(seed)
    table, pages = tables([n + N for n in lens], page, g, spare=2)
    heads = Hq + 2 * Hkv
    pad = 0 if fused is True else fused           # elements between tokens' rows
    qkv = torch.randn((B, N, heads * D + pad), generator=g).to(dt)[..., :heads * D].unflatten(2, (heads, D))
    kc = torch.randn((pages, Hkv, page, D), generator=g).to(dt)
    vc = torch.randn((pages, Hkv, page, D), generator=g).to(dt)
    rotary = pkg.rotary_table(max_pos or (max(lens) + N + 1), rot, device="cpu") if with_rotary else None
    kv = torch.tensor(lens, dtype=torch.int32)
    ql = torch.tensor(qn, dtype=torch.int32)
    return qkv, table, kc, vc, rotary, kv, ql


def strided_cuda(x):
    """The tensor on the GPU with the strides it has here."""
    out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    out.copy_(x)
    return out


def run_append(qkv, Hq, Hkv, table, kc, vc, rotary, kv, ql, inter):
    d = strided_cuda(qkv)
    kcd, vcd = kc.cuda(), vc.cuda()
    q, st = pkg.lookup_kv_append(d[:, :, :Hq], d[:, :, Hq:Hq + Hkv], d[:, :, Hq + Hkv:], kv.cuda(), table.cuda(), kcd,
                                 vcd, rotary=None if rotary is None else rotary.cuda(), q_len=ql.cuda(),
                                 interleaved=inter)
    torch.cuda.synchronize()
    return q, kcd, vcd, st


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot,inter,page,fused", [
    (1, 1, 4, 1, 128, 128, False, 16, True),
    (3, 5, 6, 2, 64, 64, True, 8, True),
    (2, 16, 8, 8, 128, 64, False, 32, True),
    (5, 3, 7, 1, 256, 128, True, 64, True),
    (2, 4, 3, 3, 80, 32, False, 16, True),
    (2, 4, 2, 1, 36, 12, False, 1, True),
    (2, 4, 2, 1, 35, 34, True, 4, True),
    (2, 3, 2, 1, 96, 72, False, 16, 1),
    (3, 7, 4, 2, 128, 128, False, 16, 3),
    (1, 70, 2, 2, 64, 16, True, 128, 8),
])
def test_append_matches_definition(dt, B, N, Hq, Hkv, D, rot, inter, page, fused):
    lens = [(37 * r + 3) % 70 if r else 0 for r in range(B)]
    qn = [(N + r) % (N + 1) if r else N for r in range(B)]
    qkv, table, kc, vc, rotary, kv, ql = append_case(B, N, Hq, Hkv, D, rot, inter, page, lens, qn, dt, B * N + D, fused)
    q, kcd, vcd, st = run_append(qkv, Hq, Hkv, table, kc, vc, rotary, kv, ql, inter)
    oq, okc, ovc, ost, bq, bk = ref.kv_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], kv, ql,
                                              table, kc, vc, rotary, inter)
    close(q, oq, bq, "q")
    close(kcd, okc, bk, "k cache")
    assert torch.equal(vcd.double().cpu(), ovc)
    assert torch.equal(st.cpu(), ost)


def test_append_without_rotation_copies():
    qkv, table, kc, vc, _, kv, ql = append_case(3, 4, 4, 2, 64, 64, False, 16, [0, 9, 15], [4, 4, 2], BF16, 5,
                                                with_rotary=False)
    q, kcd, vcd, st = run_append(qkv, 4, 2, table, kc, vc, None, kv, ql, False)
    oq, okc, ovc, ost, _, _ = ref.kv_append(qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], kv, ql, table, kc, vc, None,
                                            False)
    assert torch.equal(q.double().cpu(), oq) and torch.equal(kcd.double().cpu(), okc)
    assert torch.equal(vcd.double().cpu(), ovc) and int(st.sum()) == 0


@pytest.mark.parametrize("D,rot", [(128, 128), (36, 12)])
def test_append_reports_tokens_without_a_slot(D, rot):
    """Past the table, past the rotary table, or a table entry outside the pool: status
    1, nothing cached for that token, a row of zeros; counts out of range are clamped."""
    B, N, page = 7, 6, 8
    lens = [0, 12, 20, 3, 1, -5, 2]
    qn = [6, 6, 6, 6, 9, 6, -2]
    qkv, table, kc, vc, rotary, kv, ql = append_case(B, N, 2, 1, D, rot, False, page, [30] * B, qn, F16, 11, max_pos=16)
    kv = torch.tensor(lens, dtype=torch.int32)
    table = table[:, :3].contiguous()
    table[3, 1] = kc.shape[0]              # one past the pool
    table[4, 0] = -7
    q, kcd, vcd, st = run_append(qkv, 2, 1, table, kc, vc, rotary, kv, ql, False)
    oq, okc, ovc, ost, bq, bk = ref.kv_append(qkv[:, :, :2], qkv[:, :, 2:3], qkv[:, :, 3:], kv, ql, table, kc, vc,
                                              rotary, False)
    close(q, oq, bq, "q")
    close(kcd, okc, bk, "k cache")
    assert torch.equal(vcd.double().cpu(), ovc)
    assert torch.equal(st.cpu(), ost) and st.cpu().tolist() == [0, 1, 1, 1, 1, 0, 0]


def test_append_keeps_nonfinite_values_where_they_are():
    qkv, table, kc, vc, rotary, kv, ql = append_case(1, 3, 2, 1, 64, 64, False, 16, [5], [3], BF16, 2)
    qkv[0, 0, 2, 1] = math.inf             # in k: its pair only
    qkv[0, 1, 3, 7] = math.nan             # in v
    q, kcd, vcd, _ = run_append(qkv, 2, 1, table, kc, vc, rotary, kv, ql, False)
    row = kcd[int(table[0, 0]), 0, 5].cpu()
    assert sorted((~row.isfinite()).nonzero()[:, 0].tolist()) == [1, 33]
    assert sorted((~vcd[int(table[0, 0]), 0, 6].cpu().isfinite()).nonzero()[:, 0].tolist()) == [7]
    assert bool(q.isfinite().all())


# --------------------------------------------------------------- attention ----
def attention_case(lens, qn, N, Hq, Hkv, D, page, dt, seed, spread=2.0, junk=math.nan):
    """Pages whose unseen slots hold `junk`."""
    g = gen(seed)
    B = len(lens)
    table, pages = tables([n + c for n, c in zip(lens, qn)], page, g, spare=1)
    kc = torch.full((pages, Hkv, page, D), junk, dtype=dt)
    vc = torch.full((pages, Hkv, page, D), junk, dtype=dt)
    for r in range(B):
        for j in range(lens[r] + qn[r]):
            pg = int(table[r, j // page])
            kc[pg, :, j % page] = torch.randn((Hkv, D), generator=g).to(dt)
            vc[pg, :, j % page] = torch.randn((Hkv, D), generator=g).to(dt)
    q = (torch.randn((B, N, Hq, D), generator=g) * spread).to(dt)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), torch.tensor(qn, dtype=torch.int32)


def check_attention(q, kc, vc, table, kv, ql, scale=None, window=0, **kw):
    D = q.shape[3]
    out, lse = pkg.lookup_paged_attention(strided_cuda(q), kc.cuda(), vc.cuda(), table.cuda(), kv.cuda(),
                                          q_len=ql.cuda(), scale=scale, window=window, **kw)
    torch.cuda.synchronize()
    o, l, bo, bl = ref.attention(q, kc, vc, table, kv, ql, D ** -0.5 if scale is None else scale, window)
    close(out, o, bo, "out")
    close(lse, l, bl, "lse")
    return out, lse


LENS = [0, 1, 7, 16, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hkv,page", [(1, 4, 4, 16), (1, 8, 1, 64), (3, 5, 1, 8), (16, 8, 1, 32), (5, 14, 2, 128)])
def test_attention_over_lengths(dt, D, N, Hq, Hkv, page):
    """Lengths about every page and tile edge, every block length from none to N."""
    qn = [(r + 1) % (N + 1) if r else N for r in range(len(LENS))]
    check_attention(*attention_case(LENS, qn, N, Hq, Hkv, D, page, dt, D + N + page))


@pytest.mark.parametrize("window", [1, 5, 64, 127, 128, 130])
@pytest.mark.parametrize("N,D,page", [(1, 64, 16), (9, 128, 8)])
def test_attention_window(window, N, D, page):
    lens = [0, 3, 64, 127, 128, 260, 300]
    check_attention(*attention_case(lens, [N] * 7, N, 6, 2, D, page, BF16, window), window=window)


@pytest.mark.parametrize("N,Hq,Hkv", [(65, 8, 1), (33, 4, 1), (130, 1, 1), (17, 64, 2)])
def test_attention_of_more_rows_than_a_tile(N, Hq, Hkv):
    check_attention(*attention_case([40, 0, 129], [N, N, N // 2], N, Hq, Hkv, 64, 32, F16, N))


@pytest.mark.parametrize("page,D", [(16, 128), (1024, 64)])
def test_attention_long_context_split(page, D):
    """One request of 9001 tokens: the length is split and joined."""
    check_attention(*attention_case([9000], [1], 1, 4, 1, D, page, BF16, 3))
    check_attention(*attention_case([5000, 17], [4, 4], 4, 4, 2, D, page, F16, 4))


def filled_case(lens, qn, N, Hq, Hkv, D, page, dt, seed, spread=2.0):
    """As attention_case, drawn as a whole: only slots past a request's end hold NaN."""
    g = gen(seed)
    table, pages = tables([n + c for n, c in zip(lens, qn)], page, g, spare=1)
    kc, vc = (torch.randn((pages, Hkv, page, D), generator=g).to(dt) for _ in range(2))
    for r, (n, c) in enumerate(zip(lens, qn)):
        if (n + c) % page:
            last = int(table[r, (n + c) // page])
            kc[last, :, (n + c) % page:] = math.nan
            vc[last, :, (n + c) % page:] = math.nan
    q = (torch.randn((len(lens), N, Hq, D), generator=g) * spread).to(dt)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), torch.tensor(qn, dtype=torch.int32)


@pytest.mark.parametrize("D,N,Hq,Hkv,page,window", [
    (64, 1, 8, 4, 16, 0), (64, 9, 16, 4, 32, 0), (64, 12, 32, 4, 64, 0), (64, 9, 16, 4, 128, 700), (64, 17, 32, 4, 64, 0),
    (128, 1, 8, 4, 16, 0), (128, 9, 16, 4, 32, 0), (128, 12, 32, 4, 64, 300), (256, 5, 8, 4, 64, 0), (256, 12, 32, 4, 16, 0)])
def test_attention_of_many_tiles_per_range(D, N, Hq, Hkv, page, window):
    """Enough work that every range holds several tiles, begins and ends of items; blocks
    from one token to N, so that some warps of a tile have no rows."""
    lens = [1500 + (r * 977) % 1700 for r in range(14)] + [3, 127]
    qn = [1 + (r * 5) % N for r in range(16)]
    check_attention(*filled_case(lens, qn, N, Hq, Hkv, D, page, BF16, D + N), window=window)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 0.11])
@pytest.mark.parametrize("D,N,Hq,Hkv,page,window", [
    (64, 2, 7, 1, 16, 3), (64, 7, 14, 2, 32, 700), (128, 2, 16, 2, 8, 5), (128, 6, 16, 2, 64, 1100), (256, 3, 8, 2, 16, 40),
    (256, 16, 16, 2, 128, 900)])
def test_attention_of_cut_items_under_a_window(D, N, Hq, Hkv, page, window, scale):
    """Items cut between ranges where some of a row's parts hold nothing that it sees,
    for one, two and four copies of the block's rows, and scales of either sign."""
    lens = [2900, 2047, 1, 0, 1025, 64, 800, 2500]
    qn = [N, 1, N, 0, (N + 1) // 2, N, 1, N]
    check_attention(*filled_case(lens, qn, N, Hq, Hkv, D, page, F16, D + N + window), scale=scale, window=window)


def test_attention_many_requests_of_mixed_length():
    g = gen(9)
    lens = torch.randint(0, 90, (700,), generator=g).tolist()
    check_attention(*attention_case(lens, [1] * 700, 1, 2, 1, 64, 16, BF16, 9))


def test_attention_large_scores_and_scale():
    """Scores of hundreds: one position takes all the weight; a negative scale, a zero one."""
    case = attention_case([300, 31], [4, 4], 4, 4, 2, 128, 16, BF16, 21, spread=60.0)
    check_attention(*case)
    check_attention(*case, scale=-0.01)
    check_attention(*case, scale=0.0)


def test_attention_strided_queries():
    q, kc, vc, table, kv, ql = attention_case([33, 150], [3, 2], 3, 4, 2, 128, 16, BF16, 6)
    wide = torch.zeros((2, 5, 9, 128), dtype=BF16)
    view = wide[:, 1:4, 2:6]
    view.copy_(q)
    check_attention(view, kc, vc, table, kv, ql)


def test_attention_absent_pages_and_short_tables():
    """A table entry outside the pool reads as zeros; tokens past the table's end are absent."""
    q, kc, vc, table, kv, ql = attention_case([40, 200, 90], [3, 3, 3], 3, 4, 2, 64, 16, F16, 8)
    table[0, 1] = kc.shape[0] + 5
    table[1, 4] = -1
    table = table[:, :10].contiguous()                # request 1 needs 13 pages
    check_attention(q, kc, vc, table, kv, ql)


def test_attention_counts_out_of_range_are_clamped():
    q, kc, vc, table, kv, ql = attention_case([20, 20, 20], [4, 4, 4], 4, 2, 2, 64, 16, BF16, 12, junk=0.5)
    kv = torch.tensor([20, -9, 20], dtype=torch.int32)
    ql = torch.tensor([4, 4, 77], dtype=torch.int32)
    check_attention(q, kc, vc, table, kv, ql)
    ql = torch.tensor([-4, 4, 0], dtype=torch.int32)
    out, lse = check_attention(q, kc, vc, table, kv, ql)
    assert bool((out[0] == 0).all()) and bool((lse[2] == -math.inf).all())


def test_attention_without_q_len_and_with_outputs():
    q, kc, vc, table, kv, ql = attention_case([20, 100], [4, 4], 4, 4, 2, 128, 16, BF16, 13)
    want, wlse = check_attention(q, kc, vc, table, kv, ql)
    out, lse = torch.full_like(q, 7.0).cuda(), torch.full((2, 4, 4), 7.0, device="cuda")
    ws = torch.full((pkg.load_library().lookup_paged_attention_workspace_bytes(2, 4, 4, 2, 128),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    pkg.lookup_paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), kv.cuda(), out=out, lse=lse, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse, wlse)       # same bits: no order is left to chance


def test_attention_infinite_value_reaches_its_rows():
    """An infinite value that every row of the block sees is in every row's output."""
    q, kc, vc, table, kv, ql = attention_case([50], [2], 2, 2, 1, 64, 16, BF16, 14, junk=0.0)
    vc[int(table[0, 0]), 0, 3, 9] = math.inf
    out, _ = pkg.lookup_paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), kv.cuda(), q_len=ql.cuda())
    assert bool((out[..., 9] == math.inf).all())
    assert bool(out[..., :9].isfinite().all()) and bool(out[..., 10:].isfinite().all())


def test_attention_waits_that_run_out_give_nan():
    """A wait limit of a nanosecond: the call ends, every row says so, and the next call is
    right again."""
    case = attention_case([300, 31, 5000], [4, 3, 4], 4, 4, 2, 128, 16, BF16, 22)
    q, kc, vc, table, kv, ql = (x.cuda() for x in case)
    pkg.set_wait_limit_ns(1)
    try:
        out, lse = pkg.lookup_paged_attention(q, kc, vc, table, kv, q_len=ql)
        torch.cuda.synchronize()
    finally:
        pkg.set_wait_limit_ns(0)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    check_attention(*case)


# ------------------------------------------------------------------ verify ----
def verify_case(B, P, V, dt, mode, seed, pad=0, temps=None):
    g = gen(seed)
    z = torch.randn((B, P + 1, V), generator=g) * 2.0
    block = torch.randint(V, (B, P), generator=g).to(torch.int32)
    qprobs = point = None
    if mode == "draft":
        dz = z[:, :P] + 0.5 * torch.randn((B, P, V), generator=g)
        qprobs = torch.softmax(dz, -1)
        block = (qprobs / torch.empty((B, P, V)).exponential_(generator=g)).argmax(-1).to(torch.int32) if P else block
        point = (torch.rand((B, P), generator=g) < 0.3).to(torch.int32)
    else:
        z[:, :P].scatter_(2, block.long()[..., None], math.log(V) + 4.0 + torch.randn((B, P, 1), generator=g))
    store = torch.full((B, P + 1, V + pad), 99.0, dtype=dt)
    store[..., :V] = z
    logits = store[..., :V]
    length = torch.tensor([(P - r) % (P + 1) if r else P for r in range(B)], dtype=torch.int32)
    noise = u = temp = None
    if mode != "greedy":
        noise = torch.empty((B, V)).exponential_(generator=g).clamp_(min=1e-30)
        u = torch.rand((B, P), generator=g)
        temp = torch.tensor([(temps or [0.7, 1.0, 0.0, 1.3])[r % len(temps or [0] * 4)] for r in range(B)])
    return dict(block=block, length=length, logits=logits, noise=noise, u=u, temperature=temp, qprobs=qprobs,
                point_mass=point)


def check_verify(c, least=0.9, **kw):
    d = {k: None if v is None else strided_cuda(v) for k, v in c.items()}
    got = pkg.lookup_verify_logits(d["block"], d["length"], d["logits"], noise=d["noise"], u=d["u"],
                                   temperature=d["temperature"], qprobs=d["qprobs"], point_mass=d["point_mass"], **kw)
    torch.cuda.synchronize()
    acc, commit, nc, lps = (t.cpu() for t in got)
    wa, wc, wn, wl, bl, sure = ref.verify(c["block"], c["length"], c["logits"], c["noise"], c["u"], c["temperature"],
                                          c["qprobs"], c["point_mass"])
    assert float(sure.float().mean()) >= least            # the comparison covers nearly every request
    assert torch.equal(acc[sure], wa[sure])
    assert torch.equal(commit[sure], wc[sure])
    assert torch.equal(nc[sure], wn[sure])
    close(lps[sure], wl[sure], bl[sure], "logprobs")
    return acc, commit, nc, lps


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("mode", ["greedy", "point", "draft"])
@pytest.mark.parametrize("B,P,V,pad", [(1, 0, 1, 0), (1, 1, 2, 0), (5, 3, 37, 0), (9, 15, 1000, 1), (4, 7, 4099, 5),
                                       (2, 5, 32000, 8), (33, 2, 130, 0), (2, 33, 515, 3)])
def test_verify_matches_definition(dt, mode, B, P, V, pad):
    check_verify(verify_case(B, P, V, dt, mode, B * 31 + P + V, pad), least=0.5 if B < 3 else 0.9)


@pytest.mark.parametrize("mode", ["point", "draft"])
def test_verify_large_vocabulary(mode):
    acc, _, _, _ = check_verify(verify_case(6, 7, 151936, BF16, mode, 77), least=0.6)
    assert len(set(acc.tolist())) > 1


def test_verify_ties_take_the_lowest_index():
    c = verify_case(3, 2, 300, BF16, "greedy", 1)
    c["logits"][:] = 1.0
    c["logits"][1, 1, 40] = 2.0
    c["logits"][1, 1, 299] = 2.0
    c["block"] = torch.tensor([[0, 0], [0, 40], [1, 0]], dtype=torch.int32)
    c["length"] = torch.tensor([2, 2, 2], dtype=torch.int32)
    acc, commit, nc, _ = check_verify(c)
    assert acc.tolist() == [2, 2, 0] and commit[0].tolist() == [0, 0, 0] and commit[1].tolist() == [0, 40, 0]


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_verify_masked_and_infinite_logits(dt):
    """-infinity, NaN, the type's lowest value, +infinity, and rows with nothing left."""
    V = 700
    c = verify_case(8, 2, V, dt, "point", 3, temps=[0.8])
    z = c["logits"]
    c["length"] = torch.full((8,), 2, dtype=torch.int32)
    c["u"][:] = 0.0
    z[0] = -math.inf                                     # nothing at all
    z[1, 0] = torch.finfo(dt).min                        # the lowest value everywhere: uniform
    z[2, 0] = -math.inf
    z[2, 0, 5] = torch.finfo(dt).min                     # one token left, the lowest value
    c["block"][2, 0] = 5
    z[3, 1] = math.nan                                   # the second row holds nothing
    z[4, 0, [3, 600]] = math.inf                         # two share the row
    c["block"][4, 0] = 600
    z[5, :, ::2] = -math.inf
    z[5, :, 1::4] = math.nan
    z[6, 2, :] = torch.finfo(dt).min
    z[6, 2, 17] = torch.finfo(dt).max
    z[7, 0, :] = -math.inf
    z[7, 0, V - 1] = 0.0
    c["block"][7, 0] = V - 1
    acc, commit, nc, lps = check_verify(c, least=0.6)
    assert nc.tolist()[0] == 0 and commit[0].tolist() == [-1, -1, -1] and acc.tolist()[0] == 0
    assert acc.tolist()[3] == 1 and nc.tolist()[3] == 1 and commit[3].tolist()[1:] == [-1, -1]
    assert bool(lps.isfinite().all())
    c["noise"] = c["u"] = c["temperature"] = None        # the same rows, greedy
    _, commit, nc, _ = check_verify(c, least=0.99)
    assert nc.tolist()[0] == 0 and nc.tolist()[3] <= 1


def test_verify_error_rows_and_unusable_proposals():
    c = verify_case(6, 4, 90, F32, "point", 4)
    c["length"] = torch.tensor([4, -1, 5, 0, 4, 4], dtype=torch.int32)
    c["block"][0, 1] = -1
    c["block"][4, 0] = 90
    c["block"][5, 2] = -(1 << 31)
    c["u"][:] = 0.0
    acc, commit, nc, lps = check_verify(c, least=0.5)
    assert acc.tolist()[1:4] == [-1, -1, 0] and nc.tolist()[1:4] == [0, 0, 1]
    assert bool((commit[1:3] == -1).all()) and bool((lps[1:3] == 0).all())


def test_verify_residual_of_nothing_draws_from_p():
    """q = p exactly, a proposal refused all the same: the token is drawn from p."""
    c = verify_case(4, 1, 8, F32, "draft", 6, temps=[1.0])
    c["logits"][:] = 0.0
    c["qprobs"][:] = 0.125
    c["point_mass"][:] = 0
    c["length"] = torch.ones(4, dtype=torch.int32)
    c["block"][:] = -1                                   # no token: p = 0, refused
    acc, commit, nc, _ = check_verify(c, least=0.0)
    assert acc.tolist() == [0] * 4
    assert commit[:, 0].tolist() == c["noise"].argmin(1).tolist()


def test_verify_temperatures_that_mean_greedy():
    c = verify_case(6, 3, 500, F32, "point", 8, temps=[0.0, -1.0, math.nan, math.inf, 1e-3, 50.0])
    check_verify(c, least=0.6)


def test_verify_frequencies_follow_the_target():
    """40,000 draws of one position: the committed token is distributed as p whatever was
    proposed (chi-square over 8 tokens, 7 degrees of freedom: 35 has probability 1e-5)."""
    B, V = 40000, 8
    g = gen(10)
    z = torch.randn((1, 2, V), generator=g).expand(B, 2, V).contiguous()
    q = torch.softmax(torch.randn((1, 1, V), generator=g), -1).expand(B, 1, V).contiguous()
    block = (q[:, 0] / torch.empty((B, V)).exponential_(generator=g)).argmax(-1, keepdim=True).to(torch.int32)
    noise, u = torch.empty((B, V)).exponential_(generator=g), torch.rand((B, 1), generator=g)
    p = torch.softmax(z[0, 0].double(), -1)
    for qprobs in (q.cuda(), None):      # a point mass may be any token, whatever it was drawn from
        _, commit, _, _ = pkg.lookup_verify_logits(block.cuda(), torch.ones(B, dtype=torch.int32).cuda(), z.cuda(),
                                                   noise=noise.cuda(), u=u.cuda(), qprobs=qprobs)
        seen = torch.bincount(commit[:, 0].cpu().long(), minlength=V).double()
        chi = float(((seen - B * p) ** 2 / (B * p)).sum())
        assert chi < 35, (chi, seen.tolist(), (B * p).tolist())


def test_verify_waits_that_run_out_give_error_rows():
    """A wait limit of a nanosecond: every request reports it, and the next call is right."""
    c = verify_case(5, 3, 32000, BF16, "point", 12)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    pkg.set_wait_limit_ns(1)
    try:
        acc, commit, nc, lps = pkg.lookup_verify_logits(d["block"], d["length"], d["logits"], noise=d["noise"], u=d["u"],
                                                        temperature=d["temperature"])
        torch.cuda.synchronize()
    finally:
        pkg.set_wait_limit_ns(0)
    assert acc.tolist() == [-1] * 5 and nc.tolist() == [0] * 5
    assert bool((commit == -1).all()) and bool((lps == 0).all())
    check_verify(c, least=0.6)


# ------------------------------------------------- streams, graphs, launches ----
def test_calls_on_another_stream_and_in_a_graph():
    a = attention_case([40, 150], [4, 4], 4, 4, 2, 128, 16, BF16, 31)
    q, kc, vc, table, kv, ql = (x.cuda() for x in a)
    want, wlse = pkg.lookup_paged_attention(q, kc, vc, table, kv, q_len=ql)
    c = {k: None if v is None else v.cuda() for k, v in verify_case(4, 7, 3001, BF16, "point", 5).items()}
    vw = pkg.lookup_verify_logits(c["block"], c["length"], c["logits"], noise=c["noise"], u=c["u"],
                                  temperature=c["temperature"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = pkg.lookup_paged_attention(q, kc, vc, table, kv, q_len=ql, stream=side)
    vo = pkg.lookup_verify_logits(c["block"], c["length"], c["logits"], noise=c["noise"], u=c["u"],
                                  temperature=c["temperature"], stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert all(torch.equal(x, y) for x, y in zip(vo, vw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = pkg.lookup_paged_attention(q, kc, vc, table, kv, q_len=ql)
        vo = pkg.lookup_verify_logits(c["block"], c["length"], c["logits"], noise=c["noise"], u=c["u"],
                                      temperature=c["temperature"])
    for _ in range(2):
        out.zero_()
        vo[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(torch.equal(x, y) for x, y in zip(vo, vw))


def test_cache_class_and_empty_calls():
    cache = pkg.PagedKVCache(4, 16, 2, 64, dtype=BF16)
    q = torch.randn((1, 3, 4, 64), device="cuda").to(BF16)
    k, v = q[:, :, :2], q[:, :, 2:]
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    kv = torch.zeros(1, dtype=torch.int32, device="cuda")
    rot = pkg.rotary_table(64, 64)
    rq, st = cache.append(q, k, v, kv, table, rotary=rot)
    out, lse = cache.attention(rq, table, kv)
    # the first token sees itself only: its output is its value
    assert torch.equal(out[0, 0], v[0, 0].repeat_interleave(2, 0)) and int(st) == 0
    empty = torch.empty((0, 3, 4, 64), device="cuda", dtype=BF16)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = cache.attention(empty, table[:0], none)
    assert out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4)
    got = pkg.lookup_verify_logits(torch.empty((0, 3), dtype=torch.int32, device="cuda"), none,
                                   torch.empty((0, 4, 9), device="cuda"))
    assert got[1].shape == (0, 4)


def test_verify_step_example_follows_the_model():
    """examples/verify_step.py, greedy and sampled: every greedily committed token has a
    logit within 0.25 of the largest at its place, in a plain pass over the whole
    sequence (each 16-bit rounding of the hidden row moves a logit by 2.8 * 2^-8 / sqrt
    3 in the mean, five of them and the logits' own come to 0.03, eight times that is
    0.25), and more than one token a step is committed in the mean."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    V, steps = 64, 40
    model = ex.Model(V, hq=4, hkv=2, d=64, max_pos=2048)
    hist = ex.histories(5, V, 3)
    got = ex.generate(model, hist, steps, 7)
    assert sum(map(len, got)) > 1.2 * steps * len(hist)
    emb, qkv, wo, head = (w.float() for w in (model.embed, model.qkv, model.out, model.head))
    rot = model.rotary.float()
    for h, g in zip(hist, got):
        seq = torch.tensor(h + g, device="cuda")
        L = seq.shape[0]
        x = emb[seq]
        q, k, v = (x @ qkv).view(L, 8, 64).split([4, 2, 2], 1)
        cos, sin = rot[:L, None, :32], rot[:L, None, 32:]

        def turn(z):
            a, b = z[..., :32], z[..., 32:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

        q, k, v = turn(q), turn(k).repeat_interleave(2, 1), v.repeat_interleave(2, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / 8.0
        s.masked_fill_(torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1), -math.inf)
        a = torch.einsum("hij,jhd->ihd", s.softmax(-1), v)
        z = (x + a.reshape(L, -1) @ wo) @ head
        at = torch.arange(len(h) - 1, L - 1, device="cuda")
        gap = z[at].amax(-1) - z[at, seq[at + 1]]
        assert float(gap.max()) < 0.25
    rng = torch.Generator(device="cuda")
    rng.manual_seed(2)
    sampled = ex.generate(model, hist, 5, 7, lambda B, K: dict(
        u=torch.rand((B, K), device="cuda", generator=rng),
        noise=torch.empty((B, V), device="cuda").exponential_(generator=rng)))
    assert all(len(s) >= 5 and all(0 <= t < V for t in s) for s in sampled)


def test_append_writes_past_32_bits():
    """A pool of more than 2^32 bytes: the last page's rows are where they belong."""
    pages, page, D = 70000, 64, 256                      # 2.3 GB each for k and v: 1.1e9 elements
    kc = torch.zeros((pages, 2, page, D), dtype=BF16, device="cuda")
    vc = torch.zeros((pages, 2, page, D), dtype=BF16, device="cuda")
    assert kc.numel() > 1 << 31
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 2, 2, D), device="cuda").to(BF16)
    kv = torch.tensor([62], dtype=torch.int32, device="cuda")
    _, st = pkg.lookup_kv_append(q, q, q, kv, table, kc, vc)
    assert int(st) == 0
    assert torch.equal(kc[pages - 1, :, 62:], q[0].transpose(0, 1)) and torch.equal(vc[pages - 1, :, 62:], q[0].transpose(0, 1))
    out, lse = pkg.lookup_paged_attention(q, kc, vc, table, kv)
    k = kc[pages - 1].double()                           # [2, 64, D]
    s = torch.einsum("nhd,hjd->nhj", q[0].double(), k) / 16.0
    s[0, :, 63] = -math.inf
    p = torch.softmax(s, -1)
    want = torch.einsum("nhj,hjd->nhd", p, vc[pages - 1].double())
    mass = torch.einsum("nhj,hjd->nhd", p, vc[pages - 1].double().abs())
    assert bool(((out[0].double() - want).abs() <= mass * 2.0 ** -8 * 1.05 + 2.0 ** -16).all())
