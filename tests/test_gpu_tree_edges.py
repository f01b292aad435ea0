"""A verify step over a tree (include/lookup_tree.h), where it can go wrong: values of V that
are not finite in many items at once, and visible ones of the smallest weights."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("prompt_lookup_speculative_gb300")

import tree_reference as ref  # noqa: E402
from test_gpu_target import BF16, F16, close, gen  # noqa: E402
from test_gpu_tree import check_norm, norm_case, tree_case  # noqa: E402

pytestmark = pytest.mark.gpu


def put(vc, table, at, col, value):
    """One element of position `at`'s row of V, in every key-value head."""
    page = vc.shape[2]
    vc[table[at // page], :, at % page, col] = value


def check_odd(case, places, scale=None, window=0, again=1):
    """`places`: {request: [(node, column, value)]}, each value infinite or NaN.  What sees one
    is that value in its column (NaN where it sees infinities of both signs), what does not is as
    if it were not there."""
    q, kc, vc, table, kv, ql, mask = case
    B, N, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    v1 = vc.clone()
    want = ref.attention(q, kc, vc, table, kv, ql, mask, scale, window)
    odd = torch.zeros((B, N, 1, D), dtype=torch.float64)
    for r, some in places.items():
        n, count = int(kv[r]), int(ql[r])
        for (node, col), value in {(node, col): value for node, col, value in some}.items():     # (the last one stands)
            put(v1, table[r], n + node, col, value)
            for i in range(count):
                if n + node in ref.seen(mask[r, i], n, count, n + count, window):
                    odd[r, i, 0, col] += value
    odd = odd.expand(-1, -1, Hq, -1)
    hit = odd != 0                                       # (NaN is not 0 either)
    assert bool(hit.any()) and not bool(hit.all())
    d = [x.cuda() for x in (q, kc, v1, table, kv, mask, ql)]
    first = None
    for _ in range(again):
        out, lse = pkg.lookup_tree_attention(*d[:6], q_len=d[6], scale=scale, window=window)
        got = out.double().cpu()
        assert bool(((got == odd) | (got.isnan() & odd.isnan()))[hit].all())
        close(torch.where(hit, want[0], got), want[0], want[2], "out")
        close(lse, want[1], want[3], "lse")
        assert first is None or torch.equal(first.view(torch.int16), out.view(torch.int16))
        first = out
    return v1


@pytest.mark.parametrize("N,Hq,Hkv,D", [(64, 4, 1, 128), (40, 8, 2, 64), (20, 14, 2, 64), (12, 4, 1, 128), (5, 8, 1, 128)])
def test_values_that_are_not_finite_in_some_of_many_items(N, Hq, Hkv, D):
    """Both groups of a CTA look through the same tiles, item after item, some with such values
    and some without: the same result, to the last bit, time after time."""
    g = gen(N + D)
    lens = [(37 * r * r) % 230 for r in range(400 // N)] * 4
    qn = [N if r % 4 else max(2, N // 2) for r in range(len(lens))]
    case = tree_case(lens, qn, N, Hq, Hkv, D, 16, BF16, N)
    places = {}
    for r in range(0, len(lens), 3):
        values = [math.inf, -math.inf, math.nan]
        places[r] = [(int(torch.randint(qn[r], (1,), generator=g)), int(torch.randint(D, (1,), generator=g)),
                      values[(r + k) % 3]) for k in range(2)]
    check_odd(case, places, again=4)


SHAPES = [(5, 4, 1, 128), (12, 4, 1, 128), (30, 4, 1, 128), (64, 4, 1, 128), (7, 4, 1, 64), (40, 8, 2, 64), (9, 4, 2, 256)]


@pytest.mark.parametrize("lens", [[6000, 3000], [0, 3, 20, 9] * 80, [700, 90, 1500, 2, 300, 1100] * 6])
@pytest.mark.parametrize("N,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("dt", [BF16, F16])
def test_values_that_are_not_finite_reach_those_of_the_smallest_weights(dt, N, Hq, Hkv, D, lens):
    """Scores hundreds apart, so that most weights vanish in float32: an infinity that is seen
    with one of them is still one, in an item of many parts, of one, and of a few."""
    rows = 600 // N
    lens = lens if len(lens) < 40 else lens[:max(rows, 8)]
    qn = [N - r % 3 for r in range(len(lens))]
    case = tree_case(lens, qn, N, Hq, Hkv, D, 16, dt, N + len(lens))
    q, kc, _, table, _, _, mask = case
    places = {r: [(1 + r % 2, 5 + r % 40, math.inf), (N // 2, 60 - r % 9, -math.inf)] for r in range(0, len(lens), 2)}
    least = 0.0
    for r in places:                                     # the smallest weight that counts, of head 0
        n = lens[r]
        for row in range(qn[r]):
            at = ref.seen(mask[r, row], n, qn[r], n + qn[r], 0)
            hits = [at.index(n + node) for node, _, _ in places[r] if n + node in at]
            if hits:
                k = torch.stack([kc[table[r, x // 16], 0, x % 16] for x in at]).double()
                z = 20.0 * (k @ q[r, row, 0].double())
                least = min(least, float((z[hits] - z.max()).min()))
    assert least < -150.0
    check_odd(case, places, scale=20.0)


@pytest.mark.parametrize("lens", [[6000, 3000], [200, 330, 190, 140]])
@pytest.mark.parametrize("N,Hq,Hkv,D", SHAPES)
def test_cached_values_that_are_not_finite_reach_all_that_see_them(N, Hq, Hkv, D, lens):
    """In positions that every token sees: infinite or NaN, whatever the weight, and nothing else
    changes."""
    case = tree_case(lens, [N] * len(lens), N, Hq, Hkv, D, 16, BF16, N + len(lens))
    q, kc, vc, table, kv, ql, mask = case
    v1 = vc.clone()
    for r, n in enumerate(lens):
        put(v1, table[r], 3 + 7 * r, 9, math.inf)
        put(v1, table[r], n // 2, 33, -math.inf)
    want = ref.attention(q, kc, vc, table, kv, ql, mask, 20.0, 0)
    out, lse = pkg.lookup_tree_attention(*(x.cuda() for x in (q, kc, v1, table, kv, mask)), scale=20.0)
    got = out.double().cpu()
    assert not bool(got[..., [9, 33]].isfinite().any())
    got[..., [9, 33]] = want[0][..., [9, 33]]
    close(got, want[0], want[2], "out")
    close(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot,inter,pad", [
    (10, 63, 7, 1, 64, 64, False, 0), (12, 55, 5, 3, 32, 16, True, 0), (40, 17, 1, 1, 16, 16, False, 8),
    (9, 70, 7, 3, 128, 64, True, 0), (2, 5, 33, 7, 128, 128, False, 16), (1, 7, 16, 16, 256, 256, True, 0),
    (3, 4, 70, 3, 64, 32, False, 0), (700, 1, 3, 1, 64, 64, True, 0),
])
def test_norm_append_of_few_and_many_tokens(dt, B, N, Hq, Hkv, D, rot, inter, pad):
    """One and two heads of a thread, even and odd numbers of them, tokens that fill a CTA and those
    that one CTA goes round for."""
    lens = [(37 * r + 3) % 70 if r else 0 for r in range(B)]
    qn = [(N + r) % (N + 1) if r % 5 == 1 else N for r in range(B)]
    c = norm_case(B, N, Hq, Hkv, D, rot, 16, lens, qn, dt, B * N + D, pad)
    whole, cached = check_norm(c, inter)
    one = {n: x[:1] if n in ("q", "k", "v", "kv", "ql", "table", "depth") else x for n, x in c.items()}
    q, to = check_norm(one, inter)                           # a token's bits are its own
    assert torch.equal(q, whole[:1])
    for j in range(-(-N // 16)):
        page, rows = int(c["table"][0, j]), min(16, N - 16 * j)
        assert torch.equal(to["kc"][page, :, :rows], cached["kc"][page, :, :rows])
    q, to = check_norm(c | dict(qw=None, kw=None, depth=None), inter)
    kc, vc = c["kc"].cuda(), c["vc"].cuda()
    want, _ = pkg.lookup_kv_append(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), to["kv"], to["table"], kc, vc,
                                   rotary=to["rotary"], q_len=to["ql"], interleaved=inter)
    if not (inter and dt == BF16):
        assert torch.equal(q, want) and torch.equal(to["kc"], kc)
    assert torch.equal(to["vc"], vc)


def test_steps_of_a_loop_with_the_lookups_draft_as_one_chain():
    """Draft, merge, greedy verification and append, step after step: what is committed is what the
    target says, one token after the other, whatever the second chain proposes."""
    B, K, V, N, steps = 5, 6, 40, 14, 6
    g = gen(4)
    follow = torch.randint(V, (V, V), generator=g)           # the target: a token from the last two
    rows = []
    for r in range(B):
        x = torch.randint(V, (2,), generator=g).tolist()
        while len(x) < 60 + 11 * r:
            x.append(int(follow[x[-2], x[-1]]))
        rows.append(x)
    want = [list(x) for x in rows]
    for x in want:
        while len(x) < 400:
            x.append(int(follow[x[-2], x[-1]]))
    history = torch.tensor(sum(rows, []), dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0] + [len(x) for x in rows], dtype=torch.int64).cumsum(0).cuda()
    most = 0
    for step in range(steps):
        draft, length, _, _ = pkg.lookup_draft_ex(history, offsets, 2, 8, K)
        at = offsets.tolist()
        now = [history[at[r]:at[r + 1]].tolist() for r in range(B)]
        assert all(x == want[r][:len(x)] for r, x in enumerate(now))
        other = torch.randint(V, (B, K), generator=g).to(torch.int32)
        for r in range(0, B, 2):                             # a model that is right for a while
            other[r, :3] = torch.tensor(want[r][len(now[r]):len(now[r]) + 3])
        chains = torch.stack([draft, other.cuda()], 1)
        lengths = torch.stack([length, torch.full_like(length, K)], 1)
        root = torch.tensor([x[-1] for x in now], dtype=torch.int32, device="cuda")
        tokens, parent, depth, mask, n = pkg.lookup_tree_merge(root, chains, lengths, N)
        logits = torch.zeros((B, N, V))
        t, p = tokens.tolist(), parent.tolist()
        for r in range(B):
            for i in range(int(n[r])):
                before = t[r][p[r][i]] if i else now[r][-2]
                logits[r, i, follow[before, t[r][i]]] = 9.0
        acc, commit, ncommit, path, _ = pkg.lookup_verify_tree(tokens, parent, n, logits.cuda())
        assert torch.equal(ncommit, acc + 1) and bool((acc.cpu()[::2] >= 3).all())
        most = max(most, int(acc.max()))
        history, offsets = pkg.lookup_append(history, offsets, commit, ncommit)
    assert most >= 4                                         # (the lookup's: the target goes round)
