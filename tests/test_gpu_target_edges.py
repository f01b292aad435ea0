"""The target's operators (include/lookup_target.h) where their arithmetic and their
memory are most easily wrong: temperatures down to float32's smallest, logits of 1e8,
weights far below a row's largest, streams other than the current one.

The definitions and bounds are those of target_reference.py, as in test_gpu_target.py.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("prompt_lookup_speculative_gb300")

from test_gpu_target import BF16, F16, F32, attention_case, check_attention, check_verify, gen, verify_case  # noqa: E402

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ verify ----
def led_case(T, dt, V, shift, seed, B=6, P=3, mode="point"):
    """Rows with one logit ahead of the others by 3 to 9 (so of probability 1 at a low
    temperature), the proposals mostly that one; all logits shifted by `shift`."""
    g = gen(seed)
    z = torch.randn((B, P + 1, V), generator=g) * 2.0
    lead = torch.randint(V, (B, P + 1), generator=g)
    top = z.amax(-1, keepdim=True) + 3.0 + 6.0 * torch.rand((B, P + 1, 1), generator=g)
    z = (z.scatter(2, lead[..., None], top) + shift).to(dt)
    block = lead[:, :P].to(torch.int32)
    other = torch.rand((B, P), generator=g) < 0.2
    block = torch.where(other, torch.randint(V, (B, P), generator=g).to(torch.int32), block).contiguous()
    qprobs = point = None
    if mode == "draft":
        qprobs = torch.softmax(torch.randn((B, P, V), generator=g), -1)
        point = (torch.rand((B, P), generator=g) < 0.5).to(torch.int32)
    return dict(block=block, length=torch.full((B,), P, dtype=torch.int32), logits=z,
                noise=torch.empty((B, V)).exponential_(generator=g).clamp_(min=1e-30),
                u=torch.rand((B, P), generator=g), temperature=torch.full((B,), T), qprobs=qprobs, point_mass=point)


@pytest.mark.parametrize("T", [0.05, 0.02, 1e-2, 1e-4, 1e-5, 3e-6, 1e-6, 3e-7, 1e-7, 1e-9, 1e-15, 1e-30, 1e-38, 1e-41])
@pytest.mark.parametrize("dt,V,shift,mode", [(F32, 4099, 10.0, "point"), (F32, 515, -40.0, "draft"), (BF16, 4100, 12.0, "draft"),
                                             (BF16, 1000, -25.0, "point"), (F16, 32000, 0.0, "point")])
def test_verify_low_temperatures(T, dt, V, shift, mode):
    """Every positive finite temperature samples: at a low one the leader has all the
    weight, its proposal is accepted and its log-probability is 0 up to rounding."""
    acc, commit, nc, lps = check_verify(led_case(T, dt, V, shift, 100 + V, mode=mode))
    assert bool(lps.isfinite().all()) and bool((nc == acc + 1).all())


@pytest.mark.parametrize("T", [1.0, 0.3, 1e4, None])
@pytest.mark.parametrize("size", [1e8, -1e8, 3e30])
def test_verify_large_finite_logits(size, T):
    """Finite float32 logits of either sign and any size, sampled and greedy (None): the
    leader is 32 units in the last place ahead; and rows of equal logits."""
    c = led_case(T or 1.0, F32, 3000, 0.0, 7)
    c["logits"] = torch.full_like(c["logits"], size)
    c["logits"].scatter_(2, c["block"].long()[..., None].clone(), size + abs(size) * 2.0 ** -18)
    c["logits"][0] = size                                    # uniform: log-probability -log V
    c["block"][3, 1] = (c["block"][3, 1] + 1) % 3000
    if T is None:
        c["noise"] = c["u"] = c["temperature"] = None
    _, _, _, lps = check_verify(c, least=0.6)
    assert bool(lps.isfinite().all())


# --------------------------------------------------------------- attention ----
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 17.5, 19.0, 21.0])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,L", [(40, 1, 8, 8, 64, 16384), (1, 1, 1, 1, 128, 40000), (76, 6, 32, 4, 128, 5000),
                                            (40, 16, 64, 8, 64, 9000), (40, 3, 16, 4, 256, 4001)])
def test_attention_long_tail_behind_one_large_score(dt, gap, B, N, Hq, Hkv, D, L):
    """One position `gap` nats above all the others, which hold v = 1 where it holds 0: the
    output is what the others' small weights come to.  A weight w (the largest is 1) may
    be off by its rounding to the type, or in float16 by half a step of 2^-24 / 2^7."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(gap * 2) + D)
    page, u = 64, 2.0 ** -11 if dt == F16 else 2.0 ** -8
    width = -(-(L + N) // page)
    kc = torch.randn((B * width, Hkv, page, D), device="cuda", generator=g).to(dt)
    kc[..., 0] = (0.25 * torch.randn(kc.shape[:3], device="cuda", generator=g)).clamp(-1, 1).to(dt)
    vc = torch.ones_like(kc)
    vc[..., 1] = torch.rand(kc.shape[:3], device="cuda", generator=g).to(dt)
    table = torch.randperm(B * width, device="cuda", generator=g).to(torch.int32).view(B, width)
    at = torch.randint(L, (B,), device="cuda", generator=g)
    first = table[torch.arange(B, device="cuda"), at // page].long()
    kc[first, :, at % page, 0] = gap
    vc[first, :, at % page] = 0.0
    q = torch.zeros((B, N, Hq, D), device="cuda", dtype=dt)
    q[..., 0] = D ** 0.5 if D != 128 else 8.0            # the score is a key's first element
    scale = D ** -0.5 if D != 128 else 0.125
    out, lse = pkg.lookup_paged_attention(q, kc, vc, table, torch.full((B,), L, dtype=torch.int32, device="cuda"), scale=scale)
    torch.cuda.synchronize()
    pos = torch.arange(width * page, device="cuda")
    see = pos <= L + torch.arange(N, device="cuda")[:, None]
    tiny = 2.0 ** -32 if dt == F16 else 0.0
    for b in range(0, B, 7):
        k0 = kc[table[b].long()][..., 0].transpose(0, 1).reshape(Hkv, 1, -1).double()      # [Hkv, 1, positions]
        v = vc[table[b].long()].transpose(0, 1).reshape(Hkv, -1, D).double()
        w = torch.where(see, (k0 - gap).exp(), 0.0)                                        # [Hkv, N, positions]
        z = w.sum(-1, keepdim=True)
        o = (w / z) @ v
        lost = (torch.minimum(w, torch.full_like(w, tiny)) + w * u) / z @ v
        bound = lost * 1.01 + o * (u + 2.0 ** -18 + (L + 64) * 2.0 ** -24) + 2.0 ** -25
        o, bound = (x.repeat_interleave(Hq // Hkv, 0).transpose(0, 1) for x in (o, bound))
        assert bool(((out[b].double() - o).abs() <= bound).all()), float(((out[b].double() - o).abs() / bound).max())
        one = (gap + z[..., 0].log()).repeat_interleave(Hq // Hkv, 0).T
        assert bool(((lse[b].double() - one).abs() <= one.abs() * 2.0 ** -22 + (L + 64) * 2.0 ** -24).all())


# --------------------------------------------------------------- arguments ----
def grad_calls():
    """The three calls as functions of an input that requires a gradient, by its name."""
    q, kc, vc, table, kv, ql = (x.cuda() for x in attention_case([30, 70], [4, 4], 4, 4, 2, 64, 16, BF16, 3))
    c = {k: None if v is None else v.cuda() for k, v in verify_case(3, 2, 101, F32, "draft", 5).items()}

    def attention(**x):
        return pkg.lookup_paged_attention(*(x.get(n, t) for n, t in (("q", q), ("k_cache", kc), ("v_cache", vc))), table, kv)

    def append(**x):
        t = dict(q=q, k=q[:, :, :2], v=q[:, :, 2:]) | x
        return pkg.lookup_kv_append(t["q"], t["k"], t["v"], kv, table, kc, vc)

    def verify(**x):
        t = c | x
        return pkg.lookup_verify_logits(t["block"], t["length"], t["logits"], noise=t["noise"], u=t["u"], qprobs=t["qprobs"])

    return [(attention, "q", q), (attention, "k_cache", kc), (attention, "v_cache", vc), (append, "q", q),
            (append, "k", q[:, :, :2]), (append, "v", q[:, :, 2:]), (verify, "logits", c["logits"]), (verify, "qprobs", c["qprobs"])]


def test_a_gradient_that_would_be_lost_is_refused():
    for call, name, x in grad_calls():
        x = x.clone().requires_grad_()
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call(**{name: x})
        with torch.no_grad():
            got = call(**{name: x})
        want = call(**{name: x.detach()})
        assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))


@pytest.mark.parametrize("B,N,Hq", [(1, 3, 4), (3, 1, 4), (3, 4, 1), (1, 1, 1)])
def test_an_axis_of_one_may_have_any_stride(B, N, Hq):
    """PyTorch leaves such strides as they come out, and nothing is read by them."""
    q, kc, vc, table, kv, ql = (x.cuda() for x in attention_case([33, 70, 5][:B], [N] * B, N, Hq, 1, 64, 16, BF16, 6))
    odd = q.as_strided(q.shape, [s if n > 1 else 515 for n, s in zip(q.shape[:3], q.stride())] + [1])
    want = pkg.lookup_paged_attention(q, kc, vc, table, kv)
    got = pkg.lookup_paged_attention(odd, kc, vc, table, kv)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    kv0 = q[:, :, :1].contiguous()
    odd_kv = kv0.as_strided(kv0.shape, [s if n > 1 else 515 for n, s in zip(kv0.shape[:3], kv0.stride())] + [1])
    caches = [(kc.clone(), vc.clone()) for _ in range(2)]
    want = pkg.lookup_kv_append(q, kv0, kv0, kv, table, *caches[0])
    got = pkg.lookup_kv_append(odd, odd_kv, odd_kv, kv, table, *caches[1])
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(*caches))


def test_sampling_without_proposals_needs_no_uniforms():
    """P = 0 is plain sampling: noise alone decides."""
    c = verify_case(7, 0, 777, BF16, "point", 9)
    want = check_verify(c)
    got = pkg.lookup_verify_logits(c["block"].cuda(), c["length"].cuda(), c["logits"].cuda(), noise=c["noise"].cuda(),
                                   temperature=c["temperature"].cuda())
    assert all(torch.equal(x.cpu(), y) for x, y in zip(got, want))


# ------------------------------------------------------------- wait limits ----
@pytest.mark.parametrize("ns", [1 << 62, 1 << 63, (1 << 63) + 1, (1 << 64) - 1, 1 << 70])
def test_a_wait_limit_of_any_size_is_a_long_one(ns):
    """Limits that would pass 64 bits once doubled, or on top of the timer."""
    draft = [torch.tensor(x, device="cuda") for x in ([5, 6, 7, 8, 9, 5, 6, 7, 8], [0, 9])]
    args = draft[0].to(torch.int32), draft[1].to(torch.int64)
    want = pkg.lookup_draft(*args, min_m=2, max_m=4, K=4)
    pkg.set_wait_limit_ns(ns)
    try:
        check_attention(*attention_case([300, 31], [4, 3], 4, 4, 2, 128, 16, BF16, 22))
        check_verify(verify_case(5, 3, 3001, BF16, "point", 12), least=0.6)
        got = pkg.lookup_draft(*args, min_m=2, max_m=4, K=4)
        torch.cuda.synchronize()
    finally:
        pkg.set_wait_limit_ns(0)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# ----------------------------------------------------------------- streams ----
def calls_on(stream):
    """The three calls on `stream` (None: the current one), each as a function of nothing."""
    q, kc, vc, table, kv, ql = (x.cuda() for x in attention_case([700, 1500], [16, 16], 16, 8, 2, 128, 16, BF16, 3))
    c = {k: None if v is None else v.cuda() for k, v in verify_case(8, 15, 9001, BF16, "point", 5).items()}
    k = kc[:2, :, :, :].reshape(2, 16, 2, 128)
    into = torch.zeros_like(kc), torch.zeros_like(vc)
    return {
        "attention": lambda: pkg.lookup_paged_attention(q, kc, vc, table, kv, q_len=ql, stream=stream),
        "verify": lambda: pkg.lookup_verify_logits(c["block"], c["length"], c["logits"], noise=c["noise"], u=c["u"],
                                                   temperature=c["temperature"], stream=stream),
        "append": lambda: pkg.lookup_kv_append(q, k, k, kv, table, *into, stream=stream),
    }


@pytest.mark.parametrize("name", ["attention", "verify", "append"])
def test_another_streams_call_leaves_released_memory_alone(name):
    """Tensors of the current stream that were released while work that reads them waits: a
    call on another stream must not write there, be it outputs or its workspace."""
    side = torch.cuda.Stream()
    call, want = calls_on(side)[name], calls_on(None)[name]()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want] + [
        pkg.load_library().lookup_paged_attention_workspace_bytes(2, 16, 8, 2, 128),
        pkg.load_library().lookup_verify_logits_workspace_bytes(8, 15, 9001)]
    torch.cuda.empty_cache()
    kept = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(40)]
    released = [torch.full_like(t, 0x5A) for t in kept]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                     # 0.1 s of the current stream
    for to, t in zip(kept, released):
        to.copy_(t)
    del released, t
    got = call()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()
    assert all(bool((t == 0x5A).all()) for t in kept)


def test_an_output_released_early_is_not_used_again():
    """The output of a call on another stream, read by the current one and released before
    that has happened: the next calls there must leave it alone."""
    side = torch.cuda.Stream()
    call = calls_on(side)["attention"]
    torch.cuda.synchronize()
    out, lse = call()
    torch.cuda.current_stream().wait_stream(side)
    want = out.clone()
    torch.cuda.synchronize()
    kept = torch.zeros_like(out)
    torch.cuda._sleep(200_000_000)
    kept.copy_(out)
    del out, lse
    with torch.cuda.stream(side):
        for _ in range(20):                            # whoever takes memory of that stream next
            torch.full_like(kept, 7.0)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


@pytest.mark.parametrize("name", ["attention", "verify", "append"])
def test_a_graph_with_a_second_stream(name):
    """A capture that forks to another stream for the call: the outputs are the graph's."""
    side = torch.cuda.Stream()
    call, want = calls_on(side)[name], calls_on(None)[name]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call()
        here.wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        stream_id, device_index, device_type = 0, 1, 1

    for call in calls_on(Elsewhere()).values():
        with pytest.raises(ValueError, match="stream"):
            call()
    assert torch.cuda.current_device() == 0
