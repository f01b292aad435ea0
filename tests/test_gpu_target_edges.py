"""The target's operators (include/lookup_target.h) where their arithmetic and their
memory are most easily wrong: temperatures down to float32's smallest, logits of 1e8.

The definitions and bounds are those of target_reference.py, as in test_gpu_target.py.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("prompt_lookup_speculative_gb300")

from test_gpu_target import BF16, F16, F32, check_verify, gen  # noqa: E402

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
