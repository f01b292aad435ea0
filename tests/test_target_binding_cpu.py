"""The target's operators' Python entry: refusals that need no GPU."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import prompt_lookup_speculative_gb300 as pkg  # noqa: E402


def test_a_gradient_that_would_be_lost_is_refused():
    """Checked before the device is: under no_grad the same call gets as far as that."""
    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, requires_grad=True)
    n = torch.zeros(1, dtype=torch.int32)
    z = torch.zeros((1, 2, 8), requires_grad=True)
    for call in (lambda: pkg.lookup_paged_attention(x, x, x, n[None], n),
                 lambda: pkg.lookup_kv_append(x, x, x, n, n[None], x, x),
                 lambda: pkg.lookup_verify_logits(n[None], n, z)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
