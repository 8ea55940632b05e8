"""Clipping by factors below float32's normal numbers, where the gradients are near its largest ones: the factor rounds to 24
bits and so does an element's product (10u for both and the norm, u = 2^-24, as in the parity tests), a bfloat16 element to
2^-8 more; below the normal numbers two roundings of 2^-150 make one step of 2^-149 (2^-133 in bfloat16)."""
import numpy as np
import pytest
import torch

from oracle.select_ref import clip_ref
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,size,max_norm", [(1000, 1e38, 1e-3), (1000, 1e38, 1e-8), (20000, 3e38, 1e-30), (7, 2.0 ** 127, 1e-2),
                                             (16384, 1e38, 1e-40), (1, 2.0 ** 126, 1.0), (4, 2.0 ** 125, 1.0), (50000, 1e37, 1.0)])
def test_factors_below_the_normal_numbers(n, size, max_norm, dtype):
    """(one of 2^126 and four of 2^125, with 33 next to nothing, make factors just below 2^-126, whose first number is 1)"""
    g = torch.Generator().manual_seed(n)
    grads = [(size * (0.5 + 0.5 * torch.rand(n, generator=g)) if n > 10 else torch.full((n,), size)).to(dtype).to(DEV),
             torch.full((33,), size * 2.0 ** -17, device=DEV)]
    norm, want = clip_ref([t.double().cpu().numpy() for t in grads], float(np.float32(max_norm)), 0.0)
    assert norm / max_norm >= 2.0 ** 126
    outs = [torch.full_like(t, float("nan")) for t in grads]
    shown = O.clip_gradients(grads, max_norm, eps=0.0, out=outs)
    assert float(shown) == float("inf") if norm > 3.5e38 else abs(float(shown) - norm) <= 8 * U * norm
    O.clip_gradients(grads, max_norm, eps=0.0)
    for t, o, r in zip(grads, outs, want):
        assert torch.equal(t, o)
        half, least = (2.0 ** -8, 2.0 ** -133) if t.dtype is BF else (0.0, 2.0 ** -149)
        assert (np.abs(t.double().cpu().numpy() - r) <= (half + 10 * U) * np.abs(r) + least).all()
    # (a value below half the smallest step, 2^-134 in bfloat16 and 2^-150 in float32, is zero when rounded)
    assert float(grads[0].float().abs().max()) > 0 or float(np.abs(want[0]).max()) < (2.0 ** -134 if dtype is BF else 2.0 ** -150)
