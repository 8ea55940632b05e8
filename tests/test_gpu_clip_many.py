"""Clipping of more tensors and elements than whose partial sums every workgroup adds up for itself (more than 4096 of them:
five launches of 96 tensors that fill the card each), against float64.  Bounds as in the parity tests."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("max_norm", [1.0, 1e6])
def test_many_large_tensors(max_norm):
    torch.manual_seed(5)
    sizes = [180224 + 16384 * (i % 3) - i % 7 for i in range(480)]
    assert sum(sizes[:96]) > 1024 * 16384 and len(sizes) > 4 * 96
    grads = [torch.randn(n, device=DEV).to(BF if i % 2 else F32) for i, n in enumerate(sizes)]
    grads[37], grads[200] = grads[37][:0], grads[200][1:]
    want = float(sum(g.double().square().sum() for g in grads).sqrt())
    norm = O.grad_norm(grads)
    assert abs(float(norm.double()) - want) <= U * want * (1 + 1e-3)  # float64 sums: the rounding of the norm alone
    outs = [torch.full_like(g, float("nan")) for g in grads]
    n2 = O.clip_gradients(grads, max_norm, out=outs)
    assert torch.equal(norm, n2)
    by = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, outs):
        r = g.double() * by
        half = 2.0 ** -8 if g.dtype is BF else 0.0
        assert bool(((o.double() - r).abs() <= (half + 10 * U) * r.abs() + 2.0 ** -134).all())
    n3 = O.clip_gradients(grads, max_norm)
    assert torch.equal(norm, n3)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
