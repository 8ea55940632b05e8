"""A selective scan of no channels: sums over none of them, so b and c have gradients of zero."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,N", [(2, 5, 16), (3, 700, 8), (0, 5, 16), (2, 0, 32)])
def test_no_channels(B, T, N, dtype):
    x, w = torch.empty(B, T, 0, dtype=dtype, device=DEV), torch.empty(0, N, device=DEV)
    b = torch.randn(B, T, N, device=DEV).to(dtype).requires_grad_()
    c = torch.randn(B, T, N, device=DEV).to(dtype).requires_grad_()
    held = [torch.full_like(b, float("nan"), requires_grad=False) for _ in range(8)]
    del held  # (what the gradients' allocations are then likely to be given)
    out, state = O.selective_scan(x, x, w, b, c)
    assert out.shape == (B, T, 0) and state.shape == (B, 0, N)
    out.sum().backward()
    for t in (b, c):
        assert t.grad.shape == t.shape and not bool(t.grad.any())
