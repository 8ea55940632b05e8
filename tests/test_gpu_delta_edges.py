"""Edges of the delta rule's documented range that the parity tests do not reach."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ops():
    from rwkv_wkv_mixing_amd import ops as O

    return O


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_key_heads_without_value_heads(dtype):
    """H = 0 is a multiple of any HK: o is empty, and dr and dk are empty sums, zeros, and not whatever the
    memory held."""
    O = ops()
    e = lambda *s: torch.empty(s, device=DEV, dtype=dtype)  # noqa: E731
    w = torch.empty(2, 37, 0, device=DEV)
    r = torch.randn(2, 37, 192, device=DEV).to(dtype)
    assert O.delta_forward(w, w, r, r, e(2, 37, 0)).shape == (2, 37, 0)
    junk = [torch.full_like(r, float("nan")) for _ in range(4)]
    del junk  # what the gradients' memory holds
    dr, dk, dv, dw, dbeta, _ = O.delta_backward(w, w, r, r, e(2, 37, 0), e(2, 37, 0))
    assert dr.shape == dk.shape == r.shape and not bool(dr.any()) and not bool(dk.any())
    assert dv.shape == (2, 37, 0) and dw.shape == dbeta.shape == w.shape
    leaves = [t.requires_grad_() for t in (w, r.clone())]
    O.delta_rule(leaves[0], w.detach(), leaves[1], r, e(2, 37, 0))[0].sum().backward()
    assert not bool(leaves[1].grad.any())
