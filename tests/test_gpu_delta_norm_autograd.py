"""What the differentiable delta rule and norms refuse to differentiate."""
import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(T=5, H=2, N=64):
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    return [rn(1, T, H).abs(), rn(1, T, H).sigmoid(), rn(1, T, H * N), 0.1 * rn(1, T, H * N), rn(1, T, H * N), rn(1, H, N, N)]


@pytest.mark.parametrize("which", range(6), ids=["w", "beta", "r", "k", "v", "state"])
@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
def test_forward_mode_is_refused(which, grad):
    """A dual tensor has no requires_grad: the call must not return outputs that have lost its tangent."""
    from rwkv_wkv_mixing_amd import ops as O

    p = inputs()
    want = O.delta_rule(*p)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        got = O.delta_rule(*p)  # no input is a dual tensor
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        p[which] = forward_ad.make_dual(p[which], torch.ones_like(p[which]))
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            O.delta_rule(*p)


def test_forward_mode_of_the_norms_is_refused():
    from rwkv_wkv_mixing_amd import ops as O

    v, ones = inputs()[4], torch.ones(128, device=DEV)
    with forward_ad.dual_level(), torch.no_grad():
        d = forward_ad.make_dual(v, v)
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            O.head_norm_gated(d, ones, heads=2)
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            O.block_join(d, v, ones)


def test_functional_transforms_are_refused():
    from rwkv_wkv_mixing_amd import ops as O

    p = inputs()
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda v: O.delta_rule(*p[:4], v, p[5])[0], (p[4],), (p[4],))
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda v: O.delta_rule(*p[:4], v, p[5])[0])(torch.stack([p[4], p[4]]))
