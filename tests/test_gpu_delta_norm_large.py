"""The delta rule and the norms at sizes of 2^32 threads, which one dimension of a grid does not hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("given", [True, False], ids=["state", "zero"])
def test_state_of_2_to_the_32_elements_without_tokens(given):
    """T = 0 copies the state: 2^20 + 1 pairs of 64 x 64, the last ones behind 2^32 elements."""
    from rwkv_wkv_mixing_amd import ops as O

    B = (1 << 20) + 1
    state = torch.empty(B, 1, 64, 64, device=DEV)
    flat = state.view(-1)
    part = torch.randn(1 << 26, device=DEV)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = part[:n] + float(i >> 26)
    e = lambda c: torch.empty(B, 0, c, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    w = torch.empty(B, 0, 1, device=DEV)
    out = torch.full_like(state, float("nan"))
    O.delta_forward(w, w, e(64), e(64), e(64), state_in=state if given else None, state_out=out)
    assert torch.equal(out, state) if given else not bool(out.any())
