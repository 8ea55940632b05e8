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


def test_head_norm_gradients_of_the_most_heads():
    """2^24 - 1 heads of one channel in 128 rows: the gradients of the first and the last heads, float64's of the
    formula (eps is far from 0, so that a head of one channel has one).  Bounds: a divisor of one term and a square
    root, some ten roundings of u = 2^-24, then one to bf16; dweight a sum of 128 float32 products."""
    from rwkv_wkv_mixing_amd import ops as O

    H, rows = (1 << 24) - 1, 128
    g = torch.Generator(device=DEV).manual_seed(0)
    y, gout = (torch.empty(rows, H, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for t in (y, gout):
        for i in range(rows):
            t[i] = torch.randn(H, generator=g, device=DEV)
    weight = torch.rand(H, generator=g, device=DEV) + 0.5
    dy, dw, _, _ = O.head_norm_backward(y, gout, weight, heads=H, eps=1.0)
    ends = torch.cat((torch.arange(1000), torch.arange(H - 1000, H))).to(DEV)
    ye, ge, we = y[:, ends].double(), gout[:, ends].double(), weight[ends].double()
    inv = torch.rsqrt(ye * ye + 1)
    want_dy, terms = ge * we * inv ** 3, ge * ye * inv
    mag = (ge * we).abs() * inv * (1 + (ye * inv) ** 2)
    assert bool(((dy[:, ends].double() - want_dy).abs() <= 2.0 ** -8 * want_dy.abs() + 16 * 2.0 ** -24 * mag).all())
    assert bool(((dw[ends].double() - terms.sum(0)).abs() <= (16 + 128) * 2.0 ** -24 * terms.abs().sum(0)).all())
    assert bool(torch.isfinite(dw).all())
