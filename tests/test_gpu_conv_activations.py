"""The convolution's activations far from zero, float32: silu and sigmoid to a few roundings of their own value wherever
their argument lies (u = 2^-24: the exponential 2u of the hardware's and 1u of what is put back, 1 + e 1u, the reciprocal 2u,
products 3u, the argument and the derivative's own sums 4u: 13u of the sizes of the terms; a reciprocal below 2^-126 is
zero, which times an argument of up to 80 is below 2^-118)."""
import numpy as np
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def near(got, want, size, name):
    worst = float((np.abs(got.double().cpu().numpy() - want) / (13 * U * size + 2.0 ** -118)).max())
    assert worst <= 1.0, (name, worst)


def sigmoid(v):
    return np.where(v >= 0, 1.0, np.exp(-np.abs(v))) / (1 + np.exp(-np.abs(v)))


def arguments(C):
    g = torch.Generator().manual_seed(C)
    return torch.cat([torch.linspace(-80, 80, 3 * C), 10 * torch.randn(3 * C, generator=g)]).view(1, 6, C)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("C", [700, 701])
def test_conv(C, T, act):
    """A filter of one tap that is not zero: the argument is the input itself."""
    x = arguments(C)[:, :T].contiguous()
    weight = torch.zeros(2, C)
    weight[1] = 1.0
    v = x.double().numpy()
    p = sigmoid(v)
    q = sigmoid(-v)
    out = O.conv_forward(x.to(DEV), weight.to(DEV), act=act)
    near(out, p if act == "sigmoid" else v * p, p if act == "sigmoid" else np.abs(v) * p, "out")
    dx = O.conv_backward(x.to(DEV), torch.ones_like(x, device=DEV), weight.to(DEV), act=act)[0]
    if act == "sigmoid":  # (1 - p is good to a rounding of p)
        near(dx, p * q, p, "dx")
    else:
        near(dx, p * (1 + v * q), p * (1 + np.abs(v)), "dx")
