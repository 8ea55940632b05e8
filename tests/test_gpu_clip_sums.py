"""The norm of gradients is the float32 next to the root of the sum of squares: squares and their sums are float64, within
some n 2^-53 of the sum, which moves the nearest float32 only where the root lies that near the middle of two (the test says
how near, and that it does not)."""
import numpy as np
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 8, 24, 1000, 16384, 70001])
@pytest.mark.parametrize("seed", range(6))
def test_the_norm_is_the_nearest_float32(seed, n, dtype):
    g = torch.Generator().manual_seed(100 * seed + n)
    host = torch.randn(n, generator=g).to(dtype)
    squares = host.double().numpy() ** 2
    root = float(np.sqrt(np.longdouble(0) + np.sum(squares.astype(np.longdouble))))
    want = np.float32(root)
    middle = [(float(want) + float(np.nextafter(want, np.float32(to)))) / 2 for to in (0.0, 1e38)]
    assert min(abs(root - m) for m in middle) > 2 * (n + 8) * 2.0 ** -53 * root
    norm = O.grad_norm([host.to(DEV)])
    assert float(norm) == float(want), (float(norm), root)
