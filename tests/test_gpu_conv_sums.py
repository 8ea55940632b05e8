"""The convolution's sums over many tokens (dweight, dbias) of terms that are all alike, whose roundings in one float32 sum add
up.

Bounds (u = 2^-24, 5 K u and less for P, the sum before the activation): a term g X is within 4u + (2 K + 12)u (1 + P) / p' of
its size, p' the slope (more than 0.5 here, so 2 (2 K + 12)(1 + P)u); 128 tokens of four runs are added in float32 (132u),
workgroups in float64 with a rounding to float32 at the end (1u)."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("B,T,C", [(8, 65536, 4096), (8, 65536, 1023), (1, 3000000, 64), (70001, 5, 64)])
def test_many_tokens(B, T, C, K, dtype):
    g = torch.Generator().manual_seed(T + C + K)
    token, go = ((0.5 + 0.5 * torch.rand(C, generator=g)).to(dtype).to(DEV) for _ in range(2))
    weight, bias = (torch.rand(K, C, generator=g) / K).to(DEV), (0.2 * torch.rand(C, generator=g)).to(DEV)
    x, gout = (t.expand(B, T, C).contiguous() for t in (token, go))
    _, dweight, dbias, _ = O.conv_backward(x, gout, weight, bias, state_in=token.expand(B, K - 1, C).contiguous())
    pre = bias.double() + weight.double().sum(0) * token.double()
    p = torch.sigmoid(pre)
    slope = p * (1 + pre * (1 - p))
    assert float(slope.min()) > 0.5 and float(pre.max()) < 1.3
    want = go.double() * slope * (B * T)
    rel = (4 + 2 * (2 * K + 12) * (1 + float(pre.max())) + 133) * 2.0 ** -24
    assert float(((dbias.double() - want) / want).abs().max()) <= rel
    want = want * token.double()
    assert float(((dweight.double() - want) / want).abs().max()) <= rel
