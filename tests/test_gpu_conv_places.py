"""The short convolution's tensors next to each other in one buffer, and the carried inputs' gradient in the carried inputs'
place: what the refusals of overlapping outputs leave allowed."""
import ctypes

import pytest
import torch

from rwkv_wkv_mixing_amd import _lib as L
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def at(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,C", [(2, 64), (70, 64), (700, 7)])
def test_tensors_next_to_each_other(T, C, K, dtype):
    B, lib = 3, L.lib()
    sizes = dict(dx=T, x=T, ds_in=K - 1, gout=T, s_in=K - 1, ds_out=K - 1, s_out=K - 1, out=T)
    arena = torch.randn(B * C * sum(sizes.values()), device=DEV).to(dtype)
    p, first = {}, 0
    for n, rows in sizes.items():
        p[n] = arena[first:first + B * rows * C].view(B, rows, C)
        first += B * rows * C
    weight, bias = torch.randn(K, C, device=DEV), torch.randn(C, device=DEV)
    keep = {n: p[n].clone() for n in ("x", "gout", "s_in", "ds_out")}
    want, want_state = O.conv_forward(keep["x"], weight, bias, state_in=keep["s_in"], return_state=True)
    wg = O.conv_backward(keep["x"], keep["gout"], weight, bias, state_in=keep["s_in"], grad_state_out=keep["ds_out"], need_state_grad=True)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    head = (B, T, C, K, L.WKV_BF16 if dtype is BF else L.WKV_F32, L.WKV_ACT_SILU, None)
    L.check("forward", lib.wkv_conv_forward(*head, at(p["x"]), at(weight), at(bias), at(p["s_in"]), at(p["out"]), at(p["s_out"]), stream))
    nws = lib.wkv_conv_backward_workspace_bytes(B, T, C, K)
    ws, dw, db = torch.empty(nws, dtype=torch.uint8, device=DEV), torch.empty_like(weight), torch.empty_like(bias)
    for ds_in in ("ds_in", "s_in"):  # the second call last: it overwrites the carried inputs
        for n, v in keep.items():
            assert torch.equal(p[n], v), n
        L.check("backward", lib.wkv_conv_backward(*head, at(p["x"]), at(weight), at(bias), at(p["s_in"]), at(p["gout"]), at(p["ds_out"]),
                                                  at(p["dx"]), at(dw), at(db), at(p[ds_in]), at(ws), nws, stream))
        assert torch.equal(p["out"], want) and torch.equal(p["s_out"], want_state)
        for got, w in zip((p["dx"], dw, db, p[ds_in]), wg):
            # (a view off the vectors' grid takes one channel a thread, whose sums over tokens are grouped otherwise: 3 T terms)
            if got.dtype is F32 and got.dim() < 3:
                assert float((got - w).abs().max()) <= 2 * (B * T + 8) * 2.0 ** -24 * float(B * T * 16)
            else:
                assert torch.equal(got, w)
