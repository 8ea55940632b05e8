"""The norms through the C ABI: gradients in the place that the header allows."""
import ctypes

import pytest
import torch

from rwkv_wkv_mixing_amd import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DT = {F32: L.WKV_F32, BF: L.WKV_BF16}
GRADS = ("dx", "dy", "dgate", "dpost_w", "dpost_b", "dscale", "dpre_w", "dpre_b")


def at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def block_inputs(rows, C, tx, ty):
    g = torch.Generator().manual_seed(rows + C)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    c = dict(x_out=2 * rn(rows, C).to(tx), y=rn(rows, C).to(ty), gate=rn(rows, C).to(ty), gx=rn(rows, C).to(tx),
             gh=rn(rows, C).to(ty), post_w=1 + 0.3 * rn(C), post_b=rn(C), scale=0.5 + 0.2 * rn(C), pre_w=1 + 0.3 * rn(C),
             pre_b=rn(C))
    return {n: t.to(DEV) for n, t in c.items()}


def block_outputs(c):
    like = dict(dx="x_out", dy="y", dgate="gate", dpost_w="post_w", dpost_b="post_b", dscale="scale", dpre_w="pre_w",
                dpre_b="pre_b")
    return {n: torch.full_like(c[like[n]], float("nan")) for n in GRADS}


def block_backward(c, out, ws, center=True):
    rows, C = c["y"].shape
    L.check("wkv_block_norm_backward", L.lib().wkv_block_norm_backward(
        rows, C, DT[c["x_out"].dtype], DT[c["y"].dtype], L.WKV_NORM_CENTER if center else 0, L.WKV_ACT_SILU,
        ctypes.c_float(1e-5), *(at(c[n]) for n in ("x_out", "y", "gate", "post_w", "post_b", "scale", "pre_w", "pre_b", "gx", "gh")),
        *(at(out[n]) for n in GRADS), at(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))


@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32)], ids=["bf16", "f32-bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 10, 20, 40, 300, 777, 1000, 8200])
@pytest.mark.parametrize("C", [64, 100, 256, 511, 1000, 4101])
def test_dx_in_place_of_gx(rows, C, types):
    """dx may be gx: bit for bit what the call gives with a dx of its own, whatever the number of rows leaves of
    the last workgroup's four."""
    c = block_inputs(rows, C, *types)
    ws = torch.empty(L.lib().wkv_block_norm_backward_workspace_bytes(rows, C), dtype=torch.uint8, device=DEV)
    want = block_outputs(c)
    block_backward(c, want, ws)
    for _ in range(3):
        own = dict(c, gx=c["gx"].clone())
        got = dict(block_outputs(c), dx=own["gx"])
        block_backward(own, got, ws)
        for n in GRADS:
            assert bool(torch.isfinite(want[n]).all()) and torch.equal(got[n], want[n]), n
