"""The delta rule's gradients and time split, and the norms, through the C ABI: outputs and workspaces of exactly the
stated sizes between guards, at odd lengths and widths.  Nothing is written outside them, everything in an output is
written, and the values are those of the binding's calls."""
import ctypes

import pytest
import torch

from rwkv_wkv_mixing_amd import _lib as L
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DT = {F32: L.WKV_F32, BF: L.WKV_BF16}
TYPES = [(BF, BF), (F32, BF), (F32, F32)]
TIDS = ["bf16", "f32-bf16", "f32"]
PAD, MARK = 4096, 0xFF  # a float or bf16 of these bytes is a NaN


class Guarded:
    """Regions between guards; check() looks at all of them."""

    def __init__(self):
        self.buffers = []

    def bytes(self, n):
        buf = torch.full((2 * PAD + n,), MARK, dtype=torch.uint8, device=DEV)
        self.buffers.append(buf)
        return buf[PAD:PAD + n]

    def like(self, t):
        return self.bytes(t.nbytes).view(t.dtype).view(t.shape)

    def check(self):
        for i, buf in enumerate(self.buffers):
            assert bool((buf[:PAD] == MARK).all()) and bool((buf[-PAD:] == MARK).all()), i


def at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def delta_inputs(B, T, H, HK, N, dtype):
    g = torch.Generator().manual_seed(T + N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(w=torch.rand(B, T, H, generator=g) * 0.1, beta=torch.rand(B, T, H, generator=g), r=rn(B, T, HK * N).to(dtype),
             k=(rn(B, T, HK * N) / (2 * N ** 0.5)).to(dtype), v=rn(B, T, H * N).to(dtype), go=rn(B, T, H * N).to(dtype),
             S=rn(B, H, N, N), G=rn(B, H, N, N))
    p = {n: t.to(DEV) for n, t in p.items()}
    p["lengths"] = torch.tensor([T, max(T - 37, 0)][:B], dtype=torch.int32, device=DEV)
    return p


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,split", [(5, 64, False), (67, 64, False), (67, 128, False), (515, 64, True), (515, 64, False),
                                       (700, 128, True)])
@pytest.mark.parametrize("saved", [True, False], ids=["ckpt", "recomputed"])
def test_delta(dtype, T, N, split, saved):
    B, H, HK = 2, 2, 1
    lib, p, gd = L.lib(), delta_inputs(B, T, H, HK, N, dtype), Guarded()
    ck = gd.bytes(lib.wkv_delta_ckpt_bytes(B, T, H, N)) if saved else None
    nws = lib.wkv_delta_forward_workspace_bytes(B, T, H, HK, N)
    assert (nws > 0) == (T > 500)
    ws = gd.bytes(nws) if split else None
    o, S1 = gd.like(p["v"]), gd.like(p["S"])
    L.check("forward", lib.wkv_delta_forward(
        B, T, H, HK, N, DT[dtype], *(at(p[n]) for n in ("lengths", "w", "beta", "r", "k", "v")), at(o), at(p["S"]), at(S1), at(ck),
        at(ws), nws if split else 0, stream()))
    gd.check()
    own = O.new_delta_ckpt(B, T, H, N, DEV) if saved else None
    kw = dict(lengths=p["lengths"], state_in=p["S"], ckpt=own, split=split)
    want = O.delta_forward(*(p[n] for n in ("w", "beta", "r", "k", "v")), return_state=True, **kw)
    assert torch.equal(o, want[0]) and torch.equal(S1, want[1])
    nws = lib.wkv_delta_backward_workspace_bytes(B, T, H, HK, N, (1 if saved else 0) | (0 if split else 2))
    ws = gd.bytes(nws)
    grads = [gd.like(p[n]) for n in ("r", "k", "v", "w", "beta", "S")]
    L.check("backward", lib.wkv_delta_backward(
        B, T, H, HK, N, DT[dtype], *(at(p[n]) for n in ("lengths", "w", "beta", "r", "k", "v", "go", "S", "G")),
        *(at(t) for t in grads), at(ck), at(ws), nws, stream()))
    gd.check()
    want = O.delta_backward(*(p[n] for n in ("w", "beta", "r", "k", "v", "go")), grad_state_out=p["G"], need_state_grad=True, **kw)
    for x, y in zip(grads, want):
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())


@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("rows,H,G", [(1, 1, 1), (33, 3, 5), (7, 5, 129), (300, 3, 520), (65, 9, 8), (40, 3, 257), (9, 2, 1000)])
@pytest.mark.parametrize("shared", [False, True], ids=["own", "shared"])
def test_head_norm(rows, H, G, shared, types):
    ty, tg = types
    lib, gd = L.lib(), Guarded()
    g = torch.Generator().manual_seed(rows + G)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    n = G if shared else H * G
    p = dict(y=rn(rows, H * G).to(ty), weight=rn(n), bias=rn(n), gate=rn(rows, H * G).to(tg), gout=rn(rows, H * G).to(tg))
    p = {m: t.to(DEV) for m, t in p.items()}
    head = (rows, H, G, DT[ty], DT[tg], L.WKV_NORM_CENTER | (L.WKV_NORM_SHARED if shared else 0), L.WKV_ACT_SILU, ctypes.c_float(1e-5))
    kw = dict(heads=H, act="silu", center=True)
    out = gd.like(p["gate"])
    L.check("head norm", lib.wkv_head_norm(*head, *(at(p[m]) for m in ("y", "weight", "bias", "gate")), at(out), stream()))
    gd.check()
    assert torch.equal(out, O.head_norm(p["y"], p["weight"], p["bias"], p["gate"], **kw))
    nws = lib.wkv_head_norm_backward_workspace_bytes(rows, H, G)
    ws, grads = gd.bytes(nws), [gd.like(p[m]) for m in ("y", "weight", "bias", "gate")]
    L.check("head norm backward", lib.wkv_head_norm_backward(
        *head, *(at(p[m]) for m in ("y", "weight", "bias", "gate", "gout")), *(at(t) for t in grads), at(ws), nws, stream()))
    gd.check()
    for x, y in zip(grads, O.head_norm_backward(p["y"], p["gout"], p["weight"], p["bias"], p["gate"], **kw)):
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())


@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("rows", [1, 10, 777])
@pytest.mark.parametrize("C", [1, 64, 511, 1000, 4096, 4101, 8192])
def test_block_norm(rows, C, types):
    tx, ty = types
    lib, gd = L.lib(), Guarded()
    g = torch.Generator().manual_seed(rows + C)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    weights = ("post_w", "post_b", "scale", "pre_w", "pre_b")
    p = dict(x=rn(rows, C).to(tx), y=rn(rows, C).to(ty), gate=rn(rows, C).to(ty), gx=rn(rows, C).to(tx), gh=rn(rows, C).to(ty),
             **{m: rn(C) for m in weights})
    p = {m: t.to(DEV) for m, t in p.items()}
    head = (rows, C, DT[tx], DT[ty], L.WKV_NORM_CENTER, L.WKV_ACT_SIGMOID, ctypes.c_float(1e-5))
    kw = {m: p[m] for m in ("gate", "post_w", "post_b", "scale")}
    x_out, h = gd.like(p["x"]), gd.like(p["y"])
    L.check("block norm", lib.wkv_block_norm(*head, *(at(p[m]) for m in ("x", "y", "gate") + weights), at(x_out), at(h), stream()))
    gd.check()
    want = O.block_norm(p["x"], p["y"], p["pre_w"], p["pre_b"], **kw)
    assert torch.equal(x_out, want[0]) and torch.equal(h, want[1])
    nws = lib.wkv_block_norm_backward_workspace_bytes(rows, C)
    ws, names = gd.bytes(nws), ("dx", "dy", "dgate", "dpost_w", "dpost_b", "dscale", "dpre_w", "dpre_b")
    grads = {n: gd.like(p[n[1:]]) for n in names}
    L.check("block norm backward", lib.wkv_block_norm_backward(
        *head, at(x_out), *(at(p[m]) for m in ("y", "gate") + weights + ("gx", "gh")), *(at(grads[n]) for n in names), at(ws), nws,
        stream()))
    gd.check()
    want = O.block_norm_backward(x_out, p["y"], p["gh"], p["pre_w"], p["pre_b"], gx=p["gx"], **kw)
    for n in names:
        assert torch.equal(grads[n], want[n]) and bool(torch.isfinite(grads[n]).all()), n
