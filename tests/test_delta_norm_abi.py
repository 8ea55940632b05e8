"""CPU-side checks of the delta-rule and norm entry points: sizes, and every refusal, all decided on the host
before any HIP call (so these run without a GPU)."""
import ctypes
import os
import re

import pytest
import torch

from rwkv_wkv_mixing_amd import _lib as L
from rwkv_wkv_mixing_amd import ops as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X = 0x10000  # a fake address, never dereferenced: the calls below are refused on the host
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from rwkv_wkv_mixing_amd.build import build

        build()
    return L.lib()


def test_header_constants_match_binding():
    src = open(os.path.join(ROOT, "include", "wkv.h")).read()
    for name in ("WKV_NORM_CENTER", "WKV_NORM_SHARED"):
        assert re.search(rf"#define {name} {getattr(L, name)}\b", src)
    for name in ("WKV_ACT_NONE", "WKV_ACT_SIGMOID", "WKV_ACT_SILU"):
        assert re.search(rf"{name} = {getattr(L, name)}\b", src)


def delta_fwd(lib, B=1, T=20, H=4, HK=2, N=64, dt=L.WKV_BF16, ln=None, w=X, beta=X, r=X, k=X, v=X, o=X, s_in=None, s_out=None,
              ck=None, ws=None, nws=0):
    return lib.wkv_delta_forward(B, T, H, HK, N, dt, ln, w, beta, r, k, v, o, s_in, s_out, ck, ws, nws, None)


def delta_bwd(lib, B=1, T=20, H=4, HK=2, N=64, dt=L.WKV_BF16, ln=None, w=X, beta=X, r=X, k=X, v=X, go=X, s_in=None, ds_out=None,
              dr=X, dk=X, dv=X, dw=X, db=X, ds_in=None, ck=X, ws=X, nws=1 << 30):
    return lib.wkv_delta_backward(B, T, H, HK, N, dt, ln, w, beta, r, k, v, go, s_in, ds_out, dr, dk, dv, dw, db, ds_in, ck, ws,
                                  nws, None)


@pytest.mark.parametrize("call", [delta_fwd, delta_bwd])
def test_delta_refusals(lib, call):
    for bad in (dict(B=-1), dict(T=-1), dict(H=-4), dict(HK=-2), dict(HK=3), dict(HK=0), dict(N=32), dict(N=96), dict(N=0)):
        assert call(lib, **bad) == L.WKV_EINVAL, bad
    assert call(lib, dt=2) == L.WKV_EDTYPE
    for bad in (dict(B=1 << 31), dict(T=1 << 50), dict(H=1 << 40, HK=1 << 40), dict(H=1 << 16, HK=1 << 16),
                dict(B=1 << 20, H=1 << 12, HK=1), dict(B=1 << 22, H=1, HK=1), dict(B=1 << 25, H=1, HK=1, T=1)):
        assert call(lib, **bad) == L.WKV_ESIZE, bad
    for name in ("w", "beta", "r", "k", "v"):
        assert call(lib, **{name: None}) == L.WKV_EINVAL, name
    for name in ("r", "k", "v", "s_in"):
        assert call(lib, **{name: X + 8}) == L.WKV_EALIGN, name
    for name in ("w", "beta", "ln"):
        assert call(lib, **{name: X + 2}) == L.WKV_EALIGN, name


def test_delta_forward_refusals(lib):
    assert delta_fwd(lib, B=1 << 22, H=1, HK=1, T=16, ck=X) == L.WKV_ESIZE  # with a ckpt it walks
    assert delta_fwd(lib, B=1 << 22, H=1, HK=1, T=16, o=None) == L.WKV_EINVAL  # without, it may
    assert delta_fwd(lib, o=None) == L.WKV_EINVAL
    for name in ("o", "s_out", "ck"):
        assert delta_fwd(lib, **{name: X + 4}) == L.WKV_EALIGN, name
    need = lib.wkv_delta_forward_workspace_bytes(1, 8192, 4, 2, 64)
    assert need > 0
    assert delta_fwd(lib, T=8192, ws=X, nws=need - 1) == L.WKV_EWORKSPACE
    assert delta_fwd(lib, T=8192, ws=X + 16, nws=need) == L.WKV_EWORKSPACE
    for empty in (dict(B=0), dict(H=0, HK=0), dict(H=0)):  # nothing to do: nothing is touched
        assert delta_fwd(lib, **empty) == L.WKV_OK, empty
    assert delta_fwd(lib, T=0, w=None, r=None) == L.WKV_OK


def test_delta_backward_refusals(lib):
    for name in ("go", "dr", "dk", "dv", "dw", "db"):
        assert delta_bwd(lib, **{name: None}) == L.WKV_EINVAL, name
    for name in ("go", "dr", "dk", "dv", "ds_in", "ds_out", "ck"):
        assert delta_bwd(lib, **{name: X + 8}) == L.WKV_EALIGN, name
    for name in ("dw", "db"):
        assert delta_bwd(lib, **{name: X + 2}) == L.WKV_EALIGN, name
    for ck, flags in ((X, 1), (None, 0)):
        need = lib.wkv_delta_backward_workspace_bytes(1, 20, 4, 2, 64, flags | 2)
        assert delta_bwd(lib, ck=ck, nws=need - 1) == L.WKV_EWORKSPACE
        assert delta_bwd(lib, ck=ck, ws=None, nws=need) == L.WKV_EWORKSPACE
        assert delta_bwd(lib, ck=ck, ws=X + 64, nws=need) == L.WKV_EWORKSPACE
    assert delta_bwd(lib, B=0, w=None, ws=None) == L.WKV_OK


def test_delta_sizes(lib):
    one = 2 * 100 * 4 * 64 * 4 + 2 * 4 * 2 * 64 * 64 * 4  # errors, and the states before two tiles
    assert lib.wkv_delta_ckpt_bytes(2, 100, 4, 64) == one
    assert lib.wkv_delta_backward_workspace_bytes(2, 100, 4, 2, 64, 1 | 2) == one
    assert lib.wkv_delta_backward_workspace_bytes(2, 100, 4, 2, 64, 2) == 2 * one
    assert lib.wkv_delta_ckpt_bytes(2, 0, 4, 64) == 0 == lib.wkv_delta_ckpt_bytes(2, 100, 4, 65)
    for T in (1, 64, 256):  # too short to split
        assert lib.wkv_delta_forward_workspace_bytes(1, T, 4, 4, 64) == 0
    assert lib.wkv_delta_forward_workspace_bytes(64, 1024, 64, 64, 64) == 0  # enough pairs without
    assert lib.wkv_delta_forward_workspace_bytes(-1, 8192, 4, 4, 64) == 0
    split = lib.wkv_delta_forward_workspace_bytes(1, 8192, 4, 2, 64)
    assert split % (4 * 3 * 64 * 64 * 4) == 0  # three states a segment and pair
    assert (lib.wkv_delta_backward_workspace_bytes(1, 8192, 4, 2, 64, 1)
            == lib.wkv_delta_backward_workspace_bytes(1, 8192, 4, 2, 64, 3) + split)


def head(lib, bwd, rows=3, H=2, G=64, yd=L.WKV_F32, dt=L.WKV_BF16, flags=0, act=2, eps=1e-5, y=X, weight=X, bias=X, gate=X, out=X,
         gout=X, dy=X, dweight=X, dbias=X, dgate=X, ws=X, nws=1 << 30):
    eps = ctypes.c_float(eps)
    if not bwd:
        return lib.wkv_head_norm(rows, H, G, yd, dt, flags, act, eps, y, weight, bias, gate, out, None)
    return lib.wkv_head_norm_backward(rows, H, G, yd, dt, flags, act, eps, y, weight, bias, gate, gout, dy, dweight, dbias, dgate,
                                      ws, nws, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_head_norm_refusals(lib, bwd):
    for bad in (dict(rows=-1), dict(H=-1), dict(G=0), dict(G=1025), dict(flags=4), dict(act=3), dict(act=-1), dict(eps=-1e-3),
                dict(eps=NAN), dict(eps=INF), dict(y=None), dict(weight=None)):
        assert head(lib, bwd, **bad) == L.WKV_EINVAL, bad
    for bad in (dict(yd=L.WKV_BF16, dt=L.WKV_F32), dict(yd=5), dict(dt=-1)):
        assert head(lib, bwd, **bad) == L.WKV_EDTYPE, bad
    for bad in (dict(rows=1 << 31, H=1), dict(rows=1 << 40, H=1 << 30), dict(H=1 << 26, G=1024),
                dict(rows=0, H=1 << 58)):
        assert head(lib, bwd, **bad) == L.WKV_ESIZE, bad
    for bad in (dict(y=X + 2), dict(weight=X + 1), dict(bias=X + 2), dict(gate=X + 1)):
        assert head(lib, bwd, **bad) == L.WKV_EALIGN, bad
    if not bwd:
        assert head(lib, bwd, out=None) == L.WKV_EINVAL and head(lib, bwd, out=X + 1) == L.WKV_EALIGN
        assert head(lib, bwd, rows=0, y=None, weight=None, out=None) == L.WKV_OK
        return
    for name in ("gout", "dy", "dweight", "dbias", "dgate"):
        assert head(lib, bwd, **{name: None}) == L.WKV_EINVAL, name
    for name in ("dy", "dweight", "dbias"):
        assert head(lib, bwd, **{name: X + 2}) == L.WKV_EALIGN, name
    need = lib.wkv_head_norm_backward_workspace_bytes(3, 2, 64)
    assert need > 0
    for bad in (dict(nws=need - 1), dict(ws=None), dict(ws=X + 128)):
        assert head(lib, bwd, **bad) == L.WKV_EWORKSPACE, bad


def block(lib, bwd, rows=3, C=64, xd=L.WKV_F32, dt=L.WKV_BF16, flags=0, act=1, eps=1e-5, x=X, y=X, gate=X, post_w=X, post_b=X,
          scale=X, pre_w=X, pre_b=X, x_out=X, h=X, gx=X, gh=X, dx=X, dy=X, dgate=X, dpost_w=X, dpost_b=X, dscale=X, dpre_w=X,
          dpre_b=X, ws=X, nws=1 << 30):
    eps = ctypes.c_float(eps)
    if not bwd:
        return lib.wkv_block_norm(rows, C, xd, dt, flags, act, eps, x, y, gate, post_w, post_b, scale, pre_w, pre_b, x_out, h, None)
    return lib.wkv_block_norm_backward(rows, C, xd, dt, flags, act, eps, x, y, gate, post_w, post_b, scale, pre_w, pre_b, gx, gh,
                                       dx, dy, dgate, dpost_w, dpost_b, dscale, dpre_w, dpre_b, ws, nws, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_block_norm_refusals(lib, bwd):
    for bad in (dict(rows=-1), dict(C=-1), dict(C=8193), dict(flags=2), dict(act=7), dict(eps=NAN), dict(x=None), dict(y=None),
                dict(pre_w=None), dict(post_w=None)):  # post_b without post_w
        assert block(lib, bwd, **bad) == L.WKV_EINVAL, bad
    for bad in (dict(xd=L.WKV_BF16, dt=L.WKV_F32), dict(xd=9)):
        assert block(lib, bwd, **bad) == L.WKV_EDTYPE, bad
    assert block(lib, bwd, rows=1 << 31) == L.WKV_ESIZE
    for bad in (dict(x=X + 2), dict(y=X + 1), dict(gate=X + 1), dict(post_w=X + 2), dict(pre_b=X + 1), dict(scale=X + 3)):
        assert block(lib, bwd, **bad) == L.WKV_EALIGN, bad
    assert block(lib, bwd, C=0, x=None, y=None, pre_w=None, post_w=None, post_b=None, dpre_w=None) == L.WKV_OK
    if not bwd:
        assert block(lib, bwd, x_out=None) == L.WKV_EINVAL and block(lib, bwd, h=None) == L.WKV_EINVAL
        return
    for name in ("gh", "dx", "dy", "dgate", "dpost_w", "dpost_b", "dscale", "dpre_w", "dpre_b"):
        assert block(lib, bwd, **{name: None}) == L.WKV_EINVAL, name
    need = lib.wkv_block_norm_backward_workspace_bytes(3, 64)
    for bad in (dict(nws=need - 1), dict(ws=None), dict(ws=X + 4)):
        assert block(lib, bwd, **bad) == L.WKV_EWORKSPACE, bad


def test_binding_refuses_host_tensors():
    z = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(ValueError, match="GPU tensor"):
        O.delta_forward(z(1, 2, 1), z(1, 2, 1), z(1, 2, 64), z(1, 2, 64), z(1, 2, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        O.head_norm(z(2, 64), z(64), heads=1)
    with pytest.raises(ValueError, match="GPU tensor"):
        O.block_norm(z(2, 64), z(2, 64), z(64))
    with pytest.raises(TypeError):
        O.head_norm([1.0], z(64), heads=1)
