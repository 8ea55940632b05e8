"""CPU-side checks of the short convolution, the selective scan and the clipping of gradients: sizes, and every refusal,
all decided on the host before any HIP call (so these run without a GPU)."""
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
    assert re.search(rf"#define WKV_SELECT_SOFTPLUS {L.WKV_SELECT_SOFTPLUS}\b", src)


def conv(lib, bwd, B=2, T=20, C=8, K=4, dt=L.WKV_BF16, act=2, ln=None, x=X, weight=X, bias=X, s_in=None, out=X + 4096, s_out=None,
         gout=X, ds_out=None, dx=X + 4096, dweight=X, dbias=X, ds_in=None, ws=X, nws=1 << 30):
    if not bwd:
        return lib.wkv_conv_forward(B, T, C, K, dt, act, ln, x, weight, bias, s_in, out, s_out, None)
    return lib.wkv_conv_backward(B, T, C, K, dt, act, ln, x, weight, bias, s_in, gout, ds_out, dx, dweight, dbias, ds_in, ws, nws,
                                 None)


@pytest.mark.parametrize("bwd", [False, True])
def test_conv_refusals(lib, bwd):
    for bad in (dict(B=-1), dict(T=-1), dict(C=-1), dict(K=1), dict(K=5), dict(act=3), dict(act=-1), dict(x=None), dict(weight=None)):
        assert conv(lib, bwd, **bad) == L.WKV_EINVAL, bad
    assert conv(lib, bwd, dt=2) == L.WKV_EDTYPE
    for bad in (dict(B=1 << 31), dict(T=(1 << 31) - 64), dict(C=1 << 26), dict(B=1 << 30, T=1 << 30), dict(B=1 << 30, T=1 << 10, C=1)):
        assert conv(lib, bwd, **bad) == L.WKV_ESIZE, bad
    for bad in (dict(x=X + 1), dict(weight=X + 2), dict(bias=X + 1), dict(s_in=X + 1), dict(ln=X + 2)):
        assert conv(lib, bwd, **bad) == L.WKV_EALIGN, bad
    assert conv(lib, bwd, C=0, x=None, weight=None, out=None, bias=None, dweight=None) == L.WKV_OK
    if not bwd:
        assert conv(lib, bwd, out=None) == L.WKV_EINVAL
        assert conv(lib, bwd, out=X + 1) == L.WKV_EALIGN and conv(lib, bwd, s_out=X + 1) == L.WKV_EALIGN
        assert conv(lib, bwd, B=0, x=None, weight=None, out=None) == L.WKV_OK
        whole, carried = 2 * 20 * 8 * 2, 2 * 3 * 8 * 2  # bytes of x, and of the carried inputs
        for off in (0, 2, whole - 2, -whole + 2):
            assert conv(lib, bwd, out=X + off) == L.WKV_EINVAL, off
        for off in (0, whole - 2, -carried + 2):
            assert conv(lib, bwd, s_out=X + off) == L.WKV_EINVAL, off
            assert conv(lib, bwd, s_out=X + 4096 + off) == L.WKV_EINVAL and conv(lib, bwd, s_in=X + 4096 + off) == L.WKV_EINVAL, off
        for off in (2, carried - 2, -2):
            assert conv(lib, bwd, s_in=X + 8192, s_out=X + 8192 + off) == L.WKV_EINVAL, off
        return
    for name in ("gout", "dx", "dweight", "dbias"):
        assert conv(lib, bwd, **{name: None}) == L.WKV_EINVAL, name
    for name in ("gout", "dx", "ds_out", "ds_in"):
        assert conv(lib, bwd, **{name: X + 1}) == L.WKV_EALIGN, name
    for name in ("dweight", "dbias"):
        assert conv(lib, bwd, **{name: X + 2}) == L.WKV_EALIGN, name
    span = 2 * 3 * 8 * 2  # bytes of the carried inputs
    for off in (0, 2, span - 2, -span + 2):
        assert conv(lib, bwd, ds_out=X, ds_in=X + off, nws=0) == L.WKV_EINVAL, off
    assert conv(lib, bwd, ds_out=X, ds_in=X + span, nws=0) == L.WKV_EWORKSPACE  # (next to each other: the next check)
    whole = 2 * 20 * 8 * 2
    for off in (0, 2, whole - 2, -whole + 2):
        assert conv(lib, bwd, dx=X + off, gout=X + 8192, nws=0) == L.WKV_EINVAL, off
        assert conv(lib, bwd, dx=X + 8192 + off, gout=X + 8192, nws=0) == L.WKV_EINVAL, off
    need = lib.wkv_conv_backward_workspace_bytes(2, 20, 8, 4)
    assert need > 0 and need % (5 * 8 * 4) == 0
    for bad in (dict(nws=need - 1), dict(ws=None), dict(ws=X + 128)):
        assert conv(lib, bwd, **bad) == L.WKV_EWORKSPACE, bad


def test_conv_sizes(lib):
    for bad in ((-1, 5, 5, 4), (1, 5, 5, 1), (1, 5, 5, 9), (0, 5, 5, 4), (1, 0, 5, 4), (1 << 31, 5, 5, 4)):
        assert lib.wkv_conv_backward_workspace_bytes(*bad) == 0, bad


def select(lib, bwd, B=2, T=20, C=128, G=2, N=16, dt=L.WKV_BF16, flags=1, ln=None, x=X, dlt=X, w=X, b=X, c=X, d=X, z=X, bias=X, out=X,
           s_in=None, s_out=None, ck=None, ws=None, nws=0, go=X, ds_out=None, dx=X, ddt=X, dw=X, db=X, dc=X, dd=X, dz=X, dbias=X,
           ds_in=None):
    if not bwd:
        return lib.wkv_select_forward(B, T, C, G, N, dt, flags, ln, x, dlt, w, b, c, d, z, bias, out, s_in, s_out, ck, ws, nws, None)
    return lib.wkv_select_backward(B, T, C, G, N, dt, flags, ln, x, dlt, w, b, c, d, z, bias, go, s_in, ds_out, dx, ddt, dw, db, dc, dd,
                                   dz, dbias, ds_in, ck, ws, nws, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_select_refusals(lib, bwd):
    kw = dict(ws=X, nws=1 << 40) if bwd else {}
    for bad in (dict(B=-1), dict(T=-1), dict(C=-2), dict(G=0), dict(G=-1), dict(G=3), dict(N=4), dict(N=64), dict(N=12), dict(flags=2)):
        assert select(lib, bwd, **{**kw, **bad}) == L.WKV_EINVAL, bad
    assert select(lib, bwd, **kw, dt=5) == L.WKV_EDTYPE
    for bad in (dict(B=1 << 31), dict(T=(1 << 31) - 64), dict(C=1 << 26), dict(C=1 << 21, G=1 << 21), dict(B=1 << 21),
                dict(B=1 << 30, T=1 << 30, C=2)):
        assert select(lib, bwd, **{**kw, **bad}) == L.WKV_ESIZE, bad
    for name in ("x", "dlt", "w", "b", "c"):
        assert select(lib, bwd, **{**kw, name: None}) == L.WKV_EINVAL, name
    for name in ("w", "b", "c", "s_in", "ck"):
        assert select(lib, bwd, **{**kw, name: X + 8}) == L.WKV_EALIGN, name
    for name in ("x", "dlt", "z"):
        assert select(lib, bwd, **{**kw, name: X + 1}) == L.WKV_EALIGN, name
    for name in ("d", "bias", "ln"):
        assert select(lib, bwd, **{**kw, name: X + 2}) == L.WKV_EALIGN, name
    assert select(lib, bwd, B=0, G=1, x=None, w=None, out=None, dw=X, d=None, bias=None, C=0) == L.WKV_OK


def test_select_forward_refusals(lib):
    assert select(lib, False, out=None) == L.WKV_EINVAL and select(lib, False, out=X + 1) == L.WKV_EALIGN
    assert select(lib, False, s_out=X + 4) == L.WKV_EALIGN
    need = lib.wkv_select_forward_workspace_bytes(1, 8192, 128, 1, 16)
    assert need > 0
    for bad in (dict(ws=X, nws=need - 1), dict(ws=X + 16, nws=need)):
        assert select(lib, False, B=1, T=8192, G=1, **bad) == L.WKV_EWORKSPACE, bad
    assert select(lib, False, B=1 << 27, T=8, C=4, G=1, N=16, x=None) == L.WKV_ESIZE  # a few tokens: 2^33 numbers of state
    assert select(lib, False, B=1 << 26, T=8, C=4, G=1, N=16, x=None) == L.WKV_EINVAL  # one fewer bit passes the size check
    assert select(lib, False, B=1 << 22, T=9, C=4, G=1, N=16, x=None) == L.WKV_ESIZE  # more tokens: a tile of channels a row
    assert select(lib, False, B=1 << 22, T=8, C=4, G=1, N=16, ck=X, x=None) == L.WKV_ESIZE
    assert select(lib, False, B=0, x=None, w=None, out=None) == L.WKV_OK
    assert select(lib, False, T=0, x=None, w=None, out=None) == L.WKV_OK


def test_select_backward_refusals(lib):
    kw = dict(ws=X, nws=1 << 40)
    for name in ("go", "dx", "ddt", "dw", "db", "dc", "dd", "dz", "dbias"):
        assert select(lib, True, **{**kw, name: None}) == L.WKV_EINVAL, name
    for name in ("go", "dx", "ddt", "db", "dc", "dz"):
        assert select(lib, True, **{**kw, name: X + 1}) == L.WKV_EALIGN, name
    for name in ("dw", "ds_out", "ds_in"):
        assert select(lib, True, **{**kw, name: X + 8}) == L.WKV_EALIGN, name
    for name in ("dd", "dbias"):
        assert select(lib, True, **{**kw, name: X + 2}) == L.WKV_EALIGN, name
    assert select(lib, True, **kw, B=1 << 11, T=1 << 15, C=128, G=1) == L.WKV_ESIZE  # B T G N = 2^30
    for ck, flags in ((X, 1), (None, 0)):
        need = lib.wkv_select_backward_workspace_bytes(2, 20, 128, 2, 16, flags | 2)
        assert need > 0
        for bad in (dict(nws=need - 1, ws=X), dict(nws=need, ws=None), dict(nws=need, ws=X + 64)):
            assert select(lib, True, ck=ck, **bad) == L.WKV_EWORKSPACE, bad


def test_select_sizes(lib):
    assert lib.wkv_select_ckpt_bytes(2, 17, 5, 16) == 2 * 2 * 5 * 16 * 4
    for bad in ((2, 17, 5, 64), (-1, 17, 5, 16), (2, 0, 5, 16), (1 << 31, 17, 5, 16)):
        assert lib.wkv_select_ckpt_bytes(*bad) == 0, bad
    assert lib.wkv_select_forward_workspace_bytes(16, 4096, 4096, 1, 16) == 0  # enough channel tiles without a split
    assert lib.wkv_select_forward_workspace_bytes(1, 40, 64, 1, 16) == 0  # too short for one
    for B, T, C, G, N in ((1, 8192, 128, 2, 16), (2, 333, 1002, 2, 8), (1, 32768, 4096, 1, 16)):
        have = lib.wkv_select_backward_workspace_bytes(B, T, C, G, N, 1 | 2)
        again = lib.wkv_select_backward_workspace_bytes(B, T, C, G, N, 2)
        assert again - have == -(-lib.wkv_select_ckpt_bytes(B, T, C, N) // 256) * 256
        assert lib.wkv_select_backward_workspace_bytes(B, T, C, G, N, 1) > have


def clip(lib, n=2, grads=(X, X + 4096), sizes=(64, 64), types=(L.WKV_F32, L.WKV_BF16), outs=None, max_norm=1.0, eps=1e-6, norm=X + 65536,
         ws=X, nws=1 << 20, only_norm=False):
    arr = lambda t, v: None if v is None else (t * len(v))(*v)  # noqa: E731
    g, s, d = arr(ctypes.c_void_p, grads), arr(ctypes.c_int64, sizes), arr(ctypes.c_int, types)
    if only_norm:
        return lib.wkv_grad_norm(n, g, s, d, norm, ws, nws, None)
    return lib.wkv_clip_gradients(n, g, arr(ctypes.c_void_p, outs), s, d, max_norm, eps, norm, ws, nws, None)


@pytest.mark.parametrize("only_norm", [True, False])
def test_clip_refusals(lib, only_norm):
    kw = dict(only_norm=only_norm)
    for bad in (dict(n=-1), dict(grads=None), dict(sizes=None), dict(types=None), dict(sizes=(64, -1)), dict(grads=(X, None))):
        assert clip(lib, **kw, **bad) == L.WKV_EINVAL, bad
    assert clip(lib, **kw, types=(0, 2)) == L.WKV_EDTYPE
    assert clip(lib, **kw, n=1 << 24, grads=None) == L.WKV_ESIZE and clip(lib, **kw, sizes=(64, 1 << 51)) == L.WKV_ESIZE
    for bad in (dict(grads=(X + 2, X + 4096)), dict(grads=(X, X + 4097)), dict(norm=X + 65538)):
        assert clip(lib, **kw, **bad) == L.WKV_EALIGN, bad
    need = lib.wkv_clip_workspace_bytes(2)
    for bad in (dict(ws=None), dict(ws=X + 8), dict(nws=need - 1)):
        assert clip(lib, **kw, **bad) == L.WKV_EWORKSPACE, bad
    if only_norm:
        assert clip(lib, **kw, norm=None) == L.WKV_EINVAL
        return
    for bad in (dict(max_norm=-1.0), dict(max_norm=NAN), dict(max_norm=INF), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF),
                dict(outs=(X, None)), dict(grads=(X, X), types=(0, 0)), dict(grads=(X, X + 255), types=(0, 1), outs=(X + 8192, X + 8448 - 2)),
                dict(outs=(X + 8192, X + 8192)), dict(outs=(X + 4096, X + 12288)), dict(outs=(X, X + 128)), dict(norm=X + 4),
                dict(outs=(X + 8, X + 4096))):
        want = L.WKV_EALIGN if bad.get("grads") == (X, X + 255) else L.WKV_EINVAL
        assert clip(lib, **bad) == want, bad
    assert clip(lib, outs=(X + 8193, X + 12288)) == L.WKV_EALIGN


def test_clip_sizes(lib):
    assert lib.wkv_clip_workspace_bytes(0) == 0 == lib.wkv_clip_workspace_bytes(-1) == lib.wkv_clip_workspace_bytes(1 << 24)
    assert lib.wkv_clip_workspace_bytes(1) == lib.wkv_clip_workspace_bytes(96) < lib.wkv_clip_workspace_bytes(97)


def test_binding_refuses_host_tensors():
    z = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(ValueError, match="GPU tensor"):
        O.conv_forward(z(1, 2, 4), z(4, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        O.conv_backward(z(1, 2, 4), z(1, 2, 4), z(4, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        O.select_forward(z(1, 2, 4), z(1, 2, 4), z(4, 16), z(1, 2, 16), z(1, 2, 16))
    with pytest.raises(ValueError, match="GPU tensor"):
        O.grad_norm([z(3)])
    with pytest.raises(ValueError, match="empty"):
        O.clip_gradients([], 1.0)
    with pytest.raises(TypeError):
        O.clip_gradients([1.0], 1.0)
    with pytest.raises(ValueError, match="no ckpt"):
        O.new_select_ckpt(1, 20, 5, 12, "cpu")
