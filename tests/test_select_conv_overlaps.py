"""Outputs of the short convolution and the selective scan over tensors that other workgroups may still read: refused on the
host, before any HIP call (so these run without a GPU)."""
import os

import pytest

from rwkv_wkv_mixing_amd import _lib as L

X = 0x100000  # fake addresses, never dereferenced: the calls below are refused on the host


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from rwkv_wkv_mixing_amd.build import build

        build()
    return L.lib()


def places(names):
    """An address of its own for every tensor, far from the others'."""
    return {n: X * (i + 1) for i, n in enumerate(names)}


B, T, C, K = 2, 20, 8, 4
WHOLE, CARRIED = B * T * C * 2, B * (K - 1) * C * 2  # bytes of x, and of the carried inputs


def conv_forward(lib, T=T, **at):
    p = {**places(("x", "weight", "bias", "s_in", "out", "s_out")), **at}
    return lib.wkv_conv_forward(B, T, C, K, L.WKV_BF16, L.WKV_ACT_SILU, None, *(p[n] for n in p), None)


def conv_backward(lib, T=T, **at):
    p = {**places(("x", "weight", "bias", "s_in", "gout", "ds_out", "dx", "dweight", "dbias", "ds_in", "ws")), **at}
    return lib.wkv_conv_backward(B, T, C, K, L.WKV_BF16, L.WKV_ACT_SILU, None, *(p[n] for n in p), 1 << 30, None)


@pytest.mark.parametrize("out,of,bytes_of", [
    ("dx", "x", WHOLE), ("dx", "gout", WHOLE), ("dx", "s_in", CARRIED), ("dx", "ds_out", CARRIED), ("dx", "ds_in", CARRIED),
    ("ds_in", "x", WHOLE), ("ds_in", "gout", WHOLE), ("ds_in", "s_in", CARRIED), ("ds_in", "ds_out", CARRIED)])
def test_conv_gradients_over_what_is_read(lib, out, of, bytes_of):
    base = places(("x", "weight", "bias", "s_in", "gout", "ds_out", "dx", "dweight", "dbias", "ds_in", "ws"))[of]
    own = WHOLE if out == "dx" else CARRIED
    for off in (2, bytes_of - 2, -own + 2) + ((0,) if (out, of) != ("ds_in", "s_in") else ()):
        assert conv_backward(lib, **{out: base + off}) == L.WKV_EINVAL, off


def test_conv_carried_inputs_without_tokens(lib):
    """The copy that a call without tokens is must not run over itself either."""
    for off in (2, CARRIED - 2, -CARRIED + 2):
        assert conv_forward(lib, T=0, s_in=X, s_out=X + off) == L.WKV_EINVAL, off
        assert conv_backward(lib, T=0, ds_out=X, ds_in=X + off) == L.WKV_EINVAL, off
