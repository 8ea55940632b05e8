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


SB, ST, SC, SG, SN = 2, 20, 128, 2, 16
TOKENS, SHARED, STATES = SB * ST * SC * 2, SB * ST * SG * SN * 2, SB * SC * SN * 4
IN = ("x", "dt", "w", "b", "c", "d", "z", "dt_bias")
SIZE = {**dict.fromkeys(("x", "dt", "z", "go", "out", "dx", "ddt", "dz"), TOKENS), **dict.fromkeys(("b", "c", "db", "dc"), SHARED),
        **dict.fromkeys(("s_in", "s_out", "ds_out", "ds_in"), STATES)}


def select_forward(lib, T=ST, **at):
    p = {**places(IN + ("out", "s_in", "s_out")), **at}
    return lib.wkv_select_forward(SB, T, SC, SG, SN, L.WKV_BF16, 1, None, *(p[n] for n in p), None, None, 0, None)


def select_backward(lib, T=ST, **at):
    p = {**places(IN + ("go", "s_in", "ds_out", "dx", "ddt", "dw", "db", "dc", "dd", "dz", "dt_bias_grad", "ds_in", "ckpt", "ws")), **at}
    return lib.wkv_select_backward(SB, T, SC, SG, SN, L.WKV_BF16, 1, None, *(p[n] for n in p), 1 << 30, None)


def offsets(out, of, same):
    return (16, SIZE[of] - 16, -SIZE[out] + 16) + ((0,) if same else ())


@pytest.mark.parametrize("T", [1, ST])
@pytest.mark.parametrize("out,of", [(o, i) for o in ("out", "s_out") for i in ("x", "dt", "b", "c", "z", "s_in")] + [("s_out", "out")])
def test_select_over_what_is_read(lib, out, of, T):
    base = places(IN + ("out", "s_in", "s_out"))[of]
    if T == 1:  # (a twentieth of the tokens' bytes)
        offs = (0,) if (out, of) != ("s_out", "s_in") else (16,)
    else:
        offs = offsets(out, of, (out, of) != ("s_out", "s_in"))
    for off in offs:
        assert select_forward(lib, T=T, **{out: base + off}) == L.WKV_EINVAL, off


@pytest.mark.parametrize("out", ["dx", "ddt", "dz", "db", "dc", "ds_in"])
@pytest.mark.parametrize("of", ["x", "dt", "b", "c", "z", "go", "ds_out", "dx", "ddt", "dz", "db", "dc"])
def test_select_gradients_over_what_is_read(lib, out, of):
    if out == of:
        return
    base = places(IN + ("go", "s_in", "ds_out", "dx", "ddt", "dw", "db", "dc", "dd", "dz", "dt_bias_grad", "ds_in", "ckpt", "ws"))[of]
    for off in offsets(out, of, (out, of) != ("ds_in", "ds_out")):
        assert select_backward(lib, **{out: base + off}) == L.WKV_EINVAL, off


def test_select_states_without_tokens(lib):
    for off in (16, STATES - 16, -STATES + 16):
        assert select_forward(lib, T=0, s_in=X, s_out=X + off) == L.WKV_EINVAL, off
        assert select_backward(lib, T=0, ds_out=X, ds_in=X + off) == L.WKV_EINVAL, off
