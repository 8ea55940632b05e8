"""CPU-side checks that what the delta-rule and norm calls say of their sizes is what they take: a call whose sizes
pass is told by the error of the missing output that is looked at next, so nothing is launched."""
import pytest

from rwkv_wkv_mixing_amd import _lib as L
from rwkv_wkv_mixing_amd import ops as O

from test_delta_norm_abi import X, delta_bwd, delta_fwd, head, lib  # noqa: F401  (lib is a fixture)

STATE, ROW = 64 * 64 * 4, 64 * 4


@pytest.mark.parametrize("B,T,H,HK", [(53, 257, 64000, 1000), (1, 1 << 24, 64, 1), (4, 17, 64, 1), (3, 64, 5, 5)])
def test_ckpt_bytes_of_calls_that_are_taken(lib, B, T, H, HK):  # noqa: F811
    """The errors and the states before every 64 tokens, also where many value heads share few key heads."""
    assert delta_fwd(lib, B=B, T=T, H=H, HK=HK, ck=X, o=None) == L.WKV_EINVAL  # the sizes pass, the output is missing
    assert delta_bwd(lib, B=B, T=T, H=H, HK=HK, dr=None) == L.WKV_EINVAL
    want = B * T * H * ROW + B * H * -(-T // 64) * STATE
    assert lib.wkv_delta_ckpt_bytes(B, T, H, 64) == want == O.delta_ckpt_bytes(B, T, H, 64)
    assert lib.wkv_delta_backward_workspace_bytes(B, T, H, HK, 64, 1 | 2) == want


@pytest.mark.parametrize("B,T,H,N", [(1, 64, 1, 96), (1 << 22, 64, 1, 64), (1, 1 << 31, 1, 64), (-1, 64, 1, 64)])
def test_ckpt_of_no_call_is_refused(lib, B, T, H, N):  # noqa: F811
    assert lib.wkv_delta_ckpt_bytes(B, T, H, N) == 0
    with pytest.raises(ValueError, match="no ckpt"):
        O.new_delta_ckpt(B, T, H, N, "cpu")


def test_ckpt_of_no_tokens(lib):  # noqa: F811
    for B, T, H in ((0, 64, 2), (2, 0, 2), (2, 64, 0)):
        assert O.delta_ckpt_bytes(B, T, H, 64) == 0 and O.new_delta_ckpt(B, T, H, 64, "cpu").numel() == 1


@pytest.mark.parametrize("N,most", [(64, (1 << 25) - 1), (128, (1 << 25) - 2)])
def test_most_pairs_of_a_few_tokens(lib, N, most):  # noqa: F811
    """A wave per 64 columns of a pair, four waves a workgroup: one pair more would be a grid of 2^32 threads."""
    for T in (1, 16):
        assert delta_fwd(lib, B=most, H=1, HK=1, T=T, N=N, o=None) == L.WKV_EINVAL  # the sizes pass
        assert delta_fwd(lib, B=most + 1, H=1, HK=1, T=T, N=N, o=None) == L.WKV_ESIZE
    assert (most * N // 64 + 3) // 4 * 256 < 1 << 32


def test_gradients_of_key_heads_without_value_heads(lib):  # noqa: F811
    """dr and dk are outputs of a call without value heads too."""
    for name in ("dr", "dk"):
        assert delta_bwd(lib, H=0, HK=2, **{name: None}) == L.WKV_EINVAL, name
        assert delta_bwd(lib, H=0, HK=2, **{name: X + 8}) == L.WKV_EALIGN, name
    assert delta_bwd(lib, H=0, HK=0, dr=None, dk=None) == L.WKV_OK
    assert delta_bwd(lib, H=0, HK=2, T=0, dr=None, dk=None) == L.WKV_OK


def test_most_tiles_of_a_walk(lib):  # noqa: F811
    """With a ckpt, and backward: fewer than 2^24 (64 tokens, row, key head) places; without one, more."""
    most = ((1 << 24) - 1) * 64
    assert delta_fwd(lib, T=most, H=1, HK=1, ck=X, o=None) == delta_bwd(lib, T=most, H=1, HK=1, dr=None) == L.WKV_EINVAL
    assert delta_fwd(lib, T=most + 1, H=1, HK=1, ck=X, o=None) == delta_bwd(lib, T=most + 1, H=1, HK=1, dr=None) == L.WKV_ESIZE
    assert delta_fwd(lib, T=most + 1, H=1, HK=1, o=None) == L.WKV_EINVAL


@pytest.mark.parametrize("G", [1, 3, 5, 64, 1000, 1024])
def test_most_channels_of_a_head_norm(lib, G):  # noqa: F811
    """H G below 2^24: the largest H that the header allows passes, the next does not."""
    most = ((1 << 24) - 1) // G
    for bwd in (False, True):
        assert head(lib, bwd, rows=1, H=most, G=G, y=None) == L.WKV_EINVAL  # the sizes pass
        assert head(lib, bwd, rows=1, H=most + 1, G=G, y=None) == L.WKV_ESIZE
