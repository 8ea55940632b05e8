"""The selective scan with N = 16 in calls of more than 256 workgroups, which share out the states among waves otherwise than
smaller ones: outputs, states and every gradient against the float64 oracle, with the bounds of the parity tests."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O
from test_gpu_select import check_all, draw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DTYPES, IDS = [BF, F32], ["bf16", "f32"]


def workgroups(B, T, C, G):
    """Tiles of 64 channels times rows times segments (from the size of what the segments keep, 17 numbers a channel)."""
    split = O.L.lib().wkv_select_forward_workspace_bytes(B, T, C, G, 16)
    return B * G * -(-(C // G) // 64) * max(1, round(split / (B * C * 17 * 4)))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,T,C,G,lengths,options", [
    (5, 40, 3300, 1, None, ("d", "z", "dt_bias")), (5, 37, 3300, 3, [37, 0, 16, 5, 33], ("d", "z", "dt_bias")), (260, 9, 7, 1, None, ("z",)),
    (5, 18, 3300, 1, None, ()), (9, 1, 2000, 1, None, ("d", "z", "dt_bias"))], ids=["whole", "ragged", "narrow", "plain", "token"])
def test_many_workgroups(B, T, C, G, lengths, options, dtype):
    assert workgroups(B, T, C, G) > 256
    check_all(draw(B, T, C, G, 16, dtype), lengths=lengths, options=options)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,T,C,lengths", [(2, 333, 2100, [333, 201]), (1, 500, 3300, None)], ids=["ragged", "one"])
@pytest.mark.parametrize("saved", [True, False], ids=["ckpt", "recomputed"])
def test_many_workgroups_of_segments(B, T, C, lengths, saved, dtype):
    tiles = B * -(-C // 64)
    assert workgroups(B, T, C, 1) > 256 > tiles
    check_all(draw(B, T, C, 1, 16, dtype), lengths=lengths, saved=saved)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_the_rows_of_a_large_call_are_those_of_small_ones(dtype):
    """Some rows of a large call by themselves, where other waves hold the states: states are the same bits (a state takes the
    same multiply-adds), outputs and gradients as near as float32 sums in another grouping (1e-5 of the largest)."""
    B, T, C = 6, 50, 3300
    p = {k: v.to("cuda:0") for k, v in draw(B, T, C, 1, 16, dtype).items()}
    names = ("x", "dt", "w", "b", "c")

    def run(q, rows):
        cut = lambda n: q[n][rows].contiguous() if q[n].dim() == 3 else q[n]  # noqa: E731
        kw = dict(d=q["d"], z=cut("z"), dt_bias=q["dt_bias"], state_in=cut("state_in"), split=False)
        out, S = O.select_forward(*(cut(n) for n in names), return_state=True, **kw)
        g = O.select_backward(*(cut(n) for n in names), cut("go"), grad_state_out=cut("gstate"), need_state_grad=True, **kw)
        return out, S, g

    out, S, g = run(p, slice(0, B))
    for b in (0, B - 1):
        o1, S1, g1 = run(p, slice(b, b + 1))
        assert torch.equal(S[b], S1[0])
        for got, want in [(out[b], o1[0])] + [(g[n][b], g1[n][0]) for n in ("dx", "ddt", "dz", "db", "dc", "dstate_in")]:
            tol = 2.0 ** -7 if got.dtype is BF else 1e-5
            assert float((got.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max())
