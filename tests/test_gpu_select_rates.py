"""The selective scan at the ends of its rates and steps: infinite rates, steps that are zero or next to it, rates that are
not a number in calls with rows without tokens.  Outputs, states and every gradient against the float64 oracle.

Bounds as in the parity tests of the scan: u = 2^-24, (3 T + C + 128)u of the sizes of the terms forward, twice that with
B T for T in the gradients, and 2^-8 of a bf16 result on top."""
import numpy as np
import pytest
import torch

from oracle.select_ref import select_ref
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DTYPES, IDS = [BF, F32], ["bf16", "f32"]
ORDER = ("x", "dt", "w", "b", "c")


def draw(B, T, C, N, dtype):
    g = torch.Generator().manual_seed(11 * T + C + N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(x=rn(B, T, C), dt=rn(B, T, C), b=rn(B, T, N), c=rn(B, T, N), z=rn(B, T, C), go=rn(B, T, C))
    p = {k: v.to(dtype) for k, v in p.items()}
    p.update(w=torch.arange(1, N + 1) * torch.exp(0.2 * rn(C, N)), d=rn(C), dt_bias=torch.zeros(C), S=rn(B, C, N), Gs=rn(B, C, N))
    return p


def run(p, split, lengths=None):
    q = {k: v.to(DEV) for k, v in p.items()}
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    args = [q[k] for k in ORDER]
    kw = dict(d=q["d"], z=q["z"], dt_bias=q["dt_bias"], state_in=q["S"], split=split, lengths=ln)
    out, S1 = O.select_forward(*args, return_state=True, **kw)
    g = O.select_backward(*args, q["go"], grad_state_out=q["Gs"], need_state_grad=True, **kw)
    return dict(out=out, state=S1, **{("dstate" if k == "dstate_in" else k): v for k, v in g.items()})


def check(got, h):
    B, T, C = h["x"].shape
    kw = dict(d=h["d"], z=h["z"], dt_bias=h["dt_bias"], state_in=h["S"], go=h["go"], gstate=h["Gs"])
    r, m = (select_ref(*(h[k] for k in ORDER), mag=k, **kw) for k in (False, True))
    for n, t in got.items():
        rel = 2.0 ** -8 if t.dtype is BF else 0.0
        u = 2.0 ** -24 * (3 * T + C + 128 if n in ("out", "state") else 2 * (3 * B * T + C + 128))
        t = t.double().cpu().numpy()
        assert np.isfinite(t).all(), n
        worst = float((np.abs(t - r[n]) / (u * (1 + rel) * m[n] + rel * np.abs(r[n]) + 1e-30)).max())
        assert worst <= 1.0, (n, worst)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,split", [(3, False), (40, False), (700, True)], ids=["steps", "whole", "split"])
@pytest.mark.parametrize("N", [8, 16, 32])
def test_infinite_rates_and_steps_of_zero(N, T, split, dtype):
    """Steps that underflow keep the state whatever the rate, and have no gradient; infinite rates forget it in every other
    step, rates of zero in none; finite rates up to 1e38 in steps of zero are as any other."""
    p = draw(2, T, 70, N, dtype)
    p["dt"][:, ::3] = -200.0
    p["dt"][:, 1::3] = 60.0
    p["w"][:8] = float("inf")
    p["w"][8:16] = 0.0
    p["w"][16:20] = 1e38
    p["w"][20:24, 3] = float("inf")  # some of a channel's states
    h = {k: v.double().numpy() for k, v in p.items()}
    h["w"] = np.minimum(h["w"], 1e300)  # (0 x inf is not a decay)
    h["dt"][:, ::3] = -np.inf  # the step is below float32's smallest number: zero
    check(run(p, split), h)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,split", [(3, False), (40, False), (700, True)], ids=["steps", "whole", "split"])
def test_infinite_rates_forget_in_the_smallest_steps(T, split, dtype):
    """Steps of e^-87 = 1.6e-38, next to the smallest float32: nothing is kept of a state of 1 or of its gradient."""
    p = draw(1, T, 70, 16, dtype)
    p["dt"][:] = -87.0
    p["w"][:, ::2] = float("inf")
    got = run(p, split)
    assert float(got["state"][:, :, ::2].abs().max()) < 1e-30 and float(got["dstate"][:, :, ::2].abs().max()) < 1e-30
    h = {k: v.double().numpy() for k, v in p.items()}
    h["w"] = np.minimum(h["w"], 1e300)
    check(got, h)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,split", [(3, False), (40, False), (700, True)], ids=["steps", "whole", "split"])
def test_a_row_without_tokens_keeps_its_state_whatever_the_rates(T, split, dtype):
    p = draw(2, T, 70, 16, dtype)
    p["w"][66, 3] = float("nan")
    p["w"][5] = float("inf")
    got = run(p, split, lengths=[0, T])
    assert torch.equal(got["state"][0].cpu(), p["S"][0]) and torch.equal(got["dstate"][0].cpu(), p["Gs"][0])
    assert bool(torch.isnan(got["state"][1, 66, 3])) and bool(torch.isnan(got["out"][1, :, 66]).all())
    assert bool(torch.isfinite(got["state"][1, :66]).all())
