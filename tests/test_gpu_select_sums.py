"""The selective scan's sums over many tokens and many rows (dw, dd, the bias's gradient), of terms that are all alike: what a
float32 sum rounds off is then alike too and adds up, up to 2^-25 of the sum with every term.

Bounds as in the parity tests of the scan, without the part that grows with the number of terms: a term is within
2 (3 n + C + 128)u of its size (u = 2^-24), n the tokens that carry it.  Here a step is log 2 or more and a rate 1 or more, so
what is older than 50 tokens has decayed to 2^-50: n = min(T, 50).  Eight tiles of 16 tokens are added in float32 (128u), these,
waves and rows in float64, with a rounding to float32 between rows and two at the ends (3u)."""
import functools

import numpy as np
import pytest
import torch

from oracle.select_ref import select_ref
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DTYPES, IDS = [BF, F32], ["bf16", "f32"]
SUMS = ("dw", "dd", "ddt_bias")


def draw(T, C, N, dtype, seed):
    """One row whose tokens are all alike."""
    g = torch.Generator().manual_seed(seed)
    token = lambda *s: (0.5 + torch.rand(s, generator=g)).to(dtype).expand(1, T, *s).contiguous()  # noqa: E731
    p = dict(x=token(C), dt=token(C), b=token(N), c=token(N), z=token(C), go=token(C))
    p.update(w=1.0 + torch.rand(C, N, generator=g), d=0.5 + torch.rand(C, generator=g), dt_bias=0.5 * torch.rand(C, generator=g))
    return p


@functools.lru_cache(maxsize=None)
def draw_with_sums(T, C, N, dtype, seed):
    """... and the oracle's results and their sizes."""
    p = draw(T, C, N, dtype, seed)
    h = {k: v.double().numpy() for k, v in p.items()}
    kw = dict(d=h["d"], z=h["z"], dt_bias=h["dt_bias"], go=h["go"])
    return p, *(select_ref(*(h[k] for k in ("x", "dt", "w", "b", "c")), mag=k, **kw) for k in (False, True))


def check(T, C, B, g, r, m):
    u = (2 * (3 * min(T, 50) + C + 128) + 131) * 2.0 ** -24
    worst = {n: float((np.abs(g[n].double().cpu().numpy() / B - r[n]) / (u * m[n] + 1e-30)).max()) for n in SUMS}
    assert all(v <= 1.0 for v in worst.values()), worst


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,C,N", [(1, 20, 16), (3, 5, 32), (17, 66, 8)])
@pytest.mark.parametrize("B", [3, 1023, 70001])
def test_many_rows(B, T, C, N, dtype):
    p, r, m = draw_with_sums(T, C, N, dtype, T)
    q = {k: (v.expand(B, *v.shape[1:]).contiguous() if v.dim() == 3 else v).to(DEV) for k, v in p.items()}
    g = O.select_backward(*(q[k] for k in ("x", "dt", "w", "b", "c")), q["go"], d=q["d"], z=q["z"], dt_bias=q["dt_bias"])
    check(T, C, B, g, r, m)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("N", [8, 16, 32])
def test_many_tokens(N, split, dtype):
    p, r, m = draw_with_sums(20000, 6, N, dtype, N)
    q = {k: v.to(DEV) for k, v in p.items()}
    g = O.select_backward(*(q[k] for k in ("x", "dt", "w", "b", "c")), q["go"], d=q["d"], z=q["z"], dt_bias=q["dt_bias"], split=split)
    check(20000, 6, 1, g, r, m)
