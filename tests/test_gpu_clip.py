"""The norm of gradients and their clipping against float64: squares of eight elements are added in float32 (8 roundings of
positive terms, so 8u of the sum, u = 2^-24), the rest in float64; the norm, its root, is within 4u + u of its rounding.  The
factor is rounded once more and so is an element: 8u, and 2^-8 for a bfloat16 element."""
import numpy as np
import pytest
import torch

from oracle.select_ref import clip_ref
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def host(t):
    return t.double().cpu().numpy()


def check(grads, max_norm, eps=1e-6):
    before = [g.clone() for g in grads]
    want_norm, want = clip_ref([host(g) for g in grads], max_norm, eps)
    norm = O.grad_norm(grads)
    assert abs(float(norm.double()) - want_norm) <= 8 * U * want_norm
    out = [torch.full_like(g, float("nan")) for g in grads]
    n2 = O.clip_gradients(grads, max_norm, eps=eps, out=out)
    for a, b in zip(grads, before):
        assert torch.equal(a, b)
    n3 = O.clip_gradients(grads, max_norm, eps=eps)
    assert torch.equal(norm, n2) and torch.equal(norm, n3)
    for g, o, r in zip(grads, out, want):
        assert torch.equal(g, o)
        half = 2.0 ** -8 if g.dtype == BF else 0.0
        least = 2.0 ** -134 if g.dtype == BF else 2.0 ** -149
        assert (np.abs(host(g) - r) <= (half + 10 * U) * np.abs(r) + least).all()


def draw(shapes, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(scale * torch.randn(s, generator=g)).to(t).to(DEV) for s, t in shapes]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
@pytest.mark.parametrize("shapes", [
    [((1,), F32)], [((7,), BF)], [((3, 5), BF), ((0, 4), F32), ((8,), F32), ((), F32)], [((16384,), F32), ((16385,), BF), ((16383,), BF)],
    [((200, 333), BF), ((1000,), F32), ((70000,), F32)]], ids=["one", "seven", "empty", "chunks", "mixed"])
def test_clip(shapes, max_norm):
    check(draw(shapes), max_norm)


def test_many_tensors():
    """More tensors than one launch takes."""
    check(draw([((1 + 7 * i % 50,), BF if i % 3 else F32) for i in range(400)]), 1.0)


def test_off_the_grid():
    """Views that start anywhere, next to others."""
    flat = torch.randn(5000, device=DEV)
    half = torch.randn(5000, device=DEV).to(BF)
    cuts = [0, 1, 10, 1003, 1004, 5000]
    grads = [f[a:b] for f in (flat, half) for a, b in zip(cuts, cuts[1:])]
    check(grads, 1.0)


def test_large_and_small():
    """Squares beyond float32's range, on both sides."""
    check([torch.full((1000,), 1e25, device=DEV), torch.full((77,), 2e19, device=DEV).to(BF)], 1.0)
    check([torch.full((1000,), 1e-30, device=DEV), torch.full((77,), 1e-25, device=DEV).to(BF)], 1e-28, 0.0)
    check([torch.zeros(1000, device=DEV)], 1.0)
    check([torch.zeros(1000, device=DEV)], 0.0, 0.0)


@pytest.mark.parametrize("bad,element", [(float("inf"), 0.0), (float("nan"), float("nan"))])
def test_not_finite(bad, element):
    g = torch.ones(5000, device=DEV)
    g[4321] = bad
    norm = O.clip_gradients([g, torch.ones(3, device=DEV)], 1.0)
    assert not bool(torch.isfinite(norm))
    assert bool(torch.isnan(g[4321]))
    assert bool(torch.isnan(g[0])) if element != element else float(g[0]) == 0.0


def test_one_tensor_and_a_given_norm():
    g = torch.randn(33, device=DEV)
    norm = torch.empty((), device=DEV)
    assert O.grad_norm(g, norm=norm) is norm and abs(float(norm) - float(g.double().norm())) <= 8 * U * float(norm)


def test_refusals():
    g = torch.ones(100, device=DEV)
    for bad in ([g, g], [g[:60], g[50:]]):
        with pytest.raises(RuntimeError, match="invalid"):
            O.clip_gradients(bad, 1.0)
    with pytest.raises(RuntimeError, match="invalid"):
        O.clip_gradients([g[:50], g[50:]], 1.0, out=[g[50:], g[:50]])
    with pytest.raises(RuntimeError, match="invalid"):
        O.clip_gradients([g], 1.0, norm=g[:1].view(()))
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")), dict(max_norm=1.0, eps=-1.0)):
        with pytest.raises(RuntimeError, match="invalid"):
            O.clip_gradients([g], **kw)
    assert bool((g == 1).all())
    assert float(O.grad_norm([g, g])) == pytest.approx(200 ** 0.5)  # nothing is written: a tensor may be there twice
