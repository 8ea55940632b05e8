"""Pins of the norms' float64 oracle: torch's own norms and activations, and autograd."""
import itertools

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import block_norm_backward_ref, block_norm_ref, head_norm_backward_ref, head_norm_ref

ACTS = dict(none=lambda g: g, sigmoid=torch.sigmoid, silu=F.silu)


def norm(x, center, eps):
    return F.layer_norm(x, x.shape[-1:], eps=eps) if center else F.rms_norm(x, x.shape[-1:], eps=eps)


def draws(*shapes):
    g = torch.Generator().manual_seed(sum(map(sum, shapes)))
    return [torch.randn(s, generator=g, dtype=torch.float64) for s in shapes]


@pytest.mark.parametrize("act,center,shared,bias,gated",
                         itertools.product(ACTS, (False, True), (False, True), (False, True), (False, True)))
def test_head_norm(act, center, shared, bias, gated):
    R, H, G = 5, 3, 7
    y, gout, gate = draws((R, H * G), (R, H * G), (R, H * G))
    w, b = draws((G if shared else H * G,), (G if shared else H * G,))
    leaves = [t.clone().requires_grad_() for t in (y, w, b, gate)]
    z = norm(leaves[0].view(R, H, G), center, 1e-3) * leaves[1].view(-1, G)
    z = z + leaves[2].view(-1, G) if bias else z
    out = z.reshape(R, H * G)
    out = out * ACTS[act](leaves[3]) if gated else out
    (out * gout).sum().backward()
    args = (w, b if bias else None, gate if gated else None, H, act, center, 1e-3)
    got, mag = head_norm_ref(y, *args)
    assert np.allclose(got, out.detach(), rtol=1e-12, atol=1e-13) and (np.abs(got) <= mag * (1 + 1e-12)).all()
    g, m = head_norm_backward_ref(y, gout, *args)
    want = dict(dy=leaves[0].grad, dweight=leaves[1].grad, dbias=leaves[2].grad, dgate=leaves[3].grad)
    for n, t in want.items():
        assert (t is None) == (n not in g), n
        if t is not None:
            assert np.allclose(g[n], t, rtol=1e-11, atol=1e-12), n
            assert (np.abs(g[n]) <= m[n] * (1 + 1e-9) + 1e-12).all(), n


@pytest.mark.parametrize("act,center,post,bias,scaled,gated",
                         itertools.product(ACTS, (False, True), (False, True), (False, True), (False, True), (False, True)))
def test_block_norm(act, center, post, bias, scaled, gated):
    R, C = 4, 9
    x, y, gate, gx, gh = draws(*[(R, C)] * 5)
    names = ["x", "y", "pre_w", "pre_b", "gate", "post_w", "post_b", "scale"]
    vals = [x, y] + draws((C,)) + draws((C,)) + [gate] + draws((C,), (C,), (C,))
    L = {n: t.clone().requires_grad_() for n, t in zip(names, vals)}
    z = L["y"]
    if post:
        z = norm(z, center, 1e-3) * L["post_w"]
        z = z + L["post_b"] if bias else z
    z = z * ACTS[act](L["gate"]) if gated else z
    xo = L["x"] + (L["scale"] * z if scaled else z)
    h = norm(xo, center, 1e-3) * L["pre_w"]
    h = h + L["pre_b"] if bias else h
    ((xo * gx).sum() + (h * gh).sum()).backward()
    kw = dict(gate=gate if gated else None, act=act, post_w=vals[5] if post else None,
              post_b=vals[6] if post and bias else None, scale=vals[7] if scaled else None, center=center, eps=1e-3)
    pb = vals[3] if bias else None
    (gxo, ghh), mags = block_norm_ref(x, y, vals[2], pb, **kw)
    assert np.allclose(gxo, xo.detach(), rtol=1e-12) and np.allclose(ghh, h.detach(), rtol=1e-11, atol=1e-12)
    g, m = block_norm_backward_ref(gxo, y, gh, vals[2], pb, gx=gx, **kw)
    for n in names:
        t = L[n].grad
        assert (t is None) == ("d" + n not in g), n
        if t is not None:
            assert np.allclose(g["d" + n], t, rtol=1e-10, atol=1e-11), n
            assert (np.abs(g["d" + n]) <= m["d" + n] * (1 + 1e-9) + 1e-12).all(), n
