"""Float64 CPU oracle for the norms around the mixing.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, links or calls
this module; only ``tests/`` may.  It shares no code with the HIP path.

norm(y) = (y - m) / sqrt(mean((y - m)^2) + eps) over the last axis, m the mean (center) or 0.
    head norm:   out = act(gate) (norm(y) weight + bias), per head
    block norm:  z = act(gate) (norm(y) post_w + post_b), x_out = x + scale z, h = norm(x_out) pre_w + pre_b
The forwards return float64 arrays; the backwards dicts of gradients and, under the same names, of
magnitudes: the same sums with every term's absolute value, which bound what rounding can do to them.

Parity status: every function here is pinned (tests/test_oracle_norm_pins.py).
"""
from __future__ import annotations

import numpy as np

__all__ = ["head_norm_ref", "head_norm_backward_ref", "block_norm_ref", "block_norm_backward_ref"]


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def _act(act, g):
    if g is None:
        return 1.0, 0.0
    if act == "none":
        return g, np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-g))
    return (s, s * (1 - s)) if act == "sigmoid" else (g * s, s * (1 + g * (1 - s)))


def _stats(y, center, eps):
    """norm(y), 1 / its divisor, and the magnitude (|y| + |m|) / divisor."""
    m = y.mean(-1, keepdims=True) if center else np.zeros(y.shape[:-1] + (1,))
    inv = 1.0 / np.sqrt(((y - m) ** 2).mean(-1, keepdims=True) + eps)
    return (y - m) * inv, inv, (np.abs(y) + np.abs(m)) * inv


def _pull(d, md, yh, myh, inv, center):
    """The gradient through norm from that of its output, and its magnitude."""
    s1 = d.mean(-1, keepdims=True) if center else 0.0
    g = inv * (d - s1 - yh * (d * yh).mean(-1, keepdims=True))
    return g, inv * (md + (md.mean(-1, keepdims=True) if center else 0.0) + myh * (md * myh).mean(-1, keepdims=True))


def head_norm_ref(y, weight, bias, gate, heads, act="silu", center=False, eps=1e-5):
    """(out [rows, C], its magnitude)."""
    y, weight, bias, gate = map(_f, (y, weight, bias, gate))
    rows, C = y.shape
    G = C // heads
    yh, _, myh = _stats(y.reshape(rows, heads, G), center, eps)
    w, b = weight.reshape(-1, G), 0.0 if bias is None else bias.reshape(-1, G)
    a, _ = _act(act, None if gate is None else gate.reshape(rows, heads, G))
    return ((yh * w + b) * a).reshape(rows, C), ((myh * np.abs(w) + np.abs(b)) * np.abs(a)).reshape(rows, C)


def head_norm_backward_ref(y, gout, weight, bias, gate, heads, act="silu", center=False, eps=1e-5):
    y, gout, weight, bias, gate = map(_f, (y, gout, weight, bias, gate))
    rows, C = y.shape
    G = C // heads
    split = lambda x: x.reshape(rows, heads, G)  # noqa: E731
    yh, inv, myh = _stats(split(y), center, eps)
    w, b = weight.reshape(-1, G), 0.0 if bias is None else bias.reshape(-1, G)
    a, da = _act(act, None if gate is None else split(gate))
    go = split(gout)
    dz = go * a
    over = (0,) if w.shape[0] == heads else (0, 1)
    dy, mdy = _pull(dz * w, np.abs(dz * w), yh, myh, inv, center)
    g = dict(dy=dy.reshape(rows, C), dweight=(dz * yh).sum(over).reshape(-1))
    m = dict(dy=mdy.reshape(rows, C), dweight=(np.abs(dz) * myh).sum(over).reshape(-1))
    if bias is not None:
        g["dbias"], m["dbias"] = dz.sum(over).reshape(-1), np.abs(dz).sum(over).reshape(-1)
    if gate is not None:
        g["dgate"] = (go * (yh * w + b) * da).reshape(rows, C)
        # the derivative of silu cancels where it crosses zero: 1 + |g| bounds its terms
        m["dgate"] = (np.abs(go) * (myh * np.abs(w) + np.abs(b)) * (1 + np.abs(split(gate)))).reshape(rows, C)
    return g, m


def _inner(y, gate, post_w, post_b, act, center, eps):
    a, da = _act(act, gate)
    if post_w is None:
        return y, np.abs(y), y, np.abs(y), 1.0, a, da
    yh, iy, myh = _stats(y, center, eps)
    b = 0.0 if post_b is None else post_b
    return yh * post_w + b, myh * np.abs(post_w) + np.abs(b), yh, myh, iy, a, da


def block_norm_ref(x, y, pre_w, pre_b=None, gate=None, act="sigmoid", post_w=None, post_b=None, scale=None, center=True,
                   eps=1e-5):
    """((x_out, h), (their magnitudes))."""
    x, y, pre_w, pre_b, gate, post_w, post_b, scale = map(_f, (x, y, pre_w, pre_b, gate, post_w, post_b, scale))
    z, mz, _, _, _, a, _ = _inner(y, gate, post_w, post_b, act, center, eps)
    s = 1.0 if scale is None else scale
    x_out, mx = x + s * a * z, np.abs(x) + np.abs(s * a) * mz
    xh, inv, _ = _stats(x_out, center, eps)
    b = 0.0 if pre_b is None else pre_b
    rms = np.sqrt((mx ** 2).mean(-1, keepdims=True))  # the statistics' own error reaches every channel
    return (x_out, xh * pre_w + b), (mx, (mx + rms * (1 + np.abs(xh))) * inv * np.abs(pre_w) + np.abs(b))


def block_norm_backward_ref(x_out, y, gh, pre_w, pre_b=None, gx=None, gate=None, act="sigmoid", post_w=None, post_b=None,
                            scale=None, center=True, eps=1e-5):
    x_out, y, gh, pre_w, pre_b, gx, gate, post_w, post_b, scale = map(
        _f, (x_out, y, gh, pre_w, pre_b, gx, gate, post_w, post_b, scale))
    xh, ix, mxh = _stats(x_out, center, eps)
    d = gh * pre_w
    dx, mdx = _pull(d, np.abs(d), xh, mxh, ix, center)
    if gx is not None:
        dx, mdx = dx + gx, mdx + np.abs(gx)
    z, mz, yh, myh, iy, a, da = _inner(y, gate, post_w, post_b, act, center, eps)
    s = 1.0 if scale is None else scale
    ds, mds = dx * s, mdx * np.abs(s)
    dz, mdz = ds * a, mds * np.abs(a)
    if post_w is None:
        dy, mdy = dz, mdz
    else:
        dy, mdy = _pull(dz * post_w, mdz * np.abs(post_w), yh, myh, iy, center)
    g = dict(dx=dx, dy=dy, dpre_w=(gh * xh).sum(0))
    m = dict(dx=mdx, dy=mdy, dpre_w=(np.abs(gh) * mxh).sum(0))
    if pre_b is not None:
        g["dpre_b"], m["dpre_b"] = gh.sum(0), np.abs(gh).sum(0)
    if post_w is not None:
        g["dpost_w"], m["dpost_w"] = (dz * yh).sum(0), (mdz * myh).sum(0)
    if post_b is not None:
        g["dpost_b"], m["dpost_b"] = dz.sum(0), mdz.sum(0)
    if scale is not None:
        g["dscale"], m["dscale"] = (dx * z * a).sum(0), (mdx * mz * np.abs(a)).sum(0)
    if gate is not None:
        g["dgate"], m["dgate"] = ds * z * da, mds * mz * (1 + np.abs(gate))
    return g, m
