"""The short causal convolution, the selective scan, and gradient clipping, in float64: from their definitions, token by
token.  With ``mag`` every factor is taken by its size and every difference as a sum, which gives the summed sizes of
the terms that each result is made of: what rounding errors are measured against.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, links or calls this module; only ``tests/`` may.  It
shares no code with the HIP path.  Every function is pinned (tests/test_oracle_select_pins.py).
"""
import numpy as np

F8 = np.float64


def _sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def _act(act, v, mag=False):
    """The activation's value and derivative (mag: the sizes of silu's two terms of it, p and v p (1 - p), which cancel
    near v = -1.28)."""
    if act == "none":
        return v, np.ones_like(v)
    p = _sigmoid(v)
    return (p, p * (1 - p)) if act == "sigmoid" else (v * p, p * (1 + (np.abs(v) if mag else v) * (1 - p)))


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def conv_ref(x, weight, bias=None, act="silu", lengths=None, state_in=None, gout=None, gstate=None, mag=False):
    """out [B, T, C] and the carried inputs after each row; with gout the gradients too:
    dict(out, state, dx, dweight, dbias, dstate)."""
    x, weight = np.asarray(x, F8), np.asarray(weight, F8)
    B, T, C = x.shape
    K = weight.shape[0]
    a = np.abs if mag else (lambda v: v)
    bias = np.zeros(C) if bias is None else np.asarray(bias, F8)
    s0 = np.zeros((B, K - 1, C)) if state_in is None else np.asarray(state_in, F8)
    r = dict(out=np.zeros((B, T, C)), state=np.zeros((B, K - 1, C)), dx=np.zeros((B, T, C)), dweight=np.zeros((K, C)),
             dbias=np.zeros(C), dstate=np.zeros((B, K - 1, C)))
    pres = np.zeros((B, T, C))  # sizes of the sums, for bounds on what their errors do to the activation
    for b, n in enumerate(_lengths(lengths, B, T)):
        X = np.concatenate([s0[b], x[b, :n]])
        r["state"][b] = X[n:]
        dX = np.zeros_like(X)
        if gstate is not None:
            dX[n:] += a(np.asarray(gstate, F8)[b])
        for t in range(n):
            pre = bias + (weight * X[t:t + K]).sum(0)
            val, slope = _act(act, pre, mag)
            pres[b, t] = np.abs(bias) + np.abs(weight * X[t:t + K]).sum(0)
            r["out"][b, t] = a(val)
            if gout is not None:
                g = a(np.asarray(gout, F8)[b, t] * slope)
                dX[t:t + K] += a(weight) * g
                r["dweight"] += g * a(X[t:t + K])
                r["dbias"] += g
        r["dstate"][b], r["dx"][b, :n] = dX[:K - 1], dX[K - 1:]
    r["pre"] = pres
    return r


def select_ref(x, dt, w, b, c, d=None, z=None, dt_bias=None, softplus=True, lengths=None, state_in=None, go=None,
               gstate=None, mag=False):
    """out [B, T, C] and the state after each row; with go the gradients too: dict(out, state, dx, ddt, dw, db, dc, dd,
    dz, ddt_bias, dstate)."""
    f = lambda v: np.asarray(v, F8)  # noqa: E731
    a = np.abs if mag else (lambda v: v)
    minus = 1.0 if mag else -1.0
    x, dt, w = f(x), f(dt), f(w)
    B, T, C = x.shape
    N = w.shape[1]
    G = b.shape[2] // N
    b, c = f(b).reshape(B, T, G, N), f(c).reshape(B, T, G, N)
    wide = lambda v: np.repeat(v, C // G, axis=-2)  # noqa: E731  [.., G, N] -> [.., C, N]
    dd = np.zeros(C) if d is None else f(d)
    raw = dt + (0.0 if dt_bias is None else f(dt_bias))
    delta = np.logaddexp(0.0, raw) if softplus else raw
    slope = _sigmoid(raw) if softplus else np.ones_like(raw)
    gate, dgate = (np.ones_like(x), np.zeros_like(x)) if z is None else _act("silu", f(z), mag)
    live = np.arange(T)[None] < np.asarray(_lengths(lengths, B, T))[:, None]  # [B, T]
    h = np.zeros((B, C, N)) if state_in is None else a(f(state_in))
    hs, y = [h], np.zeros((B, T, C))
    zero3 = lambda v, t: np.where(live[:, t, None, None], v, 0.0)  # noqa: E731
    for t in range(T):
        new = np.exp(-delta[:, t, :, None] * w) * h + a((delta * x)[:, t, :, None]) * a(wide(b[:, t]))
        h = np.where(live[:, t, None, None], new, h)
        hs.append(h)
        y[:, t] = zero3(a(wide(c[:, t])) * h, t).sum(-1) + np.where(live[:, t, None], a(dd * x[:, t]), 0.0)
    only = lambda v: np.where(live[..., None], v, 0.0)  # noqa: E731
    r = dict(out=only(y * a(gate)), state=h)
    if go is None:
        return r
    go = f(go)
    gy = only(a(go * gate))
    r["dz"] = only(a(go * dgate) * y)
    g = np.zeros((B, C, N)) if gstate is None else a(f(gstate))
    dx, ddelta = np.zeros((B, T, C)), np.zeros((B, T, C))
    db, dc, dw = np.zeros((B, T, G, N)), np.zeros((B, T, G, N)), np.zeros((C, N))
    group = lambda v: v.reshape(B, G, C // G, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        gt = g + a(wide(c[:, t])) * gy[:, t, :, None]
        dc[:, t] = group(gy[:, t, :, None] * hs[t + 1])
        db[:, t] = group(zero3(gt * a((delta * x)[:, t, :, None]), t))
        du = zero3(gt * a(wide(b[:, t])), t).sum(-1)
        back = np.exp(-delta[:, t, :, None] * w) * gt
        q = zero3(back * hs[t], t)
        dw += minus * (q * a(delta[:, t, :, None])).sum(0)
        ddelta[:, t] = a(x[:, t]) * du + minus * (q * a(w)).sum(-1)
        dx[:, t] = a(delta[:, t]) * du + a(dd) * gy[:, t]
        g = np.where(live[:, t, None, None], back, g)
    ddt = only(ddelta * a(slope))
    r.update(dx=only(dx), ddt=ddt, dw=dw, db=db.reshape(B, T, G * N), dc=dc.reshape(B, T, G * N),
             dd=(gy * a(x)).sum((0, 1)) if not mag else (gy * only(np.abs(x))).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dstate=g)
    return r


def clip_ref(grads, max_norm, eps=1e-6):
    """The norm, and the gradients scaled."""
    grads = [np.asarray(g, F8) for g in grads]
    norm = float(np.sqrt(sum(float((g * g).sum()) for g in grads)))
    f = 1.0 if norm + eps <= max_norm else max_norm / (norm + eps)
    return norm, [g * f for g in grads]
