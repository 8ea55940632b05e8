"""Float64 CPU oracle for the gated delta rule.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, links or calls
this module; only ``tests/`` and ``__graft_entry__.smoke()`` may.  It shares no
code, tables or constants with the HIP path.

Per batch row and value head, from the state S_0 [N, N] (key x value):
    D_t = e^{-w_t} S_{t-1},  e_t = v_t - k_t D_t,  S_t = D_t + beta_t k_t^T e_t,  o_t = r_t S_t
Value head h reads r, k of key head h // (H // HK).  A row of n tokens ends
there: the rest give o = 0 and zero gradients.

Parity status: every function here is pinned (tests/test_oracle_delta_pins.py).
"""
from __future__ import annotations

import numpy as np

__all__ = ["delta_forward_ref", "delta_backward_ref"]


def _heads(x, n, H):
    """[B, T, n N] -> [B, T, H, N], each of the n heads repeated H // n times."""
    x = np.asarray(x, dtype=np.float64)
    B, T, C = x.shape
    return np.repeat(x.reshape(B, T, n, C // n), H // n, axis=2)


def _walk(w, beta, r, k, v, HK, S0, lengths):
    w, beta = np.asarray(w, np.float64), np.asarray(beta, np.float64)
    B, T, H = w.shape
    N = np.asarray(v).shape[2] // H
    r, k, v = _heads(r, HK, H), _heads(k, HK, H), _heads(v, H, H)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, T)
    S = np.zeros((B, H, N, N)) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((B, T, H, N))
    kept = []
    for t in range(T):
        live = (t < n)[:, None, None, None]
        a = np.exp(-w[:, t])[..., None, None]
        D = a * S
        kt, rt, vt, bt = k[:, t], r[:, t], v[:, t], beta[:, t][..., None]
        e = np.where(live[..., 0], vt - np.einsum("bhi,bhij->bhj", kt, D), 0.0)
        S2 = np.where(live, D + kt[..., None] * (bt * e)[..., None, :], S)
        o[:, t] = np.where(live[..., 0], np.einsum("bhi,bhij->bhj", rt, S2), 0.0)
        kept.append((live, a, D, e, S, S2))
        S = S2
    return o.reshape(B, T, H * N), S, kept, (B, T, H, N, r, k, v, beta)


def delta_forward_ref(w, beta, r, k, v, HK, S0=None, lengths=None):
    """(o [B, T, H N], S_T [B, H, N, N])."""
    o, S, _, _ = _walk(w, beta, r, k, v, HK, S0, lengths)
    return o, S


def delta_backward_ref(w, beta, r, k, v, go, HK, S0=None, dS=None, lengths=None, magnitude=False):
    """(dr, dk [B, T, HK N], dv [B, T, H N], dw, dbeta [B, T, H], dS0) of sum <go, o> + <dS, S_T>;
    with ``magnitude`` also |H_t| |D_t| and |e_t| |k_t G_t| [B, T, H], which bound dw and dbeta."""
    _, _, kept, (B, T, H, N, r, k, v, beta) = _walk(w, beta, r, k, v, HK, S0, lengths)
    go = np.asarray(go, np.float64).reshape(B, T, H, N)
    G = np.zeros((B, H, N, N)) if dS is None else np.array(dS, dtype=np.float64)
    dr, dk, dv = (np.zeros((B, T, H, N)) for _ in range(3))
    dw, db, mw, mb = (np.zeros((B, T, H)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        live, a, D, e, _, S2 = kept[t]
        lv = live[..., 0]
        kt, rt, gt, bt = k[:, t], r[:, t], go[:, t], beta[:, t][..., None]
        dr[:, t] = np.where(lv, np.einsum("bhij,bhj->bhi", S2, gt), 0.0)
        G1 = G + rt[..., None] * gt[..., None, :]
        y = np.einsum("bhi,bhij->bhj", kt, G1)
        lam = bt * y
        dv[:, t] = np.where(lv, lam, 0.0)
        db[:, t] = np.where(lv[..., 0], (e * y).sum(-1), 0.0)
        mb[:, t] = np.sqrt((e * e).sum(-1) * (y * y).sum(-1))
        dk[:, t] = np.where(lv, bt * np.einsum("bhij,bhj->bhi", G1, e) - np.einsum("bhij,bhj->bhi", D, lam), 0.0)
        G1 = G1 - kt[..., None] * lam[..., None, :]
        dw[:, t] = np.where(lv[..., 0], -(G1 * D).sum((-1, -2)), 0.0)
        mw[:, t] = np.sqrt((G1 * G1).sum((-1, -2)) * (D * D).sum((-1, -2)))
        G = np.where(live, a * G1, G)
    shared = lambda x: x.reshape(B, T, HK, H // HK, N).sum(3).reshape(B, T, HK * N)  # noqa: E731
    out = (shared(dr), shared(dk), dv.reshape(B, T, H * N), dw, db, G)
    return out + (mw, mb) if magnitude else out
