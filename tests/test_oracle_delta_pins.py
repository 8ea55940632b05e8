"""Pins of the gated delta rule's float64 oracle: closed forms, invariants, an
independent matrix form, differences and autograd."""
import numpy as np
import pytest
import torch

from oracle import delta_backward_ref, delta_forward_ref


def problem(B=2, T=7, H=4, HK=2, N=8, seed=0, state=True):
    g = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    r = unit(g.standard_normal((B, T, HK, N))).reshape(B, T, HK * N)
    k = unit(g.standard_normal((B, T, HK, N))).reshape(B, T, HK * N)
    v = g.standard_normal((B, T, H * N))
    w, beta = g.uniform(0, 0.5, (B, T, H)), g.uniform(0, 1, (B, T, H))
    S0 = g.standard_normal((B, H, N, N)) if state else None
    return w, beta, r, k, v, HK, S0


def test_beta_zero_only_decays():
    w, beta, r, k, v, HK, S0 = problem()
    o, S = delta_forward_ref(w, 0 * beta, r, k, v, HK, S0)
    assert np.allclose(S, np.exp(-w.sum(1))[..., None, None] * S0, rtol=1e-13)


def test_beta_one_stores_the_value():
    """With a unit key and beta = 1 the state answers the key it has just been given with its value."""
    w, beta, r, k, v, HK, S0 = problem()
    o, _ = delta_forward_ref(w, 0 * beta + 1, k, k, v, HK, S0)
    assert np.allclose(o, v, rtol=0, atol=1e-12)


def test_infinite_rate_clears_the_state():
    w, beta, r, k, v, HK, S0 = problem()
    w[:, 3] = np.inf
    o, S = delta_forward_ref(w, beta, r, k, v, HK, S0)
    w2 = w[:, 3:].copy()
    w2[:, 0] = 0
    o2, S2 = delta_forward_ref(w2, beta[:, 3:], r[:, 3:], k[:, 3:], v[:, 3:], HK, None)
    assert np.allclose(o[:, 3:], o2, atol=1e-13) and np.allclose(S, S2, atol=1e-13)


def test_matrix_form():
    """S_t = e^{-w} (I - beta k^T k) S_{t-1} + beta k^T v, by explicit matrices."""
    w, beta, r, k, v, HK, S0 = problem(B=1, H=1, HK=1)
    N = S0.shape[-1]
    S = S0[0, 0]
    for t in range(w.shape[1]):
        kt = k[0, t][:, None]
        S = np.exp(-w[0, t, 0]) * (np.eye(N) - beta[0, t, 0] * kt @ kt.T) @ S + beta[0, t, 0] * kt @ v[0, t][None]
    assert np.allclose(S, delta_forward_ref(w, beta, r, k, v, HK, S0)[1][0, 0], rtol=1e-12)


def test_lengths_end_a_row():
    w, beta, r, k, v, HK, S0 = problem()
    o, S = delta_forward_ref(w, beta, r, k, v, HK, S0, lengths=[3, 0])
    o3, S3 = delta_forward_ref(*(x[:1, :3] for x in (w, beta, r, k, v)), HK, S0[:1])
    assert np.allclose(o[0, :3], o3[0]) and (o[0, 3:] == 0).all() and np.allclose(S[0], S3[0])
    assert (o[1] == 0).all() and (S[1] == S0[1]).all()


@pytest.mark.parametrize("lengths", [None, [5, 0]])
def test_backward_against_differences(lengths):
    w, beta, r, k, v, HK, S0 = problem(T=5, N=4)
    g = np.random.default_rng(1)
    go, dS = g.standard_normal(v.shape), g.standard_normal(S0.shape)
    loss = lambda a: (lambda o, S: (o * go).sum() + (S * dS).sum())(  # noqa: E731
        *delta_forward_ref(*a[:5], HK, a[5], lengths=lengths))
    args = [w, beta, r, k, v, S0]
    dr, dk, dv, dw, db, ds = delta_backward_ref(w, beta, r, k, v, go, HK, S0, dS, lengths)
    for n, (i, d) in dict(w=(0, dw), beta=(1, db), r=(2, dr), k=(3, dk), v=(4, dv), S0=(5, ds)).items():
        for _ in range(12):
            at = tuple(g.integers(0, s) for s in args[i].shape)
            h = 1e-6
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[i][at] += h
            lo[i][at] -= h
            # central differences: error h^2 |f'''| / 6 + 2^-52 |L| / h, both below 1e-8 here
            assert abs((loss(hi) - loss(lo)) / (2 * h) - d[at]) < 1e-7, (n, at)


def test_backward_against_autograd():
    w, beta, r, k, v, HK, S0 = problem(B=1, T=6, H=2, HK=1, N=4)
    leaf = [torch.tensor(x, requires_grad=True) for x in (w, beta, r, k, v, S0)]
    W, Bt, R, K, V, S = leaf
    o = []
    for t in range(6):
        kt = K[:, t].view(1, 1, 4).repeat_interleave(2, 1)
        rt = R[:, t].view(1, 1, 4).repeat_interleave(2, 1)
        D = torch.exp(-W[:, t])[..., None, None] * S
        e = V[:, t].view(1, 2, 4) - (kt[..., None] * D).sum(-2)
        S = D + kt[..., None] * (Bt[:, t][..., None] * e)[:, :, None]
        o.append((rt[..., None] * S).sum(-2).reshape(1, 8))
    go = torch.arange(48, dtype=torch.float64).reshape(1, 6, 8).sin()
    (torch.stack(o, 1) * go).sum().backward()
    got = delta_backward_ref(w, beta, r, k, v, go.numpy(), HK, S0)
    for d, x in zip(got, (R, K, V, W, Bt, leaf[5])):
        assert np.allclose(d, x.grad.numpy(), rtol=1e-11, atol=1e-12)
