"""Pins of the oracle of the short convolution, the selective scan and clipping: closed forms, a linear filter, differences."""
import numpy as np
import pytest

from oracle.select_ref import clip_ref, conv_ref, select_ref


def draw(rng, B, T, C, G, N):
    n = rng.standard_normal
    return dict(x=n((B, T, C)), dt=n((B, T, C)) - 1.0, w=rng.uniform(0.1, 3.0, (C, N)), b=n((B, T, G * N)), c=n((B, T, G * N)),
                d=n(C), z=n((B, T, C)), dt_bias=0.3 * n(C), state_in=n((B, C, N)))


def loss(fn, p, go, gstate, **kw):
    r = fn(**p, **kw)
    return float((r["out"] * go).sum() + (r["state"] * gstate).sum())


def differences(fn, p, go, gstate, name, **kw):
    out, base = np.zeros_like(p[name]), p[name]
    for i in np.ndindex(base.shape):
        e = 1e-5
        up, down = base.copy(), base.copy()
        up[i] += e
        down[i] -= e
        out[i] = (loss(fn, {**p, name: up}, go, gstate, **kw) - loss(fn, {**p, name: down}, go, gstate, **kw)) / (2 * e)
    return out


@pytest.mark.parametrize("lengths", [None, [4, 0], [2, 7]], ids=["whole", "empty", "ragged"])
@pytest.mark.parametrize("softplus", [True, False])
def test_select_gradients_are_differences(lengths, softplus):
    rng = np.random.default_rng(3)
    B, T, C, G, N = 2, 5, 4, 2, 8
    p = draw(rng, B, T, C, G, N)
    if not softplus:  # steps are >= 0: with negative ones states grow past what differences of float64 resolve
        p["dt"], p["dt_bias"] = 0.1 + np.abs(p["dt"]), np.abs(p["dt_bias"])
    go, gs = rng.standard_normal((B, T, C)), rng.standard_normal((B, C, N))
    r = select_ref(**p, softplus=softplus, lengths=lengths, go=go, gstate=gs)
    for name, grad in dict(x="dx", dt="ddt", w="dw", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", state_in="dstate").items():
        want = differences(select_ref, p, go, gs, name, softplus=softplus, lengths=lengths)
        np.testing.assert_allclose(r[grad], want, rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("lengths", [None, [1, 0], [6, 3]], ids=["whole", "empty", "ragged"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv_gradients_are_differences(K, act, lengths):
    rng = np.random.default_rng(K)
    B, T, C = 2, 6, 3
    n = rng.standard_normal
    p = dict(x=n((B, T, C)), weight=n((K, C)), bias=n(C), state_in=n((B, K - 1, C)))
    go, gs = n((B, T, C)), n((B, K - 1, C))
    r = conv_ref(**p, act=act, lengths=lengths, gout=go, gstate=gs)
    for name, grad in dict(x="dx", weight="dweight", bias="dbias", state_in="dstate").items():
        want = differences(conv_ref, p, go, gs, name, act=act, lengths=lengths)
        np.testing.assert_allclose(r[grad], want, rtol=1e-6, atol=1e-8, err_msg=name)


def test_conv_is_a_linear_filter():
    from scipy.signal import lfilter

    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((1, 50, 2)), rng.standard_normal((4, 2))
    out = conv_ref(x, w, act="none")["out"]
    for c in range(2):
        np.testing.assert_allclose(out[0, :, c], lfilter(w[::-1, c], [1.0], x[0, :, c]), rtol=1e-12, atol=1e-12)


def test_select_constant_steps_are_a_recursive_filter():
    """Constant steps and b = c = 1: each state is a first-order recursive filter of the input."""
    from scipy.signal import lfilter

    rng = np.random.default_rng(1)
    T, C, N, step = 60, 2, 8, 0.3
    x, w = rng.standard_normal((1, T, C)), rng.uniform(0.1, 2.0, (C, N))
    one = np.ones((1, T, N))
    r = select_ref(x, np.full((1, T, C), step), w, one, one, softplus=False)
    for c in range(C):
        want = sum(lfilter([step], [1.0, -np.exp(-step * w[c, n])], x[0, :, c]) for n in range(N))
        np.testing.assert_allclose(r["out"][0, :, c], want, rtol=1e-11, atol=1e-12)


def test_select_splits_through_its_state():
    rng = np.random.default_rng(2)
    p = draw(rng, 2, 12, 4, 1, 8)
    whole = select_ref(**p)
    seq = ("x", "dt", "b", "c", "z")
    first = select_ref(**{k: (v[:, :5] if k in seq else v) for k, v in p.items()})
    second = select_ref(**{**{k: (v[:, 5:] if k in seq else v) for k, v in p.items()}, "state_in": first["state"]})
    np.testing.assert_allclose(np.concatenate([first["out"], second["out"]], 1), whole["out"], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(second["state"], whole["state"], rtol=1e-12, atol=1e-12)


def test_sizes_of_terms_bound_the_results():
    rng = np.random.default_rng(4)
    p = draw(rng, 2, 9, 4, 2, 8)
    go, gs = rng.standard_normal((2, 9, 4)), rng.standard_normal((2, 4, 8))
    r, m = (select_ref(**p, lengths=[9, 5], go=go, gstate=gs, mag=k) for k in (False, True))
    for name in r:
        assert (np.abs(r[name]) <= m[name] * (1 + 1e-12) + 1e-300).all(), name


def test_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, out = clip_ref(g, 1.0, 0.0)
    assert norm == 5.0 and np.allclose(out[0], [0.6, 0]) and np.allclose(out[1], [[0.8]])
    assert clip_ref(g, 5.0, 0.0)[1][0][0] == 3.0
    assert clip_ref([np.zeros(2)], 0.0, 0.0)[1][0][0] == 0.0
