"""The convolution, the scan and the clipping past 2^31 elements: the ends of large calls against small calls of the same
tokens."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def rand(*shape):
    """bfloat16, drawn in pieces (a generator's float32 of a whole tensor would take twice its size)."""
    t = torch.empty(shape, dtype=BF, device=DEV)
    for piece in t.view(-1).split(1 << 28):
        piece.normal_()
    return t


def test_conv():
    T, C = 530000, 4096
    x, go, w, b = rand(1, T, C), rand(1, T, C), torch.randn(4, C, device=DEV), torch.randn(C, device=DEV)
    assert x.numel() > 1 << 31
    out, state = O.conv_forward(x, w, b, return_state=True)
    tail = O.conv_forward(x[:, -50:].contiguous(), w, b, state_in=x[:, -53:-50].contiguous())
    assert torch.equal(out[:, -50:], tail) and torch.equal(state, x[:, -3:])
    del out
    dx = O.conv_backward(x, go, w, b)[0]
    want = O.conv_backward(x[:, -50:].contiguous(), go[:, -50:].contiguous(), w, b, state_in=x[:, -53:-50].contiguous())[0]
    assert torch.equal(dx[:, -50:], want)


def test_select():
    T, C, N, cut = 131100, 16384, 8, 131000
    x, dt, z, go = (rand(1, T, C) for _ in range(4))
    assert x.numel() > 1 << 31
    b, c = rand(1, T, N), rand(1, T, N)
    w, bias = torch.rand(C, N, device=DEV) + 0.5, torch.randn(C, device=DEV) - 2.0
    kw = dict(z=z, dt_bias=bias)
    out, end = O.select_forward(x, dt, w, b, c, return_state=True, **kw)
    head = [t[:, cut - 2000:cut].contiguous() for t in (x, dt, b, c, z)]
    tail = [t[:, cut:].contiguous() for t in (x, dt, b, c, z)]
    # 2000 tokens before the cut are as good as all: what is older has decayed by e^{-2000 x 0.5 x 0.1} and far more
    _, mid = O.select_forward(head[0], head[1], w, head[2], head[3], z=head[4], dt_bias=bias, return_state=True)
    o2, e2 = O.select_forward(tail[0], tail[1], w, tail[2], tail[3], z=tail[4], dt_bias=bias, state_in=mid, return_state=True)
    near = lambda p, q, tol: float((p.float() - q.float()).abs().max()) <= tol * float(q.float().abs().max())  # noqa: E731
    assert near(out[:, cut:], o2, 2.0 ** -7) and near(end, e2, 1e-5)
    del out, o2
    g = O.select_backward(x, dt, w, b, c, go, **kw)
    g2 = O.select_backward(tail[0], tail[1], w, tail[2], tail[3], go[:, cut:].contiguous(), z=tail[4], dt_bias=bias, state_in=mid)
    for n in ("dx", "ddt", "dz", "db", "dc"):
        assert near(g[n][:, cut:], g2[n], 2.0 ** -7), n
        assert bool(torch.isfinite(g[n][:, :100]).all())
    assert bool(torch.isfinite(g["dw"]).all()) and bool(torch.isfinite(g["ddt_bias"]).all())


def test_decode():
    B, C, N = 2052, 65536, 16
    state = torch.empty(B, C, N, device=DEV)
    assert state.numel() > 1 << 31
    for piece in state.view(-1).split(1 << 28):
        piece.normal_()
    x, dt, b, c = rand(B, 1, C), rand(B, 1, C), rand(B, 1, N), rand(B, 1, N)
    w = torch.rand(C, N, device=DEV)
    last = state[-3:].clone()
    o2, s2 = O.select_forward(x[-3:].contiguous(), dt[-3:].contiguous(), w, b[-3:].contiguous(), c[-3:].contiguous(), state_in=last,
                              return_state=True)
    out = O.select_forward(x, dt, w, b, c, state_in=state, state_out=state)
    assert torch.equal(out[-3:], o2) and torch.equal(state[-3:], s2)


def test_many_rows_of_one_token():
    """More rows than a grid's second dimension."""
    B, C, N = 70001, 16, 8
    x, b = rand(B, 1, C), rand(B, 1, N)
    w, state = torch.rand(C, N, device=DEV), torch.randn(B, C, N, device=DEV)
    out, s1 = O.select_forward(x, x, w, b, b, state_in=state, return_state=True)
    for s in (slice(0, 5), slice(65533, 65540), slice(B - 3, B)):
        o2, s2 = O.select_forward(x[s], x[s], w, b[s], b[s], state_in=state[s], return_state=True)
        assert torch.equal(out[s], o2) and torch.equal(s1[s], s2)


def test_clip():
    n = (1 << 31) + 12345
    g = rand(n)
    small = torch.randn(100, device=DEV)
    want = float(sum(p.float().square().sum(dtype=torch.float64) for p in g.split(1 << 28)) + small.double().square().sum()) ** 0.5
    ends = [g[:100].clone(), g[-100:].clone()]
    norm = O.clip_gradients([g, small], 1.0)
    assert abs(float(norm.double()) - want) <= 8 * 2.0 ** -24 * want
    for a, b in zip(ends, (g[:100], g[-100:])):
        assert float((b.float() - a.float() / (want + 1e-6)).abs().max()) <= 2.0 ** -8 * float(a.float().abs().max()) / want
