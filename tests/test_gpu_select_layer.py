"""A layer of the short convolution and the selective scan as a model has it (projections by torch, float32): its output and
every gradient against float64 autograd of the definitions on the CPU, the gradients clipped together, and decoding token
by token after a prompt.

Bound: every stage sums at most 200 float32 terms (u = 2^-24 each, errors of either sign), eight stages deep forward and
backward: the error of the norm is below 8 x 200 u = 2^-13.3 of the norm; 2^-13 is asked for."""
import numpy as np
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, E, R, N, K = 24, 68, 4, 16, 4  # model width, inner width, rank of the steps, states, taps


def parameters():
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(w_in=rn(D, 2 * E) / D ** 0.5, conv=rn(K, E) / 2, conv_b=0.1 * rn(E), w_x=rn(E, R + 2 * N) / E ** 0.5, w_dt=rn(R, E) / R ** 0.5,
                dt_bias=rn(E) - 3.0, w=torch.log(torch.arange(1, N + 1).float()).repeat(E, 1) + 0.1 * rn(E, N), d=1.0 + 0.1 * rn(E),
                w_out=rn(E, D) / E ** 0.5)


def layer(u, p, conv_state=None, state=None, lengths=None):
    """With the framework's calls: the output and the states for what comes next."""
    xz = u @ p["w_in"]
    x, z = xz[..., :E].contiguous(), xz[..., E:].contiguous()
    x, conv_state = O.short_conv(x, p["conv"], p["conv_b"], state_in=conv_state, lengths=lengths)
    proj = x @ p["w_x"]
    dt = proj[..., :R] @ p["w_dt"]
    b, c = proj[..., R:R + N].contiguous(), proj[..., R + N:].contiguous()
    y, state = O.selective_scan(x, dt, p["w"].exp(), b, c, p["d"], z, p["dt_bias"], state_in=state, lengths=lengths)
    return y @ p["w_out"], conv_state, state


def reference(u, p, lengths):
    """The same from the definitions, row by row and token by token."""
    silu = torch.nn.functional.silu
    rows = []
    for r, n in enumerate(lengths):
        xz = u[r, :n] @ p["w_in"]
        x, z = xz[:, :E], xz[:, E:]
        x = torch.cat([x.new_zeros(K - 1, E), x])
        x = silu(p["conv_b"] + sum(p["conv"][j] * x[j:j + n] for j in range(K)))
        proj = x @ p["w_x"]
        delta = torch.nn.functional.softplus(proj[:, :R] @ p["w_dt"] + p["dt_bias"], threshold=1e9)
        h, y = x.new_zeros(E, N), []
        for t in range(n):
            h = torch.exp(-delta[t, :, None] * p["w"].exp()) * h + (delta[t] * x[t])[:, None] * proj[t, R:R + N]
            y.append(h @ proj[t, R + N:])
        y = (torch.stack(y) + p["d"] * x) * silu(z) if n else x
        rows.append(torch.cat([y @ p["w_out"], y.new_zeros(u.shape[1] - n, D)]))
    return torch.stack(rows)


def near(a, b, tol=2.0 ** -13):
    a, b = a.detach().double().cpu(), b.detach().double()
    assert a.shape == b.shape and float((a - b).norm()) <= tol * float(b.norm()), float((a - b).norm() / b.norm())


@pytest.mark.parametrize("T,lengths", [(37, [37, 37]), (150, [150, 61]), (21, [21, 1])])
def test_training_step(T, lengths):
    g = torch.Generator().manual_seed(T)
    u, go = torch.randn(2, T, D, generator=g), torch.randn(2, T, D, generator=g)
    p64 = {k: v.double().requires_grad_() for k, v in parameters().items()}
    u64 = u.double().requires_grad_()
    y64 = reference(u64, p64, lengths)
    y64.backward(go.double())
    p = {k: v.to(DEV).requires_grad_() for k, v in parameters().items()}
    ud = u.to(DEV).requires_grad_()
    ln = None if lengths == [T, T] else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    y, _, _ = layer(ud, p, lengths=ln)
    y.backward(go.to(DEV))
    near(y, y64)
    near(ud.grad, u64.grad)
    for k in p:
        near(p[k].grad, p64[k].grad)
    grads = [v.grad for v in p.values()]
    total = float(sum(v.grad.square().sum() for v in p64.values()).sqrt())
    norm = O.clip_gradients(grads, total / 3)
    assert abs(float(norm) - total) <= 2.0 ** -13 * total
    for k in p:
        near(p[k].grad, p64[k].grad / 3)


def test_decoding_after_a_prompt():
    p = {k: v.to(DEV) for k, v in parameters().items()}
    u = torch.randn(3, 30, D, device=DEV)
    with torch.no_grad():
        whole, conv_end, end = layer(u, p)
        y, conv_state, state = layer(u[:, :17].contiguous(), p)
        near(y, whole[:, :17].cpu())
        for t in range(17, 30):
            y, conv_state, state = layer(u[:, t:t + 1].contiguous(), p, conv_state, state)
            near(y[:, 0], whole[:, t].cpu())
        near(state, end.cpu())
        near(conv_state, conv_end.cpu())


def test_gradients_are_differences():
    """Along one direction of every input, from the framework's own forward (float32 differences: 1e-2)."""
    p = {k: v.to(DEV) for k, v in parameters().items()}
    u, go = torch.randn(2, 20, D, device=DEV), torch.randn(2, 20, D, device=DEV)
    for k in p:
        q = {n: v.clone().requires_grad_(n == k) for n, v in p.items()}
        (layer(u, q)[0] * go).sum().backward()
        g = q[k].grad
        step = 1e-2 * g / g.norm()
        with torch.no_grad():
            up, down = ((layer(u, {**p, k: p[k] + s * step})[0].double() * go).sum() for s in (1, -1))
        assert abs(float((up - down) / 2e-2) - float(g.norm())) <= 1e-2 * float(g.norm()) + 1e-3 * float(go.norm()), k


def test_refused_derivatives():
    p = {k: v.to(DEV) for k, v in parameters().items()}
    x = torch.randn(1, 9, E, device=DEV, requires_grad=True)
    out, _ = O.short_conv(x, p["conv"], p["conv_b"])
    (gx,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    b = torch.randn(1, 9, N, device=DEV)
    out, _ = O.selective_scan(x, x.detach(), p["w"].exp(), b, b)
    (gx,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x))
        with pytest.raises((RuntimeError, NotImplementedError)):
            O.selective_scan(dual, x.detach(), p["w"].exp(), b, b)
        with pytest.raises((RuntimeError, NotImplementedError)):
            O.short_conv(dual, p["conv"], p["conv_b"])


def test_states_alone_and_outputs_alone():
    """A loss of the carried states only, and of the outputs only."""
    p = {k: v.to(DEV) for k, v in parameters().items()}
    x = torch.randn(2, 20, E, device=DEV, requires_grad=True)
    b = torch.randn(2, 20, N, device=DEV)
    s = torch.randn(2, E, N, device=DEV, requires_grad=True)
    out, end = O.selective_scan(x, x.detach(), p["w"].exp(), b, b, state_in=s)
    gx, gs = torch.autograd.grad(end.sum(), (x, s), retain_graph=True)
    want = O.select_backward(x.detach(), x.detach(), p["w"].exp(), b, b, torch.zeros_like(x), state_in=s.detach(),
                             grad_state_out=torch.ones_like(s), need_state_grad=True)
    assert torch.equal(gx, want["dx"]) and torch.equal(gs, want["dstate_in"])
    (gx,) = torch.autograd.grad(out.sum(), x)
    want = O.select_backward(x.detach(), x.detach(), p["w"].exp(), b, b, torch.ones_like(x), state_in=s.detach())
    assert torch.equal(gx, want["dx"])
    c0 = torch.randn(2, K - 1, E, device=DEV, requires_grad=True)
    _, c1 = O.short_conv(x, p["conv"], state_in=c0)
    gx, gc = torch.autograd.grad(c1.sum(), (x, c0))
    assert not bool(gc.any()) and torch.equal(gx[:, -3:], torch.ones_like(gx[:, -3:])) and not bool(gx[:, :-3].any())
    assert np.isfinite(float(gx.sum()))
