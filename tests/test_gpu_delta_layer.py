"""The delta rule and the norms together, as a layer uses them: a training layer's gradients against the
same formulas in float64, prompts read into states and decoded on, and the calls captured in graphs."""
import numpy as np
import pytest
import torch

from oracle import delta_forward_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def ops():
    from rwkv_wkv_mixing_amd import ops as O

    return O


def layer_inputs(B, T, H, HK, N, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    C = H * N
    p = dict(x=rn(B, T, C), y=rn(B, T, C), pre=1 + 0.1 * rn(C), pre_b=0.1 * rn(C), wr=rn(C, HK * N) / C ** 0.5,
             wk=rn(C, HK * N) / C ** 0.5, wv=rn(C, C) / C ** 0.5, wg=rn(C, C) / C ** 0.5, ww=rn(C, H) / C ** 0.5,
             wb=rn(C, H) / C ** 0.5, hn=1 + 0.1 * rn(C), wo=rn(C, C) / C ** 0.5, scale=0.5 + 0.1 * rn(C), post=1 + 0.1 * rn(C),
             gate=rn(B, T, C), pre2=1 + 0.1 * rn(C))
    return {n: t.float().double() for n, t in p.items()}


def rms(x, eps=1e-5):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def layer(x, y, pre, pre_b, wr, wk, wv, wg, ww, wb, hn, wo, scale, post, gate, pre2, *, B, T, H, HK, N, own):
    """x_out, h after: join -> projections -> unit keys -> delta rule -> gated head norm -> projection -> join."""
    C = H * N
    unit_w = torch.full((N,), N ** -0.5, dtype=x.dtype, device=x.device)
    if own:
        O = ops()
        x1, h = O.block_join(x, y, pre, pre_b, act="none", center=True)
    else:
        x1 = x + y
        h = (x1 - x1.mean(-1, keepdim=True)) / torch.sqrt(x1.var(-1, unbiased=False, keepdim=True) + 1e-5) * pre + pre_b
    r, k, v, g = h @ wr, h @ wk, h @ wv, h @ wg
    w, beta = torch.nn.functional.softplus(h @ ww - 2), torch.sigmoid(h @ wb)
    if own:
        k = O.head_norm_gated(k, unit_w, heads=HK)
        o, _ = O.delta_rule(w, beta, r, k, v)
        o = O.head_norm_gated(o, hn, None, g, heads=H, act="silu")
        return O.block_join(x1, o @ wo, pre2, gate=gate, act="sigmoid", post_w=post, scale=scale, center=False)
    k = (rms(k.view(B, T, HK, N)) * unit_w).repeat_interleave(H // HK, 2)
    r = r.view(B, T, HK, N).repeat_interleave(H // HK, 2)
    S, out = torch.zeros(B, H, N, N, dtype=x.dtype), []
    for t in range(T):
        D = torch.exp(-w[:, t])[..., None, None] * S
        e = v[:, t].view(B, H, N) - (k[:, t, :, :, None] * D).sum(-2)
        S = D + k[:, t, :, :, None] * (beta[:, t][..., None] * e)[:, :, None]
        out.append((r[:, t, :, :, None] * S).sum(-2))
    o = rms(torch.stack(out, 1)).reshape(B, T, C) * hn * torch.nn.functional.silu(g)
    z = rms(o @ wo) * post * torch.sigmoid(gate)
    x2 = x1 + scale * z
    return x2, rms(x2) * pre2


@pytest.mark.parametrize("B,T,H,HK", [(2, 40, 4, 2), (1, 530, 2, 1)])  # the second splits in time
def test_layer_gradients(B, T, H, HK):
    """Every leaf's gradient of a scalar of both outputs, float32 kernels and products against float64.
    Bound: fourteen operators in a row there and back, each adding at most the delta rule's own
    u sqrt((N + 32) T) of the norm (the norms and the products of C terms add less)."""
    N = 64
    p = layer_inputs(B, T, H, HK, N, seed=B + T)
    names = list(p)
    kw = dict(B=B, T=T, H=H, HK=HK, N=N)
    wx, wh = torch.randn(B, T, H * N, dtype=torch.float64), torch.randn(B, T, H * N, dtype=torch.float64)
    grads = {}
    for own in (False, True):
        leaves = [p[n].clone() if not own else p[n].float().to(DEV) for n in names]
        for t in leaves:
            t.requires_grad_()
        x2, h2 = layer(*leaves, own=own, **kw)
        ((x2 * wx.to(x2)).sum() + (h2 * wh.to(h2)).sum()).backward()
        grads[own] = dict(zip(names, (t.grad.double().cpu() for t in leaves)), x2=x2.detach().double().cpu(),
                          h2=h2.detach().double().cpu())
    tol = 28 * U * np.sqrt((N + 32) * T)
    for n, want in grads[False].items():
        err = float((grads[True][n] - want).norm() / want.norm())
        print(f"  {n}: {err:.2e} of {tol:.2e}", flush=True)
        assert err <= tol, n


def test_prefill_then_decode():
    """Ragged prompts read into states, then tokens one and three at a time: each row equals its whole run."""
    O = ops()
    B, T, H, HK, N, lens, more = 3, 90, 4, 2, 64, [90, 33, 64], 7
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    total = T + more
    r, v = rn(B, total, HK * N).bfloat16(), rn(B, total, H * N).bfloat16()
    k = (rn(B, total, HK, N) / 9).reshape(B, total, HK * N).bfloat16()
    w, beta = torch.rand(B, total, H, generator=g) * 0.2, torch.rand(B, total, H, generator=g)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    first = [x[:, :T].contiguous().to(DEV) for x in (w, beta, r, k, v)]
    _, S = O.delta_forward(*first, lengths=ln, return_state=True)
    outs = []
    for t0, n in ((0, 1), (1, 3), (4, 1), (5, 2)):  # the rows' own next tokens
        rows = [torch.stack([x[b, lens[b] + t0:lens[b] + t0 + n] for b in range(B)]).contiguous().to(DEV)
                for x in (w, beta, r, k, v)]
        outs.append(O.delta_forward(*rows, state_in=S, state_out=S))
    got = torch.cat(outs, 1).double().cpu().numpy()
    for b in range(B):
        n = lens[b] + more
        ref, Sref = delta_forward_ref(*(x[b:b + 1, :n].double().numpy() for x in (w, beta, r, k, v)), HK)
        err = np.abs(got[b] - ref[0, lens[b]:])
        eps = U * np.sqrt((N + 32) * n)
        assert (err <= 2.0 ** -8 * np.abs(ref[0, lens[b]:]) + 8 * eps * np.abs(ref).max()).all(), b
        assert np.linalg.norm(S[b].cpu().numpy() - Sref[0]) <= eps * np.linalg.norm(Sref), b


def step_case(seed, T, H, N, dtype):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    C = H * N
    return [t.to(DEV) for t in (torch.rand(2, T, H, generator=g) * 0.3, torch.rand(2, T, H, generator=g), rn(2, T, C).to(dtype),
                                (rn(2, T, C) / N ** 0.5).to(dtype), rn(2, T, C).to(dtype), rn(2, T, C).to(dtype),
                                rn(2, H, N, N), rn(2, T, C).to(dtype))]


@pytest.mark.parametrize("dtype,T,N", [(torch.bfloat16, 150, 64), (torch.float32, 70, 128), (torch.bfloat16, 600, 64),
                                       (torch.bfloat16, 3, 64)])
def test_graph_replays_equal_eager(dtype, T, N):
    """A captured layer step (forward with saved states, backward, both norms), replayed on new inputs with
    eager work in between, equals the eager calls bit for bit; T = 600 splits in time, T = 3 decodes too."""
    O = ops()
    H = 2
    C = H * N
    weight, pre = torch.rand(C, device=DEV) + 0.5, torch.rand(C, device=DEV) + 0.5
    static = step_case(0, T, H, N, dtype)
    lens = torch.tensor([T, max(T - 20, 1)], dtype=torch.int32, device=DEV)

    def step(w, beta, r, k, v, go, S, x):
        ck = O.new_delta_ckpt(2, T, H, N, DEV)
        o, S1 = O.delta_forward(w, beta, r, k, v, lengths=lens, state_in=S, return_state=True, ckpt=ck)
        o2, S2 = O.delta_forward(w, beta, r, k, v, lengths=lens, state_in=S, return_state=True)
        z = O.head_norm(o, weight, None, x, heads=H)
        x_out, h = O.block_norm(x, z, pre, gate=x, scale=weight)
        g = O.block_norm_backward(x_out, z, go, pre, gate=x, scale=weight)
        dz = O.head_norm_backward(o, g["dy"], weight, None, x, heads=H)
        d = O.delta_backward(w, beta, r, k, v, dz[0], lengths=lens, state_in=S, grad_state_out=S1, need_state_grad=True, ckpt=ck)
        return [o, S1, o2, S2, z, x_out, h, *(t for t in g.values() if t is not None), *(t for t in dz if t is not None), *d]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for i in range(1, 5):
        new = step_case(i, T, H, N, dtype)
        for a, b in zip(static, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(*new)
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, j)


def test_bound_calls_and_refused_shapes():
    O = ops()
    w, beta, r, k, v, go, S, x = step_case(5, 3, 2, 64, torch.bfloat16)
    call = O.delta_forward(w, beta, r, k, v, state_in=S, return_state=True, bind=True)
    o, S1 = call()
    o = o.clone()
    want = O.delta_forward(w, beta, r, k, v, state_in=S, return_state=True)
    assert torch.equal(o, want[0]) and torch.equal(S1, want[1])
    weight = torch.ones(128, device=DEV)
    call = O.head_norm(v, weight, None, x, heads=2, bind=True)
    assert torch.equal(call(), O.head_norm(v, weight, None, x, heads=2))
    g = O.block_norm_backward(x, v, go, weight, bind=True)()
    for n, t in O.block_norm_backward(x, v, go, weight).items():
        assert t is None or torch.equal(g[n], t), n
    for bad, err in ((dict(beta=beta[:, :2]), ValueError), (dict(k=k.float()), TypeError), (dict(v=v[..., :120].contiguous()), ValueError),
                     (dict(w=w.double()), TypeError), (dict(r=r.transpose(0, 1)), ValueError)):
        args = dict(w=w, beta=beta, r=r, k=k, v=v) | bad
        with pytest.raises(err):
            O.delta_forward(**args)
    for kw in (dict(state_in=S[:1]), dict(lengths=torch.ones(2, device=DEV)), dict(lengths=torch.ones(3, dtype=torch.int32, device=DEV)),
               dict(out=torch.empty_like(v, dtype=torch.float32)), dict(ckpt=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            O.delta_forward(w, beta, r, k, v, **kw)
    with pytest.raises(ValueError):
        O.delta_backward(w, beta, r, k, v, go, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(O.L.WkvError):  # off the 16-byte grid
        odd = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view_as(v)
        O.delta_forward(w, beta, r, k, odd)
    for kw in (dict(heads=3), dict(heads=0), dict(heads=2, act="relu"), dict(heads=2, eps=-1.0)):
        with pytest.raises((ValueError, O.L.WkvError)):
            O.head_norm(v, weight, None, x, **kw)
    with pytest.raises(TypeError):
        O.head_norm(v, weight, None, x.float(), heads=2)
    with pytest.raises(ValueError):
        O.block_norm(x, v, weight, post_b=weight)
    with pytest.raises(TypeError):
        O.block_norm(x, v.float(), weight)


@pytest.mark.parametrize("rows,G,act", [(1, 64, "silu"), (5, 64, "none"), (333, 80, "sigmoid")])
def test_head_norm_without_eps(rows, G, act):
    """eps 0 is allowed: slots of a workgroup that hold no row must not add 0 * inf to the weights' sums."""
    O = ops()
    g = torch.Generator().manual_seed(rows)
    y, gout, gate = (torch.randn(rows, 3 * G, generator=g, dtype=torch.float64) for _ in range(3))
    weight = torch.rand(3 * G, generator=g, dtype=torch.float64) + 0.5
    leaves = [t.requires_grad_() for t in (y, weight, gate)]
    a = {"none": gate, "sigmoid": torch.sigmoid(gate), "silu": torch.nn.functional.silu(gate)}[act]
    (rms(y.view(rows, 3, G), 0.0).reshape(rows, 3 * G) * weight * a * gout).sum().backward()
    own = [t.detach().float().to(DEV) for t in (y, gout, weight)]
    dy, dw, _, dg = O.head_norm_backward(*own, None, gate.detach().float().to(DEV), heads=3, act=act, eps=0.0)
    # a sum of G (dy) or rows (dw) terms, each of some ten roundings
    for got, leaf, n in zip((dy, dw, dg), leaves, (G, rows, 1)):
        err = (got.double().cpu() - leaf.grad).norm() / leaf.grad.norm()
        assert err <= U * (16 + n), (float(err), n)


def test_gradients_that_are_views():
    """A gradient may arrive as a view that starts off the 16-byte grid, or is not contiguous."""
    O = ops()
    w, beta, r, k, v, go, S, x = step_case(9, 40, 2, 64, torch.bfloat16)
    want = O.delta_backward(w, beta, r, k, v, go, state_in=S, grad_state_out=S, need_state_grad=True)
    for odd in (True, False):
        leaves = [t.clone().requires_grad_() for t in (w, beta, r, k, v, S)]
        o, s1 = O.delta_rule(*leaves)
        pad = torch.zeros(3, device=DEV, requires_grad=True)
        if odd:
            out = torch.cat([pad.bfloat16(), o.reshape(-1)]), torch.cat([pad, s1.reshape(-1)])
            grads = torch.cat([pad.bfloat16(), go.reshape(-1)]), torch.cat([pad, S.reshape(-1)])
        else:
            out = o.transpose(0, 1), s1.transpose(2, 3)
            grads = go.transpose(0, 1).contiguous(), S.transpose(2, 3).contiguous()
        torch.autograd.backward(out, [g.detach() for g in grads])
        for leaf, g in zip(leaves, (want[3], want[4], want[0], want[1], want[2], want[5])):
            assert torch.equal(leaf.grad, g)


def test_second_derivatives_are_refused():
    O = ops()
    w, beta, r, k, v, go, S, x = step_case(9, 20, 2, 64, torch.float32)
    v.requires_grad_()
    ones = torch.ones(128, device=DEV)
    for out in (O.delta_rule(w, beta, r, k, v)[0], O.head_norm_gated(v, ones, None, x, heads=2), O.block_join(x, v, ones)[1]):
        (g,) = torch.autograd.grad(out.square().sum(), v, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()


def test_two_streams_at_once():
    """Calls on two streams share nothing: each gives what it gives alone."""
    O = ops()
    cases = [step_case(s, 700, 2, 64, torch.bfloat16) for s in (1, 2)]
    weight = torch.ones(128, device=DEV)

    def step(w, beta, r, k, v, go, S, x):
        o, s1 = O.delta_forward(w, beta, r, k, v, state_in=S, return_state=True)  # split in time
        d = O.delta_backward(w, beta, r, k, v, go, state_in=S, grad_state_out=s1)
        g = O.block_norm_backward(x, o, go, weight, gate=v)
        h = O.head_norm_backward(o, go, weight[:64], heads=2)
        return [o, s1, *d[:5], *(t for t in (*g.values(), *h) if t is not None)]

    want = [step(*c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(step(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for j, (a, b) in enumerate(zip(run, want[i])):
                assert torch.equal(a, b), (i, j)


def test_large_offsets():
    """Arrays of more than 2^32 bytes and 2^31 elements: the last batch row, which lies behind that, holds the
    first one's data and must give the first one's results bit for bit (which other tests check)."""
    O = ops()
    B, T, H, N = 3, 300000, 40, 64  # 2.3e9 elements
    C = H * N
    g = torch.Generator(device=DEV).manual_seed(0)

    def thrice(*shape, dtype=torch.bfloat16, scale=1.0):
        x = torch.empty((B, *shape), dtype=dtype, device=DEV)
        for t0 in range(0, T, 70000):
            part = (torch.randn((min(70000, T - t0), *shape[1:]), generator=g, device=DEV) * scale).to(dtype)
            x[0, t0:t0 + 70000], x[1, t0:t0 + 70000], x[2, t0:t0 + 70000] = part, 0, part
        return x

    r, k, v = thrice(T, C // 2), thrice(T, C // 2, scale=0.1), thrice(T, C)
    w, beta = thrice(T, H, dtype=torch.float32).abs_(), thrice(T, H, dtype=torch.float32).abs_().clamp_(max=1)
    lens = torch.tensor([T - 5, 1, T - 5], dtype=torch.int32, device=DEV)
    o, S = O.delta_forward(w, beta, r, k, v, lengths=lens, return_state=True)
    assert torch.equal(S[0], S[2]) and bool(torch.isfinite(S).all()) and float(S[0].abs().max()) > 0
    assert torch.equal(o[0], o[2]) and not bool(o[:, T - 5:].any()) and bool(o[2, T - 6].any())
    grads = O.delta_backward(w, beta, r, k, v, o, lengths=lens)
    for t in grads[:5]:
        assert torch.equal(t[0], t[2]) and not bool(t[:, T - 5:].any()) and bool(t[2, T - 6].any())
    del grads
    weight = torch.ones(C, device=DEV)
    n = O.head_norm(v, weight, None, o, heads=H)
    assert torch.equal(n[0], n[2]) and bool(n[2, T - 6].any())
    x1, h = O.block_norm(v, o, weight, gate=n, post_w=weight)
    assert torch.equal(x1[0], x1[2]) and torch.equal(h[0], h[2]) and bool(h[2, T - 1].any())
    back = O.block_norm_backward(x1, o, h, weight, gate=n, post_w=weight)
    assert torch.equal(back["dx"][0], back["dx"][2]) and torch.equal(back["dy"][0], back["dy"][2])
    back = O.head_norm_backward(v, h, weight, None, o, heads=H)
    assert torch.equal(back[0][0], back[0][2]) and torch.equal(back[3][0], back[3][2])


def test_many_narrow_rows():
    """More rows than one dimension of a grid holds threads for: the last row (and the one where the second
    dimension begins) must be the first one's, whose values are checked."""
    O = ops()
    for rows, H, G in ((70_000_000, 1, 3), (5_000_000, 1, 33)):
        x = torch.zeros(rows, H * G, dtype=torch.bfloat16, device=DEV)
        first = torch.randn(H * G, device=DEV).bfloat16()
        # 2^20 workgroups of four heads, or of one row
        marks = [0, 4 << 20, (4 << 20) - 1, (1 << 20) - 1, 1 << 20, rows - 1]
        x[marks] = first
        weight = torch.rand(H * G, device=DEV) + 0.5
        want = (rms(first.double()) * weight.double()).cpu()
        n = O.head_norm(x, weight, heads=H)
        _, h = O.block_norm(x, x, weight, center=False) if G == 33 else (None, None)
        for m in marks:
            assert ((n[m].double().cpu() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-6).all(), m
            if h is not None:  # x + x, eps off by a factor of 4 in the mean square
                assert ((h[m].double().cpu() - rms(2 * first.double()).cpu() * weight.double().cpu()).abs()
                        <= want.abs() * 2.0 ** -7 + 1e-6).all(), m
        assert int((n != 0).any(-1).sum()) == len(marks)
        del x, n, h


def test_delta_rule_without_gradients():
    O = ops()
    w, beta, r, k, v, go, S, x = step_case(4, 5, 2, 64, torch.bfloat16)
    want = O.delta_forward(w, beta, r, k, v, state_in=S, return_state=True)
    with torch.no_grad():
        off = O.delta_rule(w, beta, r, k, v.clone().requires_grad_(), S)
    for got in (O.delta_rule(w, beta, r, k, v, S), off):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0].requires_grad
    assert O.delta_rule(w, beta, r, k, v, S.clone().requires_grad_())[0].requires_grad
