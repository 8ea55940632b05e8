"""GPU parity of the gated delta rule (delta_forward, delta_backward) against the float64 oracle.

Bounds, from the kernels' arithmetic: float32 throughout (u = 2^-24), outputs rounded once (half a step
of their type).  With |k| <= 1 and beta in [0, 1] every token's map of the state is a contraction, so
an error made at one token reaches later ones no larger; a token's own products have N + 16 terms and
a handful of factors.  Taking the roundings as independent, T tokens of sqrt(N + 32) u each add up to
    eps = u sqrt((N + 32) T)
of the quantity's size, twice that behind two walks (the gradients).  Per tensor, the 2-norm of the
error is held to that plus the output rounding, and every element to 8 times it of the tensor's
largest element plus half a step of its own.  dw_t = -<H_t, D_t> and dbeta_t = <e_t, k_t G_t> cancel,
so theirs is taken of the factors' norms, which the oracle returns.
"""
import numpy as np
import pytest
import torch

from oracle import delta_backward_ref, delta_forward_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.bfloat16, torch.float32]


def ops():
    from rwkv_wkv_mixing_amd import ops as O

    return O


def problem(B, T, H, HK, N, dtype, seed=0, state=True, wmax=0.5):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    p = dict(w=torch.rand(B, T, H, generator=g) ** 3 * wmax, beta=torch.rand(B, T, H, generator=g),
             r=unit(rn(B, T, HK, N)).reshape(B, T, HK * N).to(dtype),
             # neighbouring keys alike: the triangular system is far from the identity
             k=(0.99 * unit(rn(B, T, HK, N) + 2 * rn(B, 1, HK, N))).reshape(B, T, HK * N).to(dtype),
             v=rn(B, T, H * N).to(dtype), go=rn(B, T, H * N).to(dtype))
    p["S0"] = rn(B, H, N, N) if state else None
    p["dS"] = rn(B, H, N, N) if state else None
    p["HK"] = HK
    return p


def ref_fwd(p, lengths=None):
    f = lambda n: p[n].double().numpy()  # noqa: E731
    return delta_forward_ref(f("w"), f("beta"), f("r"), f("k"), f("v"), p["HK"],
                             None if p["S0"] is None else f("S0"), lengths)


def ref_bwd(p, lengths=None):
    f = lambda n: None if p[n] is None else p[n].double().numpy()  # noqa: E731
    return delta_backward_ref(f("w"), f("beta"), f("r"), f("k"), f("v"), f("go"), p["HK"], f("S0"), f("dS"), lengths,
                              magnitude=True)


def dev(p):
    return {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in p.items()}


def check(name, got, ref, eps, scale=None):
    half = HALF[got.dtype]
    g, r = got.double().cpu().numpy(), np.asarray(ref)
    assert g.shape == r.shape, (name, g.shape, r.shape)
    assert np.isfinite(g).all(), name
    if not r.size:
        return
    err = np.abs(g - r)
    size = np.abs(r) if scale is None else np.asarray(scale)
    norm = np.linalg.norm(err) / max(np.linalg.norm(size), 1e-300)
    most = float((err - half * np.abs(r)).max()) / max(float(size.max()), 1e-300)
    print(f"  {name}: norm {norm:.2e} of {eps + half:.2e}, element {most:.2e} of {8 * eps:.2e}", flush=True)
    assert norm <= eps + half, name
    assert most <= 8 * eps, name


def eps_of(p):
    T, N = p["w"].shape[1], p["v"].shape[2] // p["w"].shape[2]
    return U * np.sqrt((N + 32) * max(T, 1))


def run_fwd(p, lengths=None, **kw):
    d = dev(p)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return ops().delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], lengths=ln, state_in=d["S0"],
                               return_state=True, **kw)


def run_bwd(p, lengths=None, ckpt=None, **kw):
    d = dev(p)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return ops().delta_backward(d["w"], d["beta"], d["r"], d["k"], d["v"], d["go"], lengths=ln, state_in=d["S0"],
                                grad_state_out=d["dS"], need_state_grad=True, ckpt=ckpt, **kw)


def check_fwd(p, lengths=None, **kw):
    o, S = run_fwd(p, lengths, **kw)
    ro, rS = ref_fwd(p, lengths)
    check("o", o, ro, eps_of(p))
    check("S", S, rS, eps_of(p))


def check_bwd(p, lengths=None, ckpt=None):
    got = run_bwd(p, lengths, ckpt)
    *ref, mw, mb = ref_bwd(p, lengths)
    for n, g, r, s in zip(("dr", "dk", "dv", "dw", "dbeta", "dS0"), got, ref, (None, None, None, mw, mb, None)):
        check(n, g, r, 2 * eps_of(p), s)
    return got


SHAPES = [  # B, T, H, HK, N
    (2, 1, 2, 1, 64), (1, 16, 3, 3, 128), (2, 17, 2, 2, 64), (3, 5, 2, 2, 64), (1, 63, 1, 1, 128), (2, 64, 4, 2, 64),
    (1, 65, 2, 1, 128), (2, 200, 6, 2, 64),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_forward(shape, dtype, state):
    check_fwd(problem(*shape, dtype, seed=sum(shape), state=state))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_blocks_equal_steps_and_oracle_with_ckpt(shape, dtype):
    """With a ckpt the block kernel runs at every length."""
    B, T, H, HK, N = shape
    p = problem(*shape, dtype, seed=7)
    check_fwd(p, ckpt=ops().new_delta_ckpt(B, T, H, N, DEV))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_backward(shape, dtype, state):
    check_bwd(problem(*shape, dtype, seed=1 + sum(shape), state=state))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
def test_saved_states_give_the_same_gradients(dtype, N):
    p = problem(2, 130, 4, 2, N, dtype, seed=3)
    ck = ops().new_delta_ckpt(2, 130, 4, N, DEV)
    run_fwd(p, ckpt=ck)
    for a, b in zip(run_bwd(p, ckpt=ck), run_bwd(p)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("T,lengths", [(9, [9, 0, 4, 1]), (150, [150, 64, 65, 0]), (150, [-3, 1, 200, 149])])
def test_lengths(dtype, T, lengths):
    """Ragged rows: the rows behind a length hold NaN, and none of it is seen."""
    p = problem(4, T, 4, 2, 64, dtype, seed=5)
    for b, n in enumerate(lengths):
        for name in ("w", "beta", "r", "k", "v", "go"):
            p[name][b, max(n, 0):] = float("nan")
    q = {n: torch.nan_to_num(x) if isinstance(x, torch.Tensor) else x for n, x in p.items()}
    o, S = run_fwd(p, lengths)
    ro, rS = ref_fwd(q, lengths)
    check("o", o, ro, eps_of(p))
    check("S", S, rS, eps_of(p))
    got = run_bwd(p, lengths)
    *ref, mw, mb = ref_bwd(q, lengths)
    for n, g, r, s in zip(("dr", "dk", "dv", "dw", "dbeta", "dS0"), got, ref, (None, None, None, mw, mb, None)):
        check(n, g, r, 2 * eps_of(p), s)
    for b, n in enumerate(lengths):
        for x in (o,) + got[:5]:
            assert (x[b, max(n, 0):] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_rates_of_every_size(dtype):
    """Rates of 0, tiny, large and infinite, one after the other; beta of 0 and 1."""
    p = problem(1, 150, 2, 2, 64, dtype, seed=6)
    g = torch.Generator().manual_seed(1)
    sizes = torch.tensor([0.0, 1e-6, 1e-3, 0.1, 3.0, 40.0, 1000.0, float("inf")])
    p["w"] = sizes[torch.randint(0, 8, p["w"].shape, generator=g)]
    p["w"][:, 70:100] = 1e-4
    p["beta"][:, ::3] = 0.0
    p["beta"][:, 1::3] = 1.0
    check_fwd(p)
    check_bwd(p)


@pytest.mark.parametrize("T", [1, 40])
def test_split_sequence_chains(T):
    """A sequence in two calls, the state and its gradient handed on, equals one call's bounds."""
    O = ops()
    p = problem(2, 100, 2, 2, 64, torch.float32, seed=8)
    d = dev(p)
    names = ("w", "beta", "r", "k", "v")
    first, second = [d[n][:, :T].contiguous() for n in names], [d[n][:, T:].contiguous() for n in names]
    o1, S1 = O.delta_forward(*first, state_in=d["S0"], return_state=True)
    o2, S2 = O.delta_forward(*second, state_in=S1, return_state=True)
    ro, rS = ref_fwd(p)
    check("o", torch.cat((o1, o2), 1), ro, eps_of(p))
    check("S", S2, rS, eps_of(p))
    g2 = O.delta_backward(*second, d["go"][:, T:].contiguous(), state_in=S1, grad_state_out=d["dS"], need_state_grad=True)
    g1 = O.delta_backward(*first, d["go"][:, :T].contiguous(), state_in=d["S0"], grad_state_out=g2[5], need_state_grad=True)
    *ref, mw, mb = ref_bwd(p)
    for i, (n, s) in enumerate(zip(("dr", "dk", "dv", "dw", "dbeta"), (None, None, None, mw, mb))):
        check(n, torch.cat((g1[i], g2[i]), 1), ref[i], 2 * eps_of(p), s)
    check("dS0", g1[5], ref[5], 2 * eps_of(p))


@pytest.mark.parametrize("T", [3, 70])
def test_state_in_place_and_determinism(T):
    O = ops()
    p = problem(3, T, 4, 2, 64, torch.bfloat16, seed=9)
    d = dev(p)
    o, S = run_fwd(p)
    S2 = d["S0"].clone()
    o2, out = O.delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], state_in=S2, state_out=S2, return_state=True)
    assert out is S2 and torch.equal(S, S2) and torch.equal(o, o2)
    for a, b in zip(run_bwd(p), run_bwd(p)):
        assert torch.equal(a, b)


def test_decode_carries_the_state():
    """40 tokens one at a time, the state in place."""
    O = ops()
    p = problem(3, 40, 4, 2, 128, torch.bfloat16, seed=10)
    d = dev(p)
    S, outs = d["S0"].clone(), []
    for t in range(40):
        outs.append(O.delta_forward(*(d[n][:, t:t + 1].contiguous() for n in ("w", "beta", "r", "k", "v")), state_in=S,
                                    state_out=S))
    ro, rS = ref_fwd(p)
    check("o", torch.cat(outs, 1), ro, eps_of(p))
    check("S", S, rS, eps_of(p))


def test_empty():
    O = ops()
    p = dev(problem(2, 0, 2, 1, 64, torch.bfloat16))
    o, S = O.delta_forward(*(p[n] for n in ("w", "beta", "r", "k", "v")), state_in=p["S0"], return_state=True)
    assert o.shape == (2, 0, 128) and torch.equal(S, p["S0"])
    g = O.delta_backward(*(p[n] for n in ("w", "beta", "r", "k", "v", "go")), state_in=p["S0"], grad_state_out=p["dS"],
                         need_state_grad=True)
    assert torch.equal(g[5], p["dS"]) and g[0].shape == (2, 0, 64)
    q = dev(problem(0, 5, 2, 1, 64, torch.bfloat16))
    o, S = O.delta_forward(*(q[n] for n in ("w", "beta", "r", "k", "v")), return_state=True)
    assert o.shape == (0, 5, 128) and S.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("lengths", [None, [50, 20]])
def test_autograd(lengths):
    O = ops()
    p = problem(2, 50, 4, 2, 64, torch.float32, seed=11)
    d = dev(p)
    leaves = [d[n].clone().requires_grad_() for n in ("w", "beta", "r", "k", "v", "S0")]
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    o, S = O.delta_rule(*leaves, lengths=ln)
    (o * d["go"]).sum().add((S * d["dS"]).sum()).backward()
    *ref, mw, mb = ref_bwd(p, lengths)
    for i, (j, s) in enumerate(((2, None), (3, None), (4, None), (0, mw), (1, mb), (5, None))):
        check("grad", leaves[j].grad, ref[i], 2 * eps_of(p), s)


def test_guard_bands():
    """Nothing is written outside the outputs: each lies between NaN guards, at odd lengths."""
    O = ops()
    for dtype in DTYPES:
        for N in (64, 128):
            for T in (5, 67):
                p = dev(problem(1, T, 2, 1, N, dtype, seed=12))
                pad = 512
                buf = torch.full((2 * pad + T * 2 * N,), float("nan"), dtype=dtype, device=DEV)
                out = buf[pad:-pad].view(1, T, 2 * N)
                sbuf = torch.full((2 * pad + 2 * N * N,), float("nan"), device=DEV)
                S = sbuf[pad:-pad].view(1, 2, N, N)
                n = O.delta_ckpt_bytes(1, T, 2, N)
                cbuf = torch.full((n + 1024,), 0x5a, dtype=torch.uint8, device=DEV)
                ck = cbuf[512:512 + n] if T > 16 else None
                O.delta_forward(*(p[x] for x in ("w", "beta", "r", "k", "v")), state_in=p["S0"], state_out=S, out=out, ckpt=ck)
                for x, y in ((buf, out), (sbuf, S)):
                    assert torch.isnan(x[:pad]).all() and torch.isnan(x[-pad:]).all() and torch.isfinite(y).all()
                assert (cbuf[:512] == 0x5a).all() and (cbuf[512 + n:] == 0x5a).all()


def test_other_stream():
    O = ops()
    p = problem(2, 90, 2, 2, 64, torch.bfloat16, seed=13)
    d = dev(p)
    o, S = run_fwd(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, S2 = O.delta_forward(*(d[n] for n in ("w", "beta", "r", "k", "v")), state_in=d["S0"], return_state=True)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(S, S2)


SPLIT = [(1, 1000, 2, 1, 64), (1, 700, 1, 1, 128), (2, 515, 2, 2, 64)]  # sequences split in time


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SPLIT, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_time_split(shape, dtype, state):
    """The split and the whole walk, forward (with and without a ckpt) and backward, within the bounds."""
    O = ops()
    B, T, H, HK, N = shape
    assert O.L.lib().wkv_delta_forward_workspace_bytes(B, T, H, HK, N) > 0
    p = problem(*shape, dtype, seed=20 + sum(shape), state=state, wmax=0.05)
    for split in (True, False):
        check_fwd(p, split=split)
        ck = O.new_delta_ckpt(B, T, H, N, DEV)
        check_fwd(p, split=split, ckpt=ck)
    *ref, mw, mb = ref_bwd(p)
    for kw in (dict(ckpt=ck), dict(split=False), dict()):
        for n, g, r, s in zip(("dr", "dk", "dv", "dw", "dbeta", "dS0"), run_bwd(p, **kw), ref, (None, None, None, mw, mb, None)):
            check(n, g, r, 2 * eps_of(p), s)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1000, 0, 257], [256, 512, 1], [255, 999, 640]])
def test_time_split_lengths(dtype, lengths):
    """Rows that end before, at and inside a segment; what lies behind them is NaN."""
    p = problem(3, 1000, 2, 1, 64, dtype, seed=30, wmax=0.05)
    for b, n in enumerate(lengths):
        for name in ("w", "beta", "r", "k", "v", "go"):
            p[name][b, n:] = float("nan")
    q = {n: torch.nan_to_num(x) if isinstance(x, torch.Tensor) else x for n, x in p.items()}
    o, S = run_fwd(p, lengths)
    ro, rS = ref_fwd(q, lengths)
    check("o", o, ro, eps_of(p))
    check("S", S, rS, eps_of(p))
    *ref, mw, mb = ref_bwd(q, lengths)
    for n, g, r, s in zip(("dr", "dk", "dv", "dw", "dbeta", "dS0"), run_bwd(p, lengths), ref, (None, None, None, mw, mb, None)):
        check(n, g, r, 2 * eps_of(p), s)
