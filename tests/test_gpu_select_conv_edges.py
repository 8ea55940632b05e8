"""The short convolution, the selective scan and the clipping where calls go wrong: outputs and workspaces of exactly the
stated sizes between guards, not-a-number among the inputs, segments chained through their states, captured and replayed
calls, two streams, bound calls, the same bits twice, inputs off the vectors' grid."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.select_ref import conv_ref, select_ref
from rwkv_wkv_mixing_amd import _lib as L
from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DT = {F32: L.WKV_F32, BF: L.WKV_BF16}
DTYPES, IDS = [BF, F32], ["bf16", "f32"]
PAD, MARK = 4096, 0xFF  # a float or bf16 of these bytes is a NaN
SEQ = ("x", "dt", "b", "c", "z", "go")


class Guarded:
    """Regions between guards; check() looks at all of them."""

    def __init__(self):
        self.buffers = []

    def bytes(self, n):
        buf = torch.full((2 * PAD + n,), MARK, dtype=torch.uint8, device=DEV)
        self.buffers.append(buf)
        return buf[PAD:PAD + n]

    def like(self, t):
        return self.bytes(t.nbytes).view(t.dtype).view(t.shape)

    def check(self):
        for i, buf in enumerate(self.buffers):
            assert bool((buf[:PAD] == MARK).all()) and bool((buf[-PAD:] == MARK).all()), i


def at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def draw(B, T, C, G, N, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T + C + N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(x=rn(B, T, C), dt=rn(B, T, C), b=rn(B, T, G * N), c=rn(B, T, G * N), z=rn(B, T, C), go=rn(B, T, C))
    p = {k: v.to(dtype) for k, v in p.items()}
    p.update(w=torch.arange(1, N + 1) * torch.exp(0.2 * rn(C, N)), d=rn(C), dt_bias=rn(C) - 3.0, S=rn(B, C, N), Gs=rn(B, C, N))
    return {k: v.to(DEV) for k, v in p.items()}


def inputs(p):
    return [p[k] for k in ("x", "dt", "w", "b", "c")], dict(d=p["d"], z=p["z"], dt_bias=p["dt_bias"])


def draw_conv(B, T, C, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T + C + K)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(x=rn(B, T, C).to(dtype), weight=rn(K, C), bias=rn(C), S=rn(B, K - 1, C).to(dtype), go=rn(B, T, C).to(dtype),
             Gs=rn(B, K - 1, C).to(dtype))
    return {k: v.to(DEV) for k, v in p.items()}


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,C,G,N", [(1, 3, 1, 8), (5, 130, 2, 16), (8, 65, 1, 32), (17, 65, 1, 16), (67, 63, 3, 8), (600, 66, 2, 32),
                                     (333, 200, 1, 16)])
@pytest.mark.parametrize("saved", [True, False], ids=["ckpt", "recomputed"])
def test_select_writes_its_outputs_and_nothing_else(dtype, T, C, G, N, saved):
    B, lib, gd = 2, L.lib(), Guarded()
    p = draw(B, T, C, G, N, dtype)
    ln = torch.tensor([T, max(T - 21, 0)], dtype=torch.int32, device=DEV)
    args, kw = inputs(p)
    ck = gd.bytes(lib.wkv_select_ckpt_bytes(B, T, C, N)) if saved else None
    nws = lib.wkv_select_forward_workspace_bytes(B, T, C, G, N)
    ws = gd.bytes(nws) if nws else None
    out, S1 = gd.like(p["x"]), gd.like(p["S"])
    L.check("forward", lib.wkv_select_forward(
        B, T, C, G, N, DT[dtype], 1, at(ln), *(at(p[k]) for k in ("x", "dt", "w", "b", "c", "d", "z", "dt_bias")), at(out), at(p["S"]),
        at(S1), at(ck), at(ws), nws, stream()))
    gd.check()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(S1).all())
    own = O.new_select_ckpt(B, T, C, N, DEV) if saved else None
    want = O.select_forward(*args, lengths=ln, state_in=p["S"], return_state=True, ckpt=own, **kw)
    if T > 64 or nws == 0:  # (the binding splits from 65 tokens on)
        assert torch.equal(out, want[0]) and torch.equal(S1, want[1])
    nws = lib.wkv_select_backward_workspace_bytes(B, T, C, G, N, 1 if saved else 0)
    ws = gd.bytes(nws)
    names = ("dx", "ddt", "dw", "db", "dc", "dd", "dz", "ddt_bias", "dstate_in")
    like = dict(zip(names, ("x", "dt", "w", "b", "c", "d", "z", "dt_bias", "S")))
    g = {n: gd.like(p[like[n]]) for n in names}
    L.check("backward", lib.wkv_select_backward(
        B, T, C, G, N, DT[dtype], 1, at(ln), *(at(p[k]) for k in ("x", "dt", "w", "b", "c", "d", "z", "dt_bias", "go", "S", "Gs")),
        *(at(g[n]) for n in names), at(ck), at(ws), nws, stream()))
    gd.check()
    want = O.select_backward(*args, p["go"], lengths=ln, state_in=p["S"], grad_state_out=p["Gs"], need_state_grad=True, ckpt=ck, **kw)
    for n in names:
        assert bool(torch.isfinite(g[n]).all()), n
        assert torch.equal(g[n], want[n]), n


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,C", [(1, 1), (2, 7), (5, 64), (17, 260), (129, 1001), (400, 12)])
def test_conv_writes_its_outputs_and_nothing_else(dtype, K, T, C):
    B, lib, gd = 2, L.lib(), Guarded()
    p = draw_conv(B, T, C, K, dtype)
    ln = torch.tensor([T, max(T - 3, 0)], dtype=torch.int32, device=DEV)
    out, S1 = gd.like(p["x"]), gd.like(p["S"])
    head = (B, T, C, K, DT[dtype], L.WKV_ACT_SILU, at(ln), at(p["x"]), at(p["weight"]), at(p["bias"]), at(p["S"]))
    L.check("forward", lib.wkv_conv_forward(*head, at(out), at(S1), stream()))
    gd.check()
    want = O.conv_forward(p["x"], p["weight"], p["bias"], lengths=ln, state_in=p["S"], return_state=True)
    assert torch.equal(out, want[0]) and torch.equal(S1, want[1]) and bool(torch.isfinite(out).all())
    nws = lib.wkv_conv_backward_workspace_bytes(B, T, C, K)
    ws, g = gd.bytes(nws), [gd.like(p[k]) for k in ("x", "weight", "bias", "S")]
    L.check("backward", lib.wkv_conv_backward(*head, at(p["go"]), at(p["Gs"]), *(at(t) for t in g), at(ws), nws, stream()))
    gd.check()
    want = O.conv_backward(p["x"], p["go"], p["weight"], p["bias"], lengths=ln, state_in=p["S"], grad_state_out=p["Gs"],
                           need_state_grad=True)
    for a, b in zip(g, want):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


@pytest.mark.parametrize("sizes", [[1], [3, 16384, 0, 5], [16385, 7, 100000]])
def test_clip_writes_its_outputs_and_nothing_else(sizes):
    gd, lib = Guarded(), L.lib()
    grads = [torch.randn(n, device=DEV).to(BF if i % 2 else F32) for i, n in enumerate(sizes)]
    outs, norm = [gd.like(t) for t in grads], gd.like(torch.empty(1, device=DEV))
    nws = lib.wkv_clip_workspace_bytes(len(sizes))
    ws, n = gd.bytes(nws), len(sizes)
    arr = lambda t, v: (t * n)(*v)  # noqa: E731
    L.check("clip", lib.wkv_clip_gradients(
        n, arr(ctypes.c_void_p, [t.data_ptr() for t in grads]), arr(ctypes.c_void_p, [t.data_ptr() for t in outs]),
        arr(ctypes.c_int64, sizes), arr(ctypes.c_int, [DT[t.dtype] for t in grads]), 0.25, 1e-6, at(norm), at(ws), nws, stream()))
    gd.check()
    want = O.clip_gradients(grads, 0.25)
    assert torch.equal(norm[0], want)
    for o, g in zip(outs, grads):
        assert torch.equal(o, g)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,split", [(40, False), (700, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_select_not_a_number_stays_where_it_is_read(bad, T, split, dtype):
    """In x of one token of one channel: no earlier token, other channel or other row has anything of it."""
    B, C = 2, 70
    p = draw(B, T, C, 1, 16, dtype)
    args, kw = inputs(p)
    clean = O.select_forward(*args, split=split, **kw)
    t, ch = T - 13, 66
    p["x"][1, t, ch] = bad
    out = O.select_forward(*args, split=split, **kw)
    assert not bool(torch.isfinite(out[1, t:, ch]).all())
    out[1, t:, ch] = clean[1, t:, ch]
    assert torch.equal(out, clean)
    p["x"][1, t, ch] = 0.0
    g0 = O.select_backward(*args, p["go"], split=split, **kw)
    p["go"][1, t, ch] = bad  # a gradient's reaches earlier tokens of its channel, and what is summed over channels and rows
    g1 = O.select_backward(*args, p["go"], split=split, **kw)
    for n in ("dx", "ddt", "dz"):
        g1[n][1, :t + 1, ch] = g0[n][1, :t + 1, ch]
        assert torch.equal(g0[n], g1[n]), n
    for n in ("db", "dc"):
        assert torch.equal(g0[n][0], g1[n][0]) and torch.equal(g0[n][1, t + 1:], g1[n][1, t + 1:]), n
    other = torch.arange(C, device=DEV) != ch
    for n in ("dw", "dd", "ddt_bias"):
        assert torch.equal(g0[n][other], g1[n][other]), n


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,split", [(3, False), (40, False), (700, True)], ids=["steps", "whole", "split"])
@pytest.mark.parametrize("N", [8, 16])
def test_select_rates_that_are_not_a_number_show(N, T, split, dtype):
    """A channel with one such rate has no output, state or gradient by x that is a number (the last token's gradient by x
    needs no rate); the others are as without it."""
    B, C = 2, 70
    p = draw(B, T, C, 1, N, dtype)
    args, kw = inputs(p)
    clean, S0 = O.select_forward(*args, split=split, return_state=True, **kw)
    ch = 66
    p["w"][ch, N - 3] = float("nan")
    out, S1 = O.select_forward(*args, split=split, return_state=True, **kw)
    assert bool(torch.isnan(out[:, :, ch]).all()) and bool(torch.isnan(S1[:, ch, N - 3]).all())
    g = O.select_backward(*args, p["go"], split=split, **kw)
    assert bool(torch.isnan(g["dx"][:, :-1, ch]).all()) and bool(torch.isnan(g["dw"][ch, N - 3]))
    out[:, :, ch], S1[:, ch] = clean[:, :, ch], S0[:, ch]
    assert torch.equal(out, clean) and torch.equal(S1, S0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_conv_not_a_number_stays_where_it_is_read(dtype):
    p = draw_conv(2, 70, 68, 4, dtype)
    clean = O.conv_forward(p["x"], p["weight"], p["bias"])
    p["x"][1, 40, 5] = float("nan")
    out = O.conv_forward(p["x"], p["weight"], p["bias"])
    assert bool(torch.isnan(out[1, 40:44, 5]).all())
    out[1, 40:44, 5] = clean[1, 40:44, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_select_steps_and_rates_at_their_ends(dtype):
    """Steps that underflow, that are as large as dt itself, infinite rates (nothing kept), a rate of zero (all kept)."""
    p = draw(1, 40, 64, 1, 16, dtype)
    p["dt"][:, ::3] = -200.0
    p["dt"][:, 1::3] = 60.0
    p["w"][:8] = float("inf")
    p["w"][8:16] = 0.0
    args, kw = inputs(p)
    out, S1 = O.select_forward(*args, state_in=p["S"], return_state=True, **kw)
    h = {k: v.double().cpu().numpy() for k, v in p.items()}
    h["w"] = np.minimum(h["w"], 1e300)  # (0 x inf is not a decay)
    h["dt"][:, ::3] = -np.inf  # log(1 + e^{-200 + bias}) is below float32's smallest number: a step of zero, which keeps the state
    r, m = (select_ref(*(h[k] for k in ("x", "dt", "w", "b", "c")), d=h["d"], z=h["z"], dt_bias=h["dt_bias"], state_in=h["S"], mag=k)
            for k in (False, True))
    rel = 2.0 ** -8 if dtype is BF else 0.0
    u = (3 * 40 + 64 + 128) * 2.0 ** -24  # as in the parity tests of the scan
    for got, n in ((out, "out"), (S1, "state")):
        assert (np.abs(got.double().cpu().numpy() - r[n]) <= (u * (1 + rel) * m[n] + (rel if n == "out" else 0.0) * np.abs(r[n]) + 1e-30)).all(), n


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_segments_chain_through_their_states(dtype):
    """Two segments, forward through the state and backward through its gradient, are the whole sequence (float32 sums in
    another grouping: 1e-5 of the largest, and a bf16 rounding where an output has one)."""
    B, T, C, N, cut = 2, 90, 70, 16, 37
    p, q = draw(B, T, C, 1, N, dtype), draw_conv(B, T, C, 4, dtype)

    def near(a, b):
        tol = 2.0 ** -7 if a.dtype is BF else 1e-5
        assert float((a.float() - b.float()).abs().max()) <= tol * float(b.float().abs().max())

    args, kw = inputs(p)
    out, S1 = O.select_forward(*args, state_in=p["S"], return_state=True, **kw)
    g = O.select_backward(*args, p["go"], state_in=p["S"], grad_state_out=p["Gs"], need_state_grad=True, **kw)
    part = [{k: (v[:, s].contiguous() if k in SEQ else v) for k, v in p.items()} for s in (slice(0, cut), slice(cut, T))]
    (a0, k0), (a1, k1) = (inputs(x) for x in part)
    o0, mid = O.select_forward(*a0, state_in=p["S"], return_state=True, **k0)
    o1, end = O.select_forward(*a1, state_in=mid, return_state=True, **k1)
    near(torch.cat([o0, o1], 1), out)
    near(end, S1)
    g1 = O.select_backward(*a1, part[1]["go"], state_in=mid, grad_state_out=p["Gs"], need_state_grad=True, **k1)
    g0 = O.select_backward(*a0, part[0]["go"], state_in=p["S"], grad_state_out=g1["dstate_in"], need_state_grad=True, **k0)
    for n in ("dx", "ddt", "db", "dc", "dz"):
        near(torch.cat([g0[n], g1[n]], 1), g[n])
    for n in ("dw", "dd", "ddt_bias"):
        near(g0[n] + g1[n], g[n])
    near(g0["dstate_in"], g["dstate_in"])
    for cut in (1, 2, 37, 88, 89):  # a convolution's segments may be shorter than its filter
        full, C1 = O.conv_forward(q["x"], q["weight"], q["bias"], state_in=q["S"], return_state=True)
        gf = O.conv_backward(q["x"], q["go"], q["weight"], q["bias"], state_in=q["S"], grad_state_out=q["Gs"], need_state_grad=True)
        x0, x1, y0, y1 = (v[:, s].contiguous() for v in (q["x"], q["go"]) for s in (slice(0, cut), slice(cut, T)))
        o0, mid = O.conv_forward(x0, q["weight"], q["bias"], state_in=q["S"], return_state=True)
        o1, end = O.conv_forward(x1, q["weight"], q["bias"], state_in=mid, return_state=True)
        assert torch.equal(torch.cat([o0, o1], 1), full) and torch.equal(end, C1)
        b1 = O.conv_backward(x1, y1, q["weight"], q["bias"], state_in=mid, grad_state_out=q["Gs"], need_state_grad=True)
        b0 = O.conv_backward(x0, y0, q["weight"], q["bias"], state_in=q["S"], grad_state_out=b1[3], need_state_grad=True)
        near(torch.cat([b0[0], b1[0]], 1), gf[0])
        near(b0[1] + b1[1], gf[1])
        near(b0[2] + b1[2], gf[2])
        near(b0[3], gf[3])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,T,C,N", [(2, 40, 66, 16), (63, 33, 5, 8), (64, 33, 70, 16), (65, 20, 66, 8), (3, 400, 64, 32)])
def test_many_ragged_rows_are_each_their_own(B, T, C, N, dtype):
    """Rows of all lengths, many alike, some empty, some given as negative or too long: every row as in a call by itself."""
    p = draw(B, T, C, 1, N, dtype)
    lens = (torch.arange(B, dtype=torch.int32) * 7 % (T + 4) - 2).to(DEV)
    lens[0], lens[B - 1] = T, -5
    args, kw = inputs(p)
    split = dict(split=T > 64)
    out, S1 = O.select_forward(*args, lengths=lens, state_in=p["S"], return_state=True, **split, **kw)
    g = O.select_backward(*args, p["go"], lengths=lens, state_in=p["S"], grad_state_out=p["Gs"], need_state_grad=True, **split, **kw)
    for b in sorted({0, 1, B // 3, B // 2, B - 2, B - 1}):
        cut = lambda v: v[b:b + 1].contiguous()  # noqa: E731
        row = [cut(v) if v.dim() == 3 else v for v in args]
        k1 = {k: cut(v) if v.dim() == 3 else v for k, v in kw.items()}
        one = dict(lengths=cut(lens), state_in=cut(p["S"]), split=False)
        o1, R1 = O.select_forward(*row, return_state=True, **one, **k1)
        g1 = O.select_backward(*row, cut(p["go"]), grad_state_out=cut(p["Gs"]), need_state_grad=True, **one, **k1)
        for got, want in [(out[b], o1[0]), (S1[b], R1[0])] + [(g[n][b], g1[n][0]) for n in ("dx", "ddt", "dz", "db", "dc", "dstate_in")]:
            tol = 2.0 ** -7 if got.dtype is BF else 1e-5  # (sums over states in groups of their own, a split: other roundings)
            assert float((got.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("N,C,B", [(16, 4096, 64), (8, 4100, 130), (32, 2052, 65)])
def test_states_past_the_caches_are_the_same_bits(N, C, B, dtype):
    """In place, 16 MB of states and more in one call, and row by row in calls of less; a row without tokens keeps its own."""
    p = draw(B, 2, C, 1, N, dtype)
    assert B * C * N >= 1 << 22 > C * N
    lens = torch.full((B,), 2, dtype=torch.int32, device=DEV)
    lens[3], lens[B - 1] = 0, 1
    args, kw = inputs(p)
    S = p["S"].clone()
    out = O.select_forward(*args, lengths=lens, state_in=S, state_out=S, **kw)
    for b in (0, 3, B // 2, B - 1):
        row = [v[b:b + 1].contiguous() if v.dim() == 3 else v for v in args]
        k1 = {k: v[b:b + 1].contiguous() if v.dim() == 3 else v for k, v in kw.items()}
        o1, S1 = O.select_forward(*row, lengths=lens[b:b + 1].contiguous(), state_in=p["S"][b:b + 1].contiguous(), return_state=True, **k1)
        assert torch.equal(o1[0], out[b]) and torch.equal(S1[0], S[b])
    assert torch.equal(S[3], p["S"][3]) and not bool(out[3].any())


def test_no_tokens_and_no_rows():
    p, q = draw(2, 0, 70, 1, 16, F32), draw_conv(2, 0, 70, 4, BF)
    args, kw = inputs(p)
    out, S1 = O.select_forward(*args, state_in=p["S"], return_state=True, **kw)
    assert out.shape == (2, 0, 70) and torch.equal(S1, p["S"])
    assert not bool(O.select_forward(*args, return_state=True, **kw)[1].any())
    g = O.select_backward(*args, p["go"], grad_state_out=p["Gs"], need_state_grad=True, **kw)
    assert torch.equal(g["dstate_in"], p["Gs"]) and not any(bool(g[n].any()) for n in ("dw", "dd", "ddt_bias"))
    out, S1 = O.conv_forward(q["x"], q["weight"], q["bias"], state_in=q["S"], return_state=True)
    assert torch.equal(S1, q["S"])
    dx, dweight, dbias, ds = O.conv_backward(q["x"], q["go"], q["weight"], q["bias"], grad_state_out=q["Gs"], need_state_grad=True)
    assert torch.equal(ds, q["Gs"]) and not bool(dweight.any()) and not bool(dbias.any())
    p = draw(0, 20, 70, 1, 16, F32)
    args, kw = inputs(p)
    g = O.select_backward(*args, p["go"], **kw)
    assert not any(bool(g[n].any()) for n in ("dw", "dd", "ddt_bias"))


def layer(p, q, ck, norm, s):
    """Convolution, scan, their gradients and the clip of these, on buffers of their own."""
    args, kw = inputs(p)
    s["x"] = O.conv_forward(q["x"], q["weight"], q["bias"], state_in=q["S"])
    args = [s["x"], *args[1:]]
    s["out"], s["S1"] = O.select_forward(*args, state_in=p["S"], return_state=True, ckpt=ck, **kw)
    s["g"] = O.select_backward(*args, p["go"], state_in=p["S"], ckpt=ck, **kw)
    s["c"] = O.conv_backward(q["x"], s["g"]["dx"], q["weight"], q["bias"], state_in=q["S"])
    s["norm"] = O.clip_gradients([s["c"][1], s["c"][2], s["g"]["dw"], s["g"]["dd"]], 0.5, norm=norm)


def flat(s):
    return [s["x"], s["out"], s["S1"], *[v for v in s["g"].values() if v is not None], *[v for v in s["c"] if v is not None], s["norm"]]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T", [5, 100, 700])
def test_captured_and_replayed(T, dtype):
    """A layer's calls (with and without a time split) captured once and replayed on fresh inputs, eager work in between."""
    p, q = draw(2, T, 68, 1, 16, dtype), draw_conv(2, T, 68, 4, dtype)
    ck, norm = O.new_select_ckpt(2, T, 68, 16, DEV), torch.empty((), device=DEV)
    s, warm = {}, torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        layer(p, q, ck, norm, s)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(p, q, ck, norm, s)
    for i in range(4):
        for k, v in draw(2, T, 68, 1, 16, dtype, seed=i + 1).items():
            p[k].copy_(v)
        for k, v in draw_conv(2, T, 68, 4, dtype, seed=i + 1).items():
            q[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in flat(s)]
        eager = {}
        layer(p, q, O.new_select_ckpt(2, T, 68, 16, DEV), torch.empty((), device=DEV), eager)
        torch.cuda.synchronize()
        for a, b in zip(got, flat(eager)):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    sets = [(draw(2, 700, 68, 1, 16, BF, seed=i), draw_conv(2, 700, 68, 4, BF, seed=i)) for i in range(2)]
    want = []
    for p, q in sets:
        s = {}
        layer(p, q, O.new_select_ckpt(2, 700, 68, 16, DEV), torch.empty((), device=DEV), s)
        want.append(s)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(5):
        for i, (p, q) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                s = {}
                layer(p, q, O.new_select_ckpt(2, 700, 68, 16, DEV), torch.empty((), device=DEV), s)
                got[i].append(s)
    torch.cuda.synchronize()
    for i in range(2):
        for s in got[i]:
            for a, b in zip(flat(s), flat(want[i])):
                assert torch.equal(a, b)


def test_bound_calls():
    p, q = draw(2, 90, 68, 1, 16, BF), draw_conv(2, 90, 68, 4, BF)
    args, kw = inputs(p)
    call = O.select_forward(*args, bind=True, **kw)
    assert torch.equal(call().clone(), O.select_forward(*args, **kw))
    back = O.select_backward(*args, p["go"], bind=True, **kw)
    g = {k: v.clone() for k, v in back().items() if v is not None}
    for k, v in O.select_backward(*args, p["go"], **kw).items():
        assert v is None or torch.equal(v, g[k])
    conv = O.conv_forward(q["x"], q["weight"], q["bias"], bind=True)
    assert torch.equal(conv().clone(), O.conv_forward(q["x"], q["weight"], q["bias"]))
    grads = [torch.randn(100, device=DEV), torch.randn(50, device=DEV).to(BF)]
    out = [torch.empty_like(t) for t in grads]
    clip = O.clip_gradients(grads, 1.0, out=out, bind=True)
    del out
    for _ in range(2):
        grads[0].normal_()
        n = clip()
        assert float(n) == pytest.approx(float(O.grad_norm(grads)))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_off_the_vectors_grid(dtype):
    """Tensors that start one element off any vector's grid give what tensors on it give (the weights' sums may be grouped
    otherwise: vectors of another width make another grid)."""
    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    p, q = draw(2, 90, 68, 1, 16, dtype), draw_conv(2, 90, 68, 4, dtype)
    args, kw = inputs(p)
    want, wg = O.select_forward(*args, **kw), O.select_backward(*args, p["go"], **kw)
    shifted = [off(p["x"]), off(p["dt"]), p["w"], p["b"], p["c"]]
    kw2 = dict(d=off(p["d"]), z=off(p["z"]), dt_bias=off(p["dt_bias"]))
    assert torch.equal(O.select_forward(*shifted, out=off(p["x"]), **kw2), want)
    for k, v in O.select_backward(*shifted, off(p["go"]), **kw2).items():
        assert v is None or torch.equal(v, wg[k])
    with pytest.raises(RuntimeError, match="aligned"):
        O.select_forward(p["x"], p["dt"], p["w"], off(p["b"]), p["c"], **kw)
    want = O.conv_forward(q["x"], q["weight"], q["bias"], state_in=q["S"], return_state=True)
    got = O.conv_forward(off(q["x"]), off(q["weight"]), off(q["bias"]), state_in=off(q["S"]), return_state=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wg = O.conv_backward(q["x"], q["go"], q["weight"], q["bias"], state_in=q["S"], need_state_grad=True)
    gg = O.conv_backward(off(q["x"]), off(q["go"]), off(q["weight"]), off(q["bias"]), state_in=off(q["S"]), need_state_grad=True)
    assert torch.equal(gg[0], wg[0]) and torch.equal(gg[3], wg[3])
    for a, b in ((gg[1], wg[1]), (gg[2], wg[2])):
        assert float((a - b).abs().max()) <= 180 * 2.0 ** -24 * 2.0 * float(b.abs().max() + 40.0)  # sums of 180 terms


def test_refusals_of_the_binding():
    p, q = draw(2, 20, 68, 1, 16, BF), draw_conv(2, 20, 68, 4, BF)
    args, kw = inputs(p)
    x, dt, w, b, c = args
    for bad in ([x[0], dt, w, b, c], [x, dt[:, :-1].contiguous(), w, b, c], [x, dt, w[:-1].contiguous(), b, c],
                [x, dt, w[:, :12].contiguous(), b, c], [x, dt, w, b[..., :12].contiguous(), c], [x, dt, w, b, c[:, :-1].contiguous()],
                [x.transpose(0, 1), dt, w, b, c]):
        with pytest.raises(ValueError):
            O.select_forward(*bad)
    with pytest.raises(TypeError):
        O.select_forward(x, dt.float(), w, b, c)
    with pytest.raises(TypeError):
        O.select_forward(x, dt, w.to(BF), b, c)
    with pytest.raises(ValueError, match="ckpt"):
        O.select_forward(*args, ckpt=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        O.select_backward(*args, p["go"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="taps"):
        O.conv_forward(q["x"], q["weight"][:1].contiguous())
    with pytest.raises(ValueError, match="act"):
        O.conv_forward(q["x"], q["weight"], act="tanh")
    with pytest.raises(ValueError):
        O.conv_forward(q["x"], q["weight"], state_in=q["S"][:, :-1].contiguous())
    g = torch.ones(4, device=DEV)
    with pytest.raises(ValueError):
        O.clip_gradients([g], 1.0, out=[torch.ones(5, device=DEV)])
    with pytest.raises(ValueError, match="tensors for"):
        O.clip_gradients([g], 1.0, out=[])
    with pytest.raises(TypeError):
        O.clip_gradients([g.half()], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        O.clip_gradients([torch.ones(4, 4, device=DEV).t()], 1.0)


def test_conv_against_the_oracle_in_place_and_short_rows():
    """Rows shorter than the filter, the carried inputs in place."""
    q = draw_conv(4, 6, 10, 4, F32)
    ln = [0, 1, 2, 6]
    h = {k: v.double().cpu().numpy() for k, v in q.items()}
    r = conv_ref(h["x"], h["weight"], h["bias"], lengths=ln, state_in=h["S"])
    state = q["S"].clone()
    O.conv_forward(q["x"], q["weight"], q["bias"], lengths=torch.tensor(ln, dtype=torch.int32, device=DEV), state_in=state,
                   state_out=state)
    assert np.array_equal(state.double().cpu().numpy(), r["state"])
