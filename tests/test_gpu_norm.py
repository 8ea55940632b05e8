"""GPU parity of the norms around the mixing (head_norm, block_norm and their backwards) against the
float64 oracle.

Bounds, from the kernels' arithmetic (float32, u = 2^-24; outputs rounded once, half a step of their
type): a sum over C channels adds at most 16 in one lane, 6 rounds of shuffles and 16 waves, so it is
off by at most 38 u of its terms' magnitudes; a divisor, made of two such sums and a square root, by 60 u;
exp(-g) by (2 + |g|) u.  A forward output passes one divisor or two and the gate: within
    (160 + 4 max|g|) u of its magnitude (the sum of its terms' absolute values, from the oracle);
a gradient passes two more sums: twice that.  A sum over R rows adds at most R / 64 + 1 rows (no more
than 128 when R is at most 8192) in a lane, 32 runs and 64 partial sums: 256 u more.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm_backward_ref, block_norm_ref, head_norm_backward_ref, head_norm_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F32, BF), (F32, F32)]
TIDS = ["bf16", "f32-bf16", "f32"]


def ops():
    from rwkv_wkv_mixing_amd import ops as O

    return O


def check(name, got, ref, mag, c):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), name
    if not ref.size:
        return
    ratio = np.abs(g - ref) / (HALF[got.dtype] * np.abs(ref) + c * U * mag + 1e-30)
    print(f"  {name}: worst err / bound {ratio.max():.3f}", flush=True)
    assert ratio.max() <= 1.0, (name, np.unravel_index(ratio.argmax(), ratio.shape))


def near(a, b):
    return 160 + 4 * float(b.abs().max()) if b is not None and b.numel() else 160


def head_case(rows, H, G, ty, tg, shared=False, bias=True, gated=True, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed + rows + H + G)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    n = G if shared else H * G
    return dict(y=(rn(rows, H * G) * (0.1 + rn(rows, 1).abs()) + offset).to(ty), gout=rn(rows, H * G).to(tg),
                weight=1 + 0.3 * rn(n), bias=rn(n) if bias else None, gate=2 * rn(rows, H * G).to(tg) if gated else None)


def run_head(c, H, act, center, tg, eps=1e-5):
    d = {n: None if t is None else t.to(DEV) for n, t in c.items()}
    kw = dict(heads=H, act=act, center=center, eps=eps)
    O = ops()
    out = None if c["gate"] is not None else torch.empty(c["y"].shape, dtype=tg, device=DEV)
    got = O.head_norm(d["y"], d["weight"], d["bias"], d["gate"], out=out, **kw)
    assert got.dtype == tg
    host = [c[n] if c[n] is None else c[n].double().numpy() for n in ("weight", "bias", "gate")]
    base = near(None, c["gate"])
    ref, mag = head_norm_ref(c["y"].double().numpy(), *host, H, act, center, eps)
    check("out", got, ref, mag, base)
    grads = O.head_norm_backward(d["y"], d["gout"], d["weight"], d["bias"], d["gate"], **kw)
    ref, mag = head_norm_backward_ref(c["y"].double().numpy(), c["gout"].double().numpy(), *host, H, act, center, eps)
    for n, t in zip(("dy", "dweight", "dbias", "dgate"), grads):
        assert (t is None) == (n not in ref), n
        if t is not None:
            check(n, t, ref[n], mag[n], 2 * base + (256 if n in ("dweight", "dbias") else 0))
    return got, grads


@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 2, 5), (7, 3, 64), (130, 1, 80), (65, 5, 128), (9, 2, 1000), (4, 3, 520),
                                   (300, 8, 32), (2, 2, 999), (5, 70, 8)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
def test_head_norm(shape, types, center):
    run_head(head_case(*shape, *types), shape[1], "silu", center, types[1])


@pytest.mark.parametrize("shape", [(33, 3, 100), (20, 2, 129), (21, 2, 201), (6, 2, 257), (50, 64, 100)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("shared", [False, True], ids=["own", "shared"])
def test_head_norm_off_the_grid(shape, shared):
    """Heads that are no multiple of 8: two, four or sixteen elements a lane."""
    run_head(head_case(*shape, F32, BF, shared, True, True), shape[1], "sigmoid", True, BF)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("shared,bias,gated", [(True, True, True), (True, False, False), (False, False, True)])
def test_head_norm_options(act, shared, bias, gated):
    run_head(head_case(200, 6, 64, F32, BF, shared, bias, gated), 6, act, True, BF)


def test_head_norm_far_mean():
    """A mean a thousand times the deviation: the squares are taken of what the mean leaves."""
    run_head(head_case(20, 4, 64, F32, F32, offset=1000.0), 4, "silu", True, F32)


def test_head_norm_constant_rows():
    """A row of equal values (and of zeros): norm 0, divisor sqrt(eps)."""
    c = head_case(6, 2, 64, F32, F32)
    c["y"][0] = 0.0
    c["y"][1] = 3.0
    run_head(c, 2, "silu", True, F32)
    c["y"][1] = 0.0
    run_head(c, 2, "silu", False, F32)


def block_case(rows, C, tx, ty, post=True, bias=True, scaled=True, gated=True, later=True, seed=0):
    g = torch.Generator().manual_seed(seed + rows + C)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=2 * rn(rows, C).to(tx), y=rn(rows, C).to(ty), gate=2 * rn(rows, C).to(ty) if gated else None,
                gx=rn(rows, C).to(tx) if later else None, gh=rn(rows, C).to(ty), pre_w=1 + 0.3 * rn(C),
                pre_b=rn(C) if bias else None, post_w=1 + 0.3 * rn(C) if post else None,
                post_b=rn(C) if post and bias else None, scale=0.5 + 0.2 * rn(C) if scaled else None)


def run_block(c, act, center, eps=1e-5):
    O = ops()
    d = {n: None if t is None else t.to(DEV) for n, t in c.items()}
    h = {n: None if t is None else t.double().numpy() for n, t in c.items()}
    names = ("gate", "post_w", "post_b", "scale")
    kw = dict(act=act, center=center, eps=eps)
    base = near(None, c["gate"])
    x_out, hh = O.block_norm(d["x"], d["y"], d["pre_w"], d["pre_b"], **{n: d[n] for n in names}, **kw)
    assert x_out.dtype == c["x"].dtype and hh.dtype == c["y"].dtype
    ref, mag = block_norm_ref(h["x"], h["y"], h["pre_w"], h["pre_b"], **{n: h[n] for n in names}, **kw)
    check("x_out", x_out, ref[0], mag[0], base)
    check("h", hh, ref[1], mag[1], 2 * base)
    g = O.block_norm_backward(x_out, d["y"], d["gh"], d["pre_w"], d["pre_b"], gx=d["gx"], **{n: d[n] for n in names}, **kw)
    ref, mag = block_norm_backward_ref(x_out.double().cpu().numpy(), h["y"], h["gh"], h["pre_w"], h["pre_b"], gx=h["gx"],
                                       **{n: h[n] for n in names}, **kw)
    for n, t in g.items():
        assert (t is None) == (n not in ref), n
        if t is not None:
            check(n, t, ref[n], mag[n], 4 * base + (256 if t.dim() == 1 else 0))
    return x_out, hh, g


@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("shape", [(1, 1), (3, 5), (5, 64), (70, 250), (9, 512), (11, 520), (3, 1000), (2, 4096), (2, 4100),
                                   (600, 96), (2, 8192), (1, 8191)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("center", [False, True], ids=["rms", "layer"])
def test_block_norm(shape, types, center):
    run_block(block_case(*shape, *types), "sigmoid", center)


@pytest.mark.parametrize("shape", [(1100, 4104), (40, 5000), (30, 4101), (1030, 513), (300, 511)], ids=lambda s: "x".join(map(str, s)))
def test_block_norm_many_rows(shape):
    """Wide and odd rows, several to a workgroup of the backward."""
    run_block(block_case(*shape, F32, BF), "silu", True)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("post,bias,scaled,gated,later", [(False, False, False, False, False), (True, False, False, True, True),
                                                          (False, True, True, True, False), (True, True, True, False, True)])
def test_block_norm_options(act, post, bias, scaled, gated, later):
    run_block(block_case(40, 768, F32, BF, post, bias, scaled, gated, later), act, True)


def test_more_rows_than_partial_sums():
    run_block(block_case(1500, 40, BF, BF), "silu", True)
    run_head(head_case(9000, 2, 16, BF, BF, shared=True), 2, "silu", True, BF)


def test_misaligned_equals_aligned():
    """Rows that start off a 16-byte boundary take the element path: the same to rounding."""
    O = ops()
    for ty, tg in TYPES:
        c = head_case(33, 3, 64, ty, tg)
        d = {n: t.to(DEV) for n, t in c.items()}
        off = {n: torch.cat((t.flatten()[:1], t.flatten()))[1:].view(t.shape) for n, t in d.items()}
        want = O.head_norm(d["y"], d["weight"], d["bias"], d["gate"], heads=3)
        got = O.head_norm(off["y"], off["weight"], off["bias"], off["gate"], heads=3)
        ref, mag = head_norm_ref(*(c[n].double().numpy() for n in ("y", "weight", "bias", "gate")), 3)
        check("aligned", want, ref, mag, near(None, c["gate"]))
        check("misaligned", got, ref, mag, near(None, c["gate"]))


def test_determinism_in_place_and_streams():
    O = ops()
    c = {n: t.to(DEV) for n, t in block_case(700, 1024, F32, BF).items()}
    names = ("gate", "post_w", "post_b", "scale")
    kw = {n: c[n] for n in names}
    x_out, h = O.block_norm(c["x"], c["y"], c["pre_w"], c["pre_b"], **kw)
    x2 = c["x"].clone()
    a, b = O.block_norm(x2, c["y"], c["pre_w"], c["pre_b"], x_out=x2, **kw)
    assert a is x2 and torch.equal(a, x_out) and torch.equal(b, h)
    g1 = O.block_norm_backward(x_out, c["y"], c["gh"], c["pre_w"], c["pre_b"], gx=c["gx"], **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g2 = O.block_norm_backward(x_out, c["y"], c["gh"], c["pre_w"], c["pre_b"], gx=c["gx"], **kw)
    torch.cuda.current_stream().wait_stream(s)
    for n in g1:
        assert torch.equal(g1[n], g2[n]), n


def test_empty():
    O = ops()
    z = lambda *s: torch.zeros(s, device=DEV, dtype=BF)  # noqa: E731
    w = torch.ones(8, device=DEV)
    assert O.head_norm(z(0, 8), w, w, z(0, 8), heads=2).shape == (0, 8)
    dy, dw, db, dg = O.head_norm_backward(z(0, 8), z(0, 8), w, w, z(0, 8), heads=2)
    assert (dw == 0).all() and (db == 0).all() and dy.shape == dg.shape == (0, 8)
    xo, h = O.block_norm(z(0, 8), z(0, 8), w)
    g = O.block_norm_backward(xo, z(0, 8), z(0, 8), w, w, post_w=w, post_b=w, scale=w)
    assert all((g[n] == 0).all() for n in ("dpre_w", "dpre_b", "dpost_w", "dpost_b", "dscale"))


def test_autograd():
    O = ops()
    c = head_case(20, 4, 64, F32, F32)
    L = {n: t.to(DEV).requires_grad_() for n, t in c.items()}
    O.head_norm_gated(L["y"], L["weight"], L["bias"], L["gate"], heads=4, center=True).backward(c["gout"].to(DEV))
    ref, mag = head_norm_backward_ref(*(c[n].double().numpy() for n in ("y", "gout", "weight", "bias", "gate")), 4, "silu", True)
    for n in ("y", "weight", "bias", "gate"):
        check("d" + n, L[n].grad, ref["d" + n], mag["d" + n], 2 * near(None, c["gate"]) + 256)
    c = block_case(20, 96, F32, F32)
    L = {n: t.to(DEV).requires_grad_() for n, t in c.items()}
    names = ("gate", "post_w", "post_b", "scale")
    x_out, h = O.block_join(L["x"], L["y"], L["pre_w"], L["pre_b"], **{n: L[n] for n in names})
    (x_out * L["gx"].detach()).sum().add((h * L["gh"].detach()).sum()).backward()
    np_ = {n: t.double().numpy() for n, t in c.items()}
    ref, mag = block_norm_backward_ref(x_out.detach().double().cpu().numpy(), np_["y"], np_["gh"], np_["pre_w"], np_["pre_b"],
                                       gx=np_["gx"], **{n: np_[n] for n in names})
    for n in ("x", "y", "pre_w", "pre_b") + names:
        check("d" + n, L[n].grad, ref["d" + n], mag["d" + n], 4 * near(None, c["gate"]) + 256)
