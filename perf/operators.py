"""The gated delta rule and the norms around it, measured: real work over the range a user meets.

A case is a dict of plain values; ``kind`` says which call it is.

``prefill``       the delta rule over a batch of sequences from a carried state, returning the state
``decode``        the same for a few tokens a stream (one, or a handful when drafts are checked)
``train``         the delta rule forward and backward, every gradient returned
``head_norm``     the per-head norm of the mixing output with its gate; ``head_norm_bwd`` its gradients
``block_norm``    the residual sum behind a block with the norm before the next; ``block_norm_bwd`` its gradients

With ``own`` false, ``run`` computes them from elementary torch operations in float32 (decay sums in
float64); with ``own`` true it makes the framework's calls.
"""
import math

import torch

own = False

CHUNK = 64  # tokens a chunk of the plain delta rule
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # a small served model: one token for each of four streams, where the launch is what counts
        dict(name="decode-small", kind="decode", B=4, T=1, H=8, HK=8, N=64, dtype="bf16"),
        # one token for 256 streams of a 64-head layer: the states' trip through memory
        dict(name="decode-256", kind="decode", B=256, T=1, H=64, HK=64, N=64, dtype="bf16"),
        # prompts of unequal length read into states, two value heads to a key head, an odd longest
        dict(name="prefill-ragged", kind="prefill", B=6, T=1501, H=32, HK=16, N=128, dtype="bf16", ragged=True),
        # one long document: few (row, head) pairs, many tokens
        dict(name="prefill-long", kind="prefill", B=1, T=32768, H=32, HK=32, N=128, dtype="bf16", ragged=False),
        # a training layer at the benchmark's size
        dict(name="train-layer", kind="train", B=8, T=1024, H=64, HK=64, N=64, dtype="bf16", ragged=False),
        # a small training run in float32 with shared key heads, an odd length and ragged rows
        dict(name="train-f32-odd", kind="train", B=2, T=333, H=8, HK=4, N=64, dtype="f32", ragged=True),
        # the mixing output of a 64-head training layer, float32 as the matrix-state calls return it
        dict(name="head-norm", kind="head_norm", rows=8192, H=64, G=64, ydtype="f32", dtype="bf16", act="silu",
             center=False, bias=False, shared=False),
        # a few decode streams
        dict(name="head-norm-decode", kind="head_norm", rows=4, H=8, G=64, ydtype="bf16", dtype="bf16", act="silu",
             center=True, bias=True, shared=False),
        # its gradients in a training layer, one weight for all heads
        dict(name="head-norm-bwd", kind="head_norm_bwd", rows=8192, H=32, G=128, ydtype="bf16", dtype="bf16",
             act="silu", center=False, bias=False, shared=True),
        # between two blocks of a training layer: gate, residual scale, next norm
        dict(name="block-norm", kind="block_norm", rows=8192, C=4096, xdtype="bf16", dtype="bf16", act="sigmoid",
             center=True, post=True, scale=True),
        # the same backward
        dict(name="block-norm-bwd", kind="block_norm_bwd", rows=8192, C=4096, xdtype="bf16", dtype="bf16",
             act="sigmoid", center=True, post=True, scale=True),
        # an odd width with the residual stream in float32
        dict(name="block-norm-bwd-odd", kind="block_norm_bwd", rows=777, C=1000, xdtype="f32", dtype="bf16",
             act="none", center=False, post=False, scale=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefill", "decode", "train", "head_norm", "head_norm_bwd", "block_norm", "block_norm_bwd"])
    if kind in ("prefill", "decode", "train"):
        N = rng.choice([64, 128])
        HK = _log(rng, 1, 16)
        H = HK * rng.choice([1, 1, 2, 4])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if kind == "decode":
            return dict(kind=kind, B=_log(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 5, 8]), H=H, HK=HK, N=N, dtype=dtype)
        T = _log(rng, 17, 8192 if kind == "prefill" else 2048)
        most = max(1, (1 << 25) // (T * H * N * (1 if kind == "prefill" else 2)))
        return dict(kind=kind, B=_log(rng, 1, min(16, most)), T=T, H=H, HK=HK, N=N, dtype=dtype,
                    ragged=rng.random() < 0.5)
    act = rng.choice(["none", "sigmoid", "silu"])
    if kind.startswith("head_norm"):
        G = rng.choice([32, 64, 80, 128, 256])
        H = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, min(16384, (1 << 25) // (H * G))))
        ydtype, dtype = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        return dict(kind=kind, rows=rows, H=H, G=G, ydtype=ydtype, dtype=dtype, act=act,
                    center=rng.random() < 0.5, bias=rng.random() < 0.5, shared=rng.random() < 0.5)
    C = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        C = max(64, C // 64 * 64)
    rows = _log(rng, 1, max(1, min(16384, (1 << 25) // C)))
    xdtype, dtype = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    return dict(kind=kind, rows=rows, C=C, xdtype=xdtype, dtype=dtype, act=act, center=rng.random() < 0.5,
                post=rng.random() < 0.5, scale=rng.random() < 0.5)


def _lengths(case):
    """The tokens of each row: the case's own, so that its work is known."""
    B, T = case["B"], case["T"]
    if not case.get("ragged"):
        return [T] * B
    return [T - (b * T) // (2 * B) if b else T for b in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=gen, device=dev)  # noqa: E731
    dt = DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if case["kind"] in ("prefill", "decode", "train"):
        B, T, H, HK, N = (case[n] for n in ("B", "T", "H", "HK", "N"))
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
        s["r"] = unit(randn(B, T, HK, N)).reshape(B, T, HK * N).to(dt)
        s["k"] = unit(randn(B, T, HK, N) + 0.5 * randn(1, 1, HK, N)).reshape(B, T, HK * N).to(dt)
        s["v"] = randn(B, T, H * N).to(dt)
        s["beta"] = torch.sigmoid(randn(B, T, H))
        # rates from slow heads to fast ones, and now and then a token that clears most of the state
        w = torch.exp(math.log(1e-3) + (math.log(0.3) - math.log(1e-3)) * rand(B, T, H))
        s["w"] = torch.where(rand(B, T, H) < 0.002, w + 6.0, w)
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if case.get("ragged") else None
        if case["kind"] == "train":
            s["go"] = randn(B, T, H * N).to(dt)
        else:
            s["state"] = 0.3 * randn(B, H, N, N)
            s["state_out"] = torch.empty_like(s["state"])
        return s
    if case["kind"].startswith("head_norm"):
        rows, H, G = case["rows"], case["H"], case["G"]
        s["y"] = (randn(rows, H * G) * (0.2 + 2.0 * rand(rows, 1)) + 0.1).to(DTYPES[case["ydtype"]])
        s["gate"] = randn(rows, H * G).to(dt)
        n = G if case["shared"] else H * G
        s["weight"] = 1.0 + 0.1 * randn(n)
        s["bias"] = 0.1 * randn(n) if case["bias"] else None
        if case["kind"].endswith("bwd"):
            s["gout"] = randn(rows, H * G).to(dt)
        return s
    rows, C = case["rows"], case["C"]
    s["x"] = (2.0 * randn(rows, C)).to(DTYPES[case["xdtype"]])
    s["y"] = randn(rows, C).to(dt)
    s["gate"] = randn(rows, C).to(dt)
    s["pre_w"] = 1.0 + 0.1 * randn(C)
    s["pre_b"] = 0.1 * randn(C) if case["center"] else None
    s["post_w"] = 1.0 + 0.1 * randn(C) if case["post"] else None
    s["post_b"] = 0.1 * randn(C) if case["post"] and case["center"] else None
    s["scale"] = 0.5 + 0.1 * randn(C) if case["scale"] else None
    if case["kind"].endswith("bwd"):
        s["gx"] = randn(rows, C).to(DTYPES[case["xdtype"]])
        s["gh"] = randn(rows, C).to(dt)
    return s


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own(s, kind)
    if kind in ("prefill", "decode"):
        o, state = _delta(s, s["w"], s["beta"], s["r"].float(), s["k"].float(), s["v"].float(), s["state"])
        return dict(o=o.to(s["r"].dtype), state=state)
    if kind == "train":
        leaves = [x.float().detach().requires_grad_() for x in (s["w"], s["beta"], s["r"], s["k"], s["v"])]
        with torch.enable_grad():
            o, _ = _delta(s, *leaves, None)
        dw, dbeta, dr, dk, dv = torch.autograd.grad(o, leaves, s["go"].float())
        dt = s["r"].dtype
        return dict(o=o.detach().to(dt), dr=dr.to(dt), dk=dk.to(dt), dv=dv.to(dt), dw=dw, dbeta=dbeta)
    return {"head_norm": _head_norm, "head_norm_bwd": _head_norm_bwd, "block_norm": _block_norm,
            "block_norm_bwd": _block_norm_bwd}[kind](s)


def _own(s, kind):
    from rwkv_wkv_mixing_amd import ops

    c = s["case"]
    if kind in ("prefill", "decode"):
        o, state = ops.delta_forward(s["w"], s["beta"], s["r"], s["k"], s["v"], lengths=s["lengths"],
                                     state_in=s["state"], state_out=s["state_out"], return_state=True)
        return dict(o=o, state=state)
    if kind == "train":
        ckpt = ops.new_delta_ckpt(c["B"], c["T"], c["H"], c["N"], s["r"].device)
        o = ops.delta_forward(s["w"], s["beta"], s["r"], s["k"], s["v"], lengths=s["lengths"], ckpt=ckpt)
        dr, dk, dv, dw, dbeta, _ = ops.delta_backward(s["w"], s["beta"], s["r"], s["k"], s["v"], s["go"],
                                                      lengths=s["lengths"], ckpt=ckpt)
        return dict(o=o, dr=dr, dk=dk, dv=dv, dw=dw, dbeta=dbeta)
    if kind == "head_norm":
        return dict(out=ops.head_norm(s["y"], s["weight"], s["bias"], s["gate"], heads=c["H"], act=c["act"],
                                      center=c["center"], eps=EPS))
    if kind == "head_norm_bwd":
        dy, dweight, dbias, dgate = ops.head_norm_backward(s["y"], s["gout"], s["weight"], s["bias"], s["gate"],
                                                           heads=c["H"], act=c["act"], center=c["center"], eps=EPS)
        return dict(dy=dy, dweight=dweight, dbias=dbias, dgate=dgate)
    kw = dict(gate=s["gate"], act=c["act"], post_w=s["post_w"], post_b=s["post_b"], scale=s["scale"],
              center=c["center"], eps=EPS)
    if kind == "block_norm":
        x_out, h = ops.block_norm(s["x"], s["y"], s["pre_w"], s["pre_b"], **kw)
        return dict(x_out=x_out, h=h)
    return ops.block_norm_backward(s["x"], s["y"], s["gh"], s["pre_w"], s["pre_b"], gx=s["gx"], **kw)


# ---- plain forms


def _mask(s, x):
    """x with the tokens behind each row's length at zero."""
    if s["lengths"] is None:
        return x
    t = torch.arange(x.shape[1], device=x.device)
    return torch.where((t[None] < s["lengths"][:, None])[..., None], x, torch.zeros((), device=x.device))


def _unit_lower_inverse(m):
    """The inverses of unit lower triangular matrices [..., n, n], n a power of two: twice as large
    blocks each time, [[a, 0], [c, d]]^-1 = [[a^-1, 0], [-d^-1 c a^-1, d^-1]]."""
    n = m.shape[-1]
    i = torch.arange(n, device=m.device)
    inv = torch.eye(n, device=m.device).expand(m.shape)
    size = 1
    while size < n:
        corner = ((i[:, None] // size) == (i[None] // size) + 1) & ((i[:, None] // size) % 2 == 1)
        inv = inv - inv @ (m * corner @ inv)
        size *= 2
    return inv


def _delta(s, w, beta, r, k, v, state):
    """The gated delta rule over chunks: all that a chunk's tokens do to each other at once, then
    the state from chunk to chunk."""
    c = s["case"]
    B, T, H, HK, N = (c[n] for n in ("B", "T", "H", "HK", "N"))
    L = min(CHUNK, 1 << (T - 1).bit_length())
    n = -(-T // L)

    def chunks(x, heads):
        x = torch.nn.functional.pad(_mask(s, x), (0, 0, 0, n * L - T))
        x = x.reshape(B, n, L, heads, -1).permute(0, 3, 1, 2, 4)
        return x.repeat_interleave(H // heads, dim=1) if heads != H else x

    rc, kc, vc = chunks(r, HK), chunks(k, HK), chunks(v, H)
    bc = chunks(beta, H)
    logs = -torch.cumsum(chunks(w, H).double(), dim=3)  # [B, H, n, L, 1]
    i = torch.arange(L, device=w.device)
    low = i[:, None] >= i[None]
    gap = (logs - logs.transpose(3, 4)).masked_fill(~low, -math.inf)
    decay = torch.exp(gap).float()
    since, until = torch.exp(logs).float(), torch.exp(logs[..., -1:, :] - logs).float()
    kt = kc.transpose(3, 4).contiguous()
    among = (kc @ kt) * decay * (i[:, None] > i[None])
    solve = _unit_lower_inverse(torch.eye(L, device=w.device) + bc * among) * bc.transpose(3, 4)
    reads = (rc @ kt) * decay
    fresh, past = solve @ vc, solve @ (since * kc)
    from_past = since * rc
    put = (until * kc).transpose(3, 4).contiguous()
    if state is None:
        state = torch.zeros(B, H, N, N, device=w.device)
    out = []
    for j in range(n):
        new = fresh[:, :, j] - past[:, :, j] @ state
        out.append(from_past[:, :, j] @ state + reads[:, :, j] @ new)
        state = since[:, :, j, -1:] * state + put[:, :, j] @ new
    o = torch.stack(out, 2).permute(0, 2, 3, 1, 4).reshape(B, n * L, H * N)[:, :T]
    return o, state


def _gate(act, g):
    """The gate's value and its derivative."""
    if act == "none":
        return g, torch.ones_like(g)
    p = torch.sigmoid(g)
    return (p, p * (1 - p)) if act == "sigmoid" else (g * p, p * (1 + g * (1 - p)))


def _norm(x, center):
    """x over its last axis's deviation (or root mean square), and 1 over that."""
    if center:
        x = x - x.mean(-1, keepdim=True)
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * inv, inv


def _norm_grad(g, xhat, inv, center):
    g = g - xhat * (g * xhat).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if center else 0.0)
    return g * inv


def _head_norm(s):
    c = s["case"]
    rows, H, G = c["rows"], c["H"], c["G"]
    xhat, _ = _norm(s["y"].float().view(rows, H, G), c["center"])
    z = xhat * s["weight"].view(-1, G)
    if s["bias"] is not None:
        z = z + s["bias"].view(-1, G)
    a, _ = _gate(c["act"], s["gate"].float().view(rows, H, G))
    return dict(out=(z * a).view(rows, H * G).to(s["gate"].dtype))


def _head_norm_bwd(s):
    c = s["case"]
    rows, H, G = c["rows"], c["H"], c["G"]
    xhat, inv = _norm(s["y"].float().view(rows, H, G), c["center"])
    weight = s["weight"].view(-1, G)
    z = xhat * weight
    if s["bias"] is not None:
        z = z + s["bias"].view(-1, G)
    a, da = _gate(c["act"], s["gate"].float().view(rows, H, G))
    g = s["gout"].float().view(rows, H, G)
    dz = g * a
    over = (0, 1) if c["shared"] else (0,)
    return dict(dy=_norm_grad(dz * weight, xhat, inv, c["center"]).view(rows, H * G).to(s["y"].dtype),
                dweight=(dz * xhat).sum(over).reshape(-1),
                dbias=dz.sum(over).reshape(-1) if s["bias"] is not None else None,
                dgate=(g * z * da).view(rows, H * G).to(s["gate"].dtype))


def _block_norm(s):
    c = s["case"]
    z = s["y"].float()
    if c["post"]:
        z = _norm(z, c["center"])[0] * s["post_w"]
        z = z + s["post_b"] if s["post_b"] is not None else z
    z = z * _gate(c["act"], s["gate"].float())[0]
    x = s["x"].float() + (z * s["scale"] if c["scale"] else z)
    h = _norm(x, c["center"])[0] * s["pre_w"]
    h = h + s["pre_b"] if s["pre_b"] is not None else h
    return dict(x_out=x.to(s["x"].dtype), h=h.to(s["y"].dtype))


def _block_norm_bwd(s):
    """s["x"] holds what the forward returned as x_out."""
    c = s["case"]
    xhat, inv = _norm(s["x"].float(), c["center"])
    gh = s["gh"].float()
    dx = s["gx"].float() + _norm_grad(gh * s["pre_w"], xhat, inv, c["center"])
    a, da = _gate(c["act"], s["gate"].float())
    y = s["y"].float()
    z = y
    if c["post"]:
        yhat, yinv = _norm(y, c["center"])
        z = yhat * s["post_w"]
        z = z + s["post_b"] if s["post_b"] is not None else z
    dsum = dx * s["scale"] if c["scale"] else dx
    dz = dsum * a
    dy = _norm_grad(dz * s["post_w"], yhat, yinv, c["center"]) if c["post"] else dz
    return dict(dx=dx.to(s["x"].dtype), dy=dy.to(s["y"].dtype),
                dgate=(dsum * z * da).to(s["gate"].dtype),
                dpre_w=(gh * xhat).sum(0), dpre_b=gh.sum(0) if s["pre_b"] is not None else None,
                dpost_w=(dz * yhat).sum(0) if c["post"] else None,
                dpost_b=dz.sum(0) if s["post_b"] is not None else None,
                dscale=(dx * z * a).sum(0) if c["scale"] else None)


# ---- work


def work(case):
    size = lambda d: 2 if d == "bf16" else 4  # noqa: E731
    if case["kind"] in ("prefill", "decode", "train"):
        H, HK, N, e = case["H"], case["HK"], case["N"], size(case["dtype"])
        tokens, rows = sum(_lengths(case)), case["B"] * case["T"]
        read = tokens * (2 * HK * N * e + H * N * e + 2 * H * 4)  # r, k, v, w, beta
        if case["kind"] == "train":
            read += tokens * H * N * e  # the gradient of o
            write = rows * (2 * H * N * e + 2 * HK * N * e + 2 * H * 4)  # o, dv, dr, dk, dw, dbeta
            return dict(bytes=read + write, flops=tokens * H * 22 * N * N)
        return dict(bytes=read + rows * H * N * e + 2 * case["B"] * H * N * N * 4, flops=tokens * H * 7 * N * N)
    bwd = case["kind"].endswith("bwd")
    e = size(case["dtype"])
    if case["kind"].startswith("head_norm"):
        n, ey = case["rows"] * case["H"] * case["G"], size(case["ydtype"])
        return dict(bytes=n * (2 * ey + 3 * e if bwd else ey + 2 * e), flops=n * (30 if bwd else 12))
    n, ex = case["rows"] * case["C"], size(case["xdtype"])
    return dict(bytes=n * (3 * ex + 5 * e if bwd else 2 * ex + 3 * e), flops=n * (45 if bwd else 25))


# ---- the definitions in float64


def exact(case, seed):
    if case["kind"] in ("prefill", "decode", "train"):
        if case["kind"] == "train" and case["B"] * case["T"] * case["H"] * case["N"] ** 2 * 8 > 40e9:
            return None
        return _exact_delta(prepare(case, seed))
    s = {n: x.double() if isinstance(x, torch.Tensor) else x for n, x in prepare(case, seed).items()}
    return _exact_head(s) if case["kind"].startswith("head_norm") else _exact_block(s)


def _exact_delta(s):
    """Token by token: the state is decayed, what it says of the key is taken from the value, the
    rest written in, and the receptance read out; then the adjoint of each of these, last first."""
    c = s["case"]
    B, T, H, HK, N = (c[n] for n in ("B", "T", "H", "HK", "N"))
    dev, f8 = s["r"].device, torch.float64
    live = torch.ones(B, T, 1, dtype=f8, device=dev)
    for b, n in enumerate(_lengths(c)):
        live[b, n:] = 0
    heads = lambda x, n: x.to(f8).view(B, T, n, N).repeat_interleave(H // n, dim=2)  # noqa: E731
    r, k, v = heads(s["r"], HK), heads(s["k"], HK), heads(s["v"], H)
    a = torch.exp(-s["w"].to(f8) * live)[..., None, None]  # [B, T, H, 1, 1]
    be = (s["beta"].to(f8) * live)[..., None]
    lv = live[..., None]
    S = s["state"].to(f8) if "state" in s else torch.zeros(B, H, N, N, dtype=f8, device=dev)
    train = c["kind"] == "train"
    o = torch.zeros(B, T, H, N, dtype=f8, device=dev)
    kept, errs = [], []
    for t in range(T):
        if train:
            kept.append(S)
        D = a[:, t] * S
        err = v[:, t] - (k[:, t, :, :, None] * D).sum(-2)
        S = D + k[:, t, :, :, None] * (be[:, t] * err)[:, :, None]
        o[:, t] = (r[:, t, :, :, None] * S).sum(-2) * lv[:, t]
        errs.append(err if train else None)
    flat = lambda x: x.reshape(B, T, -1)  # noqa: E731
    if not train:
        return dict(o=flat(o), state=S)
    go = s["go"].to(f8).view(B, T, H, N) * lv
    dr, dk, dv = (torch.zeros(B, T, H, N, dtype=f8, device=dev) for _ in range(3))
    dw, db = (torch.zeros(B, T, H, dtype=f8, device=dev) for _ in range(2))
    G = torch.zeros(B, H, N, N, dtype=f8, device=dev)
    after = S
    for t in range(T - 1, -1, -1):
        dr[:, t] = (after * go[:, t, :, None]).sum(-1)
        G = G + r[:, t, :, :, None] * go[:, t, :, None]
        put = be[:, t] * errs[t]
        dput = (k[:, t, :, :, None] * G).sum(-2)
        derr = be[:, t] * dput
        D = a[:, t] * kept[t]
        db[:, t] = (errs[t] * dput).sum(-1)
        dv[:, t] = derr
        dk[:, t] = (G * put[:, :, None]).sum(-1) - (D * derr[:, :, None]).sum(-1)
        G = G - k[:, t, :, :, None] * derr[:, :, None]
        dw[:, t] = -(G * D).sum((-1, -2))
        G = a[:, t] * G
        after = kept[t]
    shared = lambda x: flat((x * lv).view(B, T, HK, H // HK, N).sum(3))  # noqa: E731
    return dict(o=flat(o), dr=shared(dr), dk=shared(dk), dv=flat(dv * lv), dw=dw * live, dbeta=db * live)


def _exact_normed(x, center):
    m = x.mean(-1, keepdim=True) if center else 0.0
    return (x - m) / torch.sqrt((x - m).pow(2).mean(-1, keepdim=True) + EPS)


def _exact_act(act, g):
    return g if act == "none" else 1 / (1 + torch.exp(-g)) if act == "sigmoid" else g / (1 + torch.exp(-g))


def _exact_head(s):
    c = s["case"]
    rows, H, G = c["rows"], c["H"], c["G"]
    names = ["y", "weight", "bias", "gate"]
    leaf = {n: s[n].clone().requires_grad_() if s[n] is not None else None for n in names}
    wide = lambda p: p.view(1, -1, G)  # noqa: E731
    z = _exact_normed(leaf["y"].view(rows, H, G), c["center"]) * wide(leaf["weight"])
    z = z + wide(leaf["bias"]) if s["bias"] is not None else z
    out = z.reshape(rows, H * G) * _exact_act(c["act"], leaf["gate"])
    if c["kind"] == "head_norm":
        return dict(out=out.detach())
    out.backward(s["gout"])
    return {"d" + n: leaf[n].grad if leaf[n] is not None else None for n in names}


def _exact_block(s):
    c = s["case"]
    names = ["x", "y", "gate", "pre_w", "pre_b", "post_w", "post_b", "scale"]
    leaf = {n: s[n].clone().requires_grad_() if s[n] is not None else None for n in names}
    z = leaf["y"]
    if c["post"]:
        z = _exact_normed(z, c["center"]) * leaf["post_w"]
        z = z + leaf["post_b"] if s["post_b"] is not None else z
    z = z * _exact_act(c["act"], leaf["gate"])
    z = z * leaf["scale"] if c["scale"] else z
    if c["kind"] == "block_norm":
        x = leaf["x"] + z
        h = _exact_normed(x, c["center"]) * leaf["pre_w"]
        h = h + leaf["pre_b"] if s["pre_b"] is not None else h
        return dict(x_out=x.detach(), h=h.detach())
    # the residual sum is given: its gradient reaches both of its terms
    h = _exact_normed(leaf["x"], c["center"]) * leaf["pre_w"]
    h = h + leaf["pre_b"] if s["pre_b"] is not None else h
    h.backward(s["gh"])
    leaf["x"].grad += s["gx"]
    z.backward(leaf["x"].grad.detach())
    return {"d" + n: leaf[n].grad if leaf[n] is not None else None for n in names}
