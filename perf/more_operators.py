"""The selective state space scan, its short causal convolution and gradient clipping, measured: real work
over the range a user meets.

A case is a dict of plain values; ``kind`` says which call it is.

``conv``        the short causal convolution over sequences, from carried inputs and returning them
``conv_train``  the convolution forward and backward, every gradient returned
``scan``        the selective scan over sequences (or single tokens) from a carried state, returning it
``scan_train``  the scan forward and backward, every gradient returned
``clip``        the global norm of a model's gradients, and the gradients scaled to a largest norm

With ``own`` false, ``run`` computes them from elementary torch operations in float32 (sums over a whole
model in float64); with ``own`` true it makes the framework's calls.
"""
import math

import torch

own = False

CHUNK = 64  # tokens a chunk of the plain scan
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_NORM = 1.0
EPS = 1e-6


def listed():
    return [
        # one token for 256 streams of a layer: the convolution's carried inputs through memory
        dict(name="conv-decode", kind="conv", B=256, T=1, C=4096, K=4, dtype="bf16", ragged=False),
        # prompts of unequal length, an odd longest one
        dict(name="conv-ragged", kind="conv", B=6, T=1501, C=4096, K=4, dtype="bf16", ragged=True),
        # a training layer at the benchmark's size
        dict(name="conv-train", kind="conv_train", B=8, T=1024, C=4096, K=4, dtype="bf16", ragged=False),
        # a small training run in float32, an odd width and length, three taps
        dict(name="conv-train-odd", kind="conv_train", B=2, T=333, C=1001, K=3, dtype="f32", ragged=True),
        # a small served model: one token for each of four streams, where the launch is what counts
        dict(name="scan-decode-small", kind="scan", B=4, T=1, C=768, G=1, N=16, dtype="bf16", ragged=False),
        # one token for 256 streams: the states' trip through memory
        dict(name="scan-decode-256", kind="scan", B=256, T=1, C=4096, G=1, N=16, dtype="bf16", ragged=False),
        # prompts of unequal length read into states
        dict(name="scan-ragged", kind="scan", B=6, T=1501, C=4096, G=1, N=16, dtype="bf16", ragged=True),
        # one long document: few channels for the card, many tokens
        dict(name="scan-long", kind="scan", B=1, T=32768, C=4096, G=1, N=16, dtype="bf16", ragged=False),
        # a training layer at the benchmark's size
        dict(name="scan-train", kind="scan_train", B=8, T=1024, C=4096, G=1, N=16, dtype="bf16", ragged=False),
        # a small training run in float32: two groups, short states, an odd length, ragged rows
        dict(name="scan-train-odd", kind="scan_train", B=2, T=333, C=1002, G=2, N=8, dtype="f32", ragged=True),
        # the gradients of two small layers: launches
        dict(name="clip-small", kind="clip", layers=2, C=64, rows=256, dtype="f32"),
        # the gradients of a model of 24 layers of 2048 channels: matrices in bfloat16, vectors in float32
        dict(name="clip-model", kind="clip", layers=24, C=2048, rows=32768, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv", "conv_train", "scan", "scan", "scan_train", "scan_train", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "clip":
        C = _log(rng, 32, 2048)
        return dict(kind=kind, layers=_log(rng, 1, 24), C=C, rows=_log(rng, 64, 32768), dtype=dtype)
    decode = not kind.endswith("train") and rng.random() < 0.35
    T = rng.choice([1, 1, 2, 5, 8]) if decode else _log(rng, 17, 2048 if kind.endswith("train") else 16384)
    groups = rng.choice([1, 1, 1, 2, 4])
    C = groups * _log(rng, 48, 4096 // groups)
    if rng.random() < 0.6:
        C = max(groups * 16, C // (groups * 16) * (groups * 16))
    if kind.startswith("conv"):
        B = _log(rng, 1, 256 if decode else max(1, min(16, (1 << 25) // (T * C))))
        return dict(kind=kind, B=B, T=T, C=C, K=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    ragged=not decode and rng.random() < 0.5)
    N = rng.choice([8, 16, 16, 32])
    B = _log(rng, 1, 256 if decode else max(1, min(16, (1 << 29) // (T * C * N))))
    return dict(kind=kind, B=B, T=T, C=C, G=groups, N=N, dtype=dtype, ragged=not decode and rng.random() < 0.5)


def _lengths(case):
    """The tokens of each row: the case's own, so that its work is known."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T - (b * T) // (2 * B) if b else T for b in range(B)]


def _tensors(case):
    """(shape, dtype) of the gradients of a model: an embedding, and per layer the projections around the
    convolution and the scan and their vectors, which are float32."""
    C, dt = case["C"], DTYPES[case["dtype"]]
    E, R, N = 2 * C, max(1, C // 16), 16
    f4 = torch.float32
    layer = [((C,), f4), ((2 * E, C), dt), ((4, E), f4), ((E,), f4), ((R + 2 * N, E), dt), ((E, R), dt), ((E,), f4),
             ((E, N), f4), ((E,), f4), ((C, E), dt)]
    return [((case["rows"], C), dt)] + layer * case["layers"] + [((C,), f4)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=gen, device=dev)  # noqa: E731
    s = dict(case=dict(case))
    if case["kind"] == "clip":
        # the tensors' gradients differ by orders of magnitude, and their norm is several times the largest allowed;
        # as in data-parallel training they lie one behind the other in a buffer for each type
        tensors = _tensors(case)
        each = 8.0 * MAX_NORM / math.sqrt(len(tensors))
        sizes = {dt: sum(math.prod(shape) for shape, d in tensors if d == dt) for _, dt in tensors}
        flat = {dt: torch.empty(n, dtype=dt, device=dev) for dt, n in sizes.items()}
        s["flat_out"] = {dt: torch.empty(n, dtype=dt, device=dev) for dt, n in sizes.items()}
        s["grads"], s["out"], used = [], [], dict.fromkeys(sizes, 0)
        for shape, dt in tensors:
            n, at = math.prod(shape), used[dt]
            s["grads"].append(flat[dt][at:at + n].view(shape))
            s["out"].append(s["flat_out"][dt][at:at + n].view(shape))
            s["grads"][-1].copy_(randn(*shape) * (each * (0.25 + 1.5 * rand(1)) / math.sqrt(n)))
            used[dt] += n
        return s
    B, T, C = case["B"], case["T"], case["C"]
    dt = DTYPES[case["dtype"]]
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    s["x"] = randn(B, T, C).to(dt)
    if case["kind"].startswith("conv"):
        s["weight"] = randn(case["K"], C) / math.sqrt(case["K"])
        s["bias"] = 0.1 * randn(C)
        if case["kind"] == "conv_train":
            s["go"] = randn(B, T, C).to(dt)
        else:
            s["state"] = randn(B, case["K"] - 1, C).to(dt)
            s["state_out"] = torch.empty_like(s["state"])
        return s
    G, N = case["G"], case["N"]
    s["b"], s["c"] = randn(B, T, G * N).to(dt), randn(B, T, G * N).to(dt)
    s["z"] = randn(B, T, C).to(dt)
    # rates of 1 .. N in every channel, steps from 0.001 to 0.1 that the tokens move about
    s["w"] = torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * randn(C, N))
    step = torch.exp(math.log(1e-3) + (math.log(0.1) - math.log(1e-3)) * rand(C))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["dt"] = (0.7 * randn(B, T, C)).to(dt)
    s["d"] = 1.0 + 0.1 * randn(C)
    if case["kind"] == "scan_train":
        s["go"] = randn(B, T, C).to(dt)
    else:
        s["state"] = 0.3 * randn(B, C, N)
        s["state_out"] = torch.empty_like(s["state"])
    return s


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own(s, kind)
    return {"conv": _conv, "conv_train": _conv_train, "scan": _scan, "scan_train": _scan_train, "clip": _clip}[kind](s)


def _own(s, kind):
    from rwkv_wkv_mixing_amd import ops

    c = s["case"]
    if kind == "clip":
        norm = ops.clip_gradients(s["grads"], MAX_NORM, eps=EPS, out=s["out"])
        return dict(norm=norm, grads=list(s["flat_out"].values()))
    if kind == "conv":
        out, state = ops.conv_forward(s["x"], s["weight"], s["bias"], act="silu", lengths=s["lengths"],
                                      state_in=s["state"], state_out=s["state_out"], return_state=True)
        return dict(out=out, state=state)
    if kind == "conv_train":
        out = ops.conv_forward(s["x"], s["weight"], s["bias"], act="silu", lengths=s["lengths"])
        dx, dweight, dbias, _ = ops.conv_backward(s["x"], s["go"], s["weight"], s["bias"], act="silu",
                                                  lengths=s["lengths"])
        return dict(out=out, dx=dx, dweight=dweight, dbias=dbias)
    args = [s[n] for n in ("x", "dt", "w", "b", "c")]
    kw = dict(d=s["d"], z=s["z"], dt_bias=s["dt_bias"], lengths=s["lengths"])
    if kind == "scan":
        out, state = ops.select_forward(*args, state_in=s["state"], state_out=s["state_out"], return_state=True, **kw)
        return dict(out=out, state=state)
    ckpt = ops.new_select_ckpt(c["B"], c["T"], c["C"], c["N"], s["x"].device)
    out = ops.select_forward(*args, ckpt=ckpt, **kw)
    g = ops.select_backward(*args, s["go"], ckpt=ckpt, **kw)
    return dict(out=out, **{n: g[n] for n in ("dx", "ddt", "dw", "db", "dc", "dd", "dz", "ddt_bias")})


# ---- plain forms


def _live(s, T, dev):
    """[B or 1, T, 1]: whether a token is one of its row's."""
    if s["lengths"] is None:
        return torch.ones(1, T, 1, dtype=torch.bool, device=dev)
    return (torch.arange(T, device=dev)[None] < s["lengths"][:, None])[..., None]


def _silu_grad(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _conv_sum(s):
    """The inputs with what came before them, and the convolution's sums."""
    c, x = s["case"], s["x"].float()
    before = s["state"].float() if "state" in s else x.new_zeros(c["B"], c["K"] - 1, c["C"])
    xs = torch.cat([before, x], 1)
    pre = s["bias"].expand_as(x)
    for j in range(c["K"]):
        pre = pre + s["weight"][j] * xs[:, j:j + c["T"]]
    return xs, pre


def _conv(s):
    c = s["case"]
    xs, pre = _conv_sum(s)
    out = torch.where(_live(s, c["T"], xs.device), pre * torch.sigmoid(pre), 0.0)
    # the state after a row of n tokens: rows n .. n + K - 2 of what came before and its tokens
    first = torch.full((c["B"],), c["T"], device=xs.device) if s["lengths"] is None else s["lengths"].long()
    at = first[:, None] + torch.arange(c["K"] - 1, device=xs.device)[None]
    state = torch.gather(xs, 1, at[..., None].expand(-1, -1, c["C"]))
    return dict(out=out.to(s["x"].dtype), state=state.to(s["x"].dtype))


def _conv_train(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    xs, pre = _conv_sum(s)
    live = _live(s, T, xs.device)
    out = torch.where(live, pre * torch.sigmoid(pre), 0.0)
    g = torch.where(live, s["go"].float() * _silu_grad(pre), 0.0)
    after = torch.nn.functional.pad(g, (0, 0, 0, K - 1))
    dx = sum(s["weight"][j] * after[:, K - 1 - j:K - 1 - j + T] for j in range(K))
    dx = torch.where(live, dx, 0.0)
    dweight = torch.stack([(g * xs[:, j:j + T]).sum((0, 1)) for j in range(K)])
    dt = s["x"].dtype
    return dict(out=out.to(dt), dx=dx.to(dt), dweight=dweight, dbias=g.sum((0, 1)))


def _scan_parts(s):
    """By chunks [B, n, L, .]: the steps (zero behind a row's length), what is written (step times input), b and
    c; every chunk's L tokens are walked at once for all the chunks."""
    c = s["case"]
    B, T, G, N = c["B"], c["T"], c["G"], c["N"]
    L = min(CHUNK, T)
    n = -(-T // L)
    chunks = lambda v: torch.nn.functional.pad(v, (0, 0, 0, n * L - T)).view(B, n, L, -1)  # noqa: E731
    raw = s["dt"].float() + s["dt_bias"]
    live = _live(s, T, raw.device)
    delta = torch.where(live, torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), 0.0)
    u = torch.where(live, delta * s["x"].float(), 0.0)
    bc = [chunks(torch.where(live, s[m].float(), 0.0)).view(B, n, L, G, 1, N) for m in ("b", "c")]
    return raw, live, chunks(delta), chunks(u), bc[0], bc[1], L, n


def _per_group(v, G):
    """[B, n, C] -> [B, n, G, C / G, 1], next to states [B, n, G, C / G, N]."""
    return v.view(*v.shape[:2], G, -1, 1)


def _scan_walk(s, want_states):
    c = s["case"]
    B, T, C, G, N = (c[m] for m in ("B", "T", "C", "G", "N"))
    raw, live, delta, u, b, cc, L, n = _scan_parts(s)
    w = s["w"].view(G, C // G, N)
    decay = lambda j: torch.exp(-_per_group(delta[:, :, j], G) * w)  # noqa: E731
    put = lambda j: _per_group(u[:, :, j], G) * b[:, :, j]  # noqa: E731
    first = s["state"].view(B, G, C // G, N) if "state" in s else torch.zeros(B, G, C // G, N, device=raw.device)
    h = torch.empty(B, n, G, C // G, N, device=raw.device)
    if n > 1:  # what each chunk does to a state of zero, then the chunks' start states one after the other
        ends = torch.zeros_like(h)
        for j in range(L):
            ends = decay(j) * ends + put(j)
        whole = torch.exp(-_per_group(delta.sum(2), G) * w)
        for i in range(n):
            h[:, i] = first
            first = whole[:, i] * first + ends[:, i]
    else:
        h[:, 0] = first
    y = torch.empty(B, n, L, C, device=raw.device)
    states = [h] if want_states else None
    for j in range(L):
        h = decay(j) * h + put(j)
        y[:, :, j] = (cc[:, :, j] * h).sum(-1).view(B, n, C)
        if want_states:
            states.append(h)
    y = y.view(B, n * L, C)[:, :T]
    y = y + s["d"] * s["x"].float()
    z = s["z"].float()
    out = torch.where(live, y * z * torch.sigmoid(z), 0.0).to(s["x"].dtype)
    return out, h[:, -1].reshape(B, C, N), y, z, raw, live, delta, u, b, cc, w, decay, states


def _scan(s):
    out, state = _scan_walk(s, False)[:2]
    return dict(out=out, state=state)


def _scan_train(s):
    c = s["case"]
    B, T, C, G, N = (c[m] for m in ("B", "T", "C", "G", "N"))
    out, _, y, z, raw, live, delta, u, b, cc, w, decay, states = _scan_walk(s, True)
    n, L = delta.shape[1:3]
    go, x = s["go"].float(), s["x"].float()
    zero = torch.zeros((), device=x.device)
    gy = torch.where(live, go * z * torch.sigmoid(z), zero)
    dz = torch.where(live, go * y * _silu_grad(z), zero)
    gyc = torch.nn.functional.pad(gy, (0, 0, 0, n * L - T)).view(B, n, L, C)
    read = lambda j: _per_group(gyc[:, :, j], G) * cc[:, :, j]  # noqa: E731
    # the states' gradients: behind each chunk from its own tokens, chunk by chunk from the last, then all of them
    g = torch.zeros(B, n, G, C // G, N, device=x.device)
    if n > 1:
        for j in range(L - 1, -1, -1):
            g = decay(j) * (g + read(j))
        whole = torch.exp(-_per_group(delta.sum(2), G) * w)
        last = torch.zeros_like(g[:, 0])
        local, g = g, torch.empty_like(g)
        for i in range(n - 1, -1, -1):
            g[:, i] = last
            last = whole[:, i] * last + local[:, i]
    du, ddelta = torch.empty_like(gyc), torch.empty_like(gyc)
    db, dc = torch.empty(B, n, L, G, N, device=x.device), torch.empty(B, n, L, G, N, device=x.device)
    dw = torch.zeros(B, n, G, C // G, N, device=x.device)
    for j in range(L - 1, -1, -1):
        gyj, uj, dj = (_per_group(v[:, :, j], G) for v in (gyc, u, delta))
        g = g + cc[:, :, j] * gyj
        dc[:, :, j] = (gyj * states[j + 1]).sum(3)
        db[:, :, j] = (g * uj).sum(3)
        du[:, :, j] = (g * b[:, :, j]).sum(-1).view(B, n, C)
        g = decay(j) * g
        q = g * states[j]
        ddelta[:, :, j] = -(q * w).sum(-1).view(B, n, C)
        dw = dw - q * dj
    line = lambda v: v.reshape(B, n * L, -1)[:, :T]  # noqa: E731
    du, ddelta = line(du), line(ddelta)
    ddt = torch.where(live, (ddelta + du * x) * torch.sigmoid(raw), zero)
    dx = torch.where(live, du * line(delta) + s["d"] * gy, zero)
    dt = s["x"].dtype
    return dict(out=out, dx=dx.to(dt), ddt=ddt.to(dt), dw=dw.sum((0, 1)).view(C, N), db=line(db).to(dt),
                dc=line(dc).to(dt), dd=(gy * x).sum((0, 1)), dz=dz.to(dt), ddt_bias=ddt.sum((0, 1)))


def _clip(s):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
    factor = torch.clamp(MAX_NORM / (norm + EPS), max=1.0).float()
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * factor)
    return dict(norm=norm.float(), grads=list(s["flat_out"].values()))


# ---- work


def work(case):
    size = lambda d: 2 if d == "bf16" else 4  # noqa: E731
    if case["kind"] == "clip":
        n = [(math.prod(shape), dt.itemsize) for shape, dt in _tensors(case)]
        return dict(bytes=sum(2 * k * e for k, e in n), flops=3 * sum(k for k, _ in n))
    B, T, C, e = case["B"], case["T"], case["C"], size(case["dtype"])
    tokens, rows = sum(_lengths(case)), B * T
    if case["kind"] == "conv":
        K = case["K"]
        return dict(bytes=(tokens + rows + 2 * B * (K - 1)) * C * e + (K + 1) * C * 4, flops=tokens * C * (2 * K + 6))
    if case["kind"] == "conv_train":
        K = case["K"]
        return dict(bytes=(2 * tokens + 2 * rows) * C * e + 2 * (K + 1) * C * 4, flops=tokens * C * (8 * K + 21))
    G, N = case["G"], case["N"]
    read = tokens * (3 * C + 2 * G * N) * e + C * (N + 2) * 4  # x, dt, z, b, c and the weights
    if case["kind"] == "scan":
        return dict(bytes=read + rows * C * e + 2 * B * C * N * 4, flops=tokens * C * (7 * N + 20))
    write = rows * (4 * C + 2 * G * N) * e + C * (N + 2) * 4  # out, dx, ddt, dz, db, dc and the weights' gradients
    return dict(bytes=read + tokens * C * e + write, flops=tokens * C * (22 * N + 50))


# ---- the definitions in float64


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "clip":
        total = math.fsum(float((g.double() ** 2).sum()) for g in s["grads"])
        f = min(1.0, MAX_NORM / (math.sqrt(total) + EPS))
        each = [torch.cat([g.double().view(-1) for g in s["grads"] if g.dtype == dt]) * f for dt in s["flat_out"]]
        return dict(norm=torch.tensor(math.sqrt(total), dtype=torch.float64, device=each[0].device), grads=each)
    if case["kind"].endswith("train") and "N" in case and case["B"] * case["T"] * case["C"] * case["N"] * 8 > 40e9:
        return None
    return _exact_conv(s) if case["kind"].startswith("conv") else _exact_scan(s)


def _exact_conv(s):
    """Row by row, each over its own tokens only, by autograd."""
    c = s["case"]
    B, T, C, K = c["B"], c["T"], c["C"], c["K"]
    f8, train = torch.float64, c["kind"] == "conv_train"
    weight, bias = (s[m].to(f8).requires_grad_(train) for m in ("weight", "bias"))
    out = torch.zeros(B, T, C, dtype=f8, device=s["x"].device)
    dx, state = torch.zeros_like(out), []
    for r, n in enumerate(_lengths(c)):
        x = s["x"][r, :n].to(f8).requires_grad_(train)
        before = s["state"][r].to(f8) if "state" in s else x.new_zeros(K - 1, C)
        line = torch.cat([before, x])
        taps = line.unfold(0, K, 1)  # [n, C, K]
        pre = (taps * weight.t()).sum(-1) + bias
        o = pre / (1 + torch.exp(-pre))
        out[r, :n] = o.detach()
        state.append(line[n:])
        if train:
            o.backward(s["go"][r, :n].to(f8))
            dx[r, :n] = x.grad
    if not train:
        return dict(out=out, state=torch.stack(state))
    return dict(out=out, dx=dx, dweight=weight.grad, dbias=bias.grad)


def _exact_scan(s):
    """Token by token: the state decays, the step's input is written in, c reads it out; then the adjoint of
    each of these, last first."""
    c = s["case"]
    B, T, C, G, N = (c[m] for m in ("B", "T", "C", "G", "N"))
    dev, f8, train = s["x"].device, torch.float64, c["kind"] == "scan_train"
    live = torch.ones(B, T, 1, dtype=f8, device=dev)
    for r, n in enumerate(_lengths(c)):
        live[r, n:] = 0
    f = {m: s[m].to(f8) for m in ("x", "dt", "z", "w", "d", "dt_bias")}
    pre = f["dt"] + f["dt_bias"]
    step = torch.logaddexp(pre, torch.zeros_like(pre)) * live
    h = s["state"].to(f8) if "state" in s else torch.zeros(B, C, N, dtype=f8, device=dev)
    y = torch.zeros(B, T, C, dtype=f8, device=dev)
    kept = []
    slab = 256  # tokens whose b and c are spread over the channels at once
    for t in range(T):
        if t % slab == 0 and G > 1:
            bw, cw = (_wide(s[m], t, min(T, t + slab), G, C, N) for m in ("b", "c"))
        bt, ct = ((bw[:, t % slab], cw[:, t % slab]) if G > 1
                  else (s["b"][:, t, None].to(f8), s["c"][:, t, None].to(f8)))
        if train:
            kept.append(h)
        h = torch.exp(-step[:, t, :, None] * f["w"]) * h + (step[:, t] * f["x"][:, t])[..., None] * bt
        y[:, t] = (ct * h).sum(-1)
    y = y + f["d"] * f["x"]
    sig = 1 / (1 + torch.exp(-f["z"]))
    out = y * f["z"] * sig * live
    if not train:
        return dict(out=out, state=h)
    go = s["go"].to(f8) * live
    gy, dz = go * f["z"] * sig, go * y * (sig + f["z"] * sig * (1 - sig))
    dstep, dx = torch.zeros_like(y), torch.zeros_like(y)
    db, dc = (torch.zeros(B, T, G, N, dtype=f8, device=dev) for _ in range(2))
    dw = torch.zeros(C, N, dtype=f8, device=dev)
    grad = torch.zeros(B, C, N, dtype=f8, device=dev)
    grouped = lambda v: v.view(B, G, C // G, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        bt, ct = (s[m][:, t].to(f8).view(B, G, N).repeat_interleave(C // G, 1) for m in ("b", "c"))
        dc[:, t] = grouped(gy[:, t, :, None] * h)
        grad = grad + gy[:, t, :, None] * ct
        db[:, t] = grouped(grad * (step[:, t] * f["x"][:, t])[..., None])
        dput = (grad * bt).sum(-1)
        dx[:, t] = dput * step[:, t] + f["d"] * gy[:, t]
        h = kept[t]
        grad = grad * torch.exp(-step[:, t, :, None] * f["w"])
        dstep[:, t] = dput * f["x"][:, t] - (grad * h * f["w"]).sum(-1)
        dw -= (grad * h * step[:, t, :, None]).sum(0)
    ddt = dstep * live / (1 + torch.exp(-pre))
    flat = lambda v: v.view(B, T, G * N) * live  # noqa: E731
    return dict(out=out, dx=dx * live, ddt=ddt, dw=dw, db=flat(db), dc=flat(dc), dd=(gy * f["x"]).sum((0, 1)), dz=dz,
                ddt_bias=ddt.sum((0, 1)))


def _wide(v, first, last, G, C, N):
    """Tokens first .. last of b or c, one copy for every channel of a group."""
    v = v[:, first:last].to(torch.float64)
    return v.view(v.shape[0], last - first, G, N).repeat_interleave(C // G, 2)
