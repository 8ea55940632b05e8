"""Edges of the delta rule's documented range that the parity tests do not reach."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ops():
    from rwkv_wkv_mixing_amd import ops as O

    return O


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_key_heads_without_value_heads(dtype):
    """H = 0 is a multiple of any HK: o is empty, and dr and dk are empty sums, zeros, and not whatever the
    memory held."""
    O = ops()
    e = lambda *s: torch.empty(s, device=DEV, dtype=dtype)  # noqa: E731
    w = torch.empty(2, 37, 0, device=DEV)
    r = torch.randn(2, 37, 192, device=DEV).to(dtype)
    assert O.delta_forward(w, w, r, r, e(2, 37, 0)).shape == (2, 37, 0)
    junk = [torch.full_like(r, float("nan")) for _ in range(4)]
    del junk  # what the gradients' memory holds
    dr, dk, dv, dw, dbeta, _ = O.delta_backward(w, w, r, r, e(2, 37, 0), e(2, 37, 0))
    assert dr.shape == dk.shape == r.shape and not bool(dr.any()) and not bool(dk.any())
    assert dv.shape == (2, 37, 0) and dw.shape == dbeta.shape == w.shape
    leaves = [t.requires_grad_() for t in (w, r.clone())]
    O.delta_rule(leaves[0], w.detach(), leaves[1], r, e(2, 37, 0))[0].sum().backward()
    assert not bool(leaves[1].grad.any())


U, TWO_TERMS = 2.0 ** -24, 2.0 ** -18


def signs(g, *shape):
    """+-1/8 in 64 channels, as many of each: of length 1 and orthogonal to all ones, both exactly."""
    x = torch.rand(*shape, 64, generator=g).argsort(-1)
    return ((x % 2) * 2 - 1) / 8.0


def held(name, got, ref, mag, c):
    import numpy as np

    g = got.double().cpu().numpy()
    ratio = np.abs(g - ref) / (2.0 ** -8 * np.abs(ref) + c * mag)
    print(f"  {name}: worst err / bound {ratio.max():.3f}, terms cancel by {np.median(mag / (np.abs(ref) + 1e-30)):.0e}", flush=True)
    assert ratio.max() <= 1.0, name


def test_bf16_output_where_its_terms_cancel():
    """o reads a state whose rows are alike through r that is orthogonal to them: the terms cancel by 2^12, and the
    bf16 rounding of what is left hides nothing.  Bound, of the sum of the terms' magnitudes, those of the state
    before the token's pair of blocks and of the pair's own tokens: 2^-18 for each term of the state and 3 2^-18 for
    each of the other block, held to two bf16 terms; and the float32 sums, of N + 32 terms at each of T tokens with
    independent roundings, u sqrt((N + 32) T), eight times that for the largest of all elements."""
    import numpy as np
    from oracle import delta_forward_ref

    T, N = 100, 64
    g = torch.Generator().manual_seed(0)
    r, k, v = signs(g, 1, T), signs(g, 1, T), torch.randn(1, T, N, generator=g).bfloat16().float()
    w, beta = torch.full((1, T, 1), 1e-3), torch.rand(1, T, 1, generator=g)
    S0 = 1000.0 + torch.randn(1, 1, N, N, generator=g)
    host = [t.double().numpy() for t in (w, beta, r, k, v)]
    ref, Sref = delta_forward_ref(*host, 1, S0.double().numpy())
    a, mag, S = np.exp(-host[0][0, :, 0]), np.zeros((T, N)), S0[0, 0].double().numpy()
    for t0 in range(0, T, 32):  # the terms of a pair of blocks
        e, D = [], S
        for t in range(t0, min(t0 + 32, T)):
            D = a[t] * D
            e.append(host[4][0, t] - host[3][0, t] @ D)
            D = D + host[1][0, t, 0] * np.outer(host[3][0, t], e[-1])
            mag[t] = np.abs(host[2][0, t]) @ np.abs(S) + sum(
                abs(host[2][0, t] @ host[3][0, t0 + s]) * host[1][0, t0 + s, 0] * np.abs(e[s]) for s in range(len(e)))
        S = D
    assert np.allclose(S, Sref[0, 0])
    d = [t.to(DEV) for t in (w, beta)] + [t.bfloat16().to(DEV) for t in (r, k, v)]
    o, S1 = ops().delta_forward(*d, state_in=S0.to(DEV), return_state=True)
    eps = U * np.sqrt((N + 32) * T)
    held("o", o[0], ref[0], mag, 3 * TWO_TERMS + 8 * eps)
    assert np.linalg.norm(S1.double().cpu().numpy() - Sref) <= eps * np.linalg.norm(Sref)  # float32 throughout


def test_bf16_gradients_where_their_terms_cancel():
    """Keys and receptances that come with their opposites: dr and dk sum a tile's pairs of tokens that cancel.
    Bound: 2^-18 of each pair's magnitude (two bf16 terms), and the float32 sums of both walks, 2 u sqrt((N + 32) T),
    eight times that for the largest of all elements."""
    import numpy as np
    from oracle import delta_backward_ref

    T, N = 64, 64
    g = torch.Generator().manual_seed(1)
    pairs = lambda x: torch.stack((x, -x), 2).reshape(1, T, N)  # noqa: E731
    r, k = pairs(signs(g, 1, T // 2)), pairs(signs(g, 1, T // 2))
    c = torch.randn(1, 1, N, generator=g).bfloat16().float()
    v, go = 8 * c.expand(1, T, N).contiguous(), c.expand(1, T, N).contiguous()
    w, beta = torch.zeros(1, T, 1), torch.full((1, T, 1), 2.0 ** -12)
    host = [t.double().numpy() for t in (w, beta, r, k, v, go)]
    dr, dk, dv, *_ = delta_backward_ref(*host, 1)
    S, e = np.zeros((N, N)), []
    for t in range(T):
        e.append(host[4][0, t] - host[3][0, t] @ S)
        S = S + 2.0 ** -12 * np.outer(host[3][0, t], e[-1])
    size = lambda x: np.linalg.norm(x, axis=-1)  # noqa: E731
    e, gn, ln, b = size(np.array(e)), size(host[5][0]), size(dv[0]), 2.0 ** -12
    ra, ka = np.abs(host[2][0]), np.abs(host[3][0])
    mr, mk = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        mr[t] = b * gn[t] * (e[:t + 1, None] * ka[:t + 1]).sum(0)
        mk[t] = b * (e[t] * (gn[t:, None] * ra[t:]).sum(0) + e[t] * (ln[t + 1:, None] * ka[t + 1:]).sum(0)
                     + ln[t] * (e[:t, None] * ka[:t]).sum(0))
    d = [t.to(DEV) for t in (w, beta)] + [t.bfloat16().to(DEV) for t in (r, k, v, go)]
    got = ops().delta_backward(*d)
    eps = U * np.sqrt((N + 32) * T)
    held("dr", got[0][0, 1::2], dr[0, 1::2], mr[1::2], TWO_TERMS + 16 * eps)  # behind a whole pair
    held("dk", got[1][0, 1::2], dk[0, 1::2], mk[1::2], TWO_TERMS + 16 * eps)
    held("dr", got[0][0], dr[0], mr, TWO_TERMS + 16 * eps)
    held("dk", got[1][0], dk[0], mk, TWO_TERMS + 16 * eps)


@pytest.mark.parametrize("B,T,HK,H,N", [(16, 130, 16, 32, 64), (11, 130, 10, 20, 128)])
def test_gradient_workgroups_that_walk_many_tiles(B, T, HK, H, N):
    """More (64 tokens, row, key head) places than workgroups of the bf16 gradient kernel (512 at N = 64, 256 at
    N = 128), rows of every length and some of none among them: each row's gradients are bit for bit those of a call
    of that row alone, in which no workgroup takes a second place, and two rows' are the oracle's."""
    import numpy as np
    from oracle import delta_backward_ref

    O = ops()
    assert -(-T // 64) * B * HK > (512 if N == 64 else 256) >= -(-T // 64) * HK
    g = torch.Generator().manual_seed(N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w, beta = torch.rand(B, T, H, generator=g) * 0.3, torch.rand(B, T, H, generator=g)
    k = rn(B, T, HK, N)
    k = (k / k.norm(dim=-1, keepdim=True)).reshape(B, T, HK * N)
    p = [w, beta] + [t.bfloat16() for t in (rn(B, T, HK * N) / N ** 0.5, k, rn(B, T, H * N), rn(B, T, H * N))]
    S0, dS = rn(B, H, N, N), rn(B, H, N, N)
    lens = [T, 0, 64, 1, 65, 129, 128, 0, 63, 17, T, 90, 0, 0, 100, T][:B]
    d = [t.to(DEV) for t in p]
    call = lambda *a, ln, S, G: O.delta_backward(*a, lengths=ln, state_in=S, grad_state_out=G, need_state_grad=True,  # noqa: E731
                                                 split=False)
    ln, S, G = torch.tensor(lens, dtype=torch.int32, device=DEV), S0.to(DEV), dS.to(DEV)
    got = call(*d, ln=ln, S=S, G=G)
    names = ("dr", "dk", "dv", "dw", "dbeta", "dS0")
    for b in range(B):
        want = call(*(t[b:b + 1].contiguous() for t in d), ln=ln[b:b + 1].contiguous(), S=S[b:b + 1], G=G[b:b + 1])
        for n, x, y in zip(names, got, want):
            assert torch.equal(x[b:b + 1], y), (n, b)
    eps = 2 * U * np.sqrt((N + 32) * T)  # of two walks with independent roundings, as the parity tests derive it
    for b in (4, 10):
        *ref, mw, mb = delta_backward_ref(*(t[b:b + 1].double().numpy() for t in p), HK, S0[b:b + 1].double().numpy(),
                                          dS[b:b + 1].double().numpy(), [lens[b]], magnitude=True)
        for n, x, y, size in zip(names, got, ref, (None, None, None, mw, mb, None)):
            half = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
            err = np.abs(x[b:b + 1].double().cpu().numpy() - y)
            size = np.abs(y) if size is None else size
            assert np.linalg.norm(err) <= (eps + half) * np.linalg.norm(size), (n, b)
            assert (err - half * np.abs(y)).max() <= 8 * eps * size.max(), (n, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("T", [9, 150, 700])  # token by token, whole, split in time
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_rows_behind_a_length_are_zeros_whatever_the_state(dtype, N, T, bad):
    """A state or a gradient that is not finite spoils its own row's tokens and nothing behind the row's length."""
    O = ops()
    B, H, HK = 3, 2, 1
    g = torch.Generator().manual_seed(T + N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    lens = [T - 4, T // 2, 1]
    p = [torch.rand(B, T, H, generator=g) * 0.1, torch.rand(B, T, H, generator=g), rn(B, T, HK * N).to(dtype),
         (rn(B, T, HK * N) / (2 * N ** 0.5)).to(dtype), rn(B, T, H * N).to(dtype), rn(B, T, H * N).to(dtype)]
    S, G = rn(B, H, N, N), rn(B, H, N, N)
    S[:2, :, 3, 5] = bad
    G[:2, :, 7, 1] = bad
    d, ln = [t.to(DEV) for t in p], torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(lengths=ln, state_in=S.to(DEV))
    ck = O.new_delta_ckpt(B, T, H, N, DEV)
    outs = [O.delta_forward(*d[:5], **kw), O.delta_forward(*d[:5], ckpt=ck, **kw)]
    for ckpt in (ck, None):
        outs += O.delta_backward(*d, grad_state_out=G.to(DEV), ckpt=ckpt, **kw)[:5]
    for i, x in enumerate(outs):
        for b, n in enumerate(lens):
            assert bool((x[b, n:] == 0).all()), (i, b)
        assert bool(torch.isfinite(x[2]).all()) and not bool(torch.isfinite(x[0, :lens[0]]).all()), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
def test_rates_that_clear_the_state_of_a_split_sequence(dtype, N):
    """Infinite and large rates at the borders of tiles and segments, and a stretch of rates of 0, in a sequence that
    is split in time.  Bounds as the parity tests derive them: u sqrt((N + 32) T), twice that for gradients."""
    import numpy as np
    from oracle import delta_backward_ref, delta_forward_ref

    O, T, H = ops(), 900, 2
    g = torch.Generator().manual_seed(N)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    k = rn(1, T, H, N)
    k = (k / k.norm(dim=-1, keepdim=True)).reshape(1, T, H * N)
    w = torch.rand(1, T, H, generator=g) * 0.1
    w[:, [0, 63, 64, 127, 128, 191, 192, 255, 256, 511, 512, 640, 899]] = float("inf")
    w[:, [100, 320, 448, 700]] = 60.0
    w[:, 400:440] = 0.0
    p = [w, torch.rand(1, T, H, generator=g), (rn(1, T, H * N) / N ** 0.5).to(dtype), k.to(dtype), rn(1, T, H * N).to(dtype),
         rn(1, T, H * N).to(dtype)]
    S, G = rn(1, H, N, N), rn(1, H, N, N)
    assert O.L.lib().wkv_delta_forward_workspace_bytes(1, T, H, H, N) > 0
    host, d = [t.double().numpy() for t in p], [t.to(DEV) for t in p]
    ref = list(delta_forward_ref(*host[:5], H, S.double().numpy()))
    *grads, mw, mb = delta_backward_ref(*host, H, S.double().numpy(), G.double().numpy(), magnitude=True)
    got = [*O.delta_forward(*d[:5], state_in=S.to(DEV), return_state=True),
           *O.delta_backward(*d, state_in=S.to(DEV), grad_state_out=G.to(DEV), need_state_grad=True)]
    eps = U * np.sqrt((N + 32) * T)
    for i, (x, y) in enumerate(zip(got, ref + grads)):
        half, c = 2.0 ** -8 if x.dtype == torch.bfloat16 else U, eps if i < 2 else 2 * eps
        err, size = np.abs(x.double().cpu().numpy() - y), np.abs(y) if i not in (5, 6) else (mw, mb)[i - 5]
        assert np.linalg.norm(err) <= (c + half) * np.linalg.norm(size), i
        assert (err - half * np.abs(y)).max() <= 8 * c * size.max(), i
