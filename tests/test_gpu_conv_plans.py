"""The short convolution's plans for large calls (long runs of tokens, several tiles a workgroup): every output and gradient
against the formulas in float64 over whole tensors.

Bounds as in the parity tests (u = 2^-24, P the largest sum of sizes before the activation; an activation's value and slope are
within (2 K + 12)u (1 + P)), but for the weights' sums, whose n terms are added in a thread's tiles, a workgroup's four runs, a
sixteenth of the workgroups and sixteen of these: a term takes as many roundings as those are long."""
import pytest
import torch

from rwkv_wkv_mixing_amd import ops as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def slope(act, v):
    p = torch.sigmoid(v)
    return v * p, p * (1 + v * (1 - p)), p * (1 + v.abs() * (1 - p))


def near(name, got, want, bound):
    rel = 2.0 ** -8 if got.dtype is BF else 2.0 ** -24
    assert bool(torch.isfinite(got).all()), name
    worst = float(((got.double() - want).abs() / (bound * (1 + rel) + rel * want.abs() + 1e-37)).max())
    print(f"  {name}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype,B,T,C,ragged", [
    (BF, 8, 40000, 68, False), (BF, 8, 40000, 67, True), (F32, 5, 30001, 68, True), (F32, 6, 50000, 67, False), (BF, 8, 1024, 4100, False),
    (F32, 8, 1024, 4100, True), (BF, 3, 2001, 4099, True)])
def test_large_plans(dtype, B, T, C, ragged, K):
    torch.manual_seed(T + C + K)
    x, go = (torch.randn(B, T, C, device=DEV).to(dtype) for _ in range(2))
    s0, gs = (torch.randn(B, K - 1, C, device=DEV).to(dtype) for _ in range(2))
    weight, bias = torch.randn(K, C, device=DEV), torch.randn(C, device=DEV)
    lens = torch.tensor([T, 0, 1, T // 2 + 1, T - 1, 2, T, 77][:B], dtype=torch.int32, device=DEV) if ragged else None
    out, s1 = O.conv_forward(x, weight, bias, lengths=lens, state_in=s0, return_state=True)
    dx, dweight, dbias, ds = O.conv_backward(x, go, weight, bias, lengths=lens, state_in=s0, grad_state_out=gs, need_state_grad=True)
    # a row at a time in float64
    w, add = weight.double(), bias.double()
    sums = {n: torch.zeros(K + 1, C, dtype=torch.float64, device=DEV) for n in ("value", "size", "flat")}
    slots = O.L.lib().wkv_conv_backward_workspace_bytes(B, T, C, K) // ((K + 1) * C * 4)
    depth = -(-B * T // (4 * slots)) + 32 + 4 + -(-slots // 16) + 16
    for b in range(B):
        n = T if lens is None else int(lens[b])
        X = torch.cat([s0[b], x[b, :n]]).double()
        assert torch.equal(s1[b], X[n:].to(dtype))
        pre = add + sum(w[j] * X[j:j + n] for j in range(K))
        size = add.abs() + sum((w[j] * X[j:j + n]).abs() for j in range(K))
        P = 1.0 + float(size.max()) if n else 1.0
        a = (2 * K + 12) * U * P
        value, der, der_size = slope("silu", pre)
        near("out", out[b, :n], value, (K + 2) * U * size + a) if n else None
        g = go[b, :n].double()
        dX, mag, flat = (torch.zeros_like(X) for _ in range(3))
        dX[n:] += gs[b].double()
        mag[n:] += gs[b].double().abs()
        flat[n:] += gs[b].double().abs()
        for j in range(K):
            dX[j:j + n] += w[j] * g * der
            mag[j:j + n] += (w[j] * g).abs() * der_size
            flat[j:j + n] += (w[j] * g).abs()
            sums["value"][j] += (g * der * X[j:j + n]).sum(0)
            sums["size"][j] += ((g * X[j:j + n]).abs() * der_size).sum(0)
            sums["flat"][j] += (g * X[j:j + n]).abs().sum(0) * a
        sums["value"][K] += (g * der).sum(0)
        sums["size"][K] += (g.abs() * der_size).sum(0)
        sums["flat"][K] += g.abs().sum(0) * a
        near("dx", dx[b, :n], dX[K - 1:], ((K + 8) * U * mag + a * flat)[K - 1:]) if n else None
        near("dstate", ds[b], dX[:K - 1], ((K + 8) * U * mag + a * flat)[:K - 1])
        assert not bool(out[b, n:].any()) and not bool(dx[b, n:].any())
    bound = (depth + 8) * U * sums["size"] + sums["flat"]
    near("dweight", dweight, sums["value"][:K], bound[:K])
    near("dbias", dbias, sums["value"][K], bound[K])
