"""RWKV-4 WKV time-mixing operator for AMD MI355X (gfx950), with the
receptance gate and the token-shift mix around it, its multi-head matrix-state
forms (RWKV-5, RWKV-6, the gated delta rule) and the norms around those, the
selective scan with its short convolution, and the clipping of gradients.

The compute path is the HIP library librwkv_wkv.so (C ABI in include/wkv.h);
``ops`` is a thin torch binding of it with the same names:

    from rwkv_wkv_mixing_amd import ops
    y = ops.wkv_forward(w, u, k, v)
    dk, dv, dw, du = ops.wkv_backward(w, u, k, v, gy)
    y = ops.wkv_step(w, u, k, v, a, b, p)
    xr_xk_xv = ops.token_shift(mu, x)          # the mixes feeding r, k, v
    x, h = ops.block_join(x, y, pre_w)         # residual sum, norm before the block
    o, state = ops.delta_rule(w, beta, r, k, v)
    o = ops.head_norm_gated(o, weight, None, gate, heads=H)
    x, carried = ops.short_conv(x, filter)
    y, state = ops.selective_scan(x, dt, w, b, c, d, z)
    norm = ops.clip_gradients([p.grad for p in parameters if p.grad is not None], 1.0)

``workloads`` draws the seeded synthetic inputs used by tests and the bench.
"""

__version__ = "0.1.0"
