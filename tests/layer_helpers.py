"""Plain float64 forms of the layer operators (decayed linear attention and
the fused block norms) for the tests, and the error bounds they are held to."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24   # half an ulp of float32, relative
U16 = 2.0 ** -8    # half an ulp of bfloat16, relative (8 significant bits)


def linattn_ref(q, k, v, decay, state, slot_idx, offsets, *, decay_is_log=False, scale=0.0):
    """Token by token in float64, on the inputs' device.  Returns (out, pool,
    out_abs, pool_abs): the values, and the same sums over absolute values,
    which the rounding errors are proportional to."""
    nv, K, V = state.shape[1:]
    r = nv // q.shape[1]
    q, k, v = q.double().repeat_interleave(r, 1), k.double().repeat_interleave(r, 1), v.double()
    lam = decay.double()
    lam = (torch.exp(lam) if decay_is_log else lam)[:, None, None]
    scale = scale if scale > 0 else K ** -0.5
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    pool = state.double().clone()
    out_abs, pool_abs = out.clone(), pool.abs()
    for b, slot in enumerate(slot_idx.tolist()):
        t0, t1 = int(offsets[b]), int(offsets[b + 1])
        if slot < 0:
            continue
        s, a = pool[slot], pool_abs[slot]
        for t in range(t0, t1):
            s = lam * s + k[t][:, :, None] * v[t][:, None, :]
            a = lam * a + (k[t][:, :, None] * v[t][:, None, :]).abs()
            out[t] = scale * (q[t][:, :, None] * s).sum(1)
            out_abs[t] = scale * (q[t][:, :, None].abs() * a).sum(1)
        pool[slot], pool_abs[slot] = s, a
    return out, pool, out_abs, pool_abs


def check_linattn(got_out, got_pool, ref, max_len, tensor_cores):
    """|error| <= (roundings on the way) x (sum of absolute values) + the last rounding.

    float32 sums: each of the row's max_len updates rounds twice (the decay
    multiply and the add), the readout adds up K <= 128 products: under
    2 max_len + 140 roundings of at most U32 of the absolute sum each, and the
    decay's powers as many again.  The chunked form rounds the score matrix
    to bfloat16 once, and the start state in two bfloat16 halves (U16^2)."""
    out, pool, out_abs, pool_abs = ref
    n = 4 * max_len + 160
    scores = U16 + U16 * U16 if tensor_cores else 0.0
    last = U16 if got_out.dtype == torch.bfloat16 else 0.0
    tol = (n * U32 + scores) * out_abs * (1 + last) + last * out.abs() + 1e-37
    err = (got_out.double() - out).abs()
    assert bool((err <= tol).all()), f"out: {float((err / tol).max()):.3g} x the bound"
    last = U16 if got_pool.dtype == torch.bfloat16 else 0.0
    tol = n * U32 * pool_abs * (1 + last) + last * pool.abs() + 1e-37
    err = (got_pool.double() - pool).abs()
    assert bool((err <= tol).all()), f"state: {float((err / tol).max()):.3g} x the bound"
    if out.numel() >= 4096 and got_out.dtype == torch.bfloat16:
        # independent roundings of the scores and of the output, rms U16 / sqrt(3) each: under U16 together
        rel = float((got_out.double() - out).norm() / out.norm())
        assert rel <= U16, f"out: relative error {rel:.3g}"


def norm_ref(x, *, gate=None, act=None, gate_first=False, post=False, post_w=None, residual=None, scale=1.0,
             pre=False, pre_w=None, eps=1e-6, centered=False):
    """(h, out) in float64: include/gdr.h, gdr_norm_args."""
    def norm(u, w):
        if centered:
            u = u - u.mean(-1, keepdim=True)
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
        return u if w is None else u * w.double()

    u = None if x is None else x.double()
    if gate is not None:
        g = gate.double()
        g = {None: g, "silu": g * torch.sigmoid(g), "sigmoid": torch.sigmoid(g)}[act]
        if gate_first:
            u = u * g
    if post:
        u = norm(u, post_w)
    if gate is not None and not gate_first:
        u = u * g
    h = u if residual is None else residual.double() + (0.0 if u is None else scale * u)
    return h, norm(h, pre_w) if pre else h
