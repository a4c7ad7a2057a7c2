"""Plain float64 forms of the state space operators (short convolution,
selective scan) and of the verification of drafts, with bounds on what float32
arithmetic may be off by."""
from __future__ import annotations

from fractions import Fraction

import torch

U32 = 2.0 ** -24   # half an ulp of float32, relative
U16 = 2.0 ** -8    # half an ulp of bfloat16, relative (8 significant bits)


def last_rounding(dtype):
    """(relative, absolute) error of the last rounding; the absolute one where values leave the normal range."""
    return (U16, 1e-38) if dtype == torch.bfloat16 else (U32, 1e-38)


def silu_error(z):
    """Relative error of z / (1 + e^-z) by the fast exponential and division: the exponential's argument is rounded
    twice (z log2 e), its power is good to 2 ulp and 2^-22, the sum rounds once, the division is good to 2 ulp."""
    return (2 * z.abs() + 12) * U32


def conv_ref(x, weight, bias, state, slot_idx, offsets, *, silu=True, counts=None, keep=True):
    """(out, bound, state): float64 values, what float32 arithmetic may be off by, and the new state (exact)."""
    T, C = x.shape
    W = weight.shape[1]
    out = torch.zeros(T, C, dtype=torch.float64, device=x.device)
    bound = out.clone()
    new = None if state is None else state.clone()
    w, b = weight.double(), (torch.zeros(C, dtype=torch.float64, device=x.device) if bias is None else bias.double())
    for r, slot in enumerate(slot_idx.tolist()):
        lo, hi = int(offsets[r]), int(offsets[r + 1])
        if slot < 0 or hi <= lo:
            continue
        old = x[:0].double() if W == 1 else state[slot].double().T
        seen = torch.cat([old, x[lo:hi].double()])
        n = hi - lo
        y, a = b.expand(n, C).clone(), b.abs().expand(n, C).clone()
        for m in range(W):
            y += seen[m:m + n] * w[:, m]
            a += (seen[m:m + n] * w[:, m]).abs()
        err = W * U32 * a  # a rounding of the running sum a tap
        if silu:
            # the slope of y / (1 + e^-y) is at most 1.1
            s = y * torch.sigmoid(y)
            err = 1.1 * err + silu_error(y) * s.abs()
            y = s
        out[lo:hi], bound[lo:hi] = y, err
        kept = n if counts is None else int(counts[r])
        if keep and W > 1 and 0 < kept <= n:
            new[slot] = seen[kept:kept + W - 1].T.to(state.dtype)
    return out, bound, new


def check_close(got, want, bound, what):
    rel, least = last_rounding(got.dtype)
    tol = bound * (1 + rel) + rel * want.abs() + least
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.3g} x the bound"


def scan_ref(x, dt, A, B, C, state, slot_idx, offsets, *, D=None, z=None, dt_bias=None, softplus=True, counts=None, keep=True,
             cut=0):
    """(out, bound, state, state bound) in float64, token by token.

    The bound follows the roundings: a decay exp(e), e = d A, is off by what its
    exponent is (d and A log2 e carry 8 roundings, the product one, and the sum of d
    over a segment of `cut` tokens as many as it has terms) and by the exponential's own
    2^-22 and a rounding of the state; a token's own d x B by 12 roundings (softplus: 8)."""
    nv, K, V = state.shape[1:]
    r = nv // B.shape[1]
    dev = x.device
    out = torch.zeros(x.shape, dtype=torch.float64, device=dev)
    bound = out.clone()
    new = state.double().clone()
    new_bound = torch.zeros_like(new)
    Ad = A.double()
    B, C = B.double().repeat_interleave(r, 1), C.double().repeat_interleave(r, 1)
    for b, slot in enumerate(slot_idx.tolist()):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        if slot < 0:
            continue
        s = state[slot].double()
        a, e = s.abs(), torch.zeros_like(s)
        kept = hi - lo if counts is None else int(counts[b])
        kept = kept if 0 <= kept <= hi - lo else 0
        for t in range(lo, hi):
            v = dt[t].double() + (0 if dt_bias is None else dt_bias.double())
            d = torch.logaddexp(v, torch.zeros_like(v)) if softplus else v
            xt = x[t].double()
            ex = d[:, None, :] * Ad
            p = torch.exp(ex)
            new_term = (d * xt)[:, None, :] * B[t][:, :, None]
            e = p * (e + ((9 + cut) * ex.abs() + 6) * U32 * a) + 12 * U32 * new_term.abs()
            a = p * a + new_term.abs()
            s = p * s + new_term
            y = (s * C[t][:, :, None]).sum(1)
            ya = (a * C[t][:, :, None].abs()).sum(1)
            ye = (e * C[t][:, :, None].abs()).sum(1) + (K + 2) * U32 * ya
            if D is not None:
                y = y + D.double() * xt
                ye = ye + U32 * (ya + (D.double() * xt).abs())
            if z is not None:
                zt = z[t].double()
                gate = zt * torch.sigmoid(zt)
                ye = ye * gate.abs() + (silu_error(zt) + U32) * (y * gate).abs()
                y = y * gate
            out[t], bound[t] = y, ye
            if keep and t + 1 - lo == kept:
                new[slot], new_bound[slot] = s, e + U32 * a
    return out, bound, new, new_bound


def accept_ref(target, draft, tokens, offsets, uniforms, row_uniforms, width):
    """(tokens, counts) by the rule, in rational numbers."""
    p = target.double().cpu().tolist()
    q = None if draft is None else draft.double().cpu().tolist()
    ids, off = tokens.tolist(), offsets.tolist()
    u, v = uniforms.double().tolist(), row_uniforms.double().tolist()
    vocab = target.shape[1]

    def clean(value):
        return Fraction(value) if 0 < value < float("inf") else Fraction(0)

    out, counts = [], []
    for b in range(len(off) - 1):
        lo, hi = off[b], off[b + 1]
        if hi == lo or hi - lo > width:
            out.append([-1] * width)
            counts.append(0)
            continue
        t, refused = lo, None
        while t + 1 < hi and 0 <= ids[t + 1] < vocab:
            d = ids[t + 1]
            chance = Fraction(1) if q is None else clean(q[t][d])
            number = u[t]
            if not (abs(number) < float("inf") and Fraction(number) * chance < clean(p[t][d])):
                refused = d
                break
            t += 1
        w = [clean(value) for value in p[t]]
        if refused is not None:
            if q is None:
                rest = [0 if i == refused else value for i, value in enumerate(w)]
            else:
                rest = [max(value - clean(o), Fraction(0)) for value, o in zip(w, q[t])]
            if any(rest):
                w = rest
        total = sum(w)
        share = Fraction(min(v[b], 1.0)) * total if v[b] > 0 else Fraction(0)
        drawn, run = -1, Fraction(0)
        for i, value in enumerate(w):
            if value:
                drawn = i
                run += value
                if run > share:
                    break
        out.append(ids[lo + 1:t + 1] + [drawn] + [-1] * (width - (t - lo) - 1))
        counts.append(t - lo + 1)
    return torch.tensor(out, dtype=torch.int32).view(len(out), width), torch.tensor(counts, dtype=torch.int32)
