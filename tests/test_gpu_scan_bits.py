"""Which bits a row of the selective scan has: float32 tokens move the states of a bfloat16 pool by float32 operations
rounded one by one, and a row's results are the same in whatever form and company it is computed."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import U32, silu_error
from tests.test_gpu_scan import BF16, DEV, F32, TYPES, Case, _clean_status, _cut, _ints  # noqa: F401

pytestmark = pytest.mark.gpu


def _plain(c, pool):
    """One call in float32 operations that are rounded one by one, token by token.  Moves pool; returns (out, bound):
    the readout in float64 from the float32 states, and what the call's float32 sums may be off by."""
    out = torch.zeros(c.x.shape, dtype=torch.float64, device=DEV)
    bound = out.clone()
    r, K = c.A.shape[0] // c.B.shape[1], c.A.shape[1]
    for b, slot in enumerate(c.slot.tolist()):
        lo, hi = int(c.off[b]), int(c.off[b + 1])
        if slot < 0 or hi <= lo:
            continue
        s = pool[slot].float()
        for t in range(lo, hi):
            v = c.dt[t].float() if c.bias is None else c.dt[t].float() + c.bias
            d = v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())) if c.softplus else v
            own = c.B[t].float().repeat_interleave(r, 0)[:, :, None] * (d * c.x[t].float())[:, None, :]
            s = torch.exp(d[:, None, :] * c.A) * s + own
            terms = s.double() * c.C[t].double().repeat_interleave(r, 0)[:, :, None]
            y, a = terms.sum(1), terms.abs().sum(1)
            err = (K + 1) * U32 * a  # a rounding a product and sum
            if c.D is not None:
                skip = c.D.double() * c.x[t].double()
                y, err = y + skip, err + 2 * U32 * (a + skip.abs())
            if c.z is not None:
                z = c.z[t].double()
                gate = z * torch.sigmoid(z)
                err = err * gate.abs() + (silu_error(z) + 2 * U32) * (y * gate).abs()
                y = y * gate
            out[t], bound[t] = y, err + U32 * y.abs() + 1e-38
        pool[slot] = s.to(pool.dtype)
    return out, 1.01 * bound


@pytest.mark.parametrize("lens,bound", [([1] * 9, 1), ([5, 1, 7, 0, 16], 16), ([40, 3, 0, 41], 0), ([2, 17, 1], 0)])
@pytest.mark.parametrize("K,V,nk,nv", [(16, 64, 1, 2), (64, 32, 1, 1), (27, 33, 3, 3), (8, 20, 1, 2), (128, 8, 1, 1)])
def test_float32_tokens_call_after_call(lens, bound, K, V, nk, nv):
    """Call after call on one pool.  A bfloat16 pool rounds what a call leaves: states that differ in their last float32
    bit can become neighbouring bfloat16 values, 2^16 times as far apart, and the next call starts there.  With the
    same bits nothing grows."""
    c = Case(lens, nk, nv, K, V, (F32, F32, BF16), pad=(1,), seed=K + V)
    got, want = c.pool.clone(), c.pool.clone()
    for call in range(6):
        c.x, c.dt = c.x.roll(1, 0), c.dt.roll(1, 0)
        out, _ = c.run(got, max_row_len=bound)
        y, tol = _plain(c, want)
        assert torch.equal(got, want), f"call {call}: {int((got != want).sum())} states differ"
        assert bool(((out.double() - y).abs() <= tol).all()), f"call {call}"


@pytest.mark.parametrize("lens,K,V", [([2500], 16, 64), ([2100, 40, 0, 1900], 16, 24), ([2300], 27, 9), ([1500, 1], 64, 8)])
def test_float32_tokens_bfloat16_pool_long_rows(lens, K, V):
    """Long rows too, whose outputs are computed by segments, with counts and without."""
    c = Case(lens, 1, 1, K, V, (F32, F32, BF16), seed=K)
    assert _cut(c, sum(lens), max(lens))
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    got, want, whole = c.pool.clone(), c.pool.clone(), c.pool.clone()
    for call in range(2):
        out, _ = c.run(got, max_row_len=max(lens))
        same, _ = c.run(whole, max_row_len=max(lens), workspace=none)
        y, tol = _plain(c, want)
        assert torch.equal(got, want) and torch.equal(whole, want)
        assert torch.equal(out, same)
        assert bool(((out.double() - y).abs() <= tol).all())
    counts = [n // 2 for n in lens]
    half, full = c.pool.clone(), c.pool.clone()
    out, _ = c.run(half, counts=counts, max_row_len=max(lens))
    same, _ = c.run(full, counts=counts, max_row_len=max(lens), workspace=none)
    assert torch.equal(out, same) and torch.equal(half, full)
    alone = c.pool.clone()
    c.run(alone, counts=counts, state_only=True, max_row_len=max(lens))
    assert torch.equal(alone, half)
    out, _ = c.run(alone, keep_state=False, max_row_len=max(lens))
    assert torch.equal(alone, half)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("K", [3, 8, 16, 27, 32, 50, 64, 100, 128])
@pytest.mark.parametrize("V", [32, 33])
def test_rows_have_the_same_bits_in_every_form(types, K, V):
    """Rows of up to 16 tokens, by the form for short rows, by chunks, alone, and among so many that blocks share
    their states out another way."""
    lens = [16, 1, 9, 2]
    c = Case(lens, 1, 2, K, V, types, seed=K)
    out, pool = c.run(max_row_len=16)
    by_chunks, state = c.run(max_row_len=0)
    assert torch.equal(out, by_chunks) and torch.equal(pool, state)
    T, copies = sum(lens), 60
    many = c.pool.repeat(copies, 1, 1, 1)
    slot = torch.cat([c.slot + i * c.pool.shape[0] for i in range(copies)])
    off = torch.cat([c.off[:-1] + i * T for i in range(copies)] + [_ints([T * copies])])
    wide = [None if t is None else t.repeat(copies, 1, 1) for t in (c.x, c.dt, c.B, c.C, c.z)]
    for bound in (0, 16):
        moved = many.clone()
        got = gdr.gdr_selective_scan(wide[0], wide[1], c.A, wide[2], wide[3], moved, slot, off, z=wide[4], D=c.D, dt_bias=c.bias,
                                     max_row_len=bound)
        assert torch.equal(got, out.repeat(copies, 1, 1)) and torch.equal(moved, pool.repeat(copies, 1, 1, 1))
    ones = Case([1] * 5, 1, 2, K, V, types, seed=K)
    single, kept = ones.run(max_row_len=1)
    for bound in (0, 2):
        got, state = ones.run(max_row_len=bound)
        assert torch.equal(got, single) and torch.equal(state, kept)
