"""Offsets that decrease or leave the tokens: the rows beside the affected ones are computed as ever."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import accept_ref, check_close, conv_ref, scan_ref
from tests.test_gpu_scan import BF16, DEV, F32, TYPES, _cut, _ints
from tests.test_gpu_scan import Case as ScanCase
from tests.test_gpu_accept import Case as AcceptCase
from tests.test_gpu_short_conv import Case as ConvCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    """Every test here makes rows that are flagged, and nothing else is."""
    gdr.gdr_get_status(clear=True)
    yield
    assert gdr.status_names(gdr.gdr_get_status(clear=True)) == ["BAD_OFFSETS"]


# Offsets, and the call's tokens.  Valid rows have no token in common.
BAD = [([0, 5, 120, 10, 20], 20), ([0, 5, -7, 10, 20], 20), ([300, 400, 0, 100, 200, 300], 400), ([-1, 3, 70, 90, 91], 90),
       ([200, 260, 100, 200, 1000, 0, 100], 260), ([64, 128, 0, 64], 128)]
BAD += [([7 * i for i in range(400, 801)] + [7 * i for i in range(0, 401)], 5600)]  # two halves the wrong way round


def _rows(off, T):
    """(row, begin, end) of the rows that there are."""
    return [(b, lo, hi) for b, (lo, hi) in enumerate(zip(off, off[1:])) if 0 <= lo < hi <= T]


def _apart(off, T, slots):
    """The same rows one behind the other, and where each of their tokens is: (order of tokens, offsets, slots)."""
    rows = _rows(off, T)
    order = [t for _, lo, hi in rows for t in range(lo, hi)]
    ends = [0]
    for _, lo, hi in rows:
        ends.append(ends[-1] + hi - lo)
    return torch.tensor(order, device=DEV), _ints(ends), slots[[b for b, _, _ in rows]]


@pytest.mark.parametrize("off,T", BAD)
@pytest.mark.parametrize("C,tok", [(64, BF16), (33, F32), (2056, BF16)])
@pytest.mark.parametrize("bound", [0, 400])
def test_convolution(off, T, C, tok, bound):
    c = ConvCase([1] * (len(off) - 1), C, 4, tok, seed=1)
    c.x = torch.randn(T, C, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(tok)
    c.off = _ints(off)
    pool, out = c.pool.clone(), torch.zeros_like(c.x)
    gdr.gdr_short_conv(*c.args(pool), out, max_row_len=bound)
    order, ends, slots = _apart(off, T, c.slot)
    want, bound, state = conv_ref(c.x[order], c.w, c.bias, c.pool, slots, ends)
    check_close(out[order], want, bound, "out")
    assert torch.equal(pool, state)
    again = c.pool.clone()
    gdr.gdr_short_conv(*c.args(again), state_only=True)
    assert torch.equal(again, pool)


@pytest.mark.parametrize("off,T", BAD)
@pytest.mark.parametrize("bound", [0, 16])
def test_scan(off, T, bound):
    rows = _rows(off, T)
    if bound and max(hi - lo for _, lo, hi in rows) > bound:
        bound = 400
    c = ScanCase([1] * (len(off) - 1), 1, 2, 16, 32, TYPES[0], seed=3)
    whole = ScanCase([T], 1, 2, 16, 32, TYPES[0], seed=4)
    c.x, c.dt, c.B, c.C, c.z, c.off = whole.x, whole.dt, whole.B, whole.C, whole.z, _ints(off)
    pool, out = c.pool.clone(), torch.zeros_like(c.x)
    c.run(pool, out=out, max_row_len=bound)
    order, ends, slots = _apart(off, T, c.slot)
    want, tol, state, state_tol = scan_ref(c.x[order], c.dt[order], c.A, c.B[order], c.C[order], c.pool, slots, ends, z=c.z[order],
                                           D=c.D, dt_bias=c.bias)
    check_close(out[order], want, tol, "out")
    check_close(pool, state, state_tol, "state")


@pytest.mark.parametrize("types", [TYPES[0], TYPES[2], TYPES[3]])
def test_scan_rows_on_one_another(types):
    """Rows that lie on one another, long enough to be cut: each moves its own slot by all of its tokens."""
    c = ScanCase([2000], 1, 1, 16, 64, types, seed=5)
    pool = torch.cat([c.pool, c.pool])
    c.slot, c.off = _ints([3, 0, 1, 2, 4]), _ints([0, 2000, 0, 1990, 0, 2000])
    if types is not TYPES[3]:  # whose state_only calls are not cut
        assert _cut(c, 2000, 2000)
    got = pool.clone()
    c.run(got, state_only=True, max_row_len=2000)
    for slot, n in ((3, 2000), (1, 1990), (4, 2000)):
        _, _, state, tol = scan_ref(c.x[:n], c.dt[:n], c.A, c.B[:n], c.C[:n], pool, _ints([slot]), _ints([0, n]), z=c.z[:n], D=c.D,
                                    dt_bias=c.bias, cut=2000)
        check_close(got[slot], state[slot], tol[slot], f"state {slot}")
    assert torch.equal(got[[0, 2, 5]], pool[[0, 2, 5]])
    out = torch.empty_like(c.x)
    again = pool.clone()
    c.run(again, out=out, max_row_len=2000)  # what they write where they meet is either's
    assert bool((out.float().abs() < 1e4).all())
    for slot in (3, 1, 4):
        check_close(again[slot], got[slot].double(), 2.0 ** -7 * got[slot].double().abs() + 1e-3, f"state {slot}")


@pytest.mark.parametrize("off,T", [([0, 5, 120, 10, 20], 20), ([8, 16, 0, 8], 16), ([-1, 3, 7, 9], 9)])
def test_verification(off, T):
    c = AcceptCase([T], 300, seed=6)
    n = len(off) - 1
    c.off, c.v = _ints(off), torch.rand(n, generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
    out, counts = gdr.gdr_accept_drafts(*c.args(), max_row_len=10)
    want, number = torch.full((n, 10), -1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    for b, lo, hi in _rows(off, T):
        part, m = accept_ref(c.target[lo:hi], c.draft[lo:hi], c.tokens[lo:hi], _ints([0, hi - lo]), c.u[lo:hi], c.v[b:b + 1], 10)
        want[b], number[b] = part[0], m[0]
    assert out.cpu().tolist() == want.tolist() and counts.cpu().tolist() == number.tolist()
