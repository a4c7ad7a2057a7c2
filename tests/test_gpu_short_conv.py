"""The short causal convolution (gdr_short_conv) against float64: types,
widths, odd sizes, layouts, ragged and padded rows, what it keeps and what it refuses."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import check_close, conv_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    gdr.gdr_get_status(clear=True)
    yield
    st = gdr.gdr_get_status(clear=True)
    assert st == 0, f"device status {gdr.status_names(st)}"


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, lens, C=64, W=4, tok=BF16, pool=F32, bias=True, pad=(), seed=0, gap=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T = sum(lens) + gap
        self.x = torch.randn(T + 3, C, generator=g, device=DEV).to(tok)[:T]
        self.w = torch.randn(C, W, generator=g, device=DEV)
        self.bias = torch.randn(C, generator=g, device=DEV) if bias else None
        slots = len(lens) + 2
        self.pool = torch.randn(slots, C, W - 1, generator=g, device=DEV).to(tok).to(pool) if W > 1 else None
        slot = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:len(lens)]
        slot[list(pad)] = -1
        self.slot = slot.to(torch.int32).to(DEV)
        off = [gap]
        for n in lens:
            off.append(off[-1] + n)
        self.off = _ints(off)
        self.gap = gap

    def args(self, pool):
        return self.x, self.w, self.bias, pool, self.slot, self.off

    def check(self, max_row_len=0, activation="silu", counts=None, keep_state=True, out=None, pool=None):
        pool = (None if self.pool is None else self.pool.clone()) if pool is None else pool
        n = None if counts is None else _ints(counts)
        got = gdr.gdr_short_conv(*self.args(pool), out, activation=activation, counts=n, keep_state=keep_state,
                                 max_row_len=max_row_len)
        want, bound, state = conv_ref(*self.args(self.pool), silu=activation == "silu", counts=counts, keep=keep_state)
        check_close(got[self.gap:], want[self.gap:], bound[self.gap:], "out")
        if pool is not None:
            assert torch.equal(pool, state)
        return got, pool


@pytest.mark.parametrize("tok,pool", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("C", [1, 7, 64, 1032, 2047])
def test_ragged_rows(tok, pool, W, C):
    lens = [1, 70, 0, 2, 64, 3, 129, 1, 1, 4]
    c = Case(lens, C, W, tok, pool, bias=C % 2 == 0, pad=(5,), seed=C + W)
    for bound in (0, 129):
        c.check(bound, activation="silu" if W > 2 else None)


@pytest.mark.parametrize("tok", [BF16, F32])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("longest", [1, 2, 5, 16])
def test_short_rows(tok, W, longest):
    Case([longest, 1, 0, longest, 1], 96, W, tok, F32, pad=(3,), seed=longest).check(longest)


def test_forms_give_the_same_bits():
    """A row's results do not depend on how the call's work is dealt out, nor on what else is in the call."""
    c = Case([5, 1, 3, 16], 264, seed=1)
    by_row, state = c.check(16)
    by_run, other = c.check(0)
    assert torch.equal(by_row, by_run) and torch.equal(state, other)
    pool = c.pool.clone()
    alone = gdr.gdr_short_conv(c.x[9:25], c.w, c.bias, pool, c.slot[3:], _ints([0, 16]))
    assert torch.equal(alone, by_run[9:25]) and torch.equal(pool[c.slot[3]], other[c.slot[3]])


def test_rows_in_two_calls_chain():
    c = Case([40], 64, seed=2, tok=F32)
    whole, state = c.check()
    for cut in (1, 2, 3, 7, 39):
        pool = c.pool.clone()
        a = gdr.gdr_short_conv(c.x[:cut], c.w, c.bias, pool, c.slot, _ints([0, cut]))
        b = gdr.gdr_short_conv(c.x[cut:], c.w, c.bias, pool, c.slot, _ints([0, 40 - cut]))
        assert torch.equal(torch.cat([a, b]), whole) and torch.equal(pool, state)


@pytest.mark.parametrize("bound", [0, 9])
@pytest.mark.parametrize("W", [2, 4])
def test_kept_counts(bound, W):
    """States behind a row's first tokens; 0 and padding leave them; nothing is kept without keep_state."""
    lens, counts = [9, 5, 1, 2, 0, 6, 3], [9, 2, 1, 0, 0, 3, 1]
    c = Case(lens, 40, W, pad=(6,), seed=W)
    c.check(bound, counts=counts)
    out, pool = c.check(bound, keep_state=False)
    assert torch.equal(pool, c.pool)
    # the verify pass, then only the states: as one call with counts
    assert gdr.gdr_short_conv(*c.args(pool), counts=_ints(counts), state_only=True, max_row_len=bound) is None
    assert torch.equal(pool, c.check(bound, counts=counts)[1])


def test_layouts():
    """Strided tokens, weights, states with the taps outermost, an output between other columns, a leading gap."""
    for tok in (BF16, F32):
        c = Case([33, 2, 20], 48, 4, tok, seed=3, gap=5)
        want, state = c.check()
        wide = torch.full((60, 160), 7.0, dtype=tok, device=DEV)
        wide[:, 5:53] = c.x
        c.x = wide[:, 5:53]
        wt = c.w.T.contiguous()
        c.w = wt.T
        pool = c.pool.transpose(1, 2).contiguous().transpose(1, 2)
        out = wide[:, 64:112]  # columns of the same rows
        got, _ = c.check(out=out, pool=pool)
        assert torch.equal(got[5:], want[5:]) and torch.equal(pool, state)
        assert bool((wide[:, :5] == 7).all()) and bool((wide[:, 53:64] == 7).all()) and bool((wide[:, 112:] == 7).all())
        assert bool((out[:5] == 7).all())  # tokens of no row


def test_rows_behind_the_last_stay_as_they_were():
    c = Case([3, 8], 64, seed=4)
    x = torch.cat([c.x, c.x])
    for bound in (0, 8):
        out = torch.full((22, 64), 5.0, dtype=BF16, device=DEV)
        gdr.gdr_short_conv(x, c.w, c.bias, c.pool.clone(), c.slot, c.off, out, max_row_len=bound)
        assert bool((out[11:] == 5.0).all()) and not bool((out[:11] == 5.0).all())


@pytest.mark.parametrize("bound", [0, 8])
def test_problems_the_device_sees(bound):
    c = Case([3, 8, 2, 4], 64, seed=5)
    c.slot[1], c.slot[2] = 99, -2
    pool = c.pool.clone()
    out = gdr.gdr_short_conv(*c.args(pool), max_row_len=bound)
    assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_SLOT"]
    assert not bool(out[3:13].any())
    want, wb, state = conv_ref(c.x, c.w, c.bias, c.pool, _ints([int(c.slot[0]), -1, -1, int(c.slot[3])]), c.off)
    check_close(out, want, wb, "out")
    assert torch.equal(pool, state)
    c = Case([3, 8, 2], 64, seed=6)
    pool = c.pool.clone()
    out = gdr.gdr_short_conv(*c.args(pool), counts=_ints([4, -1, 1]), max_row_len=bound)
    assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_COUNT"]
    want, wb, state = conv_ref(*c.args(c.pool), counts=[0, 0, 1])
    check_close(out, want, wb, "out")
    assert torch.equal(pool, state)
    pool = c.pool.clone()
    out = gdr.gdr_short_conv(*c.args(pool), max_row_len=7 if bound == 0 else 2)
    assert gdr.status_names(gdr.gdr_get_status()) == ["ROW_TOO_LONG"]
    assert not bool(out[3:11].any()) and torch.equal(pool[c.slot[1]], c.pool[c.slot[1]])
    for off in ([0, 3, 2, 13], [-1, 3, 11, 13], [0, 3, 11, 14]):
        gdr.gdr_short_conv(c.x, c.w, c.bias, pool, c.slot, _ints(off), max_row_len=bound and 14)
        assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_OFFSETS"]


def test_not_finite():
    """An infinity or NaN reaches its own channel's next width-1 tokens only."""
    for bad in (float("inf"), float("nan")):
        c = Case([12, 12], 64, seed=7)
        good = gdr.gdr_short_conv(*c.args(c.pool.clone()))
        c.x[3, 5] = bad
        got = gdr.gdr_short_conv(*c.args(c.pool.clone()))
        same = torch.ones_like(got, dtype=torch.bool)
        same[3:7, 5] = False
        assert torch.equal(got[same], good[same])


def test_streams_graphs_and_prepared_calls():
    c = Case([1, 30, 2], 128, seed=8)
    want, state = c.check()
    pool, out = c.pool.clone(), torch.empty_like(c.x)
    call = gdr.prepare_short_conv(*c.args(pool), out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pool, state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        pool.copy_(c.pool)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, state)


def test_nothing_to_do():
    c = Case([], 64)
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    out = torch.ones_like(x)
    gdr.gdr_short_conv(x, c.w, c.bias, c.pool, c.slot, c.off, out)
    assert bool((out == 1).all())
    assert gdr.gdr_short_conv(x[:0], c.w, c.bias, c.pool, _ints([0]), _ints([0, 0])).shape == (0, 64)


def test_many_rows_and_empty_ones():
    lens = [0] * 300 + [2, 0, 0, 1] * 200 + [0] * 300
    Case(lens, 16, 4, F32, seed=9).check()
    Case([1] * 1000, 16, 3, BF16, seed=10).check()


@pytest.mark.parametrize("longest", [1, 3, 6])
@pytest.mark.parametrize("W", [1, 4])
@pytest.mark.parametrize("C", [16, 13])
def test_many_short_rows(longest, W, C):
    """Blocks that take several rows: padding, empty rows and counts among them."""
    lens = [(7 * i) % (longest + 1) if i % 5 == 0 else longest for i in range(4001)]
    c = Case(lens, C, W, BF16, BF16, pad=range(4, 4001, 17), seed=11)
    c.check(longest)
    c.check(longest, counts=[i % (n + 1) for i, n in enumerate(lens)])


def test_refusals():
    c = Case([3, 4], 64)
    a = c.args(c.pool)
    with pytest.raises(gdr.GdrError, match="out lies on x"):
        gdr.gdr_short_conv(*a, c.x)
    with pytest.raises(gdr.GdrError, match="out lies on x"):
        wide = torch.zeros(7, 100, dtype=BF16, device=DEV)
        gdr.gdr_short_conv(wide[:, :64], *a[1:], wide[:, 36:])
    with pytest.raises(ValueError, match="state_only"):
        gdr.gdr_short_conv(*a, torch.empty_like(c.x), state_only=True)
    with pytest.raises(ValueError, match="keep_state"):
        gdr.gdr_short_conv(*a, counts=_ints([1, 1]), keep_state=False)
    with pytest.raises(ValueError, match="conv_state"):
        gdr.gdr_short_conv(c.x, c.w, c.bias, c.pool[:, :, :2], c.slot, c.off)
    with pytest.raises(TypeError):
        gdr.gdr_short_conv(c.x.half(), *a[1:])
    with pytest.raises(ValueError, match="activation"):
        gdr.gdr_short_conv(*a, activation="sigmoid")
    with pytest.raises(ValueError, match="offsets"):
        gdr.gdr_short_conv(*a[:5], c.off[:2])
    with pytest.raises(ValueError, match="unit channel stride"):
        gdr.gdr_short_conv(c.x.T.contiguous().T, *a[1:])
    with pytest.raises(gdr.GdrError, match="width"):
        gdr.gdr_short_conv(c.x, torch.zeros(64, 5, device=DEV), c.bias, torch.zeros(2, 64, 4, device=DEV), c.slot, c.off)
