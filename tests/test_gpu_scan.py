"""The selective scan (gdr_selective_scan) against the recurrence in float64:
types, head layouts, numbers of states, odd sizes, cut rows, what it keeps, refusals."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import check_close, scan_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16, F32), (BF16, F32, BF16), (F32, F32, F32), (F32, F32, BF16), (BF16, F32, F32), (BF16, BF16, BF16)]


@pytest.fixture(autouse=True)
def _clean_status():
    gdr.gdr_get_status(clear=True)
    yield
    st = gdr.gdr_get_status(clear=True)
    assert st == 0, f"device status {gdr.status_names(st)}"


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, lens, nk=1, nv=2, K=16, V=64, types=(BF16, BF16, F32), pad=(), seed=0, gap=0, skip=True, gate=True,
                 bias=True, softplus=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        tok, dt, pool = types
        T = sum(lens) + gap

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=DEV)

        def uniform(*shape):
            return torch.rand(*shape, generator=g, device=DEV)

        self.x = normal(T, nv, V).to(tok)
        self.z = normal(T, 2, nv, V)[:, 1].to(tok) if gate else None
        # step sizes of 0.001 to 1, as they come or by their softplus
        middle = torch.exp(-6.9 * uniform(nv, V))
        self.bias = (torch.log(torch.expm1(middle)) if softplus else middle) if bias else None
        self.dt = ((normal(T, nv, V) if softplus else uniform(T, nv, V)) * (0.5 if bias else 1.0)).to(dt)
        bc = normal(T, 2 * nk * K).to(tok)
        self.B, self.C = bc[:, :nk * K].view(T, nk, K), bc[:, nk * K:].view(T, nk, K)
        self.A = -torch.exp(2.8 * uniform(nv, K, V))
        self.D = normal(nv, V) if skip else None
        slots = len(lens) + 2
        self.pool = normal(slots, nv, K, V).to(pool)
        slot = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:len(lens)]
        slot[list(pad)] = -1
        self.slot = slot.to(torch.int32).to(DEV)
        off = [gap]
        for n in lens:
            off.append(off[-1] + n)
        self.off = _ints(off)
        self.gap, self.softplus = gap, softplus

    def args(self, pool):
        return self.x, self.dt, self.A, self.B, self.C, pool, self.slot, self.off

    def more(self):
        return {"D": self.D, "z": self.z, "dt_bias": self.bias}

    def run(self, pool=None, counts=None, **kw):
        pool = self.pool.clone() if pool is None else pool
        out = gdr.gdr_selective_scan(*self.args(pool), **self.more(), dt_softplus=self.softplus,
                                     counts=None if counts is None else _ints(counts), **kw)
        return out, pool

    def check(self, max_row_len=0, counts=None, cut=0, **kw):
        got, pool = self.run(counts=counts, max_row_len=max_row_len, **kw)
        want, bound, state, state_bound = scan_ref(*self.args(self.pool), **self.more(), softplus=self.softplus, counts=counts,
                                                   keep=kw.get("keep_state", True), cut=cut)
        check_close(got[self.gap:], want[self.gap:], bound[self.gap:], "out")
        check_close(pool, state, state_bound, "state")
        moved = set(int(s) for s, n in zip(self.slot, self.off[1:] - self.off[:-1]) if s >= 0 and n > 0)
        for s in range(pool.shape[0]):
            assert s in moved or torch.equal(pool[s], self.pool[s]), f"slot {s} is nobody's"
        return got, pool


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("K,V,nk,nv", [(16, 64, 1, 2), (8, 128, 2, 4), (16, 40, 3, 3), (32, 32, 1, 1), (64, 16, 2, 2),
                                       (128, 8, 1, 3), (27, 33, 2, 2), (1, 1, 1, 5), (5, 173, 1, 1), (100, 7, 1, 2)])
@pytest.mark.parametrize("one", [False, True])
def test_types_and_heads(types, K, V, nk, nv, one):
    lens = [1] * 5 if one else [1, 16, 0, 17, 15, 3, 40, 2]
    Case(lens, nk, nv, K, V, types, pad=(3,), seed=K + V).check(1 if one else 0)


@pytest.mark.parametrize("longest", [1, 2, 8, 16, 33])
@pytest.mark.parametrize("types", TYPES[:2])
def test_bounded_rows(types, longest):
    Case([longest, 1, 0, max(1, longest - 1), 1], 2, 4, 16, 64, types, pad=(4,), seed=longest).check(longest)


@pytest.mark.parametrize("K,V,nk,nv", [(16, 128, 1, 8), (12, 20, 2, 6), (24, 36, 1, 9), (20, 8, 1, 4), (128, 64, 1, 2), (7, 11, 1, 30)])
@pytest.mark.parametrize("longest", [1, 3])
def test_many_short_rows(K, V, nk, nv, longest):
    """Blocks that take several rows: padding, empty rows and counts among them."""
    lens = [(7 * i) % (longest + 1) if i % 5 == 0 else longest for i in range(333)]
    c = Case(lens, nk, nv, K, V, TYPES[1], pad=range(4, 333, 17), seed=K)
    c.check(longest)
    counts = [i % (n + 1) for i, n in enumerate(lens)]
    _, pool = c.check(longest, counts=counts)
    again = c.pool.clone()
    assert c.run(again, counts=counts, state_only=True, max_row_len=longest)[0] is None
    assert torch.equal(again, pool)


def test_rows_around_the_longest_short_one():
    """16 tokens go one by one, 17 in chunks; both take counts and leave the same kind of state."""
    for longest in (16, 17):
        c = Case([longest, 1, 0, longest - 1], 1, 2, 16, 32, TYPES[0], seed=longest)
        c.check(longest)
        c.check(longest, counts=[longest - 3, 1, 0, 2])


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("V", [32, 31])
def test_parts(skip, gate, bias, softplus, V):
    for lens, bound in (([20, 3], 0), ([1, 1, 1], 1)):
        Case(lens, 1, 2, 16, V, TYPES[2], skip=skip, gate=gate, bias=bias, softplus=softplus, seed=1).check(bound)


def test_rows_do_not_depend_on_their_call():
    c = Case([1, 30, 5], 1, 2, 16, 64, seed=2)
    out, pool = c.run()
    for b, (lo, hi) in enumerate([(0, 1), (1, 31), (31, 36)]):
        alone = c.pool.clone()
        part = {n: None if t is None else t[lo:hi] for n, t in (("x", c.x), ("dt", c.dt), ("B", c.B), ("C", c.C), ("z", c.z))}
        got = gdr.gdr_selective_scan(part["x"], part["dt"], c.A, part["B"], part["C"], alone, c.slot[b:b + 1], _ints([0, hi - lo]),
                                     z=part["z"], D=c.D, dt_bias=c.bias)
        assert torch.equal(got, out[lo:hi]) and torch.equal(alone[c.slot[b]], pool[c.slot[b]])


def test_rows_in_two_calls_chain():
    c = Case([37], 1, 1, 16, 32, TYPES[2], seed=3)
    whole, state = c.run()
    for cut in (1, 15, 16, 17, 36):
        pool, outs = c.pool.clone(), []
        for lo, hi in ((0, cut), (cut, 37)):
            outs.append(gdr.gdr_selective_scan(c.x[lo:hi], c.dt[lo:hi], c.A, c.B[lo:hi], c.C[lo:hi], pool, c.slot, _ints([0, hi - lo]),
                                               z=c.z[lo:hi], D=c.D, dt_bias=c.bias))
        assert torch.equal(torch.cat(outs), whole) and torch.equal(pool, state)


@pytest.mark.parametrize("K,V", [(16, 32), (16, 33), (64, 8)])
@pytest.mark.parametrize("bound", [0, 40])
def test_kept_counts(K, V, bound):
    lens, counts = [40, 5, 1, 2, 0, 16, 17, 3], [33, 5, 1, 0, 0, 16, 2, 2]
    c = Case(lens, 1, 2, K, V, TYPES[1], pad=(7,), seed=4)
    c.check(bound, counts=counts)
    out, pool = c.check(bound, keep_state=False)
    assert torch.equal(pool, c.pool)
    got, _ = c.run(pool=pool, counts=counts, state_only=True, max_row_len=bound)
    assert got is None and torch.equal(pool, c.run(counts=counts)[1])
    # what is not counted is not read
    c.x[33:40], c.dt[33:40], c.B[33:40] = float("nan"), float("nan"), float("nan")
    again = c.pool.clone()
    c.run(pool=again, counts=counts, state_only=True, max_row_len=bound)
    assert torch.equal(again, pool)


def _cut(c, T, bound):
    """Whether the call is cut into segments: it then asks for a workspace."""
    return gdr.gdr_selective_scan_workspace_bytes(*c.args(c.pool), max_row_len=bound) > 0


@pytest.mark.parametrize("types", [TYPES[0], TYPES[3], TYPES[1]])
@pytest.mark.parametrize("lens,K,V", [([2500], 16, 64), ([2100, 40, 0, 1900], 16, 24), ([2300], 27, 9), ([1500, 1], 64, 8)])
def test_cut_rows(types, lens, K, V):
    c = Case(lens, 1, 1, K, V, types, seed=K)
    bound = max(lens)
    assert _cut(c, sum(lens), bound)
    c.check(bound, cut=2500)
    # the same row without a workspace is not cut
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    whole, state = c.run(max_row_len=bound, workspace=none)
    want, wb, ws, wsb = scan_ref(*c.args(c.pool), **c.more())
    check_close(whole, want, wb, "out")
    check_close(state, ws, wsb, "state")


def test_cut_rows_with_counts_padding_and_problems():
    c = Case([2000, 1800, 2200, 30], 1, 1, 16, 32, TYPES[1], pad=(1,), seed=6)
    assert _cut(c, 6030, 2200)
    counts = [1999, 7, 1024, 30]
    c.check(2200, counts=counts, cut=2200)
    out, pool = c.run(max_row_len=2200, keep_state=False)
    assert torch.equal(pool, c.pool)
    c.run(pool=pool, counts=counts, state_only=True, max_row_len=2200)
    want = scan_ref(*c.args(c.pool), **c.more(), counts=counts, cut=2200)
    check_close(pool, want[2], want[3], "state")
    c.slot[0], c.slot[3] = 77, -5
    pool = c.pool.clone()
    out, _ = c.run(pool=pool, max_row_len=2100, counts=[5, 5, 5000, 5])
    assert sorted(gdr.status_names(gdr.gdr_get_status())) == ["BAD_SLOT", "ROW_TOO_LONG"]
    assert not bool(out.any()) and torch.equal(pool, c.pool)
    for off in ([0, 3000, 2000, 6000, 6030], [-1, 2000, 3800, 6000, 6030], [0, 2000, 3800, 6000, 6031]):
        c.off = _ints(off)
        c.slot = _ints([0, 1, 2, 3])
        c.run(pool=pool)
        assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_OFFSETS"]


@pytest.mark.parametrize("bound", [0, 1])
def test_problems_the_device_sees(bound):
    lens = [1, 1, 1, 1, 1] if bound else [3, 20, 2, 4, 5]
    c = Case(lens, 1, 2, 16, 32, TYPES[2], seed=7)
    c.slot[1], c.slot[2] = 99, -2
    out, pool = c.run(max_row_len=bound, counts=[1, 1, 1, -1, 9])
    assert sorted(gdr.status_names(gdr.gdr_get_status())) == ["BAD_COUNT", "BAD_SLOT"]
    live = c.slot.clone()
    live[1:3] = -1
    want, wb, state, sb = scan_ref(*c.args(c.pool)[:6], live, c.off, **c.more(), counts=[1, 0, 0, -1, 9])
    check_close(out, want, wb, "out")
    check_close(pool, state, sb, "state")
    T = sum(lens)
    c.slot = _ints([0, 1, 2, 3, 4])
    off = c.off.tolist()
    for bad in ([0, 2, 1] + off[3:], [-1] + off[1:], off[:5] + [T + 1]):
        c.off = _ints(bad)
        c.run(max_row_len=bound and 40)
        assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_OFFSETS"]
    c.off = _ints(off)
    if not bound:
        out, pool = c.run(max_row_len=19)
        assert gdr.status_names(gdr.gdr_get_status()) == ["ROW_TOO_LONG"]
        assert not bool(out[3:23].any()) and torch.equal(pool[1], c.pool[1]) and bool(out[:3].any())


def test_layouts():
    """Strided and misaligned tokens, shared step sizes and rates, strided pools and outputs, a leading gap."""
    for tok, V in ((BF16, 32), (F32, 32), (F32, 20)):
        c = Case([20, 1, 5], 2, 4, 16, V, (tok, tok, F32), seed=8, gap=3)
        want, state = c.check()
        T, n = c.x.shape[0], 4 * V
        for shift in (0, 8, 1):
            wide = torch.full((T, 5 * n + 80), 7.0, dtype=tok, device=DEV)
            parts = {}
            for i, (name, t) in enumerate((("x", c.x), ("dt", c.dt), ("z", c.z))):
                parts[name] = wide[:, i * n + shift:(i + 1) * n + shift].view(T, 4, V)
                parts[name].copy_(t)
            bc = torch.zeros(T, 2, 2, 24, dtype=tok, device=DEV)
            bc[:, 0, :, shift:16 + shift], bc[:, 1, :, shift:16 + shift] = c.B, c.C
            out = wide[:, 4 * n + 16 + shift:5 * n + 16 + shift].view(T, 4, V)
            pool = torch.zeros(c.pool.shape[0], 4, 18, V + 8, device=DEV)[:, :, 1:17, :V]
            pool.copy_(c.pool)
            got = gdr.gdr_selective_scan(parts["x"], parts["dt"], c.A, bc[:, 0, :, shift:16 + shift], bc[:, 1, :, shift:16 + shift],
                                         pool, c.slot, c.off, out, z=parts["z"], D=c.D, dt_bias=c.bias)
            assert got is out and torch.equal(out[3:], want[3:]) and torch.equal(pool, state)
            assert bool((out[:3] == 7).all()) and bool((wide[:, 3 * n + shift:4 * n + 16 + shift] == 7).all())
            assert bool((wide[:, 5 * n + 16 + shift:] == 7).all())
    # one step size, rate, skip and bias a head
    c = Case([20, 1, 5], 1, 3, 16, 24, TYPES[2], seed=9)
    c.dt, c.A = c.dt[:, :, :1].expand(-1, -1, 24), c.A[:, :1, :1].expand(3, 16, 24)
    c.D, c.bias = c.D[:, :1].expand(3, 24), c.bias[:, :1].expand(3, 24)
    c.check()
    c.check(20)
    one = Case([1, 1], 1, 3, 16, 24, TYPES[0], seed=10)
    one.dt, one.A = one.dt[:, :, :1].expand(-1, -1, 24), one.A[:, :, :1].expand(3, 16, 24)
    one.check(1)


def test_rows_behind_the_last_stay_as_they_were():
    for lens, bound in (([3, 20], 0), ([1, 1], 1)):
        c = Case(lens, 1, 2, 16, 64, seed=11)
        n = sum(lens)
        x, dt, B, C, z = (torch.cat([t, t]) for t in (c.x, c.dt, c.B, c.C, c.z))
        out = torch.full((2 * n, 2, 64), 5.0, dtype=BF16, device=DEV)
        gdr.gdr_selective_scan(x, dt, c.A, B, C, c.pool.clone(), c.slot, c.off, out, z=z, max_row_len=bound)
        assert bool((out[n:] == 5.0).all()) and not bool((out[:n] == 5.0).all())


def test_values_far_out():
    """Steps so large that nothing of a state is left, none at all, rates of 0 and growing ones."""
    c = Case([12], 1, 1, 16, 32, TYPES[2], seed=12)
    c.dt[3], c.dt[5], c.dt[7] = 300.0, -300.0, 88.0
    c.A[0, 0], c.A[0, 1], c.A[0, 2] = 0.0, -1e30, 0.01
    c.check()


def test_not_finite():
    """What is not finite spoils its own row, and of it its own channel where it is a channel's."""
    for bad in (float("inf"), float("nan")):
        c = Case([12, 12], 1, 2, 16, 32, seed=13)
        good, state = c.run()
        c.x[3, 0, 5] = bad
        got, pool = c.run()
        same = torch.ones_like(got, dtype=torch.bool)
        same[3:12, 0, 5] = False
        assert torch.equal(got[same], good[same])
        assert torch.equal(pool[c.slot[1]], state[c.slot[1]])


def test_repeats_and_two_calls_at_once():
    cases = [Case([300, 41, 7], 1, 2, 16, 64, seed=14), Case([2000], 1, 1, 16, 64, seed=15)]
    want = [c.run(max_row_len=2000) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.run(max_row_len=2000))
        torch.cuda.synchronize()
        for (o, p), (a, b) in zip(want, got):
            assert torch.equal(o, a) and torch.equal(p, b)


@pytest.mark.parametrize("lens", [[1, 30, 2], [2000]])
def test_graphs_and_prepared_calls(lens):
    c = Case(lens, 1, 2, 16, 32, seed=16)
    want, state = c.run()
    pool, out = c.pool.clone(), torch.empty_like(c.x)
    call = gdr.prepare_selective_scan(*c.args(pool), out, **c.more())
    call()
    torch.cuda.synchronize()
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
    c = Case([2], 1, 1, 16, 32, seed=17)
    out = torch.ones_like(c.x)
    gdr.gdr_selective_scan(c.x, c.dt, c.A, c.B, c.C, c.pool, _ints([]), _ints([0]), out)
    assert bool((out == 1).all())
    e = [t[:0] for t in (c.x, c.dt, c.B, c.C)]
    assert gdr.gdr_selective_scan(e[0], e[1], c.A, e[2], e[3], c.pool, _ints([0]), _ints([0, 0])).shape == (0, 1, 32)


def test_refusals():
    c = Case([3, 4], 1, 2, 16, 32)
    x, dt, A, B, C, pool, slot, off = c.args(c.pool)
    for args, error, match in [
            ((x, dt.half(), A, B, C, pool, slot, off), TypeError, "dt"), ((x, dt, A[:1], B, C, pool, slot, off), ValueError, "A must"),
            ((x, dt, A, B[:, :, :8], C, pool, slot, off), ValueError, "B and C"),
            ((x, dt, A, B.float(), C, pool, slot, off), TypeError, "B has"),
            ((x[:, :1], dt, A, B, C, pool, slot, off), ValueError, "x must"), ((x, dt[:2], A, B, C, pool, slot, off), ValueError, "dt must"),
            ((x, dt, A.bfloat16(), B, C, pool, slot, off), TypeError, "A has"), ((x, dt, A, B, C, pool[0], slot, off), ValueError, "state"),
            ((x, dt, A, B, C, pool, slot.long(), off), TypeError, "slot_idx"), ((x, dt, A, B, C, pool, slot, off[1:]), ValueError, "offsets"),
            ((x.float(), dt, A, B.float(), C.float(), pool, slot, off), gdr.GdrError, "dt_dtype")]:
        with pytest.raises(error, match=match):
            gdr.gdr_selective_scan(*args)
    with pytest.raises(gdr.GdrError, match="state_vdim_stride"):
        gdr.gdr_selective_scan(x, dt, A, B, C, torch.zeros(4, 2, 16, 64, device=DEV)[..., ::2], slot, off)
    with pytest.raises(gdr.GdrError, match="K=129"):
        big = torch.zeros(7, 1, 129, dtype=BF16, device=DEV)
        gdr.gdr_selective_scan(x, dt, torch.zeros(2, 129, 32, device=DEV), big, big, torch.zeros(4, 2, 129, 32, device=DEV), slot, off)
    with pytest.raises(ValueError, match="state_only"):
        gdr.gdr_selective_scan(*c.args(pool), torch.empty_like(x), state_only=True)
    with pytest.raises(ValueError, match="keep_state"):
        gdr.gdr_selective_scan(*c.args(pool), keep_state=False, state_only=True)
    with pytest.raises(ValueError, match="D must"):
        gdr.gdr_selective_scan(*c.args(pool), D=c.D[:1])
    with pytest.raises(ValueError, match="z must"):
        gdr.gdr_selective_scan(*c.args(pool), z=c.z[:2])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("K", [3, 12, 20, 27, 50, 100])
@pytest.mark.parametrize("V", [36, 64, 128])
def test_states_that_fill_no_vector(types, K, V):
    """B and C come value by value while the channels come as vectors, on a GPU whose shared memory is full of NaN."""
    full = Case([40] * 160, 1, 4, 32, 64, types, seed=1)
    full.B.fill_(float("nan"))
    full.C.fill_(float("nan"))
    full.run()
    Case([19, 3, 5, 0, 61], 2, 4, K, V, types, seed=K).check()


@pytest.mark.parametrize("types", TYPES[:2])
@pytest.mark.parametrize("lens,bound,K,V", [([1] * 9, 1, 16, 64), ([5, 1, 7], 8, 16, 64), ([100, 3, 41], 0, 16, 64),
                                            ([100, 3, 41], 0, 5, 33), ([2500], 0, 16, 64)])
@pytest.mark.parametrize("on", ["x", "z"])
def test_output_in_place_of_an_input(types, lens, bound, K, V, on):
    c = Case(lens, 1, 4, K, V, types, seed=17)
    want, state = c.run(max_row_len=bound)
    c.z = c.z.contiguous()
    pool, out = c.pool.clone(), getattr(c, on)
    assert c.run(pool, max_row_len=bound, out=out)[0] is out
    assert torch.equal(out, want) and torch.equal(pool, state)


@pytest.mark.parametrize("types", TYPES[:2])
@pytest.mark.parametrize("lens,bound", [([1] * 3, 1), ([5, 1, 7], 8), ([100, 3, 41], 0)])
def test_infinite_rates_forget(types, lens, bound):
    """A = -inf: a state is its last token's alone, as with a decay that float32 rounds to 0 (d >= 1/2, A = -1000)."""
    c = Case(lens, 1, 2, 16, 36, types, seed=18, bias=False, softplus=False)
    c.dt.clamp_(min=0.5)
    c.A[:, 3] = -1000.0
    want, state = c.run(max_row_len=bound)
    c.A[:, 3] = float("-inf")
    got, pool = c.run(max_row_len=bound)
    assert torch.equal(got, want) and torch.equal(pool, state)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("lens,bound", [([1] * 9, 1), ([5, 1, 7, 0, 8], 8), ([100, 3, 41], 0), ([1500], 0)])
@pytest.mark.parametrize("K,V,nk,nv", [(16, 64, 1, 2), (12, 36, 2, 6), (27, 20, 1, 3)])
def test_one_step_size_a_head(types, lens, bound, K, V, nk, nv):
    """dt of one value a head beside channels in vectors: the same results as with the value at every channel."""
    c = Case(lens, nk, nv, K, V, types, seed=19)
    c.dt = c.dt[:, :, 3:4].expand(-1, -1, V)
    got, pool = c.check(bound, cut=256) if max(lens) > 256 else c.check(bound)
    c.dt = c.dt.contiguous()
    want, state = c.run(max_row_len=bound)
    assert torch.equal(got, want) and torch.equal(pool, state)


@pytest.mark.parametrize("types", [TYPES[0], TYPES[3]])
@pytest.mark.parametrize("lens,bound", [([1, 1], 1), ([3, 0, 7], 7), ([40, 9], 0), ([700], 0)])
@pytest.mark.parametrize("nk,nv,K,V", [(1, 1, 1, 1), (64, 64, 4, 4), (2, 6, 31, 4), (1, 2, 128, 68), (3, 3, 65, 130)])
@pytest.mark.parametrize("shared", ["xz", "BA", "xzBAd"])
def test_inputs_that_are_shared(types, lens, bound, nk, nv, K, V, shared):
    """Strides of 0: over tokens (x, C), heads (z, B), channels (A, D, dt)."""
    c = Case(lens, nk, nv, K, V, types, seed=20)
    T = sum(lens)
    if "x" in shared:
        c.x, c.z = c.x[:1].expand(T, -1, -1), c.z[:, :1].expand(-1, nv, -1)
    if "B" in shared:
        c.B, c.C = c.B[:, :1].expand(-1, nk, -1), c.C[:1].expand(T, -1, -1)
        c.A, c.D = c.A[:1, :, :1].expand(nv, K, V), c.D[:1, :1].expand(nv, V)
    if "d" in shared:
        c.dt = c.dt[:, :1, :1].expand(-1, nv, V)
    c.check(bound, cut=max(lens))


def test_very_many_rows():
    n, h = 200001, 100000
    c = Case([1] * n, 1, 1, 8, 8, seed=21)
    got, pool = c.run(max_row_len=1)
    other, state = c.run()  # by chunks
    assert torch.equal(pool, state)
    halves = c.pool.clone()
    first = gdr.gdr_selective_scan(c.x[:h], c.dt[:h], c.A, c.B[:h], c.C[:h], halves, c.slot[:h], c.off[:h + 1], D=c.D, z=c.z[:h],
                                   dt_bias=c.bias, max_row_len=1)
    second = gdr.gdr_selective_scan(c.x[h:], c.dt[h:], c.A, c.B[h:], c.C[h:], halves, c.slot[h:], c.off[h:] - h, D=c.D, z=c.z[h:],
                                    dt_bias=c.bias, max_row_len=1)
    assert torch.equal(got, torch.cat([first, second])) and torch.equal(pool, halves)
    # the readout's eight products add up in another order: 8 roundings of the largest partial sum, and bfloat16's own
    terms = (c.C.float()[:, :, :, None].abs() * pool[c.slot.long()].abs()).sum(2) + (c.D * c.x.float()).abs()
    gate = c.z.float() * torch.sigmoid(c.z.float())
    tol = 2 * 12 * 2.0 ** -24 * terms * gate.abs() + 2.0 ** -7 * got.float().abs() + 1e-6
    assert bool(((got.float() - other.float()).abs() <= tol).all())
