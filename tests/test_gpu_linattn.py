"""Decayed linear attention (gdr_linattn_fwd) against the token-by-token
recurrence in float64: every form (single tokens, short rows, chunks, split
rows), type, head layout, odd length, stride, padding and refusal."""
from __future__ import annotations

import math

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.layer_helpers import check_linattn, linattn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    gdr.gdr_get_status(clear=True)
    yield
    st = gdr.gdr_get_status(clear=True)
    assert st == 0, f"device status {gdr.status_names(st)}"


class Case:
    """Inputs of one call: packed projections, a pool with slots nobody uses, padding rows at `pad`."""

    def __init__(self, lens, nk=2, nv=2, K=128, V=128, tok=BF16, pool=F32, pad=(), seed=0, lam=None, log=False,
                 gap=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T = sum(lens) + gap
        n = 2 * nk * K + nv * V
        self.x = torch.randn(T, n, generator=g, device=DEV).to(tok)
        self.q = self.x[:, :nk * K].view(T, nk, K)
        self.k = self.x[:, nk * K:2 * nk * K].view(T, nk, K)
        self.v = self.x[:, 2 * nk * K:].view(T, nv, V)
        if lam is None:
            lam = torch.exp(-torch.exp2(-8.0 * torch.rand(nv, generator=g, device=DEV)))
        self.lam = torch.as_tensor(lam, dtype=F32, device=DEV).expand(nv).contiguous()
        self.log = log
        self.decay = torch.log(self.lam) if log else self.lam.clone()
        slots = len(lens) + 2
        self.pool = torch.randn(slots, nv, K, V, generator=g, device=DEV).to(pool)
        slot = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:len(lens)]
        slot[list(pad)] = -1
        self.slot = slot.to(torch.int32).to(DEV)
        off = [gap]
        for n in lens:
            off.append(off[-1] + n)
        self.off = torch.tensor(off, dtype=torch.int32, device=DEV)
        self.longest = max(lens) if lens else 0

    def run(self, max_row_len=0, **kw):
        pool = self.pool.clone()
        out = gdr.gdr_linattn_fwd(self.q, self.k, self.v, self.decay, pool, self.slot, self.off, decay_is_log=self.log,
                                  max_row_len=max_row_len, **kw)
        return out, pool

    def ref(self, scale=0.0):
        return linattn_ref(self.q, self.k, self.v, self.decay, self.pool, self.slot, self.off, decay_is_log=self.log,
                           scale=scale)

    def check(self, max_row_len=0, **kw):
        out, pool = self.run(max_row_len, **kw)
        first = int(self.off[0])
        ref = self.ref(kw.get("scale", 0.0))
        check_linattn(out[first:], pool, tuple(x[first:] if i % 2 == 0 else x for i, x in enumerate(ref)), self.longest,
                      self.q.dtype == BF16 and max_row_len != 1)
        used = set(int(s) for s in self.slot.tolist() if s >= 0)
        for s in range(self.pool.shape[0]):
            if s not in used:
                assert torch.equal(pool[s], self.pool[s]), f"slot {s} is nobody's"
        return out, pool


TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]


@pytest.mark.parametrize("tok,pool", TYPES)
@pytest.mark.parametrize("K,V,nk,nv", [(128, 128, 2, 4), (64, 64, 3, 3), (16, 16, 1, 5), (32, 256, 2, 2), (96, 144, 1, 3),
                                       (128, 256, 1, 1), (80, 48, 2, 2)])
def test_single_tokens(tok, pool, K, V, nk, nv):
    Case([1] * 7, nk, nv, K, V, tok, pool, pad=(2,), seed=K + V).check(max_row_len=1)


@pytest.mark.parametrize("tok,pool", TYPES)
@pytest.mark.parametrize("K,V,nk,nv", [(128, 128, 2, 4), (64, 64, 2, 2), (16, 32, 1, 2), (128, 256, 1, 2), (96, 144, 1, 1)])
@pytest.mark.parametrize("hint", [0, 300])
def test_ragged_rows(tok, pool, K, V, nk, nv, hint):
    Case([1, 64, 0, 65, 63, 7, 128, 129, 300, 2], nk, nv, K, V, tok, pool, pad=(5,), seed=K).check(max_row_len=hint)


@pytest.mark.parametrize("longest", [2, 3, 8, 16, 17, 33])
def test_short_rows(longest):
    Case([longest, 1, 0, longest - 1, 2], 1, 2, 128, 128, BF16, BF16, pad=(3,), seed=longest).check(max_row_len=longest)


@pytest.mark.parametrize("log", [False, True])
@pytest.mark.parametrize("lam", [0.0, 1e-30, 1e-3, 0.5, 0.999, 1.0])
@pytest.mark.parametrize("hint", [0, 8])
def test_decays(log, lam, hint):
    """No memory at all, a memory that underflows inside a chunk, and one that never fades."""
    Case([8, 5, 1] if hint else [130, 64, 5, 1], 1, 2, 64, 64, BF16, F32, lam=lam, log=log, seed=3).check(max_row_len=hint)


@pytest.mark.parametrize("tok", [BF16, F32])
def test_scale_and_leading_gap(tok):
    """Rows that do not begin at token 0, and a scale of the caller's."""
    Case([70, 3], 1, 1, 64, 128, tok, F32, gap=37, seed=5).check(scale=0.37)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("tok", [BF16, F32])
def test_layouts(hint, tok):
    """Strided, odd and misaligned tokens, a strided pool, a caller's strided output."""
    lens = [1] * 5 if hint else [70, 1, 13]
    c = Case(lens, 2, 4, 64, 64, tok, F32, seed=11)
    want, want_pool = c.run(hint)
    T = c.q.shape[0]
    # heads before tokens, and rows one element off 16 bytes
    for shift in (0, 1):
        def lay(x):
            t, h, d = x.shape
            buf = torch.full((h * t * (d + 8) + 9,), float("nan"), dtype=x.dtype, device=DEV)
            y = buf[shift:].as_strided((t, h, d), (d + 8, t * (d + 8), 1))
            y.copy_(x)
            return y
        o = lay(torch.zeros_like(c.v))
        pool = torch.full((c.pool.shape[0], 4, 80, 72), float("nan"), device=DEV)[:, :, 3:67, 4:68]
        pool.copy_(c.pool)
        got = gdr.gdr_linattn_fwd(lay(c.q), lay(c.k), lay(c.v), c.decay, pool, c.slot, c.off, o, max_row_len=hint)
        assert got is o
        ref = c.ref()
        check_linattn(o, pool, ref, c.longest, tok == BF16 and hint != 1)
    # one query and key for all heads of a token, by a stride of 0
    q1 = c.q[:, :1].expand(T, 2, 64)
    pool = c.pool.clone()
    got = gdr.gdr_linattn_fwd(q1, q1, c.v, c.decay, pool, c.slot, c.off, max_row_len=hint)
    ref = linattn_ref(q1, q1, c.v, c.decay, c.pool, c.slot, c.off)
    check_linattn(got, pool, ref, c.longest, tok == BF16 and hint != 1)


def test_chained_calls_continue_the_state():
    """A prompt in two pieces and then single tokens."""
    c = Case([150], 1, 2, 128, 128, BF16, F32, seed=21)
    pool, outs = c.pool.clone(), []
    for a, b in [(0, 77), (77, 148), (148, 149), (149, 150)]:
        off = torch.tensor([0, b - a], dtype=torch.int32, device=DEV)
        outs.append(gdr.gdr_linattn_fwd(c.q[a:b], c.k[a:b], c.v[a:b], c.decay, pool, c.slot, off, max_row_len=b - a))
    check_linattn(torch.cat(outs), pool, c.ref(), 150, True)


@pytest.mark.parametrize("lens", [[1000], [700, 3, 1], [2049]])
def test_long_rows_with_and_without_a_workspace(lens):
    """Few rows: the call may cut them into segments; with no room for that it gives the same within rounding."""
    c = Case(lens, 1, 2, 64, 128, BF16, F32, seed=31)
    c.check(max_row_len=max(lens))
    c.check(max_row_len=max(lens), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    c.check()


@pytest.mark.parametrize("pool", [BF16, F32])
@pytest.mark.parametrize("lens,nk,nv,K,V,pad", [([2400], 1, 2, 128, 128, ()), ([2100, 0, 2300, 5], 2, 2, 64, 64, (2,)),
                                                ([64 * 40 + 1, 64 * 20], 1, 3, 96, 144, ()), ([3001], 2, 4, 128, 256, ()),
                                                ([64 * 36] + [70] * 8, 1, 4, 64, 128, (3,))])
def test_rows_cut_into_segments(lens, nk, nv, K, V, pad, pool):
    c = Case(lens, nk, nv, K, V, BF16, pool, pad=pad, seed=sum(lens))
    assert gdr.gdr_linattn_workspace_bytes(c.q, c.k, c.v, c.decay, c.pool, c.slot, c.off, max_row_len=max(lens)) > 0
    c.check(max_row_len=max(lens))


def test_problems_in_rows_cut_into_segments():
    c = Case([2400, 40, 2300], 1, 3, 64, 64, BF16, F32, seed=83)
    good, good_pool = c.run(2400)
    c.decay[1] = 2.0
    out, pool = _flags(lambda: c.run(2400), "BAD_DECAY")
    assert not out[:, 1].any() and torch.equal(pool[:, 1], c.pool[:, 1])
    assert torch.equal(out[:, [0, 2]], good[:, [0, 2]]) and torch.equal(pool[:, [0, 2]], good_pool[:, [0, 2]])
    c.decay[:] = c.lam
    out, pool = _flags(lambda: c.run(2350), "ROW_TOO_LONG")
    assert not out[:2400].any() and torch.equal(pool[int(c.slot[0])], c.pool[int(c.slot[0])])
    slot = c.slot.clone()
    c.slot[2] = -7
    out, pool = _flags(lambda: c.run(2400), "BAD_SLOT")
    assert not out[2440:].any() and torch.equal(out[:2440], good[:2440])
    c.slot[:] = slot
    # rows that lie on one another are not all done, and never ask for more segments than there is room for
    c = Case([2400] + [0] * 14, 1, 3, 64, 64, BF16, F32, seed=84)
    want, want_pool = c.run(2400)
    c.off[1::2] = 2400
    c.off[2::2] = 0
    out, pool = _flags(lambda: c.run(2400), "BAD_OFFSETS")
    assert torch.equal(out, want) and torch.equal(pool, want_pool)


def test_problems_in_short_rows():
    c = Case([9, 5, 12], 1, 3, 64, 64, BF16, BF16, seed=85)
    good, good_pool = c.run(12)
    c.decay[1] = -1.0
    out, pool = _flags(lambda: c.run(12), "BAD_DECAY")
    assert not out[:, 1].any() and torch.equal(pool[:, 1], c.pool[:, 1])
    assert torch.equal(out[:, [0, 2]], good[:, [0, 2]]) and torch.equal(pool[:, [0, 2]], good_pool[:, [0, 2]])
    c.decay[:] = c.lam
    out, pool = _flags(lambda: c.run(10), "ROW_TOO_LONG")
    assert not out[14:].any() and torch.equal(out[:14], good[:14])
    assert torch.equal(pool[int(c.slot[2])], c.pool[int(c.slot[2])])
    c.off[-1] = 10 ** 6
    out, pool = _flags(lambda: c.run(12), "BAD_OFFSETS")
    assert torch.equal(out[:14], good[:14]) and torch.equal(pool[int(c.slot[2])], c.pool[int(c.slot[2])])
    c.off[-1] = 26
    c.slot[0] = 5
    out, pool = _flags(lambda: c.run(12), "BAD_SLOT")
    assert not out[:9].any() and torch.equal(out[9:], good[9:])


@pytest.mark.parametrize("pool", [BF16, F32])
@pytest.mark.parametrize("K,V,nk,nv", [(128, 256, 4, 8), (16, 16, 1, 8), (96, 144, 8, 8), (64, 64, 8, 8), (48, 80, 2, 8)])
def test_short_rows_by_the_hundred(K, V, nk, nv, pool):
    """More units than the GPU takes at once, padding rows and rows of nothing among them."""
    lens = [(5 * i) % 17 for i in range(120)]
    Case(lens, nk, nv, K, V, BF16, pool, pad=(7, 40), seed=K + V).check(max_row_len=16)


@pytest.mark.parametrize("pool", [BF16, F32])
@pytest.mark.parametrize("hint,nk,nv,K,V", [(32, 2, 4, 128, 128), (33, 2, 4, 128, 144), (17, 1, 8, 96, 256), (48, 4, 4, 64, 128),
                                            (49, 1, 4, 48, 80), (47, 2, 8, 128, 64), (56, 2, 16, 64, 128), (130, 2, 16, 48, 64), (96, 8, 8, 64, 64), (97, 8, 8, 64, 64),
                                            (80, 1, 16, 16, 16)])
def test_rows_of_a_few_pieces(hint, nk, nv, K, V, pool):
    """Either side of where rows stop being short; lengths around multiples of 16, more units than fit at once."""
    lens = [min(n, hint) for n in (hint, 0, 1, 15, 16, 17, 31, 32, 33, 48, 49, 64, 65, 80, 95, 96)] * 4
    Case(lens, nk, nv, K, V, BF16, pool, pad=(6, 30), seed=hint + K).check(max_row_len=hint)


@pytest.mark.parametrize("pool", [BF16, F32])
@pytest.mark.parametrize("lens,nk,nv,K,V", [([(7 * i) % 90 for i in range(75)], 1, 2, 64, 64),  # many rows
                                            ([100, 20, 1], 2, 72, 64, 128),                      # many heads
                                            ([900, 530, 512, 64, 7, 0], 5, 40, 128, 128),        # units dealt by load
                                            ([600, 90], 1, 80, 64, 256),                         # two column tiles, more heads than CTAs
                                            ([65] * 16, 11, 11, 96, 144)])
def test_batches(lens, nk, nv, K, V, pool):
    """Every way units are dealt out, with padding rows among them."""
    Case(lens, nk, nv, K, V, BF16, pool, pad=(1,), seed=len(lens) + nv).check(max_row_len=max(lens))


def test_positions_past_32_bits():
    """A pool and token strides whose element offsets pass 2^31."""
    for hint in (1, 5, 70):
        lens = [hint, 1]
        c = Case(lens, 1, 1, 128, 256, BF16, BF16, seed=43)
        big = torch.zeros(66000, 1, 128, 256, dtype=BF16, device=DEV)  # 2.2e9 elements
        slots = torch.tensor([65999, 1], dtype=torch.int32, device=DEV)
        big[65999], big[1] = c.pool[0], c.pool[1]
        T, stride = sum(lens), 2 ** 31 // (hint + 1) // 8 * 8 + 1024
        far = torch.zeros(T * stride, dtype=BF16, device=DEV)
        v = far.as_strided((T, 1, 256), (stride, 256, 1))
        v.copy_(c.v)
        out = gdr.gdr_linattn_fwd(c.q, c.k, v, c.decay, big, slots, c.off, max_row_len=hint)
        ref = linattn_ref(c.q, c.k, c.v, c.decay, c.pool, torch.tensor([0, 1]), c.off)
        check_linattn(out, big[[65999, 1]], (ref[0], ref[1][:2], ref[2], ref[3][:2]), hint, hint > 1)
        del big, far, v


def test_a_row_of_nan_spoils_no_other():
    """Rows that share a chunk's loads with a neighbour full of NaN and infinities."""
    for hint in (0, 9):
        c = Case([9, 5, 9], 1, 2, 128, 128, BF16, F32, seed=41)
        clean = c.ref()
        c.x[9:14] = float("nan")
        c.x[10] = float("inf")
        c.pool[int(c.slot[1])] = float("nan")
        out, pool = c.run(hint)
        keep = [i for i in range(23) if not 9 <= i < 14]
        ok = [s for s in range(c.pool.shape[0]) if s != int(c.slot[1])]
        check_linattn(out[keep], pool[ok], (clean[0][keep], clean[1][ok], clean[2][keep], clean[3][ok]), 9, True)
        assert bool(torch.isnan(out[9:14]).all())


def test_nothing_to_do():
    c = Case([0, 0], 1, 1, 64, 64, BF16, BF16, seed=51)
    out, pool = c.run()
    assert out.shape[0] == 0 and torch.equal(pool, c.pool)
    c = Case([], 1, 1, 64, 64)
    c.run()


@pytest.mark.parametrize("hint", [0, 1, 5, 90, 5000])
@pytest.mark.parametrize("tok", [BF16, F32])
def test_no_tokens_at_all(hint, tok):
    c = Case([0, 0, 0], 1, 2, 64, 64, tok, BF16, pad=(1,), seed=53)
    out, pool = c.run(hint)
    assert out.shape == (0, 2, 64) and torch.equal(pool, c.pool)


@pytest.mark.parametrize("lens,hint", [([5, 9, 16, 1] * 9, 16), ([40, 3, 47] * 5, 48), ([3000, 5], 3000), ([700, 64] * 9, 700)])
def test_every_form_repeats_bit_for_bit(lens, hint):
    c = Case(lens, 2, 4, 64, 128, BF16, F32, seed=63)
    a, b = c.run(hint), c.run(hint)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("hint", [0, 1])
def test_repeats_bit_for_bit(hint):
    c = Case([1] * 9 if hint else [513, 64, 9], 2, 4, 128, 128, BF16, F32, seed=61)
    a, b = c.run(hint), c.run(hint)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_on_a_side_stream_and_in_a_graph():
    c = Case([200, 1], 1, 2, 64, 64, BF16, F32, seed=71)
    want, want_pool = c.run(200)
    pool, out = c.pool.clone(), torch.zeros_like(c.v)
    call = gdr.prepare_linattn_fwd(c.q, c.k, c.v, c.decay, pool, c.slot, c.off, out, max_row_len=200)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(pool, want_pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pool.copy_(c.pool)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(pool, want_pool)


def _flags(call, *names):
    gdr.gdr_get_status(clear=True)
    got = call()
    torch.cuda.synchronize()
    assert sorted(gdr.status_names(gdr.gdr_get_status(clear=True))) == sorted(names)
    return got


@pytest.mark.parametrize("hint", [0, 1])
def test_problems_only_the_device_sees(hint):
    """Bad decays, slots, offsets and lengths skip their rows, zero their output and are flagged."""
    lens = [1, 1, 1] if hint else [70, 5, 9]
    c = Case(lens, 1, 3, 64, 64, BF16, F32, seed=81)
    good, good_pool = c.run(hint)
    for bad in (-0.5, 1.5, math.nan):
        c.decay[1] = bad
        out, pool = _flags(lambda: c.run(hint), "BAD_DECAY")
        assert not out[:, 1].any() and torch.equal(pool[:, 1], c.pool[:, 1])
        assert torch.equal(out[:, [0, 2]], good[:, [0, 2]]) and torch.equal(pool[:, [0, 2]], good_pool[:, [0, 2]])
    c.decay[1] = c.lam[0]
    c.decay[:] = c.lam
    keep = c.slot.clone()
    c.slot[1] = 99
    out, pool = _flags(lambda: c.run(hint), "BAD_SLOT")
    a, b = int(c.off[1]), int(c.off[2])
    assert not out[a:b].any() and torch.equal(out[:a], good[:a]) and torch.equal(out[b:], good[b:])
    c.slot[:] = keep
    if not hint:
        out, pool = _flags(lambda: c.run(40), "ROW_TOO_LONG")
        assert not out[:70].any() and torch.equal(pool[int(c.slot[0])], c.pool[int(c.slot[0])])
        ref = c.ref()
        check_linattn(out[70:], pool[c.slot[1:].long()],
                      (ref[0][70:], ref[1][c.slot[1:].long()], ref[2][70:], ref[3][c.slot[1:].long()]), 9, True)
    c.off[-1] += 1000
    out, pool = _flags(lambda: c.run(hint), "BAD_OFFSETS")
    b = int(c.off[2])
    assert torch.equal(out[:b], good[:b]) and torch.equal(pool[int(c.slot[2])], c.pool[int(c.slot[2])])


def test_refusals():
    c = Case([3], 2, 4, 64, 64)
    f = lambda **o: gdr.gdr_linattn_fwd(*[o.get(n, getattr(c, a)) for n, a in (
        ("q", "q"), ("k", "k"), ("v", "v"), ("decay", "decay"), ("state", "pool"), ("slot_idx", "slot"),
        ("offsets", "off"))], o.get("out"), workspace=o.get("workspace"))
    for bad, kind in [(dict(q=c.q.cpu()), ValueError), (dict(q=c.q.half()), TypeError), (dict(k=c.k.float()), TypeError),
                      (dict(q=c.q[:2]), ValueError), (dict(v=c.v[..., :32]), ValueError),
                      (dict(q=c.q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                      (dict(decay=c.decay[:2]), ValueError), (dict(decay=c.decay.double()), TypeError),
                      (dict(slot_idx=c.slot.long()), TypeError), (dict(offsets=c.off[:1]), ValueError),
                      (dict(state=c.pool[0]), ValueError), (dict(state=c.pool.half()), TypeError),
                      (dict(out=torch.empty_like(c.v).float()), TypeError),
                      (dict(workspace=torch.empty(64, dtype=torch.uint8)), ValueError)]:
        with pytest.raises(kind):
            f(**bad)
    with pytest.raises(gdr.GdrError, match="16-byte"):
        f(state=torch.empty(c.pool.numel() + 1, device=DEV)[1:].view(c.pool.shape))
    with pytest.raises(gdr.GdrError, match="multiple of 16"):
        d = Case([3], 1, 1, 72, 64)
        d.run()
