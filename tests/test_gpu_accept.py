"""Verification of drafts (gdr_accept_drafts) against the rule in rational
numbers: whole numbers, equal."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import accept_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _clean_status():
    gdr.gdr_get_status(clear=True)
    yield
    st = gdr.gdr_get_status(clear=True)
    assert st == 0, f"device status {gdr.status_names(st)}"


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _floats(values):
    return torch.tensor(values, dtype=F32, device=DEV)


class Case:
    def __init__(self, lens, vocab, dtype=F32, drafter=True, seed=0, near=0.7):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T = sum(lens)
        logits = 3 * torch.randn(T, vocab, generator=g, device=DEV)
        self.target = torch.softmax(logits, 1).to(dtype)
        draft = torch.softmax(logits + near * torch.randn(T, vocab, generator=g, device=DEV), 1)
        self.tokens = torch.randint(vocab, (T,), generator=g, device=DEV).to(torch.int32)
        self.tokens[1:] = torch.multinomial(draft, 1, generator=g)[:-1, 0]
        self.draft = draft.to(dtype) if drafter else None
        self.off = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        self.u = torch.rand(T, generator=g, device=DEV)
        self.v = torch.rand(len(lens), generator=g, device=DEV)
        self.width = max(lens)

    def args(self):
        return self.target, self.draft, self.tokens, self.off, self.u, self.v

    def check(self, **kw):
        out, counts = gdr.gdr_accept_drafts(*self.args(), max_row_len=self.width, **kw)
        want, n = accept_ref(*self.args(), self.width)
        assert out.cpu().tolist() == want.tolist()
        assert counts.cpu().tolist() == n.tolist()
        return out, counts


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 33, 128, 1000, 1033, 4099])
def test_rows(dtype, drafter, vocab):
    lens = [1, 2, 5, 0, 9, 3, 4, 1, 6, 2, 2, 8]
    for seed in range(3):
        Case(lens, vocab, dtype, drafter, seed).check()


@pytest.mark.parametrize("rows", [1, 3, 80, 200, 330])
def test_rows_of_every_split(rows):
    """Few rows are shared by several blocks each, many have one."""
    Case([2] * rows, 515, F32, seed=rows).check()


def test_a_large_vocabulary():
    c = Case([3, 1, 4], 150001, F32, seed=5)
    c.check()
    c = Case([3, 1, 4], 131072, BF16, drafter=False, seed=6)
    c.check()


def test_draws_next_to_borders():
    """Numbers at a running sum's own value and at its neighbours, in weights whose sums are exact."""
    vocab = 64
    p = torch.zeros(1, vocab)
    p[0, [3, 10, 11, 40]] = torch.tensor([0.25, 0.125, 0.5, 0.125])
    for v in (0.0, 0.25, 0.375, 0.875, 1.0):
        for step in (-1, 0, 1):
            x = torch.tensor(v)
            if step:
                x = torch.nextafter(x, torch.tensor(float(step)) * 2)
            got, n = gdr.gdr_accept_drafts(p.to(DEV), None, _ints([0]), _ints([0, 1]), _floats([0.0]), x.view(1).to(DEV), max_row_len=1)
            want, _ = accept_ref(p, None, _ints([0]), _ints([0, 1]), _floats([0.0]), x.view(1), 1)
            assert got.cpu().tolist() == want.tolist(), (v, step)


def test_acceptance_next_to_a_border():
    """u q = p refuses, and the number below accepts: the product is not rounded."""
    third = torch.tensor(1 / 3)
    p, q = torch.zeros(2, 8), torch.zeros(2, 8)
    q[0, 2], p[0, 2], p[0, 5], p[1, 1] = third, third * torch.tensor(0.7), 0.5, 1.0
    ratio = (p[0, 2].double() / q[0, 2].double()).float()
    for u in (torch.nextafter(ratio, torch.tensor(0.0)), ratio, torch.nextafter(ratio, torch.tensor(1.0))):
        args = p, q, torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32), u.repeat(2), torch.tensor([0.3])
        got, n = gdr.gdr_accept_drafts(*(t.to(DEV) for t in args), max_row_len=2)
        want, m = accept_ref(*args, 2)
        assert got.cpu().tolist() == want.tolist() and n.cpu().tolist() == m.tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_numbers_and_probabilities_out_of_range(dtype):
    c = Case([4, 4, 4, 4, 4, 4], 200, dtype, seed=7)
    c.u[0], c.u[5], c.u[9], c.u[13] = NAN, -1.0, 1.0, INF
    c.v[:] = _floats([NAN, -0.5, 1.0, 2.0, INF, -INF])
    c.target[:, 7], c.target[:, 9], c.target[:, 150], c.target[:, 199] = NAN, -0.5, INF, 0.0
    c.draft[:, 11], c.draft[:, 12], c.draft[:, 151] = NAN, -INF, INF
    c.tokens[1], c.tokens[6], c.tokens[10], c.tokens[17] = 7, 11, 150, 199
    c.check()


def test_drafts_outside_the_vocabulary_end_a_row():
    for drafter in (True, False):
        c = Case([5, 5, 5, 5], 100, drafter=drafter, seed=8, near=0.1)
        c.u.zero_()  # accepts whatever has a chance
        c.tokens[2], c.tokens[6], c.tokens[14], c.tokens[16] = -1, 100, -2 ** 31, 2 ** 31 - 1
        out, counts = c.check()
        assert counts.tolist() == [2, 1, 4, 1]


def test_nothing_left_over():
    """Drafter and target alike, but refused (a number of 1): drawn from the target.  No weight at all: -1, and said."""
    c = Case([3, 3], 50, seed=9)
    c.draft = c.target.clone()
    c.u[0] = c.u[3] = 1.0
    c.check()
    # the one refused token is all there is
    p = torch.zeros(2, 40, device=DEV)
    p[:, 4] = 0.5
    args = p, None, _ints([1, 4]), _ints([0, 2]), _floats([0.75, 0.0]), _floats([0.5])
    got, n = gdr.gdr_accept_drafts(*args, max_row_len=2)
    assert got.tolist() == [[4, -1]] and n.tolist() == [1]
    c.target[2] = 0.0
    c.target[3] = -1.0
    c.tokens[1], c.tokens[2] = c.target[0].argmax(), c.target[1].argmax()
    c.u[:2] = 0.0
    out, counts = c.check()
    assert counts.tolist() == [3, 1] and out[:, :3].tolist()[0][2] == -1 and out[1].tolist() == [-1] * 3
    assert gdr.status_names(gdr.gdr_get_status()) == ["NO_MASS"]


def test_small_and_unnormalised_weights():
    for scale in (1e-30, 1e-42, 1e30):
        c = Case([3, 4, 2], 300, seed=10)
        c.target, c.draft = c.target * scale, c.draft * scale
        c.check()


def test_layouts():
    """Strided and misaligned probabilities, a wider result, rows behind the last left alone."""
    c = Case([3, 1, 5], 260, seed=11)
    want, n = c.check()
    wide = torch.full((9, 700), NAN, device=DEV)
    for shift in (0, 1, 2):
        wide[:, shift:260 + shift], wide[:, 300 + shift:560 + shift] = c.target, c.draft
        c.target, c.draft = wide[:, shift:260 + shift].clone(), wide[:, 300 + shift:560 + shift].clone()
        views = wide[:, shift:260 + shift], wide[:, 300 + shift:560 + shift]
        out = torch.full((4, 9), 77, dtype=torch.int32, device=DEV)
        counts = torch.full((3,), 77, dtype=torch.int32, device=DEV)
        got, m = gdr.gdr_accept_drafts(*views, *c.args()[2:], max_row_len=5, out=out[:3, 2:7], counts=counts)
        assert torch.equal(got, want) and torch.equal(m, n) and m is counts
        assert bool((out[3] == 77).all()) and bool((out[:, :2] == 77).all()) and bool((out[:, 7:] == 77).all())


def test_problems_the_device_sees():
    c = Case([3, 6, 2], 100, seed=12)
    want, n = c.check()
    got, m = gdr.gdr_accept_drafts(*c.args(), max_row_len=3)
    assert gdr.status_names(gdr.gdr_get_status()) == ["ROW_TOO_LONG"]
    assert m.tolist() == [int(n[0]), 0, int(n[2])] and got[1].tolist() == [-1] * 3
    assert got[0].tolist() == want[0, :3].tolist() and got[2].tolist() == want[2, :3].tolist()
    for off in ([0, 3, 2, 11], [-1, 3, 9, 11], [0, 3, 9, 12]):
        gdr.gdr_accept_drafts(c.target, c.draft, c.tokens, _ints(off), c.u, c.v, max_row_len=12)
        assert gdr.status_names(gdr.gdr_get_status()) == ["BAD_OFFSETS"]


def test_streams_graphs_and_prepared_calls():
    c = Case([4, 1, 6], 5000, seed=13)
    want, n = c.check()
    out, counts = torch.zeros_like(want), torch.zeros_like(n)
    call = gdr.prepare_accept_drafts(*c.args(), out, counts, max_row_len=c.width)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(counts, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(counts, n)


def test_distribution():
    """Accepted or drawn anew, the first token follows the target's probabilities."""
    vocab, rows = 8, 40000
    g = torch.Generator(device=DEV).manual_seed(14)
    p = torch.softmax(torch.randn(vocab, generator=g, device=DEV), 0)
    q = torch.softmax(torch.randn(vocab, generator=g, device=DEV), 0)
    tokens = torch.zeros(2 * rows, dtype=torch.int32, device=DEV)
    tokens[1::2] = torch.multinomial(q, rows, replacement=True, generator=g).to(torch.int32)
    off = torch.arange(0, 2 * rows + 1, 2, dtype=torch.int32, device=DEV)
    out, _ = gdr.gdr_accept_drafts(p.expand(2 * rows, vocab), q.expand(2 * rows, vocab), tokens, off,
                                   torch.rand(2 * rows, generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV),
                                   max_row_len=2)
    share = torch.bincount(out[:, 0], minlength=vocab).double() / rows
    # five standard deviations of a share
    assert bool(((share - p.double()).abs() <= 5 * (p * (1 - p) / rows).sqrt().double()).all())


def test_nothing_to_do():
    t = torch.zeros(0, 10, device=DEV)
    out, n = gdr.gdr_accept_drafts(t, t, _ints([]), _ints([0]), _floats([]), _floats([]), max_row_len=4)
    assert out.shape == (0, 4) and n.shape == (0,)
    out, n = gdr.gdr_accept_drafts(t, t, _ints([]), _ints([0, 0]), _floats([]), _floats([0.5]), max_row_len=2)
    assert out.tolist() == [[-1, -1]] and n.tolist() == [0]


def test_refusals():
    c = Case([3, 4], 64)
    a = c.args()
    with pytest.raises(ValueError, match="max_row_len"):
        gdr.gdr_accept_drafts(*a, max_row_len=0)
    with pytest.raises(TypeError):
        gdr.gdr_accept_drafts(c.target.half(), *a[1:], max_row_len=4)
    with pytest.raises(TypeError):
        gdr.gdr_accept_drafts(a[0], c.draft.bfloat16(), *a[2:], max_row_len=4)
    with pytest.raises(ValueError, match="draft"):
        gdr.gdr_accept_drafts(a[0], c.draft[:, :32], *a[2:], max_row_len=4)
    with pytest.raises(TypeError):
        gdr.gdr_accept_drafts(*a[:2], c.tokens.long(), *a[3:], max_row_len=4)
    with pytest.raises(ValueError, match="row_uniforms"):
        gdr.gdr_accept_drafts(*a[:5], c.v[:1], max_row_len=4)
    with pytest.raises(ValueError, match="stride"):
        gdr.gdr_accept_drafts(c.target.T.contiguous().T, *a[1:], max_row_len=4)
