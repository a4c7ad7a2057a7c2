"""The state space operators together, as a serving loop runs them: prompts,
single tokens, and speculative steps whose drafts are verified, with the accepted
part of each row going into the pools; beside the recurrence's own verify and fold."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from gated_deltanet_linear_gdr_gb300 import _binding as B
from tests.state_space_helpers import accept_ref, check_close, conv_ref, scan_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Layer:
    """A selective state space layer: projection, short convolution, step sizes and inputs, scan, gate."""

    def __init__(self, rows, dim=48, nv=2, V=32, K=16, W=4, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device=DEV) * std

        n = nv * V
        self.nv, self.V, self.K = nv, V, K
        self.into, self.small = normal(dim, 2 * n, std=dim ** -0.5), normal(n, n + 2 * K, std=n ** -0.5)
        self.w, self.b = normal(n, W, std=0.5), normal(n, std=0.1)
        self.A, self.D = -torch.exp(2.5 * torch.rand(nv, K, V, generator=g, device=DEV)), normal(nv, V)
        self.bias = normal(nv, V) - 2
        self.conv = torch.zeros(rows + 1, n, W - 1, dtype=BF16, device=DEV)
        self.pool = torch.zeros(rows + 1, nv, K, V, device=DEV)

    def projected(self, h):
        xz = (h.float() @ self.into).to(BF16)
        n = self.nv * self.V
        return xz[:, :n], xz[:, n:].view(-1, self.nv, self.V)

    def inputs(self, x):
        """dt, B, C of the convolved inputs."""
        n, T = self.nv * self.V, x.shape[0]
        p = (x.float() @ self.small).to(BF16)
        return p[:, :n].view(T, self.nv, self.V), p[:, n:n + self.K].view(T, 1, self.K), p[:, n + self.K:].view(T, 1, self.K)

    def __call__(self, h, slot, off, counts=None, keep_state=True, longest=0):
        x, z = self.projected(h)
        u = gdr.gdr_short_conv(x, self.w, self.b, self.conv, slot, off, keep_state=keep_state, max_row_len=longest)
        scan = u.view(-1, self.nv, self.V), *self.inputs(u)
        y = gdr.gdr_selective_scan(scan[0], scan[1], self.A, scan[2], scan[3], self.pool, slot, off, D=self.D, z=z, dt_bias=self.bias,
                                   keep_state=keep_state, max_row_len=longest)
        return y, (x, z, scan)

    def commit(self, kept, slot, off, counts, longest):
        x, z, scan = kept
        gdr.gdr_short_conv(x, self.w, self.b, self.conv, slot, off, counts=counts, state_only=True, max_row_len=longest)
        gdr.gdr_selective_scan(scan[0], scan[1], self.A, scan[2], scan[3], self.pool, slot, off, D=self.D, z=z, dt_bias=self.bias,
                               counts=counts, state_only=True, max_row_len=longest)


def test_prompts_then_single_tokens():
    """A prompt at once, or its last tokens one by one: the same up to float32 rounding, and as the formulas have it."""
    lens, more = [23, 40, 5], 3
    layer, g = Layer(3), torch.Generator(device=DEV).manual_seed(1)
    h = torch.randn(sum(lens), 48, generator=g, device=DEV)
    slot, off = _ints([2, 0, 1]), _ints([0, 23, 63, 68])
    whole, (x, z, scan) = layer(h, slot, off)
    c_out, c_bound, c_state = conv_ref(x, layer.w, layer.b, torch.zeros_like(layer.conv), slot, off)
    check_close(scan[0].reshape(sum(lens), -1), c_out, c_bound, "convolution")
    assert torch.equal(layer.conv, c_state)
    want, bound, state, sb = scan_ref(scan[0], scan[1], layer.A, scan[2], scan[3], torch.zeros_like(layer.pool), slot, off, D=layer.D,
                                      z=z, dt_bias=layer.bias)
    check_close(whole, want, bound, "scan")
    check_close(layer.pool, state, sb, "state")
    conv, pool = layer.conv.clone(), layer.pool.clone()
    layer.conv.zero_()
    layer.pool.zero_()
    starts = off[:3].tolist()
    idx = [t for s, n in zip(starts, lens) for t in range(s, s + n - more)]
    layer(h[idx], slot, _ints([0, 20, 57, 59]))
    outs = []
    for i in range(more):
        rows = [s + n - more + i for s, n in zip(starts, lens)]
        outs.append((rows, layer(h[rows], slot, _ints([0, 1, 2, 3]), longest=1)[0]))
    assert torch.equal(layer.conv, conv)
    # both ways are within the bound of the same float64 values, and bfloat16 projections round alike
    check_close(layer.pool, state, sb, "state")
    for rows, y in outs:
        check_close(y, want[rows], bound[rows], "scan")
    assert gdr.gdr_get_status() == 0


def test_speculative_steps():
    """Verify, accept, commit: the pools stand where the accepted tokens alone would have taken them, bit for bit."""
    rows, drafts, vocab = 5, 4, 50
    layer, g = Layer(rows, seed=2), torch.Generator(device=DEV).manual_seed(3)
    embed = torch.randn(vocab, 48, generator=g, device=DEV)
    head = torch.randn(64, vocab, generator=g, device=DEV) * 0.2
    slot = _ints([3, 0, 5, 1, 4])
    prompt = torch.randint(vocab, (rows * 6,), generator=g, device=DEV)
    layer(embed[prompt], slot, _ints([6 * i for i in range(rows + 1)]))
    last = prompt.view(rows, 6)[:, -1].to(torch.int32)
    accepted = []
    for step in range(4):
        width = drafts + 1
        off = _ints([width * i for i in range(rows + 1)])
        q = torch.softmax(torch.randn(rows * width, vocab, generator=g, device=DEV), -1)
        tokens = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32).roll(1)
        tokens.view(rows, width)[:, 0] = last
        conv, pool = layer.conv.clone(), layer.pool.clone()
        y, kept = layer(embed[tokens.long()], slot, off, keep_state=False, longest=width)
        assert torch.equal(layer.conv, conv) and torch.equal(layer.pool, pool)
        p = torch.softmax(y.reshape(rows * width, -1).float() @ head, -1)
        u, v = torch.rand(rows * width, generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV)
        new, counts = gdr.gdr_accept_drafts(p, q, tokens, off, u, v, max_row_len=width)
        want = accept_ref(p, q, tokens, off, u, v, width)
        assert new.tolist() == want[0].tolist() and counts.tolist() == want[1].tolist()
        layer.commit(kept, slot, off, counts, width)
        # the accepted tokens alone, from the same state
        conv, layer.conv = layer.conv, conv
        pool, layer.pool = layer.pool, pool
        n = counts.tolist()
        keep = [b * width + t for b in range(rows) for t in range(n[b])]
        alone, _ = layer(embed[tokens[keep].long()], slot, _ints([sum(n[:b]) for b in range(rows + 1)]), longest=width)
        assert torch.equal(layer.conv, conv) and torch.equal(layer.pool, pool) and torch.equal(alone, y[keep])
        last = new[torch.arange(rows, device=DEV), (counts - 1).long()]
        accepted += n
    assert len(set(accepted)) > 1  # some drafts passed, some did not
    assert gdr.gdr_get_status() == 0


def test_counts_for_the_fold():
    """The recurrence's verify pass and fold with the counts as they come."""
    rows, width, nk, nv, K, vocab = 4, 4, 1, 2, 32, 40
    g = torch.Generator(device=DEV).manual_seed(4)
    T = rows * width
    qkv = torch.randn(T, 2 * nk * K + nv * K, generator=g, device=DEV)
    decay, beta = 0.8 + 0.2 * torch.rand(T, nv, generator=g, device=DEV), torch.rand(T, nv, generator=g, device=DEV)
    pool = torch.randn(rows + 1, nv, K, K, generator=g, device=DEV) * 0.1
    slot, off = _ints([2, 0, 4, 1]), _ints([width * i for i in range(rows + 1)])
    stride = -(-gdr.gdr_ring_record_elements(K, K, nv // nk) // 8) * 8
    ring = torch.zeros(rows, nk, width, stride, device=DEV)
    before = pool.clone()
    gdr.gdr_verify_ring(qkv, decay, beta, pool, slot, off, ring, _ints([0, 1, 2, 3]), max_row_len=width)
    q = torch.softmax(torch.randn(T, vocab, generator=g, device=DEV), -1)
    p = torch.softmax(torch.log(q) + torch.randn(T, vocab, generator=g, device=DEV), -1)
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32).roll(1)
    _, counts = gdr.gdr_accept_drafts(p, q, tokens, off, torch.rand(T, generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV),
                                      max_row_len=width)
    gdr.gdr_fold(pool, slot, ring, _ints([0, 1, 2, 3]), counts)
    n = counts.tolist()
    keep = [b * width + t for b in range(rows) for t in range(n[b])]
    gdr.gdr_fwd(qkv[keep], decay[keep], beta[keep], before, slot, _ints([sum(n[:b]) for b in range(rows + 1)]))
    assert torch.equal(pool, before)
    assert gdr.gdr_get_status() == 0


def test_one_graph_of_a_speculative_step():
    """A whole step captured once and replayed on other tokens."""
    rows, width, vocab = 3, 4, 30
    layer, g = Layer(rows, seed=5), torch.Generator(device=DEV).manual_seed(6)
    slot, off = _ints([1, 3, 0]), _ints([0, 4, 8, 12])
    h = torch.randn(12, 48, generator=g, device=DEV)
    p, q = (torch.softmax(torch.randn(12, vocab, generator=g, device=DEV), -1) for _ in range(2))
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32).roll(1)
    u, v = torch.rand(12, generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV)
    new, counts = torch.empty(rows, width, dtype=torch.int32, device=DEV), torch.empty(rows, dtype=torch.int32, device=DEV)

    def step():
        y, kept = layer(h, slot, off, keep_state=False, longest=width)
        gdr.gdr_accept_drafts(p, q, tokens, off, u, v, max_row_len=width, out=new, counts=counts)
        layer.commit(kept, slot, off, counts, width)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in (7, 8):
        g.manual_seed(seed)
        h.copy_(torch.randn(12, 48, generator=g, device=DEV))
        u.copy_(torch.rand(12, generator=g, device=DEV))
        layer.conv.zero_()
        layer.pool.zero_()
        want, want_new, want_counts = step().clone(), new.clone(), counts.clone()
        conv, pool = layer.conv.clone(), layer.pool.clone()
        layer.conv.zero_()
        layer.pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(new, want_new) and torch.equal(counts, want_counts)
        assert torch.equal(layer.conv, conv) and torch.equal(layer.pool, pool)


def test_calls_switch_to_their_tensors_device(monkeypatch):
    entered = []

    class Device(torch.cuda.device):
        def __init__(self, device):
            entered.append(getattr(device, "index", device))
            super().__init__(device)

    layer = Layer(2)
    slot, off, h = _ints([0, 1]), _ints([0, 1, 2]), torch.randn(2, 48, device=DEV)
    t = torch.softmax(torch.randn(2, 9, device=DEV), -1)
    args = t, t, _ints([1, 2]), off, torch.rand(2, device=DEV), torch.rand(2, device=DEV)
    want, drawn = layer(h, slot, off, longest=1)[0], gdr.gdr_accept_drafts(*args, max_row_len=1)[0]
    layer.conv.zero_()
    layer.pool.zero_()
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    assert torch.equal(layer(h, slot, off, longest=1)[0], want) and entered == [0, 0]
    assert torch.equal(gdr.gdr_accept_drafts(*args, max_row_len=1)[0], drawn) and entered == [0, 0, 0]
