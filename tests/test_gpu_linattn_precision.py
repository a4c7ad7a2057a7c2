"""What gdr_linattn_fwd promises of its precision, form by form: results are
rounded once, and no sum's terms are held to fewer than 16 bits on the way.

Bounds.  An operand in two bfloat16 parts is off by U16^2 of itself, the terms
of an output are history or lie in its own chunk, and a state's terms for a
bfloat16 pool have a weight in two parts, a product in two parts and a sum of
them rounded (3 U16^2 in all; three parts for a float32 pool, U16^3).  float32
sums round at most 4 max_len + 160 times (two a token and the powers of the
decay as many again, 128 terms of the readout).  The recurrent form has float32
roundings only."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.layer_helpers import U16, U32, linattn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _randn(*shape, dtype=F32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def check(out, state, ref, max_len, parts):
    """Outputs to the bound above and one rounding; parts: the form splits operands."""
    want, want_state, size, size_state = ref
    n = 4 * max_len + 160
    made = (3 if state.dtype == BF16 else U16) * U16 ** 2 if parts else 0.0
    last = U16 if out.dtype == BF16 else 0.0
    tol = (n * U32 + made + (U16 ** 2 if parts else 0.0)) * size * (1 + last) + last * want.abs() + 1e-37
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"out: {float((err / tol).max()):.3g} x the bound"
    last = U16 if state.dtype == BF16 else 0.0
    tol = (n * U32 + made) * size_state * (1 + last) + last * want_state.abs() + 1e-37
    err = (state.double() - want_state).abs()
    assert bool((err <= tol).all()), f"state: {float((err / tol).max()):.3g} x the bound"


#: rows of a call, its bound on lengths, tokens one element off 16 bytes: what takes each form
FORMS = {"chunks": ([130, 70], 0, 0), "short rows": ([16, 9], 16, 0), "short rows of pieces": ([30, 17], 32, 0),
         "any layout": ([40, 20], 0, 1)}


def _call(form, q, k, v, lam, start, off, **kw):
    """The call, its tokens laid out as the form wants them."""
    lens, hint, shift = FORMS[form]
    def lay(x):
        buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device=DEV)
        y = buf[shift:shift + x.numel()].view(x.shape)
        y.copy_(x)
        return y
    slot = torch.arange(len(lens), dtype=torch.int32, device=DEV)
    state = start.clone()
    out = gdr.gdr_linattn_fwd(lay(q), lay(k), lay(v), lam, state, slot, off, max_row_len=hint, **kw)
    assert gdr.gdr_get_status() == 0
    return out, state, linattn_ref(q, k, v, lam, start, slot, off, **kw)


def _offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pool", [BF16, F32])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (64, 128), (128, 192)])
def test_random_rows(form, pool, K, V):
    lens = FORMS[form][0]
    T, off = sum(lens), _offsets(lens)
    q, k, v = _randn(T, 2, K, dtype=BF16), _randn(T, 2, K, dtype=BF16, seed=1), _randn(T, 4, V, dtype=BF16, seed=2)
    lam = torch.tensor([1.0, 0.999, 0.97, 0.6], device=DEV)
    out, state, ref = _call(form, q, k, v, lam, _randn(2, 4, K, V, dtype=pool, seed=3), off)
    check(out, state, ref, max(lens), form != "any layout")
    # what the last rounding costs, and next to nothing more: the rest is 2^-8 of it, times what cancels
    best = (ref[0].to(BF16).double() - ref[0]).norm()
    got = (out.double() - ref[0]).norm()
    assert got <= 1.02 * best, f"{float(got / best):.4f} times the rounding's own error"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pool", [BF16, F32])
def test_history_that_cancels(form, pool):
    """State entries 1 + 2^-9 and 1 - 2^-10 (both 1 in 8 bits), read by a query of 1, -1, 1, -1, ..: what is left of
    the sum is what their roundings would take away."""
    lens, K, V = FORMS[form][0], 128, 64
    T, off = sum(lens), _offsets(lens)
    sign = 1.0 - 2.0 * (torch.arange(K, device=DEV) % 2)
    q = sign.expand(T, 1, K).to(BF16).contiguous()
    k, v = torch.zeros(T, 1, K, dtype=BF16, device=DEV), torch.ones(T, 1, V, dtype=BF16, device=DEV)
    for b in range(2):  # 1s, then what they lack
        k[off[b]] = 1.0
        k[off[b] + 1] = torch.where(sign > 0, 2.0 ** -9, -2.0 ** -10).to(BF16)
    lam = torch.ones(1, device=DEV)
    start = torch.zeros(2, 1, K, V, dtype=pool, device=DEV)
    if pool == F32:  # the same from the start
        start[1] = torch.where(sign > 0, 1 + 2.0 ** -9, 1 - 2.0 ** -10)[:, None]
        k[int(off[1]):] = 0
    out, state, ref = _call(form, q, k, v, lam, start, off, scale=1.0)
    assert float((ref[0][off[1:].long() - 1] - 0.1875).abs().max()) == 0.0
    check(out, state, ref, max(lens), form != "any layout")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pool", [BF16, F32])
def test_a_chunk_that_cancels(form, pool):
    """The same for the scores inside a chunk: 1 + 2^-9 and 1 - 2^-10 for tokens of values 1 and -1."""
    lens, K, V = FORMS[form][0], 64, 128
    T, off = sum(lens), _offsets(lens)
    odd = torch.zeros(T, dtype=torch.bool, device=DEV)
    for b in range(2):
        odd[int(off[b]) + 1:int(off[b + 1]):2] = True
    q, k = torch.zeros(T, 1, K, dtype=BF16, device=DEV), torch.zeros(T, 1, K, dtype=BF16, device=DEV)
    q[..., :2] = 1.0
    k[:, 0, 0] = 1.0
    k[:, 0, 1] = torch.where(odd, -2.0 ** -10, 2.0 ** -9).to(BF16)
    v = torch.where(odd, -1.0, 1.0)[:, None, None].expand(T, 1, V).to(BF16).contiguous()
    lam = torch.ones(1, device=DEV)
    out, state, ref = _call(form, q, k, v, lam, torch.zeros(2, 1, K, V, dtype=pool, device=DEV), off, scale=1.0)
    check(out, state, ref, max(lens), form != "any layout")


@pytest.mark.parametrize("tok,shift", [(F32, 0), (F32, 1), (BF16, 1)])
@pytest.mark.parametrize("pool", [BF16, F32])
def test_long_rows_of_the_recurrent_form(tok, shift, pool):
    """float32 tokens, and bfloat16 tokens one element off 16 bytes, past 300 tokens: float32 roundings and the last."""
    lens, K, V = [777, 1, 401], 64, 96
    T, off = sum(lens), _offsets(lens)

    def lay(x):
        buf = torch.zeros(x.numel() + 8, dtype=tok, device=DEV)
        buf[shift:shift + x.numel()].view(x.shape).copy_(x)
        return buf[shift:shift + x.numel()].view(x.shape)

    q, k, v = lay(_randn(T, 1, K)), lay(_randn(T, 1, K, seed=1)), lay(_randn(T, 2, V, seed=2))
    lam, slot = torch.tensor([0.999, 0.8], device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    start = _randn(3, 2, K, V, dtype=pool, seed=3)
    state = start.clone()
    out = gdr.gdr_linattn_fwd(q, k, v, lam, state, slot, off, max_row_len=777)
    check(out, state, linattn_ref(q, k, v, lam, start, slot, off), 777, False)
    assert gdr.gdr_get_status() == 0


def test_two_calls_at_once():
    """Calls on two streams, each with a pool, an output and a workspace of its own, as when nothing else runs."""
    lens = [2400, 70, 900]
    off, slot, lam = _offsets(lens), torch.arange(3, dtype=torch.int32, device=DEV), torch.tensor([0.99, 1.0], device=DEV)
    T, jobs = sum(lens), []
    for seed, (K, V, pool) in enumerate([(128, 128, BF16), (64, 128, F32)]):
        q, k, v = (_randn(T, n, d, dtype=BF16, seed=10 * seed + i) for i, (n, d) in enumerate([(1, K), (1, K), (2, V)]))
        start = _randn(3, 2, K, V, dtype=pool, seed=seed)
        state = start.clone()
        jobs.append(((q, k, v, lam), start, gdr.gdr_linattn_fwd(q, k, v, lam, state, slot, off, max_row_len=2400), state))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, ((q, k, v, d), start, _, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                state = start.clone()
                got[i].append((gdr.gdr_linattn_fwd(q, k, v, d, state, slot, off, max_row_len=2400), state))
    torch.cuda.synchronize()
    for i, (_, _, want, want_state) in enumerate(jobs):
        for out, state in got[i]:
            assert torch.equal(out, want) and torch.equal(state, want_state)
    assert gdr.gdr_get_status() == 0
