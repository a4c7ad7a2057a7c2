"""State space operators and verification where offsets pass 32 bits: tokens, pools and probabilities far apart."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.state_space_helpers import accept_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
FAR = 2 ** 31 + 64  # elements


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _apart(t, dim, stride):
    """t with its elements along dim that far apart."""
    st = list(t.contiguous().stride())
    st[dim] = stride
    buf = torch.zeros(sum((n - 1) * s for n, s in zip(t.shape, st)) + 1, dtype=t.dtype, device=DEV)
    out = buf.as_strided(t.shape, st)
    out.copy_(t)
    return out


@pytest.mark.parametrize("lens,bound", [([3], 3), ([40], 0)])
@pytest.mark.parametrize("what", ["tokens", "pool"])
def test_convolution(lens, bound, what):
    g = torch.Generator(device=DEV).manual_seed(1)
    T, C = sum(lens), 64
    x = torch.randn(T, C, generator=g, device=DEV).to(BF16)
    w, pool = torch.randn(C, 4, generator=g, device=DEV), torch.randn(2, C, 3, generator=g, device=DEV).to(BF16)
    slot, off = _ints([1]), _ints([0, T])
    want_pool = pool.clone()
    want = gdr.gdr_short_conv(x, w, None, want_pool, slot, off, max_row_len=bound)
    if what == "tokens":
        step = FAR // (T - 1) + 8
        step -= step % 8
        x, out = _apart(x, 0, step), torch.empty_strided((T, C), (step, 1), dtype=BF16, device=DEV)
    else:
        pool, out = _apart(pool, 0, FAR), None
    got = gdr.gdr_short_conv(x, w, None, pool, slot, off, out, max_row_len=bound)
    assert torch.equal(got, want) and torch.equal(pool, want_pool)


@pytest.mark.parametrize("lens,bound", [([3], 3), ([1], 1), ([40], 0)])
@pytest.mark.parametrize("what", ["tokens", "pool"])
def test_scan(lens, bound, what):
    g = torch.Generator(device=DEV).manual_seed(2)
    T, nv, V, K = sum(lens), 2, 32, 16
    x, dt, z = (torch.randn(T, nv, V, generator=g, device=DEV).to(BF16) for _ in range(3))
    B, C = (torch.randn(T, 1, K, generator=g, device=DEV).to(BF16) for _ in range(2))
    A, pool = -torch.rand(nv, K, V, generator=g, device=DEV), torch.randn(2, nv, K, V, generator=g, device=DEV).to(BF16)
    slot, off = _ints([1]), _ints([0, T])
    want_pool = pool.clone()
    want = gdr.gdr_selective_scan(x, dt, A, B, C, want_pool, slot, off, z=z, max_row_len=bound)
    out = None
    if what == "tokens" and T > 1:
        step = FAR // (T - 1) + 8
        step -= step % 8
        x, B = _apart(x, 0, step), _apart(B, 0, step)
        out = torch.empty_strided((T, nv, V), (step, V, 1), dtype=BF16, device=DEV)
    else:
        pool = _apart(pool, 0, FAR)
    got = gdr.gdr_selective_scan(x, dt, A, B, C, pool, slot, off, out, z=z, max_row_len=bound)
    assert torch.equal(got, want) and torch.equal(pool, want_pool)


def test_verification():
    g = torch.Generator(device=DEV).manual_seed(3)
    p, q = (torch.softmax(torch.randn(4, 100, generator=g, device=DEV), -1).to(BF16) for _ in range(2))
    args = _ints([1, 2, 3, 4]), _ints([0, 4]), torch.rand(4, generator=g, device=DEV) * 0.1, torch.rand(1, generator=g, device=DEV)
    got, n = gdr.gdr_accept_drafts(_apart(p, 0, FAR // 3 + 1), _apart(q, 0, FAR // 3 + 1), *args, max_row_len=4)
    want, m = accept_ref(p, q, *args, 4)
    assert got.tolist() == want.tolist() and n.tolist() == m.tolist() and n.tolist()[0] > 1


def test_a_padding_row_of_many_tokens():
    """Its output is cleared whole, and the states stay."""
    T, nv, V = 2 ** 24 + 5, 1, 64
    one = torch.randn(1, nv, V, device=DEV).to(BF16).expand(T, nv, V)
    bc = torch.randn(1, 1, 16, device=DEV).to(BF16).expand(T, 1, 16)
    pool = torch.randn(1, nv, 16, V, device=DEV)
    keep = pool.clone()
    out = torch.full((T + 1, nv, V), 7.0, dtype=BF16, device=DEV)
    gdr.gdr_selective_scan(one, one, -torch.ones(nv, 16, V, device=DEV), bc, bc, pool, _ints([-1]), _ints([0, T]), out[:T])
    assert not bool(out[:T].any()) and bool((out[T] == 7.0).all()) and torch.equal(pool, keep)
    conv = torch.randn(1, V, 3, device=DEV)
    kept = conv.clone()
    out.fill_(7.0)
    gdr.gdr_short_conv(one[:, 0], torch.randn(V, 4, device=DEV), None, conv, _ints([-1]), _ints([0, T]),
                       out[:T, 0])
    assert not bool(out[:T].any()) and bool((out[T] == 7.0).all()) and torch.equal(conv, kept)
