"""Corners of the layer operators that a call meets seldom."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.layer_helpers import check_linattn, linattn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _randn(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("pool", [BF16, F32])
def test_units_dealt_by_load(K, pool):
    """The first chunk's tokens arrive right behind the deal of the units, and nothing of the deal may lie where they
    do: the first tokens weigh most here (a state that never fades, keys of one sign), and calls repeat bit for bit."""
    lens, nv = [513, 640, 90, 700, 515], 48
    T = sum(lens)
    q, k = _randn(T, nv // 2, K, dtype=BF16), _randn(T, nv // 2, K, dtype=BF16, seed=1).abs()
    v, lam = _randn(T, nv, 64, dtype=BF16, seed=2), torch.ones(nv, device=DEV)
    off = torch.tensor([sum(lens[:i]) for i in range(6)], dtype=torch.int32, device=DEV)
    slot = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32, device=DEV)
    start = _randn(5, nv, K, 64, dtype=pool, seed=3)
    assert gdr.gdr_linattn_workspace_bytes(q, k, v, lam, start, slot, off, max_row_len=700) == 0
    first = None
    for _ in range(30):
        state = start.clone()
        out = gdr.gdr_linattn_fwd(q, k, v, lam, state, slot, off, max_row_len=700)
        if first is None:
            first = out, state
            check_linattn(out, state, linattn_ref(q, k, v, lam, start, slot, off), 700, True)
        assert torch.equal(out, first[0]) and torch.equal(state, first[1])
    assert gdr.gdr_get_status() == 0
