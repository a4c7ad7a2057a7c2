"""The selective scan's output between its inputs' values, as parts of one projection lie, and on them."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.test_gpu_scan import BF16, DEV, F32, Case, _clean_status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,bound", [([1], 1), ([1] * 9, 1), ([5, 1, 7], 8), ([100, 3, 41], 0)])
@pytest.mark.parametrize("types", [(BF16, BF16, F32), (F32, F32, F32)])
@pytest.mark.parametrize("layout", ["token", "head", "head outside"])
def test_output_between_inputs(lens, bound, types, layout):
    c = Case(lens, 2, 4, 16, 32, types, seed=21)
    T, tok = sum(lens), types[0]
    want, state = c.run(max_row_len=bound)
    if layout == "token":  # a token's x, out, dt, B and C one behind the other
        wide = torch.zeros(T, 3 * 128 + 2 * 32, dtype=tok, device=DEV)
        x, out, dt = (wide[:, i * 128:(i + 1) * 128].view(T, 4, 32) for i in range(3))
        B, C = (wide[:, 384 + i * 32:416 + i * 32].view(T, 2, 16) for i in range(2))
        B.copy_(c.B), C.copy_(c.C)
        c.B, c.C = B, C
    else:  # a head's x, out and dt, heads within a token or tokens within a head
        wide = torch.zeros((T, 4, 96) if layout == "head" else (4, T, 96), dtype=tok, device=DEV)
        x, out, dt = (t if layout == "head" else t.transpose(0, 1) for t in wide.split(32, -1))
    x.copy_(c.x), dt.copy_(c.dt)
    c.x, c.dt = x, dt
    pool = c.pool.clone()
    c.run(pool, out=out, max_row_len=bound)
    assert torch.equal(out, want) and torch.equal(pool, state)


def test_output_on_an_input_is_refused():
    c = Case([3, 4], 1, 2, 16, 32, (BF16, BF16, F32), seed=22)
    wide = torch.zeros(8, 4, 32, dtype=BF16, device=DEV)[:7]
    for name, view in (("x", wide[:, :2]), ("z", wide[:, 2:]), ("dt", wide[:, 1:3])):
        old = getattr(c, name)
        setattr(c, name, view)
        out = wide.as_strided((7, 2, 32), view.stride(), view.storage_offset() + (0 if name == "dt" else 8))
        with pytest.raises(gdr.GdrError, match=f"out lies on {name}"):
            c.run(out=out)
        setattr(c, name, old)
