"""The short convolution over very many rows."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.test_gpu_short_conv import BF16, Case, _clean_status  # noqa: F401

pytestmark = pytest.mark.gpu


def test_very_many_rows_of_any_length():
    """Without a bound on their lengths, single tokens among some long rows: the bits of the bounded calls."""
    n = 200001
    lens = [1] * n
    lens[7], lens[n // 2], lens[n - 3] = 700, 900, 0
    c = Case(lens, 16, 4, BF16, seed=12)
    pool = c.pool.clone()
    out = gdr.gdr_short_conv(*c.args(pool))
    start = 0
    again = c.pool.clone()
    for b, e, bound in ((0, 7, 1), (7, 8, 0), (8, n // 2, 1), (n // 2, n // 2 + 1, 0), (n // 2 + 1, n, 1)):
        T = int(c.off[e]) - start
        got = gdr.gdr_short_conv(c.x[start:start + T], c.w, c.bias, again, c.slot[b:e], c.off[b:e + 1] - start, max_row_len=bound)
        assert torch.equal(got, out[start:start + T])
        start += T
    assert torch.equal(pool, again)


@pytest.mark.parametrize("tok", [BF16, torch.float32])
@pytest.mark.parametrize("C", [64, 1028, 33])
@pytest.mark.parametrize("longest", range(1, 10))
def test_rows_have_the_same_bits_in_either_form(tok, C, longest):
    """Rows that are taken whole, and the same ones by runs of tokens."""
    lens = [longest, 0, 1] + [1 + (7 * i) % longest for i in range(40)]
    c = Case(lens, C, 4, tok, seed=longest)
    pool, again = c.pool.clone(), c.pool.clone()
    out = gdr.gdr_short_conv(*c.args(pool), max_row_len=longest)
    assert torch.equal(gdr.gdr_short_conv(*c.args(again)), out) and torch.equal(again, pool)
