"""Verification where the draw's share of the sum lies on a running sum, or next to one: a token with a weight is
drawn in any case, and the right one wherever the distance is more than the sums' own error."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.test_gpu_accept import BF16, DEV, F32, _clean_status, _floats  # noqa: F401

pytestmark = pytest.mark.gpu


def _draw(p, v):
    """The token of every row of p, by the number v."""
    n = p.shape[0]
    got, counts = gdr.gdr_accept_drafts(p, None, torch.zeros(n, dtype=torch.int32, device=DEV), torch.arange(n + 1, dtype=torch.int32, device=DEV),
                                        torch.zeros(n, device=DEV), _floats([v]).expand(n).contiguous(), max_row_len=1)
    assert bool((counts == 1).all())
    return got[:, 0].long()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 40, 70, 100, 200])
@pytest.mark.parametrize("vocab", [512, 1000, 4096, 32000])
def test_a_share_on_a_border_draws_a_token(dtype, rows, vocab):
    """The second half of the weights repeats the first, and the number is a half: the share is the first half's sum
    itself, where roundings of running sums go either way.  One to eight blocks a row."""
    g = torch.Generator(device=DEV).manual_seed(rows + vocab)
    for spread in (3.0, 4.0):
        for order in (False, True):
            half = torch.softmax(spread * torch.randn(rows, vocab // 2, generator=g, device=DEV), 1).to(dtype)
            other = half[:, torch.randperm(vocab // 2, generator=g, device=DEV)] if order else half
            p = torch.cat([half, other], 1)
            got = _draw(p, 0.5)
            assert int(got.min()) >= 0 and int(got.max()) < vocab
            assert bool((p.gather(1, got[:, None]) > 0).all())
            # the sums' error is far below the weights around the middle: one of the weights next to the border
            upto = p.double().cumsum(1)
            total = upto[:, -1:]
            mine, before = upto.gather(1, got[:, None]), upto.gather(1, got[:, None]) - p.double().gather(1, got[:, None])
            near = 2.0 ** -36 * total
            assert bool((before <= total / 2 + near).all()) and bool((mine >= total / 2 - near).all())
