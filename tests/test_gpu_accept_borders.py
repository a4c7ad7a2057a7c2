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


@pytest.mark.parametrize("behind", [False, True])
def test_sums_of_many_tokens_by_one_block(behind):
    """2^27 weights of a row that one block sums up, 2^18 of them a lane: halves of equal sums, one of them larger by
    2^-34 of the total.  The share then lies 2^-35 of it away from the border between the halves, and a sum is good to
    2^-36 at worst: 64 additions to a pair of float32 lose 64^2 / 2 * 2^-48 of it, joining 64 such parts as pairs
    64 * 3 * 2^-48, and those in double, the warp's lanes and the warps far less."""
    n = 1 << 27
    g = torch.Generator(device=DEV).manual_seed(3)
    w = torch.exp(3 * torch.randn(n // 2, generator=g, device=DEV))
    w[777], w[-1] = 1.0, 100.0  # which takes the difference, and the weights beside the border
    p = torch.cat([w, w.flip(0)])
    at = n - 1 - 777 if behind else 777
    p[at] = 1.0 + float(p.double().sum()) * 2.0 ** -34
    exact = p.double()
    first, whole = exact[:n // 2].sum(), exact.sum()
    border = float((whole / 2 - first) / whole)
    assert 2.0 ** -35.1 < (border if behind else -border) < 2.0 ** -34.9
    got = _draw(p[None, :].expand(160, n), 0.5)
    assert got.tolist() == [n // 2 if behind else n // 2 - 1] * 160
