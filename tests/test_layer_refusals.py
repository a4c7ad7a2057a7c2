"""What the layer operators' Python calls refuse before they ask anything of
the GPU: arguments that are no tensors, and tensors of the host."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr

X = torch.zeros(4, 64)
BAD = [None, 3, [1.0, 2.0], "x"]


@pytest.mark.parametrize("bad", BAD)
def test_no_tensors(bad):
    for call in [lambda: gdr.gdr_gate_norm(bad, X), lambda: gdr.gdr_residual_norm(X, bad, None)]:
        with pytest.raises(TypeError, match="torch.Tensor"):
            call()
    if bad is not None:
        for call in [lambda: gdr.gdr_gate_norm(X, bad), lambda: gdr.gdr_residual_norm(bad, X, None)]:
            with pytest.raises(TypeError, match="torch.Tensor"):
                call()


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("which", range(7))
@pytest.mark.parametrize("out", [None, torch.zeros(4, 1, 64)])
def test_linear_attention_takes_tensors(which, bad, out):
    q, rows = X.view(4, 1, 64), torch.arange(5, dtype=torch.int32)
    args = [q, q, q, torch.ones(1), torch.zeros(4, 1, 64, 64), rows[:4], rows]
    args[which] = bad
    # the tensors are of the host, which is refused too where it is seen first
    with pytest.raises((TypeError, ValueError), match="torch.Tensor|CUDA tensor"):
        gdr.gdr_linattn_fwd(*args, out)


def test_tensors_of_the_host():
    for call in [lambda: gdr.gdr_gate_norm(X, X), lambda: gdr.gdr_residual_norm(X, X, None)]:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
