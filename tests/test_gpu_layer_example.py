"""The example layer: prompts, then single tokens, against the same network
in float64 over the whole sequence, and against the prompt in two pieces."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.layer_helpers import linattn_ref, norm_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("linear_attention_layer",
                                                  os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _float64(layers, x, lengths):
    """The stack over whole rows, from zero states."""
    off = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)])
    slots = torch.arange(len(lengths))
    h, y = x.double(), norm_ref(None, residual=x, pre=True, pre_w=layers[0].pre_norm)[1]
    for i, m in enumerate(layers):
        T, nk, nv, K, V = x.shape[0], m.nk, m.nv, m.K, m.V
        z = y @ m.w_in.double()
        qk = torch.nn.functional.silu(z[:, :2 * nk * K])
        pool = torch.zeros(len(lengths), nv, K, V, dtype=torch.float64, device=x.device)
        o = linattn_ref(qk[:, :nk * K].view(T, nk, K), qk[:, nk * K:].view(T, nk, K),
                        z[:, 2 * nk * K:2 * nk * K + nv * V].view(T, nv, V), m.log_decay, pool, slots, off,
                        decay_is_log=True)[0]
        o = norm_ref(o, gate=z[:, 2 * nk * K + nv * V:].view(T, nv, V), act="silu", post=True, post_w=m.head_norm)[1]
        block = o.reshape(T, nv * V) @ m.w_out.double()
        w = layers[i + 1].pre_norm if i + 1 < len(layers) else None
        h, y = norm_ref(block, post=True, post_w=m.post_norm, residual=h, scale=0.5, pre=True, pre_w=w)
    return y


def test_prompts_then_tokens(ex):
    g = torch.Generator(device="cuda").manual_seed(1)
    layers = [ex.LinearAttentionLayer(256, 2, 4, 64, 64, 6, generator=g, state_dtype=torch.float32) for _ in range(2)]
    lengths, extra = [70, 1, 130], 3
    total = [n + extra for n in lengths]
    x = torch.randn(sum(total), 256, generator=g, device="cuda").bfloat16()
    rows = [x[sum(total[:i]):sum(total[:i + 1])] for i in range(3)]
    slot = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda")
    got = [list(t.split(1)) for t in ex.run_stack(layers, torch.cat([r[:n] for r, n in zip(rows, lengths)]), slot, off,
                                                  130).split(lengths)]
    one = torch.arange(4, dtype=torch.int32, device="cuda")
    for t in range(extra):
        y = ex.run_stack(layers, torch.cat([r[n + t:n + t + 1] for r, n in zip(rows, lengths)]), slot, one, 1)
        for i in range(3):
            got[i].append(y[i:i + 1])
    got = torch.cat([torch.cat(r) for r in got])
    assert gdr.gdr_get_status() == 0
    ref = _float64(layers, x, total)
    # a dozen roundings to bfloat16 a layer, rms 2^-8 / sqrt(3) of the rms each, none amplified by the norms:
    # sqrt(24) x 2.3e-3 = 1.1e-2; the bound leaves a factor of two
    rel = float((got.double() - ref).norm() / ref.norm())
    assert rel <= 2.3e-2, rel


def test_example_runs(ex, capsys):
    ex.main()
    assert "8 tokens" in capsys.readouterr().out
