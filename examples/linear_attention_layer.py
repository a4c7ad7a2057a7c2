"""One decayed linear attention layer in serving, on the library's entry points.

    residual stream -> gdr_residual_norm -> [Q | K | V | gate] projection ->
    gdr_linattn_fwd over the slot pool -> gdr_gate_norm (per head) -> output
    projection -> gdr_residual_norm of the next layer (adds this one's output)

A ragged batch of prompts goes through a stack of such layers, then tokens one
at a time; the states live in each layer's pool, indexed by slot, so requests
of any age share a batch.  Projections are library matrix products.

    python examples/linear_attention_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_gdr_gb300 as gdr  # noqa: E402


class LinearAttentionLayer:
    """width -> nk key heads of K, nv value heads of V -> width; a pool of `slots` states."""

    def __init__(self, width, nk, nv, K, V, slots, *, generator, state_dtype=torch.bfloat16, device="cuda"):
        def normal(*shape):
            return torch.randn(*shape, generator=generator, device=device) * shape[0] ** -0.5

        self.nk, self.nv, self.K, self.V = nk, nv, K, V
        self.pre_norm = torch.ones(width, device=device)
        self.post_norm = torch.full((width,), 0.5, device=device)
        self.head_norm = torch.ones(V, device=device)
        self.w_in = normal(width, 2 * nk * K + 2 * nv * V).bfloat16()
        self.w_out = normal(nv * V, width).bfloat16()
        # half-lives from under one token to hundreds, one for each head
        self.log_decay = -torch.exp2(-8.0 * torch.arange(1, nv + 1, device=device, dtype=torch.float32) / nv)
        self.pool = torch.zeros(slots, nv, K, V, dtype=state_dtype, device=device)

    def attend(self, normed, slot_idx, offsets, max_row_len):
        """The layer between its two norms: [T, width] -> [T, width]."""
        T, nk, nv, K, V = normed.shape[0], self.nk, self.nv, self.K, self.V
        x = normed @ self.w_in
        qk = torch.nn.functional.silu(x[:, :2 * nk * K])
        o = gdr.gdr_linattn_fwd(qk[:, :nk * K].view(T, nk, K), qk[:, nk * K:].view(T, nk, K),
                                x[:, 2 * nk * K:2 * nk * K + nv * V].view(T, nv, V), self.log_decay, self.pool, slot_idx,
                                offsets, decay_is_log=True, max_row_len=max_row_len)
        o = gdr.gdr_gate_norm(o, x[:, 2 * nk * K + nv * V:].view(T, nv, V), self.head_norm)
        return o.view(T, nv * V) @ self.w_out


def run_stack(layers, x, slot_idx, offsets, max_row_len, residual_scale=0.5):
    """x [T, width] through the layers; each boundary (the layer's output norm,
    its scale, the residual add and the next layer's norm) is one call."""
    residual, normed = gdr.gdr_residual_norm(None, x, layers[0].pre_norm)
    for i, layer in enumerate(layers):
        block = layer.attend(normed, slot_idx, offsets, max_row_len)
        last = i + 1 == len(layers)
        residual, normed = gdr.gdr_residual_norm(block, residual, None if last else layers[i + 1].pre_norm,
                                                 post_weight=layer.post_norm, residual_scale=residual_scale)
    return normed


def main():
    g = torch.Generator(device="cuda").manual_seed(0)
    layers = [LinearAttentionLayer(1024, 8, 8, 128, 128, 16, generator=g) for _ in range(2)]
    lengths = [700, 33, 5]
    offsets = torch.tensor([0, 700, 733, 738], dtype=torch.int32, device="cuda")
    slot_idx = torch.tensor([3, 0, 9], dtype=torch.int32, device="cuda")
    prompts = torch.randn(sum(lengths), 1024, generator=g, device="cuda").bfloat16()
    y = run_stack(layers, prompts, slot_idx, offsets, max(lengths))
    token = y[offsets[1:].long() - 1]
    one_each = torch.arange(4, dtype=torch.int32, device="cuda")
    for _ in range(8):
        token = run_stack(layers, token, slot_idx, one_each, 1)
    torch.cuda.synchronize()
    assert gdr.gdr_get_status() == 0
    print("prompt outputs", tuple(y.shape), "then 8 tokens a request; last rms", float(token.float().pow(2).mean().sqrt()))


if __name__ == "__main__":
    main()
