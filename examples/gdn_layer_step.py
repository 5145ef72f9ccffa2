"""Serving steps of a layer with the gated delta rule (one decay per head, shared key heads) and 16-bit projections, from a
scheduler's lengths on the GPU to the new residual stream, captured once in a CUDA graph and replayed for other lengths:

  kda_batch_maps          running order, cu_seqlens and state slots of the batch
  kda_matmul              q | k | v with SiLU, the decays' and write strengths' inputs, the output gate with bias and sigmoid
  kda_gdn_chunk_prefill   the recurrence over requests of any lengths (kda_gdn_decode where every request decodes)
  kda_matmul              the output projection, added to the residual

Run:  python examples/gdn_layer_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class GdnLayer:
    """A layer's weights and state pool; step() runs one batch through it."""

    def __init__(self, hidden, key_heads, value_heads, dim, num_slots, *, device="cuda", seed=0):
        from linear_attention_state_recurrent_gb300 import kda
        self.kda, self.hidden, self.Hk, self.Hv, self.D = kda, hidden, key_heads, value_heads, dim
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, device=device, generator=g)

        def weight(n, k):
            return (randn(n, k) * k ** -0.5).to(torch.bfloat16)

        self.w_qkv = weight((2 * key_heads + value_heads) * dim, hidden)
        self.w_ab = weight(-(-2 * value_heads // 8) * 8, hidden)          # raw_g | raw_beta, rows on 16-byte boundaries
        self.w_gate, self.gate_bias = weight(value_heads * dim, hidden), randn(value_heads * dim).to(torch.bfloat16)
        self.w_out = weight(hidden, value_heads * dim)
        self.A_log, self.dt_bias = 0.5 * randn(value_heads), -2 + randn(value_heads)
        self.state = torch.zeros(num_slots, value_heads, dim, dim, device=device)

    def step(self, x, residual, cu_seqlens, state_indices, *, decode=False, out=None, err_flags=None):
        """x, residual: bf16 [rows, hidden] in the maps' running order; rows behind the last request are carried through the
        projections alone. Returns the new residual."""
        kda, Hv = self.kda, self.Hv
        qkv = kda.kda_matmul(x, self.w_qkv, activation="silu", err_flags=err_flags)
        ab = kda.kda_matmul(x, self.w_ab, err_flags=err_flags)
        gate = kda.kda_matmul(x, self.w_gate, bias=self.gate_bias, activation="sigmoid", err_flags=err_flags)
        o = torch.zeros_like(gate) if out is None else out
        args = (qkv, ab[:, :Hv], ab[:, Hv:2 * Hv], self.A_log, self.dt_bias, self.state, state_indices)
        if decode:
            kda.kda_gdn_decode(*args, num_k_heads=self.Hk, out=o, err_flags=err_flags)
        else:
            kda.kda_gdn_chunk_prefill(*args, cu_seqlens, num_k_heads=self.Hk, out=o, err_flags=err_flags)
        return kda.kda_matmul(o * gate, self.w_out, residual=residual, err_flags=err_flags)


def main():
    torch.manual_seed(0)
    layer = GdnLayer(hidden=512, key_heads=2, value_heads=4, dim=128, num_slots=8)
    kda, rows = layer.kda, 256

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    # what the graph reads: the requests' lengths and rows, for at most `rows` of them
    lens, context, slots, err = i32([0] * 4), i32([0] * 4), i32([3, 7, 1, 6]), i32([0])
    x, residual = torch.zeros(2, rows, layer.hidden, dtype=torch.bfloat16, device="cuda")
    table, pages, count = i32([[-1] * 64] * 4), torch.arange(256, dtype=torch.int32, device="cuda"), i32([256])
    maps = kda.make_batch_maps(4, rows, "cuda")

    def step():
        kda.kda_batch_maps(lens, context, slots, table, pages, count, 16, num_pages=256, out=maps, err_flags=err)
        return layer.step(x, residual, maps.cu_seqlens, maps.state_indices, err_flags=err)

    step()                                                               # the kernels' first calls are not captured
    torch.cuda.synchronize()
    layer.state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for n in ([70, 1, 130, 0], [1, 1, 1, 50], [1, 1, 1, 1]):
        lens.copy_(i32(n))
        x.copy_(torch.randn(rows, layer.hidden, device="cuda"))
        residual.copy_(torch.randn(rows, layer.hidden, device="cuda"))
        graph.replay()
        count.copy_(maps.free_left)
        context += lens
        print(f"step of {sum(n)} tokens: |y| {y[:sum(n)].float().norm().item():.3f}, |state| {layer.state.norm().item():.3f}, errors {err.item()}")
    assert err.item() == 0 and torch.isfinite(y.float()).all()


if __name__ == "__main__":
    main()
