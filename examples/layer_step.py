"""One serving step of a KDA layer with 8-bit projections, from a scheduler's lengths to the new
residual stream:

  kda_batch_maps    running order, cu_seqlens, state slots, cache pages and slots of the batch
  kda_norm_quant    residual addition, RMS norm, e4m3 output
  kda_fp8_matmul    q | k | v | raw_g | gate | raw_beta
  kda_mixed_batch   the recurrence (decodes and prefills), kda_fused_decode with the gated norm
                    where every request decodes
  kda_norm_quant    the recurrence's outputs to e4m3 (no norm)
  kda_fp8_matmul    the output projection

Run:  python examples/layer_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def quantise_weight(w):
    """e4m3 [N, K] and fp32 scales [ceil(N / 128), ceil(K / 128)] of a weight: done once, when it is loaded."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    top = torch.nn.functional.pad(w.abs().float(), (0, kb * 128 - k, 0, nb * 128 - n)).view(nb, 128, kb, 128).amax((1, 3))
    scales = top.clamp_min(448 * 2.0 ** -126) / 448
    full = scales.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    q = torch.empty(n, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=w.device)[:, :k]   # rows on 16-byte boundaries
    q.copy_((w.float() / full).clamp(-448, 448).to(torch.float8_e4m3fn))
    return q, scales


class KdaLayer:
    """A layer's weights and state pool; step() runs one batch through it."""

    def __init__(self, hidden, heads, dim, num_slots, *, num_pages=256, page_size=16, device="cuda", seed=0):
        from linear_attention_state_recurrent_gb300 import kda
        self.kda, self.hidden, self.H, self.D = kda, hidden, heads, dim
        self.num_pages, self.page_size = num_pages, page_size
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, device=device, generator=g)

        hd = heads * dim
        self.parts = (3 * hd, hd, hd, heads)                      # q | k | v, raw_g, gate, raw_beta
        self.w_in, self.w_in_scales = quantise_weight(randn(sum(self.parts), hidden) * hidden ** -0.5)
        self.w_out, self.w_out_scales = quantise_weight(randn(hidden, hd) * hd ** -0.5)
        self.norm_weight = 1 + 0.1 * randn(hidden)
        self.A_log, self.dt_bias = 0.5 * randn(heads), 0.1 * randn(hd)
        self.gated_norm_weight = torch.ones(dim, device=device)
        self.state = torch.zeros(num_slots, heads, dim, dim, device=device)

    def maps(self, query_lens, context_lens, state_slots, block_table, free_pages, free_count, num_tokens, err_flags=None):
        return self.kda.kda_batch_maps(query_lens, context_lens, state_slots, block_table, free_pages, free_count,
                                       self.page_size, num_pages=self.num_pages, num_tokens=num_tokens, err_flags=err_flags)

    def step(self, x, residual, maps, query_lens_host, err_flags=None):
        """x, residual: bf16 [tokens, hidden], rows in the maps' running order; query_lens_host: the scheduler's own
        lengths, which size the launches. Returns (output, residual) for the next layer."""
        kda, H, D = self.kda, self.H, self.D
        q, scales, residual = kda.kda_norm_quant(x, self.norm_weight, 1e-5, residual=residual)
        n = sum(self.parts)   # rows on 16-byte boundaries, as the recurrence's loads want them
        proj = torch.empty(x.shape[0], -(-n // 8) * 8, dtype=torch.bfloat16, device=x.device)[:, :n]
        kda.kda_fp8_matmul(q, scales, self.w_in, self.w_in_scales, out=proj, err_flags=err_flags)
        qkv, raw_g, gate, raw_beta = torch.split(proj, self.parts, dim=1)
        decodes = sum(n == 1 for n in query_lens_host)
        common = (qkv, raw_g, raw_beta, self.A_log, self.dt_bias, None, self.state, maps.state_indices)
        if decodes == len(query_lens_host):
            out, _ = kda.kda_fused_decode(*common, norm=(gate, self.gated_norm_weight, 1e-5), err_flags=err_flags)
        else:
            order = sorted(range(len(query_lens_host)), key=lambda r: query_lens_host[r] != 1)
            cu = torch.zeros(len(order) + 1, dtype=torch.int32)
            cu[1:] = torch.tensor([query_lens_host[r] for r in order]).cumsum(0)
            out, _ = kda.kda_mixed_batch(*common, maps.cu_seqlens, decodes, cu_seqlens_host=cu, err_flags=err_flags)
            o = out.view(-1, H, D).float()
            out = (o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-5) * self.gated_norm_weight *
                   torch.sigmoid(gate.reshape(-1, H, D).float())).to(torch.bfloat16).view(-1, H * D)
        q, scales, _ = kda.kda_norm_quant(out)
        return kda.kda_fp8_matmul(q, scales, self.w_out, self.w_out_scales, err_flags=err_flags), residual


def main():
    torch.manual_seed(0)
    layer = KdaLayer(hidden=1024, heads=4, dim=128, num_slots=16)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((4, 16), -1, dtype=torch.int32, device="cuda")
    free, count, slots = torch.arange(255, -1, -1, dtype=torch.int32, device="cuda"), i32([256]), i32([3, 7, 1, 9])
    # a first step prefills three requests and leaves the fourth waiting; then all four decode or prefill
    context = [0, 0, 0, 0]
    for lens in ([70, 1, 130, 0], [1, 1, 1, 50], [1, 1, 1, 1]):
        tokens = sum(lens)
        maps = layer.maps(i32(lens), i32(context), slots, table, free, count, tokens, err)
        x, residual = torch.randn(2, tokens, layer.hidden, device="cuda").to(torch.bfloat16)
        y, residual = layer.step(x, residual, maps, lens, err)
        count.copy_(maps.free_left)
        context = [c + n for c, n in zip(context, lens)]
        print(f"step of {tokens} tokens: |y| {y.float().norm().item():.3f}, pages left {count.item()}, "
              f"first slots {maps.slot_map[:4].tolist()}, errors {err.item()}")
    assert err.item() == 0 and torch.isfinite(y.float()).all()


if __name__ == "__main__":
    main()
