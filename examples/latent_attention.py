"""Latent attention of one decoder layer on the library's kernels: ragged prompts are cached and attended in
the expanded form, then each sequence decodes tokens in the absorbed form over the paged FP8 cache.

    python examples/latent_attention.py [--steps 4]

Weights are random. Each decoded token is computed in both forms, which have to agree: the absorbed form
multiplies the cached latents directly, the expanded one first expands them to every head's keys and values.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_bfp8_amd as bfp8  # noqa: E402

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128


def quantize_weight(w: torch.Tensor):
    """bf16 [N, K] -> (e4m3 codes, UE8M0 codes of its 128x128 blocks, the values they stand for in bf16)."""
    n, k = w.shape
    blocks = w.float().view(n // 128, 128, k // 128, 128)
    s = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax(dim=(1, 3)).clamp(min=1e-10) / 448)))
    codes = (blocks / s[:, None, :, None]).to(torch.float8_e4m3fn)
    values = (codes.float() * s[:, None, :, None]).view(n, k).to(torch.bfloat16)
    e = bfp8.ue8m0_scales((torch.log2(s) + 127).to(torch.uint8))
    return codes.view(n, k).view(torch.uint8), e, values


class LatentLayer:
    """The attention half of a decoder layer, with its slice of a paged cache."""

    def __init__(self, hidden: int, heads: int, pages: int, page: int, device, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return quantize_weight((torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16))

        self.heads, self.page, self.scale = heads, page, (NOPE + ROPE) ** -0.5
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.latent_norm = torch.ones(LATENT, dtype=torch.bfloat16, device=device)
        # queries and latents in one product; its 640 latent rows are 512 + 64 and 64 of padding to whole blocks
        self.w_in = weight(heads * (NOPE + ROPE) + LATENT + 2 * ROPE, hidden)
        self.w_up = weight(heads * (NOPE + VDIM), LATENT)
        self.w_out = weight(hidden, heads * VDIM)
        up = self.w_up[2].view(heads, NOPE + VDIM, LATENT)
        self.up_keys = up[:, :NOPE].contiguous()  # [H, 128, 512]: queries into the latent space
        self.up_values = up[:, NOPE:].transpose(1, 2).contiguous()  # [H, 512, 128]: its outputs out of it
        self.cache = torch.zeros(pages, page, bfp8.LATENT_ROW, dtype=torch.uint8, device=device)
        self.scales = torch.full((pages, page), 127, dtype=torch.uint8, device=device)

    def project(self, x, residual, positions, slots):
        """Norm, projections and rotary embedding of new tokens, which go to the cache. Returns the queries
        [T, H, 192] and the residual stream."""
        q8, s, stream = bfp8.rmsnorm_quant_ue8m0(x, self.norm, residual=residual)
        y = bfp8.gemm_ue8m0(q8, s, self.w_in[0], self.w_in[1])
        split = self.heads * (NOPE + ROPE)
        q = y[:, :split].view(-1, self.heads, NOPE + ROPE).clone()
        kv = y[:, split:split + LATENT + ROPE].clone()
        angle = positions[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, device=x.device) / ROPE)
        cos, sin = angle.cos(), angle.sin()

        def rotate(t, c, s):
            a, b = t[..., ::2].float(), t[..., 1::2].float()
            return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2).to(t.dtype)

        q[..., NOPE:] = rotate(q[..., NOPE:], cos[:, None], sin[:, None])
        kv[:, LATENT:] = rotate(kv[:, LATENT:], cos, sin)
        bfp8.latent_cache_write(kv, slots, self.cache, self.scales, norm_weight=self.latent_norm)
        return q, stream

    def output(self, heads_out, stream):
        q8, s = bfp8.quant_act_ue8m0(heads_out.reshape(heads_out.shape[0], -1))
        return bfp8.gemm_ue8m0(q8, s, self.w_out[0], self.w_out[1]), stream

    def expanded(self, q, cu_q, table, cu_k, total):
        """The cached tokens of each sequence, expanded by the up projection straight from their codes."""
        codes, e, rope = bfp8.latent_cache_gather(self.cache, self.scales, table, cu_k, total)
        kv = bfp8.gemm_ue8m0(codes, e, self.w_up[0], self.w_up[1]).view(total, self.heads, NOPE + VDIM)
        return bfp8.latent_attention_expanded(q, kv, rope, cu_q, cu_k, self.scale)

    def absorbed(self, q, lens, table):
        """One new token a sequence: the up projection is applied to the query and to the output instead."""
        into = torch.bmm(q[..., :NOPE].transpose(0, 1).contiguous(), self.up_keys).transpose(0, 1)
        o = bfp8.latent_attention(torch.cat([into, q[..., NOPE:]], dim=-1), self.cache, self.scales, table, lens, self.scale)
        return torch.bmm(o.transpose(0, 1).contiguous(), self.up_values).transpose(0, 1)


def run(device, lens=(37, 130, 1, 64), hidden=1024, heads=16, page=16, steps=4, seed=0) -> float:
    """Caches prompts, decodes `steps` tokens a sequence and returns the largest relative difference of the two
    forms' outputs."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    lens, b = list(lens), len(lens)
    width = -(-(max(lens) + steps) // page)
    layer = LatentLayer(hidden, heads, b * width + 1, page, device, seed)
    table = torch.randperm(b * width, generator=g, device=device).view(b, width).to(torch.int32)

    def starts(n):
        return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=device)

    def slots(seq, pos):
        return table[seq, pos // page].long() * page + pos % page

    def tokens(t):
        x = torch.randn(2, t, hidden, generator=g, device=device).to(torch.bfloat16)
        return x[0], x[1]

    # prompts
    seq = torch.repeat_interleave(torch.arange(b, device=device), torch.tensor(lens, device=device))
    pos = torch.cat([torch.arange(n, device=device) for n in lens])
    x, residual = tokens(sum(lens))
    q, stream = layer.project(x, residual, pos, slots(seq, pos))
    cu = starts(lens)
    layer.output(layer.expanded(q, cu, table, cu, sum(lens)), stream)

    worst = 0.0
    for _ in range(steps):
        pos = torch.tensor(lens, device=device)
        x, residual = tokens(b)
        q, stream = layer.project(x, residual, pos, slots(torch.arange(b, device=device), pos))
        lens = [n + 1 for n in lens]
        o = layer.absorbed(q, torch.tensor(lens, dtype=torch.int32, device=device), table)
        layer.output(o, stream)
        same = layer.expanded(q, starts([1] * b), table, starts(lens), sum(lens))
        worst = max(worst, float((o.float() - same.float()).norm() / same.float().norm()))
    return worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=4)
    print(f"absorbed and expanded outputs differ by {run(torch.device('cuda'), steps=parser.parse_args().steps):.2e} of their norm")
