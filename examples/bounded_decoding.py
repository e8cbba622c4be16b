"""Decoding in bounded memory: a latent-attention layer whose weights are 8-bit integers and whose cache holds at most
`limit` tokens a sequence. Attention over the paged FP8 cache records how much weight every cached token gathers; a
sequence that has reached the limit is cut down to `budget` tokens, its most recent ones and those with most weight.

    python examples/bounded_decoding.py [--steps 200] [--budget 64]

Weights and inputs are random. Prints how far the outputs are from those of the same layer with nothing evicted.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_bfp8_amd as bfp8  # noqa: E402

LATENT, ROPE = 512, 64


class BoundedLayer:
    """Absorbed latent attention between two integer projections, with its cache and its masses. One decoded token a
    sequence and step."""

    def __init__(self, batch: int, hidden: int, heads: int, limit: int, page: int, device, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):  # the channels of a weight are its rows: quantized like tokens
            return bfp8.quant_act_int8(torch.randn(n, k, generator=g, device=device) * k ** -0.5)

        self.batch, self.heads, self.limit, self.page = batch, heads, limit, page
        self.scale = (128 + ROPE) ** -0.5
        self.w_in = weight((heads + 1) * (LATENT + ROPE), hidden)  # every head's query, then the token's latents and rotary key
        self.w_out = weight(hidden, heads * LATENT)
        width = -(-limit // page)
        self.cache = torch.zeros(batch * width, page, bfp8.LATENT_ROW, dtype=torch.uint8, device=device)
        self.scales = torch.full((batch * width, page), 127, dtype=torch.uint8, device=device)
        self.table = torch.randperm(batch * width, generator=g, device=device).view(batch, width).to(torch.int32)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.mass = torch.zeros(batch, width * page, device=device)
        self.rows = torch.arange(batch, device=device)

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """One token of every sequence, x [batch, hidden] bf16. Nothing here waits for the GPU."""
        y = bfp8.linear_int8(x, *self.w_in).view(self.batch, self.heads + 1, LATENT + ROPE)
        at = self.lens.long()
        slots = self.table[self.rows, at // self.page].long() * self.page + at % self.page
        bfp8.latent_cache_write(y[:, self.heads].contiguous(), slots, self.cache, self.scales)
        self.lens += 1
        out, _ = bfp8.latent_attention_mass(y[:, :self.heads], self.cache, self.scales, self.table, self.lens, self.scale,
                                            mass=self.mass, out_mass=self.mass)
        return bfp8.linear_int8(out.view(self.batch, -1), *self.w_out)

    def evict(self, budget: int, recent: int) -> torch.Tensor:
        """Cuts every longer sequence down to `budget` tokens within its pages; returns which stayed."""
        kept, lens, _ = bfp8.latent_cache_evict(self.cache, self.scales, self.table, self.lens, self.mass, budget,
                                                recent=recent, out_mass=self.mass)
        self.lens.copy_(lens)
        return kept


def run(device, steps=200, batch=4, hidden=1024, heads=8, budget=64, room=32, page=16, seed=0):
    """Decodes `steps` tokens with at most budget + room cached, and with all of them. Returns the two runs' outputs
    [steps, batch, hidden]."""
    bounded = BoundedLayer(batch, hidden, heads, budget + room, page, device, seed)
    whole = BoundedLayer(batch, hidden, heads, steps, page, device, seed)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    outs, length = ([], []), 0
    for _ in range(steps):
        x = torch.randn(batch, hidden, generator=g, device=device).to(torch.bfloat16)
        if length == budget + room:
            bounded.evict(budget, recent=budget // 4)
            length = budget
        outs[0].append(bounded.step(x))
        outs[1].append(whole.step(x))
        length += 1
    return torch.stack(outs[0]), torch.stack(outs[1])


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=200)
    parser.add_argument("--budget", type=int, default=64)
    args = parser.parse_args()
    a, b = run(torch.device("cuda"), steps=args.steps, budget=args.budget)
    last = slice(args.steps // 2, None)
    print(f"{args.steps} tokens, {args.budget} to {args.budget + 32} of them cached: outputs of the second half differ from those with "
          f"all cached by {float((a[last].float() - b[last].float()).norm() / b[last].float().norm()):.2f} of their norm")
