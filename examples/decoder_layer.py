"""A decoder layer whose linears are W4A8 and whose cache is 8-bit, run as a server runs it
(ragged prompts, then single tokens) and, for its norms, as fine-tuning runs it.

    python examples/decoder_layer.py [--layers 2] [--tokens 8]

Random weights and inputs; there is no vocabulary: the hidden state of a sequence's last
token is fed back as its next input.
"""

from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_codebook_quantized_amd import block, synth, w4a8  # noqa: E402


@dataclass
class Batch:
    """What one step of B sequences needs beside the tokens themselves."""
    table: torch.Tensor      # int32 [B, pages of a sequence]
    ctx_len: torch.Tensor    # int32 [B], tokens cached before the step
    kv_len: torch.Tensor     # int32 [B], and after it
    start: torch.Tensor      # int32 [B + 1], first row of each sequence
    pos: torch.Tensor        # int32 [1, T]
    max_new: int
    max_kv: int

    @classmethod
    def of(cls, table: torch.Tensor, ctx, news):
        """From the host's lists of cached and of new tokens."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=table.device)
        start = [0]
        for n in news:
            start.append(start[-1] + n)
        kv = [c + n for c, n in zip(ctx, news)]
        pos = [p for c, e in zip(ctx, kv) for p in range(c, e)]
        return cls(table, i32(ctx), i32(kv), i32(start), i32([pos]), max(news), max(kv))


def rows_linear(xq, xs, layer, out_dtype=torch.bfloat16):
    """The linear on rows that are int8 already."""
    fn = w4a8.w4a8_gemv if xq.shape[0] <= w4a8.GEMV_MAX_M else w4a8.w4a8_gemm
    return fn(xq, xs, layer, out_dtype)


class DecoderLayer:
    """Norm, attention, norm, gated MLP; every product with a weight is a W4A8 linear."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, mlp: int, pages: int, page_tokens: int,
                 seed: int, device="cuda"):
        n = lambda rows, cols, i: w4a8.quantize_w4(
            synth.gaussian_weight_device(rows, cols, seed + i, device, std=cols ** -0.5))
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.qkv = n((q_heads + 2 * kv_heads) * head_dim, hidden, 0)
        self.out = n(hidden, q_heads * head_dim, 1)
        self.gate_up = n(2 * mlp, hidden, 2)        # gate and up rows interleaved
        self.down = n(hidden, mlp, 3)
        self.norm1 = torch.ones(hidden, device=device)
        self.norm2 = torch.ones(hidden, device=device)
        self.rope = block.Rope((10000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64) / (head_dim // 2)))
                               .float().to(device))
        self.cache = block.KVCache8.empty(pages, kv_heads, head_dim, page_tokens, device)

    def __call__(self, x, stream, b: Batch):
        """x [T, hidden]: the previous layer's output, not yet added to the stream.  Returns this
        layer's output (again not yet added) and the stream, which is updated in place."""
        xq, xs, stream = block.rmsnorm_quant_act(x, self.norm1, stream, h=stream)
        qkv = rows_linear(xq, xs, self.qkv).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        q = block.kv8_append(self.cache, b.table, b.ctx_len, b.start, b.max_new, k, v, q=q, pos=b.pos, rope=self.rope)
        o = block.kv8_attention(q, self.cache, b.table, b.kv_len, b.start, b.max_new, b.max_kv)
        x = w4a8.linear(o.view(x.shape[0], -1), self.out)
        xq, xs, stream = block.rmsnorm_quant_act(x, self.norm2, stream, h=stream)
        return w4a8.linear(rows_linear(xq, xs, self.gate_up, w4a8.SWIGLU), self.down), stream


def run(layers, norm, x, b: Batch):
    """All layers and the final norm: bf16 [T, hidden]."""
    stream = torch.zeros_like(x)
    for layer in layers:
        x, stream = layer(x, stream, b)
    return block.rmsnorm(x, norm, stream)[0]


def norm_linear(x, stream, weight, layer):
    """The training form of norm + linear: the output, the new stream, and what the backward needs."""
    rstd = torch.empty(x.shape[0], device=x.device)
    xq, xs, h = block.rmsnorm_quant_act(x, weight, stream, rstd=rstd)
    return rows_linear(xq, xs, layer), h, rstd


def norm_linear_grad(grad_y, grad_h, h, rstd, weight, layer):
    """Its backward, straight through the quantisers: the gradient of x and of the stream, and of the norm's weight."""
    return block.rmsnorm_grad(w4a8.grad_input(grad_y, layer), h, rstd, weight, grad_h)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=8)
    args = ap.parse_args()
    hidden, page, prompts = 1024, 64, [100, 37, 1]
    per = (max(prompts) + args.tokens + page - 1) // page
    table = torch.randperm(len(prompts) * per, device="cuda").to(torch.int32).view(len(prompts), per)
    layers = [DecoderLayer(hidden, 8, 2, 128, 2048, table.numel(), page, 100 * i) for i in range(args.layers)]
    norm = torch.ones(hidden, device="cuda")

    x = torch.randn(sum(prompts), hidden, device="cuda").to(torch.bfloat16)
    b = Batch.of(table, [0] * len(prompts), prompts)
    y = run(layers, norm, x, b)
    print(f"prompts of {prompts} tokens: out {tuple(y.shape)}, rms {y.float().square().mean().sqrt():.3f}")
    cached, last = list(prompts), y[b.start[1:].long() - 1]
    for t in range(args.tokens):
        y = run(layers, norm, last, Batch.of(table, cached, [1] * len(prompts)))
        cached, last = [n + 1 for n in cached], y
    print(f"{args.tokens} single tokens: out {tuple(y.shape)}, rms {y.float().square().mean().sqrt():.3f}, cached {cached}")

    stream = torch.randn(64, hidden, device="cuda")
    x = torch.randn(64, hidden, device="cuda").to(torch.bfloat16)
    y, h, rstd = norm_linear(x, stream, norm, layers[0].qkv)
    dx, dweight = norm_linear_grad(torch.randn_like(y), torch.zeros_like(h), h, rstd, norm, layers[0].qkv)
    print(f"norm + linear backward: dx {tuple(dx.shape)} {dx.dtype}, dweight {tuple(dweight.shape)}")


if __name__ == "__main__":
    main()
