"""The decoder-layer example: its parts composed as a user composes them."""

import os
import sys

import numpy as np
import pytest
import torch

import block_ref as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_layer as E  # noqa: E402
from bit_codebook_quantized_amd import block, w4a8  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[case]", *a, flush=True)


def stack(table, layers=2):
    return [E.DecoderLayer(512, 8, 2, 64, 768, table.numel(), 64, 100 * i) for i in range(layers)], torch.ones(512, device=DEV)


def test_later_tokens_do_not_reach_earlier_ones():
    """Rows of whole pages have the same bits whether or not more tokens follow."""
    say("causal")
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    x = torch.randn(256, 512, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    layers, norm = stack(table)
    y = E.run(layers, norm, x, E.Batch.of(table, [0, 0], [128, 128]))
    layers, norm = stack(table)
    first = torch.cat([x[:64], x[128:192]])
    z = E.run(layers, norm, first, E.Batch.of(table, [0, 0], [64, 64]))
    assert torch.equal(z[:64], y[:64]) and torch.equal(z[64:], y[128:192])


def test_single_tokens_follow_the_prompt():
    """Tokens fed one at a time reach what the whole prompt gives, to the 8-bit cache's steps: keys
    and values are requantised when a page's scale grows, at most half a step (1/254 of the page's
    maximum) each time, about log(64) times a page, so outputs agree to a few percent."""
    say("prompt against tokens")
    table = torch.arange(2, dtype=torch.int32, device=DEV).view(1, 2)
    x = torch.randn(70, 512, generator=torch.Generator(DEV).manual_seed(2), device=DEV).to(torch.bfloat16)
    layers, norm = stack(table)
    y = E.run(layers, norm, x, E.Batch.of(table, [0], [70]))
    layers, norm = stack(table)
    z = torch.cat([E.run(layers, norm, x[t:t + 1].contiguous(), E.Batch.of(table, [t], [1])) for t in range(70)])
    y, z = y.float(), z.float()
    assert ((z - y).norm(dim=1) / y.norm(dim=1)).max() < 0.1
    assert (z - y).norm() / y.norm() < 0.04


def test_norm_linear_gradient():
    """The composed backward is that of sum(g * linear(norm(x + stream))) with the straight-through weight."""
    say("norm + linear gradient")
    g = torch.Generator(DEV).manual_seed(3)
    stream = torch.randn(20, 512, generator=g, device=DEV)
    x = torch.randn(20, 512, generator=g, device=DEV).to(torch.bfloat16)
    weight = 1 + 0.1 * torch.randn(512, generator=g, device=DEV)
    layer = E.DecoderLayer(512, 8, 2, 64, 768, 1, 64, 5).qkv
    y, h, rstd = E.norm_linear(x, stream, weight, layer)
    gy = torch.randn(y.shape, generator=g, device=DEV).to(torch.bfloat16)
    gh = torch.randn(h.shape, generator=g, device=DEV)
    dx, dw = E.norm_linear_grad(gy, gh, h, rstd, weight, layer)
    f = lambda t: t.double().cpu().numpy()
    grid = f(w4a8.decode_w4_to_int8(layer)) * f(layer.s_channel)[:, None]
    ref, dw_ref, gv = R.norm_grad(f(gy) @ grid, f(h), f(weight), 1e-6, True)
    # the gradient of the rotated rows is rounded to bf16, and so is the weight: 2^-8 each, of the
    # row's 2-norm through an orthogonal map and a projection
    assert np.linalg.norm(f(dx) - f(gh) - ref) <= 2 * 2.0 ** -8 * np.linalg.norm(ref)
    assert np.linalg.norm(f(dw) - dw_ref) <= 2 * 2.0 ** -8 * np.linalg.norm(gv * f(h) * f(rstd)[:, None])


def test_example_runs(capsys):
    say("example")
    argv, sys.argv = sys.argv, ["decoder_layer.py", "--layers", "1", "--tokens", "3"]
    try:
        E.main()
    finally:
        sys.argv = argv
    out = capsys.readouterr().out
    assert "cached [103, 40, 4]" in out and "dweight (1024,)" in out
