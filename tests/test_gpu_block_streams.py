"""The decoder-layer operators on a stream that is not the default one, behind work of that stream:
what they read is ready only then, and what they leave in workspaces is read on the same stream."""

import numpy as np
import pytest
import torch

from bit_codebook_quantized_amd import block
from test_gpu_block_attention_divisions import DIVISIONS, case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[case]", *a, flush=True)


def behind_other_work(run, *tensors):
    """run(*tensors) here, and on a second stream on copies that are made there after some milliseconds of products."""
    want = run(*tensors)
    side = torch.cuda.Stream()
    late = [torch.zeros_like(t) for t in tensors]
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-4
        for a, b in zip(late, tensors):
            a.copy_(b)
        got = run(*late)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b) and a.abs().sum() > 0


def test_norm_backward():
    say("norm backward")
    g, h = torch.randn(700, 1024, device=DEV).to(torch.bfloat16), torch.randn(700, 1024, device=DEV)
    rstd, w = torch.rand(700, device=DEV) + 0.5, torch.randn(1024, device=DEV)
    behind_other_work(lambda g, h, r, w: block.rmsnorm_grad(g, h, r, w, h), g, h, rstd, w)


def test_rotation():
    say("rotation")
    x = torch.randn(900, 6, 128, device=DEV).to(torch.bfloat16)
    pos = torch.arange(1800, device=DEV).to(torch.int32).view(2, 900)
    freq = torch.rand(64, device=DEV)
    behind_other_work(lambda x, p, f: [block.rope_axes(x, p, block.Rope(f, [40, 24]))], x, pos, freq)


def test_append():
    say("append")
    x = torch.randn(150, 10, 64, device=DEV).to(torch.bfloat16)
    pos = torch.arange(150, device=DEV).to(torch.int32).view(1, 150)
    table = torch.randperm(20, device=DEV).to(torch.int32).view(2, 10)
    start, ctx = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([0, 100, 150], [7, 16]))

    def run(x, pos, table, start, ctx):
        cache = block.KVCache8.empty(20, 2, 64, 16)
        q = block.kv8_append(cache, table, ctx, start, 100, x[:, 6:8], x[:, 8:], q=x[:, :6], pos=pos,
                             rope=block.Rope(0.5 ** torch.arange(32, device=DEV)))
        return q, cache.k.float(), cache.v.float(), cache.k_scale, cache.v_scale
    behind_other_work(run, x, pos, table, start, ctx)


@pytest.mark.parametrize("name", DIVISIONS)
def test_attention(name):
    say("attention", name)
    c = case(name, 64, 16, seed=2)
    cache, t = c.cache(), lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)

    def run(q, k, v, ks, vs, table, kv, start):
        lse = torch.empty(q.shape[:2], device=DEV)
        return block.kv8_attention(q, block.KVCache8(k, v, ks, vs), table, kv, start, max(c.news), max(c.lens), lse=lse), lse
    behind_other_work(run, c.q, cache.k, cache.v, cache.k_scale, cache.v_scale, t(c.table), t(c.lens), t(c.start))
