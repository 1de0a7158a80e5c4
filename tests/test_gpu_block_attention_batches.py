"""kv8_attention over ragged batches, against softmax attention in 64 bits at the tolerance of its
other tests."""

import pytest
import torch

from bit_codebook_quantized_amd import block
from test_gpu_block_attention import DEV, Case, say

pytestmark = pytest.mark.gpu


def test_one_long_prompt_among_single_tokens():
    """64 sequences of up to 8192 new tokens: 2^24 query rows if all were as long, 2^18 as they are."""
    say("one long prompt")
    c = Case([8192] + [1 + 129 * i for i in range(63)], [8192] + [1] * 63, 32, 2, 64, 64)
    out, lse, _ = c.run()
    c.check(out, lse, rows=[0, 63, 64, 1000, 4097, 8191])


def test_no_sequences_and_no_tokens():
    say("no sequences")
    cache, rope = block.KVCache8.empty(2, 1, 64, 16), block.Rope(torch.ones(32, device=DEV))
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    for n in (0, 2):
        out = block.kv8_append(cache, i32(n, 3), i32(n), i32(n + 1), 0, x, x, q=x, pos=i32(1, 0), rope=rope)
        assert out.shape == x.shape
        assert block.kv8_attention(x, cache, i32(n, 3), i32(n), i32(n + 1), 0, 0).shape == x.shape
    assert not cache.k.any() and not cache.k_scale.any()
