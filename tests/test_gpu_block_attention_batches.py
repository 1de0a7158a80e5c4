"""kv8_attention over ragged batches, against softmax attention in 64 bits at the tolerance of its
other tests."""

import pytest

from test_gpu_block_attention import Case, say

pytestmark = pytest.mark.gpu


def test_one_long_prompt_among_single_tokens():
    """64 sequences of up to 8192 new tokens: 2^24 query rows if all were as long, 2^18 as they are."""
    say("one long prompt")
    c = Case([8192] + [1 + 129 * i for i in range(63)], [8192] + [1] * 63, 32, 2, 64, 64)
    out, lse, _ = c.run()
    c.check(out, lse, rows=[0, 63, 64, 1000, 4097, 8191])
