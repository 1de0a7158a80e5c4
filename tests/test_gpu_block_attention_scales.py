"""kv8_attention over value scales of any size, in every division of its work, at the tolerance of
its other tests."""

import numpy as np
import pytest

from test_gpu_block_attention import say
from test_gpu_block_attention_divisions import DIVISIONS, case

pytestmark = pytest.mark.gpu

ROWS = [0, 15, 17, 63, 64, 129, 1000, 2099]


def finish(c, **kw):
    out, lse, _ = c.run(**kw)
    c.check(out, lse, rows=ROWS, **kw)
    plain, _, _ = c.run(lse=None, **kw)
    c.check(plain, lse, rows=ROWS, **kw)
    return out, lse


@pytest.mark.parametrize("below", [121, 126])      # scales just above, and mostly below, the smallest normal number
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("name", DIVISIONS)
def test_tiny_values(name, D, P, below):
    """All value scales are near the smallest normal number, and the values themselves above bf16's (codes of 16 and
    more), so that the result's rounding is the relative one of the tolerance."""
    say(name, D, P, below)
    c = case(name, D, P, seed=8)
    c.v = np.where(c.v < 0, np.minimum(c.v, -16), np.maximum(c.v, 16)).astype(np.int8)
    c.vs = (c.vs * 70 * 2.0 ** -below).astype(np.float32)
    finish(c)
