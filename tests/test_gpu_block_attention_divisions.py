"""Every division of kv8_attention's work (rows of a block, chunks of a context, joined or not,
with and without lse) against softmax attention in 64 bits, at the same tolerance as its other
tests: the division changes the order of fp32 sums, which that tolerance holds."""

import numpy as np
import pytest
import torch

from test_gpu_block_attention import Case, say

pytestmark = pytest.mark.gpu

# name: contexts, new tokens, query heads, cache heads ("64 rows": in blocks of eight waves)
DIVISIONS = {
    "one launch": ([900, 5, 64], [1, 1, 3], 4, 2),
    "16 rows, a block a pair": ([400, 1, 77, 256] * 10, [1] * 40, 16, 8),
    "16 rows, dealt": ([5001, 17, 3000], [2, 1, 5], 4, 2),
    "64 rows": ([130, 300, 64], [130, 17, 64], 8, 2),
    "64 rows, many pairs": ([200, 60, 131, 64] * 10, [60, 60, 17, 1] * 10, 32, 8),
    "64 rows in chunks": ([4001, 100, 2000], [20, 17, 33], 8, 2),
    "128 rows": ([2100, 65], [2100, 65], 32, 32),
    "128 rows in chunks": ([2113, 200, 1500, 2049], [130, 128, 1, 260], 8, 8),
}
ROWS = [0, 1, 15, 16, 31, 32, 63, 64, 65, 127, 128, 129, 255, 259, 1000, 2047, 2099]


def case(name, D, P, **kw):
    lens, news, Hq, Hkv = DIVISIONS[name]
    return Case(lens, news, Hq, Hkv, D, P, **kw)


@pytest.mark.parametrize("D,P", [(64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("name", DIVISIONS)
def test_divisions(name, D, P):
    say(name, D, P)
    c = case(name, D, P, seed=3)
    out, lse, _ = c.run()
    c.check(out, lse, rows=ROWS)
    plain, _, _ = c.run(lse=None)
    c.check(plain, lse, rows=ROWS)
    again, lse2, _ = c.run()
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("window", [1, 100, 1024])
@pytest.mark.parametrize("name", DIVISIONS)
def test_divisions_with_a_window(name, window):
    say(name, window)
    c = case(name, 64, 32, seed=window)
    out, lse, _ = c.run(window=window)
    c.check(out, lse, window=window, rows=ROWS)
    out, lse, _ = c.run(window=window, causal=False)
    c.check(out, lse, window=window, causal=False, rows=ROWS)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 3e38])
@pytest.mark.parametrize("name", DIVISIONS)
def test_masked_scales_never_count(name, bad):
    """Pages past the end, and codes past the end inside a page, change nothing."""
    say(name, bad)
    c = case(name, 64, 16, room=max(DIVISIONS[name][0]) + 100)
    clean, lse0, _ = c.run()
    for b, n in enumerate(c.lens):
        used = -(-n // c.P)
        c.ks[c.table[b, used:]] = bad
        c.vs[c.table[b, used:]] = bad
        if n % c.P:
            c.k[c.table[b, n // c.P], :, n % c.P:] = 127
            c.v[c.table[b, n // c.P], :, :, n % c.P:] = -127
    out, lse, _ = c.run()
    assert np.array_equal(out, clean) and np.array_equal(lse, lse0)


@pytest.mark.parametrize("name", DIVISIONS)
def test_division_by_other_lengths(name):
    """max_kv and max_new divide the work: bounds that are too high, and a max_kv that is too low."""
    say(name)
    c = case(name, 128, 16, seed=9)
    n, m = max(c.lens), max(c.news)
    for kw in (dict(max_kv=4 * n), dict(max_kv=1), dict(max_new=2 * m), dict(max_kv=n // 3)):
        out, lse, _ = c.run(**kw)
        c.check(out, lse, rows=ROWS)
