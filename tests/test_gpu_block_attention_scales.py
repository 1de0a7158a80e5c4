"""kv8_attention over value scales of any size, in every division of its work.

test_tiny_values has the tolerance of the kernel's other tests.  Where scales lie far apart, a weight
is rounded relative to the largest one that its row has met, so the tolerance is put together anew,
with A = sum w |v| / sum w of a row and column and ds the error of the scores as in the other tests:
a weight in fp16's normal range is off by at most 2^-11 of itself, in the product and in the sum that
divides it, 2^-10 A together; one below is off by half of fp16's smallest step, 2^-40 of the largest
weight times the largest scale in the product, and 2^-32 in the sum (the step is 2^8 times larger
there, for scales down to 2^-8 of the largest; the sum takes the others unrounded); the scores give
2 ds A, exponentials and logarithms 1e-5 A, and the stored result half its distance to the next bf16
number.  lse moves by ds."""

import numpy as np
import pytest
import torch

from block_ref import U, attention, bf16_gap
from test_gpu_block_attention import DEV, Case, say
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


def check_far(c):
    """Runs a case with and without lse, against 64 bits."""
    out, lse, _ = c.run()
    plain, _, _ = c.run(lse=None)
    q, scale = c.q.double().cpu().numpy(), c.D ** -0.5
    for b, n in enumerate(c.lens):
        s, m = c.start[b], c.news[b]
        pid = c.table[b, :-(-n // c.P)]
        for hq in range(c.Hq):
            h = hq // (c.Hq // c.Hkv)
            k = (c.k[pid, h] * c.ks[pid, h].astype(np.float64)[:, None, None]).reshape(-1, c.D)[:n]
            v = (c.v[pid, h] * c.vs[pid, h].astype(np.float64)[:, None, None]).transpose(0, 2, 1).reshape(-1, c.D)[:n]
            for i in (r for r in ROWS if r < m):
                x = q[s + i, hq]
                ref, ls, size = attention(x[None], k, v, n - m + i, scale, True, 0)
                ds = scale * (c.D * U * (np.abs(k) @ np.abs(x)).max() + 2.0 ** -22 * np.abs(k @ x).max())
                bound = (2.0 ** -10 + 2.0 ** -32 * n + 2 * ds + 1e-5) * size[0] + 2.0 ** -40 * n * np.abs(v).max()
                bound = 1.01 * (bound + bf16_gap(ref[0]))       # the result may round from the next power of two
                for got in (out, plain):
                    err = np.abs(got[s + i, hq] - ref[0])
                    assert (err <= bound).all(), (b, hq, i, (err / bound).max())
                assert abs(lse[s + i, hq] - ls[0]) <= ds + 1e-5 * (1 + abs(ls[0]))


@pytest.mark.parametrize("below", [9, 20, 38, 41, 90, 128, 135])      # the last two are at and below the smallest normal number
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("name", DIVISIONS)
def test_quiet_pages_beside_loud_ones(name, D, P, below):
    """Every second page's value scale is 2^-below of the others', the quiet ones first and second."""
    say(name, D, P, below)
    for quiet in (0, 1):
        c = case(name, D, P, seed=below)
        place = np.full(c.vs.shape[0], 1 - quiet)
        for row in c.table:
            place[row] = np.arange(len(row)) % 2
        c.vs = (c.vs * 70 * np.where(place == quiet, 2.0 ** -below, 1.0)[:, None] * 4).astype(np.float32)
        check_far(c)


@pytest.mark.parametrize("quiet_first", [False, True])
@pytest.mark.parametrize("new", [1, 20, 64, 300])
def test_one_loud_key_over_many_quiet_ones(new, quiet_first):
    """A key 9.7 above all others in the exponent, in a page whose value scale is 2^28 times theirs: the others have
    half of the weights' sum."""
    say("one loud key", new, quiet_first)
    c = Case([16000], [new], 4, 1, 128, 64)
    loud = c.table[0, 249 - 5 if quiet_first else 0]
    c.k[:], c.v = 0, np.abs(c.v)
    c.k[loud, :, 0], c.ks[:] = 64, 1 / 64
    c.vs[:], c.vs[loud] = 2.0 ** -34, 2.0 ** -6
    c.q.fill_(9.7 / 128 ** 0.5)
    check_far(c)


@pytest.mark.parametrize("name", DIVISIONS)
def test_a_poisoned_page_counts_however_small_its_weights(name):
    """Rows that see a page of NaN values are NaN, also where its weights vanish.  lse does not depend on values, but
    rounds the scores near the largest, and so near itself, in another place: a few 2^-23 of it."""
    say(name)
    c = case(name, 64, 16, seed=4, q_scale=30.0)
    _, lse0, _ = c.run()
    c.vs[c.table[:, 0]] = np.nan
    out, lse, _ = c.run()
    assert np.isnan(out).all()
    assert (np.abs(lse - lse0) <= 2.0 ** -20 * (1 + np.abs(lse0))).all()


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("name", DIVISIONS)
def test_large_scores(name, D, P):
    """Scores from 2^12 to 2^27: every key's is one of three, so the result is the mean of the values of the largest."""
    say(name, D, P)
    c = case(name, D, P, seed=6)
    g = np.random.default_rng(5)
    c.k[:] = g.integers(1, 4, size=c.k.shape[:3])[..., None]
    c.ks[:] = 1.0
    c.q = torch.from_numpy(2.0 ** g.integers(6, 19, size=c.q.shape[:2]))[..., None].expand(c.q.shape).to(torch.bfloat16).to(DEV)
    c.q = c.q.contiguous()
    out, lse, _ = c.run(scale=1.0)
    for b, n in enumerate(c.lens):
        s, m = c.start[b], c.news[b]
        pid = c.table[b, :-(-n // P)]
        for hq in range(c.Hq):
            h = hq // (c.Hq // c.Hkv)
            k = c.k[pid, h].reshape(-1, D)[:n].astype(np.float64)
            v = (c.v[pid, h] * c.vs[pid, h].astype(np.float64)[:, None, None]).transpose(0, 2, 1).reshape(-1, D)[:n]
            for i in (r for r in ROWS if r < m):
                q = c.q[s + i:s + i + 1, hq].double().cpu().numpy()
                ref, ls, size = attention(q, k, v, n - m + i, 1.0, True, 0)
                # scores are exact but for the scale's rounding, the same for all keys
                bound = (2.0 ** -10 + 2.0 ** -32 * n + 1e-5) * size[0] + 2.0 ** -40 * n * np.abs(v).max()
                bound = 1.01 * (bound + bf16_gap(ref[0]))
                err = np.abs(out[s + i, hq] - ref[0])
                assert (err <= bound).all(), (b, hq, i, (err / bound).max())
                # the scale times log2(e), the score and lse are rounded to fp32
                assert abs(lse[s + i, hq] - ls[0]) <= 2.0 ** -21 * abs(ls[0]) + 1e-4
