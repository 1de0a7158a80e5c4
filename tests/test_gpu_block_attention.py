"""kv8_attention against softmax attention in 64 bits over the values that the cache stands
for.

Tolerance: with A = sum w |v| / sum w of a row and column, the weights (fp16, 11 bits) and
the stored result (bf16, 8 bits) together stay within 2^-8 A, an error ds of the scores
moves the result by 2 ds A; ds <= D 2^-24 max_j sum |q k_j| scale for the fp32 sums, plus
2^-22 of the largest score for the exponent's argument.  A weight below fp16's normal range
is rounded to a multiple of 2^-39 of the largest: 2^-40 n max |v|.  lse moves by ds."""

import numpy as np
import pytest
import torch

import block_ref as R
from bit_codebook_quantized_amd import block, synth, w4a8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[case]", *a, flush=True)


class Case:
    def __init__(self, lens, news, Hq, Hkv, D, P, seed=0, spare=2, room=None, q_scale=1.0, table=None):
        g = synth.rng(seed + 17 * D + P)
        self.lens, self.news, self.Hq, self.Hkv, self.D, self.P = lens, news, Hq, Hkv, D, P
        B = len(lens)
        per = max(1, -(-max(lens + [room or 0]) // P))
        pages = B * per + spare
        self.table = g.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
        self.k = g.integers(-127, 128, size=(pages, Hkv, P, D)).astype(np.int8)
        self.v = g.integers(-127, 128, size=(pages, Hkv, D, P)).astype(np.int8)
        self.ks = ((0.5 + g.random((pages, Hkv))) / 70).astype(np.float32)
        self.vs = ((0.1 + g.random((pages, Hkv))) / 70).astype(np.float32)
        T = sum(news)
        q = torch.from_numpy((g.standard_normal((T, Hq, D)) * q_scale).astype(np.float32)).to(torch.bfloat16)
        self.q = q.to(DEV)
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)

    def cache(self):
        t = lambda a: torch.from_numpy(a).to(DEV)
        return block.KVCache8(t(self.k), t(self.v), t(self.ks), t(self.vs))

    def run(self, **kw):
        T = sum(self.news)
        lse = torch.full((T, self.Hq), 7.0, device=DEV)
        kv = dict(max_new=max(self.news), max_kv=max(self.lens), lse=lse) | kw
        out = block.kv8_attention(kv.pop("q", self.q), self.cache(), torch.from_numpy(self.table).to(DEV),
                                  torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                                  torch.from_numpy(self.start).to(DEV), **kv)
        return out.double().cpu().numpy(), lse.double().cpu().numpy(), out

    def check(self, out, lse, scale=None, causal=True, window=0, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q.double().cpu().numpy()
        worst = 0.0
        for b, n in enumerate(self.lens):
            s, m = self.start[b], self.news[b]
            pid = self.table[b, :-(-n // self.P)]
            for h in range(self.Hkv):
                k = (self.k[pid, h] * self.ks[pid, h].astype(np.float64)[:, None, None]).reshape(-1, self.D)[:n]
                v = (self.v[pid, h] * self.vs[pid, h].astype(np.float64)[:, None, None]).transpose(0, 2, 1)
                v = v.reshape(-1, self.D)[:n]
                for j in range(self.Hq // self.Hkv):
                    hq = h * (self.Hq // self.Hkv) + j
                    pick = range(m) if rows is None else [r for r in rows if r < m]
                    for i in pick:
                        ref, ls, size = R.attention(q[s + i:s + i + 1, hq], k, v, n - m + i, scale, causal, window)
                        if np.isinf(ls[0]):
                            assert not out[s + i, hq].any() and lse[s + i, hq] == -np.inf
                            continue
                        ds = 0.0
                        if n:
                            ds = self.D * R.U * scale * (np.abs(k) @ np.abs(q[s + i, hq])).max() \
                                + 2.0 ** -22 * scale * np.abs(k @ q[s + i, hq]).max()
                        bound = (2.0 ** -8 + 2 * ds + 1e-5) * size[0] + 2.0 ** -40 * n * np.abs(v).max()
                        err = np.abs(out[s + i, hq] - ref[0])
                        worst = max(worst, (err / bound).max())
                        assert (err <= bound).all(), (b, h, j, i, (err / bound).max())
                        assert abs(lse[s + i, hq] - ls[0]) <= ds + 1e-5 * (1 + abs(ls[0]))
        print("   worst error over its bound: %.3f" % worst, flush=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_single_tokens(P, D):
    say("single tokens", P, D)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 255, 257, 700, 1030]
    c = Case(lens, [1] * len(lens), 8, 2, D, P)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (16, 2), (20, 1), (48, 2), (7, 7)])
def test_head_groups(Hq, Hkv):
    say("heads", Hq, Hkv)
    c = Case([300, 77, 1], [1, 3, 1], Hq, Hkv, 64, 32, seed=Hq)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("D,P,Hq,Hkv", [(128, 64, 8, 2), (64, 16, 6, 2), (64, 128, 4, 4)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (False, 33), (True, 200)])
def test_prompts(D, P, Hq, Hkv, causal, window):
    say("prompts", D, P, Hq, Hkv, causal, window)
    c = Case([300, 129, 64, 515], [300, 40, 64, 3], Hq, Hkv, D, P, seed=window)
    out, lse, _ = c.run(causal=causal, window=window)
    c.check(out, lse, causal=causal, window=window, rows=[0, 1, 2, 15, 16, 17, 31, 39, 63, 64, 65, 127, 128, 200, 256, 298, 299])


def test_long_context_is_split():
    """Few rows over a long context: the context is divided; all divisions agree with 64 bits."""
    say("split")
    c = Case([9001, 5000, 4097], [1, 2, 1], 4, 1, 128, 64)
    assert block.kv8_attention_workspace(3, 4, 2, 9001, 4, 1, 128) > 0
    out, lse, _ = c.run()
    c.check(out, lse)
    # max_kv divides the work and nothing else: too small, and far too large
    for max_kv in (9001 // 3, 0, 100000):
        out, lse, _ = c.run(max_kv=max_kv)
        c.check(out, lse)
    out, lse, _ = c.run(window=700)
    c.check(out, lse, window=700)


def test_chunk_of_a_long_prompt():
    say("chunk")
    c = Case([4000], [260], 8, 2, 128, 64, seed=5)
    out, lse, _ = c.run()
    c.check(out, lse, rows=[0, 1, 63, 64, 100, 127, 128, 255, 256, 259])


def test_rows_that_see_nothing():
    """Lengths of zero, no new tokens, and more new tokens than the cache holds."""
    say("empty rows")
    c = Case([0, 5, 20, 3], [2, 0, 1, 6], 4, 2, 64, 16, room=64)
    out, lse, _ = c.run(max_kv=20)
    c.check(out, lse)
    assert not out[:2].any() and not out[3:6].any()       # the last sequence's first three rows stand before its cache
    out, lse, _ = c.run(max_kv=20, causal=False)
    c.check(out, lse, causal=False)


def test_scores_far_apart():
    """A peaked softmax, scores beyond the range of exp in fp32, and a given scale."""
    say("peaked")
    c = Case([500, 130], [2, 5], 4, 2, 128, 32, q_scale=30.0)
    out, lse, _ = c.run(scale=0.3)
    c.check(out, lse, scale=0.3)
    c = Case([500, 130], [2, 5], 4, 2, 128, 32, q_scale=1e-3)
    out, lse, _ = c.run()
    c.check(out, lse)


def test_masked_places_never_count():
    """NaN scales of pages past the end, before the window and after a row's position; missing pages."""
    say("masked NaN")
    c = Case([100, 40], [36, 1], 4, 2, 64, 16, room=160)
    clean, lse0, _ = c.run(max_kv=100)
    c.check(clean, lse0)
    c.ks[c.table[0, 7:]] = np.nan            # tokens past 112: past the end
    c.vs[c.table[0, 7:]] = np.nan
    c.ks[c.table[1, 3:]] = np.nan
    out, lse, _ = c.run(max_kv=100)
    assert np.array_equal(out, clean) and np.array_equal(lse, lse0)
    c.vs[c.table[0, 6]] = np.nan             # tokens 96 .. 99: seen by the rows at positions 96 and later only
    out, lse, _ = c.run(max_kv=100)
    assert np.array_equal(out[:32], clean[:32]) and np.isnan(out[32:36]).all() and np.array_equal(out[36:], clean[36:])
    c.vs[c.table[0, 6]] = 0.01
    c.ks[c.table[0, 6]] = np.nan
    out, lse, _ = c.run(max_kv=100)
    assert np.array_equal(out[:32], clean[:32]) and np.isnan(out[32:36]).all() and np.isnan(lse[32:36]).all()
    # a window that has left the first pages behind
    c = Case([100], [3], 4, 2, 64, 16)
    clean, lse0, _ = c.run(window=30)
    c.vs[c.table[0, :4]] = np.nan
    c.ks[c.table[0, :4]] = np.nan
    out, lse, _ = c.run(window=30)
    assert np.array_equal(out, clean) and np.array_equal(lse, lse0)
    # page numbers outside the cache hide their tokens: the same as a window from page 2 on for a single row
    c = Case([90], [1], 4, 2, 64, 16)
    clean, lse0, _ = c.run(window=90 - 32)
    c.table[0, 0], c.table[0, 1] = -3, c.k.shape[0]
    out, lse, _ = c.run()
    assert np.array_equal(out, clean) and np.array_equal(lse, lse0)


def test_zero_scales():
    say("zero scales")
    c = Case([200], [2], 2, 1, 64, 16)
    c.ks[:], c.vs[c.table[0, 3]] = 0.0, 0.0
    out, lse, _ = c.run()
    c.check(out, lse)


def test_strides_and_buffers():
    """Queries and outputs inside wider tensors; rows of no sequence are left alone."""
    say("strides")
    c = Case([70, 33], [4, 2], 4, 2, 64, 16)
    clean, lse0, o = c.run()
    wide = torch.randn(9, 10, 64, device=DEV).to(torch.bfloat16)
    wide[:6, 3:7] = c.q
    buf = torch.full((9, 9, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((9, 4), 5.0, device=DEV)
    ws = torch.empty(block.kv8_attention_workspace(2, 9, 4, 70, 4, 2, 64) + 64, dtype=torch.uint8, device=DEV)
    out, _, ret = c.run(q=wide[:, 3:7], out=buf[:, 2:6], lse=lse, workspace=ws)
    assert torch.equal(buf[:6, 2:6], o)
    buf[:6, 2:6] = 5.0
    assert (buf == 5.0).all() and (lse[6:] == 5.0).all()


def test_same_bits_every_time_and_graph():
    """Joins run in a fixed order: repeated calls, and replays of a captured call, give the same bits."""
    say("repeat")
    c = Case([3000, 1500], [1, 1], 8, 2, 128, 64)
    _, _, first = c.run(lse=None)
    cache, table = c.cache(), torch.from_numpy(c.table).to(DEV)
    kv, start = torch.tensor(c.lens, dtype=torch.int32, device=DEV), torch.from_numpy(c.start).to(DEV)
    out = torch.empty_like(c.q)
    ws = torch.empty(block.kv8_attention_workspace(2, 2, 1, 4000, 8, 2, 128), dtype=torch.uint8, device=DEV)
    q = c.q.clone()
    step = lambda: block.kv8_attention(q, cache, table, kv, start, 1, 4000, out=out, workspace=ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in (3000, 17, 2000):        # the lengths are device data: a replay follows them
        kv[0] = n
        eager = step().clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    kv[0] = 3000
    for _ in range(3):
        assert torch.equal(block.kv8_attention(q, cache, table, kv, start, 1, 3000), first)


def test_refusals():
    say("refusals")
    c = Case([20, 20], [1, 1], 4, 2, 64, 16)
    cache, table = c.cache(), torch.from_numpy(c.table).to(DEV)
    kv, start = torch.tensor(c.lens, dtype=torch.int32, device=DEV), torch.from_numpy(c.start).to(DEV)
    ok = dict(q=c.q, cache=cache, table=table, kv_len=kv, q_start=start, max_new=1, max_kv=20)
    block.kv8_attention(**ok)
    for bad in (dict(q=c.q.float()), dict(q=c.q[:, :3]), dict(q=c.q[..., :32]), dict(kv_len=kv.long()), dict(table=table[:1]),
                dict(q_start=kv), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(max_kv=-1),
                dict(max_new=-1), dict(out=c.q[:1]), dict(lse=torch.empty(2, 3, device=DEV)), dict(q=c.q.cpu())):
        with pytest.raises(ValueError):
            block.kv8_attention(**(ok | bad))
    with pytest.raises(ValueError):
        block.kv8_attention(**(ok | dict(max_kv=100000, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))))
