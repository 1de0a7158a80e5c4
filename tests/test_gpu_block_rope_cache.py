"""rope_axes and kv8_append against the formulas in 64 bits.

Rotation tolerance: the angle is exact to 2^-25 of a revolution (under 2e-7 rad), cosine and
sine to a few 2^-24, and three roundings follow: 1e-6 of |a| + |b|, then half a bf16 ulp
where the result is stored as bf16.  Values, and keys without a rotation, are stored exactly
as the formula says: the scale is the fp32 quotient, codes the rounded fp32 quotients."""

import numpy as np
import pytest
import torch

import block_ref as R
from bit_codebook_quantized_amd import block, synth, w4a8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[case]", *a, flush=True)


def f64(t):
    return t.double().cpu().numpy()


def freq(n, theta=10000.0):
    return (theta ** (-np.arange(n) / n)).astype(np.float32)


def rope_bound(x, n, interleaved):
    """1e-6 (|a| + |b|) of each element's pair, 0 past the rotated part."""
    b = np.zeros_like(x)
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
        b[..., i] = b[..., j] = 1e-6 * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return b


@pytest.mark.parametrize("T,heads,D,rot,sections,interleaved,top", [
    (1, 1, 64, 64, [32], False, 10), (1, 40, 128, 128, [16, 24, 24], False, 100000), (5, 3, 64, 32, [16], False, 5000),
    (37, 5, 128, 128, [64], True, 3000), (130, 6, 96, 96, [8, 20, 20], True, 900), (33, 2, 256, 256, [128], False, 40000),
    (64, 7, 80, 48, [10, 0, 7, 7], False, 2 ** 28), (1000, 12, 128, 128, [32, 32], False, 2000),
    (3, 2, 16, 16, [8], True, 7)])
def test_rope_matches_the_formula(T, heads, D, rot, sections, interleaved, top):
    say("rope", T, heads, D, rot, sections, interleaved, top)
    g = synth.rng(T * D + heads)
    n = rot // 2
    wide = torch.from_numpy(g.standard_normal((T, heads + 3, D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    x = wide[:, 1:heads + 1]                       # a slice of a wider projection
    pos = g.integers(0, top, size=(len(sections), T)).astype(np.int32)
    inv = freq(n)
    rope = block.Rope(torch.from_numpy(inv).to(DEV), sections, interleaved)
    pd = torch.from_numpy(pos).to(DEV)
    y = block.rope_axes(x, pd, rope)
    xn = f64(x)
    ref = R.rope(xn, pos, inv, sections, interleaved)
    err = np.abs(f64(y) - ref)
    assert (err <= rope_bound(xn, n, interleaved) + R.bf16_gap(ref) * 1.0001).all(), err.max()
    assert np.array_equal(f64(y)[..., rot:], xn[..., rot:])
    back = R.rope(xn, pos, inv, sections, interleaved, inverse=True)
    z = block.rope_axes(x, pd, rope, inverse=True)
    assert (np.abs(f64(z) - back) <= rope_bound(xn, n, interleaved) + R.bf16_gap(back) * 1.0001).all()
    before = wide.clone()
    assert block.rope_axes(x, pd, rope, out=x) is x           # in place, the other heads untouched
    assert torch.equal(x, y) and torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, heads + 1:], before[:, heads + 1:])


def test_rope_backward_is_the_transpose():
    """<g, rope(x + t d)> by differences equals <rope_inverse(g), d>."""
    say("rope differences")
    g = synth.rng(3)
    T, heads, D, sections = 9, 4, 64, [12, 20]
    inv, pos = freq(32), g.integers(0, 500, size=(2, T)).astype(np.int32)
    rope = block.Rope(torch.from_numpy(inv).to(DEV), sections)
    grad = torch.from_numpy(g.standard_normal((T, heads, D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dx = f64(block.rope_axes(grad, torch.from_numpy(pos).to(DEV), rope, inverse=True))
    gn, x, d = f64(grad), g.standard_normal((T, heads, D)), g.standard_normal((T, heads, D))
    t = 1e-4
    slope = ((gn * R.rope(x + t * d, pos, inv, sections)).sum() - (gn * R.rope(x - t * d, pos, inv, sections)).sum()) / (2 * t)
    assert abs(slope - (dx * d).sum()) <= 2.0 ** -8 * np.abs(dx * d).sum()      # dx is rounded to bf16


class Cache:
    """A cache on the GPU and its mirror on the host."""

    def __init__(self, batch, per, heads, D, P, seed, spare=3):
        self.g = synth.rng(seed)
        self.P, self.D, self.heads, self.batch = P, D, heads, batch
        pages = batch * per + spare
        self.table = self.g.permutation(pages)[:batch * per].reshape(batch, per).astype(np.int32)
        self.dev = block.KVCache8.empty(pages, heads, D, P)
        # stale contents everywhere: nothing may depend on what an unused page holds
        for t in (self.dev.k, self.dev.v):
            t.copy_(torch.from_numpy(self.g.integers(-127, 128, size=tuple(t.shape)).astype(np.int8)))
        for t in (self.dev.k_scale, self.dev.v_scale):
            t.fill_(float("nan"))
        self.dtable = torch.from_numpy(self.table).to(DEV)
        self.ctx = np.zeros(batch, np.int32)

    def snapshot(self):
        d = self.dev
        return [t.cpu().numpy().copy() for t in (d.k, d.v.transpose(2, 3), d.k_scale, d.v_scale)]

    def append(self, news, rope=None, q_heads=0, pos=None, wide=True, scale=1.0):
        T = int(sum(news))
        start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        n = q_heads + 2 * self.heads
        x = torch.from_numpy((self.g.standard_normal((T, n, self.D)) * scale).astype(np.float32)).to(torch.bfloat16).to(DEV)
        q, k, v = x[:, :q_heads], x[:, q_heads:q_heads + self.heads], x[:, q_heads + self.heads:]
        if not wide:
            k, v = k.contiguous(), v.contiguous()
        before = self.snapshot()
        out = block.kv8_append(self.dev, self.dtable, torch.from_numpy(self.ctx).to(DEV), torch.from_numpy(start).to(DEV),
                               int(max(news)), k, v, q=q if q_heads else None, pos=pos, rope=rope)
        return x, (q, k, v), before, self.snapshot(), out, start

    def expect(self, before, kx, vx, start, exact_keys=True, bound=None):
        """Checks the cache against the formula given the new keys and values (64-bit); returns nothing."""
        after = self.snapshot()
        touched = np.zeros(before[0].shape[0], bool)
        for b in range(self.batch):
            n, ctx = int(start[b + 1] - start[b]), int(self.ctx[b])
            at = ctx
            while at < ctx + n:
                pid, j = self.table[b, at // self.P], at % self.P
                m = min(self.P - j, ctx + n - at)
                touched[pid] = True
                rows = slice(start[b] + at - ctx, start[b] + at - ctx + m)
                for which, new in ((0, kx), (1, vx)):
                    for h in range(self.heads):
                        piece = new[rows, h]
                        old = np.float32(before[2 + which][pid, h] if j else 0.0)
                        got_scale = after[2 + which][pid, h]
                        codes, codes0 = after[which][pid, h], before[which][pid, h]
                        if which == 1 or exact_keys:
                            want = np.maximum(old, np.float32(np.abs(piece).max()) / np.float32(127))
                            assert got_scale == want
                            q = np.rint(piece.astype(np.float32) / want) if want > 0 else np.zeros_like(piece)
                            assert np.array_equal(codes[j:j + m], q)
                        else:
                            e = bound[rows, h]
                            top = np.abs(piece).max()
                            assert abs(got_scale - max(old, top / 127)) <= e.max() / 127 + 1e-7 * got_scale
                            assert (np.abs(codes[j:j + m] - piece / got_scale) <= 0.5 + 1e-4 + e / got_scale).all()
                        if j and got_scale > old:
                            ratio = np.float32(old) / np.float32(got_scale)
                            assert np.array_equal(codes[:j], np.rint(codes0[:j].astype(np.float32) * ratio))
                        elif j:
                            assert got_scale == old and np.array_equal(codes[:j], codes0[:j])
                        tail = codes[j + m:]
                        assert np.array_equal(tail, codes0[j + m:] if j else np.zeros_like(tail))
                at += m
        for w in range(4):       # pages that no new token falls on keep every bit
            assert np.array_equal(before[w][~touched].view(np.uint8), after[w][~touched].view(np.uint8))
        self.ctx = (self.ctx + np.diff(start)).astype(np.int32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_append_without_rotation_is_exact(P, D):
    say("append", P, D)
    c = Cache(3, 300 // P + 1, 2, D, P, seed=P + D)
    for i, news in enumerate([[5, 0, 1], [1, 1, 1], [2 * P + 3, 17, 0], [1, P, 1], [0, 1, 1], [13, 0, 100]]):
        # louder and quieter calls: the scales of begun pages grow or stay
        x, (_, k, v), before, after, out, start = c.append(news, wide=i % 2 == 0, scale=[1, 3, 0.5, 2, 4, 1][i])
        assert out is None
        c.expect(before, f64(k), f64(v), start)


@pytest.mark.parametrize("D,P,rot,sections,interleaved", [(128, 64, 128, [64], False), (64, 16, 64, [8, 12, 12], False),
                                                          (128, 128, 64, [16, 16], True), (128, 32, 96, [48], False)])
def test_append_rotates_keys_and_queries(D, P, rot, sections, interleaved):
    say("append rope", D, P, rot, sections, interleaved)
    c = Cache(4, 500 // P + 1, 2, D, P, seed=D + P + rot)
    inv = freq(rot // 2)
    rope = block.Rope(torch.from_numpy(inv).to(DEV), sections, interleaved)
    for news in ([130, 1, 64, 3], [1, 1, 1, 1], [2, 200, 1, 0]):
        T = sum(news)
        pos = c.g.integers(0, 5000, size=(len(sections), T)).astype(np.int32)
        x, (q, k, v), before, after, out, start = c.append(news, rope, 6, torch.from_numpy(pos).to(DEV))
        kn = f64(k)
        c.expect(before, R.rope(kn, pos, inv, sections, interleaved), f64(v), start, exact_keys=False,
                 bound=rope_bound(kn, rot // 2, interleaved))
        assert torch.equal(out, block.rope_axes(q, torch.from_numpy(pos).to(DEV), rope))


def test_append_special_values():
    say("append special")
    c = Cache(3, 4, 1, 64, 16, seed=9)
    z = torch.zeros(12, 1, 64, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=DEV)
    k = z.clone()
    k[5, 0, 3] = float("inf")
    v = z.clone()
    v[9, 0, 60] = float("nan")
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    block.kv8_append(c.dev, c.dtable, zero, start, 4, k, v)
    p = c.table[:, 0]
    ks, vs = c.dev.k_scale.cpu()[p, 0], c.dev.v_scale.cpu()[p, 0]
    assert ks[0] == 0 and ks[2] == 0 and torch.isnan(ks[1]) and vs[0] == 0 and vs[1] == 0 and torch.isnan(vs[2])
    assert not c.dev.k[torch.from_numpy(p).long()].any() and not c.dev.v[torch.from_numpy(p).long()].any()
    # a zero page takes its first real scale later; a poisoned one stays poisoned
    one = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    s1 = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    block.kv8_append(c.dev, c.dtable, zero + 4, s1, 1, one, one)
    ks, vs = c.dev.k_scale.cpu()[p, 0], c.dev.v_scale.cpu()[p, 0]
    assert ks[0] == np.float32(1) / np.float32(127) and torch.isnan(ks[1]) and torch.isnan(vs[2])
    assert (c.dev.k.cpu()[p[0], 0, 4] == 127).all() and not c.dev.k.cpu()[p[0], 0, :4].any()


def test_append_bounds_what_the_device_says():
    """Page numbers, lengths and offsets outside their buffers write nothing outside."""
    say("append bounds")
    c = Cache(4, 3, 2, 64, 16, seed=11)
    table = c.dtable.clone()
    table[0, 0] = -1
    table[1, 0] = c.dev.k.shape[0]
    ctx = torch.tensor([0, 0, 3 * 16 - 2, -5], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 3, 6, 12, 400], dtype=torch.int32, device=DEV)
    x = torch.randn(14, 2, 64, device=DEV).to(torch.bfloat16)
    before = c.snapshot()
    block.kv8_append(c.dev, table, ctx, start, 14, x, x)
    after = c.snapshot()
    changed = {int(p) for p in np.unique(np.nonzero((before[0] != after[0]).any((1, 2, 3)))[0])}
    assert changed == {int(c.table[2, 2])}           # two tokens fitted there, the next four had no page
    block.kv8_append(c.dev, c.dtable, torch.zeros_like(ctx), start, 0, x, x)      # max_new 0: nothing appended
    assert all(np.array_equal(a.view(np.uint8), b.view(np.uint8)) for a, b in zip(after, c.snapshot()))


def test_append_long_context_offsets():
    """Pages whose byte offset passes 2^31."""
    say("append far page")
    pages = 2 ** 31 // (8 * 64 * 128) + 40
    cache = block.KVCache8(torch.zeros(pages, 8, 64, 128, dtype=torch.int8, device=DEV),
                           torch.zeros(pages, 8, 128, 64, dtype=torch.int8, device=DEV),
                           torch.zeros(pages, 8, device=DEV), torch.zeros(pages, 8, device=DEV))
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    x = torch.randn(3, 8, 128, device=DEV).to(torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    block.kv8_append(cache, table, i32(0), i32(0, 3), 3, x, x)
    scale = cache.v_scale[-1]
    # the host's IEEE quotient (torch divides by a number through its reciprocal on the GPU)
    assert np.array_equal(scale.cpu().numpy(), x.float().abs().amax((0, 2)).cpu().numpy() / np.float32(127))
    want = torch.round(x.float() / scale[None, :, None]).to(torch.int8)
    assert torch.equal(cache.v[-1, :, :, :3], want.permute(1, 2, 0)) and torch.equal(cache.k[-1, :, :3], want.transpose(0, 1))
    q = torch.randn(3, 8, 128, device=DEV).to(torch.bfloat16)
    out = block.kv8_attention(q, cache, table, i32(3), i32(0, 3), 3, 3)
    kf, vf = want.double() * scale[None, :, None], want.double() * scale[None, :, None]
    s = torch.einsum("ihd,jhd->hij", q.double().cpu(), kf.cpu()) / 128 ** 0.5
    s = s.masked_fill(torch.ones(3, 3).triu(1).bool(), float("-inf")).softmax(-1)
    ref = torch.einsum("hij,jhd->ihd", s, vf.cpu())
    assert (out.double().cpu() - ref).abs().max() <= 2.0 ** -7 * vf.abs().max()


def test_refusals():
    say("refusals")
    c = Cache(2, 4, 2, 64, 16, seed=1)
    ctx, start = torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    rope = block.Rope(torch.ones(32, device=DEV), [16, 16])
    pos = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    for bad in (dict(k=x.float()), dict(k=x[:, :1]), dict(v=x[:1]), dict(ctx_len=ctx.long()), dict(q_start=ctx),
                dict(table=c.dtable[:1]), dict(rope=rope), dict(pos=pos), dict(rope=rope, pos=pos[:1]),
                dict(k=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(q_out=x)):
        args = dict(cache=c.dev, table=c.dtable, ctx_len=ctx, q_start=start, max_new=1, k=x, v=x) | bad
        with pytest.raises(ValueError):
            block.kv8_append(**args)
    with pytest.raises(w4a8.W4A8ArgumentError):      # sections do not add up
        block.rope_axes(x, pos, block.Rope(torch.ones(32, device=DEV), [16, 15]))
    with pytest.raises(w4a8.W4A8ArgumentError):      # more pairs than the head has
        block.rope_axes(x, pos[:1], block.Rope(torch.ones(40, device=DEV)))
    with pytest.raises(w4a8.W4A8ArgumentError):      # a page of 48 tokens
        bad = block.KVCache8.empty(3, 2, 64, 48)
        block.kv8_append(bad, c.dtable, ctx, start, 1, x, x)
    with pytest.raises(w4a8.W4A8ArgumentError):      # a token stride that breaks 16-byte alignment
        y = torch.zeros(2, 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)[:, :128].view(2, 2, 64)
        block.rope_axes(y, pos, rope)
