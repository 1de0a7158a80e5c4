"""rmsnorm_quant_act, rmsnorm and rmsnorm_grad against the formulas in 64 bits and against
differences.

Tolerances, with u = 2^-24 and n_k the roundings on the longest path of a row sum (16 terms
in a lane, 4 lane steps, at most 64 slots): a sum of squares of positive terms is within
(16 + 4 + 64) u, rstd within half of that and four more roundings; y adds three; the four
rotation stages add at most 3 u of the block's 2-norm each, and errors e of y change v by at
most their 2-norm.  Together |dv| <= (50 + 3 + 12) u ||y_block||, taken as 80 u."""

import numpy as np
import pytest
import torch

import block_ref as R
from bit_codebook_quantized_amd import block, synth, w4a8

pytestmark = pytest.mark.gpu
DEV, U = "cuda", R.U
EPS = 1e-6


def say(*a):
    print("[case]", *a, flush=True)


def make(m, k, stream, seed):
    g = synth.rng(seed)
    x = torch.from_numpy(g.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16)
    r = torch.from_numpy((g.standard_normal((m, k)) * (1 + 9 * (g.random(k) < 0.01))).astype(np.float32)).to(stream)
    w = torch.from_numpy((1 + 0.1 * g.standard_normal(k)).astype(np.float32))
    return x.to(DEV), r.to(DEV), w.to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def check_rows(h, weight, xq, xs, rstd, y=None, qmax=127):
    """The outputs of one call against the norm of the stored h."""
    k = h.shape[1]
    r_ref, y_ref, v = R.norm(h, weight, EPS)
    assert (np.abs(rstd - r_ref) <= 50 * U * r_ref).all()
    if y is not None:
        assert (np.abs(y - y_ref) <= R.bf16_gap(y_ref) * 1.0001 + 60 * U * np.abs(y_ref)).all()
    if xq is None:
        return
    size = np.sqrt((y_ref.reshape(-1, k // 256, 256) ** 2).sum(2))
    dv = 80 * U * np.repeat(size, 256, axis=1)
    top = np.abs(v).max(1)
    scale = np.where(top > 0, top / qmax, 1.0)
    assert (np.abs(xs - scale) <= dv.max(1) / qmax + 2 * U * scale).all()
    # the code is the nearest to v / xs but for the error of v and the rounding of the quotient
    far = np.abs(xq - v / xs[:, None])
    assert (far <= 0.5 + dv / xs[:, None] + 2 * U * qmax).all(), far.max()
    assert (np.abs(xq) <= qmax).all()


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 256), (1, 4096), (3, 512), (5, 768), (7, 1280), (2, 2048), (33, 2304), (300, 4096),
                                 (9, 4352), (17, 12288), (2, 16384)])
def test_norm_matches_the_formula(M, K, stream):
    say("norm", M, K, stream)
    x, r, w = make(M, K, stream, 100 * K + M)
    rstd = torch.empty(M, device=DEV)
    y = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    xq, xs, h = block.rmsnorm_quant_act(x, w, r, EPS, rstd=rstd, y=y)
    assert torch.equal(h, (r.float() + x.float()).to(stream))
    check_rows(f64(h), f64(w), f64(xq), f64(xs), f64(rstd), f64(y))
    # the parts alone, and in place, give the same bits
    y2, h2 = block.rmsnorm(x, w, r, EPS)
    assert torch.equal(y2, y) and torch.equal(h2, h)
    r2 = r.clone()
    xq3, xs3, h3 = block.rmsnorm_quant_act(x, w, r2, EPS, h=r2)
    assert h3.data_ptr() == r2.data_ptr() and torch.equal(r2, h) and torch.equal(xq3, xq) and torch.equal(xs3, xs)


@pytest.mark.parametrize("M,K,qmax", [(1, 256, 127), (19, 1024, 7), (64, 4096, 127)])
def test_norm_without_a_residual(M, K, qmax):
    say("norm, no residual", M, K, qmax)
    x, _, w = make(M, K, torch.bfloat16, M)
    rstd = torch.empty(M, device=DEV)
    xq, xs, h = block.rmsnorm_quant_act(x, w, None, EPS, qmax=qmax, rstd=rstd)
    assert h is x
    check_rows(f64(x), f64(w), f64(xq), f64(xs), f64(rstd), qmax=qmax)


def test_norm_feeds_the_linear():
    """int8 rows of the fused call and of y through rotate_quant_act differ by y's rounding only."""
    say("norm to linear")
    x, r, w = make(40, 1024, torch.bfloat16, 3)
    layer = w4a8.quantize_w4(synth.gaussian_weight_device(512, 1024, 5, DEV))
    xq, xs, h = block.rmsnorm_quant_act(x, w, r, EPS)
    out = f64(w4a8.w4a8_gemm(xq, xs, layer, torch.float32))
    _, _, v = R.norm(f64(h), f64(w), EPS)
    grid = f64(w4a8.decode_w4_to_int8(layer)) * f64(layer.s_channel)[:, None]
    ref = v @ grid.T
    # the int8 step: each code is off by at most half, so the product by xs / 2 * ||row||_1
    bound = 0.51 * f64(xs)[:, None] * np.abs(grid).sum(1)[None]
    assert (np.abs(out - ref) <= bound).all()


def test_special_rows():
    say("special rows")
    x, r, w = make(6, 512, torch.float32, 4)
    x[1] = 0; r[1] = 0
    x[2, 5] = float("inf")
    r[3, 500] = float("nan")
    r[4] = 3e38
    rstd, y = torch.empty(6, device=DEV), torch.empty(6, 512, dtype=torch.bfloat16, device=DEV)
    xq, xs, h = block.rmsnorm_quant_act(x, w, r, EPS, rstd=rstd, y=y)
    for i in (2, 3, 4):     # an inf, a NaN, an overflow of the sum
        assert torch.isnan(xs[i]) and torch.isnan(rstd[i]) and not xq[i].any() and torch.isnan(y[i]).all()
    assert xs[1] == 1.0 and not xq[1].any() and not y[1].any()
    keep = [0, 5]
    check_rows(f64(h)[keep], f64(w), f64(xq)[keep], f64(xs)[keep], f64(rstd)[keep], f64(y)[keep])


def test_no_rows():
    say("no rows")
    x, r, w = make(0, 512, torch.bfloat16, 1)
    xq, xs, h = block.rmsnorm_quant_act(x, w, r)
    assert xq.shape == (0, 512) and xs.shape == (0,) and h.shape == (0, 512)
    dx, dw = block.rmsnorm_grad(x, r, torch.empty(0, device=DEV), w)
    assert dx.shape == (0, 512) and torch.equal(dw, torch.zeros(512, device=DEV))


def grad_case(M, K, stream, rotated, with_gh, seed=0):
    x, h, w = make(M, K, stream, 7 * K + M + seed)
    g = x
    rstd = torch.from_numpy((1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).astype(np.float32)).to(DEV)
    gh = torch.randn(M, K, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(stream) if with_gh else None
    return g, h, rstd, w, gh


@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,with_gh", [(1, 256, True), (4, 512, False), (77, 1280, True), (1030, 512, True),
                                         (3, 4096, False), (2500, 768, True), (600, 4096, True), (5, 12288, True),
                                         (300, 16384, True)])
def test_grad_matches_the_formula(M, K, with_gh, stream, rotated):
    say("grad", M, K, with_gh, stream, rotated)
    g, h, rstd, w, gh = grad_case(M, K, stream, rotated, with_gh)
    dx, dw = block.rmsnorm_grad(g, h, rstd, w, gh, rotated=rotated)
    hn, wn, gn = f64(h), f64(w), f64(g)
    ref, dw_ref, gy = R.norm_grad(gn, hn, wn, EPS, rotated)
    extra = f64(gh) if with_gh else 0.0
    ref = ref + extra
    r = f64(rstd)[:, None]
    # gy within 12 u of its block's 2-norm; the row sum has at most 90 roundings; the rest a few
    dg = np.repeat(np.sqrt((gn.reshape(M, -1, 256) ** 2).sum(2)), 256, axis=1) * 12 * U if rotated else 0 * gn
    u = np.abs(gy * wn)
    mean = (np.abs(gy * wn * hn)).mean(1, keepdims=True)
    dmean = 95 * U * mean + (dg * np.abs(wn * hn)).mean(1, keepdims=True)
    err = r * (dg * np.abs(wn) + 4 * U * u + np.abs(hn) * r ** 2 * (dmean + 6 * U * mean)) + 4 * U * np.abs(ref) \
        + 2 * U * np.abs(extra)
    if stream == torch.bfloat16:
        err = err + R.bf16_gap(ref) * 1.0001
    assert (np.abs(f64(dx) - ref) <= err).all(), (np.abs(f64(dx) - ref) / err).max()
    # the rows a block takes in turn (at least 256 blocks), then a lane's share of the partial
    # rows (one in 16 of at most M + 15), then 16 lanes
    path = (M + 255) // 256 + M // 16 + 32
    dw_err = (np.abs(gy * hn) * r).sum(0) * (path + 4) * U + (dg * np.abs(hn) * r).sum(0)
    assert (np.abs(f64(dw) - dw_ref) <= dw_err + 1e-30).all(), (np.abs(f64(dw) - dw_ref) / dw_err).max()
    # the same call again, in place and without dweight: the same bits
    dx2, none = block.rmsnorm_grad(g, h, rstd, w, gh, rotated=rotated, need_dweight=False,
                                   dx=gh.clone() if with_gh else None)
    assert none is None and torch.equal(dx2, dx)
    assert torch.equal(block.rmsnorm_grad(g, h, rstd, w, gh, rotated=rotated)[1], dw)


@pytest.mark.parametrize("rotated", [True, False])
def test_grad_matches_differences(rotated):
    """Central differences of sum(g * v(h, w)) in 64 bits along random directions."""
    say("grad differences", rotated)
    M, K = 6, 768
    g, h, rstd, w, _ = grad_case(M, K, torch.float32, rotated, False, seed=9)
    dx, dw = (f64(t) for t in block.rmsnorm_grad(g, h, rstd, w, rotated=rotated))
    hn, wn, gn = f64(h), f64(w), f64(g)
    rng = synth.rng(12)

    def loss(a, b):
        _, y, v = R.norm(a, b, EPS)
        return (gn * (v if rotated else y)).sum()
    for _ in range(8):
        d, e, t = rng.standard_normal((M, K)), rng.standard_normal(K), 1e-5
        slope = (loss(hn + t * d, wn) - loss(hn - t * d, wn)) / (2 * t)
        # fp32 outputs: 1e-5 of the terms' absolute sum covers their roundings, the differences' t^2 term is 1e-10
        assert abs(slope - (dx * d).sum()) <= 1e-5 * np.abs(dx * d).sum()
        slope = (loss(hn, wn + t * e) - loss(hn, wn - t * e)) / (2 * t)
        assert abs(slope - (dw * e).sum()) <= 1e-5 * np.abs(dw * e).sum()


def test_other_stream():
    """Work on another stream than the current one's default, inputs made there."""
    say("other stream")
    s = torch.cuda.Stream()
    x, r, w = make(64, 4096, torch.bfloat16, 5)
    ref = block.rmsnorm_quant_act(x, w, r)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2, r2 = x * 1, r * 1
        out = block.rmsnorm_quant_act(x2, w, r2)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_refusals():
    say("refusals")
    x, r, w = make(4, 512, torch.bfloat16, 6)
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x.float(), w, r)
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x, w[:256], r)
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x, w, r.half())
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x, w, r[:, :256])
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x, w, None, h=r)
    with pytest.raises(ValueError):
        block.rmsnorm_quant_act(x.t().contiguous().t(), w, r)
    with pytest.raises(w4a8.W4A8ArgumentError):
        block.rmsnorm_quant_act(x, w, r, eps=0.0)
    with pytest.raises(w4a8.W4A8ArgumentError):
        block.rmsnorm_quant_act(x, w, r, qmax=128)
    big = torch.zeros(1, 16384 + 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(w4a8.W4A8ArgumentError):
        block.rmsnorm_quant_act(big, torch.ones(16384 + 256, device=DEV))
    rstd = torch.ones(4, device=DEV)
    with pytest.raises(ValueError):
        block.rmsnorm_grad(x, r, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        block.rmsnorm_grad(x, r, rstd, w, grad_h=r.float())
