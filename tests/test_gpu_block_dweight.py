"""The weight's gradient of rmsnorm_grad at the tolerance of the sum that it makes."""

import numpy as np
import pytest
import torch

import block_ref as R
from bit_codebook_quantized_amd import block
from test_gpu_block_norm import f64, grad_case, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("M,K", [(1, 512), (15, 256), (77, 1280), (1030, 512), (2500, 768), (9000, 256), (4100, 2048), (600, 4096),
                                 (2077, 4096), (900, 12288)])
def test_dweight_within_the_roundings_of_its_sum(M, K, rotated):
    """A term is one rounded product and a fused multiply-add; on its way it is added to the rows that its block takes in
    turn, to the others of the block (joined in order), to one in 64 of the blocks' partial rows, and six times
    more.  The workspace holds the partial rows."""
    say("dweight", M, K, rotated)
    g, h, rstd, w, _ = grad_case(M, K, torch.float32, rotated, False)
    dw = block.rmsnorm_grad(g, h, rstd, w, rotated=rotated)[1]
    partial = block.rmsnorm_grad_workspace(M, K) // (4 * K)
    rows = max(1, 16 // (K // 256))                       # of a block at a time
    path = -(-(-(-M // rows)) // partial) + rows + -(-partial // 64) + 6
    hn, gn, r = f64(h), f64(g), f64(rstd)[:, None]
    gy = R.rotate(gn) if rotated else gn
    # of the given rstd; the rotation's stages are 12 roundings of its block's 2-norm
    ref = (gy * hn * r).sum(0)
    dg = np.repeat(np.sqrt((gn.reshape(M, -1, 256) ** 2).sum(2)), 256, axis=1) * 12 * R.U if rotated else 0 * gn
    bound = (np.abs(gy * hn) * r).sum(0) * (path + 1) * R.U * 1.001 + (dg * np.abs(hn) * r).sum(0) + 1e-30
    worst = (np.abs(f64(dw) - ref) / bound).max()
    print("   partial rows %d, path %d, worst error over its bound %.3f" % (partial, path, worst), flush=True)
    assert worst <= 1
