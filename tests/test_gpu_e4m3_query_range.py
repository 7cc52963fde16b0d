"""Query rows with one dim far above the others: the scores keep the small dims'
bits, and a row's result does not depend on how many rows share its batch."""
import math

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R
import test_gpu_step_ops as T

pytestmark = pytest.mark.gpu
KV = (700, 90)


def run(rows, dk, dv, dtype, size, seed=0):
    """`rows` query rows of two heads on one kv head, each with a dim of +-2 * size
    where the keys are zero; returns the results of the first request and the
    reference's.

    Scores: queries are exact in the products (2^-31 of the largest |q| at most is
    left out), and a product sum has 3 Dk terms of float32 size at most 1.15 times
    the row's (pieces of 1, 1/8 and 1/64): 3.5 Dk 2^-23 sm_scale sum|q k|, and the
    exponential 2^-21."""
    c = T.CacheCase(KV, 16, 1, dk, dv, seed=seed, spread=0)
    rng = np.random.default_rng(seed)
    c.codes[0][..., 5] = 0
    c.upload()
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((KV[0], 2, dk), generator=g)[:rows + 1]
    q[:, :, 5] = 2.0 * size * torch.from_numpy(rng.choice([-1.0, 1.0], (len(q), 2))).float()
    q = q.to(T.DT[dtype]).cuda()
    plan = N.nvfp4kv_decode_plan([0, rows, rows + 1], c.indptr, c.last, 2, 1, dk, dv, kernel=5,
                                 out_dtype=torch.float16)
    out, lse = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    k, v = (R.dequantised(c.codes[i], c.scale[i], c.pages(0), KV[0]) for i in (0, 1))
    vs = np.repeat(c.scale[1][c.pages(0)].T.astype(np.float64), 16, 1)[:, :KV[0]]
    scale = float(np.float32(1 / math.sqrt(dk)))
    ref, rl, mean, reach, floor = R.attention(R.to_np(q[:rows]), k, v, vs, scale, False)
    k_sum = np.abs(k).sum(-1).max()
    delta = (3.5 * dk * 2.0 ** -23 * reach + 2.0 ** -21
             + 2.0 ** -31 * scale * np.abs(R.to_np(q[:rows])).max(-1) * k_sum)
    return plan, R.to_np(out[:rows]), R.to_np(lse[:rows]), ref, rl, mean, floor, delta


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 128), (256, 256), (64, 64), (512, 256)])
@pytest.mark.parametrize("rows", [1, 6, 12, 40])
@pytest.mark.parametrize("size", [1.0, 1024.0, 16384.0])
def test_outlier_dim(rows, dk, dv, dtype, size):
    _, out, lse, ref, rl, mean, floor, delta = run(rows, dk, dv, dtype, size, seed=dk)
    eps = 2.0 ** -11
    # weights: f16 2^-11 and pieces 2^-12, at least 2^-20 + 2^-25 of the largest; f32
    # sums and a merge of split states 2^-19
    tol = (eps * np.abs(ref) + (mean * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -19 + 2 * delta[..., None])
                                + (2.0 ** -20 + 2.0 ** -25) * floor) * (1 + eps) + 2.0 ** -25)
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())
    bad = np.abs(lse - rl) / (delta + 2.0 ** -19 + np.abs(rl) * 2.0 ** -22)
    assert bad.max() <= 1, float(bad.max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_row_does_not_depend_on_its_batch(dtype):
    """The first row alone and among 6, 12, 20 and 40: the same score sums, by
    whichever kernel, up to both sides' float32 sums."""
    _, _, one, _, rl, _, _, delta = run(1, 128, 128, dtype, 4096.0)
    for rows in (6, 12, 20, 40):
        _, _, lse, _, rl2, _, _, d2 = run(rows, 128, 128, dtype, 4096.0)
        assert rl2[0, 0] == rl[0, 0]  # the same inputs
        tol = delta[0] + d2[0] + 2.0 ** -18 + np.abs(rl[0]) * 2.0 ** -21
        assert (np.abs(lse[0] - one[0]) <= tol).all()
