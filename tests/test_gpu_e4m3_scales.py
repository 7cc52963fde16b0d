"""Value scales at both ends of the allowed range [2^-64, 2^64] in one request:
the row sum has to keep every weight, however small its value's scale is."""
import math

import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import test_gpu_step_ops as T

pytestmark = pytest.mark.gpu

# query rows per kv head with two heads to one: the blocks of 8 and of 16 rows, the
# tensor-memory kernel with blocks of 32 and (at 128 dims) of 64
ROWS = [1, 6, 12, 40]


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("chunk", [0, -1, 16, 128])  # -1: whole requests
@pytest.mark.parametrize("order", [(64, -64), (-64, 64), (0, -64, 64), (64, 0, -64)])
def test_equal_scores_over_the_whole_range(rows, page, order, chunk):
    """Zero keys: every token weighs the same and lse is the logarithm of their
    number, whatever the values' scales, in any order of pages, within a tile (pages
    of one token) and between warps, tiles and splits."""
    kv = (40, 200, 300)

    def edit(c, q):
        c.codes[0][:] = 0
        for b in range(len(kv)):
            for i, pg in enumerate(c.pages(b)):
                c.scale[1][pg] = 2.0 ** order[i % len(order)]
    _, plan, _ = T.attend_case(kv, (rows, 1, rows), 2, 1, 128, 128, page=page, edit=edit,
                               force_chunk_tokens=max(chunk, 0), disable_split=chunk < 0,
                               seed=rows)
    assert not chunk or plan.info.split == (chunk > 0)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("chunk", [0, -1, 16])  # -1: whole requests
@pytest.mark.parametrize("far", [40.0, 90.0, 130.0, -40.0])
def test_scores_against_scales(rows, far, chunk):
    """The tokens of the smallest scale lie `far` score bits above those of the
    largest: the maximum of score + log2 of the scale and the maximum of the score
    are different tokens (or, from 128 on, the same); a split state of the largest
    scale then has a weight of 2^-130, and values that are 2^128 as large."""
    dk, kv = 128, (100, 260)

    def edit(c, q):
        q[:] = 0
        q[:, :, 0] = 1.0  # a score is sm_scale * code of dim 0 * the key's scale
        c.codes[0][:] = 0
        c.codes[0][..., 0] = 0x38  # 1
        for b in range(len(kv)):
            for i, pg in enumerate(c.pages(b)):
                low = i % 2
                c.scale[1][pg] = 2.0 ** (-64 if low else 64)
                c.scale[0][pg] = max(far if low else -far, 2.0 ** -20) * math.log(2) * math.sqrt(dk)
    T.attend_case(kv, (rows, 1), 2, 1, dk, 128, edit=edit, force_chunk_tokens=max(chunk, 0),
                  disable_split=chunk < 0, seed=rows)


@pytest.mark.parametrize("dk,dv,heads", [(64, 64, 2), (256, 256, 2), (512, 256, 2), (256, 128, 2)])
@pytest.mark.parametrize("rows", [1, 20])
def test_other_dims_over_the_whole_range(dk, dv, heads, rows):
    def edit(c, q):
        c.codes[0][:] = 0
        for i, pg in enumerate(c.pages(0)):
            c.scale[1][pg] = 2.0 ** (64, -64, -64, 0)[i % 4]
    T.attend_case((400,), (rows,), heads, 1, dk, dv, edit=edit, seed=dk)


def test_a_page_of_zero_values_beside_large_ones():
    """What the append itself writes: scale 2^-64 for a page of zeros, 2^64 for the
    largest values; then attention with equal scores."""
    c = N.E4m3Cache.allocate(8, 1, 128, 128)
    k = torch.zeros((48, 1, 128), device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    v[16:32] = 2.0 ** 72
    i32 = T.i32
    kvp, idx, last = i32([0, 3]), i32([4, 2, 6]), i32([16])
    N.nvfp4kv_e4m3_append(c, k, v, i32([0, 48]), kvp, idx, last)
    assert c.v_scale[[4, 2, 6], 0].tolist() == [2.0 ** -64, 2.0 ** 64, 2.0 ** -64]
    for rows in ROWS:
        plan = N.nvfp4kv_decode_plan([0, rows], [0, 3], [16], 2, 1, 128, 128, kernel=5)
        q = torch.randn((rows, 2, 128), device="cuda").to(torch.bfloat16)
        out, lse = N.nvfp4kv_e4m3_decode_run(plan, q, c, idx)
        # 16 of 48 equal weights on 2^72 (a code and scale without rounding): 2^72 / 3;
        # weight f16 2^-11, pieces 2^-12, sums and division 2^-19, output 2^-8
        tol = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -19
        assert float((out.double() * 3 / 2.0 ** 72 - 1).abs().max()) <= tol
        assert float((lse.double() - math.log(48)).abs().max()) <= 2.0 ** -19
