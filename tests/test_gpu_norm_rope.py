"""Norms of the query and key heads with their rotary positions in one pass, against 64
bits."""
import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R
import tree_reference as T

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def rows(tokens, heads, dim, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, heads + pad, dim), generator=g) * scale
    x *= torch.exp2(torch.randint(-4, 5, (tokens, heads + pad, 1), generator=g).float())
    return x.to(DT[dtype]).cuda()[:, pad:]


def weights(dim, kind, offset, seed):
    g = torch.Generator().manual_seed(seed)
    w = 1.0 - offset + 0.3 * torch.randn(dim, generator=g)
    w[::7] *= -1.0
    return w.to(kind).cuda()


def check(got, x, w, pos, rotary, interleaved, freq, offset, eps, attn):
    """Beside the result's own rounding (half a step) the float32 parts: r from a sum of
    at most 16 + 5 additions (its half counts) and rsqrtf (2 units): 2^-20; the weight's
    sum with the offset, its product with the cosine, the cosine itself (2^-23.3 from the
    angle, 2^-23 from sincospif), two products and their sum: 2^-21 of |n1| + |n2|.
    Together less than 2^-19 of the pair's sizes (of |n| where dims only pass)."""
    n = T.norm(x, w, offset, eps)
    y, size = R.rope(n, pos, rotary, interleaved, freq, attn)
    size = np.where(size > 0, size * max(attn, 1.0), np.abs(n.numpy()))
    half = torch.finfo(x.dtype).eps / 2
    tol = half * np.abs(y) + 2.0 ** -19 * size * (1 + half)
    tol += float(torch.finfo(x.dtype).smallest_normal) * half  # subnormal results
    err = np.abs(R.to_np(got) - y)
    assert (err <= tol).all(), float((err / tol).max())


CASES = [(64, 64), (128, 128), (128, 32), (128, 66), (128, 2), (256, 64), (256, 256), (512, 512),
         (512, 16), (512, 250), (8, 8), (8, 2), (40, 24), (80, 80), (80, 64), (320, 200)]


@pytest.mark.parametrize("dim,rotary", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,kind", [("bf16", torch.bfloat16), ("f16", torch.float32)])
def test_layouts(dim, rotary, interleaved, dtype, kind):
    offset = 1.0 if kind == torch.float32 else 0.0
    q, k = rows(7, 5, dim, dtype, dim), rows(7, 2, dim, dtype, dim + 1, pad=1)
    qw, kw = weights(dim, kind, offset, 1), weights(dim, kind, offset, 2)
    pos = torch.tensor([0, 1, 5, 4095, 2**31 - 1, 77, 131072], dtype=torch.int32).cuda()
    plan = N.nvfp4kv_rope_plan(dim, rotary, interleaved=interleaved, attention_factor=1.25)
    qo, ko = N.nvfp4kv_norm_rope(plan, q, k, pos, qw, kw, eps=1e-6, weight_offset=offset)
    freq = R.rope_frequencies(rotary, 10000.0)
    check(qo, q, qw, pos.tolist(), rotary, interleaved, freq, offset, 1e-6, 1.25)
    check(ko, k, kw, pos.tolist(), rotary, interleaved, freq, offset, 1e-6, 1.25)


@pytest.mark.parametrize("tokens,hq,hkv", [(1, 32, 8), (211, 16, 2), (3, 1, 1), (2, 7, 0),
                                           (2, 0, 3), (1, 67, 5), (19457, 1, 1)])
def test_sizes(tokens, hq, hkv):
    q = rows(tokens, hq, 128, "bf16", tokens) if hq else None
    k = rows(tokens, hkv, 128, "bf16", tokens + 1) if hkv else None
    w = weights(128, torch.bfloat16, 0.0, 3)
    pos = (torch.arange(tokens, dtype=torch.int32) * 37 % 9001).cuda()
    plan = N.nvfp4kv_rope_plan(128)
    qo, ko = N.nvfp4kv_norm_rope(plan, q, k, pos, w, w)
    freq = R.rope_frequencies(128, 10000.0)
    for got, x in ((qo, q), (ko, k)):
        if x is None:
            assert got is None
        else:
            check(got, x, w, pos.tolist(), 128, False, freq, 0.0, 1e-6, 1.0)


@pytest.mark.parametrize("rotary", [128, 66])
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 62, 2.0 ** -60, 2.0 ** -100, 2.0 ** -125])
def test_sizes_of_values(rotary, scale):
    """Heads whose squares leave float32's range on either side."""
    q = rows(5, 4, 128, "bf16", 9, scale)
    q[1, 1] = 0  # a head of zeros is zeros
    q[2, 2, 1:] = 0
    w = weights(128, torch.float32, 0.0, 4)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    plan = N.nvfp4kv_rope_plan(128, rotary)
    freq = R.rope_frequencies(rotary, 10000.0)
    for eps in (1e-6, 1e-20):
        got, _ = N.nvfp4kv_norm_rope(plan, q, None, pos, w, eps=eps)
        check(got, q, w, pos.tolist(), rotary, False, freq, 0.0, float(np.float32(eps)), 1.0)


def test_values_that_are_not_finite():
    """An infinite element is NaN with its pair and the others 0; a NaN makes its head NaN;
    no other head knows of either."""
    q = rows(3, 4, 64, "bf16", 10)
    clean = q.clone()
    q[0, 1, 5], q[1, 2, 40] = float("inf"), float("nan")
    w = weights(64, torch.bfloat16, 0.0, 5)
    pos = torch.arange(3, dtype=torch.int32).cuda()
    plan = N.nvfp4kv_rope_plan(64)
    got, want = (N.nvfp4kv_norm_rope(plan, x, None, pos, w)[0] for x in (q, clean))
    assert got[1, 2].isnan().all()
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[5, 37]] = True
    assert got[0, 1, bad].isnan().all() and (got[0, 1, ~bad] == 0).all()
    same = torch.ones((3, 4), dtype=torch.bool, device="cuda")
    same[0, 1] = same[1, 2] = False
    assert torch.equal(got[same], want[same])


def test_in_place_rows_behind_and_streams():
    """In place on a view of one projection's output; rows past the positions stay; the same
    on a stream of its own and from a captured graph."""
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((9, 6 + 2 + 2, 128), generator=g).to(torch.bfloat16).cuda()
    w = weights(128, torch.bfloat16, 0.0, 6)
    pos = torch.arange(7, dtype=torch.int32).cuda() * 11
    plan = N.nvfp4kv_rope_plan(128, interleaved=True)
    want = N.nvfp4kv_norm_rope(plan, qkv[:, :6], qkv[:, 6:8], pos, w, w)
    before = qkv.clone()
    out = N.nvfp4kv_norm_rope(plan, qkv[:, :6], qkv[:, 6:8], pos, w, w, q_out=qkv[:, :6],
                              k_out=qkv[:, 6:8])
    assert torch.equal(out[0][:7], want[0]) and torch.equal(out[1][:7], want[1])
    assert torch.equal(qkv[7:], before[7:]) and torch.equal(qkv[:, 8:], before[:, 8:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2, k2 = N.nvfp4kv_norm_rope(plan, before[:, :6], before[:, 6:8], pos, w, w, stream=side)
    side.synchronize()
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    q3 = torch.zeros_like(q2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.nvfp4kv_norm_rope(plan, before[:, :6], None, pos, w, q_out=q3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q3, want[0])
