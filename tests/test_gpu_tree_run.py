"""Attention of drafted trees over the 4-bit cache, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
import step_reference as R
import tree_reference as T

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def bits(mask, n, total):
    """[n, total]: what each row of one request does not see."""
    hide = np.zeros((n, total), dtype=bool)
    for i in range(n):
        for j in range(n):
            word = int(np.uint32(mask[i, j >> 5])) if j >> 5 < mask.shape[1] else 0
            hide[i, total - n + j] = not word >> (j & 31) & 1
    return hide


def tree_case(kv, new, hq, hkv, dk, dv, page=16, layout="HND", out="bf16", seed=0, masks=None,
              words=None, only=None, live=None, q_pad=0, g=(0.75, 1.25), q_scale=1.0, **plan_kw):
    """Run and check."""
    c = T.Nvfp4Case(kv, page, hkv, dk, dv, layout, seed=seed, g=g)
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn((sum(new) + 1, hq + q_pad, dk), generator=gen) * q_scale).to(torch.bfloat16)
    q = q.cuda()[:, q_pad:]
    rng = np.random.default_rng(seed + 1)
    qo = np.concatenate([[0], np.cumsum(new)])
    words = words or (max(max(new), 1) + 31) // 32
    if masks is None:
        masks = [T.mask_words(T.ancestors(T.random_parents(rng, n)), words) for n in new]
    mask = np.concatenate([m.reshape(-1, words) for m in masks])
    last = c.last
    if live is not None:
        last, plan_kw["device_last_page_len"] = live, c.last_page_len
    plan = N.nvfp4kv_decode_plan(qo, c.indptr, last, hq, hkv, dk, dv, page_size=page,
                                 out_dtype=DT[out], **plan_kw)
    tree_mask = torch.from_numpy(mask.astype(np.int32)).cuda()
    o, lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, tree_mask)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    got, gl = R.to_np(o), R.to_np(lse)
    scale = 1 / math.sqrt(dk)
    for b, n in enumerate(new):
        if not n or (only is not None and b not in only):
            continue
        rows = slice(int(qo[b]), int(qo[b + 1]))
        want = T.tree_attention(R.to_np(q[rows]), c.dense(0, b), c.dense(1, b),
                                bits(masks[b], n, kv[b]), scale)
        T.check_tree(got[rows], gl[rows], want, dk, DT[out])
    return c, plan, o, lse, q, tree_mask


DIMS = [(64, 64), (128, 128), (256, 128), (256, 256), (512, 256)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("page,layout,out", [(16, "HND", "bf16"), (16, "NHD", "f16"),
                                             (1, "HND", "bf16")])
@pytest.mark.parametrize("new", [(1, 2, 0), (3, 4, 2), (5, 16, 1), (13, 37, 40)])
def test_dims_and_rows(dk, dv, page, layout, out, new):
    """Up to 4, 8, 32 and 80 rows per kv head; the last request is nothing but its tree."""
    tree_case((37, 300, 40), new, 4, 2, dk, dv, page=page, layout=layout, out=out,
              seed=dk + sum(new))


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("hq,hkv,new", [(4, 4, (8, 1, 7)), (5, 1, (3, 1, 6)), (16, 1, (1, 4, 1)),
                                        (32, 4, (9, 65, 90)), (8, 8, (20, 33, 64))])
def test_groups(hq, hkv, new, page):
    tree_case((37, 65, 90), new, hq, hkv, 128, 128, page=page, seed=hq + sum(new))


@pytest.mark.parametrize("kernel", [1, 3])
@pytest.mark.parametrize("chunk", [16, 64, 176])
@pytest.mark.parametrize("new", [(5, 1, 0, 30), (16, 1, 17, 64)])
@pytest.mark.parametrize("num_sms", [0, 1])
def test_splits(kernel, chunk, new, num_sms):
    """Chunks that begin and end inside the tree, some that hold none of a row's tokens:
    joined by a cluster for each request and kv head, or (no room for such: one SM) folded."""
    _, plan, *_ = tree_case((300, 1, 17, 1111), new, 8, 2, 128, 128, kernel=kernel,
                            force_chunk_tokens=chunk, num_sms=num_sms, seed=chunk)
    assert plan.info.split == 1


@pytest.mark.parametrize("kernel", [1, 3])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 111, 112, 113, 127, 128, 129, 255])
def test_tree_across_tiles(kernel, before):
    """The tree's first token anywhere in a tile of 16 and of 128."""
    tree_case((before + 37,), (37,), 4, 1, 128, 128, kernel=kernel, seed=before)


@pytest.mark.parametrize("kernel,hq,hkv", [(1, 2, 2), (1, 4, 2), (1, 8, 1), (3, 4, 2), (3, 32, 1)])
def test_masks_of_any_kind(kernel, hq, hkv):
    """Rows that see nothing of the tree, nothing at all, later nodes, all; bits behind the
    request's rows set."""
    rng = np.random.default_rng(hq)
    new, kv = (7, 4, 20, 3), (60, 4, 20, 200)
    masks = [rng.integers(-2**31, 2**31, (n, 1)).astype(np.int32) for n in new]
    for m in masks:
        m[0], m[-1] = 0, -1  # (requests 1 and 2 have no token before the tree: row 0 sees none)
    _, _, out, lse, *_ = tree_case(kv, new, hq, hkv, 128, 128, masks=masks, words=1, kernel=kernel,
                                   seed=hq)
    assert (lse[7] == -math.inf).all() and (lse[11] == -math.inf).all()
    assert (out[7] == 0).all() and (out[11] == 0).all()


@pytest.mark.parametrize("rows", [17, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200])
@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 256), (512, 256)])
def test_rows_of_a_block(rows, dk, dv):
    """Row counts around the warps, the copies and the blocks of the wide kernel, one head a
    kv head, with and without a split."""
    for chunk in (0, 64):
        tree_case((rows, 300), (rows, min(rows, 70)), 1, 1, dk, dv, seed=rows,
                  force_chunk_tokens=chunk)


@pytest.mark.parametrize("kernel", [1, 3])
def test_tokens_past_the_words_are_not_seen(kernel):
    masks = [np.full((50, 1), -1, dtype=np.int32), np.full((3, 1), -1, dtype=np.int32)]
    tree_case((90, 30), (50, 3), 4, 2, 128, 128, masks=masks, words=1, kernel=kernel, seed=5)


@pytest.mark.parametrize("kernel", [1, 3])
def test_large_tree(kernel):
    """300 nodes: ten words a row, several tiles of tree, chains far apart."""
    rng = np.random.default_rng(7)
    masks = [T.mask_words(T.ancestors(T.random_parents(rng, 300, deep=True)), 10)]
    tree_case((301,), (300,), 4, 2, 128, 128, masks=masks, words=10, kernel=kernel, seed=6)


@pytest.mark.parametrize("kernel", [1, 3])
def test_values_of_all_sizes(kernel):
    """Global scales far from 1 (scores stay in range by the query)."""
    tree_case((70, 200), (9, 30), 4, 2, 128, 128, kernel=kernel, g=(0.75, 2.0 ** -60), seed=8)
    tree_case((70, 200), (9, 30), 4, 2, 128, 128, kernel=kernel, g=(2.0 ** -30, 2.0 ** 60), seed=9)


@pytest.mark.parametrize("kernel", [1, 3])
@pytest.mark.parametrize("q_scale", [2.0 ** -120, 2.0 ** -60, 0.0, 2.0 ** 60])
def test_queries_of_all_sizes(kernel, q_scale):
    """Scores that vanish (every key that is seen weighs the same, none of the others does)
    and scores kept in range by the cache's scale."""
    tree_case((70, 200, 9), (9, 30, 9), 4, 2, 128, 128, kernel=kernel, q_scale=q_scale, seed=16,
              g=(2.0 ** -64, 1.25))


def test_a_chain_is_the_causal_mask():
    """A tree without branches is the causal mask: up to 16 rows a kv head it runs in the
    causal plan's kernel (with one SM: no cluster takes a whole request) and gives the same
    bits."""
    kv, new = (37, 300, 64), (4, 1, 3)
    chains = [T.mask_words(T.ancestors(range(-1, n - 1)), 2) for n in new]
    c, plan, out, lse, q, _ = tree_case(kv, new, 8, 2, 128, 128, masks=chains, words=2, kernel=1,
                                        num_sms=1, seed=11)
    qo = np.concatenate([[0], np.cumsum(new)])
    causal = N.nvfp4kv_decode_plan(qo, c.indptr, c.last, 8, 2, 128, 128, kernel=1, causal=True,
                                   num_sms=1)
    assert plan.info.rows_per_block == 16
    o2, l2 = N.nvfp4kv_decode_run(causal, q, c.cache, c.kv_indices)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("kernel", [1, 3])
def test_chains_of_many_rows(kernel):
    kv, new = (37, 300, 64), (5, 33, 64)
    chains = [T.mask_words(T.ancestors(range(-1, n - 1)), 2) for n in new]
    tree_case(kv, new, 8, 2, 128, 128, masks=chains, words=2, kernel=kernel, seed=11)


@pytest.mark.parametrize("kernel", [1, 3])
def test_live_lengths(kernel):
    """The plan keeps page counts; the tree moves with the lengths that the device holds."""
    tree_case((21, 35), (5, 9), 8, 2, 128, 128, live=[16, 16], kernel=kernel, seed=12)


@pytest.mark.parametrize("kernel", [1, 3])
@pytest.mark.parametrize("page", [16, 1])
def test_new_tokens_in_the_same_launch(kernel, page):
    """new_k and new_v: the cache holds what nvfp4kv_quantize_append writes, the output is
    that of the call without them."""
    kv, new, hkv = (37, 300, 30), (7, 33, 30), 2
    c = T.Nvfp4Case(kv, page, hkv, 128, 128, seed=13)
    other = T.Nvfp4Case(kv, page, hkv, 128, 128, seed=13)
    g = torch.Generator().manual_seed(13)
    rows = sum(new)
    k, v = (torch.randn((rows, hkv + 1, 128), generator=g).to(torch.bfloat16).cuda()[:, 1:]
            for _ in range(2))
    q = torch.randn((rows, 8, 128), generator=g).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(13)
    mask = i32(np.concatenate([T.mask_words(T.ancestors(T.random_parents(rng, n)), 2)
                               for n in new]))
    qo = np.concatenate([[0], np.cumsum(new)])
    idx = i32([b for b, n in enumerate(new) for _ in range(n)])
    pos = i32([t for n, m in zip(new, kv) for t in range(m - n, m)])
    N.nvfp4kv_quantize_append(other.cache, k, v, idx, pos, other.kv_indices, other.kv_indptr,
                              other.last_page_len)
    plan = N.nvfp4kv_decode_plan(qo, c.indptr, c.last, 8, hkv, 128, 128, page_size=page,
                                 kernel=kernel)
    want = N.nvfp4kv_tree_run(plan, q, other.cache, other.kv_indices, mask)
    got = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask, new_k=k, new_v=v)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    mine, theirs = c.download(), other.download()
    for n in mine:
        assert np.array_equal(mine[n], theirs[n]), n
    for a, b in zip(got, want):
        assert torch.allclose(a.float(), b.float(), atol=0 if not plan.info.split else 2.0 ** -7)


@pytest.mark.parametrize("kernel", [1, 3])
def test_bad_page_ids_are_flagged(kernel):
    c = T.Nvfp4Case((100,), 16, 2, 128, 128, seed=14)
    idx = c.kv_indices.clone()
    idx[2], idx[4] = c.total, -5
    plan = N.nvfp4kv_decode_plan([0, 6], c.indptr, c.last, 8, 2, 128, 128, kernel=kernel)
    q = torch.zeros((6, 8, 128), dtype=torch.bfloat16).cuda()
    N.nvfp4kv_tree_run(plan, q, c.cache, idx, i32(np.full((6, 1), -1)))
    assert N.nvfp4kv_workspace_flags(plan, clear=True) == _lib.FLAG_BAD_PAGE_INDEX


@pytest.mark.parametrize("kernel", [1, 3])
def test_stream_graph_and_given_outputs(kernel):
    c, plan, out, lse, q, mask = tree_case((37, 300), (9, 16), 8, 2, 128, 128, kernel=kernel,
                                           seed=15, q_pad=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask, stream=side)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask, out=o3, lse=l3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    mask.zero_()  # read at replay: the rows see what stands before the tree only
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, o3) and (l3[:9] != lse[:9]).all()


@pytest.mark.parametrize("dk,dv,kv,new", [
    (128, 128, (2000, 300), (2, 3)), (128, 128, (9000, 4100), (20, 30)),
    (64, 64, (5000, 700), (9, 40)), (512, 256, (6000, 700), (9, 40))])
def test_one_plan_for_trees_and_for_causal_rows(dk, dv, kv, new):
    """A plan's workspace serves both attentions in turn: each leaves the counters of its
    split requests as it found them."""
    c, plan, o, lse, q, mask = tree_case(kv, new, 8, 2, dk, dv, seed=21)
    ref = N.nvfp4kv_decode_plan(np.concatenate([[0], np.cumsum(new)]), c.indptr, c.last, 8, 2, dk,
                                dv, causal=True)
    want, want_lse = N.nvfp4kv_decode_run(ref, q, c.cache, c.kv_indices)
    for _ in range(3):
        got, got_lse = N.nvfp4kv_tree_run(ref, q, c.cache, c.kv_indices, mask)
        assert torch.equal(got, o) and torch.equal(got_lse, lse)
        got, got_lse = N.nvfp4kv_decode_run(ref, q, c.cache, c.kv_indices)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert N.nvfp4kv_workspace_flags(ref) == 0


def test_two_streams_at_once():
    """Calls of several kernels' forms in flight together, each with a plan of its own."""
    cases = [tree_case(kv, new, 8, 2, dk, dv, seed=30 + i) for i, (kv, new, dk, dv) in enumerate(
        [((9000, 4100), (20, 30), 128, 128), ((6000, 700), (9, 40), 512, 256),
         ((5000, 7000), (16, 16), 64, 64), ((3000, 200), (3, 2), 128, 128)])]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [(torch.empty_like(o), torch.empty_like(lse)) for _, _, o, lse, _, _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, plan, _, _, q, mask), s, (o, lse) in zip(cases, streams, outs):
            N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask, out=o, lse=lse, stream=s)
    torch.cuda.synchronize()
    for (_, plan, o, lse, _, _), got in zip(cases, outs):
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert N.nvfp4kv_workspace_flags(plan) == 0


@pytest.mark.parametrize("dk,dv,hq,hkv,new,batch,most", [
    (128, 128, 16, 2, 10, 60, 5000), (64, 64, 32, 8, 9, 16, 8192), (512, 256, 16, 2, 8, 30, 8192)])
def test_uneven_batches_in_several_waves(dk, dv, hq, hkv, new, batch, most):
    """Requests of very unequal lengths, one without rows and equal ones among them: clusters
    of whole requests, the longest first, in more than one wave (checked are a few)."""
    rng = np.random.default_rng(dk)
    kv = [int(x) for x in rng.integers(300, most, batch - 3)] + [1500, 1500, 77]
    n = [new] * (batch - 1) + [0]
    tree_case(kv, n, hq, hkv, dk, dv, seed=dv, only=(0, 5, 11, batch - 3, batch - 2))
