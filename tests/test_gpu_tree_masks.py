"""Tree masks and positions from the nodes' parents, against sets of ancestors."""
import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
import tree_reference as T

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def run(trees, kv_len, words, extra_rows=0, parents=None):
    """(masks, positions, flags) with -7 where nothing is written."""
    flat = [p for t in trees for p in t] if parents is None else parents
    qo = np.concatenate([[0], np.cumsum([len(t) for t in trees])])
    rows = len(flat) + extra_rows
    mask = torch.full((rows, words), -7, dtype=torch.int32).cuda()
    pos = torch.full((rows,), -7, dtype=torch.int32).cuda()
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    N.nvfp4kv_tree_masks(i32(flat + [5] * extra_rows), i32(qo), i32(kv_len), tree_mask=mask,
                         positions=pos, device_flags=flags)
    return mask.cpu().numpy(), pos.tolist(), int(flags)


def want(trees, kv_len, words):
    masks, pos = [], []
    for t, n in zip(trees, kv_len):
        seen = T.ancestors(t)
        masks.append(T.mask_words(seen, words))
        pos += [n - len(t) + len(s) - 1 for s in seen]
    return np.concatenate(masks) if masks else np.zeros((0, words)), pos


@pytest.mark.parametrize("sizes,words", [
    ((1,), 1), ((5, 0, 7), 1), ((32, 1, 31), 1), ((33, 64, 2), 2), ((0, 0), 1), ((100, 3), 5),
    ((1024, 1, 1000), 32), ((64,) * 70, 2)])
@pytest.mark.parametrize("deep", [False, True])
def test_masks(sizes, words, deep):
    rng = np.random.default_rng(sum(sizes) + deep)
    trees = [T.random_parents(rng, n, deep) for n in sizes]
    kv = [n + int(rng.integers(0, 5000)) for n in sizes]
    mask, pos, flags = run(trees, kv, words, extra_rows=3)
    masks, positions = want(trees, kv, words)
    n = sum(sizes)
    assert flags == 0 and np.array_equal(mask[:n], masks) and pos[:n] == positions
    assert (mask[n:] == -7).all() and pos[n:] == [-7] * 3  # rows behind stay


def test_chain_and_forest():
    chain = list(range(-1, 299))
    mask, pos, flags = run([chain, [-1] * 40], [300, 1000], 10)
    masks, positions = want([chain, [-1] * 40], [300, 1000], 10)
    assert flags == 0 and np.array_equal(mask, masks) and pos == positions
    assert pos[:300] == list(range(300)) and pos[300:] == [960] * 40


def test_parents_that_are_no_tree():
    """A parent at or behind its node, or below -1: flagged, the node stands as a root."""
    given = [0, 5, 1, -2, 2, 2**30]
    mask, pos, flags = run([given], [10], 1)
    masks, positions = want([[-1, -1, 1, -1, 2, -1]], [10], 1)
    assert flags == _lib.FLAG_BAD_TREE and np.array_equal(mask, masks) and pos == positions


@pytest.mark.parametrize("sizes,kv,words", [((4, 33, 2), (9, 90, 5), 1), ((4, 6, 2), (9, 5, 5), 1)])
def test_requests_left_out(sizes, kv, words):
    """More nodes than bits, more nodes than tokens: that request alone is left out."""
    trees = [[-1] * n for n in sizes]
    mask, pos, flags = run(trees, kv, words)
    masks, positions = want(trees, kv, 2)
    a, z = sizes[0], sizes[0] + sizes[1]
    keep = np.r_[0:a, z:sum(sizes)]
    assert flags == _lib.FLAG_BAD_LENGTH
    assert np.array_equal(mask[keep], masks[keep, :words])
    assert [pos[i] for i in keep] == [positions[i] for i in keep]
    assert (mask[a:z] == -7).all() and pos[a:z] == [-7] * (z - a)


def test_rows_that_cannot_be():
    """Row lists that fall, start below 0 or pass the rows: left out, nothing else."""
    par = i32([-1] * 8)
    for qo, good in (([0, 3, 2], [0, 1, 2]), ([-1, 2, 4], [2, 3]), ([0, 2, 9], [0, 1])):
        mask = torch.full((8, 1), -7, dtype=torch.int32).cuda()
        pos = torch.full((8,), -7, dtype=torch.int32).cuda()
        flags = torch.zeros(1, dtype=torch.int32).cuda()
        N.nvfp4kv_tree_masks(par, i32(qo), i32([20, 20]), tree_mask=mask, positions=pos,
                             device_flags=flags)
        assert int(flags) == _lib.FLAG_BAD_LENGTH
        assert [i for i in range(8) if int(pos[i]) != -7] == good


def test_stream_and_graph():
    rng = np.random.default_rng(3)
    trees = [T.random_parents(rng, n) for n in (9, 20)]
    par, qo = i32(trees[0] + trees[1]), i32([0, 9, 29])
    masks, positions = want(trees, [50, 20], 1)
    kv = i32([50, 20])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mask, pos = N.nvfp4kv_tree_masks(par, qo, kv, max_nodes=20, stream=side)
    side.synchronize()
    assert np.array_equal(mask.cpu().numpy(), masks) and pos.tolist() == positions
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.nvfp4kv_tree_masks(par, qo, kv, tree_mask=mask, positions=pos)
    kv += 7  # the graph reads the lengths anew
    graph.replay()
    torch.cuda.synchronize()
    assert pos.tolist() == [x + 7 for x in positions]
