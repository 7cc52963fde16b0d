"""Rows that forks may fill, and as many entries as a call of forks takes."""
import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
import test_gpu_page_sharing as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [8, 2100, 20000])  # one CTA, a cluster, two launches
@pytest.mark.parametrize("held", [1, 32, 33, -1])
def test_a_row_that_holds_a_request_is_not_filled(width, held):
    """A child's row must be empty: its pages would leave the pool for good.  Flagged, nothing
    else written, also where it holds as many tokens as the parent (33)."""
    b = P.Both((33, 16, held if held > 0 else 0), 8, width=width)
    if held < 0:
        b.kv_len[2] = b.ref.kv_len[2] = held
    src, dst = b.fork([0, 1], [5, 2], check=False)
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_BAD_LENGTH
    b.head, b.head2 = b.head2, b.head
    b.flags.zero_()
    b.same()
    assert int(b.head2) == -1 and set(src.tolist() + dst.tolist()) == {-7}
    if held > 0:  # given up first, the row may be filled
        b.release([33, 16] + [0] * 6)
        b.fork([0, 1], [5, 2])
        b.same()


def test_as_many_entries_as_a_call_takes():
    """2^31 - 1 whole pages in one call (8192 forks of 262144 and 262143 pages): entries that
    the last warp's lanes would number past that are none."""
    n, forks = 262144, 8192
    table = torch.full((forks + 2, n), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(n, dtype=torch.int32, device="cuda")
    table[1, :n - 1] = torch.arange(n, 2 * n - 1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kv_len = i32([n, n - 1] + [0] * forks)
    parents, children = i32([0] * (forks - 1) + [1]), i32(list(range(2, forks + 2)))
    shares, free = torch.zeros(2 * n - 1, dtype=torch.int32, device="cuda"), i32([7])
    head, out, flags = i32([0]), i32([-1]), i32([0])
    src, dst = (torch.full((forks,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    N.nvfp4kv_fork_pages(parents, children, kv_len, table, shares, free, head, out, src, dst,
                         page_size=1, device_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0 and int(out) == 0 and free.tolist() == [7]
    assert (src == -1).all() and (dst == -1).all()
    assert kv_len.tolist() == [n, n - 1] + [n] * (forks - 1) + [n - 1]
    for r in range(2, forks + 1, 1024):
        assert (table[r:min(r + 1024, forks + 1)] == table[0]).all()
    assert torch.equal(table[forks + 1], table[1]) and int(table[1, n - 1]) == -1
    assert (shares[:n] == forks - 1).all() and (shares[n:] == 1).all()
    # one more entry is too many
    kv_len[2:] = 0
    kv_len[1] = n
    before = shares.clone()
    N.nvfp4kv_fork_pages(parents, children, kv_len, table, shares, free, head, out, src, dst,
                         page_size=1, device_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == _lib.FLAG_TABLE_FULL and not kv_len[2:].any()
    assert torch.equal(shares, before)


@pytest.mark.parametrize("width", [8, 2100, 20000])
def test_forks_in_a_graph_before_and_behind_calls_that_use_their_lengths(width):
    """Lengths written just before a fork, read just behind it: launched, and replayed."""
    b = P.Both((33, 50), 6, width=width)
    par, child = P.i32([0, 1, 0]), P.i32([2, 3, 4])
    src, dst = (torch.full((3,), -7, dtype=torch.int32).cuda() for _ in range(2))
    mid, seen = P.i32([0]), torch.zeros_like(b.kv_len)

    def step():
        b.kv_len[:2] += 7
        b.kv_len[:2] -= 7
        N.nvfp4kv_fork_pages(par, child, b.kv_len, b.table, b.shares, b.free, b.head, mid, src,
                             dst, device_flags=b.flags)
        seen.copy_(b.kv_len)
        N.nvfp4kv_release_pages(b.kv_len * keep, b.kv_len, b.table, b.shares, b.free, mid, b.head,
                                device_flags=b.flags)

    keep = P.i32([1, 1, 0, 0, 0, 0])
    step()
    graph = torch.cuda.CUDAGraph()
    for replay in range(4):
        copies = b.ref.fork([0, 1, 0], [2, 3, 4])
        b.ref.release([33, 50, 0, 0, 0, 0])
        b.same()
        assert seen.tolist() == [33, 50, 33, 50, 33, 0]
        assert list(zip(src.tolist(), dst.tolist())) == copies
        seen.zero_()
        if replay == 0:
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        torch.cuda.synchronize()


@pytest.mark.parametrize("width", [300, 2100])
@pytest.mark.parametrize("seed", [0, 1])
def test_many_steps_in_wide_tables(seed, width):
    """As test_many_steps, over tables whose forks take a cluster, or two launches (from 16
    forks on)."""
    rng = np.random.default_rng(seed)
    kv = [int(x) for x in rng.integers(0, 300 * 16, 20)]
    b = P.Both(kv, 60, 16, seed=seed, spare=400, width=width)
    for _ in range(6):
        rows = rng.permutation(60).tolist()
        empty = [r for r in rows if b.ref.kv_len[r] == 0]
        some = [r for r in rows if b.ref.kv_len[r] > 0]
        n = min(len(empty), int(rng.integers(1, 30)))
        if n and some:
            b.fork([some[int(rng.integers(0, len(some)))] for _ in range(n)], empty[:n])
            b.same()
        keep = list(b.ref.kv_len)
        for r in rows[:40]:
            keep[r] = int(rng.integers(0, keep[r] + 1)) if rng.random() < 0.4 else 0
        b.release(keep, out=bool(rng.integers(0, 2)))
        b.same()
    b.release([0] * 60)
    b.same()
    assert sorted(b.ref.free[b.ref.head:]) == list(range(b.total)) and not any(b.ref.shares)
