"""Forked requests, copied pages and pages given up, against lists."""
import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
from nvfp4_paged_kv_nvfp4kv_gb300 import workloads as W
import step_reference as R
import tree_reference as T

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Both:
    """The same pool on the device and in lists."""

    def __init__(self, kv, rows, page=16, seed=0, spare=200, width=None, stride=None):
        rng = np.random.default_rng(seed)
        npages = [R.pages_of(n, page) for n in kv]
        self.width = width or max(npages + [0]) + 2
        total = sum(npages) + spare
        ids = rng.permutation(total).tolist()
        table, at = [], 0
        for n in npages + [0] * (rows - len(kv)):
            table.append(ids[at:at + n] + [-1] * (self.width - n))
            at += n
        self.lead = at + 5  # entries in front of the head: the pages in use came from there
        free = [-9] * self.lead + ids[at:]
        self.ref = T.Pool(table, list(kv) + [0] * (rows - len(kv)), [0] * total, free, self.lead,
                          page)
        self.page, self.total = page, total
        wide = torch.full((rows, stride or self.width), -3, dtype=torch.int32).cuda()
        self.table = wide[:, :self.width]
        self.table.copy_(i32(table).view(rows, self.width))
        self.wide = wide
        self.kv_len, self.shares = i32(self.ref.kv_len), i32(self.ref.shares)
        self.free, self.head, self.head2 = i32(free), i32([self.lead]), i32([-1])
        self.flags = torch.zeros(1, dtype=torch.int32).cuda()

    def fork(self, parents, children, check=True, **kw):
        src, dst = (torch.full((len(parents),), -7, dtype=torch.int32).cuda() for _ in range(2))
        N.nvfp4kv_fork_pages(i32(parents), i32(children), self.kv_len, self.table, self.shares,
                             self.free, self.head, self.head2, src, dst, page_size=self.page,
                             device_flags=self.flags, **kw)
        self.head, self.head2 = self.head2, self.head
        if check:
            want = self.ref.fork(parents, children)
            torch.cuda.synchronize()
            assert list(zip(src.tolist(), dst.tolist())) == want
        return src, dst

    def release(self, keep, out=False, check=True, **kw):
        N.nvfp4kv_release_pages(i32(keep), self.kv_len, self.table, self.shares, self.free,
                                self.head, self.head2 if out else None, page_size=self.page,
                                device_flags=self.flags, **kw)
        if out:
            self.head, self.head2 = self.head2, self.head
        if check:
            self.ref.release(keep)

    def same(self):
        torch.cuda.synchronize()
        r = self.ref
        assert int(self.flags) == 0
        assert self.kv_len.tolist() == r.kv_len and self.shares.tolist() == r.shares
        assert int(self.head) == r.head and self.free.tolist() == r.free
        assert self.table.tolist() == r.table
        assert (self.wide[:, self.width:] == -3).all()


@pytest.mark.parametrize("page", [16, 1, 7])
@pytest.mark.parametrize("kv,parents", [
    ((33, 16, 0, 5), [0, 1, 2, 3]), ((40,), [0] * 9), ((16, 32), [1, 0, 1]),
    ((1000, 1, 48, 700), [3, 3, 0, 2, 1, 0]), ((5,), [])])
def test_fork_and_release(kv, parents, page):
    rows = len(kv) + len(parents) + 2
    b = Both(kv, rows, page, seed=len(parents), stride=1500)
    children = list(range(len(kv), len(kv) + len(parents)))[::-1]
    b.fork(parents, children)
    b.same()
    # the parents go first: their whole pages stay with the children
    keep = [0] * len(kv) + b.ref.kv_len[len(kv):]
    b.release(keep, out=True)
    b.same()
    b.release([n // 2 for n in b.ref.kv_len])  # the children are cut in half, at once
    b.same()
    b.release([0] * rows)
    b.same()
    assert b.ref.head == 5 and sorted(b.ref.free[5:]) == list(range(b.total))


@pytest.mark.parametrize("seed", range(6))
def test_many_steps(seed):
    """Forks of forks, cuts and ends in any order; the pool comes back whole."""
    rng = np.random.default_rng(seed)
    kv = [int(x) for x in rng.integers(0, 400, 20)]
    b = Both(kv, 60, 16, seed=seed, spare=400)
    for _ in range(12):
        rows = rng.permutation(60).tolist()
        empty = [r for r in rows if b.ref.kv_len[r] == 0]
        some = [r for r in rows if b.ref.kv_len[r] > 0]
        n = int(rng.integers(0, min(len(empty), 12) + 1))
        if n and some:
            b.fork([some[int(rng.integers(0, len(some)))] for _ in range(n)], empty[:n])
        keep = list(b.ref.kv_len)
        for r in rows[:int(rng.integers(0, 25))]:
            keep[r] = int(rng.integers(0, keep[r] + 1)) if rng.random() < 0.6 else 0
        b.release(keep, out=bool(rng.integers(0, 2)))
        b.same()
    b.release([0] * 60)
    b.same()
    assert sorted(b.ref.free[b.ref.head:]) == list(range(b.total)) and not any(b.ref.shares)


def test_many_entries():
    """More entries than the warps keep in registers, and rows of very unequal lengths."""
    b = Both([60000, 3, 0, 30000], 300, 1, seed=1, spare=10)
    b.fork([0, 3, 0, 1], [4, 299, 6, 7])
    # a faster count than the lists' for so many pages
    b.ref.table, b.ref.kv_len = b.table.tolist(), b.kv_len.tolist()
    b.same()
    keep = [0] * 300
    keep[299], keep[0] = 100, 59000
    table, kv = np.array(b.ref.table), list(b.ref.kv_len)
    shares = np.array(b.ref.shares)
    b.release(keep, check=False)
    entries = np.concatenate([table[r, k:n] for r, (k, n) in enumerate(zip(keep, kv))])
    drops = np.bincount(entries, minlength=b.total)
    first = np.full(b.total, -1)
    first[entries[::-1]] = np.arange(len(entries))[::-1]
    freed = entries[(first[entries] == np.arange(len(entries))) & (drops > shares)[entries]]
    torch.cuda.synchronize()
    assert int(b.flags) == 0 and b.kv_len.tolist() == keep
    assert b.shares.tolist() == np.maximum(shares - drops, 0).tolist()
    assert int(b.head) == b.ref.head - len(freed)
    assert b.free[int(b.head):b.ref.head].tolist() == freed.tolist()


@pytest.mark.parametrize("parents,children", [
    ([0, 1], [5, 5]), ([0, 5], [5, 6]), ([0], [0]), ([0], [8]), ([8], [5]), ([-1], [5]),
    ([0], [-1])])
def test_forks_that_cannot_be(parents, children):
    """A row filled twice, filled and read, out of range: flagged, nothing else written."""
    b = Both((33, 16), 8)
    src, dst = b.fork(parents, children, check=False)
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_BAD_LENGTH
    b.head, b.head2 = b.head2, b.head
    b.flags.zero_()
    b.same()
    assert int(b.head2) == -1 and set(src.tolist() + dst.tolist()) == {-7}


@pytest.mark.parametrize("width", [8, 1000, 20000])  # one CTA, a cluster, three launches
def test_lengths_that_cannot_be(width):
    for length in (-1, 2**30 + 1, 16 * width + 1):
        b = Both((33, 16), 8, width=width)
        b.kv_len[0] = b.ref.kv_len[0] = length
        b.fork([0], [5], check=False)
        torch.cuda.synchronize()
        assert int(b.flags) == _lib.FLAG_BAD_LENGTH
        b.head, b.head2 = b.head2, b.head
        b.flags.zero_()
        b.same()
        b.release([0] * 8, check=False)
        torch.cuda.synchronize()
        assert int(b.flags) == _lib.FLAG_BAD_LENGTH
        b.flags.zero_()
        b.same()
    for keep in ([34, 0, 0, 0, 0, 0, 0, 0], [-1, 0, 0, 0, 0, 0, 0, 0]):
        b = Both((33, 16), 8, width=width)
        b.release(keep, check=False)
        torch.cuda.synchronize()
        assert int(b.flags) == _lib.FLAG_BAD_LENGTH
        b.flags.zero_()
        b.same()


@pytest.mark.parametrize("width", [8, 1000, 20000])  # one CTA, a cluster, three launches
def test_free_lists_that_are_too_short(width):
    b = Both((33, 5, 16), 8, spare=1, width=width)
    b.fork([0, 1], [5, 6], check=False)  # two new pages, one left
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_TABLE_FULL
    b.head, b.head2 = b.head2, b.head
    b.flags.zero_()
    b.same()
    b.fork([0, 2], [5, 6])  # one new page
    b.same()
    for head in (2, 0):  # the head stands in front of fewer places than pages are freed
        b.head.fill_(head)
        b.release([0] * 8, check=False)
        torch.cuda.synchronize()
        assert int(b.flags) == _lib.FLAG_TABLE_FULL and int(b.head) == head
        b.flags.zero_()
        b.head.fill_(b.ref.head)
        b.same()
    for head in (-1, 10**6):
        b.head.fill_(head)
        b.release([0] * 8, check=False)
        torch.cuda.synchronize()
        assert int(b.flags) == _lib.FLAG_TABLE_FULL
        b.flags.zero_()
        b.head.fill_(b.ref.head)
        b.same()


@pytest.mark.parametrize("width", [8, 1000, 20000])  # one CTA, a cluster, three launches
def test_page_ids_out_of_the_pool(width):
    """Passed on by a fork and passed over by a release, flagged both times."""
    b = Both((40, 20), 6, width=width)
    b.table[0, 1] = b.ref.table[0][1] = b.total
    src, dst = b.fork([0], [3], check=False)
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_BAD_PAGE_INDEX
    assert b.table[3, :3].tolist() == [b.ref.table[0][0], b.total, int(dst[0])]
    b.flags.zero_()
    b.release([0, 20, 0, 40, 0, 0], check=False)
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_BAD_PAGE_INDEX
    assert int(b.head) == b.lead and int(b.free[b.lead]) == b.ref.table[0][2]
    assert not b.shares.any()


@pytest.mark.parametrize("width", [8, 1000, 20000])  # one CTA, a cluster, three launches
def test_a_page_given_up_too_often(width):
    """A page in two rows whose owners were not counted: freed once, flagged."""
    b = Both((16, 32), 4, width=width)
    b.table[2, 0] = b.table[0, 0]
    b.kv_len[2] = 16
    page = b.ref.table[0][0]
    b.release([0, 32, 0, 0], check=False)
    torch.cuda.synchronize()
    assert int(b.flags) == _lib.FLAG_BAD_SHARES
    assert int(b.head) == b.lead - 1 and int(b.free[b.lead - 1]) == page and not b.shares.any()


def pool(e4m3, pages, hkv, dk, dv, page, layout, seed):
    g = torch.Generator().manual_seed(seed)
    if e4m3:
        c = N.E4m3Cache.allocate(pages, hkv, dk, dv, page, layout)
        for t in (c.k_data, c.v_data):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.rand(t.shape, generator=g))
        return c, [c.k_data, c.v_data, c.k_scale, c.v_scale]
    lay = W.CacheLayout(layout, pages, page, hkv, dk, dv, pad_page_bytes=240)
    c = N.PagedCache.allocate(lay)
    bufs = [c.k_data, c.v_data, c.k_sf, c.v_sf]
    for t in bufs:
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    return c, [b.view(pages, -1)[:, :b.numel() // pages - 240] for b in bufs]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dk,dv,hkv", [(64, 64, 1), (128, 128, 8), (512, 256, 2), (32, 64, 3)])
@pytest.mark.parametrize("page,layout", [(16, "HND"), (16, "NHD"), (1, "HND")])
def test_copies(e4m3, dk, dv, hkv, page, layout):
    c, bufs = pool(e4m3, 12, hkv, dk, dv, page, layout, dk)
    want = [b.clone() for b in bufs]
    # a pair of its own, one to pass over, one source twice, a page to itself, bad ids
    src, dst = [3, -1, 5, 5, 7, 12, 2, -2, 1], [0, -1, 4, 6, 7, 8, -1, 9, 12]
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    call = N.nvfp4kv_e4m3_copy_pages if e4m3 else N.nvfp4kv_copy_pages
    call(c, i32(src[:5]), i32(dst[:5]), device_flags=flags)
    for w in want:
        w[[0, 4, 6]] = w[[3, 5, 5]].clone()
    torch.cuda.synchronize()
    assert int(flags) == 0 and all(torch.equal(a, b) for a, b in zip(bufs, want))
    call(c, i32(src), i32(dst), device_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == _lib.FLAG_BAD_PAGE_INDEX
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))


def test_graph_and_stream():
    """The three calls captured once and replayed: a continuation tried and given up again."""
    b = Both((33, 50), 6)
    c, bufs = pool(False, b.total, 2, 64, 64, 16, "HND", 1)
    par, child, keep = i32([0, 1, 0]), i32([2, 3, 4]), i32([33, 50, 0, 0, 0, 0])
    src, dst = (torch.full((3,), -7, dtype=torch.int32).cuda() for _ in range(2))
    mid = i32([0])

    def step(stream=None):
        N.nvfp4kv_fork_pages(par, child, b.kv_len, b.table, b.shares, b.free, b.head, mid, src,
                             dst, stream=stream)
        N.nvfp4kv_copy_pages(c, src, dst, stream=stream)
        N.nvfp4kv_release_pages(keep, b.kv_len, b.table, b.shares, b.free, mid, b.head,
                                stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    copies = b.ref.fork([0, 1, 0], [2, 3, 4])
    b.ref.release(keep.tolist())
    b.same()
    assert list(zip(src.tolist(), dst.tolist())) == copies
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        copies = b.ref.fork([0, 1, 0], [2, 3, 4])
        b.ref.release(keep.tolist())
        b.same()
        assert list(zip(src.tolist(), dst.tolist())) == copies
        for s, d in copies:
            assert all(torch.equal(x[s], x[d]) for x in bufs)


def test_more_entries_than_marks():
    """Nine million pages given up at once, every third of them shared: past the marks that
    the CTAs keep."""
    n = 9_000_000
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    shares = (torch.arange(n, dtype=torch.int32) % 3 == 0).int().cuda()
    kv_len, flags = i32([n, 0]), torch.zeros(1, dtype=torch.int32).cuda()
    free, head = torch.full((n + 4,), -1, dtype=torch.int32).cuda(), i32([n + 1])
    table = torch.stack([ids, torch.full_like(ids, -1)])
    want = ids[shares[ids.long()] == 0]
    N.nvfp4kv_release_pages(i32([5, 0]), kv_len, table, shares, free, head, page_size=1,
                            device_flags=flags)
    torch.cuda.synchronize()
    kept = ids[:5].long()
    want = want[(want[:, None] != kept[None, :].int()).all(1)]
    assert int(flags) == 0 and kv_len.tolist() == [5, 0]
    assert int(head) == n + 1 - want.numel()
    assert torch.equal(free[int(head):n + 1], want) and int(free[int(head) - 1]) == -1
    left = torch.zeros_like(shares)
    left[kept] = (kept % 3 == 0).int()
    assert torch.equal(shares, left)
