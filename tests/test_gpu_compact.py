"""Accepted tokens moved together in their pages, 4-bit and E4M3 cache, byte for byte."""
import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
import step_reference as R
import tree_reference as T

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def padded(paths, width=None, fill=-1):
    width = width or max(1, max(len(p) for p in paths))
    return i32([list(p) + [fill] * (width - len(p)) for p in paths])


class E4m3Case:
    def __init__(self, kv, page, hkv, dk, dv, layout="HND", seed=0, spare=2):
        rng = np.random.default_rng(seed)
        npages = [R.pages_of(n, page) for n in kv]
        self.kv, self.page, self.total = list(kv), page, sum(npages) + spare
        self.indptr = np.concatenate([[0], np.cumsum(npages)]).astype(np.int32)
        self.ids = rng.permutation(self.total)[:sum(npages)].astype(np.int32)
        self.last = [n - (m - 1) * page if m else 0 for n, m in zip(kv, npages)]
        # every code, NaN among them; scales that differ by up to 2^20
        self.codes = [rng.integers(0, 256, (self.total, hkv, page, d), dtype=np.uint8)
                      for d in (dk, dv)]
        self.scale = [np.exp2(rng.integers(-12, 9, (self.total, hkv))).astype(np.float32)
                      for _ in range(2)]
        data = [torch.from_numpy(x.copy() if layout == "HND" else
                                 np.ascontiguousarray(x.transpose(0, 2, 1, 3))).cuda()
                for x in self.codes]
        if layout == "NHD":
            data = [x.transpose(1, 2) for x in data]
        self.cache = N.E4m3Cache(*data, *(torch.from_numpy(s.copy()).cuda() for s in self.scale))
        self.kv_indices, self.kv_indptr = i32(self.ids), i32(self.indptr)
        self.last_page_len = i32(self.last)

    def pages(self, b):
        return self.ids[self.indptr[b]:self.indptr[b + 1]]

    def move(self, b, begin, path):
        """The definition, on self.codes and self.scale."""
        page, pages = self.page, self.pages(b)
        for codes, scale in zip(self.codes, self.scale):
            old_codes, old_scale = codes.copy(), scale.copy()
            for at in range(begin // page, R.pages_of(begin + len(path), page) if path else 0):
                target = pages[at]
                own = range(at * page, begin)  # tokens that stay
                src = [(i, begin + n) for i, n in enumerate(path)
                       if (begin + i) // page == at]
                for h in range(codes.shape[1]):
                    had = [old_scale[pages[s // page], h] for _, s in src]
                    now = max(had + ([old_scale[target, h]] if len(own) else []))
                    def put(slot, row, was):
                        codes[target, h, slot] = row if was == now else R.e4m3_codes(
                            R.VALUES[row] * float(np.float32(was / now)))
                    for t in own:
                        put(t % page, old_codes[target, h, t % page], old_scale[target, h])
                    for (i, s), was in zip(src, had):
                        put((begin + i) % page, old_codes[pages[s // page], h, s % page], was)
                    scale[target, h] = now

    def check(self):
        for got, want in ((self.cache.k_data, self.codes[0]), (self.cache.v_data, self.codes[1])):
            got = got.cpu().contiguous().numpy()
            nan = (want & 0x7F) == 0x7F  # a NaN that is coded anew keeps no sign
            assert np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
        for got, want in ((self.cache.k_scale, self.scale[0]), (self.cache.v_scale, self.scale[1])):
            assert np.array_equal(got.cpu().numpy(), want)


def paths_for(rng, new, most):
    out = []
    for n in new:
        c = int(rng.integers(0, min(n, most) + 1))
        out.append(sorted(rng.choice(n, c, replace=False).tolist()))
    return out


SHAPES = [((37, 300, 16, 5, 64), (5, 33, 16, 5, 0)), ((70, 40), (64, 40)), ((1, 17), (1, 2))]


@pytest.mark.parametrize("kv,new", SHAPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (512, 256), (64, 32), (32, 256)])
@pytest.mark.parametrize("page,layout,pad", [(16, "HND", 0), (16, "NHD", 48), (1, "HND", 0)])
def test_nvfp4(kv, new, dk, dv, page, layout, pad):
    rng = np.random.default_rng(dk + sum(new))
    c = T.Nvfp4Case(kv, page, 3, dk, dv, layout, seed=dk, pad=pad)
    paths = paths_for(rng, new, 64)
    qo = np.concatenate([[0], np.cumsum(new)])
    want = c.download()
    want = {n: x.copy() for n, x in want.items()}
    for b, path in enumerate(paths):
        todo = T.moved(c.pages(b), page, kv[b] - new[b], path)
        rows = {n: [x[sp, :, ss].copy() for _, _, sp, ss in todo] for n, x in want.items()}
        for n, x in want.items():
            for (tp, ts, _, _), row in zip(todo, rows[n]):
                x[tp, :, ts] = row
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    N.nvfp4kv_compact_tokens(c.cache, padded(paths), i32([len(p) for p in paths]), i32(qo),
                             c.kv_indptr, c.kv_indices, c.last_page_len, device_flags=flags)
    got = c.download()
    assert int(flags) == 0
    for n in want:
        assert np.array_equal(got[n], want[n]), n


@pytest.mark.parametrize("kv,new", SHAPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (512, 256), (96, 32)])
@pytest.mark.parametrize("page,layout", [(16, "HND"), (16, "NHD"), (1, "HND")])
def test_e4m3(kv, new, dk, dv, page, layout):
    rng = np.random.default_rng(dk + sum(new))
    c = E4m3Case(kv, page, 3, dk, dv, layout, seed=dk)
    paths = paths_for(rng, new, 64)
    qo = np.concatenate([[0], np.cumsum(new)])
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    N.nvfp4kv_e4m3_compact_tokens(c.cache, padded(paths, 70), i32([len(p) for p in paths]),
                                  i32(qo), c.kv_indptr, c.kv_indices, c.last_page_len,
                                  device_flags=flags)
    for b, path in enumerate(paths):
        c.move(b, kv[b] - new[b], path)
    assert int(flags) == 0
    c.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("path", [[300], list(range(1, 400)), list(range(0, 400, 2)),
                                  list(range(400)), [0], [0, 1, 2, 399]])
def test_long_paths(e4m3, path):
    """400 drafted tokens over 26 pages: every step of a chain, of every second one."""
    kv, new = (411, 30), (400, 3)
    c = (E4m3Case if e4m3 else T.Nvfp4Case)(kv, 16, 2, 128, 64, seed=len(path))
    paths = [path, [1]]
    call = N.nvfp4kv_e4m3_compact_tokens if e4m3 else N.nvfp4kv_compact_tokens
    if not e4m3:
        want = {n: x.copy() for n, x in c.download().items()}
        for b, p in enumerate(paths):
            todo = T.moved(c.pages(b), 16, kv[b] - new[b], p)
            rows = {n: [x[sp, :, ss].copy() for _, _, sp, ss in todo] for n, x in want.items()}
            for n, x in want.items():
                for (tp, ts, _, _), row in zip(todo, rows[n]):
                    x[tp, :, ts] = row
    call(c.cache, padded(paths), i32([len(p) for p in paths]), i32([0, 400, 403]), c.kv_indptr,
         c.kv_indices, c.last_page_len)
    if e4m3:
        for b, p in enumerate(paths):
            c.move(b, kv[b] - new[b], p)
        c.check()
    else:
        got = c.download()
        assert all(np.array_equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_paths_that_cannot_be(e4m3):
    """Nodes out of order, twice, out of the tree; counts past the path, the tree or below 0:
    that request alone is left as it is."""
    kv, new = (50,) * 8, (10,) * 8
    c = (E4m3Case if e4m3 else T.Nvfp4Case)(kv, 16, 2, 64, 64, seed=1)
    paths = [[3, 2], [4, 4], [9, 10], [-1, 3], [1, 2, 5], [2, 3], [2, 3], [1, 9]]
    kept = [2, 2, 2, 2, 4, -1, 11, 2]  # (the fifth row has three entries)
    call = N.nvfp4kv_e4m3_compact_tokens if e4m3 else N.nvfp4kv_compact_tokens
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    if not e4m3:
        want = {n: x.copy() for n, x in c.download().items()}
    call(c.cache, padded(paths), i32(kept), i32(np.arange(9) * 10), c.kv_indptr, c.kv_indices,
         c.last_page_len, device_flags=flags)
    assert int(flags) == _lib.FLAG_BAD_APPEND_TARGET
    if e4m3:
        c.move(7, 40, [1, 9])
        c.check()
    else:
        for tp, ts, sp, ss in T.moved(c.pages(7), 16, 40, [1, 9]):
            for x in want.values():
                x[tp, :, ts] = x[sp, :, ss]
        got = c.download()
        assert all(np.array_equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_page_ids(e4m3):
    """An id out of the pool: flagged, its tokens left; the other requests are served."""
    kv, new = (40, 40), (20, 20)
    c = (E4m3Case if e4m3 else T.Nvfp4Case)(kv, 16, 2, 64, 64, seed=2)
    idx = c.kv_indices.clone()
    idx[1] = c.total + 3  # page 1 of request 0: the first target
    path = [5, 6]
    call = N.nvfp4kv_e4m3_compact_tokens if e4m3 else N.nvfp4kv_compact_tokens
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    want = None if e4m3 else {n: x.copy() for n, x in c.download().items()}
    call(c.cache, padded([path, path]), i32([2, 2]), i32([0, 20, 40]), c.kv_indptr, idx,
         c.last_page_len, device_flags=flags)
    assert int(flags) == _lib.FLAG_BAD_PAGE_INDEX
    if e4m3:
        c.move(1, 20, path)
        c.check()
    else:
        for tp, ts, sp, ss in T.moved(c.pages(1), 16, 20, path):
            for x in want.values():
                x[tp, :, ts] = x[sp, :, ss]
        got = c.download()
        assert all(np.array_equal(got[n], want[n]) for n in want)


def test_scales_out_of_range_and_not_powers_of_two():
    c = E4m3Case((40,), 16, 1, 64, 64, seed=3)
    pages = c.pages(0)
    for s in c.scale:
        s[pages[1], 0], s[pages[2], 0] = 0.3, 0.7
    c.cache.k_scale.copy_(torch.from_numpy(c.scale[0]))
    c.cache.v_scale.copy_(torch.from_numpy(c.scale[1]))
    args = (i32([0, 20]), c.kv_indptr, c.kv_indices, c.last_page_len)
    flags = torch.zeros(1, dtype=torch.int32).cuda()
    N.nvfp4kv_e4m3_compact_tokens(c.cache, i32([[3, 15]]), i32([2]), *args, device_flags=flags)
    c.move(0, 20, [3, 15])
    assert int(flags) == 0
    c.check()
    c.cache.k_scale[int(pages[2])] = float("inf")
    N.nvfp4kv_e4m3_compact_tokens(c.cache, i32([[3, 15]]), i32([2]), *args, device_flags=flags)
    assert int(flags) == _lib.FLAG_BAD_SCALE
    assert float(c.cache.k_scale[int(pages[1])]) == 2.0 ** 64


@pytest.mark.parametrize("e4m3", [False, True])
def test_graph_and_stream(e4m3):
    kv, new = (50, 90), (20, 30)
    rng = np.random.default_rng(4)
    paths = paths_for(rng, new, 20)
    call = N.nvfp4kv_e4m3_compact_tokens if e4m3 else N.nvfp4kv_compact_tokens
    made = [(E4m3Case if e4m3 else T.Nvfp4Case)(kv, 16, 2, 128, 128, seed=5) for _ in range(3)]
    lists = padded(paths), i32([len(p) for p in paths]), i32([0, 20, 50])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b, c = made
    call(a.cache, *lists, a.kv_indptr, a.kv_indices, a.last_page_len)
    call(b.cache, *lists, b.kv_indptr, b.kv_indices, b.last_page_len, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c.cache, *lists, c.kv_indptr, c.kv_indices, c.last_page_len)
    graph.replay()
    torch.cuda.synchronize()
    for other in (b, c):
        assert torch.equal(a.cache.k_data, other.cache.k_data)
        assert torch.equal(a.cache.v_data, other.cache.v_data)
