"""The operators of a step that verifies drafted tokens, together as a server runs them: the
step's page table, masks and positions, normed and rotated heads, attention with the new
tokens' append, accepted tokens moved together, pages given up, requests forked."""
import math

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R
import test_gpu_tree_run as TR
import tree_reference as T

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE, LAYERS = 8, 2, 128, 16, 2


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Server:
    """Requests in the rows of a block table, over a pool whose unused slots are NaN.  What
    was accepted is kept beside it as the rows that were appended."""

    def __init__(self, rows, seed, pages=120, width=20):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.rows, self.lens = rows, [0] * rows
        self.layers = [T.Nvfp4Case((), PAGE, HKV, D, D, spare=pages, seed=seed + i, g=(0.8, 1.1))
                       for i in range(LAYERS)]
        self.table = torch.full((rows, width), -1, dtype=torch.int32).cuda()
        self.kv_len, self.shares = i32([0] * rows), i32([0] * pages)
        self.free, self.head = i32(self.rng.permutation(pages)), i32([0])
        self.step_table = N.StepTable.allocate(rows, 512, 200, slot_map=False)
        self.flags = torch.zeros(1, dtype=torch.int32).cuda()
        self.rope = N.nvfp4kv_rope_plan(D)
        self.weights = [[(1 + 0.1 * self.rand(D)) for _ in range(2)] for _ in range(LAYERS)]
        self.kept = [[[] for _ in range(rows)] for _ in range(LAYERS)]  # (K, V) row pairs

    def rand(self, *shape):
        return torch.randn(shape, generator=self.gen).to(torch.bfloat16).cuda()

    def draft(self, parents, paths):
        """The inputs of a step: `parents` and the accepted `paths` of every row's nodes."""
        new = [len(p) for p in parents]
        n, s = sum(new), dict(new=new, parents=parents, paths=paths)
        s["flat"] = i32([x for p in parents for x in p])
        s["qo_len"] = i32(new)
        s["path"] = torch.full((self.rows, max([1] + [len(p) for p in paths])), -1,
                               dtype=torch.int32)
        for b, p in enumerate(paths):
            s["path"][b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["path"], s["kept"] = s["path"].cuda(), i32([len(p) for p in paths])
        s["qkv"] = [(self.rand(n, HQ, D), self.rand(n, HKV, D), self.rand(n, HKV, D))
                    for _ in range(LAYERS)]
        lens = [a + b for a, b in zip(self.lens, new)]
        pages = [R.pages_of(a, PAGE) for a in lens]
        s["lens"] = lens
        s["plan"] = N.nvfp4kv_decode_plan(
            np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(pages)]),
            [a - (p - 1) * PAGE if p else 0 for a, p in zip(lens, pages)], HQ, HKV, D, D)
        return s

    def run(self, s):
        """What a server launches; nothing of it waits for the device."""
        t = self.step_table
        self.kv_len += s["qo_len"]
        N.nvfp4kv_build_page_table(self.kv_len, s["qo_len"], self.table, self.free, self.head, t,
                                   PAGE, device_flags=self.flags)
        s["mask"], s["pos"] = N.nvfp4kv_tree_masks(s["flat"], t.qo_indptr, self.kv_len,
                                                   max(s["new"]), device_flags=self.flags)
        s["out"] = []
        for c, (q, k, v), w in zip(self.layers, s["qkv"], self.weights):
            q, k = N.nvfp4kv_norm_rope(self.rope, q, k, s["pos"], *w)
            o, lse = N.nvfp4kv_tree_run(s["plan"], q, c.cache, t.kv_indices, s["mask"],
                                        new_k=k, new_v=v)
            s["out"].append((q, k, v, o, lse))
        return s

    def accept(self, s):
        t = self.step_table
        for c in self.layers:
            N.nvfp4kv_compact_tokens(c.cache, s["path"], s["kept"], t.qo_indptr, t.kv_indptr,
                                     t.kv_indices, t.last_page_len, device_flags=self.flags)
        keep = self.kv_len - s["qo_len"] + s["kept"]
        N.nvfp4kv_release_pages(keep, self.kv_len, self.table, self.shares, self.free,
                                t.free_head, self.head, PAGE, device_flags=self.flags)

    def note(self, s):
        at = 0
        for b, (n, path) in enumerate(zip(s["new"], s["paths"])):
            for layer, (_, k, v, _, _) in enumerate(s["out"]):
                self.kept[layer][b] += [(k[at + j].cpu(), v[at + j].cpu()) for j in path]
            self.lens[b] += len(path)
            at += n

    def check_attention(self, s):
        """Every row against 64 bits over the cache's bytes (before tokens are moved)."""
        torch.cuda.synchronize()
        t, at = self.step_table, 0
        assert N.nvfp4kv_workspace_flags(s["plan"]) == 0 and int(self.flags) == 0
        want = [T.ancestors(p) for p in s["parents"]]
        depth = [s["lens"][b] - s["new"][b] + len(a) - 1 for b, w in enumerate(want) for a in w]
        assert s["pos"].tolist() == depth
        indptr, ids = t.kv_indptr.cpu().numpy(), t.kv_indices.cpu().numpy()
        for c in self.layers:
            x = c.download()
            c.codes, c.sf = [x["k_data"], x["v_data"]], [x["k_sf"], x["v_sf"]]
            c.ids, c.indptr, c.kv = ids, indptr, s["lens"]
        for b, n in enumerate(s["new"]):
            rows = slice(at, at + n)
            at += n
            words = (max(s["new"]) + 31) // 32
            hide = TR.bits(T.mask_words(want[b], words), n, s["lens"][b])
            for c, (q, _, _, o, lse) in zip(self.layers, s["out"]):
                ref = T.tree_attention(R.to_np(q[rows]), c.dense(0, b), c.dense(1, b), hide,
                                       1 / math.sqrt(D))
                T.check_tree(R.to_np(o[rows]), R.to_np(lse[rows]), ref, D, torch.bfloat16)

    def check_bytes(self):
        """Each request's tokens hold what an append of the accepted rows in order holds."""
        torch.cuda.synchronize()
        assert int(self.flags) == 0 and self.kv_len.tolist() == self.lens
        table = self.table.cpu().numpy()
        for layer, c in enumerate(self.layers):
            have = c.download()
            for b, n in enumerate(self.lens):
                if not n:
                    continue
                fresh = T.Nvfp4Case((n,), PAGE, HKV, D, D, spare=0, g=(0.8, 1.1))
                k, v = (torch.stack([x[i] for x in self.kept[layer][b]]).cuda() for i in (0, 1))
                assert len(k) == n
                N.nvfp4kv_quantize_append(fresh.cache, k, v, i32([0] * n), i32(range(n)),
                                          fresh.kv_indices, fresh.kv_indptr, fresh.last_page_len)
                torch.cuda.synchronize()
                want, ids = fresh.download(), table[b, :R.pages_of(n, PAGE)]
                for name in want:
                    w, h = want[name][fresh.ids], have[name][ids]
                    for slot in range(n):
                        assert np.array_equal(w[slot // PAGE, :, slot % PAGE],
                                              h[slot // PAGE, :, slot % PAGE]), (layer, b, slot)

    def pages_are_owned_once(self):
        torch.cuda.synchronize()
        table, owners = self.table.cpu().numpy(), [0] * self.shares.numel()
        for b, n in enumerate(self.lens):
            for p in table[b, :R.pages_of(n, PAGE)]:
                owners[p] += 1
        free = self.free.tolist()[int(self.head):]
        assert self.shares.tolist() == [max(0, n - 1) for n in owners]
        assert sorted(free + [p for p, n in enumerate(owners) if n]) == list(range(len(owners)))

    def go(self, parents, paths):
        s = self.run(self.draft(parents, paths))
        self.check_attention(s)
        self.accept(s)
        self.note(s)

    def chains(self, lens):
        chains = [list(range(-1, n - 1)) for n in lens]
        return chains, [list(range(n)) for n in lens]

    def trees(self, most, rows=None):
        """Random trees and one accepted chain of each (none now and then)."""
        parents, paths = [], []
        for b in range(self.rows):
            n = int(self.rng.integers(1, most + 1)) if self.lens[b] else 0
            p = T.random_parents(self.rng, n)
            seen = T.ancestors(p)
            node = int(self.rng.integers(-1, n))
            parents.append(p)
            paths.append(sorted(seen[node]) if node >= 0 else [])
        return parents, paths


@pytest.mark.parametrize("most", [4, 9, 40])
def test_steps_with_forks(most):
    sv = Server(6, seed=most)
    sv.go(*sv.chains([40, 17, 5, 64, 0, 0]))
    sv.check_bytes()
    for _ in range(3):
        sv.go(*sv.trees(most))
    sv.check_bytes()
    sv.pages_are_owned_once()
    # two requests go on as two each
    src, dst = (torch.full((2,), -7, dtype=torch.int32).cuda() for _ in range(2))
    head = i32([0])
    N.nvfp4kv_fork_pages(i32([0, 3]), i32([5, 4]), sv.kv_len, sv.table, sv.shares, sv.free,
                         sv.head, head, src, dst, PAGE, device_flags=sv.flags)
    sv.head = head
    for c in sv.layers:
        N.nvfp4kv_copy_pages(c.cache, src, dst, device_flags=sv.flags)
    for a, b in ((0, 5), (3, 4)):
        sv.lens[b] = sv.lens[a]
        for kept in sv.kept:
            kept[b] = list(kept[a])
    sv.check_bytes()
    sv.pages_are_owned_once()
    for _ in range(3):
        sv.go(*sv.trees(most))
    sv.check_bytes()
    sv.pages_are_owned_once()
    # all of request 0 and of the fork of request 3 are given up
    N.nvfp4kv_release_pages(i32([0 if b in (0, 4) else n for b, n in enumerate(sv.lens)]),
                            sv.kv_len, sv.table, sv.shares, sv.free, sv.head, None, PAGE,
                            device_flags=sv.flags)
    sv.lens[0] = sv.lens[4] = 0
    for kept in sv.kept:
        kept[0], kept[4] = [], []
    sv.go(*sv.trees(most))
    sv.check_bytes()
    sv.pages_are_owned_once()


def test_a_captured_step():
    """The same step launched, and captured and replayed twice, from the same state."""
    sv = Server(4, seed=3)
    sv.go(*sv.chains([40, 17, 90, 64]))
    sv.go(*sv.trees(9))
    s = sv.draft(*sv.trees(9))
    state = [sv.table, sv.kv_len, sv.shares, sv.free, sv.head] + \
        [b for c in sv.layers for b in c.bufs.values()]
    before = [x.clone() for x in state]

    def restore():
        for x, y in zip(state, before):
            x.copy_(y)

    def results():
        torch.cuda.synchronize()
        return [x.clone() for x in state + [s["mask"], s["pos"]] +
                [y for o in s["out"] for y in o]]

    sv.run(s)
    sv.accept(s)
    want = results()
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.run(s)
        sv.accept(s)
    for _ in range(2):
        restore()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    assert N.nvfp4kv_workspace_flags(s["plan"]) == 0
    sv.note(s)
    sv.check_bytes()
    sv.pages_are_owned_once()
