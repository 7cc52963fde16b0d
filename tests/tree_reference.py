"""64-bit references of the operators of a step that verifies drafted tokens (norms with
rotary positions, tree masks, tree attention over the 4-bit cache, accepted tokens moved
together, pages with several owners), written from their definitions in plain Python and
numpy."""
from __future__ import annotations

import math

import numpy as np
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


# ---- norms with rotary positions -------------------------------------------------
def norm(x, weight, offset, eps):
    """The heads of x [tokens, heads, dim] normed, in 64 bits."""
    x = x.detach().double().cpu()
    size = x.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    y = x / size  # (squares of the largest values pass float32's range, not float64's)
    mean = (y * y).mean(-1, keepdim=True) + eps / size / size
    return y / mean.sqrt() * (weight.detach().double().cpu() + offset)


# ---- drafted trees -----------------------------------------------------------------
def ancestors(parents):
    """The set of nodes that each node of one tree sees."""
    seen = []
    for i, p in enumerate(parents):
        seen.append({i} | (seen[p] if 0 <= p < i else set()))
    return seen


def mask_words(sets, words):
    out = np.zeros((len(sets), words), dtype=np.int64)
    for i, s in enumerate(sets):
        for j in s:
            out[i, j >> 5] |= 1 << (j & 31)
    return out.astype(np.uint32).view(np.int32)


def random_parents(rng, n, deep=False):
    """A tree of n nodes: each hangs below one before it (deep: mostly the last one)."""
    return [-1 if i == 0 else (i - 1 if deep and rng.random() < 0.9 else int(rng.integers(-1, i)))
            for i in range(n)]


# ---- the 4-bit cache -----------------------------------------------------------------
class Nvfp4Case:
    """Requests of given lengths in a shuffled pool of random codes and scales; `stale`
    slots (past every length, and pages of no request) hold NaN scales."""

    def __init__(self, kv, page, hkv, dk, dv, layout="HND", seed=0, spare=3, stale=True,
                 pad=0, g=(0.75, 1.25)):
        rng = np.random.default_rng(seed)
        self.kv, self.page, self.hkv, self.dims, self.g = list(kv), page, hkv, (dk, dv), g
        npages = [R.pages_of(n, page) for n in kv]
        self.total = sum(npages) + spare
        ids = rng.permutation(self.total)
        self.indptr = np.concatenate([[0], np.cumsum(npages)]).astype(np.int32)
        self.ids = ids[:sum(npages)].astype(np.int32)
        self.unused = ids[sum(npages):].astype(np.int32)
        self.last = [n - (m - 1) * page if m else 0 for n, m in zip(kv, npages)]
        self.codes = [rng.integers(0, 256, (self.total, hkv, page, d // 2), dtype=np.uint8)
                      for d in (dk, dv)]
        # scales near a quarter, so that values are near 1
        self.sf = [rng.integers(0x24, 0x34, (self.total, hkv, page, d // 16), dtype=np.uint8)
                   for d in (dk, dv)]
        if stale:
            for sf in self.sf:
                for p in self.unused:
                    sf[p] = 0x7F
                for b, n in enumerate(self.kv):
                    if n and n % page:
                        sf[self.pages(b)[-1], :, n % page:] = 0x7F
        self.layout, self.pad = layout, pad
        self.upload()

    def pages(self, b):
        return self.ids[self.indptr[b]:self.indptr[b + 1]]

    def upload(self):
        bufs, strides = [], {}
        for name, x in (("k_data", self.codes[0]), ("v_data", self.codes[1]),
                        ("k_sf", self.sf[0]), ("v_sf", self.sf[1])):
            p, h, s, r = x.shape
            y = x if self.layout == "HND" else x.transpose(0, 2, 1, 3)
            y = y.reshape(p, -1)
            page = y.shape[1] + self.pad
            buf = np.full((p, page), 0xA5, dtype=np.uint8)
            buf[:, :y.shape[1]] = y
            bufs.append(torch.from_numpy(buf).cuda())
            strides[name] = ((page, r, s * r) if self.layout == "HND" else (page, h * r, r))
        self.bufs = dict(zip(("k_data", "v_data", "k_sf", "v_sf"), bufs))
        self.cache = N.PagedCache(*bufs, strides, self.total, self.hkv, *self.dims, *self.g,
                                  self.page)
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        self.kv_indices, self.kv_indptr = i32(self.ids), i32(self.indptr)
        self.last_page_len = i32(self.last)

    def download(self):
        """(codes, scales) of K and V as the device holds them, [pages, heads, slots, row]."""
        out = {}
        for name, like in (("k_data", self.codes[0]), ("v_data", self.codes[1]),
                           ("k_sf", self.sf[0]), ("v_sf", self.sf[1])):
            p, h, s, r = like.shape
            y = self.bufs[name].cpu().numpy()
            if self.pad:
                assert (y[:, h * s * r:] == 0xA5).all(), "bytes between pages were written"
            y = y[:, :h * s * r]
            out[name] = (y.reshape(p, h, s, r) if self.layout == "HND"
                         else y.reshape(p, s, h, r).transpose(0, 2, 1, 3))
        return out

    def dense(self, which, b):
        """[heads, tokens, dim] of request b's K (0) or V (1)."""
        codes, sf = self.codes[which][self.pages(b)], self.sf[which][self.pages(b)]
        x = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
        x[..., 0::2], x[..., 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
        x *= np.repeat(R.VALUES[sf], 16, -1) * self.g[which]
        n, h, p, d = x.shape
        return x.transpose(1, 0, 2, 3).reshape(h, n * p, d)[:, :self.kv[b]]


def tree_attention(q, k, v, hide, sm_scale):
    """One request: q [n, Hq, Dk], k [Hkv, L, Dk], v [Hkv, L, Dv], hide [n, L]: out, lse and,
    for the tolerance, the weighted mean of |v|, the largest sm_scale * sum_d |q_d k_d| of a
    row and sum_j |v_j| / sum_j p_j (p_j relative to the row's largest) over its keys."""
    n, hq, _ = q.shape
    hkv, total, dv = v.shape
    out, lse = np.zeros((n, hq, dv)), np.full((n, hq), -np.inf)
    mean, reach, floor = np.zeros((n, hq, dv)), np.zeros((n, hq)), np.zeros((n, hq, dv))
    for i in range(n):
        see = ~hide[i]
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[h // (hq // hkv)][see], v[h // (hq // hkv)][see]
            s = sm_scale * (kk @ q[i, h])
            p = np.exp(s - s.max())
            lse[i, h] = s.max() + math.log(p.sum())
            out[i, h] = p @ vv / p.sum()
            mean[i, h] = p @ np.abs(vv) / p.sum()
            reach[i, h] = sm_scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            floor[i, h] = np.abs(vv).sum(0) / p.sum()
    return out, lse, mean, reach, floor


def check_tree(got, got_lse, want, dk, dtype):
    """Rows of one request against `want` (of tree_attention).  Beside the output's own
    rounding: a weight is rounded to f16 (2^-11, at least 2^-25 of the row's largest) in the
    product and in the row sum; the scores' sums err by Dk 2^-23 of sum |q k| (`reach`) at
    most, and what follows by 2^-21; an error d of a score is one of d of a weight and of
    the sum."""
    ref, rl, mean, reach, floor = want
    eps = torch.finfo(dtype).eps / 2
    delta = dk * 2.0 ** -23 * reach + 2.0 ** -21
    tol = (eps * np.abs(ref) + (mean * (2.0 ** -10 + 2.0 ** -19 + 2 * delta[..., None])
                                + 2.0 ** -25 * floor) * (1 + eps)
           + float(torch.finfo(dtype).smallest_normal) * eps)
    none = np.isinf(rl)
    assert np.array_equal(got_lse == -np.inf, none)
    assert (got[none] == 0).all()
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    lerr = np.abs(got_lse[~none] - rl[~none])
    ltol = delta + 2.0 ** -11 + 2.0 ** -19 + np.abs(rl) * 2.0 ** -22
    assert (lerr <= ltol[~none]).all(), lerr.max()


# ---- accepted tokens -------------------------------------------------------------------
def moved(case_pages, page, begin, path):
    """(target page, slot, source page, slot) of every accepted token of one request."""
    out = []
    for i, node in enumerate(path):
        s, t = begin + node, begin + i
        out.append((case_pages[t // page], t % page, case_pages[s // page], s % page))
    return out


# ---- pages with several owners ----------------------------------------------------------
class Pool:
    """A block table, its lengths, the owners beyond the first and a free list, in lists."""

    def __init__(self, table, kv_len, shares, free, head, page):
        self.table = [list(r) for r in table]
        self.kv_len, self.shares, self.free = list(kv_len), list(shares), list(free)
        self.head, self.page = head, page

    def fork(self, parents, children):
        copies = []
        for p, c in zip(parents, children):
            n = self.kv_len[p]
            whole = n // self.page
            for col in range(whole):
                self.table[c][col] = self.table[p][col]
                self.shares[self.table[p][col]] += 1
            pair = (-1, -1)
            if n % self.page:
                pair = (self.table[p][whole], self.free[self.head])
                self.table[c][whole] = pair[1]
                self.head += 1
            copies.append(pair)
        for p, c in zip(parents, children):
            self.kv_len[c] = self.kv_len[p]
        return copies

    def release(self, keep):
        entries = [self.table[b][c] for b, k in enumerate(keep)
                   for c in range(R.pages_of(k, self.page), R.pages_of(self.kv_len[b], self.page))]
        freed = []
        left = dict()
        for e in entries:
            left[e] = left.get(e, 0) + 1
        for e in entries:
            if left[e] > self.shares[e] and e not in freed:
                freed.append(e)
        for e, n in left.items():
            self.shares[e] = max(0, self.shares[e] - n)
        self.head -= len(freed)
        self.free[self.head:self.head + len(freed)] = freed
        self.kv_len = list(keep)
