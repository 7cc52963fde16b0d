"""The serving-step operators on the GPU against 64-bit references: the page
table, rotary positions, the append into the E4M3 cache, the attention over
it, and a run of them together as a decode loop uses them."""
import math

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
from nvfp4_paged_kv_nvfp4kv_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def new_flags():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- page table ----------------------------------------------------------------
LISTS = ("qo_indptr", "kv_indptr", "last_page_len", "kv_indices", "batch_idx", "positions",
         "slot_map", "free_head")


class TableCase:
    def __init__(self, kv_len, qo_len, page, seed=0, head=2, pad=3, extra=4):
        rng = np.random.default_rng(seed)
        self.kv, self.qo, self.page, self.head = list(kv_len), list(qo_len), page, head
        held = [R.pages_of(a - n, page) for a, n in zip(kv_len, qo_len)]
        every = [R.pages_of(a, page) for a in kv_len]
        ids = rng.permutation(sum(every) + 50).tolist()
        width = max(every, default=0) + pad
        self.rows, at = [], head
        for h in held:
            self.rows.append(ids[at:at + h] + [-5] * (width - h))
            at += h
        self.free = ids[:head] + ids[at:]
        # rows apart by more than their width
        self.table = torch.full((len(held), width + 5), -9, dtype=torch.int32, device="cuda")
        if held:
            self.table[:, :width] = torch.tensor(self.rows, dtype=torch.int32)
        self.width = width
        self.out = N.StepTable.allocate(len(held), sum(qo_len) + extra, sum(every) + extra)
        for n in LISTS:
            getattr(self.out, n).fill_(-7)

    def run(self, flags=None, free_head=True):
        N.nvfp4kv_build_page_table(i32(self.kv), i32(self.qo), self.table[:, :self.width],
                                   i32(self.free), i32([self.head]) if free_head else None,
                                   self.out, page_size=self.page, device_flags=flags)

    def check(self, head=None):
        want = R.page_table(self.kv, self.qo, self.rows, self.free,
                            self.head if head is None else head, self.page)
        for n in LISTS:
            got = getattr(self.out, n).tolist()
            w = want[n]
            assert got[:len(w)] == w, n
            assert all(x == -7 for x in got[len(w):]), n  # past the step: as they were
        assert self.table[:, :self.width].tolist() == self.rows
        assert bool((self.table[:, self.width:] == -9).all())


@pytest.mark.parametrize("page", [16, 1, 7])
@pytest.mark.parametrize("batch", [1, 3, 513, 1300])
def test_page_table(batch, page):
    rng = np.random.default_rng(batch * 31 + page)
    kv = rng.integers(0, 90, batch)
    qo = [int(rng.choice([0, 1, n, min(n, 20)])) if n else 0 for n in kv]
    qo = [min(a, int(n)) for a, n in zip(qo, kv)]
    c = TableCase([int(x) for x in kv], qo, page, seed=batch)
    f = new_flags()
    c.run(f)
    c.check()
    assert int(f) == 0
    c.run(f)  # the table's own new entries change nothing
    c.check()


def test_page_table_edges():
    c = TableCase([], [], 16, head=0)
    c.run()
    c.check()
    c = TableCase([0, 0, 0], [0, 0, 0], 16, head=0, pad=0)
    c.run()
    c.check()
    c = TableCase([0, 33, 0, 16, 0], [0, 33, 0, 1, 0], 16, head=0)
    c.run(free_head=False)
    c.check()
    c = TableCase([70000, 1], [3, 1], 16, extra=0)  # one long request, exact capacities
    c.run()
    c.check()


@pytest.mark.parametrize("kv,qo,flag", [
    ([5, -1], [1, 0], _lib.FLAG_BAD_LENGTH),
    ([5, 4], [1, 5], _lib.FLAG_BAD_LENGTH),
    ([5, 4], [1, -1], _lib.FLAG_BAD_LENGTH),
    ([5, 2**31 - 1], [1, 1], _lib.FLAG_BAD_LENGTH),
    ([5, 1000], [1, 1], _lib.FLAG_BAD_LENGTH),        # more pages than a row has
    ([5, 60], [5, 60], _lib.FLAG_TABLE_FULL),         # rows, pages and new pages
    ([48, 60], [1, 1], _lib.FLAG_TABLE_FULL),         # pages
    ([5, 40], [1, 10], _lib.FLAG_TABLE_FULL),         # rows
])
def test_page_table_refuses_whole_batches(kv, qo, flag):
    c = TableCase([20, 30], [1, 1], 16, extra=1)
    before = c.table.clone()
    c.kv, c.qo = kv, qo
    f = new_flags()
    c.run(f)
    assert int(f) == flag
    assert torch.equal(c.table, before)
    assert all(bool((getattr(c.out, n) == -7).all()) for n in LISTS)


def test_page_table_free_list_runs_out():
    c = TableCase([20, 33], [1, 17], 16, extra=20)
    c.free = c.free[:c.head + 1]
    f = new_flags()
    c.run(f)
    assert int(f) == _lib.FLAG_TABLE_FULL and bool((c.out.kv_indptr == -7).all())


def test_page_table_without_slot_map():
    c = TableCase([40, 3], [2, 3], 16)
    c.out = N.StepTable.allocate(2, 9, 9, slot_map=False)
    c.run()
    want = R.page_table(c.kv, c.qo, c.rows, c.free, c.head, 16)
    assert c.out.positions.tolist()[:5] == want["positions"]


# ---- rotary positions ------------------------------------------------------------
def check_rope(got, x, positions, rotary, interleaved, freq, attn):
    """The result is rounded once (half a step of the type); before that each
    cosine and sine is off by at most 2 pi 2^-26 from the angle and 2 ulp of
    float32 (2^-23) from sincospif, times attention_factor (rounded: 2^-24),
    and two products and a sum round by 2^-24 each: below (|x1| + |x2|) *
    attn * 2^-21 together."""
    y, size = R.rope(x, positions, rotary, interleaved, freq, attn)
    eps = torch.finfo(x.dtype).eps / 2
    tol = eps * np.abs(y) * (size > 0) + size * attn * 2.0 ** -21 * (1 + eps)
    tol += (size > 0) * float(torch.finfo(x.dtype).smallest_normal) * eps  # subnormal results
    bad = np.abs(R.to_np(got) - y) > tol
    assert not bad.any(), (int(bad.sum()), np.abs(R.to_np(got) - y).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,rotary,interleaved", [
    (128, 128, False), (128, 128, True), (64, 32, False), (256, 64, True), (128, 124, True),
    (64, 30, False), (512, 512, False), (512, 510, True), (8, 2, False), (8, 2, True),
    (96, 96, False), (40, 24, False), (512, 494, False)])
@pytest.mark.parametrize("tokens", [1, 37])
def test_rope(dim, rotary, interleaved, dtype, tokens):
    g = torch.Generator().manual_seed(dim + rotary + tokens)
    hq, hkv, attn = 5, 2, 1.25
    x = torch.randn((tokens, hq + hkv + 1, dim), generator=g).to(DT[dtype]).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hkv]  # strided rows
    pos = torch.randint(-10, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    pos[0] = 2**31 - 1
    opts = dict(base=500000.0, factor=8.0)
    plan = N.nvfp4kv_rope_plan(dim, rotary, interleaved=interleaved, attention_factor=attn,
                               original_max_position=8192, high_rotations=4.0, **opts)
    freq = R.rope_frequencies(rotary, 500000.0, 8.0, 8192, 1.0, 4.0)
    before = x.clone()
    qo, ko = N.nvfp4kv_rope(plan, q, k, pos.cuda())
    assert torch.equal(x, before)
    check_rope(qo, q, pos.tolist(), rotary, interleaved, freq, attn)
    check_rope(ko, k, pos.tolist(), rotary, interleaved, freq, attn)
    # in place, one of the two alone: the same bits, and only those rows
    q_in, _ = N.nvfp4kv_rope(plan, q, None, pos.cuda(), q_out=q)
    assert q_in is q and torch.equal(q, qo) and torch.equal(x[:, hq:], before[:, hq:])
    _, k2 = N.nvfp4kv_rope(plan, None, k, pos.cuda())
    assert torch.equal(k2, ko)


def test_rope_many_tokens_and_heads():
    """Several heads a lane and several warps' columns, full occupancy."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn((2500, 40, 64), generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(2500, dtype=torch.int32) * 401
    plan = N.nvfp4kv_rope_plan(64)
    out, _ = N.nvfp4kv_rope(plan, q, None, pos.cuda())
    check_rope(out, q, pos.tolist(), 64, False, R.rope_frequencies(64, 10000.0), 1.0)


def test_rope_leaves_what_it_does_not_rotate():
    """Passing dims keep their bits (NaN and infinities too), rows past the
    positions stay as they were, and no tokens is a call that does nothing."""
    for rotary, inter in ((32, False), (30, False), (32, True), (30, True)):
        q = torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16)
        q[..., rotary:] = float("nan")
        q[..., rotary + 1] = float("inf")
        out = torch.full_like(q, 3.0)
        plan = N.nvfp4kv_rope_plan(64, rotary, interleaved=inter)
        N.nvfp4kv_rope(plan, q, None, i32([1, 2, 3]), q_out=out)
        assert torch.equal(out[:3, :, rotary:].view(torch.int16),
                           q[:3, :, rotary:].view(torch.int16))
        assert bool(out[:3, :, :rotary].isfinite().all()) and bool((out[3] == 3.0).all())
        a, b = N.nvfp4kv_rope(plan, q, q, i32([]))
        assert a.shape == b.shape == (0, 2, 64)


# ---- append into the E4M3 cache -----------------------------------------------------
class CacheCase:
    """A cache whose requests hold tokens already (random codes and scales), and
    its reference copy."""

    def __init__(self, kv_len, page, heads, dk, dv, layout="HND", seed=0, spread=3, spare=3):
        rng = np.random.default_rng(seed)
        self.kv, self.page, self.heads, self.dims = list(kv_len), page, heads, (dk, dv)
        np_ = [R.pages_of(n, page) for n in kv_len]
        total = sum(np_) + spare
        self.cache = N.E4m3Cache.allocate(total, heads, dk, dv, page, layout)
        ids = rng.permutation(total)[:sum(np_)]
        self.indptr = np.concatenate([[0], np.cumsum(np_)])
        self.ids = ids
        self.last = [n - (p - 1) * page if p else 0 for n, p in zip(kv_len, np_)]
        self.codes, self.scale = [], []
        for d in self.dims:
            c = rng.integers(0, 256, (total, heads, page, d)).astype(np.uint8)
            c[(c & 0x7F) == 0x7F] = 0x50
            self.codes.append(c)
            self.scale.append((2.0 ** rng.integers(-7 - spread, -7 + spread + 1,
                                                   (total, heads))).astype(np.float32))
        self.upload()
        self.kv_indptr, self.kv_indices = i32(self.indptr), i32(ids)
        self.last_page_len = i32(self.last)

    def upload(self):
        c = self.cache
        for t, x in ((c.k_data, self.codes[0]), (c.v_data, self.codes[1])):
            t.copy_(torch.from_numpy(x))
        c.k_scale.copy_(torch.from_numpy(self.scale[0]))
        c.v_scale.copy_(torch.from_numpy(self.scale[1]))

    def pages(self, b):
        return self.ids[self.indptr[b]:self.indptr[b + 1]]

    def append(self, new, k, v):
        """The reference of an append of new[b] rows to every request."""
        row = 0
        for b, n in enumerate(new):
            begin = self.kv[b] - n
            for c in range(begin // self.page, len(self.pages(b)) if n else 0):
                lo, hi = max(begin - c * self.page, 0), min(self.kv[b] - c * self.page, self.page)
                for i, x in enumerate((k, v)):
                    R.append(self.codes[i][self.pages(b)[c]], self.scale[i][self.pages(b)[c]],
                             R.to_np(x), self.page, lo, hi, row + c * self.page + lo - begin)
            row += n

    def check(self):
        c = self.cache
        for got, want in ((c.k_data, self.codes[0]), (c.v_data, self.codes[1]),
                          (c.k_scale, self.scale[0]), (c.v_scale, self.scale[1])):
            g = got.cpu().numpy()
            assert np.array_equal(g, want), (int((g != want).sum()), want.shape)

    def run_append(self, new, k, v, flags=None):
        N.nvfp4kv_e4m3_append(self.cache, k, v, i32(np.concatenate([[0], np.cumsum(new)])),
                              self.kv_indptr, self.kv_indices, self.last_page_len, flags)


def new_rows(rows, heads, dk, dv, dtype, seed=0, spread=6):
    g = torch.Generator().manual_seed(seed)
    out = []
    for d in (dk, dv):
        x = torch.randn((rows, heads, d), generator=g)
        x *= torch.exp2(torch.randint(-spread, spread, (rows, heads, 1), generator=g).float())
        out.append(x.to(DT[dtype]).cuda())
    return out


@pytest.mark.parametrize("dtype,layout,page,dk,dv,kv,new", [
    ("bf16", "HND", 16, 128, 128, (37, 16, 1, 100, 0), (1, 1, 1, 1, 0)),
    ("bf16", "NHD", 16, 128, 128, (37, 48, 17, 5, 33), (20, 48, 1, 5, 0)),
    ("f16", "HND", 16, 64, 64, (40, 31), (9, 31)),
    ("bf16", "HND", 16, 512, 256, (40, 17), (30, 2)),
    ("f16", "NHD", 16, 256, 512, (40, 17), (30, 2)),
    ("bf16", "HND", 16, 96, 32, (40, 17), (30, 2)),
    ("bf16", "HND", 1, 128, 64, (40, 17, 3), (30, 2, 0)),
    ("f16", "NHD", 1, 512, 512, (4, 7), (1, 7)),
])
def test_append(dtype, layout, page, dk, dv, kv, new):
    c = CacheCase(kv, page, 3, dk, dv, layout, seed=dk + page)
    k, v = new_rows(sum(new) + 2, 3, dk, dv, dtype, seed=7)  # two rows past the last request
    f = new_flags()
    c.append(new, k, v)
    c.run_append(new, k, v, f)
    c.check()
    assert int(f) == 0
    c.run_append(new, k, v, f)  # the same rows again: the same cache
    c.check()


def test_append_strided_rows_and_long_prompt():
    """Rows out of one projection, a prompt over many pages, several requests
    a call, CTAs that walk more than one block."""
    kv, new = (3001, 40, 700), (3000, 1, 655)
    c = CacheCase(kv, 16, 2, 64, 64, seed=5)
    x = torch.randn((sum(new), 7, 64), generator=torch.Generator().manual_seed(1)).cuda()
    x = x.to(torch.bfloat16)
    k, v = x[:, 1:3], x[:, 4:6]
    c.append(new, k, v)
    c.run_append(new, k, v)
    c.check()


def test_append_values_at_the_edges():
    """Zeros (and a page of nothing else), ties, saturation of the scale's
    range, infinities, NaN, a largest value just at and above 448 * 2^e."""
    c = CacheCase((16, 32, 33, 16, 16, 20), 16, 1, 32, 32, seed=9)
    new = (16, 32, 17, 16, 16, 4)
    k, v = new_rows(sum(new), 1, 32, 32, "bf16", seed=2)
    k[:16] = 0.0
    k[3, 0, 4] = -0.0
    v[:16] = 1e38
    v[5, 0, 3] = -3e38
    k[16:48] = 448.0                      # the scale is 1 exactly
    k[20, 0, :8] = torch.tensor([17., 19., 21., 23., 0.0009765625, 0.0029296875, 0.0009, -27.])
    v[16:48] = 450.0                      # rounds to bf16 450: the scale is 2
    k[48, 0, 0], k[49, 0, 1], k[50, 0, 2] = math.inf, -math.inf, math.nan
    v[48:65] = math.inf                   # nothing finite in the block
    k[65:81] = 1e-30                      # below the scale's range
    c.scale[0][c.pages(5)[1], 0] = 0.01   # a scale that is no power of two
    c.upload()
    c.append(new, k, v)
    f = new_flags()
    c.run_append(new, k, v, f)
    c.check()
    assert int(f) == 0


@pytest.mark.parametrize("dk,dv,heads", [(32, 96, 5), (128, 64, 8), (512, 256, 3), (256, 256, 1)])
def test_append_one_token_pages_at_the_edges(dk, dv, heads):
    """The same values where a warp takes all heads of a token; a page id out of
    the pool leaves its token's page as it was."""
    c = CacheCase((40, 9), 1, heads, dk, dv, seed=dk)
    k, v = new_rows(49, heads, dk, dv, "bf16", seed=2)
    k[0], k[1], v[1], k[2], v[2] = 0.0, 448.0, 450.0, math.inf, -math.inf
    k[3, :, 4], v[4, heads - 1, dv - 1], v[7, 0] = math.nan, -math.inf, math.nan
    k[5], v[6] = 1e-30, 1e38
    page = int(c.ids[11])
    old = [x[page].copy() for x in (*c.codes, *c.scale)]
    c.append((40, 9), k, v)
    for x, y in zip((*c.codes, *c.scale), old):
        x[page] = y
    c.kv_indices[11] = 10 ** 6
    f = new_flags()
    c.run_append((40, 9), k, v, f)
    c.check()
    assert int(f) == _lib.FLAG_BAD_APPEND_TARGET


def test_append_skips_and_flags():
    kv, new = (20, 20, 20, 20), (2, 2, 2, 2)
    base = CacheCase(kv, 16, 2, 64, 64, seed=3)
    k, v = new_rows(8, 2, 64, 64, "bf16")

    def run(kvp=None, idx=None, last=None, qo=(0, 2, 4, 6, 8), good=(0, 2, 3)):
        c = CacheCase(kv, 16, 2, 64, 64, seed=3)
        f = new_flags()
        N.nvfp4kv_e4m3_append(c.cache, k, v, i32(qo), i32(kvp or c.indptr), i32(idx or c.ids),
                              i32(last or c.last), f)
        row = 0
        for b, n in enumerate(new):  # the others are stored
            if b in good:
                lo = 2
                for i, x in enumerate((k, v)):
                    p = c.pages(b)[1]
                    R.append(c.codes[i][p], c.scale[i][p], R.to_np(x), 16, lo, 4, row)
            row += n
        c.check()
        assert int(f) == _lib.FLAG_BAD_APPEND_TARGET
    ids = base.ids.tolist()
    run(idx=ids[:3] + [10**6] + ids[4:])          # request 1's second page
    run(idx=ids[:3] + [-1] + ids[4:])
    run(last=[4, 17, 4, 4])
    run(last=[4, 0, 4, 4])
    run(qo=(0, 2, 4, 6, 9), good=(0, 1, 2))        # more rows than k holds
    run(kvp=[0, 2, 2, 2, 8], idx=ids[:2] + ids[2:], good=(0,), qo=(0, 2, 4, 6, 6))


def test_append_bad_old_scale_is_flagged():
    c = CacheCase((20,), 16, 1, 64, 64, seed=3)
    c.scale[0][c.pages(0)[1], 0] = math.nan
    c.upload()
    k, v = new_rows(1, 1, 64, 64, "bf16")
    f = new_flags()
    c.run_append((1,), k, v, f)
    assert int(f) == _lib.FLAG_BAD_SCALE
    assert math.isfinite(float(c.cache.k_scale[int(c.pages(0)[1]), 0]))


# ---- attention over the E4M3 cache ----------------------------------------------------
def attend_case(kv, new, hq, hkv, dk, dv, causal=False, page=16, layout="HND", dtype="bf16",
                out="bf16", seed=0, spread=3, stale=True, only=None, q_scale=1.0, live=None,
                edit=None, **plan_kw):
    """Run the attention on a random cache and compare every row with the
    64-bit reference.  The result is rounded once.  Before that: a score is off
    by at most Dk 2^-23 * sm_scale sum|q k| (f32 sums of exact f16 products)
    and the exponential by 2^-21 relative, so a weight by that delta; weights
    are rounded to f16 (2^-11 relative, 2^-25 of the row's largest weight times
    scale at least); normalised sums and a merge of split states in f32: 2^-19.  ``edit(c, q)``
    may change the reference cache and the query first; then NaN has to be where
    the reference has it.

    With more than 8 rows a block the tensor-memory kernel runs: it adds E4M3
    pieces, each the rounded rest (off by at most 2^-4 of it), of the query and
    of the weights.  Query pieces, with the row's largest |q| in [128, 256), are
    exact but for elements whose last bit is below the smallest code 2^-9: off
    by 2^-10, 2^-17 of the largest |q|, so a score by 2^-17 * sm_scale max|q|
    sum|k| more.  The three pieces of a weight, after f16, are off by 2^-12 of it
    and by half the last piece's smallest code, 2^-10 / 1024, where the row's
    largest is 1 or more: 2^-20 of that (f16's own floor is below)."""
    c = CacheCase(kv, page, hkv, dk, dv, layout, seed=seed, spread=spread)
    if stale:  # slots past every length hold NaN codes
        for b, n in enumerate(kv):
            if n and n % page:
                for x in c.codes:
                    x[c.pages(b)[-1], :, n % page:] = 0x7F
        c.upload()
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(new) + 1, hq + 1, dk), generator=g) * q_scale
    if edit is not None:
        edit(c, q[:, 1:])
        c.upload()
    q = q.to(DT[dtype]).cuda()[:, 1:]
    qo = np.concatenate([[0], np.cumsum(new)])
    plan_last = c.last
    if live is not None:
        plan_last, plan_kw["device_last_page_len"] = live, c.last_page_len
    plan = N.nvfp4kv_decode_plan(qo, c.indptr, plan_last, hq, hkv, dk, dv, page_size=page,
                                 causal=causal, kernel=5, out_dtype=DT[out], **plan_kw)
    o, lse = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    o2, lse2 = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    assert torch.equal(lse.nan_to_num(), lse2.nan_to_num()) or plan.info.split
    got, gl = R.to_np(o), R.to_np(lse)
    eps = torch.finfo(DT[out]).eps / 2
    scale = float(np.float32(1 / math.sqrt(dk)))
    for b, n in enumerate(new):
        if not n or (only is not None and b not in only):
            continue
        k, v = (R.dequantised(c.codes[i], c.scale[i], c.pages(b), kv[b]) for i in (0, 1))
        vs = np.repeat(c.scale[1][c.pages(b)].T.astype(np.float64), page, 1)[:, :kv[b]]
        rows = slice(int(qo[b]), int(qo[b + 1]))
        ref, rl, mean, reach, floor = R.attention(R.to_np(q[rows]), k, v, vs, scale, causal)
        delta = (dk * 2.0 ** -23 * reach + 2.0 ** -21)
        weight, least = 2.0 ** -11, 2.0 ** -25
        if plan.info.rows_per_block > 8:
            delta = delta + 2.0 ** -17 * scale * (np.abs(R.to_np(q[rows])).max(-1)
                                                  * np.nansum(np.abs(k), -1).max())
            weight, least = weight + 2.0 ** -12, 2.0 ** -20 + 2.0 ** -25
        tol = (eps * np.abs(ref) + (mean * (weight + 2.0 ** -19 + 2 * delta[..., None])
                                    + least * floor) * (1 + eps)
               + float(torch.finfo(DT[out]).smallest_normal) * eps)
        none, lnone = np.isnan(ref), np.isnan(rl)
        assert edit is not None or not (none.any() or lnone.any())
        assert np.array_equal(np.isnan(got[rows]), none)
        assert np.array_equal(np.isnan(gl[rows]), lnone)
        err = np.abs(got[rows] - ref)[~none]
        assert (err <= tol[~none]).all(), (b, float(err.max()), float((err / tol[~none]).max()))
        lerr = np.abs(gl[rows] - rl)
        lok = lerr <= delta + 2.0 ** -19 + np.abs(rl) * 2.0 ** -22
        assert lok[~lnone].all(), (b, lerr[~lnone].max())
    return c, plan, o


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 128), (256, 256), (512, 256)])
@pytest.mark.parametrize("page,layout", [(16, "HND"), (16, "NHD"), (1, "HND")])
def test_attention_dims(dk, dv, page, layout):
    attend_case((37, 100, 1, 16, 17, 500), (1,) * 6, 8, 2, dk, dv, page=page, layout=layout,
                seed=dk + dv)


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("hq,hkv,new,causal", [
    (4, 4, (1, 1, 1), False), (5, 1, (1, 1, 1), False), (16, 1, (1, 1, 1), False),
    (8, 1, (3, 2, 0), True), (8, 2, (7, 30, 1), True), (8, 2, (7, 30, 1), False),
    (4, 2, (37, 65, 90), True), (32, 4, (9, 65, 1), True)])
def test_attention_rows(hq, hkv, new, causal, page):
    attend_case((37, 65, 90), new, hq, hkv, 128, 128, causal=causal, page=page, seed=hq + sum(new))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 128), (256, 256), (512, 256)])
@pytest.mark.parametrize("page,layout,out", [(16, "HND", "bf16"), (16, "NHD", "f16"),
                                             (1, "HND", "bf16")])
@pytest.mark.parametrize("new", [(5, 4, 0), (9, 16, 1), (13, 16, 40)])
def test_attention_dims_many_rows(dk, dv, page, layout, out, new):
    """Up to 10, 32 and 80 rows per kv head: every kernel of every head dim."""
    attend_case((37, 300, 40), new, 4, 2, dk, dv, causal=True, page=page, layout=layout, out=out,
                seed=dk + sum(new))


@pytest.mark.parametrize("hq,hkv", [(16, 1), (48, 2), (32, 1)])
def test_attention_wide_groups_split(hq, hkv):
    """16, 24 and 32 heads to a kv head, one row each, split requests."""
    _, plan, _ = attend_case((700, 33, 5), (1, 1, 1), hq, hkv, 128, 128, force_chunk_tokens=128,
                             seed=hq)
    assert plan.info.split == 1


@pytest.mark.parametrize("chunk", [16, 64, 176])
@pytest.mark.parametrize("new,causal", [((1, 1, 1, 1), False), ((5, 1, 0, 30), True)])
def test_attention_split(chunk, new, causal):
    _, plan, _ = attend_case((300, 1, 17, 1111), new, 8, 2, 128, 128, causal=causal,
                             force_chunk_tokens=chunk, seed=chunk)
    assert plan.info.split == 1


def test_attention_prompt_from_nothing():
    """Every token is new: the causal triangle, rows that see one key."""
    attend_case((130, 16, 1), (130, 16, 1), 4, 2, 128, 128, causal=True, seed=4)
    attend_case((70,), (70,), 4, 1, 64, 64, causal=True, page=1, seed=4)


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("f16", "bf16"), ("bf16", "f16")])
def test_attention_types(dtype, out):
    attend_case((37, 200), (2, 1), 8, 2, 128, 128, dtype=dtype, out=out, seed=6)


@pytest.mark.parametrize("spread", [0, 12, 30])
def test_attention_scales_apart(spread):
    """Page scales 2^-7 apart by up to 2^(2 spread): the weights of the values
    follow the largest weight times scale, not the largest score."""
    attend_case((400, 90), (1, 3), 4, 1, 128, 128, causal=True, spread=spread, seed=spread,
                q_scale=2.0 ** -spread)
    attend_case((100, 50), (1, 1), 4, 1, 64, 64, page=1, spread=spread, seed=spread,
                q_scale=2.0 ** -spread)


def test_attention_peaked_scores():
    attend_case((400, 90), (1, 3), 4, 1, 128, 128, causal=True, seed=8, q_scale=40.0)


def test_attention_automatic_split_of_long_requests():
    _, plan, _ = attend_case((20011, 5000), (1, 1), 4, 1, 128, 128, seed=11)
    assert plan.info.split == 1 and plan.info.kernel == 5


def test_attention_live_lengths():
    """A plan made when the last pages held one token reads the current ones."""
    attend_case((37, 100, 16), (1, 1, 1), 8, 2, 128, 128, live=[1, 1, 1], seed=12)
    attend_case((45, 110, 16), (3, 2, 1), 8, 2, 128, 128, causal=True, live=[16, 1, 9], seed=12)


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("chunk", [0, 64])
@pytest.mark.parametrize("dk,dv,hq,hkv,new", [
    (128, 128, 4, 2, (1, 1, 1)), (128, 128, 8, 2, (4, 3, 2)), (64, 64, 4, 2, (7, 3, 8)),
    (128, 128, 8, 2, (20, 9, 5)), (256, 256, 4, 2, (30, 9, 5)), (256, 128, 4, 2, (2, 3, 4)),
    (512, 256, 4, 2, (7, 3, 2))])
def test_attention_nan_reaches_the_rows_that_see_it(dk, dv, hq, hkv, new, chunk, page):
    """NaN codes: in V, at tokens that some rows do not see (one dim of those that
    do) and at one that all see; in K, at the last token, alone in its page; and
    queries with a NaN or an infinite element."""
    kv = (200, 33, 150)

    def edit(c, q):
        def at(b, t):
            return c.pages(b)[t // page], t % page
        for t, d, code in ((199, 5, 0x7F), (200 - (new[0] + 1) // 2, dv - 1, 0xFF), (60, 17, 0x7F)):
            pg, slot = at(0, t)
            c.codes[1][pg, 0, slot, d] = code
        pg, slot = at(1, 32)
        c.codes[0][pg, 1, slot, 3] = 0x7F
        last = sum(new) - 1
        q[last, 0, 7], q[last, 1, 9] = math.nan, math.inf
    attend_case(kv, new, hq, hkv, dk, dv, causal=True, page=page, force_chunk_tokens=chunk,
                edit=edit, seed=dk + sum(new))


@pytest.mark.parametrize("rows", [1, 12, 40])
def test_attention_zero_scores_at_the_ends_of_the_range(rows):
    """Keys of nothing but zero codes under the largest scale, and queries as
    large as their type allows: scores of 0, so the mean of the values."""
    def edit(c, q):
        c.codes[0][:] = 0
        c.scale[0][:] = 2.0 ** 64
        q *= 2.0 ** 120
    attend_case((1, 40), (1, rows), 2, 1, 128, 128, edit=edit, seed=rows)


def test_attention_nothing_to_do():
    _, plan, o = attend_case((37, 5, 0), (0, 0, 0), 8, 2, 128, 128)
    assert plan.info.num_units == 0 and o.shape == (0, 8, 128)


def test_attention_flags():
    """A page id out of the pool and a scale that is none are flagged."""
    c, plan, _ = attend_case((37, 100), (1, 1), 4, 1, 128, 128, seed=2)
    q = torch.randn((2, 4, 128), device="cuda").to(torch.bfloat16)
    for bad in (-1, 10**6):
        idx = c.kv_indices.clone()
        idx[1] = bad
        N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, idx)
        assert N.nvfp4kv_workspace_flags(plan, clear=True) == _lib.FLAG_BAD_PAGE_INDEX
    for scale in (c.cache.k_scale, c.cache.v_scale):
        for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 65):
            keep = scale.clone()
            scale[int(c.ids[2])] = bad
            N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
            assert N.nvfp4kv_workspace_flags(plan, clear=True) == _lib.FLAG_BAD_SCALE
            scale.copy_(keep)
    N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    assert N.nvfp4kv_workspace_flags(plan) == 0


def test_attention_refusals():
    c, plan, _ = attend_case((37, 100), (1, 1), 4, 1, 128, 128, seed=2)
    q = torch.randn((2, 4, 128), device="cuda").to(torch.bfloat16)
    other = N.nvfp4kv_decode_plan([0, 1, 2], c.indptr, c.last, 4, 1, 128, 128, kernel=1)
    with pytest.raises(N.NvFp4KvError) as e:
        N.nvfp4kv_e4m3_decode_run(other, q, c.cache, c.kv_indices)
    assert e.value.status == _lib.ERR_PLAN_MISMATCH
    small = N.E4m3Cache.allocate(9, 1, 64, 64)
    with pytest.raises(N.NvFp4KvError) as e:
        N.nvfp4kv_e4m3_decode_run(plan, q, small, c.kv_indices)
    assert e.value.status == _lib.ERR_PLAN_MISMATCH
    layout = W.CacheLayout("HND", 9, 16, 1, 128, 128)
    with pytest.raises(N.NvFp4KvError) as e:
        N.nvfp4kv_decode_run(plan, q, N.PagedCache.allocate(layout), c.kv_indices)
    assert e.value.status == _lib.ERR_PLAN_MISMATCH
    with pytest.raises(ValueError):
        N.nvfp4kv_e4m3_decode_run(plan, q.float(), c.cache, c.kv_indices)
    with pytest.raises(ValueError):
        N.nvfp4kv_e4m3_decode_run(plan, q.cpu(), c.cache, c.kv_indices)
    with pytest.raises(ValueError):
        N.nvfp4kv_e4m3_decode_run(plan, q[:1], c.cache, c.kv_indices)
    with pytest.raises(ValueError):
        N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices[:2])


def test_attention_plan_with_the_other_entry_points():
    """Kernel 5's partial states merged once more by the standalone kernel; the
    NVFP4 entry points refuse the plan."""
    for new in ((1, 1), (20, 9)):
        c, plan, o = attend_case((700, 300), new, 8, 2, 128, 128, causal=True, seed=2,
                                 force_chunk_tokens=128)
        assert plan.info.split
        q = torch.randn((sum(new), 8, 128), device="cuda").to(torch.bfloat16)
        o, lse = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
        m, ml = torch.zeros_like(o), torch.zeros_like(lse)
        N.nvfp4kv_decode_merge(plan, m, ml)
        # one rounding apart from the same f32 states: a bf16 step at most
        assert bool(((m.float() - o.float()).abs() <= 2.0 ** -7 * o.float().abs() + 1e-6).all())
        assert torch.allclose(ml, lse, atol=2.0 ** -18, rtol=2.0 ** -20)
        nv = N.PagedCache.allocate(W.CacheLayout("HND", c.cache.num_pages, 16, 2, 128, 128))
        k = torch.zeros((sum(new), 2, 128), dtype=torch.bfloat16, device="cuda")
        bare = N.nvfp4kv_decode_plan([0, new[0], sum(new)], c.indptr, c.last, 8, 2, 128, 128,
                                     causal=True, kernel=5, allocate=False)
        for run in (lambda: N.nvfp4kv_decode_run_static(bare, q, nv, c.kv_indices),
                    lambda: N.nvfp4kv_decode_append_run(plan, k, k, q, nv, c.kv_indices)):
            with pytest.raises(N.NvFp4KvError) as e:
                run()
            assert e.value.status == _lib.ERR_PLAN_MISMATCH


def test_offsets_past_32_bits():
    """A cache whose pages, rows whose tokens and a table whose requests lie far
    apart: the first and last bytes of a buffer of 7 GB."""
    buf = torch.zeros(7 << 30, dtype=torch.uint8, device="cuda")
    for page in (16, 1):
        far = (7 << 30) // 40 // 1024 * 1024
        for new in ((1, 2), (9, 20)):
            c = CacheCase((250, 300) if page == 16 else (15, 20), page, 2, 128, 128, seed=page)
            total, block = c.cache.num_pages, page * 128
            assert total <= 40

            def view(first):
                return buf[first:].as_strided((total, 2, page, 128), (far, block, 128, 1))
            c.cache = N.E4m3Cache(view(0), view(4 * block), c.cache.k_scale, c.cache.v_scale)
            c.upload()
            k, v = new_rows(sum(new), 2, 128, 128, "bf16", seed=3)
            c.append(new, k, v)
            c.run_append(new, k, v)
            c.check()
            q = torch.randn((sum(new), 8, 128), generator=torch.Generator().manual_seed(1))
            q = q.to(torch.bfloat16).cuda()
            qo = [0, new[0], sum(new)]
            plan = N.nvfp4kv_decode_plan(qo, c.indptr, c.last, 8, 2, 128, 128, page_size=page,
                                         causal=True, kernel=5)
            o, lse = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
            near = N.E4m3Cache(c.cache.k_data.contiguous(), c.cache.v_data.contiguous(),
                               c.cache.k_scale, c.cache.v_scale)
            o2, lse2 = N.nvfp4kv_e4m3_decode_run(plan, q, near, c.kv_indices)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            assert N.nvfp4kv_workspace_flags(plan) == 0
    words = buf.view(torch.bfloat16)
    x = words.as_strided((7, 3, 64), ((7 << 29) // 7, 64, 1))
    x.copy_(torch.randn((7, 3, 64), device="cuda"))
    plan = N.nvfp4kv_rope_plan(64)
    pos = i32([0, 5, 2, 9, 1000, 7, 3])
    want, _ = N.nvfp4kv_rope(plan, x.contiguous(), None, pos)
    N.nvfp4kv_rope(plan, x, None, pos, q_out=x)
    assert torch.equal(x, want)
    table = buf.view(torch.int32).as_strided((7, 4), ((7 << 28) // 7, 1))
    table.fill_(-1)
    out = N.StepTable.allocate(7, 16, 32)
    kv, qo = [20, 40, 3, 64, 1, 16, 17], [1, 2, 3, 1, 1, 1, 1]
    N.nvfp4kv_build_page_table(i32(kv), i32(kv), table, i32(range(90, 120)), None, out)
    near = torch.full((7, 4), -1, dtype=torch.int32, device="cuda")
    # (all tokens new: 161 rows do not fit 16)
    assert out.kv_indices.tolist() == [0] * 32
    out = N.StepTable.allocate(7, 200, 32)
    for t in (table, near):
        N.nvfp4kv_build_page_table(i32(kv), i32(kv), t, i32(range(90, 120)), None, out)
        N.nvfp4kv_build_page_table(i32(kv), i32(qo), t, i32([]), None, out)
    assert torch.equal(table, near) and int((near >= 90).sum()) == 14


def test_two_streams_with_their_own_workspaces():
    """Two calls in flight at once, each on its stream and workspace."""
    c, plan, o = attend_case((3000, 2000), (1, 1), 8, 2, 128, 128, seed=2)
    assert plan.info.split
    q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
    plans = [N.nvfp4kv_decode_plan([0, 1, 2], c.indptr, c.last, 8, 2, 128, 128, kernel=5)
             for _ in range(2)]
    want, wl = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [N.nvfp4kv_e4m3_decode_run(p, q, c.cache, c.kv_indices, stream=s)
           for _ in range(5) for p, s in zip(plans, streams)]
    torch.cuda.synchronize()
    for o2, l2 in got:
        assert torch.allclose(l2, wl, atol=1e-5) and torch.allclose(o2.float(), want.float(),
                                                                    atol=2.0 ** -7, rtol=2.0 ** -7)


@pytest.mark.parametrize("page,new", [(16, (20, 9)), (1, (20, 9)), (16, (300, 1)), (1, (1, 2))])
def test_append_rope_and_extend_in_a_graph(page, new):
    """Every form of the kernels that a step of prompts takes, captured once and
    replayed with other inputs: the same bits as the calls one by one."""
    c = CacheCase((700, 333), page, 2, 128, 128, seed=page + new[0])
    plan = N.nvfp4kv_decode_plan([0, new[0], sum(new)], c.indptr, c.last, 8, 2, 128, 128,
                                 page_size=page, causal=True, kernel=5, force_chunk_tokens=256)
    assert plan.info.split
    rope = N.nvfp4kv_rope_plan(128, 66)          # whole columns with halves inside them
    pos = i32(range(sum(new)))
    q = torch.zeros((sum(new), 8, 128), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((sum(new), 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    o = torch.zeros((sum(new), 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((sum(new), 8), device="cuda")
    flags, qo = new_flags(), i32([0, new[0], sum(new)])

    def step(o, lse):
        q2, k2 = N.nvfp4kv_rope(rope, q, k, pos)
        N.nvfp4kv_e4m3_append(c.cache, k2, v, qo, c.kv_indptr, c.kv_indices, c.last_page_len, flags)
        N.nvfp4kv_e4m3_decode_run(plan, q2, c.cache, c.kv_indices, out=o, lse=lse)
    step(o, lse)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(o, lse)
    g = torch.Generator().manual_seed(3)
    for _ in range(3):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        c.upload()
        graph.replay()
        torch.cuda.synchronize()
        codes, scales = c.cache.k_data.clone(), c.cache.v_scale.clone()
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        c.upload()
        step(o2, lse2)
        assert torch.equal(codes, c.cache.k_data) and torch.equal(scales, c.cache.v_scale)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert int(flags) == 0 and N.nvfp4kv_workspace_flags(plan) == 0


# ---- together ---------------------------------------------------------------------------
def test_decode_steps_together_in_a_graph():
    """A decode loop: the table from device lengths, rotary positions, the
    append and the attention, captured once and replayed for the steps that
    keep the page counts; every step against the references."""
    page, hq, hkv, d, steps = 16, 8, 2, 128, 4
    held = [21, 3, 35]                      # after each step +1; no page opens within 4 steps
    rng = np.random.default_rng(0)
    total = 12
    cache = N.E4m3Cache.allocate(total, hkv, d, d, page)
    free = rng.permutation(total).tolist()
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    out = N.StepTable.allocate(3, 64, 16)
    plan_rope = N.nvfp4kv_rope_plan(d, interleaved=False)
    freq = R.rope_frequencies(d, 10000.0)
    g = torch.Generator().manual_seed(0)
    rows = sum(held)
    kr = torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16).cuda()
    vr = torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16).cuda()
    flags = new_flags()
    # the prompts
    head = i32([0])
    N.nvfp4kv_build_page_table(i32(held), i32(held), table, i32(free), head, out,
                               device_flags=flags)
    _, kt = N.nvfp4kv_rope(plan_rope, None, kr, out.positions[:rows])
    N.nvfp4kv_e4m3_append(cache, kt, vr, out.qo_indptr, out.kv_indptr, out.kv_indices,
                          out.last_page_len, flags)
    head.copy_(out.free_head)
    k_all = [[R.to_np(kt[a:b])] for a, b in zip(np.cumsum([0] + held[:-1]), np.cumsum(held))]
    # buffers of the step
    kv_len, qo_len = i32(held), i32([1, 1, 1])
    q, k, v = (torch.zeros((3, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    q_rot, k_rot = torch.zeros_like(q), torch.zeros_like(k)
    kvp = np.concatenate([[0], np.cumsum([R.pages_of(n + 1, page) for n in held])])
    last = [n + 1 - (R.pages_of(n + 1, page) - 1) * page for n in held]
    plan = N.nvfp4kv_decode_plan([0, 1, 2, 3], kvp, last, hq, hkv, d, d, kernel=5,
                                 device_last_page_len=out.last_page_len)
    o = torch.zeros((3, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((3, hq), device="cuda")
    free_dev = i32(free)

    def step():
        kv_len.add_(1)
        N.nvfp4kv_build_page_table(kv_len, qo_len, table, free_dev, head, out,
                                   device_flags=flags)
        head.copy_(out.free_head)
        N.nvfp4kv_rope(plan_rope, q, k, out.positions[:3], q_out=q_rot, k_out=k_rot)
        N.nvfp4kv_e4m3_append(cache, k_rot, v, out.qo_indptr, out.kv_indptr, out.kv_indices,
                              out.last_page_len, flags)
        N.nvfp4kv_e4m3_decode_run(plan, q_rot, cache, out.kv_indices, out=o, lse=lse)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for s in range(steps):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        now = [n + s + 1 for n in held]
        assert kv_len.tolist() == now and int(flags) == 0
        assert out.positions.tolist()[:3] == [n - 1 for n in now]
        check_rope(q_rot, q, [n - 1 for n in now], d, False, freq, 1.0)
        codes = [x.cpu().numpy() for x in (cache.k_data, cache.v_data)]
        scale = [x.cpu().numpy() for x in (cache.k_scale, cache.v_scale)]
        idx = out.kv_indices.tolist()
        for b, n in enumerate(now):
            k_all[b].append(R.to_np(k_rot[b:b + 1]))
            pages = np.array(idx[kvp[b]:kvp[b + 1]])
            kk, vv = (R.dequantised(codes[i], scale[i], pages, n) for i in (0, 1))
            # a code is half an E4M3 step off, and once more for each time its
            # page's scale grew (at most half a step of the new scale each)
            keys = np.concatenate(k_all[b]).transpose(1, 0, 2)
            big = np.repeat(scale[0][pages].T.astype(np.float64), page, 1)[:, :n, None]
            assert (np.abs(kk - keys) <= np.abs(keys) * 2.0 ** -4 * 1.01 + big * 2.0 ** -9).all()
            vs = np.repeat(scale[1][pages].T.astype(np.float64), page, 1)[:, :n]
            ref, rl, mean, reach, floor = R.attention(R.to_np(q_rot[b:b + 1]), kk, vv, vs,
                                                      float(np.float32(1 / math.sqrt(d))), False)
            delta = (d * 2.0 ** -23 * reach + 2.0 ** -21)[..., None]
            tol = 2.0 ** -8 * np.abs(ref) + (mean * (2.0 ** -11 + 2.0 ** -19 + 2 * delta)
                                             + 2.0 ** -25 * floor) * 1.01
            assert (np.abs(R.to_np(o[b:b + 1]) - ref) <= tol).all()
            assert (np.abs(R.to_np(lse[b:b + 1]) - rl) <= delta[..., 0] + 1e-5).all()
    assert N.nvfp4kv_workspace_flags(plan) == 0
