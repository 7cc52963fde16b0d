"""Every form in which the tree attention runs a plan, named by nvfp4kv_tree_form, against 64
bits; the step's tokens appended in the same launch, bit for bit; row sums.

Tolerances (of a row that sees L tokens): a weight is rounded to f16 for its product, 2^-11 of
it or 2^-25 of the row's largest; the row sum is one of unrounded weights.  A score's sum of
products errs by Dk 2^-23 of sum |q k| at most, what follows (scale, maximum, 2^x) by 2^-21;
L / 16 products of 16 tokens add up by 2^-23 each, a quarter of the row's weights by 2^-24
each; states are joined by weights out of log-sum-exps, 2^-22 of those."""
import math

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
import step_reference as R
import test_gpu_tree_run as TR
import tree_reference as T

pytestmark = pytest.mark.gpu


def check_rows(got, got_lse, want, dk, tokens, dtype):
    ref, rl, mean, reach, floor = want
    eps = torch.finfo(dtype).eps / 2
    none = np.isinf(rl)
    assert np.array_equal(got_lse == -np.inf, none) and (got[none] == 0).all()
    delta = dk * 2.0 ** -23 * reach + 2.0 ** -21
    sums = tokens * 2.0 ** -26 + 2.0 ** -19
    size = np.where(none, 0.0, np.abs(rl)) + 32
    tol = (eps * np.abs(ref) + (mean * (2.0 ** -11 + 2 * sums + (2 * delta + size * 2.0 ** -22)
                                        [..., None]) + 2.0 ** -25 * floor) * (1 + eps)
           + float(torch.finfo(dtype).smallest_normal) * eps)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    lerr = np.abs(got_lse - np.where(none, 0.0, rl))[~none]
    ltol = (delta + sums + size * 2.0 ** -22)[~none]
    assert (lerr <= ltol).all(), (float(lerr.max()), float((lerr / ltol).max()))


def run(kv, new, hq, hkv, dk, dv, page=16, layout="HND", out="bf16", seed=0, only=None,
        live=False, **plan_kw):
    """One call, checked (the requests of `only`); its plan's form."""
    c = T.Nvfp4Case(kv, page, hkv, dk, dv, layout, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(new), hq, dk), generator=gen).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(seed)
    words = (max(new) + 31) // 32
    masks = [T.mask_words(T.ancestors(T.random_parents(rng, n)), words) for n in new]
    qo = np.concatenate([[0], np.cumsum(new)])
    last = [page] * len(kv) if live else c.last
    if live:
        plan_kw["device_last_page_len"] = c.last_page_len
    plan = N.nvfp4kv_decode_plan(qo, c.indptr, last, hq, hkv, dk, dv, page_size=page,
                                 out_dtype=TR.DT[out], **plan_kw)
    mask = TR.i32(np.concatenate(masks))
    o, lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask)
    o2, lse2 = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    got, gl = R.to_np(o), R.to_np(lse)
    for b, n in enumerate(new):
        if only is not None and b not in only:
            continue
        rows = slice(int(qo[b]), int(qo[b + 1]))
        want = T.tree_attention(R.to_np(q[rows]), c.dense(0, b), c.dense(1, b),
                                TR.bits(masks[b], n, kv[b]), 1 / math.sqrt(dk))
        check_rows(got[rows], gl[rows], want, dk, kv[b], TR.DT[out])
    return N.nvfp4kv_tree_form(plan)


def assert_form(form, **want):
    assert {k: form[k] for k in want} == want, form


DIMS = [(64, 64, 1), (128, 128, 1), (256, 128, 1), (256, 256, 2), (512, 256, 2)]


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("page,out", [(16, "bf16"), (1, "f16")])
@pytest.mark.parametrize("chunk", [64, 176])
def test_folded_units_of_the_ctas_that_share_value_dims(dk, dv, value_ctas, page, out, chunk):
    """No room for clusters of tokens: each unit's partial states come from the CTAs of its
    value dims alone.  Rows in one block (fewer than 64, and more), and in two."""
    form = run((300, 1, 17, 1111), (12, 1, 17, 40), 8, 2, dk, dv, page=page, out=out, kernel=1,
               force_chunk_tokens=chunk, num_sms=1, seed=dk + chunk)
    assert_form(form, block_rows=128, row_blocks=2, cluster_ctas=value_ctas,
                value_ctas=value_ctas, whole_requests=0, folded=1)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("new", [10, 20, 40])  # rows held twice, once, in two blocks
@pytest.mark.parametrize("num_sms,ctas", [(0, 8), (14, 4), (7, 2)])  # (of a row block)
def test_folded_units_of_clusters(dk, dv, value_ctas, new, num_sms, ctas):
    """A cluster joins its CTAs' states of a unit's tokens into the unit's partial state, and
    the last unit folds three of them."""
    if ctas == 2 and dk > 128:
        pytest.skip("two CTAs of one tile size: whole requests, or no cluster of tokens")
    blocks = -(-new * 4 // 128)
    form = run((8229,), (new,), 4, 1, dk, dv, kernel=1, force_chunk_tokens=4096,
               num_sms=num_sms * blocks, layout="NHD", out="f16", seed=dk + new)
    assert_form(form, block_rows=128, row_blocks=blocks, cluster_ctas=ctas,
                value_ctas=value_ctas, whole_requests=0, folded=1)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("new", [10, 20, 40])
def test_whole_requests(dk, dv, value_ctas, new):
    """All units of a request and kv head in one cluster."""
    form = run((2200, 1500), (new, 7), 4, 1, dk, dv, kernel=1, force_chunk_tokens=64,
               seed=dk + new)
    assert_form(form, block_rows=128, cluster_ctas=8, value_ctas=value_ctas, whole_requests=1,
                longest_first=0, folded=0)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
def test_units_that_are_not_split(dk, dv, value_ctas):
    form = run((300, 50, 129), (20, 33, 5), 4, 1, dk, dv, kernel=1, disable_split=True, num_sms=1,
               seed=dk)
    assert_form(form, block_rows=128, cluster_ctas=value_ctas, whole_requests=0, folded=0)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("new,rows", [((2, 1), 8), ((4, 3), 16)])
@pytest.mark.parametrize("chunk", [0, 64])
def test_up_to_16_rows(dk, dv, value_ctas, new, rows, chunk):
    form = run((300, 1111), new, 4, 1, dk, dv, kernel=1, force_chunk_tokens=chunk, num_sms=1,
               seed=dk + rows)
    assert_form(form, block_rows=rows, row_blocks=1, cluster_ctas=1, whole_requests=0)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
def test_longest_first(dk, dv, value_ctas):
    """One long request among short ones, equal ones and one without rows."""
    rng = np.random.default_rng(dk)
    kv = [int(x) for x in rng.integers(300, 600, 16)]
    kv[5], kv[9] = 8192, kv[8]
    form = run(kv, [9] * 15 + [0], 16, 4, dk, dv, kernel=1, disable_split=True, seed=dk,
               only=(0, 5, 8, 9, 14))
    assert_form(form, block_rows=128, value_ctas=value_ctas, whole_requests=1, longest_first=1,
                folded=0)


@pytest.mark.parametrize("dk,dv,hq,hkv,new,batch,most", [
    (128, 128, 16, 2, 10, 60, 5000), (512, 256, 16, 2, 8, 30, 8192)])
def test_uneven_batches_run_longest_first(dk, dv, hq, hkv, new, batch, most):
    """The batches of test_uneven_batches_in_several_waves (where that of 64 / 64 heads runs
    unit by unit)."""
    rng = np.random.default_rng(dk)
    kv = [int(x) for x in rng.integers(300, most, batch - 3)] + [1500, 1500, 77]
    n = [new] * (batch - 1) + [0]
    npages = [R.pages_of(x, 16) for x in kv]
    plan = N.nvfp4kv_decode_plan(
        np.concatenate([[0], np.cumsum(n)]), np.concatenate([[0], np.cumsum(npages)]),
        [a - (p - 1) * 16 for a, p in zip(kv, npages)], hq, hkv, dk, dv)
    assert_form(N.nvfp4kv_tree_form(plan), block_rows=128, whole_requests=1, longest_first=1)


def test_form_of_plans_without_one():
    c = T.Nvfp4Case((100,), 16, 2, 128, 128, seed=14)
    plan = N.nvfp4kv_decode_plan([0, 0], c.indptr, c.last, 8, 2, 128, 128)
    assert not any(N.nvfp4kv_tree_form(plan).values())
    plan = N.nvfp4kv_decode_plan([0, 6], c.indptr, c.last, 8, 2, 128, 128, kernel=2)
    with pytest.raises(N.NvFp4KvError):
        N.nvfp4kv_tree_form(plan)


# the forms: requests' tokens, their nodes, the plan (see the tests above)
FORMS = [
    ((37, 300, 30), (2, 2, 1), dict(num_sms=1)), ((37, 300, 30), (4, 3, 4), dict(num_sms=1)),
    ((37, 300, 30), (7, 33, 30), dict()), ((300, 1111), (17, 40), dict(num_sms=1)),
    ((300, 1111), (17, 40), dict(num_sms=1, disable_split=True)), ((8229,), (20,), dict()),
    ((8229,), (40,), dict(num_sms=14)), ((2200, 1500), (10, 7), dict())]


@pytest.mark.parametrize("dk,dv", [(128, 128), (512, 256)])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("at", range(len(FORMS)))
def test_new_tokens_in_the_same_launch_change_no_bit(dk, dv, page, at):
    """Cache, out and lse are those of nvfp4kv_quantize_append and a call without new tokens:
    a CTA that read another's token before it was there would read the NaN scales that the
    cache holds in the new tokens' slots."""
    kv, new, kw = FORMS[at]
    if not kw.get("disable_split"):
        kw = dict(kw, force_chunk_tokens=4096 if max(kv) > 4096 else 64)
    hkv, seed = 1, 40 + at
    cases = [T.Nvfp4Case(kv, page, hkv, dk, dv, seed=seed) for _ in range(2)]
    for c in cases:
        for sf in c.sf:
            for b, (n, m) in enumerate(zip(new, kv)):
                for t in range(m - n, m):
                    sf[c.pages(b)[t // page], :, t % page] = 0x7F
        c.upload()
    one, two = cases
    g = torch.Generator().manual_seed(seed)
    rows = sum(new)
    k, v = (torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16).cuda() for d in (dk, dv))
    q = torch.randn((rows, 4 * hkv, dk), generator=g).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(seed)
    mask = TR.i32(np.concatenate([T.mask_words(T.ancestors(T.random_parents(rng, n)), 2)
                                  for n in new]))
    idx = TR.i32([b for b, n in enumerate(new) for _ in range(n)])
    pos = TR.i32([t for n, m in zip(new, kv) for t in range(m - n, m)])
    plan = N.nvfp4kv_decode_plan(np.concatenate([[0], np.cumsum(new)]), one.indptr, one.last,
                                 4 * hkv, hkv, dk, dv, page_size=page, kernel=1, **kw)
    got = N.nvfp4kv_tree_run(plan, q, one.cache, one.kv_indices, mask, new_k=k, new_v=v)
    N.nvfp4kv_quantize_append(two.cache, k, v, idx, pos, two.kv_indices, two.kv_indptr,
                              two.last_page_len)
    want = N.nvfp4kv_tree_run(plan, q, two.cache, two.kv_indices, mask)
    assert N.nvfp4kv_workspace_flags(plan) == 0
    mine, theirs = one.download(), two.download()
    for n in mine:
        assert np.array_equal(mine[n], theirs[n]), n
    for a, b in zip(got, want):
        assert torch.isfinite(b.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("at", range(len(FORMS)))
def test_outputs_that_are_4_byte_aligned(dk, dv, value_ctas, at):
    """An output may start at any multiple of 4 bytes, as for the causal attention; nothing is
    written around it.  One that is not is refused."""
    kv, new, kw = FORMS[at]
    if not kw.get("disable_split"):
        kw = dict(kw, force_chunk_tokens=4096 if max(kv) > 4096 else 64)
    c = T.Nvfp4Case(kv, 16, 1, dk, dv, seed=at)
    q = torch.randn((sum(new), 4, dk), generator=torch.Generator().manual_seed(at))
    q = q.to(torch.bfloat16).cuda()
    mask = TR.i32(np.full((sum(new), 2), -1))
    plan = N.nvfp4kv_decode_plan(np.concatenate([[0], np.cumsum(new)]), c.indptr, c.last, 4, 1,
                                 dk, dv, kernel=1, **kw)
    want, want_lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask)
    for shift in (2, 6):
        wide = torch.full((want.numel() + 8,), 9.0, dtype=torch.bfloat16).cuda()
        out = wide[shift:shift + want.numel()].view(want.shape)
        _, lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask, out=out)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (wide[:shift] == 9).all() and (wide[shift + want.numel():] == 9).all()
    with pytest.raises(N.NvFp4KvError):
        N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, mask,
                           out=wide[1:1 + want.numel()].view(want.shape))
    assert N.nvfp4kv_workspace_flags(plan) == 0


@pytest.mark.parametrize("dk,dv,value_ctas", DIMS)
@pytest.mark.parametrize("at", range(len(FORMS)))
@pytest.mark.parametrize("page", [16, 1])
def test_live_lengths_in_every_form(dk, dv, value_ctas, at, page):
    """A plan made for full last pages, run with the lengths that the device holds."""
    kv, new, kw = FORMS[at]
    if not kw.get("disable_split"):
        kw = dict(kw, force_chunk_tokens=4096 if max(kv) > 4096 else 64)
    run(kv, new, 4, 1, dk, dv, page=page, kernel=1, seed=at + dk, live=True, only=(0, 1), **kw)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (512, 256)])
@pytest.mark.parametrize("hq", [2, 4, 8, 40])
@pytest.mark.parametrize("chunk", [0, 16])
def test_row_sums_are_those_of_unrounded_weights(dk, dv, hq, chunk):
    """Queries of one dim: a score is one product, exact but for its scale (2^-23 of it) and
    2^x (2^-22), so that lse shows a row sum of weights rounded to f16."""
    kv, new = (3, 9, 40), (1, 2, 2)
    c = T.Nvfp4Case(kv, 16, 1, dk, dv, seed=dk + hq)
    rng = np.random.default_rng(hq)
    q = np.zeros((sum(new), hq, dk))
    q[:, :, 5] = rng.uniform(1, 2.5, q.shape[:2]) * math.sqrt(dk)
    q = torch.tensor(q).to(torch.bfloat16).cuda()
    masks = [T.mask_words(T.ancestors(T.random_parents(rng, n)), 1) for n in new]
    qo = np.concatenate([[0], np.cumsum(new)])
    plan = N.nvfp4kv_decode_plan(qo, c.indptr, c.last, hq, 1, dk, dv, kernel=1, num_sms=1,
                                 force_chunk_tokens=chunk, disable_split=not chunk)
    _, lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, TR.i32(np.concatenate(masks)))
    assert N.nvfp4kv_workspace_flags(plan) == 0
    gl, seen = R.to_np(lse), False
    for b, n in enumerate(new):
        k, hide = c.dense(0, b)[0], TR.bits(masks[b], n, kv[b])
        for i in range(n):
            for h in range(hq):
                row = int(qo[b]) + i
                s = k[~hide[i], 5] * float(q[row, h, 5]) / math.sqrt(dk)
                want = s.max() + math.log(np.exp(s - s.max()).sum())
                tol = np.abs(s).max() * 2.0 ** -20 + 2.0 ** -19 + abs(want) * 2.0 ** -22
                assert abs(gl[row, h] - want) <= tol, (b, i, h)
                rounded = np.exp(s - s.max()).astype(np.float16).astype(float).sum()
                seen |= abs(s.max() + math.log(rounded) - want) > 4 * tol
    assert seen  # (a sum of rounded weights would not have passed)
