"""Host-only checks of the serving-step entry points: argument validation
before anything is enqueued (so no GPU is needed), the frequency table, the
plan of the E4M3 cache and the references that the GPU tests use."""
import ctypes as C
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import step_reference as R
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib

INVALID, UNSUPPORTED = _lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED
BUF = 1 << 24  # a pointer that is never read


# ---- references -----------------------------------------------------------------
def test_reference_codes_against_torch():
    x = torch.arange(-2**15, 2**15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[x.isfinite()].float()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_codes(x.numpy()), want)
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.VALUES, v, equal_nan=True)
    mids = (R.VALUES[:0x7E] + R.VALUES[1:0x7F]) / 2  # ties go to the even code
    assert all(int(c) % 2 == 0 for c in R.e4m3_codes(mids))


def test_reference_scale():
    assert R.scale_of(0.0) == 2.0 ** -64 and R.scale_of(448.0) == 1.0
    assert R.scale_of(448.5) == 2.0 and R.scale_of(224.0) == 0.5 and R.scale_of(1e38) == 2.0 ** 64


# ---- the frequency table -----------------------------------------------------------
def frequencies(rotary, **kw):
    o = dict(base=10000.0, factor=1.0, original_max_position=0, low_rotations=1.0,
             high_rotations=32.0)
    o.update(kw)
    out = np.zeros(max(rotary // 2, 1), dtype=np.uint64)
    st = _lib.load().nvfp4kv_rope_frequencies(rotary, _lib.RopeOptions(**o), out.ctypes.data)
    return st, out


@pytest.mark.parametrize("rotary", [2, 64, 126, 512])
@pytest.mark.parametrize("kw", [{}, dict(factor=4.0), dict(
    base=500000.0, factor=32.0, original_max_position=8192, high_rotations=4.0)])
def test_frequencies(rotary, kw):
    st, got = frequencies(rotary, **kw)
    assert st == 0
    want = R.rope_frequencies(rotary, kw.get("base", 10000.0), kw.get("factor", 1.0),
                              kw.get("original_max_position", 0), 1.0,
                              kw.get("high_rotations", 32.0))
    for g, w in zip(got.tolist(), want):
        turns = Fraction(g, 1 << 64)
        # pow, pi and a few products in 64 bits: relative 2^-50, and one unit of 2^-64
        exact = Fraction(w) / Fraction(2 * math.pi)
        assert abs(turns - exact) <= exact * Fraction(1, 1 << 50) + Fraction(1, 1 << 64)


@pytest.mark.parametrize("rotary,kw,status", [
    (0, {}, UNSUPPORTED), (3, {}, UNSUPPORTED), (514, {}, UNSUPPORTED),
    (64, dict(base=1.0), INVALID), (64, dict(base=math.nan), INVALID),
    (64, dict(factor=0.0), INVALID), (64, dict(factor=math.inf), INVALID),
    (64, dict(original_max_position=-1), INVALID),
    (64, dict(original_max_position=8, low_rotations=4.0, high_rotations=4.0), INVALID),
    (64, dict(original_max_position=8, low_rotations=math.nan), INVALID)])
def test_frequencies_refuse(rotary, kw, status):
    assert frequencies(rotary, **kw)[0] == status


# ---- the page table ------------------------------------------------------------------
def build_status(**over):
    a = dict(kv_len=BUF, qo_len=BUF, batch=2, page_size=16, block_table=BUF, stride=8, width=8,
             free=BUF, num_free=4, head=BUF, flags=None)
    s = dict(qo_indptr=BUF, kv_indptr=BUF, last_page_len=BUF, kv_indices=BUF, batch_idx=BUF,
             positions=BUF, slot_map=BUF, free_head=BUF + 64, max_pages=4, max_tokens=4)
    for k, v in over.items():
        (s if k in s else a)[k] = v
    t = _lib.StepTableStruct(**s)
    return _lib.load().nvfp4kv_build_page_table(
        a["kv_len"], a["qo_len"], a["batch"], a["page_size"], a["block_table"], a["stride"],
        a["width"], a["free"], a["num_free"], a["head"], t, a["flags"], None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
    (dict(page_size=1 << 17), UNSUPPORTED), (dict(kv_len=None), INVALID),
    (dict(qo_len=None), INVALID), (dict(block_table=None), INVALID), (dict(stride=7), INVALID),
    (dict(width=-1), INVALID), (dict(free=None), INVALID), (dict(num_free=-1), INVALID),
    (dict(free_head=BUF), INVALID), (dict(free_head=None), INVALID),
    (dict(qo_indptr=None), INVALID), (dict(kv_indptr=None), INVALID),
    (dict(last_page_len=None), INVALID), (dict(kv_indices=None), INVALID),
    (dict(batch_idx=None), INVALID), (dict(positions=None), INVALID),
    (dict(max_pages=-1), INVALID), (dict(max_tokens=-1), INVALID),
    (dict(slot_map=BUF + 4), INVALID)])
def test_page_table_refuses(over, status):
    assert build_status(**over) == status
    assert _lib.load().nvfp4kv_last_error_detail()


def test_step_table_checks_its_tensors():
    t = N.StepTable.allocate(3, 8, 9, device="cpu")
    assert t.batch == 3 and t._struct.max_tokens == 8 and t._struct.max_pages == 9
    ok = [t.qo_indptr, t.kv_indptr, t.last_page_len, t.kv_indices, t.batch_idx, t.positions,
          t.slot_map, t.free_head]
    for i, bad in ((0, t.qo_indptr.long()), (1, t.kv_indptr[:3]), (5, t.positions[:7]),
                   (6, t.slot_map.int()), (3, t.kv_indices[::2]), (7, t.free_head[:0])):
        with pytest.raises(ValueError):
            N.StepTable(*(ok[:i] + [bad] + ok[i + 1:]))


# ---- rotary positions -------------------------------------------------------------------
def rope_status(**over):
    a = dict(q=BUF, qst=256, qsh=128, qo=2 * BUF, qost=256, qosh=128, hq=2, k=3 * BUF, kst=256,
             ksh=128, ko=4 * BUF, kost=256, kosh=128, hkv=2, n=1, pos=BUF, dim=128, rot=128,
             inter=0, dtype=0, freq=BUF, attn=1.0)
    a.update(over)
    return _lib.load().nvfp4kv_rope(
        a["q"], a["qst"], a["qsh"], a["qo"], a["qost"], a["qosh"], a["hq"], a["k"], a["kst"],
        a["ksh"], a["ko"], a["kost"], a["kosh"], a["hkv"], a["n"], a["pos"], a["dim"], a["rot"],
        a["inter"], a["dtype"], a["freq"], a["attn"], None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), INVALID), (dict(hq=-1), INVALID), (dict(hkv=-1), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(dim=100), UNSUPPORTED),
    (dict(dim=520), UNSUPPORTED), (dict(rot=130), UNSUPPORTED), (dict(rot=3), UNSUPPORTED),
    (dict(rot=0), UNSUPPORTED), (dict(attn=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
    (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(freq=BUF + 4), INVALID),
    (dict(q=BUF + 8), INVALID), (dict(qst=260), INVALID), (dict(kosh=-128), INVALID),
    (dict(qosh=64), INVALID), (dict(n=2, kost=64), INVALID), (dict(n=2, qost=128), INVALID),
    (dict(n=3, kost=128, kosh=256), INVALID),
    (dict(qo=BUF, qost=512), INVALID)])
def test_rope_refuses(over, status):
    assert rope_status(**over) == status


def test_rope_accepts_nothing_to_do():
    assert rope_status(n=0, q=None, k=None, pos=None) == 0
    assert rope_status(hq=0, hkv=0) == 0


def test_rope_plan():
    p = N.nvfp4kv_rope_plan(128, 64, device="cpu")
    assert p.freq.numel() == 32 and p.freq.dtype == torch.int64
    for bad in (0, 130):
        with pytest.raises(ValueError):
            N.nvfp4kv_rope_plan(128, bad, device="cpu")
    with pytest.raises(N.NvFp4KvError):
        N.nvfp4kv_rope_plan(128, 63, device="cpu")


# ---- the E4M3 cache -------------------------------------------------------------------------
def fake_cache(dk=128, dv=128, heads=2, **over):
    s = _lib.E4m3CacheStruct()
    s.k_data, s.v_data, s.k_scale, s.v_scale = BUF, 2 * BUF, 3 * BUF, 4 * BUF
    for pre, d in (("k", dk), ("v", dv)):
        setattr(s, pre + "_stride_page", 16 * heads * d)
        setattr(s, pre + "_stride_head", 16 * d)
        setattr(s, pre + "_stride_slot", d)
        setattr(s, pre + "_scale_stride_page", 4 * heads)
        setattr(s, pre + "_scale_stride_head", 4)
    s.num_pages, s.page_size, s.num_kv_heads = 10, 16, heads
    s.head_dim_qk, s.head_dim_vo = dk, dv
    for k, v in over.items():
        setattr(s, k, v)
    return s


BAD_CACHES = [
    (dict(k_data=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(head_dim_qk=100), UNSUPPORTED),
    (dict(head_dim_vo=544), UNSUPPORTED), (dict(head_dim_vo=0), UNSUPPORTED),
    (dict(k_stride_slot=136), INVALID), (dict(v_stride_head=-16), INVALID),
    (dict(k_stride_slot=64), INVALID), (dict(v_stride_page=0), INVALID),
    (dict(k_scale_stride_page=6), INVALID), (dict(v_scale_stride_head=0), INVALID),
    (dict(k_stride_page=256), INVALID), (dict(v_stride_head=128), INVALID),
    (dict(k_scale_stride_page=4), INVALID),
    (dict(k_scale_stride_page=0), INVALID), (dict(k_data=BUF + 8), INVALID),
    (dict(v_scale=BUF + 2), INVALID)]


def append_status(cache, **over):
    a = dict(k=BUF, kst=256, ksh=128, v=BUF, vst=256, vsh=128, dtype=0, rows=1, qo=BUF, kvp=BUF,
             idx=BUF, last=BUF, batch=1)
    a.update(over)
    return _lib.load().nvfp4kv_e4m3_append(
        cache, a["k"], a["kst"], a["ksh"], a["v"], a["vst"], a["vsh"], a["dtype"], a["rows"],
        a["qo"], a["kvp"], a["idx"], a["last"], a["batch"], None, None)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_e4m3_cache_refusals(over, status):
    assert append_status(fake_cache(**over)) == status
    info = _lib.PlanInfo()
    assert _lib.load().nvfp4kv_e4m3_decode_run(
        info, BUF, 256, 128, 0, fake_cache(**over), BUF, 0.0, BUF, 1 << 20, BUF, None,
        None) == status


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), INVALID), (dict(batch=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(qo=None), INVALID),
    (dict(kvp=None), INVALID), (dict(idx=None), INVALID), (dict(last=None), INVALID),
    (dict(k=BUF + 8), INVALID), (dict(kst=252), INVALID), (dict(vsh=-8), INVALID)])
def test_append_refuses(over, status):
    assert append_status(fake_cache(), **over) == status


def test_append_accepts_nothing_to_do():
    assert append_status(fake_cache(), rows=0, k=None) == 0
    assert append_status(fake_cache(), batch=0, qo=None) == 0


def test_e4m3_cache_checks_its_tensors():
    c = N.E4m3Cache.allocate(4, 2, 64, 128, layout="NHD", device="cpu")
    assert c._struct.k_stride_page == 16 * 2 * 64 and c._struct.k_stride_slot == 128
    assert c._struct.k_stride_head == 64 and c._struct.v_scale_stride_page == 8
    k, v, ks, vs = c.k_data, c.v_data, c.k_scale, c.v_scale
    for bad in ((k.int(), v, ks, vs), (k, v[:3], ks, vs), (k, v, ks.double(), vs),
                (k, v, ks, vs[:, :1]), (k.transpose(2, 3), v, ks, vs), (k[0], v, ks, vs)):
        with pytest.raises((ValueError, IndexError)):
            N.E4m3Cache(*bad)
    with pytest.raises(ValueError):
        N.E4m3Cache.allocate(4, 2, 64, 64, layout="DHN", device="cpu")


def plan5(qo, kvp, last, hq=8, hkv=2, dk=128, dv=128, **kw):
    return N.nvfp4kv_decode_plan(qo, kvp, last, hq, hkv, dk, dv, kernel=5, num_sms=152,
                                 ctas_per_sm=3, allocate=False, **kw)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 128), (256, 256), (512, 256)])
@pytest.mark.parametrize("page", [16, 1])
def test_plan(dk, dv, page):
    n = 100 if page == 1 else 7
    p = plan5([0, 1, 3], [0, n, 2 * n], [1, 1], dk=dk, dv=dv, page_size=page, causal=True)
    assert p.info.kernel == 5 and p.info.num_units >= 4 and p.info.total_qo_rows == 3
    assert p.info.rows_per_block * p.info.row_blocks >= 8


def test_plan_refuses_other_dims():
    with pytest.raises(N.NvFp4KvError) as e:
        plan5([0, 1], [0, 2], [1], dk=128, dv=256)
    assert e.value.status == UNSUPPORTED
    with pytest.raises(N.NvFp4KvError) as e:
        N.nvfp4kv_decode_plan([0, 1], [0, 2], [1], 8, 2, 128, 128, kernel=6, num_sms=152,
                              ctas_per_sm=3, allocate=False)
    assert e.value.status == INVALID


def test_runs_refuse_plans_of_the_other_cache():
    L = _lib.load()
    p5 = plan5([0, 1], [0, 2], [1])
    p1 = N.nvfp4kv_decode_plan([0, 1], [0, 2], [1], 8, 2, 128, 128, kernel=1, num_sms=152,
                               ctas_per_sm=3, allocate=False)
    e4m3 = fake_cache()
    tail = (BUF, 0.0, BUF, 1 << 30, BUF, None, None)
    run = lambda info, c: L.nvfp4kv_e4m3_decode_run(info, BUF, 256, 128, 0, c, *tail)  # noqa: E731
    assert run(p1.info, e4m3) == _lib.ERR_PLAN_MISMATCH
    assert run(p5.info, fake_cache(heads=1)) == _lib.ERR_PLAN_MISMATCH
    assert run(p5.info, fake_cache(dk=64, dv=64)) == _lib.ERR_PLAN_MISMATCH
    assert run(_lib.PlanInfo(), e4m3) == INVALID
    assert L.nvfp4kv_e4m3_decode_run(p5.info, BUF, 256, 128, 2, e4m3, *tail) == UNSUPPORTED
    s = _lib.PagedCacheStruct()
    s.k_data, s.v_data, s.k_sf, s.v_sf = BUF, 2 * BUF, 3 * BUF, 4 * BUF
    for pre, row in (("k", 64), ("v", 64), ("k_sf", 8), ("v_sf", 8)):
        setattr(s, pre + "_stride_page", 16 * 2 * row)
        setattr(s, pre + "_stride_slot", row)
        setattr(s, pre + "_stride_head", 16 * row)
    s.num_pages, s.page_size, s.num_kv_heads = 10, 16, 2
    s.head_dim_qk = s.head_dim_vo = 128
    s.k_global_scale = s.v_global_scale = 1.0
    for fn in (L.nvfp4kv_decode_run, L.nvfp4kv_decode_attend):
        assert fn(C.byref(p5.info), BUF, 256, 128, C.byref(s), *tail) == _lib.ERR_PLAN_MISMATCH


@pytest.mark.parametrize("kv,new,split", [
    ([8000] * 32, [16] * 32, False),                       # even: whole requests
    ([1000 + 1526 * i for i in range(20)], [16] * 20, True),   # a long tail on 152 SMs
    ([100, 60000] + [4000] * 11, [16] * 13, True),
    ([300] * 400, [16] * 400, False),
    ([30000] + [200] * 60, [0] + [20] * 60, None)])
def test_extend_plan_evens_out_the_sms(kv, new, split):
    """Plans of many rows a kv head may take several waves; every page of every
    request with rows is in one unit of each kv head, and the busiest SM's work
    (tiles and 12 a unit, longest first) is not above that of whole requests."""
    qo = np.concatenate([[0], np.cumsum(new)])
    np_ = [-(-n // 16) for n in kv]
    kvp = np.concatenate([[0], np.cumsum(np_)])
    last = [n - 16 * (p - 1) for n, p in zip(kv, np_)]
    plan = N.nvfp4kv_decode_plan(qo, kvp, last, 32, 8, 128, 128, causal=True, kernel=5,
                                 num_sms=152, ctas_per_sm=1, allocate=False)
    i = plan.info
    if split is not None:
        assert bool(i.split) == split
    units = plan.host[:48 * i.num_units].numpy().view(np.int32).reshape(i.num_units, -1)
    assert units.shape[1] == 12
    field = {n: units[:, k] for k, n in enumerate(
        ["b", "h", "page_begin", "pages", "tok_begin", "kv_len", "qo_begin", "qo_len", "split",
         "splits", "base", "pair"])}
    for b, n in enumerate(new):
        for h in range(8):
            at = (field["b"] == b) & (field["h"] == h)
            assert bool(at.any()) == (n > 0)
            spans = sorted(zip(field["page_begin"][at], field["pages"][at]))
            end = kvp[b]
            for begin, pages in spans:
                assert begin == end and (field["tok_begin"][at] % 128 == 0).all()
                end += pages
            assert end == (kvp[b + 1] if n else kvp[b])

    def busiest(tiles):
        sms = [0] * 152
        for t in sorted(tiles, reverse=True):
            k = sms.index(min(sms))
            sms[k] += t + 12
        return max(sms)
    whole = [-(-p // 8) for p, n in zip(np_, new) if n for _ in range(8)]
    assert busiest([-(-p // 8) for p in field["pages"]]) <= busiest(whole)
