"""Host-only checks of the entry points of a step that verifies drafted tokens: what the
library and its binding refuse before anything is launched."""
import ctypes as C

import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
from nvfp4_paged_kv_nvfp4kv_gb300 import workloads as W

OK, INVALID, UNSUPPORTED = 0, 1, 2


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def call(name, *args):
    return getattr(_lib.load(), name)(*args)


# ---- norms with rotary positions ----------------------------------------------------
def norm_rope(**change):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    a = dict(q=x, qs=(128, 64), q_out=x, qos=(128, 64), hq=2, k=None, ks=(0, 0), k_out=None,
             kos=(0, 0), hk=0, n=0, pos=i32(4), dim=64, rot=64, inter=0, dtype=0,
             freq=torch.zeros(32, dtype=torch.int64), factor=1.0, qw=w, kw=None, wt=0, off=0.0,
             eps=1e-6)
    a.update(change)
    p = lambda t: None if t is None else (t if isinstance(t, int) else t.data_ptr())  # noqa: E731
    return call("nvfp4kv_norm_rope", p(a["q"]), *a["qs"], p(a["q_out"]), *a["qos"], a["hq"],
                p(a["k"]), *a["ks"], p(a["k_out"]), *a["kos"], a["hk"], a["n"], p(a["pos"]),
                a["dim"], a["rot"], a["inter"], a["dtype"], p(a["freq"]), a["factor"], p(a["qw"]),
                p(a["kw"]), a["wt"], a["off"], a["eps"], None)


def test_norm_rope_refusals():
    assert norm_rope() == OK  # no tokens: nothing to do
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=1e30), dict(eps=-1e-6),
                dict(off=float("inf")), dict(n=4, qw=None), dict(n=-1),
                dict(n=4, qw=torch.ones(80, dtype=torch.bfloat16)[1:]),
                dict(n=4, qos=(64, 64)), dict(n=4, q_out=None), dict(factor=float("nan"))):
        assert norm_rope(**bad) == INVALID, bad
    for bad in (dict(wt=1), dict(wt=3), dict(dtype=2), dict(dim=60), dict(rot=66), dict(rot=3),
                dict(dim=520)):
        assert norm_rope(**bad) == UNSUPPORTED, bad


# ---- tree masks -----------------------------------------------------------------------
def test_tree_masks_refusals():
    p, qo, kv, m, pos = i32(4), i32(2), i32(1), i32(4, 1), i32(4)
    args = [p.data_ptr(), qo.data_ptr(), kv.data_ptr(), 1, 4, 1, m.data_ptr(), pos.data_ptr(),
            None, None]

    def st(**change):
        a = list(args)
        for k, v in change.items():
            a[int(k[1:])] = v
        return call("nvfp4kv_tree_masks", *a)
    assert st(_3=0) == OK and st(_4=0) == OK
    for bad in (dict(_3=-1), dict(_4=-1), dict(_0=None), dict(_1=None), dict(_2=None),
                dict(_6=None), dict(_7=None)):
        assert st(**bad) == INVALID, bad
    for bad in (dict(_5=0), dict(_5=33), dict(_5=-1)):
        assert st(**bad) == UNSUPPORTED, bad


@pytest.fixture
def no_device(monkeypatch):
    """The binding's checks with host tensors: the device is taken as the host (-1), and
    nothing may reach the library."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)

    def reached(name):
        raise AssertionError("%s was called" % name)
    import nvfp4_paged_kv_nvfp4kv_gb300.step as step
    import nvfp4_paged_kv_nvfp4kv_gb300.tree as tree
    monkeypatch.setattr(step, "_entry", reached)
    monkeypatch.setattr(tree, "_entry", reached)


def test_tree_masks_binding(no_device):
    ok = dict(parents=i32(4), qo_indptr=i32(3), kv_len=i32(2))
    for change in (dict(max_nodes=None), dict(max_nodes=0), dict(max_nodes=1025),
                   dict(tree_mask=i32(3, 1)), dict(tree_mask=i32(4, 1).long()),
                   dict(tree_mask=i32(4, 2)[:, :1]), dict(tree_mask=i32(4, 1), max_nodes=33),
                   dict(max_nodes=4, positions=i32(3)), dict(max_nodes=4, qo_indptr=i32(2)),
                   dict(max_nodes=4, parents=i32(4).long())):
        with pytest.raises(ValueError):
            N.nvfp4kv_tree_masks(**{**ok, **change})


def test_norm_rope_binding(no_device):
    plan = N.nvfp4kv_rope_plan(64, device="cpu")
    x, w = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    assert N.nvfp4kv_norm_rope(plan, None, None, i32(3)) == (None, None)
    for qw, kw in ((None, w), (w, None), (w[:63], w), (w.half(), w), (w, w.float()),
                   (w.double(), w.double()), (torch.ones(128, dtype=torch.bfloat16)[::2], w)):
        with pytest.raises(ValueError):
            N.nvfp4kv_norm_rope(plan, x, x, i32(3), qw, kw)


# ---- tree attention ----------------------------------------------------------------------
def host_plan(kernel=0, **kw):
    plan = N.nvfp4kv_decode_plan([0, 3, 4], [0, 2, 4], [5, 16], 8, 2, 128, 128, num_sms=152,
                                 ctas_per_sm=3, allocate=False, kernel=kernel, **kw)
    plan.workspace = torch.zeros(int(plan.info.workspace_bytes) + 256, dtype=torch.uint8)
    return plan


def paged(pages=8, hkv=2, dk=128, dv=128):
    layout = W.CacheLayout("HND", pages, 16, hkv, dk, dv)
    return N.PagedCache.allocate(layout, device="cpu")


def test_tree_run_refusals():
    """Statuses come before the plan's device or any launch."""
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    out, lse = torch.zeros((4, 8, 128), dtype=torch.bfloat16), torch.zeros((4, 8))
    mask, idx, cache = i32(4, 1), i32(4), paged()

    def st(plan, mask_ptr=mask.data_ptr(), words=1, k=None, v=None, kst=256, c=cache):
        at = (plan.workspace.data_ptr() + 255) // 256 * 256
        return call("nvfp4kv_tree_run", C.byref(plan.info), mask_ptr, words, k, kst, 128, v, 256,
                    128, q.data_ptr(), 1024, 128, c.struct(), idx.data_ptr(), 0.0, at,
                    int(plan.info.workspace_bytes), out.data_ptr(), lse.data_ptr(), None)
    for kernel in (1, 3):
        plan = host_plan(kernel)
        plan.info.device = -1
        assert st(plan, mask_ptr=None) == INVALID
        assert st(plan, mask_ptr=mask.data_ptr() + 2) == INVALID
        assert st(plan, words=0) == UNSUPPORTED and st(plan, words=33) == UNSUPPORTED
        assert st(plan, k=q.data_ptr()) == INVALID and st(plan, v=q.data_ptr()) == INVALID
        assert st(plan, k=q.data_ptr(), v=q.data_ptr(), kst=3) == INVALID
        assert st(plan, c=paged(hkv=4)) == _lib.ERR_PLAN_MISMATCH
    plan = host_plan(2)
    plan.info.device = -1
    assert st(plan) == UNSUPPORTED  # the CUDA-core kernel has no trees
    plan = host_plan(5)
    plan.info.device = -1
    assert st(plan) == _lib.ERR_PLAN_MISMATCH  # a plan for the E4M3 cache


def test_tree_run_binding(no_device):
    plan, cache = host_plan(), paged()
    ok = dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16), kv_indices=i32(4),
              tree_mask=i32(4, 1))
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    for change in (dict(q=ok["q"][:3]), dict(q=ok["q"].half()), dict(q=ok["q"][:, :4]),
                   dict(tree_mask=i32(3, 1)), dict(tree_mask=i32(4)),
                   dict(tree_mask=i32(4, 1).long()), dict(tree_mask=i32(4, 2)[:, ::2]),
                   dict(kv_indices=i32(3)), dict(kv_indices=i32(4).long()), dict(new_k=k),
                   dict(new_k=k, new_v=k[:3]), dict(new_k=k, new_v=k.float()),
                   dict(out=torch.zeros((4, 8, 64), dtype=torch.bfloat16)),
                   dict(lse=torch.zeros((4, 7))),
                   dict(out=torch.zeros((4, 8, 128), dtype=torch.float16))):
        with pytest.raises(ValueError):
            N.nvfp4kv_tree_run(plan, cache=cache, **{**ok, **change})
    plan.workspace = None
    with pytest.raises(ValueError):
        N.nvfp4kv_tree_run(plan, cache=cache, **ok)


# ---- accepted tokens ------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [False, True])
def test_compact_refusals(e4m3):
    cache = N.E4m3Cache.allocate(8, 2, 64, 64, device="cpu") if e4m3 else paged(dk=64, dv=64)
    name = "nvfp4kv_e4m3_compact_tokens" if e4m3 else "nvfp4kv_compact_tokens"
    lists = [i32(4) for _ in range(5)]
    path, kept, qo, kvp, idx = (t.data_ptr() for t in lists)
    struct = cache._struct if e4m3 else cache.struct()

    def st(c=struct, path=path, stride=2, width=2, kept=kept, last=qo, batch=2, idx=idx):
        return call(name, c, path, stride, width, kept, qo, kvp, idx, last, batch, None, None)
    assert st(batch=0) == OK and st(width=0) == OK
    for bad in (dict(batch=-1), dict(width=-1), dict(stride=1), dict(stride=-2), dict(path=None),
                dict(kept=None), dict(last=None), dict(idx=None)):
        assert st(**bad) == INVALID, bad
    assert st(batch=1 << 30) == UNSUPPORTED
    struct.page_size = 8
    assert st(c=struct) == UNSUPPORTED


def test_compact_binding(no_device):
    ok = dict(path=i32(2, 3), num_kept=i32(2), qo_indptr=i32(3), kv_indptr=i32(3),
              kv_indices=i32(5), last_page_len=i32(2))
    for change in (dict(path=i32(3, 3)), dict(path=i32(2, 6)[:, ::2]), dict(path=i32(6)),
                   dict(path=i32(2, 3).long()), dict(num_kept=i32(3)), dict(qo_indptr=i32(2)),
                   dict(kv_indptr=i32(4)), dict(kv_indices=i32(5).long())):
        with pytest.raises(ValueError):
            N.nvfp4kv_compact_tokens(paged(), **{**ok, **change})


# ---- pages with several owners -----------------------------------------------------------------
def fork(**change):
    lists = {n: i32(8) for n in ("par", "child", "kv", "table", "shares", "free", "head", "out",
                                 "src", "dst")}
    a = dict({n: t.data_ptr() for n, t in lists.items()}, forks=2, rows=4, page=16, stride=2,
             width=2, pages=8, nfree=8)
    a.update(change)
    return call("nvfp4kv_fork_pages", a["par"], a["child"], a["forks"], a["kv"], a["rows"],
                a["page"], a["table"], a["stride"], a["width"], a["shares"], a["pages"], a["free"],
                a["nfree"], a["head"], a["head"] if change.get("out") == "head" else a["out"],
                a["src"], a["dst"], None, None)


def test_fork_refusals():
    for bad in (dict(forks=-1), dict(rows=-1), dict(width=-1), dict(pages=-1), dict(nfree=-1),
                dict(par=None), dict(child=None), dict(kv=None), dict(table=None),
                dict(shares=None), dict(free=None), dict(head=None), dict(out=None),
                dict(src=None), dict(dst=None), dict(stride=1), dict(out="head")):
        assert fork(**bad) == INVALID, bad
    for bad in (dict(forks=8193), dict(rows=65537), dict(page=0), dict(page=65537)):
        assert fork(**bad) == UNSUPPORTED, bad


def release(**change):
    lists = {n: i32(8) for n in ("keep", "kv", "table", "shares", "free", "head", "out")}
    a = dict({n: t.data_ptr() for n, t in lists.items()}, rows=4, page=16, stride=2, width=2,
             pages=8, nfree=8)
    a.update(change)
    return call("nvfp4kv_release_pages", a["keep"], a["kv"], a["rows"], a["page"], a["table"],
                a["stride"], a["width"], a["shares"], a["pages"], a["free"], a["nfree"],
                a["head"], a["out"], None, None)


def test_release_refusals():
    for bad in (dict(rows=-1), dict(width=-1), dict(pages=-1), dict(nfree=-1), dict(keep=None),
                dict(kv=None), dict(table=None), dict(shares=None), dict(free=None),
                dict(head=None), dict(out=None), dict(stride=1)):
        assert release(**bad) == INVALID, bad
    for bad in (dict(rows=8193), dict(page=0), dict(page=65537)):
        assert release(**bad) == UNSUPPORTED, bad


def test_copy_refusals():
    src, dst = i32(4), i32(4)
    for name, struct in (("nvfp4kv_copy_pages", paged().struct()),
                         ("nvfp4kv_e4m3_copy_pages",
                          N.E4m3Cache.allocate(8, 2, 64, 64, device="cpu")._struct)):
        assert call(name, struct, None, None, 0, None, None) == OK
        assert call(name, struct, None, dst.data_ptr(), 4, None, None) == INVALID
        assert call(name, struct, src.data_ptr(), None, 4, None, None) == INVALID
        assert call(name, struct, src.data_ptr(), dst.data_ptr(), -1, None, None) == INVALID
        assert call(name, struct, src.data_ptr(), dst.data_ptr(), 1 << 30, None, None) == UNSUPPORTED
        assert call(name, None, src.data_ptr(), dst.data_ptr(), 4, None, None) == INVALID


def test_page_binding(no_device):
    f = dict(parents=i32(2), children=i32(2), kv_len=i32(4), block_table=i32(4, 3),
             page_shares=i32(9), free_pages=i32(5), free_head=i32(1), free_head_out=i32(1),
             copy_src=i32(2), copy_dst=i32(2))
    for change in (dict(children=i32(3)), dict(copy_src=i32(1)), dict(copy_dst=i32(3)),
                   dict(block_table=i32(3, 3)), dict(block_table=i32(4, 6)[:, ::2]),
                   dict(block_table=i32(4, 3).long()), dict(free_head=i32(0)),
                   dict(free_head_out=i32(0)), dict(kv_len=i32(4).long()),
                   dict(page_shares=i32(18)[::2])):
        with pytest.raises(ValueError):
            N.nvfp4kv_fork_pages(**{**f, **change})
    r = dict(keep_len=i32(4), kv_len=i32(4), block_table=i32(4, 3), page_shares=i32(9),
             free_pages=i32(5), free_head=i32(1))
    for change in (dict(keep_len=i32(3)), dict(block_table=i32(5, 3)), dict(free_head=i32(0)),
                   dict(free_head_out=i32(0)), dict(free_pages=i32(5).long())):
        with pytest.raises(ValueError):
            N.nvfp4kv_release_pages(**{**r, **change})
    for src, dst in ((i32(2), i32(3)), (i32(2).long(), i32(2))):
        with pytest.raises(ValueError):
            N.nvfp4kv_copy_pages(paged(), src, dst)
