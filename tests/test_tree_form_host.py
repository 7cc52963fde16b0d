"""Host-only checks of nvfp4kv_tree_form: what it refuses, and the form that needs no device."""
import ctypes as C

import pytest

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib


def plan(rows, kernel=1, **kw):
    return N.nvfp4kv_decode_plan([0, rows], [0, 20], [16], 4, 1, 128, 128, kernel=kernel,
                                 num_sms=152, ctas_per_sm=1, allocate=False, **kw)


def test_refusals():
    fn, form = _lib.load().nvfp4kv_tree_form, _lib.TreeLaunch()
    p = plan(2)
    assert fn(C.byref(p.info), C.byref(form)) == 0
    assert fn(None, C.byref(form)) == 1 and fn(C.byref(p.info), None) == 1
    assert fn(C.byref(_lib.PlanInfo()), C.byref(form)) == 1  # (not a plan)
    for kernel in (2, 4, 5):
        assert fn(C.byref(plan(1, kernel).info), C.byref(form)) == 2
        with pytest.raises(N.NvFp4KvError):
            N.nvfp4kv_tree_form(plan(1, kernel))


def test_few_rows_run_in_the_plans_kernel():
    form = N.nvfp4kv_tree_form(plan(2, force_chunk_tokens=64))
    assert form == dict(block_rows=8, row_blocks=1, cluster_ctas=1, value_ctas=1,
                        whole_requests=0, longest_first=0, folded=1)
    assert not any(N.nvfp4kv_tree_form(plan(0)).values())
