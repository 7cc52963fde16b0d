"""Host-only checks of the serving-step binding against calls that the library
itself cannot refuse (a pointer carries no length)."""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib


def plan_on_host(qo, kvp, last):
    """A plan with kernel 5 whose workspace is host memory: a run gets as far as the
    checks of its arguments."""
    plan = N.nvfp4kv_decode_plan(qo, kvp, last, 2, 1, 128, 128, kernel=5, num_sms=152,
                                 ctas_per_sm=3, allocate=False)
    plan.workspace = torch.zeros(max(int(plan.info.workspace_bytes), 256), dtype=torch.uint8)
    return plan


def run(plan, entries):
    rows = plan.info.total_qo_rows
    q = torch.zeros((rows, 2, 128), dtype=torch.bfloat16)
    cache = N.E4m3Cache.allocate(200, 1, 128, 128, device="cpu")
    N.nvfp4kv_e4m3_decode_run(plan, q, cache, torch.zeros(entries, dtype=torch.int32))


@pytest.mark.parametrize("qo,kvp,last,need", [
    ([0, 0, 1], [0, 100, 102], [3, 5], 102),        # an idle request in front
    ([0, 1, 1, 2], [0, 2, 60, 63], [3, 5, 1], 63),  # and in the middle
    ([0, 1, 1], [0, 2, 60], [3, 5], 2),             # one behind is not read
    ([0, 1], [0, 7], [16], 7)])
def test_kv_indices_reach_the_last_request_with_rows(qo, kvp, last, need):
    plan = plan_on_host(qo, kvp, last)
    assert plan.kv_end == need
    units = plan.host[:48 * plan.info.num_units].view(torch.int32).reshape(-1, 12)
    assert int((units[:, 2] + units[:, 3]).max()) == need  # first page and pages of a unit
    with pytest.raises(ValueError, match="kv_indices has %d entries, the plan reads %d"
                       % (need - 1, need)):
        run(plan, need - 1)


def test_a_plan_without_rows_reads_nothing():
    assert plan_on_host([0, 0], [0, 9], [1]).kv_end == 0
    assert plan_on_host([0], [0], []).kv_end == 0


def test_rope_plan_checks_its_table():
    """A table of the caller's own must hold every pair that the kernel reads."""
    table = N.nvfp4kv_rope_plan(128, 64, device="cpu").freq
    assert N.RopePlan(128, 64, False, 1.0, table).rotary_dim == 64
    for bad in (table[:31], table.int(), table.double(), table.repeat(2)[::2]):
        with pytest.raises(ValueError):
            N.RopePlan(128, 64, False, 1.0, bad)


@pytest.mark.parametrize("heads,dims", [(40, 128), (40, 64), (64, 128)])
def test_chunks_of_one_page_tiles_fill_the_wave(heads, dims):
    """9 to 16 rows a kv head stream tiles of one page: a chunk is not rounded up to
    the 8 pages of the tensor-memory kernel's tiles (9 requests of 70 pages, 4 kv
    heads, 304 CTAs: 8 chunks a request, where 5 of whole tiles would leave 124 idle)."""
    kvp = [70 * b for b in range(10)]
    plan = N.nvfp4kv_decode_plan(list(range(10)), kvp, [7] * 9, heads, 4, dims, dims, kernel=5,
                                 num_sms=152, ctas_per_sm=2, allocate=False)
    assert plan.info.rows_per_block == 16
    assert 288 <= plan.info.num_units <= 304


_MANY_SMS = """
import ctypes as C, importlib.util, resource, sys, types
sys.modules["torch"] = types.ModuleType("torch")  # (its address space is not the library's)
resource.setrlimit(resource.RLIMIT_AS, (4 << 30, 4 << 30))
pkg = types.ModuleType("pkg"); pkg.__path__ = [sys.argv[1]]; sys.modules["pkg"] = pkg
import pkg._lib as L
lib = L.load()
a = lambda x: (C.c_int32 * len(x))(*x)
qo, kv, last = a([0, 20, 40]), a([0, 200, 500]), a([3, 4])
for sms in (152, 4096, 2 ** 31 - 1):
    opts, info = L.PlanOptions(1, 0, 0, 0, 5, sms, 1, 0, None), L.PlanInfo()
    st = lib.nvfp4kv_decode_plan(qo, kv, last, 2, 8, 2, 128, 128, 16, C.byref(opts), -1, None, 0,
                                 None, 0, None, C.byref(info))
    print(sms, st, info.num_units)
"""


def test_plan_for_any_number_of_sms():
    """The option num_sms names any number: the plan's model of their loads takes no
    memory for SMs that stay idle, and the C entry does not end the process (4 GB of
    address space)."""
    run = subprocess.run([sys.executable, "-c", _MANY_SMS, os.path.dirname(_lib.__file__)],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    lines = [line.split() for line in run.stdout.splitlines()]
    assert [int(x[0]) for x in lines] == [152, 4096, 2 ** 31 - 1]
    assert all(int(x[1]) in (_lib.OK, _lib.ERR_WORKSPACE_TOO_SMALL) for x in lines)
    assert all(int(x[2]) > 0 for x in lines)
