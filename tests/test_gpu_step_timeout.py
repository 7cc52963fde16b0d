"""A bounded wait of the E4M3 extend kernel runs out: the kernel returns, reports
NVFP4KV_FLAG_COPY_TIMEOUT, and the context stays usable.

As for the NVFP4 extend kernel, the failure is made in a separate build of the
library: the first loader of CTA (0, 0) withholds its arrival for the first
tile, the S^T issuer's wait (about a millisecond in this build) runs out and
raises flag 0x4 and the CTA's abort word, and every other wait returns; copies
and products in flight are drained before the tensor memory is released.  The
other CTAs' rows are right all the same."""
import ctypes as C
import os

import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import test_gpu_step_ops as T
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
from nvfp4_paged_kv_nvfp4kv_gb300 import build as B

pytestmark = pytest.mark.gpu


@pytest.fixture
def withholding_lib(monkeypatch):
    prod = _lib.load()
    path = B.build(defines=["NVFP4KV_E4M3_TEST_SKIP_ARRIVE=1", "NVFP4KV_TG5_POLLS=50"],
                   out=os.path.join(B.BUILD, "e4m3_timeout", "libnvfp4kv.so"))
    lib = C.CDLL(path)
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    monkeypatch.setattr(_lib, "_lib", lib)
    yield lib
    monkeypatch.setattr(_lib, "_lib", prod)


def run():
    c = T.CacheCase((300, 900), 16, 2, 128, 128, seed=3)
    q = torch.randn((40, 4, 128), generator=torch.Generator().manual_seed(1))
    q = q.to(torch.bfloat16).cuda()
    plan = N.nvfp4kv_decode_plan([0, 20, 40], c.indptr, c.last, 4, 2, 128, 128, causal=True,
                                 kernel=5, disable_split=True)
    assert plan.info.rows_per_block > 16
    out, _ = N.nvfp4kv_e4m3_decode_run(plan, q, c.cache, c.kv_indices)
    torch.cuda.synchronize()
    return out, N.nvfp4kv_workspace_flags(plan, clear=True)


def test_extend_wait_runs_out_and_reports(withholding_lib, monkeypatch):
    out, flags = run()
    assert flags == _lib.FLAG_COPY_TIMEOUT
    assert float(torch.arange(1000, device="cuda", dtype=torch.float32).sum()) == 499500.0
    monkeypatch.undo()
    good, flags = run()
    assert flags == 0
    # unit 0 is the first request's first kv head; the other rows and heads stand
    same = (out == good).all(-1)
    assert bool(same[20:].all()) and bool(same[:, 2:].all()) and not bool(same.all())
