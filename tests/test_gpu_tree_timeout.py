"""A bounded wait of the kernel of 128-row tree blocks runs out: the kernel returns, reports
NVFP4KV_FLAG_COPY_TIMEOUT, and the context stays usable.

As for the other kernels, the failure is made in a separate build of the library: the first
K loader of CTA (0, 0) withholds its arrival for the first tile, the issuer's wait (about a
millisecond in this build) runs out and raises flag 0x4 and the CTA's abort word, and every
other wait returns; products in flight are drained before the tensor memory is released.  The
rows of other CTAs are right all the same."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
import tree_reference as T
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib
from nvfp4_paged_kv_nvfp4kv_gb300 import build as B

pytestmark = pytest.mark.gpu


@pytest.fixture
def withholding_lib(monkeypatch):
    prod = _lib.load()
    path = B.build(defines=["NVFP4KV_TREE_TEST_SKIP_ARRIVE=1", "NVFP4KV_TG5_POLLS=50"],
                   out=os.path.join(B.BUILD, "tree_timeout", "libnvfp4kv.so"))
    lib = C.CDLL(path)
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    monkeypatch.setattr(_lib, "_lib", lib)
    yield lib
    monkeypatch.setattr(_lib, "_lib", prod)


def run(dk, dv, kv, new):
    c = T.Nvfp4Case(kv, 16, 2, dk, dv, seed=4)
    q = torch.randn((sum(new), 8, dk), generator=torch.Generator().manual_seed(1))
    q = q.to(torch.bfloat16).cuda()
    rng = np.random.default_rng(5)
    words = (max(new) + 31) // 32
    mask = np.concatenate([T.mask_words(T.ancestors(T.random_parents(rng, n)), words)
                           for n in new]).astype(np.int32)
    plan = N.nvfp4kv_decode_plan(np.concatenate([[0], np.cumsum(new)]), c.indptr, c.last, 8, 2,
                                 dk, dv, disable_split=True)
    out, lse = N.nvfp4kv_tree_run(plan, q, c.cache, c.kv_indices, torch.from_numpy(mask).cuda())
    torch.cuda.synchronize()
    return out, N.nvfp4kv_workspace_flags(plan, clear=True)


# 128-row blocks, rows held twice, a cluster that joins its states, shared halves' states
@pytest.mark.parametrize("dk,dv,kv,new", [
    (128, 128, (300, 900), (32, 20)), (64, 64, (300, 900), (9, 20)),
    (128, 128, (4000, 3000), (12, 12)), (512, 256, (300, 2000), (20, 12))])
def test_wait_runs_out_and_reports(withholding_lib, monkeypatch, dk, dv, kv, new):
    out, flags = run(dk, dv, kv, new)
    assert flags == _lib.FLAG_COPY_TIMEOUT
    assert float(torch.arange(1000, device="cuda", dtype=torch.float32).sum()) == 499500.0
    monkeypatch.undo()
    good, flags = run(dk, dv, kv, new)
    assert flags == 0
    # one request's first rows of one kv head are missing; every other row stands
    same = (out == good).all(-1).view(sum(new), 2, 4).all(-1)  # [rows, kv heads]
    first = torch.arange(sum(new)).cuda() < new[0]
    wrong = [(r, h) for r, rows in enumerate((first, ~first)) for h in (0, 1)
             if not bool(same[rows][:, h].all())]
    assert len(wrong) == 1, wrong
