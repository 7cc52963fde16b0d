"""The page table of the largest batches (its sums need more shared memory than a
kernel has unasked), also from two host threads at once."""
import threading

import numpy as np
import pytest
import torch

import test_gpu_step_ops as T

pytestmark = pytest.mark.gpu


def case(batch, seed=0, page=16):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, 60, batch)
    new = np.minimum(kv, rng.integers(0, 4, batch))
    return T.TableCase(kv.tolist(), new.tolist(), page, seed=seed)


@pytest.mark.parametrize("batch", [2559, 2560, 3000, 8191, 8192])
def test_large_batches(batch):
    c = case(batch, seed=batch)
    f = T.new_flags()
    c.run(f)
    c.check()
    assert int(f) == 0


def test_two_threads_with_batches_of_different_sizes():
    """The limit of one call must not fall under another's need between that one's
    setting it and its launch: every launch of both threads succeeds."""
    cases, errors = {}, []
    for batch in (8192, 3000):
        cases[batch] = case(batch, seed=batch)
    torch.cuda.synchronize()

    def work(batch):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    cases[batch].run()
                torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append((batch, e))
    threads = [threading.Thread(target=work, args=(b,)) for b in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c in cases.values():
        c.check()
