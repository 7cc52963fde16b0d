"""An old page scale outside the format's range: the append takes the nearer end of
[2^-64, 2^64] (the lower for a NaN), as the attention does, and flags it."""
import math

import pytest

import test_gpu_step_ops as T
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad,taken", [
    (0.0, 2.0 ** -64), (-0.0, 2.0 ** -64), (-1.0, 2.0 ** -64), (math.nan, 2.0 ** -64),
    (2.0 ** -65, 2.0 ** -64), (-math.inf, 2.0 ** -64), (math.inf, 2.0 ** 64),
    (2.0 ** 65, 2.0 ** 64), (1.5 * 2.0 ** 64, 2.0 ** 64)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** 80])
def test_append_old_scale_out_of_range(bad, taken, size):
    """Older codes and the new scale are those of an append onto the end that is
    taken: under 2^64 nothing older changes, whatever the new tokens' size."""
    c = T.CacheCase((20, 30), 16, 2, 64, 128, seed=3)
    page = c.pages(0)[1]
    k, v = T.new_rows(3, 2, 64, 128, "bf16")
    k, v = k * size, v * size
    for i in (0, 1):
        c.scale[i][page, 1] = bad
    c.upload()
    for i in (0, 1):
        c.scale[i][page, 1] = taken
    c.append((2, 1), k, v)
    f = T.new_flags()
    c.run_append((2, 1), k, v, f)
    c.check()
    assert int(f) == _lib.FLAG_BAD_SCALE


def test_the_ends_of_the_range_are_scales():
    c = T.CacheCase((20, 30), 16, 2, 64, 128, seed=4)
    k, v = T.new_rows(3, 2, 64, 128, "bf16")
    c.scale[0][c.pages(0)[1], :] = 2.0 ** 64
    c.scale[1][c.pages(0)[1], :] = 2.0 ** -64
    c.upload()
    c.append((2, 1), k, v)
    f = T.new_flags()
    c.run_append((2, 1), k, v, f)
    c.check()
    assert int(f) == 0
