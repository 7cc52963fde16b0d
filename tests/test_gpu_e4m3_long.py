"""The E4M3 extend kernel over units of many tiles: every ring (K, V, S^T,
scales, weights) wraps several times, and the last tile, which some rows or all
of them see in part, is one of a ring that has been round before."""
import math

import pytest

import test_gpu_step_ops as T

pytestmark = pytest.mark.gpu


def rows_of(plan):
    return plan.info.rows_per_block


# 128 tokens a tile: lengths that end inside the tile, at its first token, one
# short of its end and at its end
@pytest.mark.parametrize("dk,dv", [(256, 256), (256, 128), (128, 128)])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("tiles,over", [(5, 88), (6, 1), (9, 127), (9, 128), (17, 40)])
def test_units_of_many_tiles(dk, dv, page, tiles, over):
    """Whole requests: stale NaN codes past the end must not reach the output, and
    every value before it must."""
    kv = 128 * (tiles - 1) + over
    _, plan, _ = T.attend_case((kv, 600), (12, 15), 4, 2, dk, dv, causal=True, page=page,
                               disable_split=True, seed=kv + page)
    assert rows_of(plan) > 16 and plan.info.split == 0
    T.attend_case((kv,), (40,), 4, 2, dk, dv, causal=False, page=page, disable_split=True, seed=kv)


@pytest.mark.parametrize("dk,dv", [(256, 256), (256, 128), (128, 128)])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("chunk", [640, 768, 1152])
def test_split_units_of_many_tiles(dk, dv, page, chunk):
    """Chunks of 5, 6 and 9 tiles, the last of a request in part."""
    _, plan, _ = T.attend_case((2176 + 17, 2 * chunk + 5), (18, 9), 4, 2, dk, dv, causal=True,
                               page=page, force_chunk_tokens=chunk, seed=chunk)
    assert rows_of(plan) > 16 and plan.info.split == 1


@pytest.mark.parametrize("tiles", [5, 9])
@pytest.mark.parametrize("dk,dv,out", [(256, 256, "f16"), (128, 128, "f16"), (256, 128, "bf16")])
def test_prompts_end_two_tiles_in_part(dk, dv, out, tiles):
    """A block of rows whose limits lie in two tiles: the last two of its unit are
    both seen in part.  (64 or 32 rows a block, one head to a kv head: their limits
    are as many tokens apart.)"""
    kv = 128 * tiles + 20
    T.attend_case((kv,), (kv,), 2, 2, dk, dv, causal=True, out=out, seed=tiles)


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("dk,dv", [(256, 256), (256, 128), (128, 128)])
@pytest.mark.parametrize("chunk", [0, 640])
def test_nan_in_the_last_of_many_tiles(dk, dv, chunk):
    """NaN value codes that some rows see and some do not, in the last two tiles of
    nine, and one in an early tile that all see."""
    kv = 128 * 8 + 10
    new = 24

    def edit(c, q):
        for t, d in ((kv - 1, 3), (kv - 12, dv - 1), (kv - 20, 40), (130, 17)):
            c.codes[1][c.pages(0)[t // 16], 0, t % 16, d] = 0x7F
    _, plan, o = T.attend_case((kv, 700), (new, 9), 4, 2, dk, dv, causal=True, edit=edit,
                               force_chunk_tokens=chunk, seed=dv)
    assert rows_of(plan) > 16
    assert math.isnan(float(o[new - 1, 0, 3])) and not math.isnan(float(o[0, 0, 3]))


@pytest.mark.parametrize("dk,dv", [(256, 256), (128, 128)])
@pytest.mark.parametrize("chunk", [0, 640])
def test_live_lengths_of_many_tiles(dk, dv, chunk):
    """A plan made with other last page lengths reads the current ones: the tile in
    which the request ends, and the rows' limits, move with them."""
    for kv, planned in (((1110, 700), [1, 16]), ((1121, 690), [16, 1])):
        T.attend_case(kv, (20, 33), 4, 2, dk, dv, causal=True, live=planned, layout="NHD",
                      force_chunk_tokens=chunk, seed=dk)
