"""The frequency table against 60 decimal digits, and the rotation at the ends of
the position range against angles from the same digits."""
import math
from decimal import Decimal, getcontext, localcontext

import numpy as np
import pytest
import torch

import nvfp4_paged_kv_nvfp4kv_gb300 as N
from nvfp4_paged_kv_nvfp4kv_gb300 import _lib

DIGITS = 60


def two_pi():
    """2 pi = 8 (4 atan(1/5) - atan(1/239)) to DIGITS digits (Machin)."""
    def atan_inverse(n):
        term, total, k = Decimal(1) / n, Decimal(0), 0
        while abs(term) > Decimal(10) ** -(DIGITS + 5):
            total += term / (2 * k + 1) * (-1 if k % 2 else 1)
            term /= n * n
            k += 1
        return total
    return 8 * (4 * atan_inverse(5) - atan_inverse(239))


def exact_turns(rotary, base=10000.0, factor=1.0, original_max_position=0, low=1.0, high=32.0):
    """Turns a position of every pair, from the formulas in the header."""
    with localcontext() as ctx:
        ctx.prec = DIGITS + 10
        tau, out = two_pi(), []
        for i in range(rotary // 2):
            f = (Decimal(base).ln() * Decimal(-2 * i) / rotary).exp()
            if original_max_position:
                g = (original_max_position * f / tau - Decimal(low)) / (Decimal(high) - Decimal(low))
                g = min(max(g, Decimal(0)), Decimal(1))
                f = f * (1 - g) / Decimal(factor) + f * g
            else:
                f /= Decimal(factor)
            out.append(f / tau)
        return out


OPTIONS = [{}, dict(factor=4.0), dict(base=500000.0), dict(base=1000003.7, factor=0.37),
           dict(factor=0.001), dict(base=2.0), dict(base=1.0000001), dict(base=1e300),
           dict(base=500000.0, factor=32.0, original_max_position=8192, low=1.0, high=4.0),
           dict(factor=7.3, original_max_position=(1 << 40) + 12345, low=0.1, high=1e9)]


def table(rotary, base=10000.0, factor=1.0, original_max_position=0, low=1.0, high=32.0):
    out = np.zeros(rotary // 2, dtype=np.uint64)
    st = _lib.load().nvfp4kv_rope_frequencies(
        rotary, _lib.RopeOptions(base, factor, original_max_position, low, high), out.ctypes.data)
    return st, out.tolist()


@pytest.mark.parametrize("rotary", [2, 4, 64, 126, 128, 510, 512])
@pytest.mark.parametrize("kw", OPTIONS, ids=range(len(OPTIONS)))
def test_table_is_rounded_once(rotary, kw):
    """Every entry is the exact value to half a unit of 2^-64 turns (and 2^-90 of the
    turns, from 106 bits)."""
    st, got = table(rotary, **kw)
    assert st == 0
    getcontext().prec = DIGITS
    for g, want in zip(got, exact_turns(rotary, **kw)):
        units = want * (1 << 64)
        off = (Decimal(g) - units) % (1 << 64)
        off = min(off, (1 << 64) - off)
        slack = Decimal(2) ** -20 if kw.get("base", 0) == 1e300 else Decimal(2) ** -90
        assert off <= Decimal("0.5") + units * slack


def test_frequencies_without_end_are_refused():
    assert table(64, factor=1e-320)[0] == _lib.ERR_INVALID_ARGUMENT  # 1 / factor is infinite
    assert table(64, factor=2.0 ** -45)[0] == _lib.ERR_INVALID_ARGUMENT
    assert table(64, factor=2.0 ** -40)[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kw", [{}, dict(factor=0.001), OPTIONS[-2]], ids=["plain", "dense", "parts"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_at_the_ends_of_the_positions(dtype, kw, interleaved):
    dim, pos = 128, [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1000003, 2 ** 30 + 1, 2 ** 24 + 1, -7, 0]
    args = dict(kw)
    for short in ("low", "high"):
        if short in args:
            args[short + "_rotations"] = args.pop(short)
    plan = N.nvfp4kv_rope_plan(dim, interleaved=interleaved, **args)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((len(pos), 6, dim), generator=g).to(dtype).cuda()
    x[:, 5, :] = 0
    if interleaved:
        x[:, 5, 0::2] = 1.0  # cosine and sine alone
    else:
        x[:, 5, :dim // 2] = 1.0
    y, _ = N.nvfp4kv_rope(plan, x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"))
    with localcontext() as ctx:
        ctx.prec = DIGITS + 10
        turns = [[float((t * p) % 1) for t in exact_turns(dim, **kw)] for p in pos]
    angle = 2 * math.pi * np.array(turns)[:, None, :]
    c, s = np.cos(angle), np.sin(angle)
    half = dim // 2
    lo, hi = ((slice(0, dim, 2), slice(1, dim, 2)) if interleaved
              else (slice(0, half), slice(half, dim)))
    x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
    a, b = x[..., lo], x[..., hi]
    eps = torch.finfo(dtype).eps / 2
    for got, want in ((y[..., lo], a * c - b * s), (y[..., hi], b * c + a * s)):
        # the angle, 1.02 * 2^-26 turns; sincospif (two units of float32), two products
        # and a sum in float32; one rounding
        size = np.abs(a) + np.abs(b)
        err = size * (2 * math.pi * 1.02 * 2.0 ** -26 + 2.0 ** -22 + 3 * 2.0 ** -24)
        tol = err + eps * (np.abs(want) + err) + 2.0 ** -25
        assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
