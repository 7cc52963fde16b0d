"""64-bit references of the serving-step operators (page table, rotary
positions, E4M3 append, attention over the E4M3 cache), written from their
definitions in plain Python and numpy."""
from __future__ import annotations

import math

import numpy as np
import torch


def pages_of(n, page):
    return -(-n // page)


# ---- page table ------------------------------------------------------------
def page_table(kv_len, qo_len, table, free, head, page):
    """The lists of a step; extends the rows of ``table`` (a list of lists)."""
    qo, kvp, last, idx, req, pos, slot = [0], [0], [], [], [], [], []
    for b, (total, n) in enumerate(zip(kv_len, qo_len)):
        held, every = pages_of(total - n, page), pages_of(total, page)
        for c in range(held, every):
            table[b][c] = free[head]
            head += 1
        idx += table[b][:every]
        kvp.append(len(idx))
        last.append(total - (every - 1) * page if every else 0)
        for p in range(total - n, total):
            req.append(b)
            pos.append(p)
            slot.append(table[b][p // page] * page + p % page)
        qo.append(len(req))
    return dict(qo_indptr=qo, kv_indptr=kvp, last_page_len=last, kv_indices=idx, batch_idx=req,
                positions=pos, slot_map=slot, free_head=[head])


# ---- rotary positions --------------------------------------------------------
def rope_frequencies(rotary, base, factor=1.0, orig=0, low=1.0, high=32.0):
    f = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if not orig:
        return [x / factor for x in f]
    out = []
    for x in f:
        g = min(max((orig * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
        out.append(x * (1 - g) / factor + x * g)
    return out


def rope(x, positions, rotary, interleaved, freq, attn=1.0):
    """(y, |x1| + |x2| of every element's pair; 0 where dims pass) in 64 bits."""
    x = x.double().cpu().numpy()
    y, size = x.copy(), np.zeros_like(x)
    # angles modulo a turn in extended precision: positions up to 2^31
    turns = np.longdouble(freq) / (2 * np.longdouble(math.pi))
    turns = turns[None, :] * np.asarray(positions, dtype=np.longdouble)[:, None]
    angle = (2 * math.pi * (turns - np.rint(turns)).astype(np.float64))[:, None, :]
    c, s = attn * np.cos(angle), attn * np.sin(angle)
    half = rotary // 2
    lo, hi = ((slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved
              else (slice(0, half), slice(half, rotary)))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = np.abs(a) + np.abs(b)
    return y, size


# ---- the E4M3 cache ------------------------------------------------------------
def e4m3_values():
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = (math.nan if e == 15 and m == 7 else x) * (-1 if c & 128 else 1)
    return out


VALUES = e4m3_values()


def e4m3_codes(x):
    """Codes of the nearest E4M3 values, ties to the even code, saturating;
    NaN gives 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    grid = VALUES[:0x7F]  # 0 .. 448 in order
    size = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0)
    up = np.searchsorted(grid, size).clip(0, 0x7E)
    down = np.maximum(up - 1, 0)
    du, dd = grid[up] - size, size - grid[down]
    code = np.where(du < dd, up, np.where(dd < du, down, np.where(up % 2 == 0, up, down)))
    code = np.where(size == grid[up], up, code)
    return np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def scale_of(m):
    """2^e, the smallest e in [-64, 64] with 448 * 2^e >= m."""
    e = -64
    while e < 64 and 448.0 * 2.0 ** e < m:
        e += 1
    return 2.0 ** e


def append(codes, scale, x, page, lo, hi, first_row):
    """One page of one (K or V) tensor: codes [heads, page_size, dim] uint8 and
    scale [heads] are changed; slots [lo, hi) take rows first_row .. of x."""
    for h in range(codes.shape[0]):
        block = x[first_row:first_row + hi - lo, h]
        finite = np.abs(block[np.isfinite(block)])
        s = scale_of(finite.max() if finite.size else 0.0)
        if lo:
            old = float(scale[h])
            s = max(s, old)
            if s > old:
                codes[h, :lo] = e4m3_codes(VALUES[codes[h, :lo]] * float(np.float32(old / s)))
        codes[h, lo:hi] = e4m3_codes((block / s).astype(np.float32))
        scale[h] = s


def dequantised(codes, scale, pages, total):
    """[heads, total, dim] of the tokens in the listed pages, 64 bits."""
    x = VALUES[codes[pages]] * scale[pages].astype(np.float64)[:, :, None, None]
    n, h, p, d = x.shape
    return x.transpose(1, 0, 2, 3).reshape(h, n * p, d)[:, :total]


def attention(q, k, v, v_scale, sm_scale, causal):
    """One request: q [n, Hq, Dk], k [Hkv, L, Dk], v [Hkv, L, Dv] and the value
    scale of every token v_scale [Hkv, L] in 64 bits.  Returns out, lse and,
    for the tolerance, the softmax-weighted mean of |v|, the largest
    sm_scale * sum_d |q_d k_d| of a row, and the f16 floor of the weights:
    max_j(p_j b_j) * sum_j |d_j| / sum_j p_j (d_j the codes, b_j the scales)."""
    n, hq, _ = q.shape
    hkv, total, dv = v.shape
    group = hq // hkv
    out, lse = np.zeros((n, hq, dv)), np.zeros((n, hq))
    mean, reach, floor = np.zeros((n, hq, dv)), np.zeros((n, hq)), np.zeros((n, hq, dv))
    for i in range(n):
        seen = total - n + i + 1 if causal else total
        for h in range(hq):
            kk, vv, b = k[h // group, :seen], v[h // group, :seen], v_scale[h // group, :seen]
            s = sm_scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + math.log(p.sum())
            out[i, h] = p @ vv / p.sum()
            mean[i, h] = p @ np.abs(vv) / p.sum()
            reach[i, h] = sm_scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            floor[i, h] = (p * b).max() * np.abs(vv / b[:, None]).sum(0) / p.sum()
    return out, lse, mean, reach, floor


def to_np(t):
    return t.detach().double().cpu().numpy() if isinstance(t, torch.Tensor) else np.asarray(t)
