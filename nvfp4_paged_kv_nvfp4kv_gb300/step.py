"""Python binding of the serving-step entry points beside the NVFP4 attention
(include/nvfp4kv.h, same names): the step's page table, rotary positions and
the E4M3 cache with its attention.

Argument marshalling only, as in ``api``.  Tensors are checked for device,
type and shape here, because a pointer carries none of them; what the library
can check it checks itself (``NvFp4KvError``).  A decode step waits for these
calls, so they take what they need of a tensor once and keep what belongs to a
plan or a cache.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import _lib
from ._lib import E4m3CacheStruct, RopeOptions, StepTableStruct, check
from .api import Plan

__all__ = ["StepTable", "nvfp4kv_build_page_table", "RopePlan", "nvfp4kv_rope_plan",
           "nvfp4kv_rope", "nvfp4kv_norm_rope", "E4m3Cache", "nvfp4kv_e4m3_append",
           "nvfp4kv_e4m3_decode_run"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1}


def _entry(name):
    """The library's function (an attribute of the loaded library)."""
    return getattr(_lib._lib or _lib.load(), name)


def _check_device(dev, *tensors):
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensor on %s, the current device is cuda:%d" % (t.device, dev))


def _ints(dtype, **tensors):
    for name, t in tensors.items():
        if t is not None and (t.dtype != dtype or not t.is_contiguous()):
            raise ValueError("%s must be contiguous %s" % (name, dtype))


def _flag_ptr(flags, dev):
    if flags is None:
        return None
    if flags.dtype not in (torch.int32, torch.uint32) or flags.numel() < 1:
        raise ValueError("device_flags must be a 32-bit integer tensor")
    _check_device(dev, flags)
    return flags.data_ptr()


def _stream_of(stream, dev):
    if stream is None:  # (torch.cuda.current_stream() builds an object on every call)
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _empty(shape, dtype, device, stream, like=None):
    """An output of a call on `stream`, allocated in that stream's order (the
    caching allocator may hand its memory on as soon as it is freed).  ``like``: a
    tensor of that type and device (sooner done)."""
    if stream is None:
        if like is not None:
            return like.new_empty(shape)
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device if like is None else like.device)


# ---- the step's page table ------------------------------------------------------
class StepTable:
    """The device lists of one step: ``qo_indptr`` [batch + 1], ``kv_indptr``
    [batch + 1], ``last_page_len`` [batch], ``kv_indices`` [max_pages],
    ``batch_idx`` and ``positions`` [max_tokens], all int32, ``slot_map``
    [max_tokens] int64 (or None) and ``free_head`` [1] int32."""

    def __init__(self, qo_indptr, kv_indptr, last_page_len, kv_indices, batch_idx, positions,
                 slot_map, free_head):
        _ints(torch.int32, qo_indptr=qo_indptr, kv_indptr=kv_indptr,
              last_page_len=last_page_len, kv_indices=kv_indices, batch_idx=batch_idx,
              positions=positions, free_head=free_head)
        _ints(torch.int64, slot_map=slot_map)
        self.qo_indptr, self.kv_indptr, self.last_page_len = qo_indptr, kv_indptr, last_page_len
        self.kv_indices, self.batch_idx, self.positions = kv_indices, batch_idx, positions
        self.slot_map, self.free_head = slot_map, free_head
        self.batch = last_page_len.numel()
        if qo_indptr.numel() != self.batch + 1 or kv_indptr.numel() != self.batch + 1:
            raise ValueError("indptrs must have one entry more than last_page_len")
        tokens = batch_idx.numel()
        if positions.numel() != tokens or (slot_map is not None and slot_map.numel() != tokens):
            raise ValueError("batch_idx, positions and slot_map must have one length")
        if free_head.numel() < 1:
            raise ValueError("free_head is empty")
        tensors = [t for t in (qo_indptr, kv_indptr, last_page_len, kv_indices, batch_idx,
                               positions, slot_map, free_head) if t is not None]
        if len({t.device for t in tensors}) != 1:
            raise ValueError("the table's tensors are on different devices")
        s = StepTableStruct()
        for name in ("qo_indptr", "kv_indptr", "last_page_len", "kv_indices", "batch_idx",
                     "positions", "slot_map", "free_head"):
            t = getattr(self, name)
            setattr(s, name, None if t is None else t.data_ptr())
        s.max_pages, s.max_tokens = kv_indices.numel(), tokens
        self._struct, self._ref = s, C.byref(s)

    @classmethod
    def allocate(cls, batch, max_tokens, max_pages, device="cuda", slot_map=True):
        def i32(n):
            return torch.zeros(n, dtype=torch.int32, device=device)
        slots = torch.zeros(max_tokens, dtype=torch.int64, device=device) if slot_map else None
        return cls(i32(batch + 1), i32(batch + 1), i32(batch), i32(max_pages), i32(max_tokens),
                   i32(max_tokens), slots, i32(1))


def nvfp4kv_build_page_table(kv_len, qo_len, block_table, free_pages, free_head,
                             table: StepTable, page_size: int = 16, device_flags=None,
                             stream=None) -> StepTable:
    """Fill ``table`` (and the new entries of ``block_table`` [batch, pages])
    from the requests' lengths after the step and their new rows, on the
    device.  ``free_head`` [1] (or None: 0) is the first free entry of
    ``free_pages``; the head after the step is ``table.free_head``."""
    _ints(torch.int32, kv_len=kv_len, qo_len=qo_len, free_pages=free_pages, free_head=free_head)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be int32 [batch, pages] with contiguous rows")
    batch = table.batch
    if not (kv_len.numel() == qo_len.numel() == block_table.shape[0] == batch):
        raise ValueError("kv_len, qo_len and block_table must have the table's batch")
    dev = torch.cuda.current_device()
    _check_device(dev, kv_len, qo_len, block_table, free_pages, table.kv_indptr,
                  *(() if free_head is None else (free_head,)))
    st = _entry("nvfp4kv_build_page_table")(
        kv_len.data_ptr(), qo_len.data_ptr(), batch, page_size, block_table.data_ptr(),
        block_table.stride(0), block_table.shape[1], free_pages.data_ptr(), free_pages.numel(),
        None if free_head is None else free_head.data_ptr(), table._ref,
        _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_build_page_table")
    return table


# ---- rotary positions -------------------------------------------------------------
class RopePlan:
    """Frequencies on the device and the layout they belong to: ``freq`` holds, for
    each of the rotary_dim / 2 pairs, the turns of a position in units of 2^-64 (a
    64-bit integer tensor; ``nvfp4kv_rope_plan`` fills one, other tables may come
    from the caller)."""

    def __init__(self, head_dim, rotary_dim, interleaved, attention_factor, freq):
        self.head_dim, self.rotary_dim = int(head_dim), int(rotary_dim)
        if freq.dtype not in (torch.int64, torch.uint64) or not freq.is_contiguous():
            raise ValueError("freq must be a contiguous 64-bit integer tensor")
        if freq.numel() < self.rotary_dim // 2:
            raise ValueError("freq has fewer entries than rotary_dim / 2")
        self.interleaved = int(bool(interleaved))
        self.attention_factor = float(attention_factor)
        self.freq = freq  # int64 tensor, the bits of the uint64 table
        self.device, self.table = freq.get_device(), freq.data_ptr()
        self.layout = (self.head_dim, self.rotary_dim, self.interleaved)


def nvfp4kv_rope_plan(head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0,
                      interleaved: bool = False, factor: float = 1.0,
                      original_max_position: int = 0, low_rotations: float = 1.0,
                      high_rotations: float = 32.0, attention_factor: float = 1.0,
                      device="cuda") -> RopePlan:
    """The frequency table of ``nvfp4kv_rope`` (nvfp4kv_rope_frequencies): the
    first ``rotary_dim`` dims (all by default) rotate, as halves or as
    neighbouring pairs (``interleaved``).  ``factor`` > 1 stretches positions:
    every frequency alike, or, with ``original_max_position``, by parts."""
    rotary_dim = head_dim if rotary_dim is None else int(rotary_dim)
    if not 2 <= rotary_dim <= head_dim:
        raise ValueError("rotary_dim must lie in [2, head_dim]")
    host = torch.empty(max(rotary_dim // 2, 1), dtype=torch.int64)
    opts = RopeOptions(base, factor, original_max_position, low_rotations, high_rotations)
    check(_lib.load().nvfp4kv_rope_frequencies(rotary_dim, opts, host.data_ptr()),
          "nvfp4kv_rope_frequencies")
    return RopePlan(head_dim, rotary_dim, interleaved, attention_factor, host.to(device))


def _rows(name, t, head_dim, tokens, dtype):
    """Check [tokens, heads, head_dim]; returns the strides and the heads."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != head_dim or strides[2] != 1:
        raise ValueError("%s must be [tokens, heads, %d] with contiguous rows" % (name, head_dim))
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if shape[0] < tokens:
        raise ValueError("%s has fewer rows than the call needs" % name)
    return strides, shape[1]


def nvfp4kv_rope(plan: RopePlan, q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions,
                 q_out=None, k_out=None, stream=None):
    """Rotate q [tokens, Hq, D] and k [tokens, Hkv, D] (either may be None) by
    ``positions`` [tokens] int32: returns (q_out, k_out), new tensors unless
    given; ``q_out=q`` rotates in place."""
    if q is None and k is None:
        return None, None
    args, outs, dev = _rope_args(plan, q, k, positions, q_out, k_out, stream)
    st = _entry("nvfp4kv_rope")(*args, _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_rope")
    return outs


def nvfp4kv_norm_rope(plan: RopePlan, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                      positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                      weight_offset: float = 0.0, q_out=None, k_out=None, stream=None):
    """Norm every head of q [tokens, Hq, D] and k [tokens, Hkv, D] (either may be
    None), x / sqrt(mean x^2 + eps) * (weight + weight_offset), and rotate it as
    ``nvfp4kv_rope`` does, in one pass: returns (q_out, k_out).  ``q_weight`` and
    ``k_weight`` [D] are of the rows' type or both float32."""
    if q is None and k is None:
        return None, None
    args, outs, dev = _rope_args(plan, q, k, positions, q_out, k_out, stream)
    first, w = (q, q_weight) if q is not None else (k, k_weight)
    kind = _weight("q_weight" if q is not None else "k_weight", w, plan, first.dtype, dev)
    if q is not None and k is not None and \
            _weight("k_weight", k_weight, plan, first.dtype, dev) is not kind:
        raise ValueError("the weights must be of one type")
    st = _entry("nvfp4kv_norm_rope")(
        *args, None if q is None else q_weight.data_ptr(),
        None if k is None else k_weight.data_ptr(), _WEIGHT[kind], weight_offset, eps,
        _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_norm_rope")
    return outs


_WEIGHT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _weight(name, w, plan, dtype, dev):
    """Check the weights of a norm; returns their type."""
    if w is None or w.shape != (plan.head_dim,) or not w.is_contiguous():
        raise ValueError("%s must be contiguous [%d]" % (name, plan.head_dim))
    kind = w.dtype
    if kind is not dtype and kind is not torch.float32:
        raise ValueError("%s must be of the rows' type or torch.float32" % name)
    if w.get_device() != dev:
        _check_device(dev, w)
    return kind


def _rope_args(plan, q, k, positions, q_out, k_out, stream):
    """The arguments that both rotations take up to the frequencies and their factor,
    the outputs, and the device."""
    dtype = (q if q is not None else k).dtype
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError("q and k must be torch.bfloat16 or torch.float16")
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        raise ValueError("positions must be contiguous torch.int32")
    n, dev = positions.numel(), torch.cuda.current_device()
    if not positions.get_device() == plan.device == dev:
        _check_device(dev, positions, plan.freq)
    qa, q_out = _rope_rows(plan.head_dim, "q", q, q_out, n, dtype, dev, stream)
    ka, k_out = _rope_rows(plan.head_dim, "k", k, k_out, n, dtype, dev, stream)
    return ((*qa, *ka, n, positions.data_ptr(), *plan.layout, code, plan.table,
             plan.attention_factor), (q_out, k_out), dev)


def _rope_rows(dim, name, x, out, n, dtype, dev, stream):
    """The seven arguments of one of q and k, and its output."""
    if x is None:
        return (None, 0, 0, None, 0, 0, 0), None
    rows, heads = _rows(name, x, dim, n, dtype)
    if out is None:
        out = _empty((n, heads, dim), dtype, None, stream, x)
        to0, to1 = heads * dim, dim
    else:
        (to0, to1, _), out_heads = _rows(name + "_out", out, dim, n, dtype)
        if out_heads != heads:
            raise ValueError("%s_out has another number of heads" % name)
    if not x.get_device() == out.get_device() == dev:
        _check_device(dev, x, out)
    return (x.data_ptr(), rows[0], rows[1], out.data_ptr(), to0, to1, heads), out


# ---- the E4M3 cache ----------------------------------------------------------------
class E4m3Cache:
    """A paged cache of E4M3 codes: ``k_data`` [pages, Hkv, page_size, Dk] and
    ``v_data`` [pages, Hkv, page_size, Dv] (uint8 or float8_e4m3fn, any strides
    with contiguous rows, so a transposed view gives the [page, slot, head]
    layout) and float32 scales ``k_scale``, ``v_scale`` [pages, Hkv].  The
    tensors are those of its making: for others make another cache."""

    def __init__(self, k_data, v_data, k_scale, v_scale):
        pages, heads, page_size = k_data.shape[:3]
        s = E4m3CacheStruct()
        for pre, data, scale in (("k", k_data, k_scale), ("v", v_data, v_scale)):
            if data.dtype not in (torch.uint8, torch.float8_e4m3fn) or data.dim() != 4 or \
                    data.stride(3) != 1 or data.shape[:3] != k_data.shape[:3]:
                raise ValueError("%s_data must be [pages, heads, page_size, dim] bytes with "
                                 "contiguous rows" % pre)
            if scale.dtype != torch.float32 or tuple(scale.shape) != (pages, heads):
                raise ValueError("%s_scale must be float32 [pages, heads]" % pre)
            setattr(s, pre + "_data", data.data_ptr())
            setattr(s, pre + "_scale", scale.data_ptr())
            for i, n in ((0, "page"), (1, "head"), (2, "slot")):
                setattr(s, "%s_stride_%s" % (pre, n), data.stride(i))
            setattr(s, pre + "_scale_stride_page", 4 * scale.stride(0))
            setattr(s, pre + "_scale_stride_head", 4 * scale.stride(1))
        if len({t.device for t in (k_data, v_data, k_scale, v_scale)}) != 1:
            raise ValueError("the cache's tensors are on different devices")
        self.k_data, self.v_data, self.k_scale, self.v_scale = k_data, v_data, k_scale, v_scale
        self.device = k_data.get_device()
        self.num_pages, self.num_kv_heads, self.page_size = pages, heads, page_size
        self.head_dim_qk, self.head_dim_vo = k_data.shape[3], v_data.shape[3]
        s.num_pages, s.page_size, s.num_kv_heads = pages, page_size, heads
        s.head_dim_qk, s.head_dim_vo = self.head_dim_qk, self.head_dim_vo
        self._struct, self._ref = s, C.byref(s)

    @classmethod
    def allocate(cls, num_pages, num_kv_heads, head_dim_qk, head_dim_vo, page_size=16,
                 layout="HND", device="cuda"):
        """Buffers of an empty cache, [page][head][slot] (HND) or
        [page][slot][head] (NHD) in memory."""
        def data(dim):
            if layout == "HND":
                return torch.zeros((num_pages, num_kv_heads, page_size, dim), dtype=torch.uint8,
                                   device=device)
            if layout == "NHD":
                return torch.zeros((num_pages, page_size, num_kv_heads, dim), dtype=torch.uint8,
                                   device=device).transpose(1, 2)
            raise ValueError(layout)

        def scale():
            return torch.ones((num_pages, num_kv_heads), dtype=torch.float32, device=device)
        return cls(data(head_dim_qk), data(head_dim_vo), scale(), scale())


def nvfp4kv_e4m3_append(cache: E4m3Cache, k: torch.Tensor, v: torch.Tensor, qo_indptr, kv_indptr,
                        kv_indices, last_page_len, device_flags=None, stream=None):
    """Quantise the step's new tokens, k [rows, Hkv, Dk] and v [rows, Hkv, Dv]
    (request b's rows qo_indptr[b] .. qo_indptr[b + 1) are its last tokens),
    into their pages; the page table (int32, device) is that after the step."""
    code = _DTYPE.get(k.dtype)
    if code is None:
        raise ValueError("k must be torch.bfloat16 or torch.float16")
    rows, batch = k.shape[0], last_page_len.numel()
    ks, k_heads = _rows("k", k, cache.head_dim_qk, rows, k.dtype)
    vs, v_heads = _rows("v", v, cache.head_dim_vo, rows, k.dtype)
    if k_heads != cache.num_kv_heads or v_heads != k_heads or v.shape[0] != rows:
        raise ValueError("k and v must have the cache's heads and one number of rows")
    _ints(torch.int32, qo_indptr=qo_indptr, kv_indptr=kv_indptr, kv_indices=kv_indices,
          last_page_len=last_page_len)
    if qo_indptr.numel() != batch + 1 or kv_indptr.numel() != batch + 1:
        raise ValueError("indptrs must have one entry more than last_page_len")
    dev = torch.cuda.current_device()
    _check_device(dev, cache.k_data, k, v, qo_indptr, kv_indptr, kv_indices, last_page_len)
    st = _entry("nvfp4kv_e4m3_append")(
        cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], code, rows,
        qo_indptr.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(),
        last_page_len.data_ptr(), batch, _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_e4m3_append")


class _Run:
    """What every run of a plan with kernel 5 needs, taken from it once."""

    def __init__(self, plan: Plan):
        i = plan.info
        if plan.workspace is None:
            raise ValueError("the plan has no workspace (allocate=False)")
        self.rows, self.heads = i.total_qo_rows, i.num_qo_heads
        self.dk, self.dv = i.head_dim_qk, i.head_dim_vo
        # total_kv_pages leaves out requests without rows, which may stand in between
        self.pages = max(plan.kv_end, i.total_kv_pages)
        self.dtype = torch.float16 if i.out_dtype == 1 else torch.bfloat16
        self.of = plan.workspace
        self.workspace, self.nbytes = plan.workspace.data_ptr(), plan.workspace.numel()
        self.device = plan.workspace.get_device()
        self.info = C.byref(i)
        self.out_shape, self.lse_shape = (self.rows, self.heads, self.dv), (self.rows, self.heads)


def nvfp4kv_e4m3_decode_run(plan: Plan, q: torch.Tensor, cache: E4m3Cache, kv_indices,
                            sm_scale: float = 0.0, out=None, lse=None, stream=None):
    """Attention over an E4M3 cache with a plan made with ``kernel=5``: returns
    (out [rows, Hq, Dv], lse [rows, Hq])."""
    r = plan.__dict__.get("_e4m3_run")
    if r is None or r.of is not plan.workspace:
        r = plan._e4m3_run = _Run(plan)
    code = _DTYPE.get(q.dtype)
    if code is None:
        raise ValueError("q must be torch.bfloat16 or torch.float16")
    qs, heads = _rows("q", q, r.dk, r.rows, q.dtype)
    if heads != r.heads:
        raise ValueError("q must have the plan's heads")
    if kv_indices.dtype != torch.int32 or not kv_indices.is_contiguous():
        raise ValueError("kv_indices must be contiguous torch.int32")
    if kv_indices.numel() < r.pages:
        raise ValueError("kv_indices has %d entries, the plan reads %d"
                         % (kv_indices.numel(), r.pages))
    dev = torch.cuda.current_device()
    if not (q.get_device() == kv_indices.get_device() == cache.device == r.device == dev):
        _check_device(dev, q, kv_indices, cache.k_data, plan.workspace)
    if out is None:
        out = _empty(r.out_shape, r.dtype, q.device, stream)
    elif tuple(out.shape) != r.out_shape or out.dtype != r.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous %s [rows, Hq, Dv]" % r.dtype)
    if lse is None:
        lse = _empty(r.lse_shape, torch.float32, q.device, stream)
    elif tuple(lse.shape) != r.lse_shape or lse.dtype != torch.float32 or \
            not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [rows, Hq]")
    if out.get_device() != dev or lse.get_device() != dev:
        _check_device(dev, out, lse)
    st = _entry("nvfp4kv_e4m3_decode_run")(
        r.info, q.data_ptr(), qs[0], qs[1], code, cache._ref, kv_indices.data_ptr(),
        sm_scale or 0.0, r.workspace, r.nbytes, out.data_ptr(), lse.data_ptr(),
        _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_e4m3_decode_run")
    return out, lse
