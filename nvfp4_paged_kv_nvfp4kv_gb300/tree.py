"""Python binding of the entry points of a step that verifies drafted tokens
(include/nvfp4kv.h, same names): what the nodes of a tree see, their attention,
the accepted tokens moved together, and pages that several requests share.

Argument marshalling only, as in ``step``: tensors are checked for device, type
and shape here, what the library can check it checks itself (``NvFp4KvError``).
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from ._lib import TreeLaunch, check
from .api import PagedCache, Plan
from .step import E4m3Cache, _check_device, _empty, _entry, _flag_ptr, _stream_of

__all__ = ["nvfp4kv_tree_masks", "nvfp4kv_tree_run", "nvfp4kv_tree_form", "nvfp4kv_compact_tokens",
           "nvfp4kv_e4m3_compact_tokens", "nvfp4kv_fork_pages", "nvfp4kv_copy_pages",
           "nvfp4kv_e4m3_copy_pages", "nvfp4kv_release_pages"]

_MOST_NODES = 1024


def nvfp4kv_tree_masks(parents, qo_indptr, kv_len, max_nodes: Optional[int] = None,
                       tree_mask=None, positions=None, device_flags=None, stream=None):
    """What each drafted node sees of its tree, and its position, from ``parents``
    [rows] int32 (the index of a node's parent among its request's nodes, -1 for a
    root), ``qo_indptr`` [batch + 1] and ``kv_len`` [batch] (tokens with the nodes):
    returns (tree_mask [rows, words] int32, positions [rows] int32).  The words hold
    ``max_nodes`` nodes a request, unless ``tree_mask`` is given."""
    _i32("parents, qo_indptr and kv_len", parents, qo_indptr, kv_len)
    rows, batch, dev = parents.numel(), kv_len.numel(), torch.cuda.current_device()
    if qo_indptr.numel() != batch + 1:
        raise ValueError("qo_indptr must have one entry more than kv_len")
    if tree_mask is None:
        if max_nodes is None or not 1 <= max_nodes <= _MOST_NODES:
            raise ValueError("max_nodes must lie in [1, %d]" % _MOST_NODES)
        words = (max_nodes + 31) // 32
        tree_mask = _empty((rows, words), torch.int32, None, stream, parents)
    else:
        words = _mask_words(tree_mask, rows, rows)
        if max_nodes is not None and max_nodes > 32 * words:
            raise ValueError("tree_mask has too few words for max_nodes")
    if positions is None:
        positions = _empty((rows,), torch.int32, None, stream, parents)
    else:
        _i32("positions", positions)
        if positions.numel() != rows:
            raise ValueError("positions must have one entry a row")
    _check_device(dev, parents, qo_indptr, kv_len, tree_mask, positions)
    st = _entry("nvfp4kv_tree_masks")(
        parents.data_ptr(), qo_indptr.data_ptr(), kv_len.data_ptr(), batch, rows, words,
        tree_mask.data_ptr(), positions.data_ptr(), _flag_ptr(device_flags, dev),
        _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_tree_masks")
    return tree_mask, positions


def _i32(names, *tensors):
    for t in tensors:
        if t.dtype is not torch.int32 or not t.is_contiguous():
            raise ValueError("%s must be contiguous torch.int32" % names)


def _mask_words(mask, least, most):
    """Check a mask of `least` rows at least (`most` at most); its words a row."""
    shape = mask.shape
    if mask.dtype is not torch.int32 or len(shape) != 2 or shape[0] < least or \
            (most is not None and shape[0] > most) or not mask.is_contiguous():
        raise ValueError("tree_mask must be contiguous int32 [rows, words]")
    return shape[1]


class _Run:
    """What every tree run of a plan needs, taken from it once."""

    def __init__(self, plan: Plan):
        i = plan.info
        if plan.workspace is None:
            raise ValueError("the plan has no workspace (allocate=False)")
        self.of, self.info = plan.workspace, C.byref(i)
        self.rows, self.heads, self.kv_heads = i.total_qo_rows, i.num_qo_heads, i.num_kv_heads
        self.dk, self.dv = i.head_dim_qk, i.head_dim_vo
        # total_kv_pages leaves out requests without rows, which may stand in between
        self.pages = max(plan.kv_end, i.total_kv_pages)
        self.dtype = torch.float16 if i.out_dtype == 1 else torch.bfloat16
        self.workspace, self.nbytes = plan.workspace.data_ptr(), plan.workspace.numel()
        self.device = plan.workspace.get_device()
        self.out_shape = (self.rows, self.heads, self.dv)
        self.lse_shape = (self.rows, self.heads)


def _rows_of(name, x, rows, heads, dim):
    """Check bf16 [rows, heads, dim] with contiguous rows; the two strides."""
    shape, strides = x.shape, x.stride()
    if x.dtype is not torch.bfloat16 or len(shape) != 3 or strides[2] != 1 or \
            shape[0] < rows or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s must be bfloat16 [%d, %d, %d] with contiguous rows"
                         % (name, rows, heads, dim))
    return strides[0], strides[1]


def nvfp4kv_tree_run(plan: Plan, q, cache: PagedCache, kv_indices, tree_mask,
                     sm_scale: float = 0.0, new_k=None, new_v=None, out=None, lse=None,
                     stream=None):
    """Attention of the nodes of drafted trees: row i of q [rows, Hq, Dk] sees what stood
    before its request's rows, and of these those whose bits are set in its words of
    ``tree_mask`` [rows, words] int32; q is finite.  With ``new_k`` and ``new_v`` [rows, Hkv, D] the
    step's tokens are quantised into their pages by the same launch.  ``plan`` is one of
    kernel 0, 1 or 3.  Returns (out [rows, Hq, Dv], lse [rows, Hq])."""
    r = plan.__dict__.get("_tree_run")
    if r is None or r.of is not plan.workspace:
        r = plan._tree_run = _Run(plan)
    q0, q1 = _rows_of("q", q, r.rows, r.heads, r.dk)
    words = _mask_words(tree_mask, r.rows, None)
    _i32("kv_indices", kv_indices)
    if kv_indices.numel() < r.pages:
        raise ValueError("kv_indices has %d entries, the plan reads %d"
                         % (kv_indices.numel(), r.pages))
    dev = torch.cuda.current_device()
    if new_k is None and new_v is None:
        new = (None, 0, 0, None, 0, 0)
    elif new_k is None or new_v is None:
        raise ValueError("new_k and new_v: both or neither")
    else:
        new = (new_k.data_ptr(), *_rows_of("new_k", new_k, r.rows, r.kv_heads, r.dk),
               new_v.data_ptr(), *_rows_of("new_v", new_v, r.rows, r.kv_heads, r.dv))
        _check_device(dev, new_k, new_v)
    if not (q.get_device() == tree_mask.get_device() == kv_indices.get_device() == r.device
            == cache.k_data.get_device() == dev):
        _check_device(dev, q, tree_mask, kv_indices, cache.k_data, plan.workspace)
    if out is None:
        out = _empty(r.out_shape, r.dtype, q.device, stream,
                     q if r.dtype is torch.bfloat16 else None)
    elif out.shape != r.out_shape or out.dtype is not r.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous %s [rows, Hq, Dv]" % r.dtype)
    if lse is None:
        lse = _empty(r.lse_shape, torch.float32, q.device, stream)
    elif lse.shape != r.lse_shape or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [rows, Hq]")
    if out.get_device() != dev or lse.get_device() != dev:
        _check_device(dev, out, lse)
    st = _entry("nvfp4kv_tree_run")(
        r.info, tree_mask.data_ptr(), words, *new, q.data_ptr(), q0, q1, cache.struct(),
        kv_indices.data_ptr(), sm_scale or 0.0, r.workspace, r.nbytes, out.data_ptr(),
        lse.data_ptr(), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_tree_run")
    return out, lse


def nvfp4kv_tree_form(plan: Plan) -> dict:
    """How ``nvfp4kv_tree_run`` runs a plan on the current device: ``block_rows``,
    ``row_blocks``, ``cluster_ctas``, ``value_ctas``, ``whole_requests``, ``longest_first``
    and ``folded`` of include/nvfp4kv.h.  Nothing is launched."""
    form = TreeLaunch()
    check(_entry("nvfp4kv_tree_form")(C.byref(plan.info), C.byref(form)), "nvfp4kv_tree_form")
    return {name: getattr(form, name) for name, _ in TreeLaunch._fields_}


def _compact(name, cache, ref, path, num_kept, qo_indptr, kv_indptr, kv_indices, last_page_len,
             device_flags, stream):
    _i32("num_kept, the indptrs, kv_indices and last_page_len", num_kept, qo_indptr, kv_indptr,
         kv_indices, last_page_len)
    batch, shape, strides = last_page_len.numel(), path.shape, path.stride()
    if path.dtype is not torch.int32 or len(shape) != 2 or shape[0] != batch or \
            (shape[1] > 1 and strides[1] != 1):
        raise ValueError("path must be int32 [batch, most nodes] with contiguous rows")
    if num_kept.numel() != batch or qo_indptr.numel() != batch + 1 or \
            kv_indptr.numel() != batch + 1:
        raise ValueError("num_kept must have the batch's entries, the indptrs one more")
    dev = torch.cuda.current_device()
    _check_device(dev, cache.k_data, path, num_kept, qo_indptr, kv_indptr, kv_indices,
                  last_page_len)
    st = _entry(name)(
        ref, path.data_ptr(), strides[0], shape[1], num_kept.data_ptr(),
        qo_indptr.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(),
        last_page_len.data_ptr(), batch, _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, name)


def nvfp4kv_compact_tokens(cache: PagedCache, path, num_kept, qo_indptr, kv_indptr, kv_indices,
                           last_page_len, device_flags=None, stream=None):
    """Move the accepted tokens of every request together: of its rows of the step
    (qo_indptr), its last tokens in the page table of the step, those of the nodes
    ``path`` [batch, most] int32 (rising, the first ``num_kept[b]`` entries count) go to
    the first places.  A page with a drafted token is one request's alone."""
    _compact("nvfp4kv_compact_tokens", cache, cache.struct(), path, num_kept, qo_indptr,
             kv_indptr, kv_indices, last_page_len, device_flags, stream)


def nvfp4kv_e4m3_compact_tokens(cache: E4m3Cache, path, num_kept, qo_indptr, kv_indptr,
                                kv_indices, last_page_len, device_flags=None, stream=None):
    """``nvfp4kv_compact_tokens`` for an E4M3 cache (whose own attention is causal: for
    programs that attend to the tree in another way)."""
    _compact("nvfp4kv_e4m3_compact_tokens", cache, cache._ref, path, num_kept, qo_indptr,
             kv_indptr, kv_indices, last_page_len, device_flags, stream)


def _table(block_table, rows):
    """Check the block table; its rows' stride and its columns."""
    shape, strides = block_table.shape, block_table.stride()
    if block_table.dtype is not torch.int32 or len(shape) != 2 or \
            (shape[1] > 1 and strides[1] != 1):
        raise ValueError("block_table must be int32 [rows, pages] with contiguous rows")
    if shape[0] != rows:
        raise ValueError("block_table must have a row for every entry of kv_len")
    return strides[0], shape[1]


def _word(*heads):
    for t in heads:
        if t.numel() < 1:
            raise ValueError("a free head is empty")


def nvfp4kv_fork_pages(parents, children, kv_len, block_table, page_shares, free_pages,
                       free_head, free_head_out, copy_src, copy_dst, page_size: int = 16,
                       device_flags=None, stream=None):
    """Make rows ``children`` [forks] of the block table, which are empty (``kv_len`` 0:
    release what is there first), requests that share the whole pages of rows ``parents``
    [forks]; a last page that is not full is replaced by a new one off the free list, and
    the pair stands in ``copy_src`` / ``copy_dst`` [forks] (-1 where there is none) for
    ``nvfp4kv_copy_pages`` on every layer's cache.  ``kv_len`` [rows] and ``page_shares``
    [pages of the pool] (owners beyond the first) are updated; ``free_head`` [1] is read,
    ``free_head_out`` [1], another word, is written."""
    _i32("the lists", parents, children, kv_len, page_shares, free_pages, free_head,
         free_head_out, copy_src, copy_dst)
    forks, rows = parents.numel(), kv_len.numel()
    if not children.numel() == copy_src.numel() == copy_dst.numel() == forks:
        raise ValueError("parents, children, copy_src and copy_dst must have one length")
    table_stride, width = _table(block_table, rows)
    _word(free_head, free_head_out)
    dev = torch.cuda.current_device()
    _check_device(dev, parents, children, kv_len, block_table, page_shares, free_pages,
                  free_head, free_head_out, copy_src, copy_dst)
    st = _entry("nvfp4kv_fork_pages")(
        parents.data_ptr(), children.data_ptr(), forks, kv_len.data_ptr(), rows, page_size,
        block_table.data_ptr(), table_stride, width,
        page_shares.data_ptr(), page_shares.numel(), free_pages.data_ptr(), free_pages.numel(),
        free_head.data_ptr(), free_head_out.data_ptr(), copy_src.data_ptr(),
        copy_dst.data_ptr(), _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_fork_pages")


def _copy(name, cache, ref, src, dst, device_flags, stream):
    _i32("src and dst", src, dst)
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have one length")
    dev = torch.cuda.current_device()
    _check_device(dev, cache.k_data, src, dst)
    st = _entry(name)(ref, src.data_ptr(), dst.data_ptr(), src.numel(),
                      _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, name)


def nvfp4kv_copy_pages(cache: PagedCache, src, dst, device_flags=None, stream=None):
    """Copy pages ``src`` [n] of the cache to pages ``dst`` [n] (int32, device; a pair
    (-1, -1) is passed over).  A page that is written must not be in another pair."""
    _copy("nvfp4kv_copy_pages", cache, cache.struct(), src, dst, device_flags, stream)


def nvfp4kv_e4m3_copy_pages(cache: E4m3Cache, src, dst, device_flags=None, stream=None):
    """``nvfp4kv_copy_pages`` for an E4M3 cache."""
    _copy("nvfp4kv_e4m3_copy_pages", cache, cache._ref, src, dst, device_flags, stream)


def nvfp4kv_release_pages(keep_len, kv_len, block_table, page_shares, free_pages, free_head,
                          free_head_out=None, page_size: int = 16, device_flags=None,
                          stream=None):
    """Row b of the block table keeps its first ``keep_len[b]`` of ``kv_len[b]`` tokens and
    gives the pages behind them up: a page without another owner goes back in front of
    the free list's head (``free_head`` [1]; the new one goes to ``free_head_out``, by
    default the same word).  ``kv_len`` and ``page_shares`` are updated.  A request cut
    inside a page with other owners must not grow there, over their tokens (fork it
    first)."""
    if free_head_out is None:
        free_head_out = free_head
    _i32("the lists", keep_len, kv_len, page_shares, free_pages, free_head, free_head_out)
    rows = kv_len.numel()
    if keep_len.numel() != rows:
        raise ValueError("keep_len and kv_len must have one length")
    table_stride, width = _table(block_table, rows)
    _word(free_head, free_head_out)
    dev = torch.cuda.current_device()
    _check_device(dev, keep_len, kv_len, block_table, page_shares, free_pages, free_head,
                  free_head_out)
    st = _entry("nvfp4kv_release_pages")(
        keep_len.data_ptr(), kv_len.data_ptr(), rows, page_size, block_table.data_ptr(),
        table_stride, width, page_shares.data_ptr(),
        page_shares.numel(), free_pages.data_ptr(), free_pages.numel(), free_head.data_ptr(),
        free_head_out.data_ptr(), _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_release_pages")
