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

from ._lib import check
from .api import PagedCache, Plan
from .step import E4m3Cache, _check_device, _empty, _entry, _flag_ptr, _ints, _stream_of

__all__ = ["nvfp4kv_tree_masks", "nvfp4kv_tree_run", "nvfp4kv_compact_tokens",
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
    _ints(torch.int32, parents=parents, qo_indptr=qo_indptr, kv_len=kv_len, positions=positions)
    rows, batch, dev = parents.numel(), kv_len.numel(), torch.cuda.current_device()
    if qo_indptr.numel() != batch + 1:
        raise ValueError("qo_indptr must have one entry more than kv_len")
    if tree_mask is None:
        if max_nodes is None or not 1 <= max_nodes <= _MOST_NODES:
            raise ValueError("max_nodes must lie in [1, %d]" % _MOST_NODES)
        tree_mask = _empty((rows, (max_nodes + 31) // 32), torch.int32, parents.device, stream)
    elif tree_mask.dtype != torch.int32 or tree_mask.dim() != 2 or \
            tree_mask.shape[0] != rows or not tree_mask.is_contiguous():
        raise ValueError("tree_mask must be contiguous int32 [rows, words]")
    elif max_nodes is not None and max_nodes > 32 * tree_mask.shape[1]:
        raise ValueError("tree_mask has too few words for max_nodes")
    if positions is None:
        positions = _empty((rows,), torch.int32, parents.device, stream)
    elif positions.numel() != rows:
        raise ValueError("positions must have one entry a row")
    _check_device(dev, parents, qo_indptr, kv_len, tree_mask, positions)
    st = _entry("nvfp4kv_tree_masks")(
        parents.data_ptr(), qo_indptr.data_ptr(), kv_len.data_ptr(), batch, rows,
        tree_mask.shape[1], tree_mask.data_ptr(), positions.data_ptr(),
        _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_tree_masks")
    return tree_mask, positions


def _rows_of(name, x, rows, heads, dim):
    """Check bf16 [rows, heads, dim] with contiguous rows; the two strides."""
    if x.dtype != torch.bfloat16 or x.dim() != 3 or x.stride(2) != 1 or x.shape[0] < rows or \
            x.shape[1] != heads or x.shape[2] != dim:
        raise ValueError("%s must be bfloat16 [%d, %d, %d] with contiguous rows"
                         % (name, rows, heads, dim))
    return x.stride(0), x.stride(1)


def nvfp4kv_tree_run(plan: Plan, q, cache: PagedCache, kv_indices, tree_mask,
                     sm_scale: float = 0.0, new_k=None, new_v=None, out=None, lse=None,
                     stream=None):
    """Attention of the nodes of drafted trees: row i of q [rows, Hq, Dk] sees what stood
    before its request's rows, and of these those whose bits are set in its words of
    ``tree_mask`` [rows, words] int32.  With ``new_k`` and ``new_v`` [rows, Hkv, D] the
    step's tokens are quantised into their pages by the same launch.  ``plan`` is one of
    kernel 0, 1 or 3.  Returns (out [rows, Hq, Dv], lse [rows, Hq])."""
    i = plan.info
    if plan.workspace is None:
        raise ValueError("the plan has no workspace (allocate=False)")
    rows, hkv, dk, dv = i.total_qo_rows, i.num_kv_heads, i.head_dim_qk, i.head_dim_vo
    qs = _rows_of("q", q, rows, i.num_qo_heads, dk)
    if tree_mask.dtype != torch.int32 or tree_mask.dim() != 2 or tree_mask.shape[0] < rows or \
            not tree_mask.is_contiguous():
        raise ValueError("tree_mask must be contiguous int32 [rows, words]")
    _ints(torch.int32, kv_indices=kv_indices)
    pages = max(plan.kv_end, i.total_kv_pages)
    if kv_indices.numel() < pages:
        raise ValueError("kv_indices has %d entries, the plan reads %d"
                         % (kv_indices.numel(), pages))
    if (new_k is None) != (new_v is None):
        raise ValueError("new_k and new_v: both or neither")
    new = (None, 0, 0, None, 0, 0)
    if new_k is not None:
        new = (new_k.data_ptr(), *_rows_of("new_k", new_k, rows, hkv, dk),
               new_v.data_ptr(), *_rows_of("new_v", new_v, rows, hkv, dv))
    dev = torch.cuda.current_device()
    _check_device(dev, q, tree_mask, kv_indices, cache.k_data, plan.workspace,
                  *(() if new_k is None else (new_k, new_v)))
    dtype = torch.float16 if i.out_dtype == 1 else torch.bfloat16
    if out is None:
        out = _empty((rows, i.num_qo_heads, dv), dtype, q.device, stream)
    elif tuple(out.shape) != (rows, i.num_qo_heads, dv) or out.dtype != dtype or \
            not out.is_contiguous():
        raise ValueError("out must be contiguous %s [rows, Hq, Dv]" % dtype)
    if lse is None:
        lse = _empty((rows, i.num_qo_heads), torch.float32, q.device, stream)
    elif tuple(lse.shape) != (rows, i.num_qo_heads) or lse.dtype != torch.float32 or \
            not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [rows, Hq]")
    _check_device(dev, out, lse)
    st = _entry("nvfp4kv_tree_run")(
        C.byref(i), tree_mask.data_ptr(), tree_mask.shape[1], *new, q.data_ptr(), *qs,
        cache.struct(), kv_indices.data_ptr(), sm_scale or 0.0, plan.workspace.data_ptr(),
        plan.workspace.numel(), out.data_ptr(), lse.data_ptr(), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_tree_run")
    return out, lse


def _compact(name, cache, ref, path, num_kept, qo_indptr, kv_indptr, kv_indices, last_page_len,
             device_flags, stream):
    _ints(torch.int32, num_kept=num_kept, qo_indptr=qo_indptr, kv_indptr=kv_indptr,
          kv_indices=kv_indices, last_page_len=last_page_len)
    batch = last_page_len.numel()
    if path.dtype != torch.int32 or path.dim() != 2 or path.shape[0] != batch or \
            (path.shape[1] > 1 and path.stride(1) != 1):
        raise ValueError("path must be int32 [batch, most nodes] with contiguous rows")
    if num_kept.numel() != batch or qo_indptr.numel() != batch + 1 or \
            kv_indptr.numel() != batch + 1:
        raise ValueError("num_kept must have the batch's entries, the indptrs one more")
    dev = torch.cuda.current_device()
    _check_device(dev, cache.k_data, path, num_kept, qo_indptr, kv_indptr, kv_indices,
                  last_page_len)
    st = _entry(name)(
        ref, path.data_ptr(), path.stride(0), path.shape[1], num_kept.data_ptr(),
        qo_indptr.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(),
        last_page_len.data_ptr(), batch, _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, name)


def nvfp4kv_compact_tokens(cache: PagedCache, path, num_kept, qo_indptr, kv_indptr, kv_indices,
                           last_page_len, device_flags=None, stream=None):
    """Move the accepted tokens of every request together: of its rows of the step
    (qo_indptr), its last tokens in the page table of the step, those of the nodes
    ``path`` [batch, most] int32 (rising, the first ``num_kept[b]`` entries count) go to
    the first places."""
    _compact("nvfp4kv_compact_tokens", cache, cache.struct(), path, num_kept, qo_indptr,
             kv_indptr, kv_indices, last_page_len, device_flags, stream)


def nvfp4kv_e4m3_compact_tokens(cache: E4m3Cache, path, num_kept, qo_indptr, kv_indptr,
                                kv_indices, last_page_len, device_flags=None, stream=None):
    """``nvfp4kv_compact_tokens`` for an E4M3 cache."""
    _compact("nvfp4kv_e4m3_compact_tokens", cache, cache._ref, path, num_kept, qo_indptr,
             kv_indptr, kv_indices, last_page_len, device_flags, stream)


def _table(block_table, rows):
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [rows, pages] with contiguous rows")
    if block_table.shape[0] != rows:
        raise ValueError("block_table must have a row for every entry of kv_len")


def _word(**tensors):
    for name, t in tensors.items():
        if t.numel() < 1:
            raise ValueError("%s is empty" % name)


def nvfp4kv_fork_pages(parents, children, kv_len, block_table, page_shares, free_pages,
                       free_head, free_head_out, copy_src, copy_dst, page_size: int = 16,
                       device_flags=None, stream=None):
    """Make rows ``children`` [forks] of the block table requests that share the whole
    pages of rows ``parents`` [forks]; a last page that is not full is replaced by a new
    one off the free list, and the pair stands in ``copy_src`` / ``copy_dst`` [forks] (-1
    where there is none) for ``nvfp4kv_copy_pages`` on every layer's cache.  ``kv_len``
    [rows] and ``page_shares`` [pages of the pool] (owners beyond the first) are updated;
    ``free_head`` [1] is read, ``free_head_out`` [1], another word, is written."""
    _ints(torch.int32, parents=parents, children=children, kv_len=kv_len,
          page_shares=page_shares, free_pages=free_pages, free_head=free_head,
          free_head_out=free_head_out, copy_src=copy_src, copy_dst=copy_dst)
    forks, rows = parents.numel(), kv_len.numel()
    if not children.numel() == copy_src.numel() == copy_dst.numel() == forks:
        raise ValueError("parents, children, copy_src and copy_dst must have one length")
    _table(block_table, rows)
    _word(free_head=free_head, free_head_out=free_head_out)
    dev = torch.cuda.current_device()
    _check_device(dev, parents, children, kv_len, block_table, page_shares, free_pages,
                  free_head, free_head_out, copy_src, copy_dst)
    st = _entry("nvfp4kv_fork_pages")(
        parents.data_ptr(), children.data_ptr(), forks, kv_len.data_ptr(), rows, page_size,
        block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
        page_shares.data_ptr(), page_shares.numel(), free_pages.data_ptr(), free_pages.numel(),
        free_head.data_ptr(), free_head_out.data_ptr(), copy_src.data_ptr(),
        copy_dst.data_ptr(), _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_fork_pages")


def _copy(name, cache, ref, src, dst, device_flags, stream):
    _ints(torch.int32, src=src, dst=dst)
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
    default the same word).  ``kv_len`` and ``page_shares`` are updated."""
    if free_head_out is None:
        free_head_out = free_head
    _ints(torch.int32, keep_len=keep_len, kv_len=kv_len, page_shares=page_shares,
          free_pages=free_pages, free_head=free_head, free_head_out=free_head_out)
    rows = kv_len.numel()
    if keep_len.numel() != rows:
        raise ValueError("keep_len and kv_len must have one length")
    _table(block_table, rows)
    _word(free_head=free_head, free_head_out=free_head_out)
    dev = torch.cuda.current_device()
    _check_device(dev, keep_len, kv_len, block_table, page_shares, free_pages, free_head,
                  free_head_out)
    st = _entry("nvfp4kv_release_pages")(
        keep_len.data_ptr(), kv_len.data_ptr(), rows, page_size, block_table.data_ptr(),
        block_table.stride(0), block_table.shape[1], page_shares.data_ptr(),
        page_shares.numel(), free_pages.data_ptr(), free_pages.numel(), free_head.data_ptr(),
        free_head_out.data_ptr(), _flag_ptr(device_flags, dev), _stream_of(stream, dev))
    if st:
        check(st, "nvfp4kv_release_pages")
