"""Tensor-level calls of the decode's forms for long and shared contexts (include/gqa_paged_decode.h).

A batch that shares prefixes (``shared_run``); blocks bounded, chosen and attended to (``block_bounds``,
``block_select``, ``block_sparse_run``); attention weights accumulated beside the decode and the eviction by them
(``run_weighted``, ``kv_evict``). As in ``serving``: argument checks and marshalling only, no CPU path; a call runs on
the current stream of its tensors' device unless ``stream`` is given, and what it allocates, its workspace among it,
belongs to that stream.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from ._lib import HEAD_DIM, NUM_KV_HEADS, NUM_QO_HEADS, load
from .serving import CACHE_BF16, _INT_MAX, _cache_format, _call, _check, _empty_strided_cuda, _entries, _index, _new


_SCALE = HEAD_DIM ** -0.5
_OUT_STRIDE, _LSE_STRIDE = (NUM_QO_HEADS * HEAD_DIM, HEAD_DIM, 1), (NUM_QO_HEADS, 1)
_BF16_PAGE = (1, NUM_KV_HEADS, HEAD_DIM)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _plain(index, dtype, dim, *tensors):
    """Whether all are contiguous tensors of `dtype` with `dim` dimensions on GPU `index`: the common case, in few steps."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != index or t.ndim != dim or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return True


def _need(index, dtype, dim, **tensors):
    """Raises unless all are contiguous tensors of `dtype` with `dim` dimensions on GPU `index`."""
    for name, t in tensors.items():
        _check(index, dtype, True, **{name: t})
        if t.dim() != dim:
            raise ValueError(f"{name} must have {dim} dimension{'s' if dim > 1 else ''}, not {t.dim()}")


def _queries(index, q):
    if not _plain(index, _BF16, 3, q):
        _need(index, _BF16, 3, q=q)
    n, heads, dim = q.shape
    if heads != NUM_QO_HEADS or dim != HEAD_DIM:
        raise ValueError("expected q [N, 32, 128]")
    return n


def _paged(index, k_cache, v_cache):
    """(format, pages) of CSR-paged caches."""
    if _plain(index, _BF16, 4, k_cache, v_cache):
        shape = k_cache.shape
        if shape[1:] == _BF16_PAGE and v_cache.shape == shape:
            return CACHE_BF16, shape[0]
    _check(index, None, True, k_cache=k_cache, v_cache=v_cache)
    return _cache_format(k_cache, v_cache)


_current = torch._C._cuda_getDevice


def _alloc(index, shape, stride, dtype, stream):
    """_new with the strides of a contiguous tensor of that shape, known to the caller."""
    if stream is None and _empty_strided_cuda is not None and index == _current():
        return _empty_strided_cuda(shape, stride, dtype)
    return _new(index, shape, dtype, stream)


def _results(index, n, out, lse, with_lse, stream):
    """out [n, 32, 128] and lse [n, 32] (or None), allocated where they are not given."""
    if out is None:
        out = _alloc(index, (n, NUM_QO_HEADS, HEAD_DIM), _OUT_STRIDE, _BF16, stream)
    else:
        _check(index, _BF16, True, out=out)
        if out.shape != (n, NUM_QO_HEADS, HEAD_DIM):
            raise ValueError(f"out must be {(n, NUM_QO_HEADS, HEAD_DIM)}")
    if lse is not None:
        _check(index, _F32, True, lse=lse)
        if lse.shape != (n, NUM_QO_HEADS):
            raise ValueError(f"lse must be {(n, NUM_QO_HEADS)}")
    elif with_lse:
        lse = _alloc(index, (n, NUM_QO_HEADS), _LSE_STRIDE, _F32, stream)
    return out, lse


def _workspace(index, given, stream, what, *sizes):
    """(tensor, bytes) of the call's own workspace, or the given one."""
    if given is not None:
        _check(index, None, True, workspace=given)
        return given, given.numel() * given.element_size()
    size_of = _entries.get(what)
    if size_of is None:
        size_of = _entries[what] = getattr(load(), what)
    if index == _current():
        size = size_of(*sizes)
    else:
        with torch.cuda.device(index):
            size = size_of(*sizes)
    if size == 0:
        raise ValueError(f"sizes {sizes} are out of range")
    return _alloc(index, (size,), (1,), torch.uint8, stream), size


def _fit(*counts):
    """Raises for counts that a C int would cut."""
    if max(counts) > _INT_MAX:
        raise ValueError(f"more than {_INT_MAX} entries")


def _pointer(t):
    return None if t is None else t.data_ptr()


def shared_run(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, prefix_indptr: torch.Tensor,
               prefix_indices: torch.Tensor, group_indptr: torch.Tensor, kv_indptr: torch.Tensor,
               kv_indices: torch.Tensor, sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``run`` (bf16 caches [P, 1, 4, 128]) or ``run_fp8`` (FP8 caches [P, 528]) for a batch whose sequences share
    prefixes, each read once: sequence b of group g (group_indptr[g] <= b < group_indptr[g + 1]) attends to the pages
    prefix_indices[prefix_indptr[g]:prefix_indptr[g + 1]], then to its own in kv_indptr and kv_indices; sequences of no
    group to their own alone. Returns (out [B, 32, 128] bf16, lse [B, 32] fp32, base 2)."""
    index = _index("q", q)
    n = _queries(index, q)
    fmt, pages = _paged(index, k_cache, v_cache)
    if not _plain(index, _I32, 1, prefix_indptr, prefix_indices, group_indptr, kv_indptr, kv_indices):
        _need(index, _I32, 1, prefix_indptr=prefix_indptr, prefix_indices=prefix_indices, group_indptr=group_indptr,
              kv_indptr=kv_indptr, kv_indices=kv_indices)
    groups = group_indptr.shape[0] - 1
    _fit(n, groups, prefix_indices.shape[0], kv_indices.shape[0], pages)
    if groups < 0 or prefix_indptr.shape[0] != groups + 1 or kv_indptr.shape[0] != n + 1:
        raise ValueError(f"expected prefix_indptr and group_indptr [G + 1] and kv_indptr [{n + 1}]")
    out, lse = _results(index, n, out, lse, True, stream)
    if n == 0:
        return out, lse
    ws, size = _workspace(index, workspace, stream, "gqa_shared_paged_decode_ws_size", n, groups, fmt)
    _call("gqa_shared_paged_decode", index, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          prefix_indptr.data_ptr(), prefix_indices.data_ptr(), group_indptr.data_ptr(), kv_indptr.data_ptr(),
          kv_indices.data_ptr(), _SCALE if sm_scale is None else sm_scale, out.data_ptr(), lse.data_ptr(), n,
          groups, prefix_indices.shape[0], kv_indices.shape[0], pages, fmt, ws.data_ptr(), size)
    return out, lse


def _blocked(index, name, cache):
    """(blocks, page size) of a block-table cache [blocks, page, 4, 128]."""
    if not _plain(index, _BF16, 4, cache):
        _need(index, _BF16, 4, **{name: cache})
    blocks, page, heads, dim = cache.shape
    if heads != NUM_KV_HEADS or dim != HEAD_DIM:
        raise ValueError(f"expected {name} [blocks, page_size, 4, 128]")
    return blocks, page


def _table(index, block_table):
    if not _plain(index, _I32, 2, block_table):
        _need(index, _I32, 2, block_table=block_table)
    return block_table.shape


def _bounds(index, bounds):
    if not _plain(index, _BF16, 4, bounds):
        _need(index, _BF16, 4, bounds=bounds)
    blocks, two, heads, dim = bounds.shape
    if two != 2 or heads != NUM_KV_HEADS or dim != HEAD_DIM:
        raise ValueError("expected bounds [blocks, 2, 4, 128]")
    return blocks


def block_bounds(k_cache: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 first: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The largest (bounds[:, 0]) and smallest (bounds[:, 1]) key values of the blocks that hold the new tokens
    first[r] <= t < lens[r] (first None: from 0) of each request of block_table [requests, width], over all of the
    block's tokens below lens[r]; k_cache [blocks, page_size, 4, 128], bounds [blocks, 2, 4, 128], in place. To be
    called after the tokens' rows are stored. Returns bounds."""
    index = _index("k_cache", k_cache)
    blocks, page = _blocked(index, "k_cache", k_cache)
    requests, width = _table(index, block_table)
    if not _plain(index, _I32, 1, lens):
        _need(index, _I32, 1, lens=lens)
    if first is not None and not _plain(index, _I32, 1, first):
        _need(index, _I32, 1, first=first)
    _fit(requests, width, blocks, page)
    if _bounds(index, bounds) != blocks or lens.shape[0] != requests or (first is not None and first.shape[0] != requests):
        raise ValueError("expected bounds [blocks, 2, 4, 128], and lens and first [requests]")
    _call("gqa_block_bounds", index, stream, k_cache.data_ptr(), bounds.data_ptr(), block_table.data_ptr(),
          lens.data_ptr(), _pointer(first), requests, page, blocks, width)
    return bounds


def block_select(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, token_to_req: torch.Tensor,
                 lens: torch.Tensor, top: int, page_size: int, keep_first: int = 1, keep_last: int = 1,
                 blocks: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The `top` blocks of each query row and KV head: of the blocks that hold tokens below lens[row] of request
    token_to_req[row], the first keep_first and last keep_last, then those whose bounds allow the largest product with
    one of the head's 8 queries (ties to the lower block). q [rows, 32, 128]. Returns their numbers in the table,
    ascending, then -1: int32 [rows, 4, top]."""
    index = _index("q", q)
    rows = _queries(index, q)
    held = _bounds(index, bounds)
    requests, width = _table(index, block_table)
    _fit(rows, requests, width, held)
    if not _plain(index, _I32, 1, token_to_req, lens):
        _need(index, _I32, 1, token_to_req=token_to_req, lens=lens)
    if token_to_req.shape[0] != rows or lens.shape[0] != rows:
        raise ValueError(f"token_to_req and lens must be [{rows}]")
    if not (0 <= keep_first and 0 <= keep_last and 0 < top <= _INT_MAX and 0 < page_size <= _INT_MAX):
        raise ValueError("top, page_size, keep_first or keep_last is out of range")
    if keep_first + keep_last > top:
        raise ValueError("keep_first and keep_last take more than top blocks")
    if blocks is None:
        blocks = _alloc(index, (rows, NUM_KV_HEADS, top), (NUM_KV_HEADS * top, top, 1), _I32, stream)
    else:
        _check(index, torch.int32, True, blocks=blocks)
        if blocks.shape != (rows, NUM_KV_HEADS, top):
            raise ValueError(f"blocks must be {(rows, NUM_KV_HEADS, top)}")
    if rows == 0:
        return blocks
    ws, size = _workspace(index, workspace, stream, "gqa_block_select_ws_size", rows, width)
    _call("gqa_block_select", index, stream, q.data_ptr(), bounds.data_ptr(), block_table.data_ptr(),
          token_to_req.data_ptr(), lens.data_ptr(), blocks.data_ptr(), rows, requests, page_size, held, width, top,
          keep_first, keep_last, ws.data_ptr(), size)
    return blocks


def block_sparse_run(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, blocks: torch.Tensor,
                     block_table: torch.Tensor, token_to_req: torch.Tensor, lens: torch.Tensor,
                     sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, with_lse: bool = True,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``sparse_run`` with a list of blocks for each KV head, as ``block_select`` returns: row r attends, with the
    query heads of KV head g, to the tokens below lens[r] of the blocks blocks[r, g] of request token_to_req[r].
    Returns (out [rows, 32, 128] bf16, lse [rows, 32] fp32, base 2, or None)."""
    index = _index("q", q)
    rows = _queries(index, q)
    held, page = _blocked(index, "k_cache", k_cache)
    if _blocked(index, "v_cache", v_cache) != (held, page):
        raise ValueError("k_cache and v_cache must have the same shape")
    requests, width = _table(index, block_table)
    if not _plain(index, _I32, 1, token_to_req, lens):
        _need(index, _I32, 1, token_to_req=token_to_req, lens=lens)
    if not _plain(index, _I32, 3, blocks):
        _need(index, _I32, 3, blocks=blocks)
    listed, heads, top = blocks.shape
    _fit(rows, requests, width, held, page, top)
    if listed != rows or heads != NUM_KV_HEADS:
        raise ValueError(f"blocks must be [{rows}, 4, top]")
    if token_to_req.shape[0] != rows or lens.shape[0] != rows:
        raise ValueError(f"token_to_req and lens must be [{rows}]")
    out, lse = _results(index, rows, out, lse, with_lse, stream)
    if rows == 0:
        return out, lse
    ws, size = _workspace(index, workspace, stream, "gqa_block_sparse_decode_ws_size", rows, top, page)
    _call("gqa_block_sparse_decode", index, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          blocks.data_ptr(), block_table.data_ptr(), token_to_req.data_ptr(), lens.data_ptr(),
          _SCALE if sm_scale is None else sm_scale, out.data_ptr(), _pointer(lse), rows, requests, top, page,
          held, width, ws.data_ptr(), size)
    return out, lse


def run_weighted(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_indptr: torch.Tensor,
                 kv_indices: torch.Tensor, weights: torch.Tensor, decay: float = 1.0,
                 sm_scale: Optional[float] = None, weights_out: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``run`` (bf16 caches) or ``run_fp8`` (FP8 caches) that also accumulates the attention each token gets: for the
    j-th token of sequence b, weights_out[b, j] = decay * weights[b, j] + the sum over the 32 heads of its softmax
    weight. weights: fp32 [B, width]; places past a sequence's length are copied, tokens past width not accumulated.
    weights_out: a tensor like weights, possibly weights itself (default: a new one). Returns (out [B, 32, 128] bf16,
    lse [B, 32] fp32, base 2, weights_out)."""
    index = _index("q", q)
    n = _queries(index, q)
    fmt, pages = _paged(index, k_cache, v_cache)
    if not (_plain(index, _I32, 1, kv_indptr, kv_indices) and _plain(index, _F32, 2, weights)):
        _need(index, _I32, 1, kv_indptr=kv_indptr, kv_indices=kv_indices)
        _need(index, _F32, 2, weights=weights)
    rows, width = weights.shape
    _fit(n, width, kv_indices.shape[0], pages)
    if rows != n or kv_indptr.shape[0] != n + 1:
        raise ValueError(f"expected weights [{n}, width] and kv_indptr [{n + 1}]")
    if not math.isfinite(decay):
        raise ValueError("decay must be finite")
    if weights_out is None:
        weights_out = _alloc(index, (n, width), (max(width, 1), 1), _F32, stream)
    else:
        _check(index, torch.float32, True, weights_out=weights_out)
        if weights_out.shape != weights.shape:
            raise ValueError("weights_out must have weights' shape")
    out, lse = _results(index, n, out, lse, True, stream)
    if n == 0:
        return out, lse, weights_out
    ws, size = _workspace(index, workspace, stream, "gqa_paged_decode_weighted_ws_size", kv_indices.shape[0], fmt)
    _call("gqa_paged_decode_weighted", index, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          kv_indptr.data_ptr(), kv_indices.data_ptr(), _SCALE if sm_scale is None else sm_scale,
          weights.data_ptr(), decay, weights_out.data_ptr(), out.data_ptr(), lse.data_ptr(), n, width,
          kv_indices.shape[0], pages, fmt, ws.data_ptr(), size)
    return out, lse, weights_out


def kv_evict(weights: torch.Tensor, kv_indptr: torch.Tensor, kv_indices: torch.Tensor, budget: int, keep_first: int = 0,
             keep_last: int = 0, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """Cuts sequences of more than `budget` tokens back to it: the first keep_first and last keep_last tokens stay and,
    of those between, the ones of the largest weights[b, j] (ties: the lower j), in order. Returns (weights [B, width]
    at the tokens' new places, then zeros; kv_indptr [B + 1]; kv_indices; freed_indptr [B + 1]; freed): the tokens kept
    as a page table, and the other tokens' pages in the same form. kv_indices and freed are as long as the given
    kv_indices, -1 behind the last sequence's."""
    index = _index("weights", weights)
    if not (_plain(index, _F32, 2, weights) and _plain(index, _I32, 1, kv_indptr, kv_indices)):
        _need(index, _F32, 2, weights=weights)
        _need(index, _I32, 1, kv_indptr=kv_indptr, kv_indices=kv_indices)
    (n, width), total = weights.shape, kv_indices.shape[0]
    if kv_indptr.shape[0] != n + 1:
        raise ValueError("expected weights [B, width] and kv_indptr [B + 1]")
    _fit(n, width, total)
    if not (0 <= keep_first and 0 <= keep_last and 0 <= budget <= _INT_MAX):
        raise ValueError("budget, keep_first or keep_last is out of range")
    if keep_first + keep_last > budget:
        raise ValueError("keep_first and keep_last take more than the budget")
    got = _alloc(index, (n, width), (max(width, 1), 1), _F32, stream)
    indptr = _alloc(index, (n + 1,), (1,), _I32, stream)
    freed_indptr = _alloc(index, (n + 1,), (1,), _I32, stream)
    indices = _alloc(index, (total,), (1,), _I32, stream)
    freed = _alloc(index, (total,), (1,), _I32, stream)
    if n == 0:
        with torch.cuda.stream(stream):
            indptr.zero_(), freed_indptr.zero_(), indices.fill_(-1), freed.fill_(-1)
        return got, indptr, indices, freed_indptr, freed
    _call("gqa_kv_evict", index, stream, weights.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(), budget,
          keep_first, keep_last, got.data_ptr(), indptr.data_ptr(), indices.data_ptr(), freed_indptr.data_ptr(),
          freed.data_ptr(), n, width, total)
    return got, indptr, indices, freed_indptr, freed
