"""Tensor-level calls of the decode's forms for long and shared contexts (include/gqa_paged_decode.h).

A batch that shares prefixes (``shared_run``); blocks bounded, chosen and attended to (``block_bounds``,
``block_select``, ``block_sparse_run``); attention weights accumulated beside the decode and the eviction by them
(``run_weighted``, ``kv_evict``). As in ``serving``: argument checks and marshalling only, no CPU path; a call runs on
the current stream of its tensors' device unless ``stream`` is given, and what it allocates, its workspace among it,
belongs to that stream.

A call's tensors are looked at in one step of C++ (csrc/context_host.cpp), or one by one where that finds anything amiss
or is not built: a call of one step of 16 sequences with accumulated weights took 24 us one by one, its kernels 21.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from ._lib import HEAD_DIM, NUM_KV_HEADS, NUM_QO_HEADS, load
from .serving import CACHE_BF16, CACHE_FP8, _INT_MAX, _cache_format, _call, _check, _empty_strided_cuda, _entries, _index, _new


_SCALE = HEAD_DIM ** -0.5
_OUT_STRIDE, _LSE_STRIDE = (NUM_QO_HEADS * HEAD_DIM, HEAD_DIM, 1), (NUM_QO_HEADS, 1)
_BF16_PAGE, _FP8_PAGE = (1, NUM_KV_HEADS, HEAD_DIM), (NUM_KV_HEADS * (HEAD_DIM + 4),)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


_TYPES = {"b": _BF16, "f": _F32, "i": _I32, "u": torch.uint8}
_CACHES = {_BF16: (b"b4b4", CACHE_BF16, 4), torch.uint8: (b"u2u2", CACHE_FP8, 2)}
_gather = None


def _no_gather(spec, *tensors):
    return None


def _built():
    """The C++ step if it was built for this PyTorch, or one that finds nothing."""
    global _gather
    _gather = _no_gather
    try:
        from . import _context_host
        if _context_host.torch_version == torch.__version__.split("+")[0]:
            _gather = _context_host.gather
    except ImportError:
        pass
    return _gather


def _look(spec, names, *tensors):
    """(GPU index, the tensors' addresses, then the sizes of each) of tensors that are contiguous, on one GPU, and of the
    types and dimensions that `spec` gives, two characters each; raises otherwise."""
    got = (_gather or _built())(spec, *tensors)
    if got is not None:
        return got
    index = _index(names.split()[0], tensors[0])
    spec, sizes = spec.decode(), []
    for at, (name, t) in enumerate(zip(names.split(), tensors)):
        _check(index, _TYPES[spec[2 * at]], True, **{name: t})
        if t.dim() != int(spec[2 * at + 1]):
            raise ValueError(f"{name} must have {spec[2 * at + 1]} dimension(s), not {t.dim()}")
        sizes += t.shape
    return (index, *(t.data_ptr() for t in tensors), *sizes)


def _paged(q, k_cache, v_cache):
    """(spec, format, caches) of CSR-paged caches; other FP8 caches of 528-byte rows as [P, 528]."""
    spec, fmt, dim = _CACHES.get(getattr(k_cache, "dtype", None), (None, None, None))
    if spec is None or k_cache.dim() != dim:
        _check(_index("q", q), None, True, k_cache=k_cache, v_cache=v_cache)
        fmt, _ = _cache_format(k_cache, v_cache)
        return _CACHES[torch.uint8][:2] + (k_cache.view(-1, _FP8_PAGE[0]), v_cache.view(-1, _FP8_PAGE[0]))
    return spec, fmt, k_cache, v_cache


def _pages(fmt, pages, sizes, k_cache, v_cache):
    """Checks the sizes of both caches, the first one's pages apart."""
    page = _BF16_PAGE if fmt == CACHE_BF16 else _FP8_PAGE
    if sizes[:2 * len(page) + 1] != [*page, pages, *page]:
        _cache_format(k_cache, v_cache)
        raise ValueError("k_cache and v_cache must have the same shape")


def _heads(heads, dim):
    if heads != NUM_QO_HEADS or dim != HEAD_DIM:
        raise ValueError("expected q [N, 32, 128]")


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
    group to their own alone. Returns (out [B, 32, 128] bf16, lse [B, 32] fp32, base 2).

    Faster than ``run`` on the joined lists from about 8 sequences a prefix on (4 behind 4000 tokens and more), with FP8
    caches from 16 (6 behind 16384 and more); a single sequence takes 3 to 10 us longer than there (FP8 caches 5 to 26)."""
    caches, fmt, k_cache, v_cache = _paged(q, k_cache, v_cache)
    index, q_at, k_at, v_at, p_indptr, p_indices, g_indptr, indptr, indices, n, heads, dim, pages, *sizes = _look(
        b"b3" + caches + b"i1i1i1i1i1",
        "q k_cache v_cache prefix_indptr prefix_indices group_indptr kv_indptr kv_indices", q, k_cache, v_cache,
        prefix_indptr, prefix_indices, group_indptr, kv_indptr, kv_indices)
    _heads(heads, dim)
    _pages(fmt, pages, sizes, k_cache, v_cache)
    prefixes, prefix_count, groups, sequences, count = sizes[-5:]
    _fit(n, groups, prefix_count, count, pages)
    groups -= 1
    if groups < 0 or prefixes != groups + 1 or sequences != n + 1:
        raise ValueError(f"expected prefix_indptr and group_indptr [G + 1] and kv_indptr [{n + 1}]")
    out, lse = _results(index, n, out, lse, True, stream)
    if n == 0:
        return out, lse
    ws, size = _workspace(index, workspace, stream, "gqa_shared_paged_decode_ws_size", n, groups, fmt)
    _call("gqa_shared_paged_decode", index, stream, q_at, k_at, v_at, p_indptr, p_indices, g_indptr, indptr, indices,
          _SCALE if sm_scale is None else sm_scale, out.data_ptr(), lse.data_ptr(), n, groups, prefix_count, count, pages,
          fmt, ws.data_ptr(), size)
    return out, lse


def _blocked(name, heads, dim):
    if heads != NUM_KV_HEADS or dim != HEAD_DIM:
        raise ValueError(f"expected {name} [blocks, page_size, 4, 128]")


def _bounded(two, heads, dim):
    if two != 2 or heads != NUM_KV_HEADS or dim != HEAD_DIM:
        raise ValueError("expected bounds [blocks, 2, 4, 128]")


def block_bounds(k_cache: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 first: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The largest (bounds[:, 0]) and smallest (bounds[:, 1]) key values of the blocks that hold the new tokens
    first[r] <= t < lens[r] (first None: from 0) of each request of block_table [requests, width], over all of the
    block's tokens below lens[r]; k_cache [blocks, page_size, 4, 128], bounds [blocks, 2, 4, 128], in place. To be
    called after the tokens' rows are stored. Returns bounds."""
    if first is None:
        first_at = None
        index, k_at, bounds_at, table, lens_at, blocks, page, heads, dim, held, two, b_heads, b_dim, requests, width, n = _look(
            b"b4b4i2i1", "k_cache bounds block_table lens", k_cache, bounds, block_table, lens)
    else:
        (index, k_at, bounds_at, table, lens_at, first_at, blocks, page, heads, dim, held, two, b_heads, b_dim, requests,
         width, n, firsts) = _look(b"b4b4i2i1i1", "k_cache bounds block_table lens first", k_cache, bounds, block_table,
                                   lens, first)
        if firsts != requests:
            raise ValueError("expected first [requests]")
    _blocked("k_cache", heads, dim)
    _bounded(two, b_heads, b_dim)
    _fit(requests, width, blocks, page)
    if held != blocks or n != requests:
        raise ValueError("expected bounds [blocks, 2, 4, 128], and lens and first [requests]")
    _call("gqa_block_bounds", index, stream, k_at, bounds_at, table, lens_at, first_at, requests, page, blocks, width)
    return bounds


def block_select(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, token_to_req: torch.Tensor,
                 lens: torch.Tensor, top: int, page_size: int, keep_first: int = 1, keep_last: int = 1,
                 blocks: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The `top` blocks of each query row and KV head: of the blocks that hold tokens below lens[row] of request
    token_to_req[row], the first keep_first and last keep_last, then those whose bounds allow the largest product with
    one of the head's 8 queries (ties to the lower block). q [rows, 32, 128]. Returns their numbers in the table,
    ascending, then -1: int32 [rows, 4, top]."""
    (index, q_at, bounds_at, table, req, lens_at, rows, heads, dim, held, two, b_heads, b_dim, requests, width, reqs,
     lengths) = _look(b"b3b4i2i1i1", "q bounds block_table token_to_req lens", q, bounds, block_table, token_to_req, lens)
    _heads(heads, dim)
    _bounded(two, b_heads, b_dim)
    _fit(rows, requests, width, held)
    if reqs != rows or lengths != rows:
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
    _call("gqa_block_select", index, stream, q_at, bounds_at, table, req, lens_at, blocks.data_ptr(), rows, requests,
          page_size, held, width, top, keep_first, keep_last, ws.data_ptr(), size)
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
    (index, q_at, k_at, v_at, listed_at, table, req, lens_at, rows, heads, dim, held, page, k_heads, k_dim, v_held, v_page,
     v_heads, v_dim, listed, per_row, top, requests, width, reqs, lengths) = _look(
        b"b3b4b4i3i2i1i1", "q k_cache v_cache blocks block_table token_to_req lens", q, k_cache, v_cache, blocks, block_table,
        token_to_req, lens)
    _heads(heads, dim)
    _blocked("k_cache", k_heads, k_dim)
    if v_held != held or v_page != page or v_heads != k_heads or v_dim != k_dim:
        raise ValueError("k_cache and v_cache must have the same shape")
    _fit(rows, requests, width, held, page, top)
    if listed != rows or per_row != NUM_KV_HEADS:
        raise ValueError(f"blocks must be [{rows}, 4, top]")
    if reqs != rows or lengths != rows:
        raise ValueError(f"token_to_req and lens must be [{rows}]")
    out, lse = _results(index, rows, out, lse, with_lse, stream)
    if rows == 0:
        return out, lse
    ws, size = _workspace(index, workspace, stream, "gqa_block_sparse_decode_ws_size", rows, top, page)
    _call("gqa_block_sparse_decode", index, stream, q_at, k_at, v_at, listed_at, table, req, lens_at,
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
    caches, fmt, k_cache, v_cache = _paged(q, k_cache, v_cache)
    index, q_at, k_at, v_at, indptr, indices, weights_at, n, heads, dim, pages, *sizes = _look(
        b"b3" + caches + b"i1i1f2", "q k_cache v_cache kv_indptr kv_indices weights", q, k_cache, v_cache, kv_indptr,
        kv_indices, weights)
    _heads(heads, dim)
    _pages(fmt, pages, sizes, k_cache, v_cache)
    sequences, count, rows, width = sizes[-4:]
    _fit(n, width, count, pages)
    if rows != n or sequences != n + 1:
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
    ws, size = _workspace(index, workspace, stream, "gqa_paged_decode_weighted_ws_size", count, fmt)
    _call("gqa_paged_decode_weighted", index, stream, q_at, k_at, v_at, indptr, indices,
          _SCALE if sm_scale is None else sm_scale, weights_at, decay, weights_out.data_ptr(), out.data_ptr(),
          lse.data_ptr(), n, width, count, pages, fmt, ws.data_ptr(), size)
    return out, lse, weights_out


def kv_evict(weights: torch.Tensor, kv_indptr: torch.Tensor, kv_indices: torch.Tensor, budget: int, keep_first: int = 0,
             keep_last: int = 0, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """Cuts sequences of more than `budget` tokens back to it: the first keep_first and last keep_last tokens stay and,
    of those between, the ones of the largest weights[b, j] (ties: the lower j), in order. Returns (weights [B, width]
    at the tokens' new places, then zeros; kv_indptr [B + 1]; kv_indices; freed_indptr [B + 1]; freed): the tokens kept
    as a page table, and the other tokens' pages in the same form. kv_indices and freed are as long as the given
    kv_indices, -1 behind the last sequence's."""
    index, weights_at, indptr_at, indices_at, n, width, sequences, total = _look(
        b"f2i1i1", "weights kv_indptr kv_indices", weights, kv_indptr, kv_indices)
    _fit(n, width, total)
    if sequences != n + 1:
        raise ValueError("expected weights [B, width] and kv_indptr [B + 1]")
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
    _call("gqa_kv_evict", index, stream, weights_at, indptr_at, indices_at, budget, keep_first, keep_last, got.data_ptr(),
          indptr.data_ptr(), indices.data_ptr(), freed_indptr.data_ptr(), freed.data_ptr(), n, width, total)
    return got, indptr, indices, freed_indptr, freed
