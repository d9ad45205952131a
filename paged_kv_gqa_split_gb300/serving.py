"""Tensor-level calls of the operators around the paged decode (include/gqa_paged_decode.h).

Rotary positions (``rope_inv_freq``, ``rope``), the cache's write and read
(``rope_kv_append``, ``kv_append_fp8``, ``kv_read_fp8``, ``mla_kv_append``) and
latent attention's projections and prompt pass (``mla_absorb_q``,
``mla_expand_out``, ``mla_absorbed_run``, ``mla_prefill``). As in ``_lib``:
argument checks and marshalling only, no CPU path; a call runs on the current
stream of its tensors' device unless ``stream`` is given. What the call
allocates then belongs to that stream, as under ``torch.cuda.stream``: a result
that another stream reads needs its ``record_stream``, beside the wait. (``run``,
``run_fp8``, ``sparse_run`` and ``mla_run`` allocate from the current stream.)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from ._lib import (FP8_ROW_BYTES, GQA_OK, GqaError, HEAD_DIM, MLA_D_QK, MLA_D_V, NUM_KV_HEADS, NUM_QO_HEADS, load,
                   mla_run, mla_workspace_size)

try:  # the allocation that compiled PyTorch programs call: no dispatch (3 us of a 14 us call on the GPU's host)
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "by_parts": 3}
CACHE_BF16, CACHE_FP8 = 0, 1
FILL_OUT, FILL_LSE = 1, 2
MLA_NOPE, MLA_ROPE, MLA_HEAD_V = 128, 64, 128
MLA_D_HEAD = MLA_NOPE + MLA_ROPE  # query and expanded key values a head
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _on(index, t, dtype):
    """Whether t is a tensor of `dtype` on GPU `index`."""
    return isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype


def _ready(index, t, dtype):
    """Whether t is a contiguous tensor of `dtype` on GPU `index`: the common case, in few steps."""
    return isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.is_contiguous()


_OPTIONAL = {"q", "q_out", "out", "lse", "k_out", "v_out"}  # arguments that may be None where _check sees them
_INT_MAX = 2 ** 31 - 1


def _check(index, dtype, contiguous, **tensors):
    """Raises for the first tensor (None only where it is optional) that is not on GPU `index` (a CPU tensor's is -1),
    of `dtype` (None: any) and, if asked, contiguous."""
    for name, t in tensors.items():
        if t is None and name in _OPTIONAL:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} is on {t.device}: the CUDA library has no CPU path; move inputs to the GPU")
        if t.get_device() != index:
            raise ValueError(f"all tensors must be on cuda:{index}; {name} is on {t.device}")
        if dtype is not None and t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _index(name, t):
    """The GPU of t, the tensor that sets the call's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        _check(index, None, False, **{name: t})
    return index


def _new(index, shape, dtype, stream):
    """An uninitialised contiguous tensor on GPU `index`, in the memory of the stream that the call runs on."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    if _empty_strided_cuda is None or index != torch._C._cuda_getDevice():
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    stride, step = [], 1
    for size in reversed(shape):
        stride.insert(0, step)
        step *= max(size, 1)
    return _empty_strided_cuda(shape, tuple(stride), dtype)


def _layout(layout):
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    return code


def _rotation(index, n, positions, inv_freq, pairs=None, rot_offset=0):
    """(positions pointer, inv_freq pointer, pairs); inv_freq None: no rotation."""
    if inv_freq is None:
        return None, None, 0
    if not 0 <= rot_offset <= _INT_MAX:  # a C int would drop the upper bits
        raise ValueError("rot_offset must not be negative or past the head")
    if positions is None:
        raise ValueError("a rotation needs positions")
    if not _ready(index, positions, torch.int32) or not _ready(index, inv_freq, torch.float64):
        _check(index, torch.int32, True, positions=positions)
        _check(index, torch.float64, True, inv_freq=inv_freq)
    if positions.dim() != 1 or positions.shape[0] != n:
        raise ValueError(f"positions must be [{n}]")
    have = inv_freq.shape[0] if inv_freq.dim() == 1 else 0
    if have < 1 or (pairs is not None and have != pairs):
        raise ValueError(f"inv_freq must be [{'pairs' if pairs is None else pairs}]")
    return positions.data_ptr(), inv_freq.data_ptr(), have


_entries = {}  # C entry points already looked up


def _call(name, index, stream, *args):
    """Calls the C entry on `stream` (default: GPU `index`'s current stream) and raises on an error code."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(load(), name)
    # the current stream's handle, without building a Stream
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != GQA_OK:
        raise GqaError(rc, name)


def _token_stride(name, t, heads, dim):
    """Token stride of t [n, heads, dim] whose heads lie one after another."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or stride[2] != 1 or stride[1] != dim:
        raise ValueError(f"{name} must be [N, {heads}, {dim}] with contiguous heads")
    return stride[0] if shape[0] > 1 else heads * dim


# ------------------------------------------------------------------ rotary
def rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                  original_positions: float = 4096.0, slow_turns: float = 1.0, fast_turns: float = 32.0,
                  device="cuda") -> Tuple[torch.Tensor, float]:
    """(inv_freq float64 [rot_dim / 2] on `device`, scale): radians a position of each pair, and the factor
    that goes with them (0.1 ln(factor) + 1 for "by_parts", else 1). scaling: None, "linear", "base" or "by_parts".
    "by_parts" ramps linearly in a pair's turns over original_positions; a model trained with a ramp over the pairs'
    index needs frequencies of its own (any float64 [pairs] tensor will do)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}")
    freq = torch.empty(max(int(rot_dim), 2) // 2, dtype=torch.float64)
    scale = ctypes.c_float(1.0)
    rc = load().gqa_rope_inv_freq(int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                  float(original_positions), float(slow_turns), float(fast_turns), freq.data_ptr(),
                                  ctypes.byref(scale))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_rope_inv_freq")
    return freq.to(device), scale.value


def rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, scale: float = 1.0, rot_offset: int = 0,
         layout: str = "half", inverse: bool = False, out: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rotary positions on x [N, heads, dim] (bf16, fp16 or fp32; any token and head strides): the window of
    2 * len(inv_freq) values from rot_offset is turned, the rest copied. out: a tensor like x, possibly x itself
    (default: a new contiguous one). inverse turns back, and is the gradient."""
    index = _index("x", x)
    code = _TYPES.get(x.dtype)
    if code is None or x.dim() != 3:
        raise ValueError("x must be [N, heads, dim] in bfloat16, float16 or float32")
    n, heads, dim = x.shape
    if inv_freq is None:
        raise ValueError("rope needs inv_freq")
    pos, freq, pairs = _rotation(index, n, positions, inv_freq, rot_offset=rot_offset)
    if out is None:
        out = _new(index, (n, heads, dim), x.dtype, stream)
    else:
        _check(index, x.dtype, False, out=out)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    (xt, xh, xe), (ot, oh, oe) = x.stride(), out.stride()
    if (xe != 1 or oe != 1) and dim > 1:
        raise ValueError("a head's values must be contiguous")
    _call("gqa_rope", index, stream, x.data_ptr(), pos, freq, scale, out.data_ptr(), n, heads, dim, rot_offset,
          2 * pairs, _layout(layout), 1 if inverse else 0, code, xt, xh, ot, oh)
    return out


# -------------------------------------------------------------- cache write
def _cache_format(k_cache, v_cache):
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same shape and type")
    if k_cache.dtype == torch.uint8:
        if k_cache.dim() < 2 or k_cache.shape[-1] != FP8_ROW_BYTES:
            raise ValueError(f"FP8 caches must be uint8 rows of {FP8_ROW_BYTES} bytes ([P, {FP8_ROW_BYTES}])")
        return CACHE_FP8, k_cache.numel() // FP8_ROW_BYTES
    if k_cache.dtype != torch.bfloat16 or k_cache.dim() != 4 or \
            tuple(k_cache.shape[1:]) != (1, NUM_KV_HEADS, HEAD_DIM):
        raise ValueError("expected k_cache / v_cache [P, 1, 4, 128] bfloat16 or [P, 528] uint8")
    return CACHE_BF16, k_cache.shape[0]


def rope_kv_append(q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, positions: Optional[torch.Tensor] = None,
                   inv_freq: Optional[torch.Tensor] = None, scale: float = 1.0, rot_offset: int = 0,
                   layout: str = "half", q_out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """One pass over a step's new tokens: q [N, 32, 128] and k_new [N, 4, 128] turned by their positions (inv_freq
    None: not turned), k_new and v_new stored in pages slots[r] of bf16 caches [P, 1, 4, 128] or FP8 caches [P, 528]
    (quantised). q, k_new and v_new may be views of one fused row. Returns the turned q (None without q)."""
    index, bf = _index("k_cache", k_cache), torch.bfloat16
    if not (_on(index, k_new, bf) and _on(index, v_new, bf) and (q is None or _on(index, q, bf)) and
            (q_out is None or _ready(index, q_out, bf)) and k_cache.is_contiguous() and
            _ready(index, v_cache, k_cache.dtype) and _ready(index, slots, torch.int32)):
        _check(index, bf, False, q=q, k_new=k_new, v_new=v_new, q_out=q_out)
        _check(index, None, True, k_cache=k_cache, v_cache=v_cache, q_out=q_out)
        _check(index, torch.int32, True, slots=slots)
    fmt, pages = _cache_format(k_cache, v_cache)
    if slots.dim() != 1:
        raise ValueError("slots must be [N]")
    n = slots.shape[0]
    ks, vs = _token_stride("k_new", k_new, NUM_KV_HEADS, HEAD_DIM), _token_stride("v_new", v_new, NUM_KV_HEADS, HEAD_DIM)
    qs, q_ptr, out_ptr = 0, None, None
    if q is not None:
        qs = _token_stride("q", q, NUM_QO_HEADS, HEAD_DIM)
        if q_out is None:
            q_out = _new(index, (n, NUM_QO_HEADS, HEAD_DIM), torch.bfloat16, stream)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if k_new.shape[0] != n or v_new.shape[0] != n or (q is not None and (q.shape[0] != n or q_out.shape != q.shape)):
        raise ValueError("q, k_new, v_new and q_out must have one row per slot")
    pos, freq, pairs = _rotation(index, n, positions, inv_freq, rot_offset=rot_offset)
    _call("gqa_rope_kv_append", index, stream, q_ptr, k_new.data_ptr(), v_new.data_ptr(), pos, slots.data_ptr(),
          freq, scale, rot_offset, 2 * pairs, _layout(layout), out_ptr, k_cache.data_ptr(), v_cache.data_ptr(), fmt, n,
          pages, qs, ks, vs)
    return q_out


def kv_append_fp8(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise each new token's K/V rows [N, 4, 128] into page slots[r] of FP8 caches [P, 528] (in place); slots
    outside [0, P) are skipped."""
    _check(_index("k_cache", k_cache), None, False, v_cache=v_cache)
    if _cache_format(k_cache, v_cache)[0] != CACHE_FP8:
        raise ValueError("kv_append_fp8 needs FP8 caches; kv_append stores bfloat16 ones")
    rope_kv_append(None, k_new, v_new, slots, k_cache, v_cache, stream=stream)


def kv_read_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, indices: torch.Tensor,
                k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of pages indices[r] of FP8 caches [P, 528] as bfloat16 ([N, 4, 128] each); zeros for a page outside
    [0, P)."""
    index = _index("k_cache", k_cache)
    if not (_ready(index, k_cache, torch.uint8) and _ready(index, v_cache, torch.uint8) and
            _ready(index, indices, torch.int32)):
        _check(index, torch.uint8, True, k_cache=k_cache, v_cache=v_cache)
        _check(index, torch.int32, True, indices=indices)
    pages = _cache_format(k_cache, v_cache)[1]
    if indices.dim() != 1:
        raise ValueError("indices must be [N]")
    n = indices.shape[0]
    shape = (n, NUM_KV_HEADS, HEAD_DIM)
    _check(index, torch.bfloat16, True, k_out=k_out, v_out=v_out)
    if k_out is None:
        k_out = _new(index, shape, torch.bfloat16, stream)
    if v_out is None:
        v_out = _new(index, shape, torch.bfloat16, stream)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out and v_out must be {shape}")
    _call("gqa_paged_kv_read_fp8", index, stream, k_cache.data_ptr(), v_cache.data_ptr(), indices.data_ptr(),
          k_out.data_ptr(), v_out.data_ptr(), n, pages)
    return k_out, v_out


def _latent_cache(kv_cache):
    if kv_cache.dim() != 4 or kv_cache.shape[2] != 1 or kv_cache.shape[3] != MLA_D_QK:
        raise ValueError("expected kv_cache [num_blocks, page_size, 1, 576] bf16 (one latent KV head)")
    return kv_cache.shape[0], kv_cache.shape[1]


def mla_kv_append(latent: torch.Tensor, k_rope: torch.Tensor, slots: torch.Tensor, kv_cache: torch.Tensor,
                  positions: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                  scale: float = 1.0, layout: str = "interleaved",
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Store latent [N, 512] and the (turned) rotary key k_rope [N, 64] in slots[r] = block * page_size + offset of
    kv_cache [num_blocks, page_size, 1, 576] (in place); other slots are skipped."""
    index = _index("kv_cache", kv_cache)
    _check(index, torch.bfloat16, True, kv_cache=kv_cache)
    _check(index, torch.bfloat16, False, latent=latent, k_rope=k_rope)
    _check(index, torch.int32, True, slots=slots)
    blocks, page = _latent_cache(kv_cache)
    n = slots.shape[0] if slots.dim() == 1 else -1
    for name, t, d in (("latent", latent, MLA_D_V), ("k_rope", k_rope, MLA_ROPE)):
        if t.dim() != 2 or t.shape != (n, d) or t.stride(1) != 1:
            raise ValueError(f"{name} must be [N, {d}] with contiguous rows, one per slot")
    pos, freq, _ = _rotation(index, n, positions, inv_freq, MLA_ROPE // 2)
    _call("gqa_mla_kv_append", index, stream, latent.data_ptr(), k_rope.data_ptr(), pos, slots.data_ptr(), freq, scale,
          _layout(layout), kv_cache.data_ptr(), n, blocks * page, latent.stride(0) if n > 1 else MLA_D_V,
          k_rope.stride(0) if n > 1 else MLA_ROPE)


# --------------------------------------------------------- latent attention
def _weights(w_kv, heads, index):
    if not _ready(index, w_kv, torch.bfloat16):
        _check(index, torch.bfloat16, True, w_kv=w_kv)
    if w_kv.shape != (heads, MLA_NOPE + MLA_HEAD_V, MLA_D_V):
        raise ValueError(f"w_kv must be [{heads}, {MLA_NOPE + MLA_HEAD_V}, {MLA_D_V}]")
    return w_kv.data_ptr()


def _query(q):
    """(N, heads, token stride, head stride) of q [N, heads, 192]."""
    if q.dtype is not torch.bfloat16 or q.dim() != 3 or q.shape[2] != MLA_D_HEAD or q.stride(2) != 1:
        raise ValueError(f"q must be bfloat16 [N, heads, {MLA_D_HEAD}] with contiguous heads")
    n, h, d = q.shape
    ts, hs, _ = q.stride()
    return n, h, ts if n > 1 else h * d, hs if h > 1 else d


def mla_absorb_q(q: torch.Tensor, w_kv: torch.Tensor, positions: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None, scale: float = 1.0, layout: str = "interleaved",
                 out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """q [N, heads, 192] to the latent decode's queries [N, heads, 576]: q[..., :128] w_kv[h, :128], then the 64 rotary
    values (turned by positions if inv_freq [32] is given). w_kv: [heads, 256, 512]."""
    index = _index("q", q)
    n, h, ts, hs = _query(q)
    w = _weights(w_kv, h, index)
    pos, freq, _ = _rotation(index, n, positions, inv_freq, MLA_ROPE // 2)
    if out is None:
        out = _new(index, (n, h, MLA_D_QK), torch.bfloat16, stream)
    else:
        _check(index, torch.bfloat16, True, out=out)
        if out.shape != (n, h, MLA_D_QK):
            raise ValueError(f"out must be {(n, h, MLA_D_QK)}")
    _call("gqa_mla_absorb_q", index, stream, q.data_ptr(), w, pos, freq, scale, _layout(layout), out.data_ptr(), n, h,
          ts, hs)
    return out


def mla_expand_out(o_latent: torch.Tensor, w_kv: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The latent decode's output [N, heads, 512] to the heads' values [N, heads, 128]: w_kv[h, 128:] o_latent."""
    index = _index("o_latent", o_latent)
    if not _ready(index, o_latent, torch.bfloat16):
        _check(index, torch.bfloat16, True, o_latent=o_latent)
    if o_latent.dim() != 3 or o_latent.shape[2] != MLA_D_V:
        raise ValueError(f"o_latent must be [N, heads, {MLA_D_V}]")
    n, h, _ = o_latent.shape
    w = _weights(w_kv, h, index)
    if out is None:
        out = _new(index, (n, h, MLA_HEAD_V), torch.bfloat16, stream)
    else:
        _check(index, torch.bfloat16, True, out=out)
        if out.shape != (n, h, MLA_HEAD_V):
            raise ValueError(f"out must be {(n, h, MLA_HEAD_V)}")
    _call("gqa_mla_expand_out", index, stream, o_latent.data_ptr(), w, out.data_ptr(), n, h)
    return out


def mla_absorbed_run(q: torch.Tensor, w_kv: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                     cache_seqlens: torch.Tensor, positions: Optional[torch.Tensor] = None,
                     inv_freq: Optional[torch.Tensor] = None, scale: float = 1.0, layout: str = "interleaved",
                     softmax_scale: Optional[float] = None, with_lse: bool = True,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Latent attention for new tokens, absorbed form: ``mla_absorb_q``, ``mla_run`` and ``mla_expand_out`` in turn.
    q: [B, s_q, heads, 192] (s_q * heads a multiple of 16; not causal within the s_q tokens); positions: [B * s_q].
    Each call allocates its workspace, so calls in several streams and captured ones do not share one.
    Returns (out [B, s_q, heads, 128] bf16, lse [B, heads, s_q] fp32 natural log, or None)."""
    if stream is not None:  # the intermediate tensors then belong to that stream
        with torch.cuda.stream(stream):
            return mla_absorbed_run(q, w_kv, kv_cache, block_table, cache_seqlens, positions, inv_freq, scale, layout,
                                    softmax_scale, with_lse)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError(f"expected q [B, s_q, heads, {MLA_D_HEAD}]")
    b, s, h, d = q.shape
    flat = mla_absorb_q(q.reshape(b * s, h, d), w_kv, positions, inv_freq, scale, layout)
    flat, index = flat.view(b, s, h, MLA_D_QK), flat.get_device()
    if not (_ready(index, kv_cache, torch.bfloat16) and _ready(index, block_table, torch.int32)):
        _check(index, torch.bfloat16, True, kv_cache=kv_cache)
        _check(index, torch.int32, True, block_table=block_table)
    blocks, page = _latent_cache(kv_cache)
    if block_table.dim() != 2:
        raise ValueError("expected block_table [B, width]")
    # a workspace of the call's own: other streams' calls and captured graphs do not share it
    if index == torch._C._cuda_getDevice():  # without the switch of devices, 5 us
        size = load().gqa_mla_decode_ws_size(b, s, h, page, blocks, block_table.shape[1])
    else:
        size = mla_workspace_size(flat, kv_cache, block_table)
    if size == 0 and b > 0:
        raise ValueError("the batch, the heads or the block table are out of range")
    workspace = _new(index, (size,), torch.uint8, None)
    o, lse = mla_run(flat, kv_cache, block_table, cache_seqlens,
                     MLA_D_HEAD ** -0.5 if softmax_scale is None else softmax_scale, with_lse=with_lse,
                     workspace=workspace)
    return mla_expand_out(o.view(b * s, h, MLA_D_V), w_kv).view(b, s, h, MLA_HEAD_V), lse


def mla_prefill(q: torch.Tensor, w_kv: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                cache_seqlens: torch.Tensor, cu_seqlens_q: torch.Tensor, softmax_scale: Optional[float] = None,
                causal: bool = True, max_kv_tokens: Optional[int] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, with_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Latent attention for prompts and prompt chunks, expanded form: packed queries q [total, heads, 192] (sequence
    b's rows from cu_seqlens_q[b] on, rotary part turned) over the cached tokens that block_table [B, width] and
    cache_seqlens [B] list, the new ones among them. max_kv_tokens: a bound on the sum of cache_seqlens, which sizes
    the workspace and how many heads a pass takes (default: what the block table can list; with a table far wider
    than the lengths that costs memory and up to several times the time). Sequences past a bound that is too small
    come back as 0 and -inf; bit 64 of ``_lib.gqa_paged_decode_device_error`` is all that tells. Rows of no sequence
    are 0 (lse -inf) in outputs that the call allocates, and left as they were in given ones. Returns (out
    [total, heads, 128] bf16, lse [heads, total] fp32 natural log, or None)."""
    index = _index("q", q)
    n, h, ts, hs = _query(q)
    w = _weights(w_kv, h, index)
    if not (_ready(index, kv_cache, torch.bfloat16) and _ready(index, block_table, torch.int32) and
            _ready(index, cache_seqlens, torch.int32) and _ready(index, cu_seqlens_q, torch.int32)):
        _check(index, torch.bfloat16, True, kv_cache=kv_cache)
        _check(index, torch.int32, True, block_table=block_table, cache_seqlens=cache_seqlens, cu_seqlens_q=cu_seqlens_q)
    _check(index, torch.bfloat16, True, out=out)
    blocks, page = _latent_cache(kv_cache)
    if block_table.dim() != 2 or cache_seqlens.shape != (block_table.shape[0],) or \
            cu_seqlens_q.shape != (block_table.shape[0] + 1,):
        raise ValueError("expected block_table [B, width], cache_seqlens [B] and cu_seqlens_q [B + 1]")
    b, width = block_table.shape
    if max_kv_tokens is None:
        max_kv_tokens = b * width * page
    if not 0 <= max_kv_tokens <= _INT_MAX:
        raise ValueError(f"max_kv_tokens {max_kv_tokens} is out of range")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(MLA_D_HEAD)
    fill = 0  # outputs of the call's own have no rows left as they were
    if out is None:
        fill |= FILL_OUT
        out = _new(index, (n, h, MLA_HEAD_V), torch.bfloat16, stream)
    elif out.shape != (n, h, MLA_HEAD_V):
        raise ValueError(f"out must be {(n, h, MLA_HEAD_V)}")
    if lse is not None:
        _check(index, torch.float32, True, lse=lse)
        if lse.shape != (h, n):
            raise ValueError(f"lse must be {(h, n)}")
    elif with_lse:
        fill |= FILL_LSE
        lse = _new(index, (h, n), torch.float32, stream)
    if b == 0 or n == 0:
        with torch.cuda.stream(stream):
            if fill & FILL_OUT:
                out.zero_()
            if fill & FILL_LSE:
                lse.fill_(-math.inf)
        return out, lse
    if workspace is None:
        size = load().gqa_mla_prefill_ws_size(b, h, max_kv_tokens)
        if size == 0:
            raise ValueError(f"batch {b}, heads {h} and max_kv_tokens {max_kv_tokens} are out of range")
        workspace = _new(index, (size,), torch.uint8, stream)
    else:
        _check(index, None, True, workspace=workspace)
    _call("gqa_mla_prefill_fill", index, stream, q.data_ptr(), w, kv_cache.data_ptr(), block_table.data_ptr(),
          cache_seqlens.data_ptr(), cu_seqlens_q.data_ptr(), softmax_scale, 1 if causal else 0, fill, out.data_ptr(),
          lse.data_ptr() if lse is not None else None, b, n, h, page, blocks, width, max_kv_tokens, ts, hs,
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse
