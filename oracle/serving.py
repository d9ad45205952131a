"""Float64 CPU oracles of the operators around the paged decode.

TEST INFRASTRUCTURE. Only the test suite may import or run this module. The
CUDA library never calls it, and it imports nothing from the CUDA package.

Each function states the operator's definition in float64 without any rounding
of its result; the tests compare with tolerances derived from the roundings
the library makes.
"""
from __future__ import annotations

import math
from typing import Tuple

import numpy as np
import torch

from .fp8 import ROW_BYTES, e4m3_decode
from .oracle import HEAD_DIM, NUM_KV_HEADS

LATENT, ROPE, NOPE, HEAD_V = 512, 64, 128, 128


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, dtype=np.float64)


def inv_freq_oracle(rot_dim, base=10000.0, scaling=None, factor=1.0, original=4096.0, slow=1.0, fast=32.0):
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        keep = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return f * keep + f / factor * (1 - keep)
    return f


def rope_oracle(x, positions, inv_freq, scale=1.0, rot_offset=0, layout="half", inverse=False) -> np.ndarray:
    """x [N, heads, dim] with the window's pairs turned."""
    y = f64(x).copy()
    a = f64(positions)[:, None] * f64(inv_freq)[None]
    c, s = np.cos(a)[:, None] * scale, np.sin(a)[:, None] * (-scale if inverse else scale)
    r = a.shape[1]
    first = rot_offset + (np.arange(r) if layout == "half" else 2 * np.arange(r))
    second = first + (r if layout == "half" else 1)
    x1, x2 = f64(x)[..., first], f64(x)[..., second]
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def rope_pair_size(x, rot_dim, rot_offset, layout) -> np.ndarray:
    """|x1| + |x2| of every element's pair, 0 outside the window (for error bounds)."""
    ax, out = np.abs(f64(x)), np.zeros(x.shape)
    r = rot_dim // 2
    first = rot_offset + (np.arange(r) if layout == "half" else 2 * np.arange(r))
    second = first + (r if layout == "half" else 1)
    out[..., first] = out[..., second] = ax[..., first] + ax[..., second]
    return out


def fp8_scale_oracle(x) -> np.ndarray:
    """Smallest power of two that keeps the finite values of x [..., 128] within 448; 1 where all are 0."""
    ax = np.abs(f64(x))
    top = np.where(np.isfinite(ax), ax, 0.0).max(-1)
    m, e = np.frexp(top)
    s = np.where(m > 0.875, np.ldexp(1.0, e - 8), np.ldexp(1.0, e - 9))
    return np.where(top > 0, np.maximum(s, 2.0 ** -126), 1.0)


_CODES = e4m3_decode(np.arange(127))  # the finite codes without sign, ascending


def e4m3_encode(x) -> np.ndarray:
    """Nearest e4m3 code, ties to the even code; beyond 448 saturates, NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    ax = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    hi = np.clip(np.searchsorted(_CODES, ax), 1, 126)
    lo = hi - 1
    dl, dh = ax - _CODES[lo], _CODES[hi] - ax
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def fp8_rows_oracle(x) -> np.ndarray:
    """uint8 rows [N, 528] of x [N, 4, 128]."""
    s = fp8_scale_oracle(x)
    codes = e4m3_encode(f64(x) / s[..., None]).reshape(-1, NUM_KV_HEADS * HEAD_DIM)
    rows = np.empty((codes.shape[0], ROW_BYTES), dtype=np.uint8)
    rows[:, :NUM_KV_HEADS * HEAD_DIM] = codes
    rows[:, NUM_KV_HEADS * HEAD_DIM:] = s.astype("<f4").reshape(-1, NUM_KV_HEADS).view(np.uint8)
    return rows


def mla_absorb_q_oracle(q, w_kv) -> np.ndarray:
    """[N, h, 512]: q[..., :128] w_kv[h, :128]."""
    return np.einsum("nhd,hdl->nhl", f64(q)[..., :NOPE], f64(w_kv)[:, :NOPE])


def mla_expand_out_oracle(o, w_kv) -> np.ndarray:
    return np.einsum("nhl,hdl->nhd", f64(o), f64(w_kv)[:, NOPE:])


def mla_prefill_oracle(q, w_kv, kv_cache, block_table, cache_seqlens, cu_q, scale, causal=True) -> Tuple[
        np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """(out [T, h, 128], lse [h, T], out_bound [T, h, 128], lse_bound [h, T]).

    The bounds follow the roundings of an fp16 expansion and fp16 probabilities, with fp32 accumulation whose
    steps are off by at most u = 2^-23 (the sum may be cut instead of rounded):
      an expanded key or value: half a step of fp16 (2^-11 of it, 2^-25 at least) plus 512 u sum |c w|;
      a score: ds = scale * (sum |q| dk + 192 u sum |q k|);
      a weight p / sum p: a factor within exp(+-2 max ds), and half a step, 2^-11, on p;
      an output: sum p |v| times those, sum p dv, accumulation n u, then half a step of bf16 (2^-8);
      lse: max ds, plus 2^-20 of its terms for the exponentials and logarithm.
    """
    qf, w = f64(q), f64(w_kv)
    t_all, h = qf.shape[0], w.shape[0]
    blocks, page = int(kv_cache.shape[0]), int(kv_cache.shape[1])
    flat = f64(kv_cache).reshape(-1, LATENT + ROPE)
    out, lse = np.full((t_all, h, HEAD_V), np.nan), np.full((h, t_all), np.nan)
    ob, lb = np.zeros_like(out), np.zeros_like(lse)
    u = 2.0 ** -23
    cu = [int(x) for x in cu_q]
    table = np.asarray(block_table.cpu(), dtype=np.int64)
    for b in range(len(cu) - 1):
        nq = cu[b + 1] - cu[b]
        if nq == 0:
            continue
        n = min(max(int(cache_seqlens[b]), 0), table.shape[1] * page)
        t = np.arange(n)
        blk = table[b, t // page]
        keep = (blk >= 0) & (blk < blocks)
        rows = flat[(blk * page + t % page)[keep]]
        t = t[keep]
        c = rows[:, :LATENT]
        for a in range(h):
            full, mag = c @ w[a].T, np.abs(c) @ np.abs(w[a]).T
            dfull = 2.0 ** -11 * np.abs(full) + 2.0 ** -25 + 512 * u * mag
            k = np.concatenate([full[:, :NOPE], rows[:, LATENT:]], 1)
            dk = np.concatenate([dfull[:, :NOPE], np.zeros((len(t), ROPE))], 1)
            x = qf[cu[b]:cu[b + 1], a]
            s = scale * (x @ k.T)
            ds = abs(scale) * (np.abs(x) @ dk.T + 192 * u * (np.abs(x) @ np.abs(k).T))
            if causal:
                hide = t[None, :] > (n - nq + np.arange(nq))[:, None]
                s[hide] = -np.inf
                ds[hide] = 0.0
            if len(t) == 0:
                out[cu[b]:cu[b + 1], a], lse[a, cu[b]:cu[b + 1]] = 0.0, -np.inf
                continue
            m = s.max(1, keepdims=True)
            empty = np.isneginf(m[:, 0])
            p = np.exp(s - np.where(np.isneginf(m), 0.0, m))
            total = p.sum(1, keepdims=True)
            pn = p / np.where(total == 0, 1.0, total)
            v, dv = full[:, NOPE:], dfull[:, NOPE:]
            o = pn @ v
            d = ds.max(1)
            bound = (np.expm1(2 * d) + 2.0 ** -10 + 2.0 ** -20 + n * u)[:, None] * (pn @ np.abs(v)) + pn @ dv
            out[cu[b]:cu[b + 1], a] = o
            ob[cu[b]:cu[b + 1], a] = 2.0 ** -8 * (np.abs(o) + bound) + bound
            with np.errstate(divide="ignore"):
                lse[a, cu[b]:cu[b + 1]] = np.where(empty, -np.inf, (m + np.log(total))[:, 0])
            lb[a, cu[b]:cu[b + 1]] = d + 2.0 ** -20 * (1 + np.where(empty, 0.0, np.abs(m[:, 0]) + np.log(n)))
    return out, lse, ob, lb
