"""Float64 CPU oracles of the decode's forms for long and shared contexts.

TEST INFRASTRUCTURE. Only the test suite may import or run this module. The CUDA library never calls it, and it imports
nothing from the CUDA package.

Each function states the operator's definition in float64; ``attend`` also returns what error bounds are made of.
"""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import numpy as np
import torch

from .fp8 import dequantize_rows
from .oracle import GQA_GROUP, HEAD_DIM, NUM_KV_HEADS, NUM_QO_HEADS

# An MMA of 16 products and an accumulator cuts each off at 2^-23 of the largest: 17 * 2^-23 of the sum of sizes, 8 MMAs
# a score of 128 dims.
SCORE_ERROR = 8 * 17 * 2.0 ** -23


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, dtype=np.float64)


def ints(t) -> List[int]:
    return [int(x) for x in (t.detach().cpu().reshape(-1).tolist() if isinstance(t, torch.Tensor) else t)]


def rows64(cache, pages: List[int]) -> np.ndarray:
    """[t, 4, 128] values of the listed pages that lie in the pool, in order."""
    count = cache.shape[0]
    sel = [p for p in pages if 0 <= p < count]
    if cache.dtype == torch.uint8:
        return dequantize_rows(cache.cpu().numpy()[sel]).reshape(-1, NUM_KV_HEADS, HEAD_DIM)
    return f64(cache.view(count, NUM_KV_HEADS, HEAD_DIM)[torch.as_tensor(sel, dtype=torch.long, device=cache.device)])


class Attended:
    """One query row over rows k, v [t, 4, 128] (or lists of four [t_g, 128]): out [32, 128], lse [32] (base 2),
    p [32] lists, and sizes: abs_v = sum p |v| [32, 128], size [32] the largest sum of |q_d k_d| of a score, room [32, 128]
    the sum of the |v| of all tokens."""

    def __init__(self, q, k, v, sm_scale):
        q = f64(q)
        self.out, self.abs_v, self.room = (np.zeros((NUM_QO_HEADS, HEAD_DIM)) for _ in range(3))
        self.lse, self.size, self.p = np.full(NUM_QO_HEADS, -np.inf), np.zeros(NUM_QO_HEADS), []
        for h in range(NUM_QO_HEADS):
            g = h // GQA_GROUP
            kk, vv = (k[g], v[g]) if isinstance(k, list) else (k[:, g], v[:, g])
            if kk.shape[0] == 0:
                self.p.append(np.zeros(0))
                continue
            s = kk @ q[h] * sm_scale
            self.size[h] = (np.abs(kk) @ np.abs(q[h])).max() * abs(sm_scale)
            top = s.max()
            e = np.exp(s - top)
            self.lse[h] = (top + math.log(e.sum())) / math.log(2.0)
            p = e / e.sum()
            self.p.append(p)
            self.out[h], self.abs_v[h], self.room[h] = p @ vv, p @ np.abs(vv), np.abs(vv).sum(0)

    def out_bound(self, fp8: bool) -> np.ndarray:
        """Probabilities rounded to bf16 (2^-8) or, with an FP8 cache, fp16 (2^-11, and 2^-25 of the largest one's size
        times a V scale of up to twice the token's), scores off by SCORE_ERROR of their size, the result rounded to bf16."""
        step = 2.0 ** -11 if fp8 else 2.0 ** -8
        off = np.expm1(2 * SCORE_ERROR * self.size)[:, None]
        low = 2.0 ** -24 * self.room if fp8 else 0.0
        inner = self.abs_v * (step + off + 2.0 ** -16) + low
        return inner + (np.abs(self.out) + inner) * 2.0 ** -8 + 1e-30

    def lse_bound(self) -> np.ndarray:
        return SCORE_ERROR * self.size / math.log(2.0) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(self.lse), self.lse, 0)))


def shared_oracle(q, k_cache, v_cache, prefix_indptr, prefix_indices, group_indptr, kv_indptr, kv_indices,
                  sm_scale: float) -> List[Attended]:
    pi, px, gi, ki, kx = (ints(t) for t in (prefix_indptr, prefix_indices, group_indptr, kv_indptr, kv_indices))
    got = []
    for b in range(q.shape[0]):
        pages = list(kx[ki[b]:ki[b + 1]])
        for g in range(len(gi) - 1):
            if gi[g] <= b < gi[g + 1]:
                pages = px[pi[g]:pi[g + 1]] + pages
        got.append(Attended(q[b], rows64(k_cache, pages), rows64(v_cache, pages), sm_scale))
    return got


def bounds_oracle(k_cache, bounds, block_table, lens, first=None) -> np.ndarray:
    """The new bounds [blocks, 2, 4, 128]."""
    got, k = f64(bounds).copy(), f64(k_cache)
    table, page = block_table.cpu().numpy(), k_cache.shape[1]
    for r, n in enumerate(ints(lens)):
        n = max(0, min(n, table.shape[1] * page))
        at = 0 if first is None else max(0, ints(first)[r])
        for i in range(at // page, -(-n // page) if at < n else 0):
            block = int(table[r, i])
            if 0 <= block < k.shape[0]:
                x = k[block, :min(page, n - i * page)]
                got[block, 0], got[block, 1] = x.max(0), x.min(0)  # NaN spreads
    return got


def select_oracle(q, bounds, block_table, token_to_req, lens, top, page, keep_first, keep_last) -> np.ndarray:
    """blocks [rows, 4, top]."""
    q, b, table = f64(q), f64(bounds), block_table.cpu().numpy()
    got = np.full((q.shape[0], NUM_KV_HEADS, top), -1, dtype=np.int32)
    for r, (req, n) in enumerate(zip(ints(token_to_req), ints(lens))):
        if not 0 <= req < table.shape[0]:
            continue
        n = max(0, min(n, table.shape[1] * page))
        count = -(-n // page)
        cand = [i for i in range(count) if 0 <= table[req, i] < b.shape[0]]
        if not cand:
            continue
        x = b[table[req, cand]]  # [c, 2, 4, 128]
        for g in range(NUM_KV_HEADS):
            qg = q[r, g * GQA_GROUP:(g + 1) * GQA_GROUP]
            with np.errstate(invalid="ignore", over="ignore"):
                each = (np.maximum(qg, 0)[None] * x[:, 0, g][:, None] + np.minimum(qg, 0)[None] * x[:, 1, g][:, None])
                s = each.sum(-1).max(1)  # NaN if a head's is
                score = np.where(np.isfinite(s.astype(np.float32)), s, np.inf)
            order = sorted(range(len(cand)),
                           key=lambda c: (not (cand[c] < keep_first or cand[c] >= count - keep_last), -score[c], cand[c]))
            pick = sorted(cand[c] for c in order[:top])
            got[r, g, :len(pick)] = pick
    return got


def block_sparse_oracle(q, k_cache, v_cache, blocks, block_table, token_to_req, lens, sm_scale) -> List[Attended]:
    held, page = k_cache.shape[:2]
    table, picks = block_table.cpu().numpy(), blocks.cpu().numpy()
    k, v = f64(k_cache), f64(v_cache)
    got = []
    for r, (req, n) in enumerate(zip(ints(token_to_req), ints(lens))):
        ks, vs = [], []
        n = max(0, min(n, table.shape[1] * page))
        for g in range(NUM_KV_HEADS):
            kg, vg = [np.zeros((0, HEAD_DIM))], [np.zeros((0, HEAD_DIM))]
            for i in picks[r, g].tolist():
                if not (0 <= req < table.shape[0] and 0 <= i and i * page < n and 0 <= table[req, i] < held):
                    continue
                kg.append(k[table[req, i], :min(page, n - i * page), g])
                vg.append(v[table[req, i], :min(page, n - i * page), g])
            ks.append(np.concatenate(kg))
            vs.append(np.concatenate(vg))
        got.append(Attended(q[r], ks, vs, sm_scale))
    return got


def weighted_oracle(q, k_cache, v_cache, kv_indptr, kv_indices, weights, decay, sm_scale
                    ) -> Tuple[List[Attended], np.ndarray, np.ndarray]:
    """(attended, weights, their error bounds)."""
    ki, kx, old = ints(kv_indptr), ints(kv_indices), f64(weights)
    count, got, rows = k_cache.shape[0], [], []
    new, bound = old.copy(), np.zeros_like(old)
    for b in range(q.shape[0]):
        pages = kx[ki[b]:ki[b + 1]]
        a = Attended(q[b], rows64(k_cache, pages), rows64(v_cache, pages), sm_scale)
        rows.append(a)
        held = [j for j, page in enumerate(pages) if 0 <= page < count]
        add = np.zeros(len(pages))
        off = np.zeros(len(pages))
        for h in range(NUM_QO_HEADS):
            add[held] += a.p[h]
            off[held] += a.p[h] * np.expm1(2 * SCORE_ERROR * a.size[h] + 2.0 ** -19 * (1 + abs(a.lse[h]) if held else 1))
        n = min(len(pages), old.shape[1])
        base = decay * old[b, :n] if decay else np.zeros(n)
        new[b, :n] = base + add[:n]
        bound[b, :n] = off[:n] + 2.0 ** -22 * (np.abs(base) + add[:n]) + 2.0 ** -120
    return rows, new, bound


def evict_oracle(weights, kv_indptr, kv_indices, budget, keep_first=0, keep_last=0):
    """(weights, kv_indptr, kv_indices, freed_indptr, freed)."""
    ki, kx, w = ints(kv_indptr), ints(kv_indices), weights.detach().cpu().numpy()
    width = w.shape[1]
    new = np.zeros_like(w)
    stay, go, a, f = [], [], [0], [0]
    for b in range(w.shape[0]):
        pages = kx[ki[b]:ki[b + 1]]
        n = len(pages)
        x = np.zeros(n, dtype=np.float64)
        x[:min(n, width)] = w[b, :min(n, width)]
        rank = np.where(np.isnan(x), np.inf, x)
        order = sorted(range(n), key=lambda j: (not (j < keep_first or j >= n - keep_last), not np.isnan(x[j]), -rank[j], j))
        keep = sorted(order[:budget])
        gone = sorted(set(range(n)) - set(keep))
        m = min(len(keep), width)
        new[b, :m] = x[keep[:m]]
        stay += [pages[j] for j in keep]
        go += [pages[j] for j in gone]
        a.append(len(stay))
        f.append(len(go))
    total = len(kx)
    return (new, np.array(a), np.array(stay + [-1] * (total - len(stay))), np.array(f),
            np.array(go + [-1] * (total - len(go))))
