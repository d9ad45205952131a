// Latent attention's expanded form: the prompt pass. Queries of several
// sequences, packed one after another, attend to their sequence's paged latent
// rows through per-head keys and values expanded from them:
//   k[t][h] = [ W_k[h] c_t (128) ; rotary key of t (64) ],  v[t][h] = W_v[h] c_t (128)
//   out[i][h] = sum_t softmax_t(scale * q[i][h] . k[t][h]) v[t][h]
// over the t that the sequence holds and, if causal, t <= n - nq + i. Expanding
// costs 2 * 512 * 256 FLOP a token and head once, after which a pair costs
// 2 * (192 + 128) FLOP where the absorbed form costs 2 * (576 + 512): cheaper
// from about 170 queries a sequence on.
//
// Precision. Queries, keys, values and probabilities are fp16 operands (11
// bits against bf16's 8: with bf16 the output was 1.6 x further from the 64-bit
// result than one rounding of it, with fp16 1.01 x). fp16's range is kept by
// powers of two, which change nothing else: a query row is brought to a largest
// value in [2^10, 2^11); keys and values of a sequence have one exponent each, from the
// bound 512 * max|c| * max|W| (and the rotary keys). A sequence whose tokens' own maxima
// lie more than 2^8 apart is "wide": there each token has exponents of its own, so that a
// huge one costs no bits of the others (rows that do not see it, or give it no weight, are
// what they are without it), and the attention has a second, slower loop for it. The maxima
// are taken over finite values, so an infinity stays with its row: a token whose latent is
// not all finite gets NaN keys and zero values, which makes the rows that see it NaN
// and, a weight of 0 times 0 being 0, no others.
// Scores, softmax statistics and outputs accumulate in fp32.
//
// Steps, each a kernel that starts while the one before it ends: the plan (prefix
// sums over the sequences), the gather (paged rows to packed rows, 128-aligned per
// sequence and zero-filled, and the maxima), the expansion, the attention, and a join
// where that was split. Bound by
// the tensor cores: 8192 tokens x 16 heads 250 to 260 us in all (1460 to 1510 TFLOP/s, 78 to
// 81 % of the measured cuBLAS bf16 rate); five short prompts 35 us, the chain's latency.
#include <cuda_bf16.h>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_ptx.cuh"
#include "gqa_tc.cuh"

namespace gqa {
namespace {

constexpr int kLat = 512, kNope = 128, kRope = 64, kHeadV = 128, kRow = kLat + kRope;
constexpr int kAlign = 128;    // packed rows of a sequence start at a multiple of this
constexpr int kQTile = 512;   // query rows a pair of CTAs takes
constexpr int64_t kExpandBytes = int64_t{1} << 30;  // expanded keys and values of one pass over the heads
constexpr int64_t kGroupBytes = int64_t{96} << 20;  // and of the heads whose CTAs run together (they stay in L2)

// Splitting the attention's units over their keys (see there): at most this many units (query tiles x heads) and pairs
// of CTAs, from this many packed rows on; steps (key tiles' time) that a unit, and joining one, cost besides; the least
// piece.
constexpr int kSplitTiles = 152, kSplitPairs = 76, kSplitRows = 2048;
constexpr int kUnitSteps = 5, kJoinSteps = 16, kPieceSteps = 12;
constexpr int kPartFloats = 32 * (kHeadV + 4);  // a warp's piece: 32 rows of output, then their maxima, sums and output units
constexpr unsigned kWindow = 8;  // binades that the tokens of a sequence with one exponent may be apart

// ------------------------------------------------------------------- plan
// One block: lengths clamped to the table, packed starts, query tiles. Prefix
// sums run over chunks of 1024 sequences (a warp's by shuffles, then the warps'). What this and
// the later kernels write into the workspace is read with __ldcg throughout: the readers start
// before the writers end, and the non-coherent load is for words that no one writes meanwhile. Only
// malformed offsets, whose sequences share rows, have more query tiles than p.q_tiles;
// those past it are left out.
__global__ void __launch_bounds__(1024) gqa_mla_prefill_plan_kernel(const MlaPrefillParams p) {
  __shared__ int64_t sk[32];
  __shared__ int sq[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  if (tid < 2) p.amax[tid] = 0;
  int64_t base_k = 0, base_q = 0;
  const int64_t table = static_cast<int64_t>(p.width) * p.page_size;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + tid;
    int len = 0, tiles = 0;
    if (b < p.batch) {
      // a malformed cu_q never makes a row out of range: entries are clamped to
      // [0, total_q], and a decreasing pair counts as an empty sequence
      const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), n = __ldg(p.cache_seqlens + b);
      const int qs = min(max(c0, 0), p.total_q), qe = min(max(c1, 0), p.total_q);
      if (c1 < c0 || c0 < 0 || c1 > p.total_q) atomicOr(p.err, kErrBadIndptr);
      const int nq = max(qe - qs, 0);
      tiles = (nq + kQTile - 1) / kQTile;
      if (nq > 0) len = static_cast<int>(min(static_cast<int64_t>(max(n, 0)), table));
      p.q_start[2 * b] = qs;
      p.q_start[2 * b + 1] = nq;
      *reinterpret_cast<uint4*>(p.amax + 4 + 4 * b) = make_uint4(0, 0, 0, 0);
    }
    const int64_t rows = (static_cast<int64_t>(len) + kAlign - 1) / kAlign * kAlign;
    int64_t k = rows;
    int q = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t vk = __shfl_up_sync(0xffffffffu, k, o);
      const int vq = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) {
        k += vk;
        q += vq;
      }
    }
    if (lane == 31) {
      sk[warp] = k;
      sq[warp] = q;
    }
    __syncthreads();
    int64_t before_k = base_k;
    int64_t before_q = base_q;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) {
        before_k += sk[w];
        before_q += sq[w];
      }
      base_k += sk[w];
      base_q += sq[w];
    }
    if (b < p.batch) {
      const int64_t end = before_k + k;
      if (end > p.cap) {  // more tokens than the caller's bound: these sequences see no key
        atomicOr(p.err, kErrKvBound);
        len = 0;
      }
      p.kv_len[b] = len;
      p.kv_start[b] = static_cast<int>(min(end - rows, static_cast<int64_t>(p.cap)));
      p.qt_start[b] = static_cast<int>(min(before_q + q - tiles, static_cast<int64_t>(p.q_tiles)));
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.kv_start[p.batch] = static_cast<int>(min(base_k, static_cast<int64_t>(p.cap)));
    p.qt_start[p.batch] = static_cast<int>(min(base_q, static_cast<int64_t>(p.q_tiles)));
  }
}

// Largest b in [0, batch) with start[b] <= x (start[0] = 0).
__device__ __forceinline__ int find_seq(const int* start, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(start + mid) <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Whether to split, by steps: the time of the pass without it and an even share of a pair. An eighth off, because with
// every pair busy the clock falls by as much (1024 tokens behind 16384 x 32 heads, 64 units: 186 us whole, on 64 pairs at
// 1.87 GHz; 186 us and the join split over 76, at 1.75 GHz). 4096 tokens x 4 heads: 60 us split, 70 whole; x 16 heads,
// where it is not: 118 and 94.
__host__ __device__ __forceinline__ bool split_pays(int64_t whole, int64_t even) {
  return (even < kPieceSteps ? kPieceSteps : even) + kJoinSteps < whole - whole / 8;
}
// The split of a pass's units over the pairs. Without it the end is the longest unit's or, with more units than pairs, the
// pairs-th and the next one's (units are taken the longest first). Every pair takes an equal run of the steps of all
// units, and so at most one piece that begins inside a unit and one that ends inside one. Unit u of the steps
// [first, first + steps) is in pieces 0, 1, ... of pairs pair0, pair0 + 1, ...; its first kUnitSteps stand for no keys.
struct Split {
  int64_t per_head, run;  // steps of a head, of a pair (0: units are not split)
  __device__ __forceinline__ Split(const MlaPrefillParams& p, int tiles, int pairs) {
    per_head = run = 0;
    if (!p.split || static_cast<int64_t>(tiles) * p.heads > kSplitTiles) return;
    per_head = __ldcg(p.steps + tiles);
    const int64_t most = __ldcg(p.steps + 255), even = (per_head * p.heads + pairs - 1) / pairs;
    run = max(even, static_cast<int64_t>(kPieceSteps));
    const int64_t second = tiles * p.heads <= pairs ? 0 : 2 * static_cast<int64_t>(__ldcg(p.steps + 256 + (pairs - 1) / p.heads));
    const int64_t whole = max(most, second);
    if (!split_pays(whole, even)) run = 0;
  }
  __device__ __forceinline__ int pieces(int64_t first, int steps, int& pair0) const {
    pair0 = static_cast<int>(first / run);
    if (steps <= kUnitSteps) return 1;
    if ((pair0 + 1) * run - first <= kUnitSteps) ++pair0;
    return static_cast<int>((first + steps - 1) / run) - pair0 + 1;
  }
  __device__ __forceinline__ int slot(int64_t first, int pair0, int piece) const {  // two for each pair
    return 2 * (pair0 + piece) + (piece == 0 && first > pair0 * run ? 1 : 0);
  }
};

__device__ __forceinline__ unsigned finite_bits2(uint32_t two, unsigned top) {  // larger finite |bf16| of a pair, as fp32 bits
  const unsigned lo = (two << 16) & 0x7fffffffu, hi = two & 0x7fff0000u;
  if (lo < 0x7f800000u) top = max(top, lo);
  if (hi < 0x7f800000u) top = max(top, hi);
  return top;
}
__device__ __forceinline__ unsigned finite_bits(uint4 v, unsigned top) {
  return finite_bits2(v.w, finite_bits2(v.z, finite_bits2(v.y, finite_bits2(v.x, top))));
}

__device__ __forceinline__ bool not_finite2(uint32_t two) {
  return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool not_finite(uint4 v) {
  return not_finite2(v.x) || not_finite2(v.y) || not_finite2(v.z) || not_finite2(v.w);
}

// Query rows of no sequence, before the first one's and behind the last one's: out 0 and lse -inf, as asked. Runs ahead
// of the attention, which overwrites what malformed offsets make overlap.
__device__ __forceinline__ void fill_rows(const MlaPrefillParams& p) {
  const int q0 = min(max(__ldg(p.cu_q), 0), p.total_q), q1 = min(max(__ldg(p.cu_q + p.batch), 0), p.total_q);
  const int64_t rows = static_cast<int64_t>(q0) + (p.total_q - q1), step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int per_row = p.num_heads * (kHeadV / 8);
  for (int64_t i = t0; i < rows * per_row && (p.fill & 1) != 0; i += step) {
    const int64_t r = i / per_row, row = r < q0 ? r : q1 + (r - q0);
    reinterpret_cast<uint4*>(p.out)[row * per_row + (i - r * per_row)] = make_uint4(0, 0, 0, 0);
  }
  for (int64_t i = t0; i < rows * p.num_heads && (p.fill & 2) != 0; i += step) {
    const int64_t h = i / rows, r = i - h * rows;
    p.lse[h * p.total_q + (r < q0 ? r : q1 + (r - q0))] = -INFINITY;
  }
}

// ----------------------------------------------------------------- gather
// A block per 32 packed rows, four rows a warp with all their loads in flight; before that, and before the
// plan's results are needed, a warp per weight row for the maxima.
__global__ void __launch_bounds__(256) gqa_mla_prefill_gather_kernel(const MlaPrefillParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned top_k = 0, top_v = 0;
  // of each warp: rows not finite; largest latent and rotary key of its rows; the smallest row's, inverted
  __shared__ unsigned group_s[5][8];
  pdl_launch_dependents();
  if (p.fill != 0) fill_rows(p);
  if (blockIdx.x == gridDim.x - 1)
    for (int i = threadIdx.x; i < p.num_heads; i += 256) p.units[i] = 0;
  const int wrows = p.num_heads * (kNope + kHeadV);
#pragma unroll 4
  for (int r = blockIdx.x * 8 + warp; r < wrows; r += gridDim.x * 8) {
    const uint4* src = reinterpret_cast<const uint4*>(p.w) + static_cast<int64_t>(r) * (kLat / 8);
    const unsigned t = finite_bits(__ldg(src + 32 + lane), finite_bits(__ldg(src + lane), 0));
    if ((r & 255) < kNope) top_k = max(top_k, t); else top_v = max(top_v, t);
  }
  pdl_wait();
  const int groups = __ldcg(p.kv_start + p.batch) / 32;  // 32 packed rows share a word of valid bits and a sequence
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    // the last sequence that starts at or before the row (empty ones start where the next does)
    const int b = find_seq(p.kv_start, p.batch, 32 * g);
    const int t0 = 32 * g - __ldcg(p.kv_start + b), n = __ldcg(p.kv_len + b);
    // lane l looks up row l's slot
    int64_t slot = -1;
    if (t0 + lane < n) {
      const int t = t0 + lane, blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.width + t / p.page_size);
      if (blk >= 0 && blk < p.num_blocks) slot = static_cast<int64_t>(blk) * p.page_size + t % p.page_size;
    }
    const unsigned ok = __ballot_sync(0xffffffffu, slot >= 0);
    uint4 v[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t from = __shfl_sync(0xffffffffu, slot, 4 * warp + i);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.kv) + from * kRow);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      v[i][0] = from >= 0 ? __ldg(src + lane) : zero;
      v[i][1] = from >= 0 ? __ldg(src + 32 + lane) : zero;
      v[i][2] = from >= 0 && lane < 8 ? __ldg(src + 64 + lane) : zero;
    }
    unsigned bad = 0, top_c = 0, top_r = 0, low_c = 0, low_r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = 32 * g + 4 * warp + i;
      uint4* lat = reinterpret_cast<uint4*>(p.lat) + row * (kLat / 8);
      lat[lane] = v[i][0];
      lat[32 + lane] = v[i][1];
      if (lane < 8) reinterpret_cast<uint4*>(p.kr)[row * (kRope / 8) + lane] = v[i][2];
      const unsigned c = __reduce_max_sync(0xffffffffu, finite_bits(v[i][1], finite_bits(v[i][0], 0)));
      const unsigned r = __reduce_max_sync(0xffffffffu, finite_bits(v[i][2], 0));
      if (lane == 0) p.row_top[row] = make_uint2(c, r);
      top_c = max(top_c, c);
      top_r = max(top_r, r);
      if (c != 0) low_c = max(low_c, ~c);
      if (r != 0) low_r = max(low_r, ~r);
      if (__any_sync(0xffffffffu, not_finite(v[i][0]) || not_finite(v[i][1]))) bad |= 1u << (4 * warp + i);
    }
    if (lane == 0) {
      group_s[0][warp] = bad;
      group_s[1][warp] = top_c;
      group_s[2][warp] = top_r;
      group_s[3][warp] = low_c;
      group_s[4][warp] = low_r;
    }
    __syncthreads();
    if (warp == 0) {  // eight lanes combine each of the first four
      unsigned m = group_s[lane >> 3][lane & 7];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const unsigned other = __shfl_xor_sync(0xffffffffu, m, o);
        m = lane < 8 ? m | other : max(m, other);
      }
      if (lane == 0) {
        p.valid[g] = ok;
        p.bad[g] = m;
      }
      // a maximum of integers: the order of the atomics does not matter
      if (lane != 0 && (lane & 7) == 0 && m != 0) atomicMax(p.amax + 3 + 4 * b + (lane >> 3), m);
    } else if (warp == 1) {
      const unsigned m = __reduce_max_sync(0xffffffffu, lane < 8 ? group_s[4][lane] : 0);
      if (lane == 0 && m != 0) atomicMax(p.amax + 7 + 4 * b, m);
    }
    __syncthreads();
  }
  if (p.split && blockIdx.x == gridDim.x - 1) {
    // first step of each query tile: a step a key tile that its last row sees, and those that a unit costs besides
    __shared__ int steps_s[256];
    steps_s[threadIdx.x] = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.batch) {  // at most kSplitTiles sequences; malformed offsets may make more tiles
      const int b = threadIdx.x, nq = __ldcg(p.q_start + 2 * b + 1), n = __ldcg(p.kv_len + b), t0 = __ldcg(p.qt_start + b);
      for (int i = 0; i * kQTile < nq && t0 + i < 256; ++i) {
        const int see = p.causal ? min(n, n - nq + min(kQTile * (i + 1), nq)) : n;
        steps_s[t0 + i] = (max(see, 0) + kAlign - 1) / kAlign + kUnitSteps;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int v[8], sum = 0, most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = steps_s[8 * lane + i];
        most = max(most, v[i]);
        sum += v[i];
      }
      int at = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += x;
      }
      at -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (8 * lane + i < 255) p.steps[8 * lane + i] = at;
        at += v[i];
      }
      most = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(most));
      if (lane == 0) p.steps[255] = most;
    }
    // query tiles, the longest first
    const int mine = steps_s[threadIdx.x];
    int longer = 0;
#pragma unroll 8
    for (int i = 0; i < kSplitTiles; ++i)
      longer += steps_s[i] > mine || (steps_s[i] == mine && i < static_cast<int>(threadIdx.x));
    if (mine > 0) p.steps[256 + longer] = mine;
  }
  __shared__ unsigned top_s[2][8];
  top_k = __reduce_max_sync(0xffffffffu, top_k);
  top_v = __reduce_max_sync(0xffffffffu, top_v);
  if (lane == 0) {
    top_s[0][warp] = top_k;
    top_s[1][warp] = top_v;
  }
  __syncthreads();
  if (warp == 0) {  // one atomic a block (one a warp took 10 us)
    unsigned m = lane < 16 ? top_s[lane >> 3][lane & 7] : 0;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((lane == 0 || lane == 8) && m != 0) atomicMax(p.amax + (lane >> 3), m);
  }
}

// Exponents that bring keys and values into fp16 (value * 2^-e), from the largest latent c and rotary key r:
// |c . w| <= 512 max|c| max|w| < 2^(Ec + 1 + Ew + 1 + 9), to be below 2^15.
__device__ __forceinline__ int exponent_of(unsigned bits) { return static_cast<int>(bits >> 23) - 127; }
__device__ __forceinline__ void exponents(const unsigned* amax, unsigned c, unsigned r, int& ek, int& ev) {
  const uint2 w = __ldcg(reinterpret_cast<const uint2*>(amax));
  const unsigned wk = w.x, wv = w.y;
  ek = r != 0 ? exponent_of(r) + 1 - 15 : -126;
  if (c != 0 && wk != 0) ek = max(ek, exponent_of(c) + exponent_of(wk) + 11 - 15);
  ev = c != 0 && wv != 0 ? exponent_of(c) + exponent_of(wv) + 11 - 15 : 0;
  ek = min(max(ek, -126), 126);
  ev = min(max(ev, -126), 126);
}
// A sequence's, and whether its tokens have their own instead.
__device__ __forceinline__ bool kv_exponents(const unsigned* amax, int b, int& ek, int& ev) {
  const uint4 t = __ldcg(reinterpret_cast<const uint4*>(amax + 4 + 4 * b));
  exponents(amax, t.x, t.y, ek, ev);
  return (t.x != 0 && (t.x >> 23) - (~t.z >> 23) > kWindow) || (t.y != 0 && (t.y >> 23) - (~t.w >> 23) > kWindow);
}
// Whether keys or values of a sequence may pass fp32's range as they accumulate.
__device__ __forceinline__ bool may_overflow(const unsigned* amax, int b) {
  const uint2 w = __ldcg(reinterpret_cast<const uint2*>(amax));
  return exponent_of(__ldcg(amax + 4 + 4 * b)) + exponent_of(max(w.x, w.y)) + 11 > 127;
}
// Those of a packed row of sequence b; a row of zeros has the sequence's.
__device__ __forceinline__ bool row_exponents(const MlaPrefillParams& p, int b, int64_t row, int& ek, int& ev) {
  const bool wide = kv_exponents(p.amax, b, ek, ev);
  if (wide) {
    const uint2 top = __ldcg(p.row_top + row);
    int rk, rv;
    exponents(p.amax, top.x, top.y, rk, rv);
    if ((top.x | top.y) != 0) ek = rk;
    if (top.x != 0) ev = rv;
  }
  return wide;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }


// ------------------------------------------------------------------ waits
// Whole warp: every lane waits (bounded; no lane runs apart from the others), every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_s, int* err, int bit,
                                          uint64_t limit = kWaitNs) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_s, err, bit, limit));
}
// The same for a barrier that both CTAs' threads arrive on.
__device__ __forceinline__ bool warp_wait_pair(uint32_t bar, uint32_t parity, volatile int* abort_s, int* err, int bit,
                                               uint64_t limit = kWaitNs) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_s, err, bit, limit) && mbar_try_wait_cluster(bar, parity));
}

// -------------------------------------------------------------- expansion
// Keys and values of one head for 256 packed rows are a unit: D [256 rows x 256 columns] =
// rows [256 x 512] W[h]^T, columns 0..127 the head's keys and 128..255 its values (32 MMAs
// of M = 256, N = 256, K = 16, 128 clocks each), by a pair of CTAs. Every pair takes an
// equal run of the units (all heads of a row tile, then the next tile). A CTA keeps its 128
// rows of the latents in shared memory (128 KB) for all heads of the tile and streams its
// half of the weights (the even CTA the key rows, the odd one the value rows) through four
// slots of 64 of the 512 values; the next tile's rows replace the old ones region by region
// behind the MMAs. The accumulators of two units fill tensor memory, so a unit's epilogue
// (scale, round to fp16, through shared memory and a tensor copy out) runs beside the next
// unit's MMAs. Bound by the MMAs and, a fifth over them, the traffic of the copies out:
// 32 heads of 16384 rows take 94 us (1460 TFLOP/s), without the copies out 77.
//
// Roles in each CTA: an MMA warp (the even CTA's issues for both), a copy warp, a warp that
// turns the rotary keys into scaled fp16 (once, with the first head), two epilogue
// warpgroups (keys and values; one for both took 5700 clocks a head).
constexpr int kExThreads = 384, kExSlots = 4, kExRegion = 128 * 128;
constexpr int kExB = 8 * kExRegion, kExOut = kExB + kExSlots * kExRegion, kExBars = kExOut + 2 * kExRegion;
// Barriers. The even CTA's: regions of A and slots of B landed (both halves' bytes), accumulators read (8 warps of each
// CTA). Both CTAs' (MMA commits): regions and slots free, accumulators written, all done.
enum : int { E_A = 0, E_BFULL = E_A + 8, E_DFREE = E_BFULL + kExSlots, E_AFREE = E_DFREE + 2, E_BFREE = E_AFREE + 8,
             E_DFULL = E_BFREE + kExSlots, E_DONE = E_DFULL + 2, E_COUNT = E_DONE + 1 };
constexpr int kExSlot = kExBars + E_COUNT * 8, kExAbort = kExSlot + 4, kExSmem = kExAbort + 4 + 1024;
static_assert(kExSmem <= 227 * 1024, "expansion exceeds shared memory");

struct ExpandMaps {  // boxes of 64 values x 128 rows
  CUtensorMap lat, w, kn, vv;
};

__global__ void __launch_bounds__(kExThreads, 1)
    gqa_mla_prefill_expand_kernel(const MlaPrefillParams p, const __grid_constant__ ExpandMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  pdl_wait();
  pdl_launch_dependents();  // after the wait: what the next kernel reads before its own is then complete
  const int total = __ldcg(p.kv_start + p.batch);
  const int64_t all = static_cast<int64_t>((total + 255) / 256) * p.heads;
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const int u0 = static_cast<int>(all * pair / pairs), u1 = static_cast<int>(all * (pair + 1) / pairs);
  if (u0 >= u1) return;
  const uint32_t half = cluster_rank();
  // unit u: tile u / heads; the heads of a tile start at another one in each tile, so that pairs do not read the same
  // weights at once
  auto tile_of = [&](int u) { return u / p.heads; };
  auto head_of = [&](int u) {
    const int t = u / p.heads, r = u - t * p.heads + t % p.heads;
    return r < p.heads ? r : r - p.heads;
  };
  auto first_of_tile = [&](int u) { return u == u0 || u % p.heads == 0; };
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_s = reinterpret_cast<volatile int*>(sm + kExAbort);
  auto bar = [&](int i) { return base + kExBars + 8u * static_cast<uint32_t>(i); };
  if (tid == 0) {
    for (int i = 0; i < E_COUNT; ++i) mbar_init(bar(i), i >= E_DFREE && i < E_AFREE ? 16u : 1u);
    *abort_s = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 3) tc2_alloc(base + kExSlot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the barriers and the tensor memory of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + kExSlot);
  int* err = p.err;

  if (warp == 0) {
    if (half == 0) {
      constexpr uint32_t idesc = tc_idesc_bf16(256, 256, false, false);
      const uint64_t da0 = tc_sdesc(base, 16, 1024, kSwizzle128B), db0 = tc_sdesc(base + kExB, 16, 1024, kSwizzle128B);
      bool good = true;
      int s = 0;
      uint32_t ph = 0, aph = 1;  // parities of the slot and of the tile's regions
#pragma unroll 1
      for (int u = u0; u < u1 && good; ++u) {
        const int i = u - u0;
        const bool first = first_of_tile(u), last = u + 1 == u1 || (u + 1) % p.heads == 0;
        if (first) aph ^= 1;
        const uint32_t d = tmem + 256 * (i & 1);
        if (i >= 2) good = warp_wait(bar(E_DFREE + (i & 1)), ((i >> 1) - 1) & 1, abort_s, err, kErrTimeoutEmpty);
        tc_fence_after();
#pragma unroll 1
        for (uint32_t c = 0; c < 8 && good; ++c) {
          if (first) good = warp_wait(bar(E_A + c), aph, abort_s, err, kErrTimeoutFull);
          good = good && warp_wait(bar(E_BFULL + s), ph, abort_s, err, kErrTimeoutFull);
          if (!good) break;
          const uint64_t da = da0 + c * (kExRegion >> 4), db = db0 + s * (kExRegion >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc2_mma_warp(d, da + ((kk * 32) >> 4), db + ((kk * 32) >> 4), idesc, kk ? 1u : c);
          tc2_commit_warp(bar(E_BFREE + s));
          if (last) tc2_commit_warp(bar(E_AFREE + c));
          if (++s == kExSlots) {
            s = 0;
            ph ^= 1;
          }
        }
        if (good) tc2_commit_warp(bar(E_DFULL + (i & 1)));
      }
      tc2_commit_warp(bar(E_DONE));
      __syncwarp();
      if (lane == 0) drain_wait(bar(E_DONE), 0);
    }
  } else if (warp == 1) {
    const uint32_t a_full = cluster_addr(bar(E_A), 0), b_full = cluster_addr(bar(E_BFULL), 0);
    const uint32_t expect = half == 0 ? 2 * kExRegion : 0;
    int s = 0, n = 0, tiles = 0, a_regions = 0;
    uint32_t ph = 1;  // parity of the slot's previous release
    bool good = true;
#pragma unroll 1
    for (int u = u0; u < u1 && good; ++u) {
      const int y = (p.head0 + head_of(u)) * 256 + 128 * half, m0 = tile_of(u) * 256 + 128 * half;
      const bool first = first_of_tile(u);
      if (first) ++tiles;
#pragma unroll 1
      for (int c = 0; c < 8; ++c, ++n) {
        if (first) {
          if (tiles > 1) good = warp_wait(bar(E_AFREE + c), tiles & 1, abort_s, err, kErrTimeoutEmpty);
          if (!good) break;
          a_regions = c + 1;
          tma2_load_2d_warp(base + c * kExRegion, &maps.lat, 64 * c, m0, bar(E_A + c), expect, a_full + 8 * c);
        }
        if (n >= kExSlots) good = warp_wait(bar(E_BFREE + s), ph, abort_s, err, kErrTimeoutEmpty);
        if (!good) break;
        tma2_load_2d_warp(base + kExB + s * kExRegion, &maps.w, 64 * c, y, bar(E_BFULL + s), expect, b_full + 8 * s);
        if (++s == kExSlots) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (half == 0 && lane == 0) {  // no copy may still be writing either CTA's shared memory when the pair leaves
      for (int i = n > kExSlots ? n - kExSlots : 0; i < n; ++i) drain_wait(bar(E_BFULL + i % kExSlots), (i / kExSlots) & 1);
      for (int c = 0; c < a_regions; ++c) drain_wait(bar(E_A + c), (tiles - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 2) {
    for (int u = u0; u < u1 && p.head0 == 0; ++u) {
      const int m0 = tile_of(u) * 256 + 128 * half;
      if (u % p.heads != 0 || m0 >= total) continue;  // once a tile, whichever pair has its first unit
      int ek, ev;
      const int b = find_seq(p.kv_start, p.batch, m0);  // 128 rows are one sequence's
      const bool wide = kv_exponents(p.amax, b, ek, ev);
      const float f = pow2(-ek);
      uint4* kr = reinterpret_cast<uint4*>(p.kr) + static_cast<int64_t>(m0) * (kRope / 8);
      auto scaled = [](uint4 v, float f) {
        auto half2 = [&](uint32_t w) { return pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
        return make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
      };
      if (!wide) {
#pragma unroll 4
        for (int i = lane; i < 128 * kRope / 8; i += 32) kr[i] = scaled(kr[i], f);
        continue;
      }
      for (int i = lane; i < 128; i += 32) {
        int rk, rv;
        row_exponents(p, b, m0 + i, rk, rv);
        // factors of the row's scores (0 below 2^-126) and, in base 2, of its values; none for values that are all 0
        p.row_scale[m0 + i] = make_float2(rk - ek < -126 ? 0.f : pow2(rk - ek),
                                          __ldcg(p.row_top + m0 + i).x != 0 ? static_cast<float>(rv - ev) : -INFINITY);
        for (int c = 0; c < kRope / 8; ++c) kr[i * (kRope / 8) + c] = scaled(kr[i * (kRope / 8) + c], pow2(-rk));
      }
    }
  } else if (warp >= 4) {
    const int part = (warp >> 2) - 1;  // 0: keys, 1: values
    const int wq = warp & 3, row = 32 * wq + lane;
    const bool issuer = wq == 0 && lane == 0;
    float f = 1.f;
    const uint32_t of_bad = part == 0 ? 0x7fff7fffu : 0u;
    const uint32_t dfree = cluster_addr(bar(E_DFREE), 0);
    const uint32_t dst = base + kExOut + part * kExRegion;
    bool bad = false, over = false;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      const int i = u - u0, m0 = tile_of(u) * 256 + 128 * half;  // this CTA's packed rows (may lie past the last one)
      const bool out = m0 < total;
      if (first_of_tile(u) && out) {  // 128 rows are one sequence's
        int ek, ev;
        const int b = find_seq(p.kv_start, p.batch, m0);
        row_exponents(p, b, m0 + row, ek, ev);
        f = pow2(part == 0 ? -ek : -ev);
        over = may_overflow(p.amax, b);
        bad = ((__ldcg(p.bad + (m0 >> 5) + wq) >> lane) & 1u) != 0;
      }
      const bool good = warp_wait(bar(E_DFULL + (i & 1)), (i >> 1) & 1, abort_s, err, kErrTimeoutFull);
      int every;  // the four warps agree, so that none is left at the barriers below
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
          : "=r"(every)
          : "r"(good ? 1 : 0), "r"(1 + part)
          : "memory");
      if (!every) break;
      tc_fence_after();
      const uint32_t d = tmem + (static_cast<uint32_t>(32 * wq) << 16) + 256 * (i & 1) + 128 * part;
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {  // 64 columns
        uint32_t v[64];
        tc_ld32(d + 64 * r, v);
        tc_ld32(d + 64 * r + 32, v + 32);
        tc_wait_ld();
        if (over) {  // a weight of 0 times an infinity would be NaN in rows that do not see the token
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e] = __float_as_uint(fminf(fmaxf(__uint_as_float(v[e]), -FLT_MAX), FLT_MAX));
        }
        if (r == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(dfree + 8 * (i & 1));
        }
        if (issuer) bulk_wait_read<0>();  // the last copy out has read the buffer
        asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = bad ? of_bad : pack_f16(__uint_as_float(v[8 * c + 2 * e]) * f, __uint_as_float(v[8 * c + 2 * e + 1]) * f);
          st_shared_u4(sw128(dst, row, c), o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
        if (issuer && out) {
          tma_store_2d(part == 0 ? &maps.kn : &maps.vv, 64 * r, head_of(u) * p.cap + m0, dst);
          bulk_commit();
        }
      }
    }
    if (issuer) bulk_wait_read<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's arrivals, MMAs and copies are done too
  if (warp == 3) tc2_dealloc(tmem, 512);
}

// -------------------------------------------------------------- attention
// A pair of CTAs takes 512 query rows of one head as two tiles of 256 (128 rows
// a CTA each) and walks the keys in tiles of 128. Per tile and key tile, S = Q K^T
// (M = 256, N = 128 keys, 12 MMAs of K = 16) lands in tensor memory, a thread per
// row turns it into fp16 probabilities that overwrite it there, and O += P V (8
// MMAs, P read from tensor memory) accumulates beside it. The two tiles alternate:
// while one is in its softmax, the tensor cores do the other's O and next S.
//
// Why pairs: the queries take 96 KB of a CTA's shared memory, and V and the next K
// are in use at once (80 KB at 128 keys). One CTA alone has room for 1.6 key tiles
// in flight, and its MMAs waited for loads (measured: 3900 to 4000 clocks a key tile of
// both query tiles, against 2560 of MMAs). A pair keeps half of each key and value tile
// in each CTA, which gives a ring of three tiles, and halves the L2 reads: 2520 to 2600
// clocks once caches and clock have settled, all of them MMAs (the clock then holds
// 1.75 to 1.87 GHz of 2.07: the power is what is left to save).
//
// The pairs are persistent: a unit is the 512 query rows of one head; a pair begins with the unit of its own number
// and takes the next ones from a counter (heads in groups, the query tiles of the most keys first), a few key tiles
// before it needs them. What a unit costs beside its key tiles is then the copy and turning of its queries, the first
// scores and the last output: 7 us, where a pair launched per unit took 13 to 15. The barriers' phases, the rings and
// the turns simply run on from unit to unit.
//
// With few units (a chunk of a prompt behind a long prefix, few heads) pairs would be idle: then each takes an equal run
// of the key tiles of all units (as the plan's lengths make them), writes outputs and statistics of the pieces of units
// that others have a part of in fp32, and a kernel behind it joins them. 200 tokens behind 16384 x 16 heads: 123 us
// instead of 228 in all, 1024 behind 32768 x 16 heads 305 instead of 456, 256 behind 131072 x 1 head 189 instead of
// 1346. The pass that may split has a kernel of its own: a key tile takes 2 % longer in it.
//
// Roles in each CTA: two softmax warpgroups and two MMA warps (one of each per tile;
// the even CTA's issue for both CTAs, in turns), a copy warp. Issuing an MMA takes
// nearly as long as its 64 clocks, so with one MMA warp for both tiles its waits and
// commits stood between the MMAs (1690 clocks a step of 1280); without turns the two
// tiles fall into step and the tensor cores idle during their softmax. Shared memory: the queries (2 x 48 KB, fp16,
// 128-byte swizzle), three slots of half a key tile (64 keys x 192) and three of
// half a value tile (128 keys x 64 values). Tensor memory: S at columns 0 and 128
// (P over its first 64), O at 256 and 384.
//
// The running maximum moves only when a row's scores pass it by 2^8, so O is
// seldom rescaled; probabilities are held times 2^7, at most 2^15, which keeps
// small ones fp16 normals.
//
// A wide sequence's keys and values have an exponent a token. Scores are then scaled by column, and the weights of O are
// 2^(score + value exponent) against a running maximum of their own (the sum keeps the scores'): a second exponential a
// score and two passes over the tile. 8192 tokens x 16 heads, one of them 2^60 times as large: 764 us in all (239
// without it).
//
// Every wait is bounded: on a timeout the CTA flags
// the device error word and leaves after draining its copies and MMAs.
//
// Measured: 8192 causal tokens x 16 heads 198 us (1740 TFLOP/s), 1024 tokens behind
// 16384 x 32 heads 193 us (1720 TFLOP/s, on 64 of the 76 pairs).
//
// A timeout frees what the CTA holds and leaves, after the drains of its own copies and MMAs. A pair's copies are counted
// by the even CTA alone, so the odd one's last are only known to have landed because every wait lasts 2 s: this path is
// not for shorter limits, and the test hook's does not reach it.
constexpr int kKTile = 128, kSlots = 3;
constexpr int kQRegion = 128 * 128, kQTileBytes = 3 * kQRegion;  // 128 rows x 64 values; a CTA's half of a query tile
constexpr int kKRegion = 64 * 128, kKSlot = 3 * kKRegion;        // 64 keys x 64 values
constexpr int kVSlot = kKTile * 128;                             // 128 keys x 64 values
constexpr int kAtThreads = 384, kCopyWarp = 2, kSoftWarp = 4;  // MMA warps 0 and 1; warp 3 only allots registers
// 168 registers a thread at launch (384 x 168 of the SM's 65536); the split below is no more
constexpr int kSoftRegs = 216, kRoleRegs = 72;
static_assert(256 * kSoftRegs + 128 * kRoleRegs <= kAtThreads * 168, "register split");
constexpr float kShift = 7.f, kMoveBy = 8.f;
constexpr int kAtK = 2 * kQTileBytes, kAtV = kAtK + kSlots * kKSlot, kAtBars = kAtV + kSlots * kVSlot;
// Barriers. The even CTA's: K and V landed (both halves' bytes), queries and the halves of P written (4 warps of
// each CTA), whose turn it is to issue, a unit's number read by the other CTA. Both CTAs': K and V
// slots free (a commit of each MMA warp), S and O written, queries read (MMA commits), all done; bf16 queries landed;
// unit published, unit taken (every warp with a role); the odd CTA's: the unit's number has come.
enum : int { B_KFULL = 0, B_VFULL = B_KFULL + kSlots, B_Q = B_VFULL + kSlots, B_P = B_Q + 2, B_KFREE = B_P + 4,
             B_VFREE = B_KFREE + kSlots, B_S = B_VFREE + kSlots, B_O = B_S + 2, B_QFREE = B_O + 2, B_DONE = B_QFREE + 2,
             B_TURN = B_DONE + 1, B_QRAW = B_TURN + 2, B_UFULL = B_QRAW + 2, B_UFREE = B_UFULL + 2, B_MFULL = B_UFREE + 2,
             B_MFREE = B_MFULL + 2, B_COUNT = B_MFREE + 2 };
__device__ __forceinline__ uint32_t attn_bar_count(int i, uint32_t half) {
  if (i >= B_Q && i < B_KFREE) return 8;
  if ((i >= B_KFREE && i < B_S) || i == B_DONE) return 2;
  if (i >= B_UFREE && i < B_MFULL) return half == 0 ? 10 : 8;  // softmax and, in the even CTA, MMA warps
  return 1;
}
constexpr int kAtSlot = kAtBars + B_COUNT * 8, kAtAbort = kAtSlot + 4;
constexpr int kAtUnits = (kAtAbort + 4 + 15) / 16 * 16, kAtMail = kAtUnits + 2 * 64;  // two units of 13 words, two numbers
constexpr int kAtSmem = kAtMail + 8 + 1024;  // the base is rounded up to 1024 bytes (swizzle atoms)
static_assert(kAtSmem <= 227 * 1024, "prompt attention exceeds shared memory");

struct AttnMaps {  // boxes of 64 values x 64 rows (keys) and x 128 rows (values, queries of one head)
  CUtensorMap kn, vv, kr, q;
};

// Two scores to probabilities 2^(s sc + off): packed fp16, and their sum added to l.
__device__ __forceinline__ uint32_t exp_pair(uint32_t s0, uint32_t s1, uint64_t sc2, uint64_t off2, uint64_t& l) {
  float x0, x1;
  unpack2(fma2(pack2(__uint_as_float(s0), __uint_as_float(s1)), sc2, off2), x0, x1);
  x0 = ex2(x0);
  x1 = ex2(x1);
  l = add2(l, pack2(x0, x1));
  return pack_f16(x0, x1);
}

// Bits c of a word whose key 32 k + c (of the key tile at t0) is at most lim.
__device__ __forceinline__ unsigned upto(int lim, int t0, int k) {
  const int c = lim - t0 - 32 * k;
  return c < 0 ? 0u : (c >= 31 ? 0xffffffffu : (2u << c) - 1u);
}

// A word into the shared memory of a CTA of the cluster, counted by that CTA's mbarrier.
__device__ __forceinline__ void st_async(uint32_t addr, int value, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];" ::"r"(addr), "r"(value), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float natural_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
}

// Words of a unit in shared memory: whether there is one, head of the pass, first query row of the sequence, its
// queries, their first row among all, its keys (from the piece's first on), that one's packed row, key tiles of the two
// query tiles, exponents; where a piece's rows go, -1: the unit is in one piece; whether tokens have their own exponents.
enum : int { U_OK = 0, U_HEAD, U_ROW, U_NQ, U_Q0, U_KEYS, U_KV0, U_NT0, U_NT1, U_EK, U_EV, U_SLOT, U_WIDE };
constexpr uint64_t kUnitWaitNs = 10 * kWaitNs;  // a unit may last longer than any wait inside it

template <bool kSplit>
__global__ void __launch_bounds__(kAtThreads, 1)
    gqa_mla_prefill_attn_kernel(const MlaPrefillParams p, const __grid_constant__ AttnMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t half = cluster_rank();  // which 128 rows of a tile, which half of the keys and values
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_s = reinterpret_cast<volatile int*>(sm + kAtAbort);
  auto bar = [&](int i) { return base + kAtBars + 8u * static_cast<uint32_t>(i); };
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), attn_bar_count(i, half));
    *abort_s = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) tc2_alloc(base + kAtSlot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the barriers and the tensor memory of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + kAtSlot);
  int* err = p.err;

  // Waits for unit number `it` of this pair, for a warp with a role; false at the end (or on a timeout). A role reads a
  // unit's words where it needs them (in registers they spilled) and leaves the unit when it has read the last.
  auto unit_word = [&](int it, int w) { return reinterpret_cast<const volatile int*>(sm + kAtUnits + 64 * (it & 1))[w]; };
  auto enter_unit = [&](int it) -> bool {
    return warp_wait(bar(B_UFULL + (it & 1)), (it >> 1) & 1, abort_s, err, kErrTimeoutFull, kUnitWaitNs) &&
           unit_word(it, U_OK) != 0;
  };
  auto leave_unit = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_UFREE + (it & 1)));
  };

  if (warp < kSoftWarp) {
    setmaxnreg_dec<kRoleRegs>();
    if (warp == kCopyWarp) {
      // What the plan and the gather wrote is complete when this kernel may start (the expansion lets it start after its
      // own wait); only the copies of keys and values wait for the expansion. Read past L1, which an earlier call's
      // values of the same workspace may still be in.
      const int tiles = __ldcg(p.qt_start + p.batch), pairs = gridDim.x >> 1;
      const int start = lane + 1 < p.batch ? __ldcg(p.qt_start + lane + 1) : INT_MAX;  // of the first 32 after sequence 0
      const uint32_t kfull = cluster_addr(bar(B_KFULL), 0), vfull = cluster_addr(bar(B_VFULL), 0);
      const uint32_t k_bytes = half == 0 ? 2 * kKSlot : 0, v_bytes = half == 0 ? 2 * kVSlot : 0;
      int s = 0, keys = 0, values = 0;  // slot, counts of copies begun
      uint32_t ph = 1;                  // parity of the slot's previous release
      int queries[2] = {0, 0};          // loads of each tile's queries
      const int pair = blockIdx.x >> 1;
      int rank = pair, next = 0;
      bool good = true;
      const Split cut(p, tiles, pairs);
      const bool split = kSplit && cut.run > 0;
      int64_t x = cut.run * pair;
      const int64_t x_end = min(x + cut.run, cut.per_head * p.heads);
#pragma unroll 1
      for (int it = 0;; ++it) {
        const int us = it & 1;
        if (it > 0 && !split) {  // the even CTA took the unit's number, the odd one gets it
          const uint32_t mail = base + kAtMail + 4 * us;
          if (half == 0) {
            rank = pairs + __shfl_sync(0xffffffffu, next, 0);
            if (it > 2) {
              good = warp_wait_pair(bar(B_MFREE + us), ((it - 3) >> 1) & 1, abort_s, err, kErrTimeoutEmpty, kUnitWaitNs);
              if (!good) break;
            }
            if (lane == 0) st_async(cluster_addr(mail, 1), rank, cluster_addr(bar(B_MFULL + us), 1));
          } else {
            if (lane == 0) mbar_arrive_expect_tx(bar(B_MFULL + us), 4);
            good = warp_wait(bar(B_MFULL + us), ((it - 1) >> 1) & 1, abort_s, err, kErrTimeoutFull, kUnitWaitNs);
            if (!good) break;
            rank = *reinterpret_cast<volatile int*>(sm + kAtMail + 4 * us);
          }
          __syncwarp();
        }
        bool ok = false, wide = false;
        int hp = 0, b = 0, i0 = 0, n = 0, kv0 = 0, ek = 0, ev = 0, nt[2] = {0, 0};
        int qt = 0, k0 = 0, k1 = INT_MAX, slot = -1;
        int2 qs = {0, 0};
        if (!split) {
          ok = rank < static_cast<int64_t>(tiles) * p.heads;
          if (ok) {
            // in order: groups of heads whose keys and values stay in L2 together, within a group the last query tiles
            // (the most keys, if causal) first
            const int group = static_cast<int>(rank / (static_cast<int64_t>(tiles) * p.head_group));
            const int in_group = static_cast<int>(rank - static_cast<int64_t>(group) * tiles * p.head_group);
            const int gh = min(p.head_group, p.heads - group * p.head_group);
            qt = tiles - 1 - in_group / gh;
            hp = group * p.head_group + in_group % gh;
          }
        }
        while (split && !ok && x < x_end) {
          hp = static_cast<int>(x / cut.per_head);
          const int at = static_cast<int>(x - hp * cut.per_head);
          qt = 0;
#pragma unroll
          for (int i = 0; i < kSplitTiles / 32 + 1; ++i) {
            const int t = 32 * i + lane + 1;
            qt += __popc(__ballot_sync(0xffffffffu, t < tiles && __ldcg(p.steps + min(t, tiles)) <= at));
          }
          const int u0 = __ldcg(p.steps + qt), steps = __ldcg(p.steps + qt + 1) - u0;
          const int64_t first = hp * cut.per_head + u0;
          const int begin = at - u0, end = static_cast<int>(min(x_end - first, static_cast<int64_t>(steps)));
          k0 = max(begin - kUnitSteps, 0);
          k1 = max(end - kUnitSteps, 0);
          ok = k1 > k0 || (steps == kUnitSteps && begin == 0);
          x = first + end;
          int pair0;
          slot = cut.pieces(first, steps, pair0) > 1 ? cut.slot(first, pair0, pair - pair0) : -1;
        }
        if (ok) {
          // the last sequence that starts at this tile or before it
          b = __popc(__ballot_sync(0xffffffffu, start <= qt));
          for (int k = 33; b == k - 1 && k < p.batch; k += 32)
            b += __popc(__ballot_sync(0xffffffffu, k + lane < p.batch && __ldcg(p.qt_start + min(k + lane, p.batch)) <= qt));
          qs = __ldcg(reinterpret_cast<const int2*>(p.q_start) + b);
          n = __ldcg(p.kv_len + b);
          kv0 = __ldcg(p.kv_start + b);
          i0 = (qt - __ldcg(p.qt_start + b)) * kQTile;
          wide = kv_exponents(p.amax, b, ek, ev);
          // key tiles of each query tile (the same in both CTAs): up to the last key that its last row sees
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int last_row = min(i0 + 256 * (a + 1), qs.y) - 1;
            int see = last_row < i0 + 256 * a ? 0 : (p.causal ? min(n, n - qs.y + last_row + 1) : n);
            nt[a] = max(min((max(see, 0) + kKTile - 1) / kKTile, k1) - k0, 0);
          }
          n -= kKTile * k0;
          kv0 += kKTile * k0;
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          if (!good || nt[a] == 0) continue;
          if (queries[a] > 0) good = warp_wait(bar(B_QFREE + a), (queries[a] - 1) & 1, abort_s, err, kErrTimeoutEmpty);
          if (!good) continue;
          ++queries[a];
#pragma unroll 1
          for (int r = 0; r < 3; ++r)
            tma_load_3d_warp(base + a * kQTileBytes + r * kQRegion, &maps.q, 64 * r, p.head0 + hp,
                             qs.x + i0 + 256 * a + 128 * half, bar(B_QRAW + a), r == 0 ? kQTileBytes : 0);
        }
        if (!good) break;
        if (it >= 2 && !warp_wait(bar(B_UFREE + us), ((it >> 1) - 1) & 1, abort_s, err, kErrTimeoutEmpty, kUnitWaitNs)) break;
        if (lane == 0) {
          volatile int* w = reinterpret_cast<volatile int*>(sm + kAtUnits + 64 * us);
          w[U_OK] = ok ? 1 : 0;
          w[U_HEAD] = hp;
          w[U_EK] = ek;
          w[U_EV] = ev;
          w[U_ROW] = i0;
          w[U_NQ] = qs.y;
          w[U_Q0] = qs.x;
          w[U_KEYS] = n;
          w[U_KV0] = kv0;
          w[U_NT0] = nt[0];
          w[U_NT1] = nt[1];
          w[U_SLOT] = slot;
          w[U_WIDE] = wide ? 1 : 0;
          mbar_arrive(bar(B_UFULL + us));
        }
        __syncwarp();
        if (!ok) break;
        if (it == 0) pdl_wait();
        const int total = max(nt[0], nt[1]), ask_at = max(total - 6, 0);
        const int y0 = hp * p.cap + kv0 + 64 * half, r0 = kv0 + 64 * half, v0 = hp * p.cap + kv0;
#pragma unroll 1
        for (int j = 0; j < total && good; ++j) {
          // the next unit is taken a few key tiles before the end of this one, not sooner: another pair may be free
          if (j == ask_at && !split && half == 0 && lane == 0) next = atomicAdd(p.units + p.pass, 1);
          __syncwarp();
          const uint32_t kd = base + kAtK + s * kKSlot, vd = base + kAtV + s * kVSlot;
          if (keys >= kSlots) good = warp_wait(bar(B_KFREE + s), ph, abort_s, err, kErrTimeoutEmpty);
          if (!good) break;
          tma2_load_2d_warp(kd, &maps.kn, 0, y0 + j * kKTile, bar(B_KFULL + s), k_bytes, kfull + 8 * s);
          tma2_load_2d_warp(kd + kKRegion, &maps.kn, 64, y0 + j * kKTile, 0, 0, kfull + 8 * s);
          tma2_load_2d_warp(kd + 2 * kKRegion, &maps.kr, 0, r0 + j * kKTile, 0, 0, kfull + 8 * s);
          ++keys;
          if (values >= kSlots) good = warp_wait(bar(B_VFREE + s), ph, abort_s, err, kErrTimeoutEmpty);
          if (!good) break;
          tma2_load_2d_warp(vd, &maps.vv, 64 * half, v0 + j * kKTile, bar(B_VFULL + s), v_bytes, vfull + 8 * s);
          ++values;
          if (++s == kSlots) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!good) break;
        if (total == 0 && !split && half == 0 && lane == 0) next = atomicAdd(p.units + p.pass, 1);
        if (it > 0 && !split && half == 1 && lane == 0) mbar_arrive_cluster(cluster_addr(bar(B_MFREE + us), 0));
        __syncwarp();
      }
      if (keys == 0) pdl_wait();
      // no copy may still be writing either CTA's shared memory when the pair leaves
      if (lane == 0)
        for (int a = 0; a < 2; ++a)
          if (queries[a] > 0) drain_wait(bar(B_QRAW + a), (queries[a] - 1) & 1);
      if (half == 0 && lane == 0)
        for (int k = 0; k < kSlots; ++k) {
          const int i = keys - 1 - k, v = values - 1 - k;
          if (i >= 0) drain_wait(bar(B_KFULL + i % kSlots), (i / kSlots) & 1);
          if (v >= 0) drain_wait(bar(B_VFULL + v % kSlots), (v / kSlots) & 1);
        }
      __syncwarp();
    } else if (warp < 2 && half == 0) {
      // tile a: the whole warp walks the keys (warp-uniform operands), one elected lane issues
      const int a = static_cast<int>(uniform(warp));
      const uint32_t ub = uniform(base), ut = uniform(tmem);
      constexpr uint32_t idesc_s = tc_idesc_f16(256, kKTile, false, false);
      constexpr uint32_t idesc_o = tc_idesc_f16(256, kHeadV, false, true);
      const uint64_t dq0 = tc_sdesc(ub + a * kQTileBytes, 16, 1024, kSwizzle128B);
      const uint64_t dk0 = tc_sdesc(ub + kAtK, 16, 1024, kSwizzle128B);
      // V as B: N = 64 values a CTA (one swizzle atom), K = keys in 8-row groups (SBO)
      const uint64_t dv0 = tc_sdesc(ub + kAtV, kVSlot, 1024, kSwizzle128B);
      const uint32_t s_col = ut + 128 * a, o_col = ut + 256 + 128 * a;
      auto bar = [&](int i) { return ub + kAtBars + 8u * static_cast<uint32_t>(i); };
      int s = 0;  // slot and parity of tile j
      uint32_t ph = 0, np = 0, nq = 0, turn = 0;  // counts of P read, queries taken, turns had
      bool good = true;
#pragma unroll 1
      for (int it = 0; good && enter_unit(it); ++it) {
        const int mine = static_cast<int>(uniform(unit_word(it, U_NT0 + a)));
        const int total = max(mine, static_cast<int>(uniform(unit_word(it, U_NT0 + 1 - a))));
        leave_unit(it);
        if (total == 0) continue;
#pragma unroll 1
        for (int j = 0; j <= total; ++j, ++turn) {
          // O += P(j - 1) V(j - 1), then S(j) = Q K(j), in turn with the other tile's warp. Slots of keys that this
          // tile does not see are freed as they land, not sooner: an arrival for the slot's next use would count for
          // this one.
          const int vs = s == 0 ? kSlots - 1 : s - 1;
          const uint32_t vp = s == 0 ? ph ^ 1u : ph;
          const bool pv = j > 0 && j <= mine, qk = j < mine;
          if (j > 0) good = warp_wait(bar(B_VFULL + vs), vp, abort_s, err, kErrTimeoutFull);
          if (j < total) good = good && warp_wait(bar(B_KFULL + s), ph, abort_s, err, kErrTimeoutFull);
          if (j == 0 && qk) good = good && warp_wait_pair(bar(B_Q + a), nq & 1, abort_s, err, kErrTimeoutFull);
          if (a == 1 || turn > 0)
            good = good && warp_wait(bar(B_TURN + a), (a == 1 ? turn : turn - 1) & 1, abort_s, err, kErrTimeoutFull);
          if (pv) good = good && warp_wait(bar(B_P + 2 * a), np & 1, abort_s, err, kErrTimeoutFull);
          if (!good) break;
          tc_fence_after();
          if (pv) {
            const uint64_t dv = dv0 + vs * (kVSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc2_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, kk ? 1u : j - 1);
            good = warp_wait(bar(B_P + 2 * a + 1), np & 1, abort_s, err, kErrTimeoutFull);
            if (!good) break;
            ++np;
            tc_fence_after();
#pragma unroll
            for (int kk = 4; kk < 8; ++kk)
              tc2_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, 1u);
          }
          const uint64_t dk = dk0 + s * (kKSlot >> 4);
          auto scores = [&](int r) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc2_mma_warp(s_col, dq0 + ((r * kQRegion + kk * 32) >> 4), dk + ((r * kKRegion + kk * 32) >> 4), idesc_s,
                           (r | kk) ? 1u : 0u);
          };
          if (qk) scores(0);
          if (lane == 0) mbar_arrive(bar(B_TURN + 1 - a));  // early: the rest is issued before the other warp gets going
          __syncwarp();
          if (qk) {
            scores(1);
            scores(2);
            tc2_commit_warp(bar(B_S + a));
            if (j == mine - 1) tc2_commit_warp(bar(B_QFREE + a));
          }
          if (j > 0) tc2_commit_warp(bar(B_VFREE + vs));
          if (pv && j == mine) tc2_commit_warp(bar(B_O + a));
          if (j < total) {
            tc2_commit_warp(bar(B_KFREE + s));
            if (++s == kSlots) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (mine > 0) ++nq;
      }
      tc2_commit_warp(bar(B_DONE));  // every MMA done before tensor memory is freed
      __syncwarp();
      if (lane == 0) drain_wait(bar(B_DONE), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------- a softmax warpgroup: tile a, row 32 wq + lane
    setmaxnreg_inc<kSoftRegs>();
    const int a = (warp - kSoftWarp) >> 2, wq = warp & 3;
    const uint32_t quarter = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t s_col = tmem + quarter + 128 * a, o_col = tmem + quarter + 256 + 128 * a;
    const uint32_t q_bar = cluster_addr(bar(B_Q + a), 0), p_bar = cluster_addr(bar(B_P + 2 * a), 0);
    uint32_t scored = 0, turned = 0;  // counts of S read and of queries turned
    bool good = true;
#pragma unroll 1
    for (int it = 0; good && enter_unit(it); ++it) {
      const int nt = unit_word(it, U_NT0 + a);
      int row_exp = 0;
      if (nt > 0) {
        // this row's query, copied in as bf16, to fp16 with its largest value in [2^10, 2^11). Small loops: straight-line
        // code for the whole row took 6 to 8 us a CTA, most of it instruction fetch. Rows past the sequence's queries hold
        // whatever follows them; their results are not stored.
        good = warp_wait(bar(B_QRAW + a), turned & 1, abort_s, err, kErrTimeoutFull);
        if (!good) break;
        const uint32_t q_row = base + a * kQTileBytes;
        unsigned top = 0;
#pragma unroll 4
        for (int k = 0; k < 24; ++k) {
          uint4 v;
          ld_shared_u4(sw128(q_row + (k >> 3) * kQRegion, 32 * wq + lane, k & 7), v.x, v.y, v.z, v.w);
          top = finite_bits(v, top);
        }
        row_exp = top != 0 ? max(exponent_of(top), -116) - 10 : 0;
        const float f = p.scale_log2 < 0.f ? -pow2(-row_exp) : pow2(-row_exp);
        auto half2 = [&](uint32_t w) { return pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
#pragma unroll 2
        for (int k = 0; k < 24; ++k) {
          const uint32_t at = sw128(q_row + (k >> 3) * kQRegion, 32 * wq + lane, k & 7);
          uint4 v;
          ld_shared_u4(at, v.x, v.y, v.z, v.w);
          st_shared_u4(at, half2(v.x), half2(v.y), half2(v.z), half2(v.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(q_bar);
      }
      const int sc_exp = row_exp + unit_word(it, U_EK);  // in two factors, so that nothing between leaves the range
      const float sc = fmaxf(fabsf(p.scale_log2) * pow2(sc_exp >> 1) * pow2(sc_exp - (sc_exp >> 1)), 1e-37f);  // > 0: -inf * sc stays -inf
      // the last key that the warp's first row and this row see
      const int row0 = unit_word(it, U_ROW) + 256 * a + 128 * half + 32 * wq;
      const int lim0 = p.causal ? unit_word(it, U_KEYS) - unit_word(it, U_NQ) + row0 : INT_MAX;
      const int lim = p.causal ? lim0 + lane : INT_MAX;
      const uint4* valid = reinterpret_cast<const uint4*>(p.valid) + (unit_word(it, U_KV0) >> 7);
      float m = -INFINITY, m_out = -INFINITY;  // O's unit, where it is not the maximum
      uint64_t l2 = 0;
      const bool wide = unit_word(it, U_WIDE) != 0;
      if (wide) {
        const float2* scales = p.row_scale + unit_word(it, U_KV0);
        float l = 0.f;
        pdl_wait();  // the expansion's row scales
#pragma unroll 1
        for (int j = 0; j < nt && good; ++j) {
          const int t0 = j * kKTile;
          const uint4 vw = __ldcg(valid + j);
          good = warp_wait(bar(B_S + a), scored & 1, abort_s, err, kErrTimeoutFull);
          if (!good) break;
          ++scored;
          tc_fence_after();
          // columns [32 c, 32 c + 32): scores in base 2, and the exponents of their values
          auto columns = [&](int c, auto&& each) {
            uint32_t s[32];
            tc_ld32(s_col + 32 * c, s);
            tc_wait_ld();
            const unsigned w = (c == 0 ? vw.x : c == 1 ? vw.y : c == 2 ? vw.z : vw.w) & upto(lim, t0, c);
            const float4* fg = reinterpret_cast<const float4*>(scales + t0 + 32 * c);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float4 v = __ldcg(fg + k);
              each(2 * k, ((w >> (2 * k)) & 1u) != 0 ? __uint_as_float(s[2 * k]) * v.x * sc : -INFINITY, v.y);
              each(2 * k + 1, ((w >> (2 * k + 1)) & 1u) != 0 ? __uint_as_float(s[2 * k + 1]) * v.z * sc : -INFINITY, v.w);
            }
          };
          float top = -INFINITY, top_out = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
            columns(c, [&](int, float x, float g) {
              top = fmaxf(top, x);
              top_out = fmaxf(top_out, x + g);
            });
          if (top > m + kMoveBy) {
            l = m == -INFINITY ? 0.f : l * ex2(m - top);
            m = top;
          }
          const bool move = top_out > m_out + kMoveBy;
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = !move ? 1.f : (m_out == -INFINITY ? 0.f : ex2(m_out - top_out));
            if (move) m_out = top_out;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tc_ld16(o_col + 16 * c, o);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tc_st16(o_col + 16 * c, o);
              }
            }
          }
          const float off = m == -INFINITY ? 0.f : kShift - m, off_out = m_out == -INFINITY ? 0.f : kShift - m_out;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            float last = 0.f;
            columns(c, [&](int k, float x, float g) {
              l += ex2(x + off);
              const float y = ex2(x + g + off_out);
              if (k & 1) pk[k >> 1] = pack_f16(last, y);
              last = y;
            });
            tc_st16(s_col + 16 * c, pk);  // over scores that have been read
            if (c & 1) {
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(p_bar + 8 * (c >> 1));
            }
          }
        }
        l2 = pack2(l, 0.f);
      }
      for (int j = 0; j < nt && good && !wide; ++j) {
        const uint4 vw = __ldcg(valid + j);
        good = warp_wait(bar(B_S + a), scored & 1, abort_s, err, kErrTimeoutFull);
        if (!good) break;
        ++scored;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(s_col + 32 * c, s + 32 * c);
        tc_wait_ld();
        const int t0 = j * kKTile;
        if ((vw.x & vw.y & vw.z & vw.w) != 0xffffffffu || t0 + kKTile - 1 > lim0) {
          const unsigned w[4] = {vw.x & upto(lim, t0, 0), vw.y & upto(lim, t0, 1), vw.z & upto(lim, t0, 2), vw.w & upto(lim, t0, 3)};
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (((w[c >> 5] >> (c & 31)) & 1u) == 0) s[c] = 0xff800000u;  // -inf
        }
        // Optimistic: the first half's probabilities are formed with the running maximum as it stands, beside the search
        // for this tile's; only if a row passed it by 2^8 (the first tile, and seldom after) are they formed again.
        const uint64_t sc2 = pack2(sc, sc);
        uint64_t off2 = pack2(kShift - m, kShift - m), l_new = 0;
        uint32_t pk[32];
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          pk[k] = exp_pair(s[2 * k], s[2 * k + 1], sc2, off2, l_new);
          mx[k & 3] = max3(mx[k & 3], max3(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1]), __uint_as_float(s[4 * k + 2])),
                           __uint_as_float(s[4 * k + 3]));
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;
        const bool move = top > m + kMoveBy;
        if (__any_sync(0xffffffffu, move || m == -INFINITY)) {
          const float alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2(m - top));
          if (move) m = top;
          float lo, hi;
          unpack2(l2, lo, hi);
          l2 = pack2(lo * alpha, hi * alpha);
          if (j > 0) {  // the commit that signalled S also covers the previous tile's O
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tc_ld16(o_col + 16 * c, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tc_st16(o_col + 16 * c, o);
            }
          }
          const float off = m == -INFINITY ? 0.f : kShift - m;
          off2 = pack2(off, off);
          l_new = 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) pk[k] = exp_pair(s[2 * k], s[2 * k + 1], sc2, off2, l_new);
        }
        tc_st32(s_col, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(p_bar + 8 * 0);  // half of the keys: the MMAs may start on it
#pragma unroll
        for (int k = 0; k < 32; ++k) pk[k] = exp_pair(s[64 + 2 * k], s[64 + 2 * k + 1], sc2, off2, l_new);
        l2 = add2(l2, l_new);
        tc_st32(s_col + 32, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(p_bar + 8 * 1);
      }
      if (nt > 0 && good) good = warp_wait(bar(B_O + a), turned++ & 1, abort_s, err, kErrTimeoutFull);
      tc_fence_after();
      if (good) {  // (the MMAs of the next unit's O follow this warp's next P)
        float l, hi;
        unpack2(l2, l, hi);
        l += hi;
        const int slot = kSplit ? unit_word(it, U_SLOT) : -1;
        float scale = pow2(unit_word(it, U_EV)), scale2 = 1.f;
        if (wide) scale = scale2 = ex2(0.5f * (static_cast<float>(unit_word(it, U_EV)) + (m_out - m)));  // in two: see the range
        else m_out = m;
        const int i = unit_word(it, U_ROW) + 256 * a + 128 * half + 32 * wq + lane, nq = unit_word(it, U_NQ);
        const int64_t q0 = unit_word(it, U_Q0);
        const int h = p.head0 + unit_word(it, U_HEAD);
        leave_unit(it);
        if (slot >= 0) {
          // a piece: this warp's rows as 32 groups of four columns, a lane's row each, then the rows' (m, l, O's unit)
          int w = 8 * half + 4 * a + wq, ln = lane;
          asm volatile("" : "+r"(w), "+r"(ln));  // (else their products are formed before the loop over units, and spilled)
          float4* to = reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(slot) * 16 + w) * kPartFloats) + ln;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            if (nt > 0) {
              tc_ld16(o_col + 16 * c, o);
              tc_wait_ld();
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = 0;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              to[32 * (4 * c + k)] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                 __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
          to[32 * (kHeadV / 4)] = make_float4(m, l, m_out, 0.f);
        } else {
          const bool none = l == 0.f;  // the row sees no token
          const float inv = scale / l;
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + ((q0 + i) * p.num_heads + h) * kHeadV);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            if (nt > 0) {
              tc_ld32(o_col + 32 * c, o);
              tc_wait_ld();
            } else {  // (undefined values would be kept from unit to unit, and spilled)
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0;
            }
            if (i < nq)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  r[e] = none ? 0u : pack_bf16(__uint_as_float(o[8 * k + 2 * e]) * inv * scale2,
                                               __uint_as_float(o[8 * k + 2 * e + 1]) * inv * scale2);
                out[4 * c + k] = make_uint4(r[0], r[1], r[2], r[3]);
              }
          }
        }
        if (slot < 0 && p.lse != nullptr && i < nq)
          p.lse[static_cast<int64_t>(h) * p.total_q + q0 + i] = natural_lse(m, l);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's arrivals, MMAs and copies are done too
  if (warp == 0) tc2_dealloc(tmem, 512);
}

// Joins the pieces of the units that were split: a warp per 32 rows and kJoinCols columns, a lane a row, the pieces in order.
// Bound by reading them, out of L2: 512 bytes a row and piece (8192 tokens x 4 heads in all: 107 us with 8 columns a warp,
// 100 with 16 or 32).
constexpr int kJoinThreads = 256, kJoinCols = 16;
__global__ void __launch_bounds__(kJoinThreads) gqa_mla_prefill_join_kernel(const MlaPrefillParams p, int pairs) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int tiles = __ldcg(p.qt_start + p.batch);
  const Split cut(p, tiles, pairs);
  if (cut.run == 0) return;
  const int tasks = tiles * p.heads * 16 * (kHeadV / kJoinCols), warps = gridDim.x * (kJoinThreads / 32);
  for (int task = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); task < tasks; task += warps) {
    const int c = task % (kHeadV / kJoinCols), rows = task / (kHeadV / kJoinCols) % 16, unit = task / (kHeadV / kJoinCols) / 16;
    const int hp = unit / tiles, qt = unit - hp * tiles;
    const int u0 = __ldcg(p.steps + qt), steps = __ldcg(p.steps + qt + 1) - u0;
    const int64_t first = hp * cut.per_head + u0;
    int pair0;
    const int pieces = cut.pieces(first, steps, pair0);
    if (pieces == 1) continue;
    const int b = find_seq(p.qt_start, p.batch, qt);
    const int2 qs = __ldcg(reinterpret_cast<const int2*>(p.q_start) + b);
    const int row0 = (qt - __ldcg(p.qt_start + b)) * kQTile + 256 * ((rows >> 2) & 1) + 128 * (rows >> 3) + 32 * (rows & 3);
    if (row0 >= qs.y) continue;
    auto part = [&](int k) { return p.part + (static_cast<int64_t>(cut.slot(first, pair0, k)) * 16 + rows) * kPartFloats; };
    auto stats = [&](int k) { return __ldcg(reinterpret_cast<const float4*>(part(k) + 32 * kHeadV) + lane); };
    float m = -INFINITY, m_out = -INFINITY, l = 0.f, o[kJoinCols];
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float4 ml = stats(k);
      if (ml.y == 0.f) continue;  // the row sees none of the piece's keys
      m = fmaxf(m, ml.x);
      m_out = fmaxf(m_out, ml.z);
    }
    const float ref = m_out == -INFINITY ? 0.f : m_out;
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float4 ml = stats(k);
      float4 v[kJoinCols / 4];
#pragma unroll
      for (int e = 0; e < kJoinCols / 4; ++e)
        v[e] = __ldcg(reinterpret_cast<const float4*>(part(k)) + 32 * (kJoinCols / 4 * c + e) + lane);
      if (ml.y == 0.f) continue;
      const float f = ex2(ml.z - ref);
      l += ex2(ml.x - m) * ml.y;
#pragma unroll
      for (int e = 0; e < kJoinCols / 4; ++e) {
        o[4 * e] += f * v[e].x;
        o[4 * e + 1] += f * v[e].y;
        o[4 * e + 2] += f * v[e].z;
        o[4 * e + 3] += f * v[e].w;
      }
    }
    int ek, ev;
    const bool wide = kv_exponents(p.amax, b, ek, ev);
    float scale = pow2(ev), scale2 = 1.f;
    if (wide) scale = scale2 = ex2(0.5f * (static_cast<float>(ev) + (m_out - m)));
    const float inv = scale / l;
    const int i = row0 + lane, h = p.head0 + hp;
    if (i >= qs.y) continue;
    const int64_t row = static_cast<int64_t>(qs.x) + i;
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (row * p.num_heads + h) * kHeadV);
#pragma unroll
    for (int k = 0; k < kJoinCols / 8; ++k) {
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = l == 0.f ? 0u : pack_bf16(o[8 * k + 2 * e] * inv * scale2, o[8 * k + 2 * e + 1] * inv * scale2);
      out[kJoinCols / 8 * c + k] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    if (c == 0 && p.lse != nullptr) p.lse[static_cast<int64_t>(h) * p.total_q + row] = natural_lse(m, l);
  }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t mla_prefill_workspace(MlaPrefillParams* p, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = base != nullptr ? base + at : nullptr;
    at += round256(bytes);
    return q;
  };
  const size_t B = static_cast<size_t>(p->batch), cap = static_cast<size_t>(p->cap);
  const int64_t per_head = static_cast<int64_t>(cap) * (kNope + kHeadV) * 2;
  int64_t hp = per_head > 0 ? kExpandBytes / per_head : p->num_heads;
  hp = hp < 1 ? 1 : (hp > p->num_heads ? p->num_heads : hp);
  p->heads_per_pass = static_cast<int>(hp);
  p->kv_len = reinterpret_cast<int*>(take(B * 4));
  p->kv_start = reinterpret_cast<int*>(take((B + 1) * 4));
  p->q_start = reinterpret_cast<int*>(take(B * 8));
  p->qt_start = reinterpret_cast<int*>(take((B + 1) * 4));
  p->amax = reinterpret_cast<unsigned*>(take((4 + 4 * B) * 4));
  p->units = reinterpret_cast<int*>(take(static_cast<size_t>(p->num_heads) * 4));
  p->valid = reinterpret_cast<unsigned*>(take(cap / 32 * 4));
  p->bad = reinterpret_cast<unsigned*>(take(cap / 32 * 4));
  p->row_top = reinterpret_cast<uint2*>(take(cap * 8));
  p->row_scale = reinterpret_cast<float2*>(take(cap * 8));
  p->lat = take(cap * kLat * 2);
  p->kr = take(cap * kRope * 2);
  p->kn = take(cap * kNope * 2 * hp);
  p->vv = take(cap * kHeadV * 2 * hp);
  if (cap >= kSplitRows) {
    p->steps = reinterpret_cast<int*>(take(512 * 4));
    p->part = reinterpret_cast<float*>(take(static_cast<size_t>(2 * kSplitPairs) * 16 * kPartFloats * 4));
  }
  return at;
}

namespace {

// Kernel that may start while the one before it ends (it waits for that one itself), over clusters of `cluster` CTAs.
template <typename... Args>
cudaError_t launch_next(void (*fn)(Args...), int cluster, dim3 grid, int threads, int smem, cudaStream_t stream,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t launch_mla_prefill(MlaPrefillParams p, int sm_count, cudaStream_t stream) {
  const int64_t q_tiles = (p.total_q + int64_t{kQTile - 1} * p.batch) / kQTile;  // at most
  p.q_tiles = static_cast<int>(q_tiles);
  const int all_pairs = sm_count / 2;
  // Whether sequences of the average lengths would be split (the plan's lengths then decide): a pass that may split but
  // does not takes 6 us longer (its own attention kernel 2 to 3, an empty join 3, the steps 1).
  auto may_split = [&](int heads) {
    const int64_t units = q_tiles * heads, n = p.cap / p.batch, nq = p.total_q / p.batch;
    const int64_t most = n / kAlign + kUnitSteps;
    const int64_t mean = most - (p.causal && nq > kQTile ? (nq - kQTile) / (2 * kAlign) : 0);
    return p.part != nullptr && units <= kSplitTiles && mean > 0 &&
           split_pays(units <= all_pairs || most > 2 * mean ? most : 2 * mean, (units * mean + all_pairs - 1) / all_pairs);
  };
  const int tail = p.num_heads % p.heads_per_pass;
  p.split = may_split(p.num_heads < p.heads_per_pass ? p.num_heads : p.heads_per_pass) || (tail != 0 && may_split(tail));
  gqa_mla_prefill_plan_kernel<<<1, 1024, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_next(gqa_mla_prefill_gather_kernel, 1, dim3(sm_count * 8), 256, 0, stream, p);
  if (e != cudaSuccess) return e;
  static std::atomic<int> ex_done[kMaxDevices], at_done[kMaxDevices], sp_done[kMaxDevices];
  e = set_smem_limit_once(ex_done, reinterpret_cast<const void*>(gqa_mla_prefill_expand_kernel), kExSmem);
  if (e != cudaSuccess) return e;
  e = set_smem_limit_once(at_done, reinterpret_cast<const void*>(gqa_mla_prefill_attn_kernel<false>), kAtSmem);
  if (e != cudaSuccess) return e;
  e = set_smem_limit_once(sp_done, reinterpret_cast<const void*>(gqa_mla_prefill_attn_kernel<true>), kAtSmem);
  if (e != cudaSuccess) return e;
  const int64_t fit = kGroupBytes / (static_cast<int64_t>(p.cap) * (kNope + kHeadV) * 2);
  p.pass = 0;
  for (int h0 = 0; h0 < p.num_heads; h0 += p.heads_per_pass, ++p.pass) {
    p.head0 = h0;
    p.heads = p.num_heads - h0 < p.heads_per_pass ? p.num_heads - h0 : p.heads_per_pass;
    const int groups = static_cast<int>(fit < 1 ? p.heads : (p.heads + fit - 1) / fit);
    p.head_group = (p.heads + groups - 1) / groups;
    ExpandMaps ex;
    AttnMaps at;
    const int64_t rows = static_cast<int64_t>(p.heads) * p.cap;
    constexpr CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kF = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!tc_encode_2d(&ex.lat, kBf, p.lat, kLat, p.cap, kLat * 2, 64, 128) ||
        !tc_encode_2d(&ex.w, kBf, p.w, kLat, static_cast<int64_t>(p.num_heads) * (kNope + kHeadV), kLat * 2, 64, 128) ||
        !tc_encode_2d(&ex.kn, kF, p.kn, kNope, rows, kNope * 2, 64, 128) ||
        !tc_encode_2d(&ex.vv, kF, p.vv, kHeadV, rows, kHeadV * 2, 64, 128) ||
        !tc_encode_2d(&at.kn, kF, p.kn, kNope, rows, kNope * 2, 64, kKTile / 2) ||
        !tc_encode_2d(&at.kr, kF, p.kr, kRope, p.cap, kRope * 2, 64, kKTile / 2))
      return cudaErrorInvalidValue;
    at.vv = ex.vv;  // the same boxes
    const int64_t q_size[3] = {kNope + kRope, p.num_heads, p.total_q}, q_pitch[2] = {2 * p.q_head_stride, 2 * p.q_token_stride};
    const int q_box[3] = {64, 1, 128};
    if (!tc_encode(&at.q, kBf, p.q, 3, q_size, q_pitch, q_box)) return cudaErrorInvalidValue;
    e = launch_next(gqa_mla_prefill_expand_kernel, 2, dim3(sm_count / 2 * 2), kExThreads, kExSmem, stream, p, ex);
    if (e != cudaSuccess) return e;
    const int64_t units = q_tiles * p.heads;
    int64_t pairs = all_pairs;
    p.split = may_split(p.heads);
    if (p.split) {
      pairs = pairs < kSplitPairs ? pairs : kSplitPairs;
      const dim3 grid(static_cast<unsigned>(2 * pairs));
      e = launch_next(gqa_mla_prefill_attn_kernel<true>, 2, grid, kAtThreads, kAtSmem, stream, p, at);
      if (e != cudaSuccess) return e;
      e = launch_next(gqa_mla_prefill_join_kernel, 1, dim3(sm_count * 4), kJoinThreads, 0, stream, p,
                      static_cast<int>(pairs));
    } else {
      const dim3 grid(static_cast<unsigned>(2 * (units < pairs ? units : pairs)));
      e = launch_next(gqa_mla_prefill_attn_kernel<false>, 2, grid, kAtThreads, kAtSmem, stream, p, at);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace gqa
