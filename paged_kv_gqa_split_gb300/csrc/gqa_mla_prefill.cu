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
// value in [2^10, 2^11); keys and values have one exponent each, from the bound
// 512 * max|c| * max|W| (and the rotary keys). The maxima are taken over finite
// values, so an infinity stays with its row: a token whose latent is not all
// finite gets NaN keys and zero values, which makes the rows that see it NaN
// and, a weight of 0 times 0 being 0, no others.
// Scores, softmax statistics and outputs accumulate in fp32.
//
// Steps, each a kernel: the plan (prefix sums over the sequences), the gather
// (paged rows to packed rows, 128-aligned per sequence and zero-filled, and the
// maxima), the expansion, the attention. Tensor-core bound.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_ptx.cuh"

namespace gqa {
namespace {

constexpr int kLat = 512, kNope = 128, kRope = 64, kHeadV = 128, kRow = kLat + kRope, kDqk = kNope + kRope;
constexpr int kAlign = 128;    // packed rows of a sequence start at a multiple of this
constexpr int kQTile = 64;    // query rows a CTA takes
constexpr int64_t kExpandBytes = int64_t{1} << 30;  // expanded keys and values of one pass over the heads

// ------------------------------------------------------------------- plan
// One block: lengths clamped to the table, packed starts, query tiles. Prefix
// sums run over chunks of 1024 sequences.
__global__ void __launch_bounds__(1024) gqa_mla_prefill_plan_kernel(const MlaPrefillParams p) {
  __shared__ int64_t sk[1024];
  __shared__ int sq[1024];
  __shared__ int64_t base_k;
  __shared__ int base_q;
  const int tid = threadIdx.x;
  if (tid < 4) p.amax[tid] = 0;
  if (tid == 0) {
    base_k = 0;
    base_q = 0;
  }
  const int64_t table = static_cast<int64_t>(p.width) * p.page_size;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + tid;
    int len = 0, tiles = 0, qs = 0;
    if (b < p.batch) {
      // a malformed cu_q never makes a row out of range: entries are clamped to
      // [0, total_q], and a decreasing pair counts as an empty sequence
      qs = min(max(__ldg(p.cu_q + b), 0), p.total_q);
      const int qe = min(max(__ldg(p.cu_q + b + 1), 0), p.total_q);
      if (__ldg(p.cu_q + b + 1) < __ldg(p.cu_q + b) || __ldg(p.cu_q + b) < 0 || __ldg(p.cu_q + b + 1) > p.total_q)
        atomicOr(p.err, kErrBadIndptr);
      const int nq = max(qe - qs, 0);
      tiles = (nq + kQTile - 1) / kQTile;
      if (nq > 0) len = static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.cache_seqlens + b), 0)), table));
      p.q_start[2 * b] = qs;
      p.q_start[2 * b + 1] = nq;
    }
    sk[tid] = (static_cast<int64_t>(len) + kAlign - 1) / kAlign * kAlign;
    sq[tid] = tiles;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      const int64_t vk = tid >= o ? sk[tid - o] : 0;
      const int vq = tid >= o ? sq[tid - o] : 0;
      __syncthreads();
      sk[tid] += vk;
      sq[tid] += vq;
      __syncthreads();
    }
    if (b < p.batch) {
      const int64_t end = base_k + sk[tid];
      const int64_t start = end - (static_cast<int64_t>(len) + kAlign - 1) / kAlign * kAlign;
      if (end > p.cap) {  // more tokens than the caller's bound: these sequences see no key
        atomicOr(p.err, kErrKvBound);
        len = 0;
      }
      p.kv_len[b] = len;
      p.kv_start[b] = static_cast<int>(min(start, static_cast<int64_t>(p.cap)));
      p.qt_start[b] = base_q + sq[tid] - tiles;
    }
    __syncthreads();
    if (tid == 0) {
      base_k += sk[1023];
      base_q += sq[1023];
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.kv_start[p.batch] = static_cast<int>(min(base_k, static_cast<int64_t>(p.cap)));
    p.qt_start[p.batch] = base_q;
  }
}

// Largest b in [0, batch) with start[b] <= x (start[0] = 0).
__device__ __forceinline__ int find_seq(const int* start, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(start + mid) <= x) lo = mid; else hi = mid;
  }
  return lo;
}

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

// ----------------------------------------------------------------- gather
// A warp per packed row (rows [0, cap) in turn, 32 rows a block), then a warp
// per weight row.
__global__ void __launch_bounds__(256) gqa_mla_prefill_gather_kernel(const MlaPrefillParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int total = __ldg(p.kv_start + p.batch);
  const int groups = total / 32;  // 32 packed rows share a word of valid bits and a sequence
  unsigned top_c = 0, top_r = 0, top_k = 0, top_v = 0;
  __shared__ unsigned bad_s;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    if (threadIdx.x == 0) bad_s = 0;
    __syncthreads();
    // the last sequence that starts at or before the row (empty ones start where the next does)
    const int b = find_seq(p.kv_start, p.batch, 32 * g);
    const int t0 = 32 * g - __ldg(p.kv_start + b), n = __ldg(p.kv_len + b);
    if (warp == 0) {
      const int t = t0 + lane;
      bool ok = false;
      if (t < n) {
        const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.width + t / p.page_size);
        ok = blk >= 0 && blk < p.num_blocks;
      }
      const unsigned m = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) p.valid[g] = m;
    }
    for (int i = warp; i < 32; i += 8) {
      const int t = t0 + i;
      const uint4* src = nullptr;
      if (t < n) {
        const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.width + t / p.page_size);
        if (blk >= 0 && blk < p.num_blocks)
          src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.kv) +
                                               (static_cast<int64_t>(blk) * p.page_size + t % p.page_size) * kRow);
      }
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 a = src ? __ldg(src + lane) : zero, c = src ? __ldg(src + 32 + lane) : zero;
      const uint4 r = src && lane < 8 ? __ldg(src + 64 + lane) : zero;
      uint4* lat = reinterpret_cast<uint4*>(p.lat) + static_cast<int64_t>(32 * g + i) * (kLat / 8);
      lat[lane] = a;
      lat[32 + lane] = c;
      if (lane < 8) reinterpret_cast<uint4*>(p.kr)[static_cast<int64_t>(32 * g + i) * (kRope / 8) + lane] = r;
      top_c = finite_bits(c, finite_bits(a, top_c));
      top_r = finite_bits(r, top_r);
      if (__any_sync(0xffffffffu, not_finite(a) || not_finite(c)) && lane == 0) atomicOr(&bad_s, 1u << i);
    }
    __syncthreads();
    if (threadIdx.x == 0) p.bad[g] = bad_s;
  }
  const int wrows = p.num_heads * (kNope + kHeadV);
  for (int r = blockIdx.x * 8 + warp; r < wrows; r += gridDim.x * 8) {
    const uint4* src = reinterpret_cast<const uint4*>(p.w) + static_cast<int64_t>(r) * (kLat / 8);
    const unsigned t = finite_bits(__ldg(src + 32 + lane), finite_bits(__ldg(src + lane), 0));
    if ((r & 255) < kNope) top_k = max(top_k, t); else top_v = max(top_v, t);
  }
  const unsigned top[4] = {top_c, top_r, top_k, top_v};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a maximum of integers: the order of the atomics does not matter
    const unsigned m = __reduce_max_sync(0xffffffffu, top[i]);
    if (lane == 0 && m != 0) atomicMax(p.amax + i, m);
  }
}

// Exponents that bring keys and values into fp16 (value * 2^-e):
// |c . w| <= 512 max|c| max|w| < 2^(Ec + 1 + Ew + 1 + 9), to be below 2^15.
__device__ __forceinline__ int exponent_of(unsigned bits) { return static_cast<int>(bits >> 23) - 127; }
__device__ __forceinline__ void kv_exponents(const unsigned* amax, int& ek, int& ev) {
  const unsigned c = __ldg(amax), r = __ldg(amax + 1), wk = __ldg(amax + 2), wv = __ldg(amax + 3);
  ek = r != 0 ? exponent_of(r) + 1 - 15 : -126;
  if (c != 0 && wk != 0) ek = max(ek, exponent_of(c) + exponent_of(wk) + 11 - 15);
  ev = c != 0 && wv != 0 ? exponent_of(c) + exponent_of(wv) + 11 - 15 : 0;
  ek = min(max(ek, -126), 126);
  ev = min(max(ev, -126), 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }

__device__ __forceinline__ uint32_t sw128(uint32_t base, int r, int c) { return base + r * 128 + ((c ^ (r & 7)) << 4); }

// -------------------------------------------------------------- expansion
// [128 packed rows x 512] x W[h]^T [512 x 128 columns] on mma.sync; column
// block 0 gives the head's keys, 1 its values. Block column 2 of head 0 turns
// the rotary keys into scaled fp16.
constexpr int kExBM = 128, kExStage = (kExBM + 128) * 128;
__global__ void __launch_bounds__(256) gqa_mla_prefill_expand_kernel(const MlaPrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp >> 2, wn = warp & 3;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kExBM;
  if (m0 >= __ldg(p.kv_start + p.batch)) return;
  const int part = blockIdx.y & 1, hp = blockIdx.y >> 1;
  int ek, ev;
  kv_exponents(p.amax, ek, ev);
  if (hp >= p.heads) {  // the last block column: rotary keys, once (the first pass over the heads)
    if (part != 0 || p.head0 != 0) return;
    uint32_t* kr = static_cast<uint32_t*>(p.kr) + m0 * (kRope / 2);
    const float f = pow2(-ek);
    for (int i = tid; i < kExBM * kRope / 2; i += 256) {
      const uint32_t v = kr[i];
      kr[i] = pack_f16(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
    }
    return;
  }
  const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.lat) + m0 * kLat;
  const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(p.w) + (static_cast<int64_t>(p.head0 + hp) * 256 + part * 128) * kLat;
  auto load = [&](int ck) {
    const uint32_t as = sb + (ck % 3) * kExStage, bs = as + kExBM * 128;
    for (int i = tid; i < 128 * 8; i += 256) {
      const int r = i >> 3, c = i & 7;
      cp_async_16(sw128(as, r, c), a + static_cast<int64_t>(r) * kLat + ck * 64 + c * 8, 16u);
      cp_async_16(sw128(bs, r, c), b + static_cast<int64_t>(r) * kLat + ck * 64 + c * 8, 16u);
    }
  };
  float acc[4][4][4] = {};
  load(0);
  cp_async_commit();
  load(1);
  cp_async_commit();
  for (int ck = 0; ck < 8; ++ck) {
    cp_async_wait<1>();
    __syncthreads();
    if (ck + 2 < 8) load(ck + 2);
    cp_async_commit();
    const uint32_t as = sb + (ck % 3) * kExStage, bs = as + kExBM * 128;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t af[4][4];
#pragma unroll
      for (int mi = 0; mi < 4; ++mi)
        ldsm_x4(sw128(as, (wm * 4 + mi) * 16 + (lane & 15), 2 * kk + (lane >> 4)), af[mi][0], af[mi][1], af[mi][2], af[mi][3]);
#pragma unroll
      for (int nj = 0; nj < 4; nj += 2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(sw128(bs, wn * 32 + nj * 8 + ((lane >> 4) << 3) + (lane & 7), 2 * kk + ((lane >> 3) & 1)), b0, b1, b2, b3);
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) {
          mma_bf16_16816(acc[mi][nj], af[mi][0], af[mi][1], af[mi][2], af[mi][3], b0, b1);
          mma_bf16_16816(acc[mi][nj + 1], af[mi][0], af[mi][1], af[mi][2], af[mi][3], b2, b3);
        }
      }
    }
  }
  const float f = pow2(part == 0 ? -ek : -ev);
  __half* o = static_cast<__half*>(part == 0 ? p.kn : p.vv) + (static_cast<int64_t>(hp) * p.cap + m0) * 128;
#pragma unroll
  for (int mi = 0; mi < 4; ++mi)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = (wm * 4 + mi) * 16 + (lane >> 2) + 8 * half;
      const bool bad = ((__ldg(p.bad + (m0 >> 5) + (r >> 5)) >> (r & 31)) & 1u) != 0;
#pragma unroll
      for (int nj = 0; nj < 4; ++nj)
        *reinterpret_cast<uint32_t*>(o + r * 128 + wn * 32 + nj * 8 + 2 * (lane & 3)) =
            bad ? (part == 0 ? 0x7fff7fffu : 0u) : pack_f16(acc[mi][nj][2 * half] * f, acc[mi][nj][2 * half + 1] * f);
    }
}

// -------------------------------------------------------------- attention
// 64 query rows of one head a CTA, 16 a warp; tiles of 64 keys, two in flight.
constexpr int kKTile = 64;
constexpr int kQBytes = kQTile * kDqk * 2, kKBytes = kKTile * kDqk * 2, kVBytes = kKTile * kHeadV * 2;
constexpr int kAttnSmem = kQBytes + 2 * (kKBytes + kVBytes) + kQTile * 4;
__global__ void __launch_bounds__(128) gqa_mla_prefill_attn_kernel(const MlaPrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  float* rowfac = reinterpret_cast<float*>(smem + kQBytes + 2 * (kKBytes + kVBytes));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qt = blockIdx.x, hp = blockIdx.y, h = p.head0 + hp;
  if (qt >= __ldg(p.qt_start + p.batch)) return;
  const int b = find_seq(p.qt_start, p.batch, qt);
  const int nq = __ldg(p.q_start + 2 * b + 1), i0 = (qt - __ldg(p.qt_start + b)) * kQTile;
  const int64_t q0 = __ldg(p.q_start + 2 * b);
  const int n = __ldg(p.kv_len + b), kv0 = __ldg(p.kv_start + b);
  // the sequence's own length places the queries (n may be cut by the table or the bound)
  const int seq_n = n;
  const int last = p.causal ? min(n, seq_n - nq + min(i0 + kQTile, nq)) : n;  // keys any row of the tile sees
  const int ntiles = last > 0 ? (last + kKTile - 1) / kKTile : 0;

  // queries to fp16, each row brought to a largest value in [2^10, 2^11)
  for (int r = warp * 16; r < warp * 16 + 16; ++r) {
    uint32_t v[3];
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      v[j] = i0 + r < nq ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                   (q0 + i0 + r) * p.q_token_stride + h * p.q_head_stride) +
                                 32 * j + lane)
                         : 0u;
      top = finite_bits2(v[j], top);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = top != 0 ? max(exponent_of(top), -116) - 10 : 0;
    if (lane == 0) rowfac[r] = pow2(max(e, -126));
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const float f = pow2(min(-e, 127));
      const uint32_t h2 = pack_f16(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sw128(sb + j * (kQTile * 128), r, lane >> 2) + (lane & 3) * 4), "r"(h2)
                   : "memory");
    }
  }
  const __half* kn = static_cast<const __half*>(p.kn) + (static_cast<int64_t>(hp) * p.cap + kv0) * 128;
  const __half* vv = static_cast<const __half*>(p.vv) + (static_cast<int64_t>(hp) * p.cap + kv0) * 128;
  const __half* kr = static_cast<const __half*>(p.kr) + static_cast<int64_t>(kv0) * kRope;
  auto load = [&](int j) {
    const uint32_t ks = sb + kQBytes + (j & 1) * (kKBytes + kVBytes), vs = ks + kKBytes;
    for (int i = tid; i < kKTile * 16; i += 128) {
      const int r = i >> 4, c = i & 15;
      const int64_t t = static_cast<int64_t>(j) * kKTile + r;
      cp_async_16(sw128(ks + (c >> 3) * (kKTile * 128), r, c & 7), kn + t * 128 + c * 8, 16u);
      cp_async_16(sw128(vs + (c >> 3) * (kKTile * 128), r, c & 7), vv + t * 128 + c * 8, 16u);
    }
    for (int i = tid; i < kKTile * 8; i += 128) {
      const int r = i >> 3, c = i & 7;
      cp_async_16(sw128(ks + 2 * (kKTile * 128), r, c), kr + (static_cast<int64_t>(j) * kKTile + r) * kRope + c * 8, 16u);
    }
  };
  float o[16][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  __syncthreads();
  int ek, ev;
  kv_exponents(p.amax, ek, ev);
  float sc[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) sc[half] = rowfac[warp * 16 + (lane >> 2) + 8 * half] * p.scale_log2 * pow2(ek);
  if (ntiles > 0) load(0);
  cp_async_commit();
  for (int j = 0; j < ntiles; ++j) {
    if (j + 1 < ntiles) load(j + 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t ks = sb + kQBytes + (j & 1) * (kKBytes + kVBytes), vs = ks + kKBytes;
    float s[8][4] = {};
#pragma unroll
    for (int kk = 0; kk < 12; ++kk) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4(sw128(sb + (kk >> 2) * (kQTile * 128), warp * 16 + (lane & 15), 2 * (kk & 3) + (lane >> 4)), a0, a1, a2, a3);
#pragma unroll
      for (int nj = 0; nj < 8; nj += 2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(sw128(ks + (kk >> 2) * (kKTile * 128), nj * 8 + ((lane >> 4) << 3) + (lane & 7), 2 * (kk & 3) + ((lane >> 3) & 1)),
                b0, b1, b2, b3);
        mma_f16_16816(s[nj], a0, a1, a2, a3, b0, b1);
        mma_f16_16816(s[nj + 1], a0, a1, a2, a3, b2, b3);
      }
    }
    const unsigned v0 = __ldg(p.valid + (kv0 >> 5) + 2 * j), v1 = __ldg(p.valid + (kv0 >> 5) + 2 * j + 1);
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int nj = 0; nj < 8; ++nj)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = nj * 8 + 2 * (lane & 3) + (e & 1), half = e >> 1;
        const int t = j * kKTile + col, i = i0 + warp * 16 + (lane >> 2) + 8 * half;
        const bool ok = (((col < 32 ? v0 : v1) >> (col & 31)) & 1u) != 0 && (!p.causal || t <= seq_n - nq + i);
        s[nj][e] = ok ? s[nj][e] * sc[half] : -INFINITY;
        mx[half] = fmaxf(mx[half], s[nj][e]);
      }
    float fix[2], base[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 2));
      fix[half] = mx[half] == -INFINITY ? 1.f : ex2(m[half] - mx[half]);
      // probabilities are held times 2^14, so that small ones stay fp16 normals
      base[half] = mx[half] == -INFINITY ? 0.f : 14.f - mx[half];
      m[half] = mx[half];
      l[half] *= fix[half];
    }
#pragma unroll
    for (int nd = 0; nd < 16; ++nd) {
      o[nd][0] *= fix[0];
      o[nd][1] *= fix[0];
      o[nd][2] *= fix[1];
      o[nd][3] *= fix[1];
    }
#pragma unroll
    for (int nj = 0; nj < 8; ++nj)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[nj][e] = ex2(s[nj][e] + base[e >> 1]);
        l[e >> 1] += s[nj][e];
      }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t a0 = pack_f16(s[2 * kk][0], s[2 * kk][1]), a1 = pack_f16(s[2 * kk][2], s[2 * kk][3]);
      const uint32_t a2 = pack_f16(s[2 * kk + 1][0], s[2 * kk + 1][1]), a3 = pack_f16(s[2 * kk + 1][2], s[2 * kk + 1][3]);
#pragma unroll
      for (int nd = 0; nd < 16; nd += 2) {
        uint32_t b0, b1, b2, b3;
        const int c = nd + (lane >> 4);
        ldsm_x4_trans(sw128(vs + (c >> 3) * (kKTile * 128), kk * 16 + (lane & 15), c & 7), b0, b1, b2, b3);
        mma_f16_16816(o[nd], a0, a1, a2, a3, b0, b1);
        mma_f16_16816(o[nd + 1], a0, a1, a2, a3, b2, b3);
      }
    }
    __syncthreads();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    const int i = i0 + warp * 16 + (lane >> 2) + 8 * half;
    if (i >= nq) continue;
    const bool none = l[half] == 0.f;  // the row sees no token
    const float inv = pow2(ev) / l[half];
    __nv_bfloat16* row = static_cast<__nv_bfloat16*>(p.out) + ((q0 + i) * p.num_heads + h) * kHeadV;
#pragma unroll
    for (int nd = 0; nd < 16; ++nd)
      *reinterpret_cast<uint32_t*>(row + nd * 8 + 2 * (lane & 3)) =
          none ? 0u : pack_bf16(o[nd][2 * half] * inv, o[nd][2 * half + 1] * inv);
    if (p.lse != nullptr && (lane & 3) == 0)
      p.lse[static_cast<int64_t>(h) * p.total_q + q0 + i] =
          none ? -INFINITY : (m[half] - 14.f + log2f(l[half])) * 0.6931471805599453f;
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
  p->amax = reinterpret_cast<unsigned*>(take(16));
  p->valid = reinterpret_cast<unsigned*>(take(cap / 32 * 4));
  p->bad = reinterpret_cast<unsigned*>(take(cap / 32 * 4));
  p->lat = take(cap * kLat * 2);
  p->kr = take(cap * kRope * 2);
  p->kn = take(cap * kNope * 2 * hp);
  p->vv = take(cap * kHeadV * 2 * hp);
  return at;
}

cudaError_t launch_mla_prefill(MlaPrefillParams p, int sm_count, cudaStream_t stream) {
  gqa_mla_prefill_plan_kernel<<<1, 1024, 0, stream>>>(p);
  gqa_mla_prefill_gather_kernel<<<sm_count * 8, 256, 0, stream>>>(p);
  static std::atomic<int> ex_done[kMaxDevices], at_done[kMaxDevices];
  cudaError_t e = set_smem_limit_once(ex_done, reinterpret_cast<const void*>(gqa_mla_prefill_expand_kernel), 3 * kExStage);
  if (e != cudaSuccess) return e;
  e = set_smem_limit_once(at_done, reinterpret_cast<const void*>(gqa_mla_prefill_attn_kernel), kAttnSmem);
  if (e != cudaSuccess) return e;
  const int q_tiles = p.total_q / kQTile + p.batch;
  for (int h0 = 0; h0 < p.num_heads; h0 += p.heads_per_pass) {
    p.head0 = h0;
    p.heads = p.num_heads - h0 < p.heads_per_pass ? p.num_heads - h0 : p.heads_per_pass;
    gqa_mla_prefill_expand_kernel<<<dim3(p.cap / kExBM, 2 * p.heads + 1), 256, 3 * kExStage, stream>>>(p);
    gqa_mla_prefill_attn_kernel<<<dim3(q_tiles, p.heads), 128, kAttnSmem, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gqa
