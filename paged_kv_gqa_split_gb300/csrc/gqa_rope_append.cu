// The cache's write side: one pass over a step's new tokens that turns Q and K
// by their positions, quantises (FP8 cache) and stores K and V in their pages;
// and the read side that expands FP8 rows back to bf16.
//
// FP8 rows hold, per KV head, 128 e4m3 codes and one fp32 scale. The scale
// written here is the smallest power of two that keeps the head's largest
// finite value within 448 (1 for a head of zeros): dividing by it is exact, so
// a code is one rounding of the fp32 value, and nothing is lost against
// amax / 448, because e4m3 keeps three fraction bits in every binade.
// Infinities saturate to +-448 * scale and NaN stays NaN; neither enters the
// scale, so the other values of the head keep their precision.
//
// All of it is bounded by HBM. Append: a token's 40 head rows (32 Q, 4 K, 4 V) are
// ten batches of four; a warp takes all of them, or with few tokens a share, with the
// next batch's loads in flight. A row is 128 values, four consecutive ones per lane. A
// lane's four (cos, sin) pairs are formed once and serve every Q and K row the warp
// handles (the frequencies' fixed-point fractions once per CTA); partners come from another lane by shuffle when the pairs' distance is a
// whole number of lanes, else through a row staged in shared memory. K before
// quantisation stays fp32 (not rounded to bf16 first). Measured: 16384 tokens, FP8
// cache, 56 us (5.7 TB/s), bf16 cache 60 us; 256 tokens 5.5 us; keys and values alone, 16384
// tokens, 14.4 us (FP8; a floor of 7.5) and 16.0 us (bf16; 9.9).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_plan.h"
#include "gqa_ptx.cuh"
#include "gqa_rope.cuh"

namespace gqa {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kBatch = 4;                                          // rows: a batch is all of Q, K or V
constexpr int kBatches = (kQoHeads + 2 * kKvHeads) / kBatch;       // 10: eight of Q, then K, then V
static_assert(kKvHeads == kBatch && kQoHeads % kBatch == 0, "batches of four rows");
constexpr int kF8Codes = kKvHeads * kHeadDim;           // 512
constexpr int kF8Row = kF8Codes + 4 * kKvHeads;         // 528

__device__ __forceinline__ float4 unpack_row4(uint2 v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

// A lane's four elements of the rotary window: cos and (signed) sin factors,
// y_j = x_j * c[j] + partner_j * s[j]; c = 1, s = 0 outside the window.
struct LaneTurn {
  float c[4], s[4];
};

template <int LAYOUT>
__device__ __forceinline__ int partner_of(int e, int pairs) {  // window element -> window element
  return LAYOUT == kRopeInterleaved ? (e ^ 1) : (e < pairs ? e + pairs : e - pairs);
}

template <int LAYOUT>
__device__ __forceinline__ LaneTurn lane_turn(const AppendParams& p, const unsigned long long* turns, int pos, int lane) {
  LaneTurn t;
  const int pairs = p.rot_dim >> 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * lane + j - p.rot_offset;
    t.c[j] = 1.f;
    t.s[j] = 0.f;
    if (e >= 0 && e < p.rot_dim) {
      const int i = LAYOUT == kRopeInterleaved ? e >> 1 : (e < pairs ? e : e - pairs);
      const bool second = LAYOUT == kRopeInterleaved ? (e & 1) != 0 : e >= pairs;
      const float2 v = rope_cos_sin(pos, turns[i], p.scale);
      t.c[j] = v.x;
      t.s[j] = second ? v.y : -v.y;
    }
  }
  return t;
}

// Turns one row held four elements per lane. SHUFFLE: the partner of element
// 4 lane + j is element j of another lane (half layout, distance and offset
// multiples of 4) or of this lane (interleaved, even offset).
template <int LAYOUT, bool SHUFFLE>
__device__ __forceinline__ float4 turn_row(const AppendParams& p, float4 x, const LaneTurn& t, int lane, float* row) {
  const int pairs = p.rot_dim >> 1;
  float xi[4] = {x.x, x.y, x.z, x.w}, pr[4];
  if (SHUFFLE && LAYOUT == kRopeInterleaved) {
    pr[0] = xi[1];
    pr[1] = xi[0];
    pr[2] = xi[3];
    pr[3] = xi[2];
  } else if (SHUFFLE) {
    const int e = 4 * lane - p.rot_offset;
    const int src = (e >= 0 && e < p.rot_dim) ? (partner_of<LAYOUT>(e, pairs) + p.rot_offset) >> 2 : lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) pr[j] = __shfl_sync(0xffffffffu, xi[j], src);
  } else {
    __syncwarp();
    *reinterpret_cast<float4*>(row + 4 * lane) = x;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * lane + j - p.rot_offset;
      pr[j] = (e >= 0 && e < p.rot_dim) ? row[partner_of<LAYOUT>(e, pairs) + p.rot_offset] : 0.f;
    }
  }
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * lane + j - p.rot_offset;
    y[j] = (e >= 0 && e < p.rot_dim) ? xi[j] * t.c[j] + pr[j] * t.s[j] : xi[j];
  }
  return make_float4(y[0], y[1], y[2], y[3]);
}

// |x| as ordered bits, 0 for infinities and NaN.
__device__ __forceinline__ unsigned finite_abs(float x) {
  const unsigned b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Exponent field of the smallest power of two s >= 2^-126 with amax <= 448 s
// (448 = 1.75 * 2^8), and 1 for amax = 0.
__device__ __forceinline__ unsigned scale_field(unsigned amax_bits) {
  if (amax_bits == 0) return 127;
  const int f = static_cast<int>(amax_bits >> 23) - ((amax_bits & 0x7fffffu) > 0x600000u ? 7 : 8);
  return static_cast<unsigned>(f < 1 ? 1 : f);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <int LAYOUT, bool SHUFFLE, bool FP8>
__global__ void __launch_bounds__(kAppendWarps * 32) gqa_rope_append_kernel(const AppendParams p) {
  __shared__ float stage[SHUFFLE ? 1 : kAppendWarps][SHUFFLE ? 4 : kHeadDim];
  __shared__ unsigned long long turns[kHeadDim / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (p.inv_freq != nullptr) {
    if (threadIdx.x < p.rot_dim / 2) turns[threadIdx.x] = rope_turn(__ldg(p.inv_freq + threadIdx.x));
    __syncthreads();
  }
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
  const int n = static_cast<int>(w / p.splits);
  const int part = static_cast<int>(w - static_cast<int64_t>(n) * p.splits);
  if (n >= p.num_tokens) return;
  const int first = p.q != nullptr ? 0 : kBatches - 2;  // no queries: the batches of K and V
  const int slot = __ldg(p.slots + n);
  const int count = slot >= 0 && slot < p.num_pages ? kBatches : kBatches - 2;  // not stored: the queries only
  const int b0 = first + part * (kBatches - first) / p.splits;
  const int b1 = min(first + (part + 1) * (kBatches - first) / p.splits, count);
  if (b0 >= b1) return;

  auto load = [&](int b, uint2 (&v)[kBatch]) {
    const void* from = b < kBatches - 2 ? p.q : (b == kBatches - 2 ? p.k : p.v);
    const int64_t stride = b < kBatches - 2 ? p.q_stride : (b == kBatches - 2 ? p.k_stride : p.v_stride);
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(from) + n * stride +
                                                      (b < kBatches - 2 ? b * kBatch * kHeadDim : 0)) + lane;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v[i] = __ldcs(src + i * (kHeadDim / 4));
  };
  uint2 next[kBatch];
  load(b0, next);
  const bool turned = p.inv_freq != nullptr && b0 < kBatches - 1;
  LaneTurn t;
  if (turned) t = lane_turn<LAYOUT>(p, turns, __ldg(p.positions + n), lane);
  float* row = stage[SHUFFLE ? 0 : warp];
  for (int b = b0; b < b1; ++b) {
    uint2 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v[i] = next[i];
    if (b + 1 < b1) load(b + 1, next);
    const bool is_q = b < kBatches - 2, is_k = b == kBatches - 2;
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      x[i] = unpack_row4(v[i]);
      if (turned && (is_q || is_k)) x[i] = turn_row<LAYOUT, SHUFFLE>(p, x[i], t, lane, row);
    }
    if (is_q || !FP8) {
      __nv_bfloat16* dst = is_q ? static_cast<__nv_bfloat16*>(p.q_out) + (static_cast<int64_t>(n) * kQoHeads + b * kBatch) * kHeadDim
                                : static_cast<__nv_bfloat16*>(is_k ? p.k_cache : p.v_cache) +
                                      static_cast<int64_t>(slot) * (kKvHeads * kHeadDim);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        reinterpret_cast<uint2*>(dst + i * kHeadDim)[lane] = make_uint2(pack_bf16(x[i].x, x[i].y), pack_bf16(x[i].z, x[i].w));
    } else {
      uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + static_cast<int64_t>(slot) * kF8Row;
      unsigned f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        f[i] = scale_field(__reduce_max_sync(
            0xffffffffu, max(max(finite_abs(x[i].x), finite_abs(x[i].y)), max(finite_abs(x[i].z), finite_abs(x[i].w)))));
        const float inv = __uint_as_float((254u - f[i]) << 23);
        reinterpret_cast<uint32_t*>(dst + i * kHeadDim)[lane] =
            e4m3x4(x[i].x * inv, x[i].y * inv, x[i].z * inv, x[i].w * inv);
      }
      if (lane == 0)
        *reinterpret_cast<uint4*>(dst + kF8Codes) = make_uint4(f[0] << 23, f[1] << 23, f[2] << 23, f[3] << 23);
    }
  }
}

template <int LAYOUT, bool SHUFFLE>
cudaError_t launch_append(const AppendParams& p, int grid, cudaStream_t stream) {
  if (p.fp8)
    gqa_rope_append_kernel<LAYOUT, SHUFFLE, true><<<grid, kAppendWarps * 32, 0, stream>>>(p);
  else
    gqa_rope_append_kernel<LAYOUT, SHUFFLE, false><<<grid, kAppendWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------ FP8 read back
// A warp takes four tokens, their eight rows' loads in flight together. Lane l reads
// the codes [8 l, 8 l + 8) of each half of a row (heads 0 and 1, 2 and 3) and writes
// their eight bf16 values: both sides contiguous over the warp. Measured: 262144 tokens
// 121 us (6.7 TB/s, 99 % of the measured copy rate); 777 tokens 4.5 us.
constexpr int kReadTokens = 4;
__device__ __forceinline__ uint4 dequantise8(uint2 codes, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t h2 = cvt_e4m3x2_f16x2((j < 2 ? codes.x : codes.y) >> (16 * (j & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    o[j] = pack_bf16(v.x * scale, v.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(256) gqa_kv_read_fp8_kernel(const uint8_t* __restrict__ k_cache,
                                                              const uint8_t* __restrict__ v_cache,
                                                              const int* __restrict__ indices, uint4* __restrict__ k_out,
                                                              uint4* __restrict__ v_out, int n, int num_pages) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kReadTokens;
  if (i0 >= n) return;
  int page = -1;
  if (lane < kReadTokens && i0 + lane < n) {
    page = __ldg(indices + i0 + lane);
    if (page >= num_pages) page = -1;
  }
  uint2 codes[2 * kReadTokens][2];
  float scale[2 * kReadTokens][2];
#pragma unroll
  for (int t = 0; t < kReadTokens; ++t) {
    const int pg = __shfl_sync(0xffffffffu, page, t);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        codes[2 * t + c][h] = make_uint2(0, 0);
        scale[2 * t + c][h] = 0.f;
        if (pg >= 0) {
          const uint8_t* row = (c == 0 ? k_cache : v_cache) + static_cast<int64_t>(pg) * kF8Row;
          codes[2 * t + c][h] = __ldg(reinterpret_cast<const uint2*>(row) + 32 * h + lane);
          scale[2 * t + c][h] = __ldg(reinterpret_cast<const float*>(row + kF8Codes) + 2 * h + (lane >> 4));
        }
      }
  }
#pragma unroll
  for (int t = 0; t < kReadTokens; ++t) {
    if (i0 + t >= n) break;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        ((c == 0 ? k_out : v_out) + (i0 + t) * (kF8Codes / 8))[32 * h + lane] =
            dequantise8(codes[2 * t + c][h], scale[2 * t + c][h]);
  }
}

// ------------------------------------------------------- latent cache append
// One warp per token: the 512 latent values as 16-byte vectors (two per lane),
// then the 64 rotary values, one pair per lane. 2.3 KB moved a token, bound by HBM:
// 131072 tokens 50.5 us (6.0 TB/s), 16384 tokens 9.3 us (a floor of 5.6), 256 tokens 2.7 us.
template <int LAYOUT>
__global__ void __launch_bounds__(256) gqa_mla_append_kernel(const MlaAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int stride = gridDim.x * (blockDim.x >> 5);
  const unsigned long long turn = p.inv_freq != nullptr ? rope_turn(__ldg(p.inv_freq + lane)) : 0;  // of the lane's pair
  for (int n = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); n < p.num_tokens; n += stride) {
    const int slot = __ldg(p.slots + n);
    if (slot < 0 || slot >= p.num_slots) continue;
    const uint4* lat = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.latent) + n * p.latent_stride);
    const uint4 a = __ldcs(lat + lane), b = __ldcs(lat + 32 + lane);
    const __nv_bfloat16* rope = static_cast<const __nv_bfloat16*>(p.k_rope) + n * p.rope_stride;
    const int e1 = LAYOUT == kRopeInterleaved ? 2 * lane : lane, e2 = LAYOUT == kRopeInterleaved ? e1 + 1 : lane + 32;
    float x1 = __bfloat162float(rope[e1]), x2 = __bfloat162float(rope[e2]);
    if (p.inv_freq != nullptr) {
      const float2 c = rope_cos_sin(__ldg(p.positions + n), turn, p.scale);
      const float y1 = x1 * c.x - x2 * c.y;
      x2 = x2 * c.x + x1 * c.y;
      x1 = y1;
    }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.kv_cache) + static_cast<int64_t>(slot) * 576;
    reinterpret_cast<uint4*>(dst)[lane] = a;
    reinterpret_cast<uint4*>(dst)[32 + lane] = b;
    dst[512 + e1] = __float2bfloat16_rn(x1);
    dst[512 + e2] = __float2bfloat16_rn(x2);
  }
}

}  // namespace

cudaError_t launch_rope_append(AppendParams p, int sm_count, cudaStream_t stream) {
  // a warp a token, or with few tokens more warps each: ten (a batch each), five or two, while a wave of 64 warps an
  // SM holds them
  const int64_t wave = static_cast<int64_t>(sm_count) * 64;
  const int batches = p.q != nullptr ? kBatches : 2;
  p.splits = 1;
  for (int s : {10, 5, 2})
    if (p.splits == 1 && s <= batches && p.num_tokens * static_cast<int64_t>(s) <= wave) p.splits = s;
  const int64_t warps = static_cast<int64_t>(p.num_tokens) * p.splits;
  const int grid = static_cast<int>((warps + kAppendWarps - 1) / kAppendWarps);
  const int pairs = p.rot_dim >> 1;
  if (p.layout == kRopeInterleaved)
    return (p.rot_offset & 1) == 0 ? launch_append<kRopeInterleaved, true>(p, grid, stream)
                                   : launch_append<kRopeInterleaved, false>(p, grid, stream);
  return ((p.rot_offset | pairs) & 3) == 0 ? launch_append<kRopeHalf, true>(p, grid, stream)
                                           : launch_append<kRopeHalf, false>(p, grid, stream);
}

cudaError_t launch_kv_read_fp8(const void* k_cache, const void* v_cache, const int* indices, void* k_out, void* v_out,
                               int n, int num_pages, int sm_count, cudaStream_t stream) {
  (void)sm_count;
  const int grid = (n + 8 * kReadTokens - 1) / (8 * kReadTokens);
  gqa_kv_read_fp8_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(k_cache),
                                                   static_cast<const uint8_t*>(v_cache), indices,
                                                   static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), n, num_pages);
  return cudaGetLastError();
}

cudaError_t launch_mla_append(const MlaAppendParams& p, int sm_count, cudaStream_t stream) {
  int grid = (p.num_tokens + 7) / 8;
  const int cap = sm_count * 8;
  if (grid > cap) grid = cap;
  if (p.layout == kRopeInterleaved)
    gqa_mla_append_kernel<kRopeInterleaved><<<grid, 256, 0, stream>>>(p);
  else
    gqa_mla_append_kernel<kRopeHalf><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
