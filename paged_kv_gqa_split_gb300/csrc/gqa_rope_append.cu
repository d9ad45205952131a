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
// All of it is bounded by HBM. Append: a warp takes `rows` of one token's 40
// head rows (32 Q, 4 K, 4 V); a row is 128 values, four consecutive ones per
// lane. A lane's four (cos, sin) pairs are formed once and serve every Q and K
// row the warp handles; partners come from another lane by shuffle when the
// pairs' distance is a whole number of lanes, else through a row staged in
// shared memory. K before quantisation stays fp32 (not rounded to bf16 first).
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
constexpr int kRowsPerToken = kQoHeads + 2 * kKvHeads;  // 40
constexpr int kF8Codes = kKvHeads * kHeadDim;           // 512
constexpr int kF8Row = kF8Codes + 4 * kKvHeads;         // 528

__device__ __forceinline__ float4 load_row4(const __nv_bfloat16* row, int lane) {
  const uint2 v = __ldcs(reinterpret_cast<const uint2*>(row) + lane);
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
__device__ __forceinline__ LaneTurn lane_turn(const AppendParams& p, int pos, int lane) {
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
      const float2 v = rope_cos_sin(pos, rope_turn(__ldg(p.inv_freq + i)), p.scale);
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
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
  const int n = static_cast<int>(w / p.splits);
  const int part = static_cast<int>(w - static_cast<int64_t>(n) * p.splits);
  if (n >= p.num_tokens) return;
  const int first_row = p.q != nullptr ? 0 : kQoHeads;
  const int rows = kRowsPerToken - first_row;
  const int r0 = first_row + part * rows / p.splits, r1 = first_row + (part + 1) * rows / p.splits;
  const int slot = __ldg(p.slots + n);
  const bool stored = slot >= 0 && slot < p.num_pages;
  const bool turned = p.inv_freq != nullptr && r0 < kQoHeads + kKvHeads;
  LaneTurn t;
  if (turned) t = lane_turn<LAYOUT>(p, __ldg(p.positions + n), lane);
  float* row = stage[SHUFFLE ? 0 : warp];
  for (int r = r0; r < r1; ++r) {
    const bool is_q = r < kQoHeads, is_k = !is_q && r < kQoHeads + kKvHeads;
    if (!is_q && !stored) break;
    const int h = is_q ? r : (is_k ? r - kQoHeads : r - kQoHeads - kKvHeads);
    const __nv_bfloat16* src =
        static_cast<const __nv_bfloat16*>(is_q ? p.q : (is_k ? p.k : p.v)) +
        n * (is_q ? p.q_stride : (is_k ? p.k_stride : p.v_stride)) + h * kHeadDim;
    float4 x = load_row4(src, lane);
    if (turned && (is_q || is_k)) x = turn_row<LAYOUT, SHUFFLE>(p, x, t, lane, row);
    if (is_q || !FP8) {
      __nv_bfloat16* dst = is_q ? static_cast<__nv_bfloat16*>(p.q_out) + (static_cast<int64_t>(n) * kQoHeads + h) * kHeadDim
                                : static_cast<__nv_bfloat16*>(is_k ? p.k_cache : p.v_cache) +
                                      (static_cast<int64_t>(slot) * kKvHeads + h) * kHeadDim;
      reinterpret_cast<uint2*>(dst)[lane] = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
    } else {
      const unsigned top = __reduce_max_sync(
          0xffffffffu, max(max(finite_abs(x.x), finite_abs(x.y)), max(finite_abs(x.z), finite_abs(x.w))));
      const unsigned f = scale_field(top);
      const float inv = __uint_as_float((254u - f) << 23);
      uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + static_cast<int64_t>(slot) * kF8Row;
      reinterpret_cast<uint32_t*>(dst + h * kHeadDim)[lane] = e4m3x4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
      if (lane == 0) reinterpret_cast<float*>(dst + kF8Codes)[h] = __uint_as_float(f << 23);
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
// One warp per token and cache half: lane l reads the 16 codes [16 l, 16 l + 16)
// (head l / 8) and writes their 16 bf16 values.
__global__ void __launch_bounds__(256) gqa_kv_read_fp8_kernel(const uint8_t* __restrict__ k_cache,
                                                              const uint8_t* __restrict__ v_cache,
                                                              const int* __restrict__ indices, uint4* __restrict__ k_out,
                                                              uint4* __restrict__ v_out, int n, int num_pages) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < n; i += stride) {
    const int page = __ldg(indices + i);
    const bool ok = page >= 0 && page < num_pages;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint4 codes = make_uint4(0, 0, 0, 0);
      float scale = 0.f;
      if (ok) {
        const uint8_t* row = (c == 0 ? k_cache : v_cache) + static_cast<int64_t>(page) * kF8Row;
        codes = __ldg(reinterpret_cast<const uint4*>(row) + lane);
        scale = __ldg(reinterpret_cast<const float*>(row + kF8Codes) + (lane >> 3));
      }
      const uint32_t in[4] = {codes.x, codes.y, codes.z, codes.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t h2 = cvt_e4m3x2_f16x2(in[j >> 1] >> (16 * (j & 1)));
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        o[j] = ok ? pack_bf16(v.x * scale, v.y * scale) : 0u;
      }
      uint4* dst = (c == 0 ? k_out : v_out) + i * (kF8Codes / 8) + 2 * lane;
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// ------------------------------------------------------- latent cache append
// One warp per token: the 512 latent values as 16-byte vectors (two per lane),
// then the 64 rotary values, one pair per lane.
template <int LAYOUT>
__global__ void __launch_bounds__(256) gqa_mla_append_kernel(const MlaAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int stride = gridDim.x * (blockDim.x >> 5);
  for (int n = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); n < p.num_tokens; n += stride) {
    const int slot = __ldg(p.slots + n);
    if (slot < 0 || slot >= p.num_slots) continue;
    const uint4* lat = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.latent) + n * p.latent_stride);
    const uint4 a = __ldcs(lat + lane), b = __ldcs(lat + 32 + lane);
    const __nv_bfloat16* rope = static_cast<const __nv_bfloat16*>(p.k_rope) + n * p.rope_stride;
    const int e1 = LAYOUT == kRopeInterleaved ? 2 * lane : lane, e2 = LAYOUT == kRopeInterleaved ? e1 + 1 : lane + 32;
    float x1 = __bfloat162float(rope[e1]), x2 = __bfloat162float(rope[e2]);
    if (p.inv_freq != nullptr) {
      const float2 c = rope_cos_sin(__ldg(p.positions + n), rope_turn(__ldg(p.inv_freq + lane)), p.scale);
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
  (void)sm_count;
  p.splits = 4;
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
  int grid = (n + 7) / 8;
  const int cap = sm_count * 8;
  if (grid > cap) grid = cap;
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
