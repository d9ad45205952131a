// Decode of a batch whose sequences share prefixes: what a sequence reads is its group's prefix, then its own tokens.
//   out = (sum over prefix and own tokens of 2^(s - m) v) / (the same sum of 2^(s - m))
// is formed from parts: the prefix's (computed here, once a group for all its sequences), the own tokens' (the split
// decode, kFormParts) and their join by log-sum-exp weights.
#include <cuda_runtime.h>

#include "gqa_common.cuh"
#include "gqa_kernels.h"

namespace gqa {

// Group of sequence b, or -1: the largest g with group_indptr[g] <= b, if it reaches past b.
__device__ __forceinline__ int group_of(const SharedParams& p, int b) {
  int lo = 0, hi = p.groups;  // group_indptr[lo] <= b wherever any entry is
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.group_indptr + mid) <= b) lo = mid; else hi = mid;
  }
  return p.groups > 0 && __ldg(p.group_indptr + lo) <= b && b < __ldg(p.group_indptr + lo + 1) ? lo : -1;
}

// First prefix token of group g and their count, cut to the table.
__device__ __forceinline__ int prefix_range(const SharedParams& p, int g, int& first) {
  first = max(0, min(__ldg(p.prefix_indptr + g), p.prefix_count));
  return max(0, min(__ldg(p.prefix_indptr + g + 1), p.prefix_count) - first);
}

// ----------------------------------------------------------------- prefix
// A warp per sequence and KV head: lane l holds dims 4 l .. 4 l + 3 of the 8 query heads.
__global__ void __launch_bounds__(128) gqa_shared_prefix_kernel(const SharedParams p) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    const int group = group_of(p, b);
    int first = 0;
    const int n = group < 0 ? 0 : prefix_range(p, group, first);
    float q[8][4], acc[8][4], m[8], l[8];
    const uint2* qr = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(b) * kQoHeads + g * kGroup) * kHeadDim) + lane;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const uint2 x = __ldg(qr + h * (kHeadDim / 4));
      q[h][0] = bf16_lo(x.x); q[h][1] = bf16_hi(x.x); q[h][2] = bf16_lo(x.y); q[h][3] = bf16_hi(x.y);
      acc[h][0] = acc[h][1] = acc[h][2] = acc[h][3] = 0.f;
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
    for (int t = 0; t < n; ++t) {
      const int page = __ldg(p.prefix_indices + first + t);
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) continue;
      float k[4], v[4];
      if (p.fp8) {
        const uint8_t* kr = static_cast<const uint8_t*>(p.k_cache) + static_cast<int64_t>(page) * 528;
        const uint8_t* vr = static_cast<const uint8_t*>(p.v_cache) + static_cast<int64_t>(page) * 528;
        const float sk = __ldg(reinterpret_cast<const float*>(kr + 512) + g), sv = __ldg(reinterpret_cast<const float*>(vr + 512) + g);
        const uint32_t kc = __ldg(reinterpret_cast<const uint32_t*>(kr + g * 128) + lane), vc = __ldg(reinterpret_cast<const uint32_t*>(vr + g * 128) + lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = cvt_e4m3x2_f16x2(kc >> (16 * i)), c = cvt_e4m3x2_f16x2(vc >> (16 * i));
          const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&a)), vf = __half22float2(*reinterpret_cast<const __half2*>(&c));
          k[2 * i] = kf.x * sk; k[2 * i + 1] = kf.y * sk; v[2 * i] = vf.x * sv; v[2 * i + 1] = vf.y * sv;
        }
      } else {
        const int64_t at = (static_cast<int64_t>(page) * kKvHeads + g) * kHeadDim;
        const uint2 kx = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.k_cache) + at) + lane);
        const uint2 vx = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.v_cache) + at) + lane);
        k[0] = bf16_lo(kx.x); k[1] = bf16_hi(kx.x); k[2] = bf16_lo(kx.y); k[3] = bf16_hi(kx.y);
        v[0] = bf16_lo(vx.x); v[1] = bf16_hi(vx.x); v[2] = bf16_lo(vx.y); v[3] = bf16_hi(vx.y);
      }
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        float s = q[h][0] * k[0] + q[h][1] * k[1] + q[h][2] * k[2] + q[h][3] * k[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.scale_log2;
        const float mn = fmaxf(m[h], s), sh = mn == -INFINITY ? 0.f : mn, a = ex2(m[h] - sh), w = ex2(s - sh);
        m[h] = mn;
        l[h] = l[h] * a + w;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[h][i] = acc[h][i] * a + w * v[i];
      }
    }
    float* po = p.pre_o + (static_cast<int64_t>(b) * kKvHeads + g) * (kHeadDim * kGroup);
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) po[(4 * lane + i) * kGroup + h] = acc[h][i] * inv;
      if (lane == 0) p.pre_lse[(static_cast<int64_t>(b) * kKvHeads + g) * kGroup + h] = l[h] > 0.f ? m[h] + log2f(l[h]) : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------- join
// A block per sequence and KV head, a thread per dim: the parts' running join by 2^(LSE - max).
struct Join {
  float m[8], den[8], acc[8];
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int h = 0; h < 8; ++h) m[h] = -INFINITY, den[h] = acc[h] = 0.f;
  }
  __device__ __forceinline__ void add(const float* o, const float* lse) {  // a part's row of this dim, its LSEs
    const float4 la = __ldcg(reinterpret_cast<const float4*>(lse)), lb = __ldcg(reinterpret_cast<const float4*>(lse) + 1);
    const float4 oa = __ldcg(reinterpret_cast<const float4*>(o)), ob = __ldcg(reinterpret_cast<const float4*>(o) + 1);
    const float l8[8] = {la.x, la.y, la.z, la.w, lb.x, lb.y, lb.z, lb.w}, o8[8] = {oa.x, oa.y, oa.z, oa.w, ob.x, ob.y, ob.z, ob.w};
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const float mn = fmaxf(m[h], l8[h]), sh = mn == -INFINITY ? 0.f : mn, sc = ex2(m[h] - sh), wt = ex2(l8[h] - sh);
      den[h] = den[h] * sc + wt;
      acc[h] = acc[h] * sc + wt * o8[h];
      m[h] = mn;
    }
  }
};

__global__ void __launch_bounds__(kHeadDim) gqa_shared_join_kernel(const SharedParams p) {
  const int d = threadIdx.x, g = blockIdx.x % kKvHeads;
  constexpr int kBlock = kHeadDim * kGroup;
  const int total = max(0, min(__ldg(p.kv_indptr + p.batch), p.index_count));
  for (int b = blockIdx.x / kKvHeads; b < p.batch; b += gridDim.x / kKvHeads) {
    Join j;
    j.init();
    const int64_t part = static_cast<int64_t>(b) * kKvHeads + g;
    j.add(p.pre_o + part * kBlock + d * kGroup, p.pre_lse + part * kGroup);
    const int lo = max(0, min(__ldg(p.kv_indptr + b), total)), hi = min(__ldg(p.kv_indptr + b + 1), total);
    if (hi > lo) {
      const Plan pl = make_plan(total, p.plan);
      const SeqSplit sp = seq_split(pl, lo, hi);
      const int n = static_cast<int>(sp.last_cta - sp.first_cta) + 1;
      for (int i = 0; i < n; ++i) {
        const int64_t sid = n == 1 ? p.whole_base + b : slot_id(sp.first_cta + i, i == 0 ? sp.first_slot : 0);
        const int64_t at = sid * kKvHeads + g;
        j.add(p.own_o + at * kBlock + d * kGroup, p.own_lse + at * kGroup);
      }
    }
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(b) * kQoHeads + g * kGroup) * kHeadDim + d;
#pragma unroll
    for (int h = 0; h < 8; ++h) ob[h * kHeadDim] = __float2bfloat16_rn(j.den[h] > 0.f ? j.acc[h] / j.den[h] : 0.f);
    if (p.lse != nullptr && d < kGroup) {
      float mm = j.m[0], dd = j.den[0];
#pragma unroll
      for (int h = 1; h < 8; ++h)
        if (d == h) mm = j.m[h], dd = j.den[h];
      p.lse[static_cast<int64_t>(b) * kQoHeads + g * kGroup + d] = dd > 0.f ? mm + log2f(dd) : -INFINITY;
    }
  }
}

cudaError_t launch_shared(const SharedParams& p, const DecodeParams& own, cudaStream_t stream) {
  const int grid = p.batch < (1 << 16) ? p.batch : (1 << 16);
  gqa_shared_prefix_kernel<<<grid, 128, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_decode_lsu_form(kFormParts, p.fp8 != 0, own, own.plan.tier1_ctas + own.plan.tier2_ctas, stream, kLaunchPlain);
  if (e != cudaSuccess) return e;
  gqa_shared_join_kernel<<<grid * kKvHeads, kHeadDim, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
