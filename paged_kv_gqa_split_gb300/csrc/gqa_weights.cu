// Attention weights accumulated beside the decode, and the eviction by them.
//   weights[b][j] = decay * weights[b][j] + sum over the 32 query heads of 2^(s[j] - lse)
// from the scores that the decode stored (kFormScores) and the LSE that it returned.
#include <cuda_runtime.h>

#include "gqa_common.cuh"
#include "gqa_kernels.h"
#include "gqa_select.cuh"

namespace gqa {

constexpr int kWeighThreads = 256;

__global__ void __launch_bounds__(kWeighThreads) gqa_weigh_kernel(const WeighParams p) {
  __shared__ float lse[kQoHeads];
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    __syncthreads();
    if (threadIdx.x < kQoHeads) lse[threadIdx.x] = __ldcg(p.lse + static_cast<int64_t>(b) * kQoHeads + threadIdx.x);
    __syncthreads();
    const int total = max(0, min(__ldg(p.kv_indptr + p.batch), p.index_count));
    const int lo = max(0, min(__ldg(p.kv_indptr + b), total)), n = min(__ldg(p.kv_indptr + b + 1), total) - lo;
    const int j = blockIdx.x * kWeighThreads + threadIdx.x;
    if (j >= p.width || (j >= n && p.weights == p.out)) continue;
    const int64_t at = static_cast<int64_t>(b) * p.width + j;
    if (j >= n) {
      p.out[at] = p.weights[at];
      continue;
    }
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kKvHeads; ++g) {
      const float4* s = reinterpret_cast<const float4*>(p.scores + (static_cast<int64_t>(g) * p.index_count + lo + j) * kGroup);
      const float4 x = __ldcg(s), y = __ldcg(s + 1);
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int h = 0; h < kGroup; ++h) {
        const float l = lse[g * kGroup + h];
        sum += l == -INFINITY ? 0.f : ex2(v[h] - l);
      }
    }
    p.out[at] = p.decay == 0.f ? sum : p.decay * p.weights[at] + sum;
  }
}

cudaError_t launch_weigh(const WeighParams& p, cudaStream_t stream) {
  if (p.width == 0) return cudaSuccess;
  const dim3 grid((p.width + kWeighThreads - 1) / kWeighThreads, p.batch < 65535 ? p.batch : 65535);
  gqa_weigh_kernel<<<grid, kWeighThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// --------------------------------------------------------------- eviction
// A block per sequence. Of more than `budget` tokens the first keep_first and the last keep_last stay, and of those
// between them the heaviest; the sequence's share of the new lists begins where the sequences before it end, which every
// block sums up by itself.
constexpr int kEvictThreads = 1024;

__global__ void __launch_bounds__(kEvictThreads) gqa_evict_kernel(const EvictParams p) {
  __shared__ SelectSpace<kEvictThreads> sp;
  const int tid = threadIdx.x;
  auto length = [&](int b, int& lo) {
    lo = max(0, min(__ldg(p.kv_indptr + b), p.index_count));
    return max(0, min(__ldg(p.kv_indptr + b + 1), p.index_count) - lo);
  };
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    int before = 0, before_all = 0, lo = 0;
    for (int i = tid; i < b; i += kEvictThreads) {
      const int n = length(i, lo);
      before += min(n, p.budget);
      before_all += n;
    }
    before = block_sum(sp, before);
    before_all = block_sum(sp, before_all);
    const int n = length(b, lo), keep = min(n, p.budget);
    int gone = before_all - before;
    if (tid == 0) {
      if (b == 0) p.new_indptr[0] = p.freed_indptr[0] = 0;
      p.new_indptr[b + 1] = before + keep;
      p.freed_indptr[b + 1] = gone + n - keep;
    }
    const float* w = p.weights + static_cast<int64_t>(b) * p.width;
    float* wo = p.weights_out + static_cast<int64_t>(b) * p.width;
    const int mid_lo = min(p.keep_first, n), mid_hi = max(n - p.keep_last, mid_lo);
    auto weight = [&](int j) { return j < p.width ? w[j] : 0.f; };
    auto key = [&](int j) { return ordered_bits(weight(j)); };
    const int take = keep - (n - (mid_hi - mid_lo));  // of the middle
    uint32_t least = 0;
    int ties = 0;
    if (n > p.budget && take > 0) {
      int above = 0;
      least = block_kth<kEvictThreads, uint32_t>(sp, mid_hi - mid_lo, take, [](int) { return true; },
                                                 [&](int i) { return key(mid_lo + i); }, above);
      ties = take - above;
    }
    int at = 0;  // kept so far
    for (int j0 = 0; j0 < n; j0 += kEvictThreads) {
      const int j = j0 + tid;
      bool stay = j < n, tie = false;
      if (j < n && n > p.budget && j >= mid_lo && j < mid_hi) {
        const uint32_t x = key(j);
        tie = take > 0 && x == least;
        stay = take > 0 && x > least;
      }
      int tied, kept;
      const int tie_rank = block_rank(sp, tie, tied);
      stay = stay || (tie && tie_rank < ties);
      ties -= min(ties, tied);
      const int rank = block_rank(sp, stay, kept);
      if (j < n) {
        const int page = __ldg(p.kv_indices + lo + j);
        if (stay) {
          if (before + at + rank < p.index_count) p.new_indices[before + at + rank] = page;  // offsets that decrease
          if (at + rank < p.width) wo[at + rank] = weight(j);
        } else {
          if (gone + j - (at + rank) < p.index_count) p.freed[gone + j - (at + rank)] = page;
        }
      }
      at += kept;
    }
    for (int j = keep + tid; j < p.width; j += kEvictThreads) wo[j] = 0.f;
    if (b == p.batch - 1) {  // behind the last sequence's
      for (int i = before + keep + tid; i < p.index_count; i += kEvictThreads) p.new_indices[i] = -1;
      for (int i = gone + n - keep + tid; i < p.index_count; i += kEvictThreads) p.freed[i] = -1;
    }
  }
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  gqa_evict_kernel<<<p.batch < (1 << 16) ? p.batch : (1 << 16), kEvictThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
