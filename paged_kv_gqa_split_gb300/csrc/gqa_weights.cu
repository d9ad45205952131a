// Attention weights accumulated beside the decode, and the eviction by them.
//   weights[b][j] = decay * weights[b][j] + sum over the 32 query heads of 2^(s[j] - lse)
// from the scores that the decode stored (kFormScores) and the LSE that it returned. Bound by the launch and the round trips
// of loads; the scores (128 bytes a token) come from L2 and are read while the merge runs (6019 tokens of 16 sequences, the
// whole call: 20.8 us; behind the merge: 22.8).
#include <cuda_runtime.h>

#include "gqa_common.cuh"
#include "gqa_kernels.h"
#include "gqa_select.cuh"

namespace gqa {

constexpr int kWeighThreads = 256;

__global__ void __launch_bounds__(kWeighThreads) gqa_weigh_kernel(const WeighParams p) {
  __shared__ float lse[kQoHeads];
  bool waited = false;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    // ahead of the wait: the call's inputs, and the scores, which the merge let this kernel start behind
    const int total = max(0, min(__ldcg(p.kv_indptr + p.batch), p.index_count));
    const int lo = max(0, min(__ldcg(p.kv_indptr + b), total)), n = min(__ldcg(p.kv_indptr + b + 1), total) - lo;
    const int j = blockIdx.x * kWeighThreads + threadIdx.x;
    const int64_t at = static_cast<int64_t>(b) * p.width + j;
    const bool in = j < p.width, add = in && j < n;
    float4 s[2 * kKvHeads];
    if (add) {
#pragma unroll
      for (int g = 0; g < kKvHeads; ++g) {
        const float4* from = reinterpret_cast<const float4*>(p.scores + (static_cast<int64_t>(g) * p.index_count + lo + j) * kGroup);
        s[2 * g] = __ldcg(from);
        s[2 * g + 1] = __ldcg(from + 1);
      }
    }
    const float old = in && !(add && p.decay == 0.f) ? __ldcg(p.weights + at) : 0.f;
    if (!waited) {
      pdl_wait();
      pdl_launch_dependents();
      waited = true;
    }
    __syncthreads();
    if (threadIdx.x < kQoHeads) lse[threadIdx.x] = __ldcg(p.lse + static_cast<int64_t>(b) * kQoHeads + threadIdx.x);
    __syncthreads();
    if (add) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * kKvHeads; ++k) {
        const float v[4] = {s[k].x, s[k].y, s[k].z, s[k].w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float l = lse[4 * k + h];
          sum += v[h] == -INFINITY ? 0.f : ex2(v[h] - l);  // 0: left out, where l may be -inf or NaN
        }
      }
      p.out[at] = p.decay == 0.f ? sum : p.decay * old + sum;
    } else if (in && p.weights != p.out) {
      p.out[at] = old;
    }
  }
}

cudaError_t launch_weigh(const WeighParams& p, cudaStream_t stream) {
  if (p.width == 0) return cudaSuccess;
  const dim3 grid((p.width + kWeighThreads - 1) / kWeighThreads, p.batch < 65535 ? p.batch : 65535);
  return launch_chained(gqa_weigh_kernel, grid, kWeighThreads, 0, stream, 1, p);
}

// --------------------------------------------------------------- eviction
// A cluster of blocks per sequence, each with an equal run of its tokens. Of more than `budget` tokens the first
// keep_first and the last keep_last stay, and of those between them the heaviest; the sequence's share of the new lists
// begins where the sequences before it end, which every block sums up by itself, or for many sequences a kernel ahead for
// all of them. The weights are read once into shared memory as ordered words (from global memory each time where a run does
// not fit).
constexpr int kEvictHeld = 48 * 1024;   // words of shared memory at most
constexpr int kEvictRun = 4 * 1024;     // tokens a block of a cluster at least
constexpr int kEvictAlone = 1024;       // sequences that every block sums up by itself
static_assert(kMostBlocks == 16, "evict_us goes up to 16 blocks a cluster");
constexpr uint32_t kStays = 1, kGoes = 0;  // marks below any key

// Tokens of sequence b, as far as the indices reach, and where they begin.
__device__ __forceinline__ int evict_length(const EvictParams& p, int b, int& lo) {
  lo = max(0, min(__ldcg(p.kv_indptr + b), p.index_count));
  return max(0, min(__ldcg(p.kv_indptr + b + 1), p.index_count) - lo);
}

// Both new offsets of every sequence: prefix sums by one block, 8192 sequences at a time. Sequences of 20 tokens cut to 10 with
// this kernel, and with each block of the eviction summing up by itself: 300: 12.2 us and 10.1, 1024: 29.5 and 29.8, 4096: 97 and
// 106, 20000: 450 and 701, 65536: 1460 and 3900.
constexpr int kSumThreads = 1024, kSumEach = 8;

__global__ void __launch_bounds__(kSumThreads) gqa_evict_sums_kernel(const EvictParams p) {
  __shared__ int2 warp_sum[kSumThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  int2 base = make_int2(0, 0);  // tokens kept and freed before these sequences
  if (tid == 0) p.new_indptr[0] = p.freed_indptr[0] = 0;
  for (int64_t b0 = 0; b0 < p.batch; b0 += kSumThreads * kSumEach) {
    const int64_t first = b0 + tid * kSumEach;
    int2 each[kSumEach], sum = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kSumEach; ++i) {
      int lo, n = first + i < p.batch ? evict_length(p, static_cast<int>(first) + i, lo) : 0;
      sum.x += min(n, p.budget);
      sum.y += n - min(n, p.budget);
      each[i] = sum;
    }
    int2 upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto.x, o), y = __shfl_up_sync(0xffffffffu, upto.y, o);
      if (lane >= o) upto.x += x, upto.y += y;
    }
    __syncthreads();  // (the sums of the sequences before have been read)
    if (lane == 31) warp_sum[tid >> 5] = upto;
    __syncthreads();
    const int2 w = warp_sum[lane];
    const bool ahead = lane < (tid >> 5);
    const int2 from = make_int2(base.x + upto.x - sum.x + __reduce_add_sync(0xffffffffu, ahead ? w.x : 0),
                                base.y + upto.y - sum.y + __reduce_add_sync(0xffffffffu, ahead ? w.y : 0));
#pragma unroll
    for (int i = 0; i < kSumEach; ++i) {
      if (first + i < p.batch) {
        p.new_indptr[first + i + 1] = from.x + each[i].x;
        p.freed_indptr[first + i + 1] = from.y + each[i].y;
      }
    }
    base.x += __reduce_add_sync(0xffffffffu, w.x);
    base.y += __reduce_add_sync(0xffffffffu, w.y);
  }
}

template <bool CLUSTERED, int THREADS>
__global__ void __launch_bounds__(THREADS) gqa_evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t held[];
  __shared__ SelectSpace<THREADS> sp;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int blocks = p.cluster, rank = CLUSTERED ? static_cast<int>(blockIdx.x) % blocks : 0;
  for (int b = blockIdx.x / blocks; b < p.batch; b += gridDim.x / blocks) {
    int lo = 0, before, gone;  // tokens kept and freed of the sequences before this one
    int2 all;                  // of all sequences
    if (p.sums) {
      before = __ldcg(p.new_indptr + b);
      gone = __ldcg(p.freed_indptr + b);
      all = make_int2(__ldcg(p.new_indptr + p.batch), __ldcg(p.freed_indptr + p.batch));
    } else {
      int2 ahead = make_int2(0, 0);
      all = make_int2(0, 0);
      for (int i = tid; i < p.batch; i += THREADS) {
        const int n = evict_length(p, i, lo), kept = min(n, p.budget);
        all.x += kept;
        all.y += n - kept;
        if (i < b) ahead.x += kept, ahead.y += n - kept;
      }
      ahead = block_sum2<THREADS>(sp.sums, ahead);
      all = block_sum2<THREADS>(sp.sums, all);
      before = ahead.x;
      gone = ahead.y;
    }
    const int n = evict_length(p, b, lo), keep = min(n, p.budget);
    if (!p.sums && tid == 0 && rank == 0) {
      if (b == 0) p.new_indptr[0] = p.freed_indptr[0] = 0;
      p.new_indptr[b + 1] = before + keep;
      p.freed_indptr[b + 1] = gone + n - keep;
    }
    const float* w = p.weights + static_cast<int64_t>(b) * p.width;
    float* wo = p.weights_out + static_cast<int64_t>(b) * p.width;
    const int mid_lo = min(p.keep_first, n), mid_hi = max(n - p.keep_last, mid_lo);
    const int take = keep - (n - (mid_hi - mid_lo));  // of the middle
    const int run = (n + blocks - 1) / blocks, first = min(rank * run, n), mine = min(run, n - first);
    const bool cut = n > p.budget, hold = mine <= p.held;
    auto weight = [&](int j) { return p.width > 0 && j < p.width ? __ldcg(w + j) : 0.f; };
    auto word_of = [&](int j, float x) -> uint32_t { return j < mid_lo || j >= mid_hi ? kStays : (take > 0 ? ordered_bits(x) : kGoes); };
    auto word = [&](int i) { return word_of(first + i, weight(first + i)); };
    uint32_t least = kKeyLeast;
    int ties = 0;
    if (cut) {
      if (hold) {
        __syncthreads();  // (the words of the sequence before)
#pragma unroll 1
        for (int i0 = tid; i0 < mine; i0 += 8 * THREADS) {  // eight words a thread, their loads together
          float x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = weight(first + min(i0 + u * THREADS, mine - 1));
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (i0 + u * THREADS < mine) held[i0 + u * THREADS] = word_of(first + i0 + u * THREADS, x[u]);
        }
        __syncthreads();
      }
      if (take > 0) {
        least = hold ? select_kth<THREADS, CLUSTERED, uint32_t>(sp, mine, take, [&](int i) { return held[i]; }, ties)
                     : select_kth<THREADS, CLUSTERED, uint32_t>(sp, mine, take, word, ties);
      }
    }
    struct Token {
      int page;
      float weight;
    };
    select_in_order<THREADS, CLUSTERED, 8>(
        sp, mine, ties,
        [&](int i) {
          if (!cut) return 2;
          const uint32_t x = hold ? held[i] : word(i);
          return x == kStays || x > least ? 2 : (x == least ? 1 : 0);
        },
        [&](int i) {
          const int j = first + i;
          return Token{__ldcg(p.kv_indices + lo + j), weight(j)};
        },
        [&](int i, const Token& t, int at, bool stay) {
          const int to = stay ? before + at : gone + first + i - at;
          // (offsets that decrease could pass either end)
          if (static_cast<unsigned>(to) < static_cast<unsigned>(p.index_count)) (stay ? p.new_indices : p.freed)[to] = t.page;
          if (stay && at < p.width) wo[at] = t.weight;
        });
    for (int j = keep + rank * THREADS + tid; j < p.width; j += blocks * THREADS) wo[j] = 0.f;
    // behind the last sequence's, a share a block
    const int64_t shares = static_cast<int64_t>(p.batch) * blocks, share = (p.index_count + shares - 1) / shares;
    const int64_t from = (static_cast<int64_t>(b) * blocks + rank) * share, to = min(from + share, static_cast<int64_t>(p.index_count));
    for (int64_t i = max(from, static_cast<int64_t>(all.x)) + tid; i < to; i += THREADS) p.new_indices[i] = -1;
    for (int64_t i = max(from, static_cast<int64_t>(all.y)) + tid; i < to; i += THREADS) p.freed[i] = -1;
  }
}

constexpr int kClusterThreads = 1024;
static std::atomic<int> g_cluster_limit{0};
void set_evict_cluster_limit(int blocks) { g_cluster_limit.store(blocks); }

// The largest cluster of the eviction that the current device can hold: those of 16 blocks need a part of the GPU with that
// many SMs, which not every one has. Asked for once a device.
static cudaError_t evict_cluster_limit(int* most) {
  static std::atomic<int> known[kMaxDevices], configured[kMaxDevices], allowed[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(gqa_evict_kernel<true, kClusterThreads>);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = set_smem_limit_once(configured, fn, kEvictHeld * 4);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < kMaxDevices;
  *most = tracked ? known[dev].load(std::memory_order_acquire) : 0;
  if (*most == 0) {
    *most = 1;
    for (int blocks = kMostBlocks; blocks > 1 && *most == 1; blocks /= 2) {
      int fit = 0;
      if (blocks > 8 && set_attribute_once(allowed, fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        continue;
      }
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(blocks);
      cfg.blockDim = dim3(kClusterThreads);
      cfg.dynamicSmemBytes = kEvictHeld * 4;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = blocks;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&fit, fn, &cfg) != cudaSuccess) cudaGetLastError();
      else if (fit > 0) *most = blocks;
    }
    if (tracked) known[dev].store(*most, std::memory_order_release);
  }
  const int limit = g_cluster_limit.load();
  if (limit > 0 && limit < *most) *most = limit;
  return cudaSuccess;
}

template <bool CLUSTERED, int THREADS>
static cudaError_t launch_evict_form(const EvictParams& p, cudaStream_t stream) {
  if (!CLUSTERED) {
    static std::atomic<int> configured[kMaxDevices];
    const cudaError_t e = set_smem_limit_once(configured, reinterpret_cast<const void*>(gqa_evict_kernel<CLUSTERED, THREADS>), kEvictHeld * 4);
    if (e != cudaSuccess) return e;
  }
  const int64_t units = p.batch < (1 << 16) ? p.batch : (1 << 16);
  return launch_chained(gqa_evict_kernel<CLUSTERED, THREADS>, dim3(static_cast<unsigned>(units * p.cluster)), THREADS, p.held * 4, stream, p.cluster, p);
}

// What an eviction takes with clusters of `blocks`, in us: a line in the tokens a block for each kernel, twice where they are
// not held, times the rounds (a cluster stays within a part of the GPU, so that of larger ones fewer fit at once). Measured,
// for 1, 2, 4, 8, 16 blocks: 1 sequence of 16384 tokens 27, 19, 16, 16, 16; 48 of 16384 29, 21, 33, 33, 33; 128 of 16384 31, 40,
// 64, 64, 64; 2 of 131072 -, -, -, 30, 24; 8 of 131072 -, 126, 49, 32, 48; 64 of 131072 412, 137, 100, 151, 235.
static double evict_us(int batch, int width, int blocks, int sms) {
  const int run = (width - 1) / blocks + 1;
  const int at_once = blocks == 1 ? 2 * sms : (blocks <= 4 ? sms : (blocks == 8 ? sms * 2 / 3 : sms * 5 / 9)) / blocks;
  if (at_once == 0) return 1e30;
  const int rounds = (batch - 1) / at_once + 1;
  return rounds * (blocks == 1 ? 5.0 + run * (1.4 / 1024) : 11.5 + run * (1.05 / 1024)) * (run > kEvictHeld ? 2 : 1);
}

cudaError_t launch_evict(EvictParams p, int sm_count, cudaStream_t stream) {
  const int width = p.width > 0 ? p.width : 1;
  p.cluster = 1;
  int most = 1;
  if (width >= 2 * kEvictRun) {
    const cudaError_t e = evict_cluster_limit(&most);
    if (e != cudaSuccess) return e;
  }
  for (int blocks = 2; blocks <= most && width >= blocks * kEvictRun; blocks *= 2)
    if (evict_us(p.batch, width, blocks, sm_count) < evict_us(p.batch, width, p.cluster, sm_count)) p.cluster = blocks;
  const int run = (width - 1) / p.cluster + 1;
  p.held = run < kEvictHeld ? run : kEvictHeld;
  p.sums = p.batch > kEvictAlone;
  if (p.sums) {
    const cudaError_t e = launch_chained(gqa_evict_sums_kernel, dim3(1), kSumThreads, 0, stream, 1, p);
    if (e != cudaSuccess) return e;
  }
  return p.cluster > 1 ? launch_evict_form<true, kClusterThreads>(p, stream) : launch_evict_form<false, 512>(p, stream);
}

}  // namespace gqa
