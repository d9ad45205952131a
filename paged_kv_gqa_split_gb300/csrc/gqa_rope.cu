// Rotary positions on the heads of Q and K.
//
// For token n at position p and pair i of the r / 2 pairs inside the window
// [offset, offset + r) of a head, with a = p * inv_freq[i]:
//   y1 = scale * (x1 cos a - x2 sin a),   y2 = scale * (x2 cos a + x1 sin a)
// where (x1, x2) are elements (i, i + r / 2) of the window (half layout) or
// (2 i, 2 i + 1) (interleaved). Elements outside the window are copied.
// `inverse` turns by -a, which undoes a rotation and is also its gradient.
//
// Bounded by HBM: every element is read and written once. A thread stays at one
// vector of a head and one token and walks that token's heads (or, with few tokens,
// a share of them), a few rows' loads in flight; it forms its pairs' (cos, sin) once
// for all of them, while the first rows load; the frequencies' fixed-point fractions are
// formed once per CTA. (With a table of all pairs' (cos, sin) in
// shared memory the two barriers and the table's latency held HBM at 50 %.) With 16-byte
// vectors (bf16 / fp16: 8 elements) a half-layout item holds the vectors of both
// partners, so a rotation never crosses threads and in-place calls are safe. Windows,
// strides or addresses that do not fit 16-byte vectors take the one-element form.
// Rotation is in fp32; the one rounding is the store to the tensor's type.
// Measured: 32768 tokens x 16 heads x 192 bf16, 64 values turned, 69 us (5.8 TB/s, 86 %
// of the measured copy rate); x 36 heads x 128, whole heads, interleaved 97 us (6.2 TB/s), half
// layout 118 us (5.1); 16 heads x 128 fp32, half layout, 83 us (6.5); 64 tokens x 36 heads x 128,
// 4.4 us. The one-element form: 2.6 TB/s (rows off 16-byte boundaries, or 20 of 80 values turned).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_rope.cuh"

namespace gqa {
namespace {

constexpr int kRopeThreads = 256;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ float load(float v) { return v; }
  static __device__ float store(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ float load(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __nv_bfloat16 store(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ float load(__half v) { return __half2float(v); }
  static __device__ __half store(float v) { return __float2half_rn(v); }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// One item of a row: reads its vectors, then turns (or copies) and writes them.
template <typename T, int V, int LAYOUT>
struct Item {
  using VecT = Vec<T, V>;
  VecT a, b;  // b: the partners (half layout), or the pair's second element (interleaved, V = 1)

  __device__ __forceinline__ void load(const T* x, int e, int pairs, bool turn) {
    a = *reinterpret_cast<const VecT*>(x + e);
    if (turn && LAYOUT == kRopeHalf) b = *reinterpret_cast<const VecT*>(x + e + pairs);
    if (turn && LAYOUT == kRopeInterleaved && V == 1) b = *reinterpret_cast<const VecT*>(x + e + 1);
  }
  __device__ __forceinline__ void finish(T* y, int e, int pairs, bool turn, const float2 (&cs)[LAYOUT == kRopeHalf ? V : (V + 1) / 2]) {
    if (!turn) {
      *reinterpret_cast<VecT*>(y + e) = a;
    } else if (LAYOUT == kRopeHalf || V == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 c = cs[j];
        const float x1 = Elem<T>::load(a.e[j]), x2 = Elem<T>::load(b.e[j]);
        a.e[j] = Elem<T>::store(x1 * c.x - x2 * c.y);
        b.e[j] = Elem<T>::store(x2 * c.x + x1 * c.y);
      }
      *reinterpret_cast<VecT*>(y + e) = a;
      *reinterpret_cast<VecT*>(y + e + (LAYOUT == kRopeHalf ? pairs : 1)) = b;
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 c = cs[j >> 1];
        const float x1 = Elem<T>::load(a.e[j]), x2 = Elem<T>::load(a.e[j + 1]);
        a.e[j] = Elem<T>::store(x1 * c.x - x2 * c.y);
        a.e[j + 1] = Elem<T>::store(x2 * c.x + x1 * c.y);
      }
      *reinterpret_cast<VecT*>(y + e) = a;
    }
  }
};

template <typename T, int V, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) gqa_rope_kernel(const RopeParams p) {
  extern __shared__ unsigned long long turns[];  // [r / 2]
  // Items of a head: the window's (pairs of vectors, vectors or pairs), then the vectors outside it unless in place.
  constexpr int kTurned = LAYOUT == kRopeHalf ? V : (V + 1) / 2;  // pairs an item turns
  constexpr int U = LAYOUT == kRopeHalf ? 2 : 4;                  // rows in flight
  const int pairs = p.rot_dim >> 1;
  const int turn_items = pairs / kTurned;
  const int per_head = turn_items + (p.copy_rest ? (p.head_dim - p.rot_dim) / V : 0);
  const bool wide = per_head > kRopeThreads;  // a head holds more items than threads
  const int tokens = wide ? 1 : kRopeThreads / per_head;
  const int y = wide ? 0 : threadIdx.x / per_head;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * tokens + y;
  const int h0 = blockIdx.y * p.heads_each, h1 = min(h0 + p.heads_each, p.num_heads);
  const bool active = y < tokens && n < p.num_tokens;
  const T* x = static_cast<const T*>(p.x) + n * p.x_token_stride;
  T* out = static_cast<T*>(p.out) + n * p.out_token_stride;
  Item<T, V, LAYOUT> it[U];
  int e = 0;
  bool turn = false;
  auto place = [&](int k) {
    turn = k < turn_items;
    e = turn ? p.rot_offset + k * kTurned * (LAYOUT == kRopeHalf ? 1 : 2) : (k - turn_items) * V;
    if (!turn && e >= p.rot_offset) e += p.rot_dim;
  };
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < h1) it[u].load(x + (h + u) * p.x_head_stride, e, pairs, turn);
  };
  int k = threadIdx.x - y * per_head;
  int pos = 0;
  if (active) {
    place(k);
    load(h0);
    pos = __ldg(p.positions + n);
  }
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) turns[i] = rope_turn(__ldg(p.inv_freq + i));
  __syncthreads();
  if (!active) return;

  for (;;) {
    float2 cs[kTurned];
    if (turn) {
#pragma unroll
      for (int j = 0; j < kTurned; ++j) {
        cs[j] = rope_cos_sin(pos, turns[k * kTurned + j], p.scale);
        if (p.inverse) cs[j].y = -cs[j].y;
      }
    }
    for (int h = h0; h < h1; h += U) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u < h1) it[u].finish(out + (h + u) * p.out_head_stride, e, pairs, turn, cs);
      if (h + U < h1) load(h + U);
    }
    k += kRopeThreads;
    if (!wide || k >= per_head) break;
    place(k);
    load(h0);
  }
}

template <typename T, int V>
cudaError_t launch(RopeParams p, int sm_count, cudaStream_t stream) {
  const int pairs = p.rot_dim / 2;
  const int turned = p.layout == kRopeHalf ? V : (V + 1) / 2;
  const int per_head = pairs / turned + (p.copy_rest ? (p.head_dim - p.rot_dim) / V : 0);
  const int tokens = per_head > kRopeThreads ? 1 : kRopeThreads / per_head;
  const int64_t blocks = (static_cast<int64_t>(p.num_tokens) + tokens - 1) / tokens;
  // all heads of a token a thread, or, where that leaves fewer than 8 CTAs an SM, a share of them
  const int64_t want = 8 * static_cast<int64_t>(sm_count);
  int64_t splits = blocks >= want ? 1 : (want + blocks - 1) / blocks;
  if (splits > p.num_heads) splits = p.num_heads;
  p.heads_each = static_cast<int>((p.num_heads + splits - 1) / splits);
  const dim3 grid(static_cast<unsigned>(blocks), (p.num_heads + p.heads_each - 1) / p.heads_each);
  const int smem = pairs * static_cast<int>(sizeof(unsigned long long));
  if (p.layout == kRopeHalf)
    gqa_rope_kernel<T, V, kRopeHalf><<<grid, kRopeThreads, smem, stream>>>(p);
  else
    gqa_rope_kernel<T, V, kRopeInterleaved><<<grid, kRopeThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(RopeParams p, int sm_count, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const int64_t strides = p.x_token_stride | p.x_head_stride | p.out_token_stride | p.out_head_stride;
  const bool addr = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0;
  const int window = p.layout == kRopeHalf ? p.rot_dim / 2 : p.rot_dim;
  const bool vec = addr && (strides | p.rot_offset | window | (p.head_dim - p.rot_dim)) % V == 0;
  p.copy_rest = p.x != p.out || p.x_token_stride != p.out_token_stride || p.x_head_stride != p.out_head_stride;
  return vec ? launch<T, V>(p, sm_count, stream) : launch<T, 1>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int sm_count, cudaStream_t stream) {
  if (dtype == kTypeF32) return launch_type<float>(p, sm_count, stream);
  if (dtype == kTypeF16) return launch_type<__half>(p, sm_count, stream);
  return launch_type<__nv_bfloat16>(p, sm_count, stream);
}

}  // namespace gqa
