// Rotary positions on the heads of Q and K.
//
// For token n at position p and pair i of the r / 2 pairs inside the window
// [offset, offset + r) of a head, with a = p * inv_freq[i]:
//   y1 = scale * (x1 cos a - x2 sin a),   y2 = scale * (x2 cos a + x1 sin a)
// where (x1, x2) are elements (i, i + r / 2) of the window (half layout) or
// (2 i, 2 i + 1) (interleaved). Elements outside the window are copied.
// `inverse` turns by -a, which undoes a rotation and is also its gradient.
//
// Bounded by HBM: every element is read and written once, and an angle costs
// one sincos shared by all heads of its token. A CTA takes a few tokens: it fills
// a table of their (cos, sin) pairs in shared memory (the frequencies' 64-bit
// arithmetic once per CTA: the part has few FP64 lanes), then its threads walk the
// (token, head) rows, a thread always at the same vector of a head, four rows'
// loads in flight. With 16-byte vectors (bf16 / fp16: 8 elements) a half-layout
// item holds the vectors of both partners, so a rotation never crosses threads and
// in-place calls are safe. Windows, strides or addresses that do not fit 16-byte
// vectors take the one-element form. Rotation is in fp32; the one rounding is the
// store to the tensor's type.
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
  __device__ __forceinline__ void finish(T* y, int e, int pairs, bool turn, const float2* cs) {
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
  extern __shared__ float2 cs[];  // [tokens_per_block][r / 2], then the frequencies [r / 2]
  const int pairs = p.rot_dim >> 1;
  const int n0 = blockIdx.x * p.tokens_per_block;
  const int nt = min(p.tokens_per_block, p.num_tokens - n0);

  // Items of a head: the window's (pairs of vectors, vectors or pairs), then the vectors outside it unless in place.
  constexpr int kTurned = LAYOUT == kRopeHalf ? V : (V == 1 ? 1 : V / 2);  // pairs an item turns
  const int turn_items = pairs / kTurned;
  const int per_head = turn_items + (p.copy_rest ? (p.head_dim - p.rot_dim) / V : 0);
  const int rows = nt * p.num_heads;
  const bool wide = per_head > kRopeThreads;  // a head holds more items than threads: one row at a time
  const int rows_at_once = wide ? 1 : kRopeThreads / per_head;
  const int y = wide ? 0 : threadIdx.x / per_head;
  const int k0 = threadIdx.x - y * per_head;
  const uint32_t magic = p.head_magic;
  constexpr int U = 4;
  Item<T, V, LAYOUT> it[U];
  int e = 0;
  bool turn = false;
  auto place = [&](int k) {
    turn = k < turn_items;
    e = turn ? p.rot_offset + k * kTurned * (LAYOUT == kRopeHalf ? 1 : 2) : (k - turn_items) * V;
    if (!turn && e >= p.rot_offset) e += p.rot_dim;
  };
  auto token = [&](int row) { return magic != 0 ? static_cast<int>(__umulhi(row, magic)) : row; };  // row / num_heads
  auto load = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r + u * rows_at_once;
      if (row >= rows) break;
      const int t = token(row), h = row - t * p.num_heads;
      it[u].load(static_cast<const T*>(p.x) + (n0 + t) * p.x_token_stride + h * p.x_head_stride, e, pairs, turn);
    }
  };
  const bool active = y < rows_at_once;
  place(k0);
  if (active) load(y);  // in flight while the table is filled

  unsigned long long* turns = reinterpret_cast<unsigned long long*>(cs + p.tokens_per_block * pairs);
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) turns[i] = rope_turn(__ldg(p.inv_freq + i));
  __syncthreads();
  for (int i = threadIdx.x; i < pairs * nt; i += kRopeThreads) {
    const int t = i / pairs;
    float2 v = rope_cos_sin(__ldg(p.positions + n0 + t), turns[i - t * pairs], p.scale);
    if (p.inverse) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();
  if (!active) return;

  for (int k = k0; k < per_head; k += kRopeThreads) {
    if (k != k0) {
      place(k);
      load(y);
    }
    const float2* mine = cs + (turn ? k * kTurned : 0);
    for (int r = y; r < rows; r += U * rows_at_once) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = r + u * rows_at_once;
        if (row >= rows) break;
        const int t = token(row), h = row - t * p.num_heads;
        it[u].finish(static_cast<T*>(p.out) + (n0 + t) * p.out_token_stride + h * p.out_head_stride, e, pairs, turn,
                     mine + t * pairs);
      }
      load(r + U * rows_at_once);
    }
    if (!wide) break;
  }
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, int grid, int smem, cudaStream_t stream) {
  if (p.layout == kRopeHalf)
    gqa_rope_kernel<T, V, kRopeHalf><<<grid, kRopeThreads, smem, stream>>>(p);
  else
    gqa_rope_kernel<T, V, kRopeInterleaved><<<grid, kRopeThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(RopeParams p, int sm_count, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const int pairs = p.rot_dim / 2;
  const int64_t strides = p.x_token_stride | p.x_head_stride | p.out_token_stride | p.out_head_stride;
  const bool addr = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0;
  const int window = p.layout == kRopeHalf ? pairs : p.rot_dim;
  const bool vec = addr && (strides | p.rot_offset | window | (p.head_dim - p.rot_dim)) % V == 0;
  p.copy_rest = p.x != p.out || p.x_token_stride != p.out_token_stride || p.x_head_stride != p.out_head_stride;
  // one token a CTA until the CTAs fill the GPU 16 times over, then up to 8 share a table
  const int most = p.num_tokens / (16 * sm_count);
  p.tokens_per_block = most < 1 ? 1 : (most > 8 ? 8 : most);
  const int smem = (p.tokens_per_block + 1) * pairs * static_cast<int>(sizeof(float2));
  const int grid = (p.num_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  // row / heads as the upper half of row * magic: exact below 2^32 / heads rows (a CTA has at most 8 * heads)
  p.head_magic = p.num_heads > 1 ? static_cast<uint32_t>(((1ull << 32) + p.num_heads - 1) / p.num_heads) : 0;
  return vec ? launch<T, V>(p, grid, smem, stream) : launch<T, 1>(p, grid, smem, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int sm_count, cudaStream_t stream) {
  if (dtype == kTypeF32) return launch_type<float>(p, sm_count, stream);
  if (dtype == kTypeF16) return launch_type<__half>(p, sm_count, stream);
  return launch_type<__nv_bfloat16>(p, sm_count, stream);
}

}  // namespace gqa
