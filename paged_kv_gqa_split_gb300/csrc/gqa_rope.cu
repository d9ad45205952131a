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
// one sincos shared by all heads of its token. A CTA takes `tpb` tokens: its
// threads first fill a table of their (cos, sin) pairs in shared memory, then
// walk the (token, head, vector) items. With 16-byte vectors (bf16 / fp16: 8
// elements) a half-layout item holds the vectors of both partners, so a
// rotation never crosses threads and in-place calls are safe. Windows, strides
// or addresses that do not fit 16-byte vectors take the one-element form.
// Rotation is in fp32; the one rounding is the store to the tensor's type.
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

template <typename T, int V, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) gqa_rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs[];  // [tpb][r / 2]
  const int pairs = p.rot_dim >> 1;
  const int n0 = blockIdx.x * p.tokens_per_block;
  const int nt = min(p.tokens_per_block, p.num_tokens - n0);
  for (int i = threadIdx.x; i < pairs * nt; i += kRopeThreads) {
    const int t = i / pairs;
    float2 v = rope_cos_sin(__ldg(p.positions + n0 + t), rope_turn(__ldg(p.inv_freq + (i - t * pairs))), p.scale);
    if (p.inverse) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();

  // Items of a head. Half layout: pairs / V items of two vectors in the window;
  // interleaved: r / W vectors of W elements, W = V rounded up to a whole pair.
  // Then the vectors outside the window, unless the call is in place.
  constexpr int W = (LAYOUT == kRopeInterleaved && V == 1) ? 2 : V;  // elements of an interleaved item
  const int turn_items = LAYOUT == kRopeHalf ? pairs / V : p.rot_dim / W;
  const int copy_items = p.copy_rest ? (p.head_dim - p.rot_dim) / V : 0;
  const int per_head = turn_items + copy_items;
  const int per_token = per_head * p.num_heads;
  for (int it = threadIdx.x; it < per_token * nt; it += kRopeThreads) {
    const int t = it / per_token;
    const int rem = it - t * per_token;
    const int h = rem / per_head;
    const int k = rem - h * per_head;
    const T* x = static_cast<const T*>(p.x) + (n0 + t) * p.x_token_stride + h * p.x_head_stride;
    T* y = static_cast<T*>(p.out) + (n0 + t) * p.out_token_stride + h * p.out_head_stride;
    const float2* a = cs + t * pairs;
    using VecT = Vec<T, V>;
    if (k >= turn_items) {
      int e = (k - turn_items) * V;
      if (e >= p.rot_offset) e += p.rot_dim;
      *reinterpret_cast<VecT*>(y + e) = *reinterpret_cast<const VecT*>(x + e);
    } else if (LAYOUT == kRopeHalf) {
      const int e = p.rot_offset + k * V;
      const VecT v1 = *reinterpret_cast<const VecT*>(x + e);
      const VecT v2 = *reinterpret_cast<const VecT*>(x + e + pairs);
      VecT w1, w2;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 c = a[k * V + j];
        const float x1 = Elem<T>::load(v1.e[j]), x2 = Elem<T>::load(v2.e[j]);
        w1.e[j] = Elem<T>::store(x1 * c.x - x2 * c.y);
        w2.e[j] = Elem<T>::store(x2 * c.x + x1 * c.y);
      }
      *reinterpret_cast<VecT*>(y + e) = w1;
      *reinterpret_cast<VecT*>(y + e + pairs) = w2;
    } else if (V == 1) {
      const int e = p.rot_offset + 2 * k;
      const float2 c = a[k];
      const float x1 = Elem<T>::load(x[e]), x2 = Elem<T>::load(x[e + 1]);
      y[e] = Elem<T>::store(x1 * c.x - x2 * c.y);
      y[e + 1] = Elem<T>::store(x2 * c.x + x1 * c.y);
    } else {
      const int e = p.rot_offset + k * V;
      const VecT v = *reinterpret_cast<const VecT*>(x + e);
      VecT w;
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 c = a[(k * V + j) >> 1];
        const float x1 = Elem<T>::load(v.e[j]), x2 = Elem<T>::load(v.e[j + 1]);
        w.e[j] = Elem<T>::store(x1 * c.x - x2 * c.y);
        w.e[j + 1] = Elem<T>::store(x2 * c.x + x1 * c.y);
      }
      *reinterpret_cast<VecT*>(y + e) = w;
    }
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
  p.tokens_per_block = 1;
  const int smem = p.tokens_per_block * pairs * static_cast<int>(sizeof(float2));
  const int grid = (p.num_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  (void)sm_count;
  return vec ? launch<T, V>(p, grid, smem, stream) : launch<T, 1>(p, grid, smem, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int sm_count, cudaStream_t stream) {
  if (dtype == kTypeF32) return launch_type<float>(p, sm_count, stream);
  if (dtype == kTypeF16) return launch_type<__half>(p, sm_count, stream);
  return launch_type<__nv_bfloat16>(p, sm_count, stream);
}

}  // namespace gqa
