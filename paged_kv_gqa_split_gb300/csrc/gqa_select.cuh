// Choosing the k largest of n keys with one block, ties to the lowest index: a radix select from the top digit down, 8 bits a
// pass, then the chosen in index order.
#pragma once

#include <cstdint>

namespace gqa {

// Order-preserving bits of a float: larger float, larger word; -0 and +0 alike, NaN above everything.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int THREADS>
struct SelectSpace {
  int hist[256];
  int warp_sum[THREADS / 32];
  int digit, above;
};

// Sum over the block; every thread gets it. `space` is free again after the next barrier.
template <int THREADS>
__device__ __forceinline__ int block_sum(SelectSpace<THREADS>& sp, int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sp.warp_sum[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += sp.warp_sum[w];
  return s;
}

// Exclusive prefix sum of `flag` over the block's threads; total gets the sum.
template <int THREADS>
__device__ __forceinline__ int block_rank(SelectSpace<THREADS>& sp, bool flag, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sp.warp_sum[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = all;
    all += sp.warp_sum[w];
  }
  total = all;
  return before + __popc(m & ((1u << lane) - 1u));
}

// The k-th largest (k >= 1) of key(i), 0 <= i < n, over the i for which in(i) holds (at least k of them): returns its
// value, and in `above` how many are larger. Key: uint32_t or uint64_t.
template <int THREADS, typename Key, typename In, typename Get>
__device__ __forceinline__ Key block_kth(SelectSpace<THREADS>& sp, int n, int k, In in, Get key, int& above) {
  constexpr int kBits = 8 * sizeof(Key);
  Key prefix = 0;
  int left = k;
  above = 0;
#pragma unroll 1
  for (int shift = kBits - 8; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += THREADS) sp.hist[i] = 0;
    __syncthreads();
    const Key mask = shift == kBits - 8 ? Key(0) : (~Key(0)) << (shift + 8);
    for (int i0 = 0; i0 < n; i0 += THREADS) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      int d = 256;
      if (i < n && in(i)) {
        const Key x = key(i);
        if ((x & mask) == prefix) d = static_cast<int>((x >> shift) & 255);
      }
      // many keys share their top digits: one addition for all lanes of a digit
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d < 256 && (threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&sp.hist[d], __popc(same));
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // lane l holds digits 255 - 8 l .. 248 - 8 l, the largest first
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = sp.hist[255 - 8 * static_cast<int>(threadIdx.x) - j];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (static_cast<int>(threadIdx.x) >= o) incl += up;
      }
      int before = incl - sum;
      if (before < left && left <= incl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < left && left <= before + c[j]) {
            sp.digit = 255 - 8 * static_cast<int>(threadIdx.x) - j;
            sp.above = before;
          }
          before += c[j];
        }
      }
    }
    __syncthreads();
    prefix |= static_cast<Key>(sp.digit) << shift;
    left -= sp.above;
    above += sp.above;
  }
  return prefix;
}

}  // namespace gqa
