// Choosing the k largest of many keys, ties to the lowest index: a radix select from the top digit down, 8 bits a pass, by
// one block or a cluster of them, then the chosen in index order from one pass of counts. Keys are 32-bit words that order
// as their numbers do; they are read four or five times, from shared memory where they fit.
#pragma once

#include <cooperative_groups.h>

#include <cstdint>

namespace gqa {

// Order-preserving bits of a float: larger float, larger word; -0 and +0 alike, NaN above everything. No float has a word
// below kKeyLeast, so smaller words are free for marks.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_float(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kKeyLeast = 0x007fffffu, kKeyInf = 0xff800000u;  // -inf, +inf

// Sum over the block of two numbers; every thread gets them. `sums` holds 2 words a warp.
template <int THREADS>
__device__ __forceinline__ int2 block_sum2(int2* sums, int2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  const int2 v = (threadIdx.x & 31) < THREADS / 32 ? sums[threadIdx.x & 31] : make_int2(0, 0);
  return make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
}

constexpr int kMostBlocks = 16;  // of a cluster

template <int THREADS>
struct SelectSpace {
  alignas(16) int hist[3][256];  // of this block, in turns
  alignas(16) int all[256];      // of the cluster
  int2 sums[THREADS / 32];
  int2 counts;                   // this block's, for the others of its cluster
  unsigned long long least;
};

// The k-th largest (k >= 1) of this cluster's keys, of which this block has keys[0 .. n), and in `ties` at least how many
// of the keys equal to it are among the k largest. Every block of the cluster calls it (CLUSTERED), or a block alone.
// A pass counts the keys of a prefix by their next 8 bits; every warp finds the digit by itself, so that a pass needs one
// barrier (a cluster one of its own more). As soon as all keys of the digit are among the k largest, the smallest of them is the k-th.
template <int THREADS, bool CLUSTERED, typename Key, typename Get>
__device__ __forceinline__ Key select_kth(SelectSpace<THREADS>& sp, int n, int k, Get key, int& ties) {
  constexpr int kBits = 8 * sizeof(Key);
  const int lane = threadIdx.x & 31;
  Key prefix = 0;
  int left = k;
  for (int i = threadIdx.x; i < 256; i += THREADS) sp.hist[0][i] = 0;
  if (threadIdx.x == 0) sp.least = ~0ull;
  __syncthreads();
  int turn = 0;
  bool whole = false;
#pragma unroll 1
  for (int shift = kBits - 8; shift >= 0 && !whole; shift -= 8) {
    int* hist = sp.hist[turn];
    turn = turn == 2 ? 0 : turn + 1;
    for (int i = threadIdx.x; i < 256; i += THREADS) sp.hist[turn][i] = 0;  // the next pass's: read last two passes ago
    const Key mask = shift == kBits - 8 ? Key(0) : (~Key(0)) << (shift + 8);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 4 * THREADS) {  // four keys a thread, their loads together
      Key x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = key(min(i0 + u * THREADS + static_cast<int>(threadIdx.x), n - 1));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int d = i0 + u * THREADS + static_cast<int>(threadIdx.x) < n && (x[u] & mask) == prefix ? static_cast<int>((x[u] >> shift) & 255) : 256;
        // keys of one size share their top digits: one addition where all lanes have the same
        const int d0 = __shfl_sync(0xffffffffu, d, 0);
        if (__all_sync(0xffffffffu, d == d0)) {
          if (d0 < 256 && lane == 0) atomicAdd(&hist[d0], 32);
        } else if (d < 256) {
          atomicAdd(&hist[d], 1);
        }
      }
    }
    if constexpr (CLUSTERED) {
      auto cluster = cooperative_groups::this_cluster();
      cluster.sync();  // (others read this turn's counts until the next pass's, and they are cleared after that)
      for (int i = threadIdx.x; i < 256; i += THREADS) {
        int x[kMostBlocks], sum = 0;  // (their loads together)
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) x[r] = r < static_cast<int>(cluster.num_blocks()) ? cluster.map_shared_rank(hist, r)[i] : 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) sum += x[r];
        sp.all[i] = sum;
      }
      hist = sp.all;
    }
    __syncthreads();
    // lane l holds digits 8 l .. 8 l + 7, counted from the largest down
    const int4 ca = reinterpret_cast<const int4*>(hist)[2 * lane], cb = reinterpret_cast<const int4*>(hist)[2 * lane + 1];
    const int c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += c[j];
    int upto = sum;  // of this lane's digits and all larger ones
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int more = __shfl_down_sync(0xffffffffu, upto, o);
      if (lane + o < 32) upto += more;
    }
    int before = upto - sum, digit = -1, above = 0, count = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      if (before < left && left <= before + c[j]) digit = 8 * lane + j, above = before, count = c[j];
      before += c[j];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, digit >= 0)) - 1;
    digit = __shfl_sync(0xffffffffu, digit, src);
    above = __shfl_sync(0xffffffffu, above, src);
    count = __shfl_sync(0xffffffffu, count, src);
    prefix |= static_cast<Key>(digit) << shift;
    left -= above;
    whole = count == left && shift > 0;
    if (whole) {  // the smallest key that is at least the prefix
      Key least = ~Key(0);
      for (int i = threadIdx.x; i < n; i += THREADS) {
        const Key x = key(i);
        if (x >= prefix && x < least) least = x;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Key x = __shfl_xor_sync(0xffffffffu, least, o);
        least = x < least ? x : least;
      }
      if (lane == 0) atomicMin(&sp.least, static_cast<unsigned long long>(least));
      __syncthreads();
      if constexpr (CLUSTERED) {
        auto cluster = cooperative_groups::this_cluster();
        cluster.sync();
        unsigned long long all = ~0ull;
        for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
          const unsigned long long x = *cluster.map_shared_rank(&sp.least, r);
          all = x < all ? x : all;
        }
        cluster.sync();
        prefix = static_cast<Key>(all);
      } else {
        prefix = static_cast<Key>(sp.least);
      }
    }
    if constexpr (CLUSTERED) __syncthreads();  // sp.all is written anew
  }
  __syncthreads();
  ties = left;  // (all of them, where the digit's keys were taken whole)
  return prefix;
}

// The k-th largest of up to 32 * OWN words, by one warp and without a barrier: bit by bit the largest word that k words
// reach, until exactly k do. For short rows (choosing among 144 blocks for 128 rows: 22.9 us with select_kth, 21.6 with this,
// where counting by ballots, under a condition each, took 35).
template <int OWN>
__device__ __forceinline__ uint32_t warp_kth(const uint32_t* words, int n, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t x[OWN];
#pragma unroll
  for (int u = 0; u < OWN; ++u) x[u] = 32 * u + lane < n ? words[32 * u + lane] : 0;
  uint32_t t = 0;
  bool exact = false;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit != 0 && !exact; bit >>= 1) {
    int reach = 0;
#pragma unroll
    for (int u = 0; u < OWN; ++u) reach += x[u] >= (t | bit) ? 1 : 0;
    reach = __reduce_add_sync(0xffffffffu, reach);
    if (reach >= k) t |= bit;
    exact = reach == k;
  }
  uint32_t least = 0xffffffffu;  // of those that reach it
#pragma unroll
  for (int u = 0; u < OWN; ++u)
    if (x[u] >= t && x[u] < least) least = x[u];
  return __reduce_min_sync(0xffffffffu, least);
}

// Walks this block's items 0 .. n in index order: cls(i) is 2 for a chosen item, 1 for one that ties with the last chosen
// (the first `ties` of the cluster's are chosen too), 0 for others; put(i, x, rank, chosen) is called for every item, rank
// being the number of chosen items before it in the cluster and x what get(i) returned: those are called AHEAD at a time,
// so that their loads do not wait for the stores of the items before. A warp takes a run of items, 32 at a time.
template <int THREADS, bool CLUSTERED, int AHEAD, typename Class, typename Get, typename Put>
__device__ __forceinline__ void select_in_order(SelectSpace<THREADS>& sp, int n, int ties, Class cls, Get get, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = ((n + THREADS - 1) / THREADS) * 32, first = warp * run, end = min(first + run, n);
  int2 mine = make_int2(0, 0);  // chosen outright, ties
#pragma unroll 1
  for (int i0 = first; i0 < end; i0 += 128) {
    int c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) c[u] = i0 + 32 * u + lane < end ? cls(i0 + 32 * u + lane) : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      mine.x += __popc(__ballot_sync(0xffffffffu, c[u] == 2));
      mine.y += __popc(__ballot_sync(0xffffffffu, c[u] == 1));
    }
  }
  __syncthreads();
  if (lane == 0) sp.sums[warp] = mine;
  __syncthreads();
  const int2 v = lane < THREADS / 32 ? sp.sums[lane] : make_int2(0, 0);
  const bool ahead = lane < warp;
  int2 at = make_int2(__reduce_add_sync(0xffffffffu, ahead ? v.x : 0), __reduce_add_sync(0xffffffffu, ahead ? v.y : 0));
  if constexpr (CLUSTERED) {
    auto cluster = cooperative_groups::this_cluster();
    const int2 all = make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
    if (threadIdx.x == 0) sp.counts = all;
    cluster.sync();
    for (unsigned r = 0; r < cluster.block_rank(); ++r) {
      const int2 c = *cluster.map_shared_rank(&sp.counts, r);
      at.x += c.x;
      at.y += c.y;
    }
    cluster.sync();  // no block leaves, or counts anew, while another reads
  }
#pragma unroll 1
  for (int i0 = first; i0 < end; i0 += 32 * AHEAD) {
    decltype(get(0)) x[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) x[u] = get(min(i0 + 32 * u + lane, end - 1));
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + 32 * u + lane;
      const int c = i < end ? cls(i) : 0;
      const unsigned sure = __ballot_sync(0xffffffffu, c == 2), tied = __ballot_sync(0xffffffffu, c == 1);
      const unsigned below = (1u << lane) - 1u;
      const int tie = at.y + __popc(tied & below);
      if (i < end) put(i, x[u], at.x + __popc(sure & below) + min(tie, ties), c == 2 || (c == 1 && tie < ties));
      at.x += __popc(sure);
      at.y += __popc(tied);
    }
  }
}

}  // namespace gqa
