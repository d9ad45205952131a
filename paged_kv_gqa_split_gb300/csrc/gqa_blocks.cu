// Attention over blocks that a cheap score selects. A block is a page of a block-table cache.
//   bounds:  hi[block][g][d], lo[block][g][d] = largest and smallest k[t][g][d] of the block's tokens (bf16, exact)
//   score:   score[row][g][block] = max over the 8 query heads h of g of
//                sum_d max(q[h][d], 0) hi[d] + min(q[h][d], 0) lo[d],
//            which no q . k of the block's tokens passes
//   choice:  the first and last blocks of a row's tokens, then those of the largest scores
//   slots:   the chosen blocks' tokens for the selected-token decode (kFormHeads)
#include <cuda_runtime.h>

#include "gqa_common.cuh"
#include "gqa_kernels.h"
#include "gqa_select.cuh"

namespace gqa {

constexpr int kRowValues = kKvHeads * kHeadDim;  // of a token, or of a block's upper or lower bounds

// ----------------------------------------------------------------- bounds
// Teams of 64 lanes, 16 bytes a lane and token. The blocks to renew, request by request, are numbered by prefix sums that
// every block of threads forms by itself, 256 requests at a time, and taken in turns: by a block of threads, its four teams
// sharing one, or by a team where they are many and of few tokens (131072 tokens in pages of 16: 31 us by teams, 34 shared;
// of 32: 29 and 27; of 64: 37 and 31). Bound by the keys' bytes (524288 tokens: 5.6 TB/s) and, below that, by how many
// loads a block's tokens give a team at once; one new token each of 64 requests takes 5 us, the launch and four dependent loads.
constexpr int kBoundThreads = 256, kBoundTeams = kBoundThreads / 64, kSharedPage = 32;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

struct MinMax {
  uint4 hi, lo;
  __device__ __forceinline__ void init() {
    hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);
  }
  __device__ __forceinline__ void add(const uint4& a, const uint4& b) {
    hi = make_uint4(max2(hi.x, a.x), max2(hi.y, a.y), max2(hi.z, a.z), max2(hi.w, a.w));
    lo = make_uint4(min2(lo.x, b.x), min2(lo.y, b.y), min2(lo.z, b.z), min2(lo.w, b.w));
  }
};

__global__ void __launch_bounds__(kBoundThreads) gqa_block_bounds_kernel(const BoundsParams p) {
  __shared__ MinMax part[kBoundTeams][64];
  __shared__ int64_t start[kBoundThreads + 1], warp_sum[kBoundThreads / 32];
  __shared__ int first_block[kBoundThreads], length[kBoundThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 63, team = tid >> 6;
  // tokens t0, t0 + step, ... of the i-th block of request r; false if its table names no block of the pool
  auto walk = [&](int r, int i, int n, int t0, int step, MinMax& mm, int64_t& block) {
    const int b = __ldcg(p.block_table + static_cast<int64_t>(r) * p.width + i);
    if (static_cast<unsigned>(b) >= static_cast<unsigned>(p.num_blocks)) return false;
    block = b;
    const int tokens = min(p.page_size, n - i * p.page_size);
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_cache) + block * p.page_size * kRowValues) + lane;
    mm.init();
    int t = t0;  // (up to 2^30 tokens a block: their numbers have 31 bits, the offsets of those from 2^25 on have not)
    for (; t + 15 * step < tokens; t += 16 * step) {
      uint4 x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) x[u] = __ldcg(k + static_cast<int64_t>(t + u * step) * 64);
#pragma unroll
      for (int u = 0; u < 16; ++u) mm.add(x[u], x[u]);
    }
#pragma unroll 4
    for (; t < tokens; t += step) {
      const uint4 x = __ldcg(k + static_cast<int64_t>(t) * 64);
      mm.add(x, x);
    }
    return true;
  };
  auto store = [&](int64_t block, const MinMax& mm) {
    uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.bounds) + block * 2 * kRowValues) + lane;
    to[0] = mm.hi;
    to[64] = mm.lo;
  };
  for (int r0 = 0; r0 < p.requests; r0 += kBoundThreads) {
    const int r = r0 + tid;
    int count = 0, at = 0, n = 0;
    if (r < p.requests) {
      n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(__ldcg(p.lens + r)), static_cast<int64_t>(p.width) * p.page_size)));
      const int first = p.first == nullptr ? 0 : max(0, __ldcg(p.first + r));
      at = first / p.page_size;
      if (first < n) count = (n - 1) / p.page_size + 1 - at;
    }
    int64_t upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if ((tid & 31) >= o) upto += up;
    }
    __syncthreads();  // the requests before have been walked
    if ((tid & 31) == 31) warp_sum[tid >> 5] = upto;
    first_block[tid] = at;
    length[tid] = n;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) upto += warp_sum[w];
    start[tid + 1] = upto;
    if (tid == 0) start[0] = 0;
    __syncthreads();
    const int64_t total = start[kBoundThreads];
    const bool shared = total <= gridDim.x || p.page_size >= kSharedPage;
    const int64_t teams = shared ? gridDim.x : gridDim.x * kBoundTeams;
    for (int64_t x = shared ? blockIdx.x : blockIdx.x + team * gridDim.x; x < total; x += teams) {
      int lo = 0, hi = kBoundThreads;  // the request: start[lo] <= x < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid;
      }
      MinMax mm;
      int64_t block = 0;
      const bool ok = walk(r0 + lo, first_block[lo] + static_cast<int>(x - start[lo]), length[lo], shared ? team : 0, shared ? kBoundTeams : 1, mm, block);
      if (!ok) continue;  // the same for the team, and for the block of threads where it shares
      if (shared) {
        part[team][lane] = mm;
        __syncthreads();
        if (team == 0)
#pragma unroll
          for (int j = 1; j < kBoundTeams; ++j) mm.add(part[j][lane].hi, part[j][lane].lo);
        __syncthreads();
        if (team != 0) continue;
      }
      store(block, mm);
    }
  }
}

cudaError_t launch_block_bounds(const BoundsParams& p, int sm_count, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(p.requests) * p.width;
  return launch_chained(gqa_block_bounds_kernel, dim3(most < 8 * sm_count ? most : 8 * sm_count), kBoundThreads, 0, stream, 1, p);
}

// ------------------------------------------------------------------ score
// A warp per KV head and 16 blocks at a time: S^T (16 blocks x 8 heads) += [hi lo] (16 x 16) . [q+ q-]^T, 16 MMAs of
// m16n8k16 in all. A lane reads 16 consecutive bytes of a block's bounds, the contraction's order following: within 32
// dims, lane c's k indices 2c, 2c + 1, 2c + 8, 2c + 9 of the first MMA are dims 8c .. 8c + 3, of the second 8c + 4 .. + 7.
// Beside the score goes a bound of its error, kGamma * max_h |q_h|_1 * max |bounds|, for the choice: products of bf16 are
// exact in fp32; an MMA sums 16 of them and the accumulator, each cut off at 2^-23 of the largest, and no partial sum
// passes |q|_1 max|bounds|: 16 MMAs x 17 terms x 2^-23 < 2^-14.9. Bound by the round trips row, table, bounds (one row of 2048
// blocks 4.3 us), with many rows by the bounds' bytes (128 rows of 32 to 256 blocks 9 us).
constexpr int kScoreBlocks = 16;  // of a row, a block of threads
constexpr float kGamma = 0x1p-14f;
constexpr float kBounded = kGamma * 0x1p126f;  // an error below it: no partial sum of the MMAs can pass fp32's range
constexpr uint32_t kNoBlock = 0xffffffffu;  // in a score's place where the table names no block of the pool

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct RowView {
  int n, count, req;  // tokens, blocks
};
__device__ __forceinline__ RowView row_view(const BlockParams& p, int row) {
  RowView v;
  v.req = __ldcg(p.token_to_req + row);
  const bool ok = v.req >= 0 && v.req < p.requests;
  v.n = ok ? static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(__ldcg(p.lens + row)), static_cast<int64_t>(p.width) * p.page_size))) : 0;
  v.count = v.n > 0 ? (v.n - 1) / p.page_size + 1 : 0;
  return v;
}

__global__ void __launch_bounds__(128) gqa_block_score_kernel(const BlockParams p) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  for (int row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const uint4* qr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(row) * kQoHeads + g * kGroup + r) * kHeadDim) + c;
    uint4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = __ldcg(qr + 4 * j);
    const RowView v = row_view(p, row);
    const int first = blockIdx.x * kScoreBlocks;
    if (first >= v.count) continue;
    const int* table = p.block_table + static_cast<int64_t>(v.req) * p.width;
    const int ia = first + r, ib = first + r + 8;
    const int pa = ia < v.count ? __ldcg(table + ia) : -1, pb = ib < v.count ? __ldcg(table + ib) : -1;
    const bool oka = static_cast<unsigned>(pa) < static_cast<unsigned>(p.num_blocks), okb = static_cast<unsigned>(pb) < static_cast<unsigned>(p.num_blocks);
    const uint4* xa = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) + (static_cast<int64_t>(oka ? pa : 0) * 2 * kKvHeads + g) * kHeadDim) + c;
    const uint4* xb = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) + (static_cast<int64_t>(okb ? pb : 0) * 2 * kKvHeads + g) * kHeadDim) + c;
    uint4 a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // 0 .. 3 hi, 4 .. 7 lo
      const int at = (j >> 2) * (kRowValues / 8) + 4 * (j & 3);
      a[j] = oka ? __ldcg(xa + at) : make_uint4(0, 0, 0, 0);
      b[j] = okb ? __ldcg(xb + at) : make_uint4(0, 0, 0, 0);
    }
    float norm = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) norm += fabsf(bf16_lo(w[i])) + fabsf(bf16_hi(w[i]));
    }
    norm += __shfl_xor_sync(0xffffffffu, norm, 1);
    norm += __shfl_xor_sync(0xffffffffu, norm, 2);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) norm = max_nan(norm, __shfl_xor_sync(0xffffffffu, norm, o));
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t ta = 0, tb = 0;  // largest |bound| so far, two at a time
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 qj = q[j & 3];
      const bool up = j < 4;
      auto part = [&](uint32_t x) { return up ? max2(x, 0u) : min2(x, 0u); };
      mma_bf16_16816(s, a[j].x, b[j].x, a[j].y, b[j].y, part(qj.x), part(qj.y));
      mma_bf16_16816(s, a[j].z, b[j].z, a[j].w, b[j].w, part(qj.z), part(qj.w));
      ta = max2(max2(ta, a[j].x & 0x7fff7fffu), max2(max2(a[j].y & 0x7fff7fffu, a[j].z & 0x7fff7fffu), a[j].w & 0x7fff7fffu));
      tb = max2(max2(tb, b[j].x & 0x7fff7fffu), max2(max2(b[j].y & 0x7fff7fffu, b[j].z & 0x7fff7fffu), b[j].w & 0x7fff7fffu));
    }
    float sa = max_nan(s[0], s[1]), sb = max_nan(s[2], s[3]);
    float ea = kGamma * norm * max_nan(bf16_lo(ta), bf16_hi(ta)), eb = kGamma * norm * max_nan(bf16_lo(tb), bf16_hi(tb));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sa = max_nan(sa, __shfl_xor_sync(0xffffffffu, sa, o));
      sb = max_nan(sb, __shfl_xor_sync(0xffffffffu, sb, o));
      ea = max_nan(ea, __shfl_xor_sync(0xffffffffu, ea, o));
      eb = max_nan(eb, __shfl_xor_sync(0xffffffffu, eb, o));
    }
    // a score whose sums may have passed fp32's range on the way is to be formed again, as one that is no number
    if (!(ea < kBounded)) sa = __uint_as_float(0x7fc00000u), ea = 0.f;
    if (!(eb < kBounded)) sb = __uint_as_float(0x7fc00000u), eb = 0.f;
    float e = fmaxf(ea, eb);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
    const int64_t unit = static_cast<int64_t>(row) * kKvHeads + g;
    float* scores = p.scores + unit * p.width;
    if (c == 0 && ia < v.count) scores[ia] = oka ? sa : __uint_as_float(kNoBlock);
    if (c == 0 && ib < v.count) scores[ib] = okb ? sb : __uint_as_float(kNoBlock);
    if (lane == 0) p.errors[unit * ((p.width + kScoreBlocks - 1) / kScoreBlocks) + blockIdx.x] = e;
  }
}

// ----------------------------------------------------------------- choice
// A block of threads per row and KV head. The MMA's scores decide all blocks but those within the error of the k-th
// largest; of these the score is formed again in two floats (products of bf16 are exact, sums are carried with their
// rounding errors: 2^-40 of the terms), and the larger ones, then the lower ones, fill what is left. They are few unless
// scores tie: up to kListed are compared with one another, more by a second radix select over both floats. Scores are held
// in shared memory as ordered words, up to kHeldWords of them (else in their place in global memory).
// Small blocks of threads for short rows: their barriers are cheap and all fit the GPU at once. Bound by barriers and round
// trips: one row of 2048 blocks 15 us, of which the k-th largest takes 3.4 and the exact scores 2; 128 rows of 32 to 256 13.
constexpr int kHeldWords = 48 * 1024, kListed = 128;
constexpr uint32_t kAbsent = 0, kChosen = 1;  // marks below any score's word
constexpr uint32_t kUnknown = 0xffffffffu;    // of a score whose sums may have left fp32's range: it is formed again in any case

// s + e += x, exactly but for e's own rounding.
__device__ __forceinline__ void add_exact(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// Lane (h = lane >> 2, c = lane & 3): the score of head h from its four lanes' 32 dims each, as t + rest, rounded into t
// first; t is NaN if a term is. With u = 2^-24 and S the sum of the terms' sizes a lane's four sums leave 36 u^2 S (eight
// terms' errors are added up in fp32), their join 66, the two joins of lanes 52 and the last rounding 2: 2^-40 S in all.
// SCALED: products of both factors times 2^-70, whose sums of 128 stay in range (2^256 becomes 2^116; what underflows is
// below 2^-70 of terms whose sum passed the range unscaled). Only the score itself then decides whether it is past fp32's.
template <bool SCALED>
__device__ __forceinline__ void exact_sum(const uint4 (&x4)[4], const uint4 (&a4)[4], const uint4 (&b4)[4], float& t, float& rest) {
  constexpr float kDown = SCALED ? 0x1p-70f : 1.f;
  float sum[4], rest_of[4], other = 0.f;  // four sums at once: each term waits for the one before
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] = rest_of[i] = 0.f;
    const uint32_t xs[4] = {x4[i].x, x4[i].y, x4[i].z, x4[i].w}, as[4] = {a4[i].x, a4[i].y, a4[i].z, a4[i].w}, bs[4] = {b4[i].x, b4[i].y, b4[i].z, b4[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = bf16_lo(xs[k]), x1 = bf16_hi(xs[k]);
      const bool up0 = x0 > 0.f, up1 = x1 > 0.f;
      add_exact(sum[i], rest_of[i], __fmul_rn(kDown * x0, kDown * (up0 ? bf16_lo(as[k]) : bf16_lo(bs[k]))));
      add_exact(sum[i], rest_of[i], __fmul_rn(kDown * x1, kDown * (up1 ? bf16_hi(as[k]) : bf16_hi(bs[k]))));
      other = fmaf(up0 ? bf16_lo(bs[k]) : bf16_lo(as[k]), 0.f, other);  // the products of 0: nothing, or NaN
      other = fmaf(up1 ? bf16_hi(bs[k]) : bf16_hi(as[k]), 0.f, other);
    }
  }
  float s = sum[0] + other, e = rest_of[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    add_exact(s, e, sum[i]);
    e = __fadd_rn(e, rest_of[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
    add_exact(s, e, s2);
    e = __fadd_rn(e, e2);
  }
  t = __fadd_rn(s, e);
  rest = __fadd_rn(__fsub_rn(s, __fsub_rn(t, __fsub_rn(t, s))), __fsub_rn(e, __fsub_rn(t, s)));
  if (!isfinite(s)) t = s;  // (s is the plain sum, infinite or NaN as the terms make it; its error is no number)
  if constexpr (SCALED) {
    t = t * 0x1p70f * 0x1p70f;
    rest = rest * 0x1p70f * 0x1p70f;
  }
  if (!isfinite(t)) rest = 0.f;
}

// A block's score for the 8 query heads at q, the largest of theirs, by one warp, as hi + lo; false if it is no finite
// fp32 number, or a head's is none at all.
__device__ __forceinline__ bool exact_score(const __nv_bfloat16* q, const __nv_bfloat16* bounds, int lane, float& hi, float& lo) {
  const uint4* qr = reinterpret_cast<const uint4*>(q + (lane >> 2) * kHeadDim) + 4 * (lane & 3);
  const uint4* up = reinterpret_cast<const uint4*>(bounds) + 4 * (lane & 3);
  const uint4* down = up + kRowValues / 8;
  uint4 x4[4], a4[4], b4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x4[i] = __ldcg(qr + i);
    a4[i] = __ldcg(up + i);
    b4[i] = __ldcg(down + i);
  }
  float t, rest;
  exact_sum<false>(x4, a4, b4, t, rest);
  if (!__all_sync(0xffffffffu, isfinite(t))) {  // a sum passed the range, at its end or on the way
    float t2, rest2;
    exact_sum<true>(x4, a4, b4, t2, rest2);
    if (!isfinite(t)) t = t2, rest = rest2;  // (the other heads' terms may be too small for the scaled form)
  }
  bool nan = t != t;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {  // the largest of the heads
    const float t2 = __shfl_xor_sync(0xffffffffu, t, o), r2 = __shfl_xor_sync(0xffffffffu, rest, o);
    nan = __shfl_xor_sync(0xffffffffu, nan ? 1 : 0, o) != 0 || nan;
    if (t2 > t || (t2 == t && r2 > rest)) t = t2, rest = r2;
  }
  hi = t;
  lo = rest;
  return !nan && isfinite(t);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) gqa_block_choose_kernel(const BlockParams p) {
  extern __shared__ uint32_t held[];
  __shared__ SelectSpace<THREADS> sp;
  __shared__ float widest[THREADS / 32];
  __shared__ int unknown_s[THREADS / 32];
  __shared__ int list[kListed], listed;
  __shared__ uint64_t listed_key[kListed];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the call's inputs are there: the score kernel let this one start behind its own wait
  RowView v = row_view(p, static_cast<int>(blockIdx.x / kKvHeads));
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t unit = blockIdx.x; unit < static_cast<int64_t>(p.rows) * kKvHeads; unit += gridDim.x) {
    const int row = static_cast<int>(unit / kKvHeads), g = static_cast<int>(unit % kKvHeads);
    if (unit != blockIdx.x) v = row_view(p, row);
    const int* table = p.block_table + static_cast<int64_t>(max(v.req, 0)) * p.width;
    const float* scores = p.scores + unit * p.width;
    uint32_t* words = p.width <= kHeldWords ? held : reinterpret_cast<uint32_t*>(p.scores + unit * p.width);
    // candidates and those of them that are kept in any case; the widest error
    int2 mine = make_int2(0, 0);
    int unknown = 0;
    float wide = 0.f;
    const int tiles = (p.width + kScoreBlocks - 1) / kScoreBlocks;
    for (int i = tid; i < (v.count + kScoreBlocks - 1) / kScoreBlocks; i += THREADS) wide = fmaxf(wide, __ldcg(p.errors + unit * tiles + i));
#pragma unroll 4
    for (int i = tid; i < v.count; i += THREADS) {
      const float s = __ldcg(scores + i);
      uint32_t x = kAbsent;
      if (__float_as_uint(s) != kNoBlock) {
        const bool fixed = i < p.keep_first || i >= v.count - p.keep_last;
        const bool number = fabsf(s) < INFINITY;
        x = fixed ? kChosen : (number ? ordered_bits(s) : kUnknown);
        ++mine.x;
        mine.y += fixed;
        unknown += !fixed && !number;
      }
      words[i] = x;
    }
    if (tid == 0) listed = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    unknown = __reduce_add_sync(0xffffffffu, unknown);
    if (lane == 0) widest[warp] = wide, unknown_s[warp] = unknown;
    mine = block_sum2<THREADS>(sp.sums, mine);  // (its barriers: the words and the widest errors are there too)
    wide = widest[lane & (THREADS / 32 - 1)];  // (a power of two of warps)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    unknown = __reduce_add_sync(0xffffffffu, lane < THREADS / 32 ? unknown_s[lane] : 0);
    const int take = min(p.top, mine.x) - mine.y;  // of the others; mine.y <= top
    const int others = mine.x - mine.y;
    const bool all = mine.x <= p.top;
    // words above `above` are chosen, below `below` not; those between, and the unknown, are to be decided
    uint32_t above = all ? kAbsent : 0xffffffffu, below = all ? kAbsent : 0xffffffffu;
    bool settled = all, again = false;
    uint64_t least = 0;
    int ties = 0;
    auto open = [&](uint32_t x) { return x > kChosen && (x == kUnknown || (x >= below && x <= above)); };
    if (!all && take > 0) {
      auto rank = [&](int k) {  // the k-th largest word
        if (THREADS == 128 && v.count <= 256) return warp_kth<8>(words, v.count, k);
        int unused = 0;
        return select_kth<THREADS, false, uint32_t>(sp, v.count, k, [&](int i) { return words[i]; }, unused);
      };
      // the unknown may come out above all others or below them: chosen for sure is what passes the (take - unknown)-th of
      // the others (the take-th with the unknown on top), and what their take-th passes is not
      const uint32_t kth = rank(take), kth_low = unknown == 0 ? kth : (take + unknown <= others ? rank(take + unknown) : kAbsent);
      if (kth != kUnknown) above = ordered_bits(__fadd_ru(ordered_float(kth), __fmul_ru(2.f, wide)));
      below = kth_low == kAbsent ? kKeyLeast : ordered_bits(__fadd_rd(ordered_float(kth_low), __fmul_rd(-2.f, wide)));
      mine = make_int2(0, 0);  // chosen by their words, to be decided
      for (int i = tid; i < v.count; i += THREADS) {
        const uint32_t x = words[i];
        if (open(x)) {
          ++mine.y;
          const int at = atomicAdd(&listed, 1);
          if (at < kListed) list[at] = i;
        } else if (x > above) {
          ++mine.x;
        }
      }
      mine = block_sum2<THREADS>(sp.sums, mine);
      const int left = take - mine.x;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(row) * kQoHeads + g * kGroup) * kHeadDim;
      auto formed = [&](int i) {  // block i's score, by a warp
        float hi, lo;
        const int64_t block = __ldcg(table + i);
        const bool number = exact_score(q, static_cast<const __nv_bfloat16*>(p.bounds) + (block * 2 * kKvHeads + g) * kHeadDim, lane, hi, lo);
        return number ? make_float2(hi, lo) : make_float2(INFINITY, 0.f);
      };
      auto key_of = [](float2 x) { return (static_cast<uint64_t>(ordered_bits(x.x)) << 32) | ordered_bits(x.y); };
      if (left >= mine.y) {
        settled = true;
      } else if (mine.y <= kListed) {
        for (int i = warp; i < mine.y; i += THREADS / 32) {
          const uint64_t k = key_of(formed(list[i]));
          if (lane == 0) listed_key[i] = k;
        }
        __syncthreads();
        if (tid < mine.y) {
          const uint64_t k = listed_key[tid];
          const int at = list[tid];
          int better = 0;
          for (int i = 0; i < mine.y; ++i) better += listed_key[i] > k || (listed_key[i] == k && list[i] < at);
          words[at] = better < left ? kChosen : kAbsent;
        }
        __syncthreads();
        settled = true;  // (none is left open)
      } else {
        again = true;
        for (int i0 = 32 * warp; i0 < v.count; i0 += THREADS) {
          const int i = i0 + lane;
          for (unsigned m = __ballot_sync(0xffffffffu, i < v.count && open(words[i])); m != 0; m &= m - 1) {
            const int at = i0 + __ffs(m) - 1;
            const float2 x = formed(at);
            if (lane == 0) p.again[unit * p.width + at] = x;
          }
        }
        __syncthreads();
        least = select_kth<THREADS, false, uint64_t>(
            sp, v.count, left, [&](int i) { return open(words[i]) ? key_of(p.again[unit * p.width + i]) : uint64_t{0}; }, ties);
      }
    }
    int* out = p.blocks + unit * p.top;
    const int chosen = all ? mine.x : p.top;
    select_in_order<THREADS, false, 1>(
        sp, v.count, ties,
        [&](int i) {
          const uint32_t x = words[i];
          if (x <= kChosen) return x == kChosen ? 2 : 0;
          if (all) return 2;
          if (!open(x)) return x > above ? 2 : 0;
          if (!again) return settled ? 2 : 0;
          const float2 y = p.again[unit * p.width + i];
          const uint64_t k = (static_cast<uint64_t>(ordered_bits(y.x)) << 32) | ordered_bits(y.y);
          return k > least ? 2 : (k == least ? 1 : 0);
        },
        [](int) { return 0; },
        [&](int i, int, int at, bool stay) {
          if (stay && at < p.top) out[at] = i;
        });
    for (int i = chosen + tid; i < p.top; i += THREADS) out[i] = -1;
    __syncthreads();
  }
}

template <int THREADS>
static cudaError_t launch_choose(const BlockParams& p, cudaStream_t stream) {
  static std::atomic<int> configured[kMaxDevices];
  const cudaError_t e = set_smem_limit_once(configured, reinterpret_cast<const void*>(gqa_block_choose_kernel<THREADS>), kHeldWords * 4);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(p.rows) * kKvHeads;
  return launch_chained(gqa_block_choose_kernel<THREADS>, dim3(units < (1 << 20) ? units : (1 << 20)), THREADS,
                        p.width <= kHeldWords ? p.width * 4 : 0, stream, 1, p);
}

cudaError_t launch_block_select(const BlockParams& p, cudaStream_t stream) {
  const dim3 grid((p.width + kScoreBlocks - 1) / kScoreBlocks, p.rows < 65535 ? p.rows : 65535);
  const cudaError_t e = launch_chained(gqa_block_score_kernel, grid, 128, 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  return p.width <= 1024 ? launch_choose<128>(p, stream) : launch_choose<512>(p, stream);
}

// ------------------------------------------------------------------ slots
// A warp per kSlotBlocks listed blocks: a lane looks a block up, then the warp writes the blocks' slots in a row. Bound by its
// launch and three dependent loads (4 to 5 us).
constexpr int kSlotThreads = 128, kSlotBlocks = 8;

__global__ void __launch_bounds__(kSlotThreads) gqa_block_slots_kernel(const BlockParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per_row = static_cast<int64_t>(p.top) * p.page_size, parts = (p.top + kSlotBlocks - 1) / kSlotBlocks;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kSlotThreads / 32);
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * (kSlotThreads / 32) + (threadIdx.x >> 5); x < p.rows * kKvHeads * parts; x += warps) {
    const int64_t unit = x / parts;
    const int j0 = static_cast<int>(x - unit * parts) * kSlotBlocks, row = static_cast<int>(unit / kKvHeads), g = static_cast<int>(unit % kKvHeads);
    const int i = lane < kSlotBlocks && j0 + lane < p.top ? __ldcg(p.blocks + unit * p.top + j0 + lane) : -1;
    const RowView v = row_view(p, row);
    int block = -1, tokens = 0;
    if (i >= 0 && i < v.count) {
      block = __ldcg(p.block_table + static_cast<int64_t>(v.req) * p.width + i);
      tokens = static_cast<unsigned>(block) < static_cast<unsigned>(p.num_blocks) ? min(p.page_size, v.n - i * p.page_size) : 0;
    }
    int* slots = p.slots + (static_cast<int64_t>(g) * p.rows + row) * per_row + static_cast<int64_t>(j0) * p.page_size;
    const int count = min(kSlotBlocks, p.top - j0) * p.page_size;  // at most 2^31 - 1: rows * top * page_size is
    for (unsigned z0 = 0; z0 < static_cast<unsigned>(count); z0 += 32) {
      const int z = static_cast<int>(min(z0 + lane, static_cast<unsigned>(count) - 1)), j = z / p.page_size, t = z - j * p.page_size;
      const int b = __shfl_sync(0xffffffffu, block, j), n = __shfl_sync(0xffffffffu, tokens, j);
      if (z0 + lane < static_cast<unsigned>(count)) slots[z] = t < n ? b * p.page_size + t : -1;
    }
  }
}

cudaError_t launch_block_slots(const BlockParams& p, int sm_count, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(p.rows) * kKvHeads * ((p.top + kSlotBlocks - 1) / kSlotBlocks);
  const int64_t blocks = (warps + kSlotThreads / 32 - 1) / (kSlotThreads / 32), most = 16 * static_cast<int64_t>(sm_count);
  return launch_chained(gqa_block_slots_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), kSlotThreads, 0, stream, 1, p);
}

}  // namespace gqa
