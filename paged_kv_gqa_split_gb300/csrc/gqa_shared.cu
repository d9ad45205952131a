// Decode of a batch whose sequences share prefixes: what a sequence reads is its group's prefix, then its own tokens.
//   out = (sum over prefix and own tokens of 2^(s - m) v) / (the same sum of 2^(s - m))
// is formed from parts: the prefix's (computed here, once a group for all its sequences), the own tokens' (the split
// decode, kFormParts, which fills the SMs as the prefix pass leaves them) and their join by log-sum-exp weights.
//
// These kernels start while the ones before them on the stream end, and what those wrote is read with ld.cg, behind the
// wait: the non-coherent load is for words that no kernel under way writes.
#include <cuda_runtime.h>

#include "gqa_common.cuh"
#include "gqa_kernels.h"
#include "gqa_tc.cuh"

namespace gqa {

// Group of sequence b, or -1: the largest g with group_indptr[g] <= b, if it reaches past b.
__device__ __forceinline__ int group_of(const SharedParams& p, int b) {
  int lo = 0, hi = p.groups;  // group_indptr[lo] <= b wherever any entry is
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(p.group_indptr + mid) <= b) lo = mid; else hi = mid;
  }
  return p.groups > 0 && __ldcg(p.group_indptr + lo) <= b && b < __ldcg(p.group_indptr + lo + 1) ? lo : -1;
}

// First prefix token of group g and their count, cut to the table.
__device__ __forceinline__ int prefix_range(const SharedParams& p, int g, int& first) {
  first = max(0, min(__ldcg(p.prefix_indptr + g), p.prefix_count));
  return max(0, min(__ldcg(p.prefix_indptr + g + 1), p.prefix_count) - first);
}

// ----------------------------------------------------------------- prefix
// Query rows of one KV head are its 8 query heads of up to 32 sequences of a group: two tiles of 128 rows, a row a lane
// of tensor memory. A unit is these rows and the group's prefix, walked in steps of 128 tokens: S = Q K^T (M = 128,
// N = 128 tokens, 8 MMAs of K = 16) lands in tensor memory, a thread per row turns it into probabilities that overwrite
// it there, and O += P V (8 MMAs, P read from tensor memory) accumulates beside it; while one tile is in its softmax the
// tensor cores do the other's MMAs. Rows without a sequence are zeros; with 16 sequences or fewer there is one tile.
//
// The steps of all units (groups, then row tiles, then KV heads) are one line, cut into equal runs, one a CTA, one CTA
// an SM: prefixes of any number and length fill the GPU. What a CTA has of a unit is a piece. Its outputs and LSE go out
// in fp32, as blocks of [128 dims][8 heads] a sequence: the piece that begins the unit to the sequence's own block, one
// that goes on with it to the CTA's (a CTA has one such piece at most, its first).
//
// Pages are single tokens in any order, so a token's 256 bytes of a KV head are gathered by 16-byte cp.async, written
// where the 128-byte swizzle wants them; four warps keep five 32 KB slots (128 tokens of K or V) in flight. An FP8
// cache's codes go through a ring of their own and become fp16 (exact) on the way to three such slots; a token's K
// scale is taken on its score, its V scale on its probability (over a running power of two), Q is fp16 times a power of
// two a row, as in the decode.
//
// The running maximum moves only when a row's scores pass it by 2^8, so O is seldom rescaled; fp16 probabilities are held
// times 2^7. Every wait is bounded: on a timeout the CTA flags the device error word, waits for its copies and MMAs in
// flight, frees tensor memory and leaves.
constexpr int kStep = 128, kSeqTile = 16, kUnitSeqs = 2 * kSeqTile;
constexpr int kPreThreads = 512, kCopyWarps = 4, kMmaWarp = 4, kRowWarp = 8;  // two MMA warps; from 8 on two warpgroups of rows
constexpr int kRowRegs = 200, kOtherRegs = 56;
static_assert(256 * kRowRegs + 256 * kOtherRegs <= 65536, "register split");
constexpr int kHalfTile = 128 * 128, kSlotBytes = 2 * kHalfTile;  // 128 rows of 64 values; of 128
constexpr int kInfo = 4;  // steps whose masks and scales are held: the copies are at most three ahead of the softmax
constexpr float kMoveBy = 8.f;

template <bool F8>
struct PrefixCfg {
  static constexpr int kSlots = F8 ? 3 : 5;
  static constexpr int kRaw = F8 ? 3 : 0;  // slots of codes, 16 KB each
  static constexpr float kShift = F8 ? 7.f : 0.f;
  static constexpr int kSlotOff = 2 * kSlotBytes;  // behind the two query tiles
  static constexpr int kRawOff = kSlotOff + kSlots * kSlotBytes;
  static constexpr int kRawBytes = kStep * kHeadDim + 2 * kStep * 4;  // codes; with K's the scales of K and V
  static constexpr int kMaskOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kScaleOff = kMaskOff + kInfo * 16;                   // K, then V scales of a step; their largest, a warp's each
  static constexpr int kTopOff = kScaleOff + (F8 ? kInfo * 2 * kStep * 4 : 0);
  static constexpr int kRowOff = kTopOff + (F8 ? kInfo * 16 : 0);           // the queries' factors
  static constexpr int kBarOff = kRowOff + (F8 ? 256 * 4 : 0);
  // barriers: slots full and free; queries written, S and O there, the halves of P written, a tile each; all done
  static constexpr int kFull = 0, kFree = kSlots, kQ = 2 * kSlots, kS = kQ + 2, kO = kS + 2, kP = kO + 2, kDone = kP + 4, kBars = kDone + 1;
  static constexpr int kWordOff = kBarOff + kBars * 8;
  static constexpr int kBytes = kWordOff + 16 + 1024;  // the base is rounded up to 1024 bytes (swizzle atoms)
  static_assert(kBytes <= 227 * 1024, "prefix pass exceeds shared memory");
};

// Steps of group g's units together.
__device__ __forceinline__ int64_t group_steps(const SharedParams& p, int g, int& tiles, int& seq0, int& members) {
  int first;
  tiles = (prefix_range(p, g, first) + kStep - 1) / kStep;
  seq0 = max(0, min(__ldcg(p.group_indptr + g), p.batch));
  members = max(0, min(__ldcg(p.group_indptr + g + 1), p.batch) - seq0);
  return static_cast<int64_t>((members + kUnitSeqs - 1) / kUnitSeqs) * kKvHeads * tiles;
}

__host__ __device__ __forceinline__ int64_t steps_per_cta(int64_t total, int ctas) {
  return total > ctas ? (total + ctas - 1) / ctas : 1;
}

// A role's walk over the pieces of its CTA.
struct Walk {
  int64_t x, end, group_end;  // next step, the run's end, the end of group g's steps
  int g, tiles, seq0, members, first, n;  // the group: steps a unit, sequences, prefix tokens
  int head, row0, step0, steps;           // the piece: KV head, first sequence (within the group), steps

  __device__ __forceinline__ bool next(const SharedParams& p) {
    if (x >= end) return false;
    while (x >= group_end) {
      ++g;
      group_end += group_steps(p, g, tiles, seq0, members);
    }
    n = prefix_range(p, g, first);
    const int64_t per_group = static_cast<int64_t>((members + kUnitSeqs - 1) / kUnitSeqs) * kKvHeads * tiles;
    const int64_t at = x - (group_end - per_group);
    const int unit = static_cast<int>(at / tiles);
    step0 = static_cast<int>(at - static_cast<int64_t>(unit) * tiles);
    steps = static_cast<int>(min(static_cast<int64_t>(tiles - step0), end - x));
    head = unit % kKvHeads;
    row0 = unit / kKvHeads * kUnitSeqs;
    x += steps;
    return true;
  }
  __device__ __forceinline__ int seqs(int a) const { return max(0, min(members - row0 - a * kSeqTile, kSeqTile)); }
};

template <bool F8>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  return F8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}

template <bool F8>
__global__ void __launch_bounds__(kPreThreads, 1) gqa_shared_prefix_kernel(const SharedParams p) {
  using C = PrefixCfg<F8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_s = reinterpret_cast<volatile int*>(sm + C::kWordOff + 4);
  auto bar = [&](int i) { return base + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  __shared__ int64_t warp_steps[kPreThreads / 32], begin_s;
  __shared__ int begin_g;
  pdl_wait();
  pdl_launch_dependents();  // the own tokens' decode: by now all that it reads is there

  // total steps, then where this CTA's run begins
  Walk walk;
  {
    int64_t mine = 0;
    int t, s0, m;
    for (int g = tid; g < p.groups; g += kPreThreads) mine += group_steps(p, g, t, s0, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) warp_steps[warp] = mine;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kPreThreads / 32; ++w) total += warp_steps[w];
    const int64_t run = steps_per_cta(total, gridDim.x);
    walk.x = run * blockIdx.x;
    walk.end = min(walk.x + run, total);
    int64_t carry = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kPreThreads) {
      const int g = g0 + tid;
      const int64_t steps = g < p.groups ? group_steps(p, g, t, s0, m) : 0;
      int64_t upto = steps;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      __syncthreads();
      if (lane == 31) warp_steps[warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += warp_steps[w];
      upto += carry;
      if (g < p.groups) {
        if (blockIdx.x == 0) p.group_start[g + 1] = upto;
        if (upto - steps <= walk.x && walk.x < upto) begin_g = g, begin_s = upto;
      }
      for (int w = 0; w < kPreThreads / 32; ++w) carry += warp_steps[w];
    }
    if (blockIdx.x == 0 && tid == 0) p.group_start[0] = 0;
    __syncthreads();
    if (walk.x >= total) return;
    walk.g = begin_g;
    walk.group_end = begin_s;
    group_steps(p, walk.g, walk.tiles, walk.seq0, walk.members);
  }

  if (tid == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      int count = 1;  // S, O: a commit
      if (i < C::kFree) count = F8 ? kCopyWarps : kCopyWarps * 32 + kCopyWarps;
      else if (i < C::kQ || i == C::kDone) count = 2;  // a commit of each MMA warp
      else if (i < C::kS || (i >= C::kP && i < C::kDone)) count = 4;  // warps of a tile's rows
      mbar_init(bar(i), count);
    }
    *abort_s = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) tc_alloc(base + C::kWordOff, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::kWordOff);
  auto wait = [&](int i, uint32_t parity, int bit) {
    return __all_sync(0xffffffffu, tc_wait_limited(bar(i), parity, abort_s, p.err, bit, p.wait_limit_ns)) != 0;
  };

  if (warp < kRowWarp) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp < kCopyWarps) {
      // ------------------------------------------------------------- copies
      const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
      const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
      int s = 0, info = 0, filled = 0;
      uint32_t ph = 1;  // parity of the slot's previous release
      bool good = true;
      if constexpr (!F8) {
        const int c = lane & 15;  // 16-byte column of a token's 256 bytes
        const uint32_t to = (c >> 3) * kHalfTile;
        while (good && walk.next(p)) {
          int t = walk.step0 * kStep + 32 * warp + lane;
          int id = t < walk.n ? __ldcg(p.prefix_indices + walk.first + t) : -1;
#pragma unroll 1
          for (int j = 0; j < walk.steps && good; ++j) {
            const bool live = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages);
            const unsigned mask = __ballot_sync(0xffffffffu, live);
            const int page = live ? id : 0;
            t += kStep;
            id = t < walk.n ? __ldcg(p.prefix_indices + walk.first + t) : -1;  // of the next step, behind this one's copies
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              if (filled >= C::kSlots) good = wait(C::kFree + s, ph, kErrTimeoutEmpty);
              if (!good) break;
              ++filled;
              const uint8_t* from = (kv == 0 ? kc : vc) + walk.head * (kHeadDim * 2) + 16 * c;
              const uint32_t slot = base + C::kSlotOff + s * kSlotBytes + to;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + (lane >> 4);
                const int64_t pg = __shfl_sync(0xffffffffu, page, r);
                cp_async_16(sw128(slot, 32 * warp + r, c & 7), from + pg * kPageBytes, (mask >> r) & 1u ? 16u : 0u);
              }
              cp_async_arrive(bar(C::kFull + s));
              if (lane == 0) {
                if (kv == 0) reinterpret_cast<volatile unsigned*>(sm + C::kMaskOff)[4 * info + warp] = mask;
                mbar_arrive(bar(C::kFull + s));
              }
              if (++s == C::kSlots) {
                s = 0;
                ph ^= 1;
              }
            }
            info = (info + 1) % kInfo;
          }
        }
      } else {
        // A thread converts the chunks that it copied itself: row r = 4 i + lane / 8 of the warp's 32, 16 codes at lane % 8.
        const int c = lane & 7;
        constexpr int kRow = kKvHeads * kHeadDim + 4 * kKvHeads;
        Walk ahead = walk;  // the copies' walk, kRaw - 1 slots ahead of the conversion's
        bool more = ahead.next(p);
        int aj = 0, akv = 0, as = 0, page = 0;
        unsigned mask = 0;
        auto copy = [&]() {
          if (more) {
            if (akv == 0) {
              const int t = (ahead.step0 + aj) * kStep + 32 * warp + lane;
              const int id = t < ahead.n ? __ldcg(p.prefix_indices + ahead.first + t) : -1;
              const bool live = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages);
              mask = __ballot_sync(0xffffffffu, live);
              page = live ? id : 0;
            }
            const uint8_t* from = akv == 0 ? kc : vc;
            const uint32_t slot = base + C::kRawOff + as * C::kRawBytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              const int64_t pg = __shfl_sync(0xffffffffu, page, r);
              cp_async_16(slot + (32 * warp + r) * kHeadDim + 16 * c, from + pg * kRow + ahead.head * kHeadDim + 16 * c,
                          (mask >> r) & 1u ? 16u : 0u);
            }
            if (akv == 0) {  // V's scales with K's: the softmax reads both when the scores are there
              const int64_t at = static_cast<int64_t>(page) * kRow + kKvHeads * kHeadDim + 4 * ahead.head;
              const uint32_t to = slot + kStep * kHeadDim + 4 * (32 * warp + lane);
              cp_async_4(to, kc + at, (mask >> lane) & 1u ? 4u : 0u);
              cp_async_4(to + 4 * kStep, vc + at, (mask >> lane) & 1u ? 4u : 0u);
            }
            as = as + 1 == C::kRaw ? 0 : as + 1;
            akv ^= 1;
            if (akv == 0 && ++aj == ahead.steps) {
              aj = 0;
              more = ahead.next(p);
            }
          }
          cp_async_commit();  // one group a call, even when empty
        };
#pragma unroll 1
        for (int i = 0; i < C::kRaw - 1; ++i) copy();
        int rs = 0;
        while (good && walk.next(p)) {
#pragma unroll 1
          for (int j = 0; j < walk.steps && good; ++j) {
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              __syncwarp();
              copy();
              cp_async_wait<C::kRaw - 1>();
              if (filled >= C::kSlots) good = wait(C::kFree + s, ph, kErrTimeoutEmpty);
              if (!good) break;
              ++filled;
              const uint32_t slot = base + C::kSlotOff + s * kSlotBytes + (c >> 2) * kHalfTile;
              const uint32_t codes = base + C::kRawOff + rs * C::kRawBytes;
#pragma unroll 4
              for (int i = 0; i < 8; ++i) {
                const int r = 32 * warp + 4 * i + (lane >> 3);
                uint32_t x[4], y[8];
                ld_shared_u4(codes + r * kHeadDim + 16 * c, x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  y[2 * k] = cvt_e4m3x2_f16x2(x[k]);
                  y[2 * k + 1] = cvt_e4m3x2_f16x2(x[k] >> 16);
                }
                st_shared_u4(sw128(slot, r, 2 * (c & 3)), y[0], y[1], y[2], y[3]);
                st_shared_u4(sw128(slot, r, 2 * (c & 3) + 1), y[4], y[5], y[6], y[7]);
              }
              if (kv == 0) {
                const uint32_t at = codes + kStep * kHeadDim + 4 * (32 * warp + lane);
                const float sk = ld_shared_f32(at), sv = ld_shared_f32(at + 4 * kStep);
                volatile float* scales = reinterpret_cast<volatile float*>(sm + C::kScaleOff) + 2 * info * kStep + 32 * warp + lane;
                scales[0] = sk;
                scales[kStep] = sv;
                float top = fabsf(sv) < INFINITY ? fabsf(sv) : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (lane == 0) reinterpret_cast<volatile float*>(sm + C::kTopOff)[4 * info + warp] = top;
                const int t = (walk.step0 + j) * kStep + 32 * warp + lane;
                const int id = t < walk.n ? __ldcg(p.prefix_indices + walk.first + t) : -1;
                const unsigned mk = __ballot_sync(0xffffffffu, static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages));
                if (lane == 0) reinterpret_cast<volatile unsigned*>(sm + C::kMaskOff)[4 * info + warp] = mk;
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::kFull + s));
              rs = rs + 1 == C::kRaw ? 0 : rs + 1;
              if (++s == C::kSlots) {
                s = 0;
                ph ^= 1;
              }
            }
            info = (info + 1) % kInfo;
          }
        }
      }
      cp_async_commit();
      cp_async_wait<0>();  // no copy may still be writing when the CTA leaves
    } else if (warp < kMmaWarp + 2) {
      // --------------------------------------------------------------- MMAs
      // tile a: the whole warp walks (warp-uniform operands), one elected lane issues
      const int a = static_cast<int>(uniform(warp - kMmaWarp));
      const uint32_t ub = uniform(base), ut = uniform(tmem);
      constexpr uint32_t idesc_s = F8 ? tc_idesc_f16(128, kStep, false, false) : tc_idesc_bf16(128, kStep, false, false);
      constexpr uint32_t idesc_o = F8 ? tc_idesc_f16(128, kHeadDim, false, true) : tc_idesc_bf16(128, kHeadDim, false, true);
      const uint64_t dq0 = tc_sdesc(ub + a * kSlotBytes, 16, 1024, kSwizzle128B);
      const uint64_t dk0 = tc_sdesc(ub + C::kSlotOff, 16, 1024, kSwizzle128B);
      // V as B: N = 128 dims in two regions (LBO), K = tokens in 8-row groups (SBO)
      const uint64_t dv0 = tc_sdesc(ub + C::kSlotOff, kHalfTile, 1024, kSwizzle128B);
      const uint32_t s_col = ut + 128 * a, o_col = ut + 256 + 128 * a;
      auto ubar = [&](int i) { return ub + C::kBarOff + 8u * static_cast<uint32_t>(i); };
      int s = 0;
      uint32_t ph = 0, np = 0, nq = 0;
      bool good = true;
      auto advance = [&]() {
        if (++s == C::kSlots) {
          s = 0;
          ph ^= 1;
        }
      };
      while (good && walk.next(p)) {
        const int steps = static_cast<int>(uniform(walk.steps));
        const bool mine = uniform(walk.seqs(a)) > 0;
        if (mine) good = wait(C::kQ + a, nq++ & 1, kErrTimeoutFull);
        int vs = 0;
#pragma unroll 1
        for (int j = 0; j <= steps && good; ++j) {
          // O += P(j - 1) V(j - 1) behind S(j) = Q K(j) in the slots' order K(0) V(0) K(1) ..., so V's slot is the last one
          int v_slot = vs;
          const bool have_v = j > 0;
          if (have_v) {
            good = wait(C::kFull + s, ph, kErrTimeoutFull);
            v_slot = s;
            if (!good) break;
            advance();
          }
          const int k_slot = s;
          if (j < steps) {
            good = wait(C::kFull + s, ph, kErrTimeoutFull);
            if (!good) break;
          }
          if (!F8) fence_proxy_async_smem();  // the copies' writes, seen behind the barrier, for the MMAs
          if (have_v && mine) {
            good = wait(C::kP + 2 * a, np & 1, kErrTimeoutFull);
            if (!good) break;
            tc_fence_after();
            const uint64_t dv = dv0 + v_slot * (kSlotBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, kk ? 1u : (j > 1 ? 1u : 0u));
            good = wait(C::kP + 2 * a + 1, np & 1, kErrTimeoutFull);
            if (!good) break;
            ++np;
            tc_fence_after();
#pragma unroll
            for (int kk = 4; kk < 8; ++kk) tc_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, 1u);
          }
          if (j < steps && mine) {
            const uint64_t dk = dk0 + k_slot * (kSlotBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_bf16_warp(s_col, dq0 + (((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4),
                               dk + (((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4), idesc_s, kk ? 1u : 0u);
            tc_commit_warp(ubar(C::kS + a));
          }
          if (have_v) {
            tc_commit_warp(ubar(C::kFree + v_slot));
            if (mine && j == steps) tc_commit_warp(ubar(C::kO + a));
          }
          if (j < steps) {
            tc_commit_warp(ubar(C::kFree + k_slot));
            advance();
          }
        }
      }
      tc_commit_warp(ubar(C::kDone));  // every MMA done before tensor memory is freed
      __syncwarp();
    }
    __syncwarp();
  } else {
    // -------------------------- a warpgroup of rows: tile a, row 32 wq + lane
    setmaxnreg_inc<kRowRegs>();
    const int a = (warp - kRowWarp) >> 2, wq = warp & 3, t = 32 * wq + lane;
    const uint32_t quarter = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t s_col = tmem + quarter + 128 * a, o_col = tmem + quarter + 256 + 128 * a;
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes to the queries
    uint32_t scored = 0, units = 0, info = 0;
    bool good = true;
    while (good && walk.next(p)) {
      const int seqs = walk.seqs(a);
      if (seqs == 0) {
        info = (info + walk.steps) % kInfo;
        continue;
      }
      // the queries: sequence i's 8 rows are 2 KB in a row, 16 bytes a thread
      const int seq = walk.seq0 + walk.row0 + a * kSeqTile;
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         (static_cast<int64_t>(seq) * kQoHeads + walk.head * kGroup) * kHeadDim) + t;
      const uint32_t to = base + a * kSlotBytes + ((t & 15) >> 3) * kHalfTile;
#pragma unroll 4
      for (int i = 0; i < kSeqTile; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i < seqs) x = __ldcg(from + i * (kQoHeads * kHeadDim / 8));
        x = make_uint4(x.x ^ sign, x.y ^ sign, x.z ^ sign, x.w ^ sign);
        if constexpr (F8) {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float lo = fabsf(bf16_lo(w[k])), hi = fabsf(bf16_hi(w[k]));
            top = fmaxf(top, fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f));
          }
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = top > 0.f ? max(1, min(253, 127 + 13 + 127 - static_cast<int>(__float_as_uint(top) >> 23))) : 127;
          const float f = __uint_as_float(static_cast<uint32_t>(e) << 23);
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = pack_f16(bf16_lo(w[k]) * f, bf16_hi(w[k]) * f);
          x = make_uint4(y[0], y[1], y[2], y[3]);
          if ((t & 15) == 0) reinterpret_cast<volatile float*>(sm + C::kRowOff)[128 * a + 8 * i + (t >> 4)] = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        }
        st_shared_u4(sw128(to, 8 * i + (t >> 4), t & 7), x.x, x.y, x.z, x.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kQ + a));
      float sc = fabsf(p.scale_log2);
      if constexpr (F8) {
        asm volatile("bar.sync %0, 128;" ::"r"(1 + a) : "memory");
        sc *= reinterpret_cast<volatile float*>(sm + C::kRowOff)[128 * a + t];
      }
      sc = fmaxf(sc, 1e-37f);  // > 0: -inf * sc stays -inf
      float m = -INFINITY, cv = 0.f;
      uint64_t l2 = 0;
#pragma unroll 1
      for (int j = 0; j < walk.steps; ++j) {
        good = wait(C::kS + a, scored & 1, kErrTimeoutFull);
        if (!good) break;
        ++scored;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(s_col + 32 * c, s + 32 * c);
        tc_wait_ld();
        if constexpr (F8) {
          const uint32_t scales = base + C::kScaleOff + info * 2 * kStep * 4;
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            uint32_t x[4];
            ld_shared_u4(scales + 4 * c, x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[c + k] = __float_as_uint(__uint_as_float(s[c + k]) * __uint_as_float(x[k]));
          }
        }
        uint32_t w[4];
        ld_shared_u4(base + C::kMaskOff + 16 * info, w[0], w[1], w[2], w[3]);
        if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (((w[c >> 5] >> (c & 31)) & 1u) == 0) s[c] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 32; ++k)
          mx[k & 3] = max3(mx[k & 3], max3(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1]), __uint_as_float(s[4 * k + 2])),
                           __uint_as_float(s[4 * k + 3]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;
        const bool move = top > m + kMoveBy;
        float cv_new = cv, iv = 1.f;
        if constexpr (F8) {
          uint32_t x[4];
          ld_shared_u4(base + C::kTopOff + 16 * info, x[0], x[1], x[2], x[3]);
          const float vm = fminf(fmaxf(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]))), 0x1p126f);
          cv_new = fmaxf(cv, vm > 0.f ? pow2_ceil(fmaxf(vm, 0x1p-126f)) : 0.f);
          iv = cv_new > 0.f ? pow2_recip(cv_new) : 0.f;
        }
        if (__any_sync(0xffffffffu, move || cv_new != cv)) {
          const float alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2(m - top));
          if (move) m = top;
          float lo, hi;
          unpack2(l2, lo, hi);
          l2 = pack2(lo * alpha, hi * alpha);
          if (j > 0) {  // the commit that signalled S also covers the previous step's O
            const float beta = F8 ? alpha * (cv * iv) : alpha;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tc_ld16(o_col + 16 * c, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * beta);
              tc_st16(o_col + 16 * c, o);
            }
          }
          cv = cv_new;
        }
        const float off = m == -INFINITY ? 0.f : C::kShift - m;
        const uint64_t sc2 = pack2(sc, sc), off2 = pack2(off, off);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
          const uint32_t vscales = base + C::kScaleOff + (info * 2 + 1) * kStep * 4 + 256 * half;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float x0, x1;
            unpack2(fma2(pack2(__uint_as_float(s[64 * half + 2 * k]), __uint_as_float(s[64 * half + 2 * k + 1])), sc2, off2), x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            l2 = add2(l2, pack2(x0, x1));
            if constexpr (F8) {
              x0 *= ld_shared_f32(vscales + 8 * k) * iv;
              x1 *= ld_shared_f32(vscales + 8 * k + 4) * iv;
            }
            pk[k] = pack_p<F8>(x0, x1);
          }
          tc_st32(s_col + 32 * half, pk);  // over scores that have been read
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kP + 2 * a + half));  // half of the tokens: the MMAs may start on it
        }
        info = (info + 1) % kInfo;
      }
      if (!good) break;
      good = wait(C::kO + a, units++ & 1, kErrTimeoutFull);
      if (!good) break;
      tc_fence_after();
      float l, hi;
      unpack2(l2, l, hi);
      l += hi;
      const float inv = l == 0.f ? 0.f : (F8 ? cv : 1.f) / l;
      const int i = t >> 3, h = t & 7;
      const bool begins = walk.step0 == 0;
      const int64_t block = begins ? static_cast<int64_t>(seq + i) * kKvHeads + walk.head
                                   : static_cast<int64_t>(p.batch) * kKvHeads + static_cast<int64_t>(blockIdx.x) * kUnitSeqs + a * kSeqTile + i;
      float* po = p.part_o + block * (kHeadDim * kGroup) + h;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tc_ld32(o_col + 32 * c, o);
        tc_wait_ld();
        if (i < seqs)
#pragma unroll
          for (int k = 0; k < 32; ++k) po[(32 * c + k) * kGroup] = __uint_as_float(o[k]) * inv;
      }
      if (i < seqs) p.part_lse[block * kGroup + h] = l == 0.f ? -INFINITY : m - C::kShift + log2f(l);
      tc_fence_before();
    }
  }
  if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    if (lane == 0) drain_wait(bar(C::kDone), 0);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- join
// A block per sequence and KV head, a thread per dim. The parts are taken 16 at a time: a thread per part and head finds
// the part and its LSE, their largest gives the weights 2^(LSE - max), and every thread sums its dim of the parts, whose
// loads do not depend on one another. Bound by two round trips of loads, and by 4 KB a part.
constexpr int kJoinParts = 16;

__global__ void __launch_bounds__(kHeadDim) gqa_shared_join_kernel(const SharedParams p) {
  __shared__ float lse_s[kJoinParts][kGroup];
  __shared__ __align__(16) float weight_s[kJoinParts][kGroup];
  __shared__ int64_t part_s[kJoinParts];
  constexpr int kPart = kHeadDim * kGroup;
  const int tid = threadIdx.x, g = blockIdx.x % kKvHeads;
  // What the call's inputs tell is read ahead of the wait: the kernels before this one do not write it. Steps before
  // each group and in all, where a thread a group can count them; else the prefix pass has left them.
  const bool few = p.groups <= kHeadDim;
  __shared__ int64_t start_s[kHeadDim + 1];
  if (few && p.pre_ctas > 0) {
    int t, s0, m;
    int64_t upto = tid < p.groups ? group_steps(p, tid, t, s0, m) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if ((tid & 31) >= o) upto += up;
    }
    if ((tid & 31) == 31) part_s[tid >> 5] = upto;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) upto += part_s[w];
    start_s[tid + 1] = upto;
    if (tid == 0) start_s[0] = 0;
    __syncthreads();
  } else if (!few) {
    pdl_wait();
  }
  const int total = max(0, min(__ldcg(p.kv_indptr + p.batch), p.index_count));
  bool waited = false;
  for (int b = blockIdx.x / kKvHeads; b < p.batch; b += gridDim.x / kKvHeads) {
    // pieces of the prefix: the first in the sequence's block, the others in their CTA's
    int pre = 0, own = 0, cta0 = 0, local = 0;
    const int lo = max(0, min(__ldcg(p.kv_indptr + b), total)), hi = min(__ldcg(p.kv_indptr + b + 1), total);
    const int group = p.pre_ctas > 0 ? group_of(p, b) : -1;
    if (group >= 0) {
      int tiles, seq0, members;
      group_steps(p, group, tiles, seq0, members);
      if (tiles > 0) {
        const int64_t run = steps_per_cta(few ? start_s[p.groups] : __ldcg(p.group_start + p.groups), p.pre_ctas);
        const int64_t first = (few ? start_s[group] : __ldcg(p.group_start + group)) + (static_cast<int64_t>((b - seq0) / kUnitSeqs) * kKvHeads + g) * tiles;
        cta0 = static_cast<int>(first / run);
        pre = min(static_cast<int>((first + tiles - 1) / run), p.pre_ctas - 1) - cta0 + 1;
        local = (b - seq0) % kUnitSeqs;
      }
    }
    SeqSplit sp{0, 0, 0};
    if (hi > lo) {
      sp = seq_split(make_plan(total, p.plan), lo, hi);
      own = static_cast<int>(sp.last_cta - sp.first_cta) + 1;
    }
    if (!waited) pdl_wait();
    waited = true;
    auto part_of = [&](int i) -> int64_t {
      if (i < pre) return i == 0 ? static_cast<int64_t>(b) * kKvHeads + g : static_cast<int64_t>(p.batch) * kKvHeads + (cta0 + i) * kUnitSeqs + local;
      i -= pre;
      const int64_t sid = own == 1 ? p.whole_base + b : slot_id(sp.first_cta + i, i == 0 ? sp.first_slot : 0);
      return p.own_base + sid * kKvHeads + g;
    };
    float m[8], den[8], acc[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) m[h] = -INFINITY, den[h] = acc[h] = 0.f;
    for (int i0 = 0; i0 < pre + own; i0 += kJoinParts) {
      const int n = min(kJoinParts, pre + own - i0);
      const int i = tid >> 3, h = tid & 7;
      __syncthreads();  // the parts before have been read
      float l = -INFINITY;
      if (i < n) {
        const int64_t part = part_of(i0 + i);
        l = __ldcg(p.part_lse + part * kGroup + h);
        if (h == 0) part_s[i] = part;
      }
      lse_s[i][h] = l;
      __syncthreads();
      float top = -INFINITY;  // of head h over these parts (NaN aside: it goes into its own part's weight)
#pragma unroll
      for (int k = 0; k < kJoinParts; ++k) top = fmaxf(top, lse_s[k][h]);
      // head h's running maximum is the same in every thread that holds it
      float mh = m[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) mh = h == k ? m[k] : mh;
      const float mn = fmaxf(mh, top);
      weight_s[i][h] = ex2(l - (mn == -INFINITY ? 0.f : mn));
      // every thread: all heads' new maxima, and what was summed under the old ones
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = fmaxf(m[k], __shfl_sync(0xffffffffu, top, k));
        const float sc = ex2(m[k] - (t == -INFINITY ? 0.f : t));
        m[k] = t;
        den[k] *= sc;
        acc[k] *= sc;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float4* o = reinterpret_cast<const float4*>(p.part_o + part_s[k] * kPart + tid * kGroup);
        const float4 oa = __ldcg(o), ob = __ldcg(o + 1);
        const float4 wa = *reinterpret_cast<const float4*>(weight_s[k]), wb = *reinterpret_cast<const float4*>(weight_s[k] + 4);
        const float o8[8] = {oa.x, oa.y, oa.z, oa.w, ob.x, ob.y, ob.z, ob.w}, w8[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          den[e] += w8[e];
          acc[e] += w8[e] * o8[e];
        }
      }
    }
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(b) * kQoHeads + g * kGroup) * kHeadDim + tid;
#pragma unroll
    for (int h = 0; h < 8; ++h) ob[h * kHeadDim] = __float2bfloat16_rn(den[h] == 0.f ? 0.f : acc[h] / den[h]);
    if (p.lse != nullptr && tid < kGroup) {
      float mm = m[0], dd = den[0];
#pragma unroll
      for (int h = 1; h < 8; ++h)
        if (tid == h) mm = m[h], dd = den[h];
      p.lse[static_cast<int64_t>(b) * kQoHeads + g * kGroup + tid] = dd == 0.f ? -INFINITY : mm + log2f(dd);
    }
  }
}

template <bool F8>
static cudaError_t launch_prefix(const SharedParams& p, cudaStream_t stream) {
  static std::atomic<int> configured[kMaxDevices];
  const cudaError_t e = set_smem_limit_once(configured, reinterpret_cast<const void*>(gqa_shared_prefix_kernel<F8>), PrefixCfg<F8>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_chained(gqa_shared_prefix_kernel<F8>, dim3(p.pre_ctas), kPreThreads, PrefixCfg<F8>::kBytes, stream, 1, p);
}

int shared_prefix_blocks(int batch, int ctas) { return batch * kKvHeads + ctas * kUnitSeqs; }

cudaError_t launch_shared(const SharedParams& p, const DecodeParams& own, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.pre_ctas > 0) e = p.fp8 ? launch_prefix<true>(p, stream) : launch_prefix<false>(p, stream);
  if (e != cudaSuccess) return e;
  e = launch_decode_lsu_form(kFormParts, p.fp8 != 0, own, own.plan.tier1_ctas + own.plan.tier2_ctas, stream,
                             p.pre_ctas > 0 ? kLaunchPdl : kLaunchPlain);
  if (e != cudaSuccess) return e;
  const int grid = p.batch < (1 << 16) ? p.batch : (1 << 16);
  return launch_chained(gqa_shared_join_kernel, dim3(grid * kKvHeads), kHeadDim, 0, stream, 1, p);
}

}  // namespace gqa
