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
// Query rows of one KV head are its 8 query heads of up to 64 sequences of a group. A pair of CTAs takes them as two tiles
// of 256 rows (128 a CTA, 16 sequences, a row a lane of tensor memory) and walks the group's prefix in steps of 128 tokens:
// S = Q K^T (M = 256, N = 128 tokens, 8 MMAs of K = 16) lands in tensor memory, a thread per row turns it into
// probabilities that overwrite it there, and O += P V (8 MMAs, P read from tensor memory) accumulates beside it. The two
// tiles alternate: while one is in its softmax the tensor cores do the other's MMAs. Rows without a sequence are zeros;
// with 32 sequences or fewer there is one tile.
//
// A unit is these rows and the prefix. The steps of all units (groups, then 64 sequences at a time, then KV heads) are one
// line, cut into equal runs, one a pair, one CTA an SM: prefixes of any number and length fill the GPU. What a pair has of
// a unit is a piece. Its outputs and LSE go out in fp32, as blocks of [8 heads][128 dims] a sequence: the piece that begins
// the unit to the sequence's own block, one that goes on with it to the pair's (a pair has one such piece at most, its
// first).
//
// Why pairs: a CTA alone reads 64 KB a step of 256 rows, and its copies took 2500 of the step's 4050 clocks. In a pair
// each CTA copies and keeps half (K of 64 of the tokens, V of 64 of the 128 dims).
//
// What bounds it: a step of both tiles takes 3330 clocks, 2048 of them MMAs; a tile's chain is its softmax (1880 clocks from
// scores to the second half of P), its MMAs (1024 at least) and the barriers between them. 16384 tokens for 128 sequences on 43
// pairs: 54 us, 53 % of the tensor pipe's cycles (the own tokens' decode has the other SMs; on 47 pairs 49.5 us). With an FP8 cache a step takes 4800
// clocks: twice the operations a score, and warps that convert beside them. Two threads a row (64 tokens each, 768 threads) took
// 1270 clocks for the softmax, but 79 us for the whole call where this form took 68 (FP8 103 and 81): more warps for the same issue slots.
//
// Pages are single tokens in any order, so their rows are gathered by 16-byte cp.async, written where the 128-byte swizzle
// wants them; four warps keep up to four steps (32 KB each, a CTA) in flight. The odd CTA's copies are counted there, and its MMA warp
// tells the even CTA, which issues for both. An FP8 cache's codes go through a ring of their own and become fp16 (exact) on
// the way to three such stages; a token's K scale is taken on its score, its V scale on its probability (over a running power of
// two), Q is fp16 times a power of two a row, as in the decode.
//
// The running maximum moves only when a row's scores pass it by 2^8, so O is seldom rescaled; fp16 probabilities are held
// times 2^7. Every wait is bounded: on a timeout the CTA flags the device error word, waits for its copies and MMAs in
// flight, frees tensor memory and leaves.
constexpr int kStep = 128, kSeqTile = 16, kUnitSeqs = 4 * kSeqTile;
constexpr int kPreThreads = 512, kCopyWarps = 4, kMmaWarp = 4, kRowWarp = 8;  // two MMA warps; from 8 on two warpgroups of rows
constexpr int kRowRegs = 200, kOtherRegs = 56;
static_assert(256 * kRowRegs + 256 * kOtherRegs <= 65536, "register split");
constexpr int kQRegion = 128 * 128, kQTile = 2 * kQRegion;  // 128 rows of 64 values; of 128
constexpr int kKRegion = 64 * 128, kVOff = 2 * kKRegion;   // 64 tokens x 128 values of K in two regions, then 128 x 64 of V
constexpr int kStageBytes = kVOff + 128 * 128;
constexpr int kInfo = 8;  // steps whose masks and scales are held: the copies are at most six ahead of the softmax
constexpr float kMoveBy = 8.f;

// A role's walk over the pieces of its pair, kept in shared memory.
struct Walk {
  int64_t x, end, group_end;         // next step, the run's end, the end of group g's steps
  int g, tiles, seq0, members, first, n;  // the group: steps a unit, sequences, prefix tokens
};
struct Piece {
  int head, row0, step0, steps;  // KV head, first sequence (within the group), steps
  int seq0, members, first, n;
  // sequences of tile a; those of one CTA's half of it
  __device__ __forceinline__ int seqs(int a) const { return max(0, min(members - row0 - a * 2 * kSeqTile, 2 * kSeqTile)); }
  __device__ __forceinline__ int seqs(int a, int half) const { return max(0, min(seqs(a) - half * kSeqTile, kSeqTile)); }
};

template <bool F8>
struct PrefixCfg {
  static constexpr int kStages = F8 ? 3 : 4;
  static constexpr int kRaw = F8 ? 3 : 0;  // stages of codes
  static constexpr float kShift = F8 ? 7.f : 0.f;
  static constexpr int kStageOff = 2 * kQTile;
  static constexpr int kRawOff = kStageOff + kStages * kStageBytes;
  static constexpr int kRawV = kVOff / 2, kRawScales = kStageBytes / 2, kRawBytes = kRawScales + 2 * kStep * 4;  // codes of K, of V; scales of K, of V
  static constexpr int kMaskOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kScaleOff = kMaskOff + kInfo * 16;           // K, then V scales of a step; V's largest, a warp's each
  static constexpr int kTopOff = kScaleOff + (F8 ? kInfo * 2 * kStep * 4 : 0);
  static constexpr int kRowOff = kTopOff + (F8 ? kInfo * 16 : 0);   // the queries' factors
  static constexpr int kWalkOff = kRowOff + (F8 ? 256 * 4 : 0);
  static constexpr int kBarOff = kWalkOff + kPreThreads / 32 * static_cast<int>(sizeof(Walk));
  // Barriers. Both CTAs': stages full (the even one's counts the odd one's too) and free, S and O there (MMA commits), all
  // done; for an FP8 cache, the factors of a tile's rows written. The even CTA's: queries written, the halves of P written
  // (4 warps of each CTA), whose turn it is to issue.
  static constexpr int kFull = 0, kFree = kStages, kQ = 2 * kStages, kS = kQ + 2, kO = kS + 2, kP = kO + 2, kTurn = kP + 4,
                       kRows = kTurn + 2, kDone = kRows + 2, kBars = kDone + 1;
  static constexpr int kWordOff = kBarOff + kBars * 8;
  static constexpr int kBytes = kWordOff + 16 + 1024;  // the base is rounded up to 1024 bytes (swizzle atoms)
  static_assert(kBytes <= 226 * 1024 && sizeof(Walk) % 8 == 0, "prefix pass exceeds shared memory");
};

// Steps of group g's units together; its steps a unit, first sequence, sequences, first prefix token and their count.
__device__ __forceinline__ int64_t group_steps(const SharedParams& p, int g, int& tiles, int& seq0, int& members, int& first, int& n) {
  n = prefix_range(p, g, first);
  tiles = (n + kStep - 1) / kStep;
  seq0 = max(0, min(__ldcg(p.group_indptr + g), p.batch));
  members = max(0, min(__ldcg(p.group_indptr + g + 1), p.batch) - seq0);
  return static_cast<int64_t>((members + kUnitSeqs - 1) / kUnitSeqs) * kKvHeads * tiles;
}

__device__ __forceinline__ int64_t steps_per_pair(int64_t total, int pairs) {
  return total > pairs ? (total + pairs - 1) / pairs : 1;
}

// The next piece of the warp's walk; false at the run's end. Every lane gets it.
__device__ __forceinline__ bool next_piece(const SharedParams& p, volatile Walk* w, int lane, Piece& pc) {
  __syncwarp();
  int64_t x = w->x, group_end = w->group_end;
  const int64_t end = w->end;
  if (x >= end) return false;
  int g = w->g, tiles = w->tiles;
  pc.seq0 = w->seq0;
  pc.members = w->members;
  pc.first = w->first;
  pc.n = w->n;
  while (x >= group_end) {
    ++g;
    group_end += group_steps(p, g, tiles, pc.seq0, pc.members, pc.first, pc.n);
  }
  const int64_t per_group = static_cast<int64_t>((pc.members + kUnitSeqs - 1) / kUnitSeqs) * kKvHeads * tiles;
  const int64_t at = x - (group_end - per_group);
  const int unit = at < INT32_MAX ? static_cast<int>(at) / tiles : static_cast<int>(at / tiles);
  pc.step0 = static_cast<int>(at - static_cast<int64_t>(unit) * tiles);
  pc.steps = static_cast<int>(min(static_cast<int64_t>(tiles - pc.step0), end - x));
  pc.head = unit % kKvHeads;
  pc.row0 = unit / kKvHeads * kUnitSeqs;
  __syncwarp();
  if (lane == 0) {
    w->x = x + pc.steps;
    w->group_end = group_end;
    w->g = g;
    w->tiles = tiles;
    w->seq0 = pc.seq0;
    w->members = pc.members;
    w->first = pc.first;
    w->n = pc.n;
  }
  return true;
}

template <bool F8>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  return F8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}

// Two scores to weights x = 2^(s sc + off), their sum added to l: packed operands x, or x (w iv) with an FP8 cache.
template <bool F8>
__device__ __forceinline__ uint32_t weigh_pair(uint32_t s0, uint32_t s1, uint64_t sc2, uint64_t off2, float w0, float w1, uint64_t iv2, uint64_t& l) {
  float x0, x1;
  unpack2(fma2(pack2(__uint_as_float(s0), __uint_as_float(s1)), sc2, off2), x0, x1);
  x0 = ex2(x0);
  x1 = ex2(x1);
  const uint64_t x = pack2(x0, x1);
  l = add2(l, x);
  if constexpr (F8) unpack2(mul2(x, mul2(pack2(w0, w1), iv2)), x0, x1);
  return pack_p<F8>(x0, x1);
}

// 16 consecutive floats of shared memory, their loads together.
__device__ __forceinline__ void load16(uint32_t addr, float (&x)[16]) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) ld_shared_u4(addr + 16 * i, u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ void store_f8(float* to, const uint32_t* x, float f) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(__uint_as_float(x[0]) * f),
               "f"(__uint_as_float(x[1]) * f), "f"(__uint_as_float(x[2]) * f), "f"(__uint_as_float(x[3]) * f),
               "f"(__uint_as_float(x[4]) * f), "f"(__uint_as_float(x[5]) * f), "f"(__uint_as_float(x[6]) * f),
               "f"(__uint_as_float(x[7]) * f)
               : "memory");
}

template <bool F8>
__global__ void __launch_bounds__(kPreThreads, 1) gqa_shared_prefix_kernel(const SharedParams p) {
  using C = PrefixCfg<F8>;
  extern __shared__ uint8_t smem_raw[];
  const int half = static_cast<int>(cluster_rank());
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort_s = reinterpret_cast<volatile int*>(sm + C::kWordOff + 4);
  auto bar = [&](int i) { return base + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  __shared__ int64_t warp_steps[kPreThreads / 32];
  Walk* walks = reinterpret_cast<Walk*>(sm + C::kWalkOff);
  if (tid == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      int count = 1;  // S, O, turns
      if (i < C::kFree) count = (F8 ? kCopyWarps : kCopyWarps * 32 + kCopyWarps) + (half == 0 ? 1 : 0);
      else if (i < C::kQ || i == C::kDone) count = 2;  // a commit of each MMA warp
      else if (i < C::kS || (i >= C::kP && i < C::kTurn)) count = 8;
      else if (i >= C::kRows && i < C::kDone) count = 4;
      mbar_init(bar(i), count);
    }
    *abort_s = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  pdl_wait();
  pdl_launch_dependents();  // the own tokens' decode: by now all that it reads is there

  // total steps, then where this pair's run begins; groups 512 at a time
  {
    int t = 0, s0 = 0, m = 0, f = 0, n = 0;
    int64_t total = 0, carry = 0, steps = 0, upto = 0;
    const bool once = p.groups <= kPreThreads;
    auto scan = [&](int g0) {  // steps of group g0 + tid, and up to its end within these 512
      steps = g0 + tid < p.groups ? group_steps(p, g0 + tid, t, s0, m, f, n) : 0;
      upto = steps;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      __syncthreads();
      if (lane == 31) warp_steps[warp] = upto;
      __syncthreads();
      int64_t all = 0;
#pragma unroll 1
      for (int w = 0; w < kPreThreads / 32 && (g0 + 32 * w < p.groups); ++w) {
        if (w == warp) upto += all;
        all += warp_steps[w];
      }
      return all;
    };
    for (int g0 = 0; g0 < p.groups; g0 += kPreThreads) total += scan(g0);
    const int64_t run = steps_per_pair(total, pairs), begin = run * pair;
    for (int g0 = 0; g0 < p.groups; g0 += kPreThreads) {
      const int64_t all = once ? total : scan(g0);
      upto += carry;
      if (g0 + tid < p.groups) {
        if (blockIdx.x == 0) p.group_start[g0 + tid + 1] = upto;
        if (upto - steps <= begin && begin < upto)
          for (int w = 0; w < kPreThreads / 32; ++w) walks[w] = Walk{begin, min(begin + run, total), upto, g0 + tid, t, s0, m, f, n};
      }
      carry += all;
    }
    if (blockIdx.x == 0 && tid == 0) p.group_start[0] = 0;
    if (begin >= total) return;  // both CTAs of the pair
  }
  if (warp == kMmaWarp) tc2_alloc(base + C::kWordOff, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the barriers and the tensor memory of both CTAs are ready
  volatile Walk* walk = walks + warp;
  Piece pc;
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::kWordOff);
  auto wait = [&](int i, uint32_t parity, int bit) {
    return __all_sync(0xffffffffu, tc_wait_limited(bar(i), parity, abort_s, p.err, bit, p.wait_limit_ns)) != 0;
  };
  // for barriers that releases of the other CTA's threads complete
  auto wait_pair = [&](int i, uint32_t parity, int bit) {
    return __all_sync(0xffffffffu, mbar_try_wait_cluster(bar(i), parity) ||
                                       (tc_wait_limited(bar(i), parity, abort_s, p.err, bit, p.wait_limit_ns) &&
                                        mbar_try_wait_cluster(bar(i), parity))) != 0;
  };

  if (warp < kRowWarp) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp < kCopyWarps) {
      // ------------------------------------------------------------- copies
      // Warp w: K of tokens 16 w .. of this CTA's 64, V of tokens 32 w .. of the 128.
      const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
      const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
      int s = 0, info = 0, filled = 0;
      uint32_t ph = 1;  // parity of the stage's previous release
      bool good = true;
      const int k_token = 64 * half + 16 * warp + (lane & 15), v_token = 32 * warp + lane;
      auto id_of = [&](const Piece& w, int t) { return t < w.n ? __ldcg(p.prefix_indices + w.first + t) : -1; };
      auto live = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages); };
      if constexpr (!F8) {
        const uint8_t* k_from = kc + 16 * (lane & 15);
        const uint8_t* v_from = vc + 128 * half + 16 * (lane & 7);
        // rows 2 i + lane / 16 of K (8 apart: every fourth i), 4 i + lane / 8 of V: the swizzle of i and i + 4, or i + 2, is one
        const uint32_t k_to = ((lane & 15) >> 3) * kKRegion;
        while (good && next_piece(p, walk, lane, pc)) {
          int t0 = pc.step0 * kStep;
          int kid = id_of(pc, t0 + k_token), vid = id_of(pc, t0 + v_token);
          const int64_t head_off = pc.head * (kHeadDim * 2);
#pragma unroll 1
          for (int j = 0; j < pc.steps; ++j) {
            const unsigned k_mask = __ballot_sync(0xffffffffu, live(kid)), v_mask = __ballot_sync(0xffffffffu, live(vid));
            const int k_page = live(kid) ? kid : 0, v_page = live(vid) ? vid : 0;
            t0 += kStep;
            kid = id_of(pc, t0 + k_token);  // of the next step, behind this one's copies
            vid = id_of(pc, t0 + v_token);
            if (filled >= C::kStages) good = wait(C::kFree + s, ph, kErrTimeoutEmpty);
            if (!good) break;
            ++filled;
            const uint32_t stage = base + C::kStageOff + s * kStageBytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 2 * i + (lane >> 4);
              const int64_t pg = __shfl_sync(0xffffffffu, k_page, r);
              cp_async_16(sw128(stage + k_to, 16 * warp + r, lane & 7), k_from + head_off + pg * kPageBytes, (k_mask >> r) & 1u ? 16u : 0u);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              const int64_t pg = __shfl_sync(0xffffffffu, v_page, r);
              cp_async_16(sw128(stage + kVOff, 32 * warp + r, lane & 7), v_from + head_off + pg * kPageBytes, (v_mask >> r) & 1u ? 16u : 0u);
            }
            cp_async_arrive(bar(C::kFull + s));
            if (lane == 0) {
              reinterpret_cast<volatile unsigned*>(sm + C::kMaskOff)[4 * info + warp] = v_mask;
              mbar_arrive(bar(C::kFull + s));
            }
            if (++s == C::kStages) {
              s = 0;
              ph ^= 1;
            }
            info = (info + 1) % kInfo;
          }
        }
      } else {
        // A thread converts the chunks that it copied itself: 16 codes of rows 4 i + lane / 8 of K, 8 i + lane / 4 of V. The
        // copies run kRaw - 1 steps ahead of the conversion; the conversions are counted by the copies' walk.
        constexpr int kRow = kKvHeads * kHeadDim + 4 * kKvHeads;
        bool more = next_piece(p, walk, lane, pc);
        int aj = 0, as = 0, ainfo = 0, copied = 0, kid = -1, vid = -1;
        auto ids = [&]() {
          if (more) {
            const int t0 = (pc.step0 + aj) * kStep;
            kid = id_of(pc, t0 + k_token);
            vid = id_of(pc, t0 + v_token);
          }
        };
        ids();
        auto copy = [&]() {
          if (more) {
            const uint32_t stage = base + C::kRawOff + as * C::kRawBytes;
            const int64_t head_off = pc.head * kHeadDim;
            const unsigned k_mask = __ballot_sync(0xffffffffu, live(kid)), v_mask = __ballot_sync(0xffffffffu, live(vid));
            const int k_page = live(kid) ? kid : 0, v_page = live(vid) ? vid : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 4 * i + (lane >> 3);
              const int64_t pg = __shfl_sync(0xffffffffu, k_page, r);
              cp_async_16(stage + (16 * warp + r) * kHeadDim + 16 * (lane & 7), kc + pg * kRow + head_off + 16 * (lane & 7),
                          (k_mask >> r) & 1u ? 16u : 0u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2);
              const int64_t pg = __shfl_sync(0xffffffffu, v_page, r);
              cp_async_16(stage + C::kRawV + (32 * warp + r) * 64 + 16 * (lane & 3), vc + pg * kRow + head_off + 64 * half + 16 * (lane & 3),
                          (v_mask >> r) & 1u ? 16u : 0u);
            }
            const int64_t at = static_cast<int64_t>(v_page) * kRow + kKvHeads * kHeadDim + 4 * pc.head;
            const uint32_t to = stage + C::kRawScales + 4 * v_token;
            cp_async_4(to, kc + at, (v_mask >> lane) & 1u ? 4u : 0u);
            cp_async_4(to + 4 * kStep, vc + at, (v_mask >> lane) & 1u ? 4u : 0u);
            if (lane == 0) reinterpret_cast<volatile unsigned*>(sm + C::kMaskOff)[4 * ainfo + warp] = v_mask;
            as = as + 1 == C::kRaw ? 0 : as + 1;
            ainfo = (ainfo + 1) % kInfo;
            ++copied;
            if (++aj == pc.steps) {
              aj = 0;
              more = next_piece(p, walk, lane, pc);
            }
            ids();  // of the next step, behind this one's copies
          }
          cp_async_commit();  // one group a call, even when empty
        };
        auto convert = [&](uint32_t from, uint32_t region, int r, int c) {  // 16 codes to columns c and c + 1 of row r
          uint32_t x[4], y[8];
          ld_shared_u4(from, x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = cvt_e4m3x2_f16x2(x[k]);
            y[2 * k + 1] = cvt_e4m3x2_f16x2(x[k] >> 16);
          }
          st_shared_u4(sw128(region, r, c), y[0], y[1], y[2], y[3]);
          st_shared_u4(sw128(region, r, c + 1), y[4], y[5], y[6], y[7]);
        };
#pragma unroll 1
        for (int i = 0; i < C::kRaw - 1; ++i) copy();
        int rs = 0;
#pragma unroll 1
        while (filled < copied || more) {
          __syncwarp();
          copy();
          cp_async_wait<C::kRaw - 1>();
          if (filled >= C::kStages) good = wait(C::kFree + s, ph, kErrTimeoutEmpty);
          if (!good) break;
          ++filled;
          const uint32_t stage = base + C::kStageOff + s * kStageBytes;
          const uint32_t codes = base + C::kRawOff + rs * C::kRawBytes;
          const uint32_t at = codes + C::kRawScales + 4 * v_token;
          const float sk = ld_shared_f32(at), sv = ld_shared_f32(at + 4 * kStep);
          volatile float* scales = reinterpret_cast<volatile float*>(sm + C::kScaleOff) + 2 * info * kStep + v_token;
          scales[0] = sk;
          scales[kStep] = sv;
          const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, fabsf(sv) < INFINITY ? __float_as_uint(fabsf(sv)) : 0u));
          if (lane == 0) reinterpret_cast<volatile float*>(sm + C::kTopOff)[4 * info + warp] = top;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = lane & 7, r = 16 * warp + 4 * i + (lane >> 3);
            convert(codes + r * kHeadDim + 16 * c, stage + (c >> 2) * kKRegion, r, 2 * (c & 3));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 32 * warp + 8 * i + (lane >> 2);
            convert(codes + C::kRawV + r * 64 + 16 * (lane & 3), stage + kVOff, r, 2 * (lane & 3));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kFull + s));
          rs = rs + 1 == C::kRaw ? 0 : rs + 1;
          info = (info + 1) % kInfo;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      cp_async_commit();
      cp_async_wait<0>();  // no copy may still be writing when the CTA leaves
    } else if (warp == kMmaWarp && half == 1) {
      // the odd CTA's stages, told to the even one as they are full
      const uint32_t peer = cluster_addr(bar(C::kFull), 0);
      int s = 0;
      uint32_t ph = 0;
      bool good = true;
      while (good && next_piece(p, walk, lane, pc)) {
#pragma unroll 1
        for (int j = 0; j < pc.steps; ++j) {
          good = wait(C::kFull + s, ph, kErrTimeoutFull);
          if (!good) break;
          fence_proxy_async_smem();  // the copies' writes, seen behind the barrier, for the MMAs
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(peer + 8 * s);
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp < kMmaWarp + 2 && half == 0) {
      // --------------------------------------------------------------- MMAs
      // tile a: the whole warp walks (warp-uniform operands), one elected lane issues
      const int a = static_cast<int>(uniform(warp - kMmaWarp));
      const uint32_t ub = uniform(base), ut = uniform(tmem);
      constexpr uint32_t idesc_s = F8 ? tc_idesc_f16(256, kStep, false, false) : tc_idesc_bf16(256, kStep, false, false);
      constexpr uint32_t idesc_o = F8 ? tc_idesc_f16(256, kHeadDim, false, true) : tc_idesc_bf16(256, kHeadDim, false, true);
      const uint64_t dq0 = tc_sdesc(ub + a * kQTile, 16, 1024, kSwizzle128B);
      const uint64_t dk0 = tc_sdesc(ub + C::kStageOff, 16, 1024, kSwizzle128B);
      // V as B: N = 64 dims a CTA (one swizzle atom), K = tokens in 8-row groups (SBO)
      const uint64_t dv0 = tc_sdesc(ub + C::kStageOff + kVOff, 128 * 128, 1024, kSwizzle128B);
      const uint32_t s_col = ut + 128 * a, o_col = ut + 256 + 128 * a;
      auto ubar = [&](int i) { return ub + C::kBarOff + 8u * static_cast<uint32_t>(i); };
      int s = 0;  // stage and parity of step j
      uint32_t ph = 0, np = 0, nq = 0, turn = 0;
      bool good = true;
      while (good && next_piece(p, walk, lane, pc)) {
        const int steps = static_cast<int>(uniform(pc.steps));
        const bool mine = uniform(pc.seqs(a)) > 0;
        if (mine) good = wait_pair(C::kQ + a, nq++ & 1, kErrTimeoutFull);
#pragma unroll 1
        for (int j = 0; j <= steps; ++j, ++turn) {
          // O += P(j - 1) V(j - 1), then S(j) = Q K(j), in turn with the other tile's warp
          const int vs = s == 0 ? C::kStages - 1 : s - 1;
          if (j < steps) good = good && wait_pair(C::kFull + s, ph, kErrTimeoutFull);
          if (a == 1 || turn > 0) good = good && wait(C::kTurn + a, (a == 1 ? turn : turn - 1) & 1, kErrTimeoutFull);
          const bool pv = j > 0 && mine, qk = j < steps && mine;
          if (pv) good = good && wait(C::kP + 2 * a, np & 1, kErrTimeoutFull);
          if (!good) break;
          if (!F8) fence_proxy_async_smem();  // the copies' writes, seen behind the barrier, for the MMAs
          tc_fence_after();
          if (pv) {
            const uint64_t dv = dv0 + vs * (kStageBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc2_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, kk ? 1u : (j > 1 ? 1u : 0u));
            good = wait(C::kP + 2 * a + 1, np & 1, kErrTimeoutFull);
            if (!good) break;
            ++np;
            tc_fence_after();
#pragma unroll
            for (int kk = 4; kk < 8; ++kk) tc2_mma_tmem_a_warp(o_col, s_col + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, 1u);
          }
          const uint64_t dk = dk0 + s * (kStageBytes >> 4);
          auto scores = [&](int r) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc2_mma_warp(s_col, dq0 + ((r * kQRegion + kk * 32) >> 4), dk + ((r * kKRegion + kk * 32) >> 4), idesc_s, (r | kk) ? 1u : 0u);
          };
          if (qk) scores(0);
          if (lane == 0) mbar_arrive(bar(C::kTurn + 1 - a));  // early: the rest is issued before the other warp gets going
          __syncwarp();
          if (qk) {
            scores(1);
            tc2_commit_warp(ubar(C::kS + a));
          }
          if (j > 0) {
            tc2_commit_warp(ubar(C::kFree + vs));
            if (mine && j == steps) tc2_commit_warp(ubar(C::kO + a));
          }
          if (j < steps && ++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      tc2_commit_warp(ubar(C::kDone));  // every MMA done before tensor memory is freed
      __syncwarp();
    }
    __syncwarp();
  } else {
    // -------------------------- a warpgroup of rows: tile a, row 32 wq + lane
    setmaxnreg_inc<kRowRegs>();
    const int a = (warp - kRowWarp) >> 2, wq = warp & 3, t = 32 * wq + lane;
    const uint32_t quarter = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t s_col = tmem + quarter + 128 * a, o_col = tmem + quarter + 256 + 128 * a;
    const uint32_t q_bar = cluster_addr(bar(C::kQ + a), 0), p_bar = cluster_addr(bar(C::kP + 2 * a), 0);
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes to the queries
    uint32_t scored = 0, units = 0, info = 0;
    bool good = true;
    while (good && next_piece(p, walk, lane, pc)) {
      if (pc.seqs(a) == 0) {
        info = (info + pc.steps) % kInfo;
        continue;
      }
      // the queries: sequence i's 8 rows are 2 KB in a row, 16 bytes a thread
      const int seqs = pc.seqs(a, half), seq = pc.seq0 + pc.row0 + (2 * a + half) * kSeqTile;
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         (static_cast<int64_t>(seq) * kQoHeads + pc.head * kGroup) * kHeadDim) + t;
      const uint32_t to = base + a * kQTile + ((t & 15) >> 3) * kQRegion;
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
      if (lane == 0) mbar_arrive_cluster(q_bar);
      float sc = fabsf(p.scale_log2);
      if constexpr (F8) {
        if (lane == 0) mbar_arrive(bar(C::kRows + a));
        good = wait(C::kRows + a, units & 1, kErrTimeoutFull);
        if (!good) break;
        sc *= reinterpret_cast<volatile float*>(sm + C::kRowOff)[128 * a + t];
      }
      sc = fmaxf(sc, 1e-37f);  // > 0: -inf * sc stays -inf
      const uint64_t sc2 = pack2(sc, sc);
      float m = -INFINITY, cv = 0.f;
      uint64_t l2 = 0;
#pragma unroll 1
      for (int j = 0; j < pc.steps; ++j) {
        good = wait(C::kS + a, scored & 1, kErrTimeoutFull);
        if (!good) break;
        ++scored;
        tc_fence_after();
        const uint32_t k_scales = base + C::kScaleOff + info * 2 * kStep * 4, v_scales = k_scales + kStep * 4;
        uint32_t w[4];
        ld_shared_u4(base + C::kMaskOff + 16 * info, w[0], w[1], w[2], w[3]);
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(s_col + 32 * c, s + 32 * c);
        tc_wait_ld();
        if constexpr (F8) {
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            float x[16];
            load16(k_scales + 4 * c, x);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float lo, hi;
              unpack2(mul2(pack2(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), pack2(x[e], x[e + 1])), lo, hi);
              s[c + e] = __float_as_uint(lo);
              s[c + e + 1] = __float_as_uint(hi);
            }
          }
        }
        if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (((w[c >> 5] >> (c & 31)) & 1u) == 0) s[c] = 0xff800000u;  // -inf
        }
        float iv = 1.f, cv_new = cv;
        uint64_t iv2 = 0;
        if constexpr (F8) {
          uint32_t x[4];
          ld_shared_u4(base + C::kTopOff + 16 * info, x[0], x[1], x[2], x[3]);
          const float vm = fminf(fmaxf(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]))), 0x1p126f);
          cv_new = fmaxf(cv, vm > 0.f ? pow2_ceil(fmaxf(vm, 0x1p-126f)) : 0.f);
          iv = cv_new > 0.f ? pow2_recip(cv_new) : 0.f;
          iv2 = pack2(iv, iv);
        }
        auto weigh = [&](int c, uint64_t off2, uint32_t* pk, uint64_t& l) {  // of tokens 64 c .. 64 c + 63
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float v[16];
            if constexpr (F8) load16(v_scales + 256 * c + 8 * k, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              pk[k + e] = weigh_pair<F8>(s[64 * c + 2 * (k + e)], s[64 * c + 2 * (k + e) + 1], sc2, off2, v[2 * e], v[2 * e + 1], iv2, l);
          }
        };
        // Optimistic: the first half's weights are formed with the running maximum as it stands, beside the search for this
        // step's; only if a row passed it by 2^8 (the first step, and seldom after) are they formed again.
        uint32_t pk[32];
        uint64_t l_new = 0, off2 = pack2(C::kShift - m, C::kShift - m);
        weigh(0, off2, pk, l_new);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 32; ++k)
          mx[k & 3] = max3(mx[k & 3], max3(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1]), __uint_as_float(s[4 * k + 2])),
                           __uint_as_float(s[4 * k + 3]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;
        const bool move = top > m + kMoveBy;
        if (__any_sync(0xffffffffu, move || m == -INFINITY || cv_new != cv)) {
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
          const float off = m == -INFINITY ? 0.f : C::kShift - m;
          off2 = pack2(off, off);
          l_new = 0;
          weigh(0, off2, pk, l_new);
        }
        tc_st32(s_col, pk);  // over scores that have been read
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(p_bar);  // half of the tokens: the MMAs may start on it
        weigh(1, off2, pk, l_new);
        l2 = add2(l2, l_new);
        tc_st32(s_col + 32, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(p_bar + 8);
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
      const int64_t block = pc.step0 == 0 ? static_cast<int64_t>(seq + i) * kKvHeads + pc.head
                                            : static_cast<int64_t>(p.batch) * kKvHeads + static_cast<int64_t>(pair) * kUnitSeqs + (2 * a + half) * kSeqTile + i;
      float* po = p.part_o + block * (kHeadDim * kGroup) + h * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tc_ld32(o_col + 32 * c, o);
        tc_wait_ld();
        if (i < seqs)
#pragma unroll
          for (int k = 0; k < 32; k += 8) store_f8(po + 32 * c + k, o + k, inv);
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
  cluster_sync();  // the other CTA's arrivals and MMAs are done too
  if (warp == kMmaWarp) tc2_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- join
// A block per sequence and KV head, a thread per dim. The parts are taken 16 at a time: a thread per part and head finds
// the part and its LSE, their largest gives the weights 2^(LSE - max), and every thread sums its dim of the parts, whose
// loads do not depend on one another. Bound by two round trips of loads, and by 4 KB a part (8 sequences 11 us, 128 10 to 14).
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
    int t, s0, m, f, n;
    int64_t upto = tid < p.groups ? group_steps(p, tid, t, s0, m, f, n) : 0;
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
    // pieces of the prefix: the first in the sequence's block, the others in their pair's
    int pre = 0, own = 0, cta0 = 0, local = 0;
    const int lo = max(0, min(__ldcg(p.kv_indptr + b), total)), hi = min(__ldcg(p.kv_indptr + b + 1), total);
    const int group = p.pre_ctas > 0 ? group_of(p, b) : -1;
    if (group >= 0) {
      int tiles, seq0, members, first_token, n;
      group_steps(p, group, tiles, seq0, members, first_token, n);
      if (tiles > 0) {
        const int64_t run = steps_per_pair(few ? start_s[p.groups] : __ldcg(p.group_start + p.groups), p.pre_ctas / 2);
        const int64_t first = (few ? start_s[group] : __ldcg(p.group_start + group)) + (static_cast<int64_t>((b - seq0) / kUnitSeqs) * kKvHeads + g) * tiles;
        cta0 = static_cast<int>(first / run);
        pre = min(static_cast<int>((first + tiles - 1) / run), p.pre_ctas / 2 - 1) - cta0 + 1;
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
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float* o = p.part_o + part_s[k] * kPart;
        float4 oa, ob;
        if (i0 + k < pre) {  // [8 heads][128 dims]
          o += tid;
          oa = make_float4(__ldcg(o), __ldcg(o + kHeadDim), __ldcg(o + 2 * kHeadDim), __ldcg(o + 3 * kHeadDim));
          ob = make_float4(__ldcg(o + 4 * kHeadDim), __ldcg(o + 5 * kHeadDim), __ldcg(o + 6 * kHeadDim), __ldcg(o + 7 * kHeadDim));
        } else {             // [128 dims][8 heads]
          oa = __ldcg(reinterpret_cast<const float4*>(o + tid * kGroup));
          ob = __ldcg(reinterpret_cast<const float4*>(o + tid * kGroup) + 1);
        }
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
  return launch_chained(gqa_shared_prefix_kernel<F8>, dim3(p.pre_ctas), kPreThreads, PrefixCfg<F8>::kBytes, stream, 2, p);
}

int shared_prefix_blocks(int batch, int ctas) { return batch * kKvHeads + ctas / 2 * kUnitSeqs; }

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
