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
// A block of threads per cache block: 64 lanes of 16 bytes a token, four tokens at a time.
constexpr int kBoundThreads = 256;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__global__ void __launch_bounds__(kBoundThreads) gqa_block_bounds_kernel(const BoundsParams p) {
  __shared__ uint4 part[2][4][64];
  const int lane = threadIdx.x & 63, team = threadIdx.x >> 6;
  for (int r = blockIdx.y; r < p.requests; r += gridDim.y) {
    const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(__ldg(p.lens + r)), static_cast<int64_t>(p.width) * p.page_size)));
    const int first = p.first == nullptr ? 0 : max(0, __ldg(p.first + r));
    if (first >= n) continue;
    for (int i = first / p.page_size + blockIdx.x; i <= (n - 1) / p.page_size; i += gridDim.x) {
      const int block = __ldg(p.block_table + static_cast<int64_t>(r) * p.width + i);
      if (static_cast<unsigned>(block) >= static_cast<unsigned>(p.num_blocks)) continue;  // the same for all threads
      const int tokens = min(p.page_size, n - i * p.page_size);
      const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_cache) + static_cast<int64_t>(block) * p.page_size * kRowValues) + lane;
      uint4 hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u), lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);
#pragma unroll 8
      for (int t = team; t < tokens; t += 4) {
        const uint4 x = __ldg(k + t * 64);
        hi = make_uint4(max2(hi.x, x.x), max2(hi.y, x.y), max2(hi.z, x.z), max2(hi.w, x.w));
        lo = make_uint4(min2(lo.x, x.x), min2(lo.y, x.y), min2(lo.z, x.z), min2(lo.w, x.w));
      }
      __syncthreads();  // the last block's parts have been read
      part[0][team][lane] = hi;
      part[1][team][lane] = lo;
      __syncthreads();
      if (team < 2) {
        uint4 a = part[team][0][lane];
#pragma unroll
        for (int j = 1; j < 4; ++j) {
          const uint4 x = part[team][j][lane];
          a = team == 0 ? make_uint4(max2(a.x, x.x), max2(a.y, x.y), max2(a.z, x.z), max2(a.w, x.w))
                        : make_uint4(min2(a.x, x.x), min2(a.y, x.y), min2(a.z, x.z), min2(a.w, x.w));
        }
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.bounds) + static_cast<int64_t>(block) * 2 * kRowValues)[team * 64 + lane] = a;
      }
    }
  }
}

cudaError_t launch_block_bounds(const BoundsParams& p, int sm_count, cudaStream_t stream) {
  const int y = p.requests < 65535 ? p.requests : 65535;
  const int most = (8 * sm_count + y - 1) / y;
  gqa_block_bounds_kernel<<<dim3(p.width < most ? p.width : most, y), kBoundThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ score
// A warp per KV head and 16 blocks at a time: S^T (16 blocks x 8 heads) += [hi lo] (16 x 16) . [q+ q-]^T, 16 MMAs of
// m16n8k16 in all. A lane reads 16 consecutive bytes of a block's bounds, the contraction's order following: within 32
// dims, lane c's k indices 2c, 2c + 1, 2c + 8, 2c + 9 of the first MMA are dims 8c .. 8c + 3, of the second 8c + 4 .. + 7.
// Beside the score goes a bound of its error, kGamma * max_h |q_h|_1 * max |bounds|, for the choice: products of bf16 are
// exact in fp32; an MMA sums 16 of them and the accumulator, each cut off at 2^-23 of the largest, and no partial sum
// passes |q|_1 max|bounds|: 16 MMAs x 17 terms x 2^-23 < 2^-14.9.
constexpr int kScoreBlocks = 64;  // of a row, a block of threads
constexpr float kGamma = 0x1p-14f;

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
  v.req = __ldg(p.token_to_req + row);
  const bool ok = v.req >= 0 && v.req < p.requests;
  v.n = ok ? static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(__ldg(p.lens + row)), static_cast<int64_t>(p.width) * p.page_size))) : 0;
  v.count = (v.n + p.page_size - 1) / p.page_size;
  return v;
}

__global__ void __launch_bounds__(128) gqa_block_score_kernel(const BlockParams p) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  for (int row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const RowView v = row_view(p, row);
    const int first = blockIdx.x * kScoreBlocks;
    if (first >= v.count) continue;
    const int* table = p.block_table + static_cast<int64_t>(v.req) * p.width;
    const uint4* qr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(row) * kQoHeads + g * kGroup + r) * kHeadDim) + c;
    uint4 q[4];
    float norm = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[j] = __ldg(qr + 4 * j);
      const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) norm += fabsf(bf16_lo(w[i])) + fabsf(bf16_hi(w[i]));
    }
    norm += __shfl_xor_sync(0xffffffffu, norm, 1);
    norm += __shfl_xor_sync(0xffffffffu, norm, 2);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) norm = max_nan(norm, __shfl_xor_sync(0xffffffffu, norm, o));
    float* scores = p.scores + (static_cast<int64_t>(row) * kKvHeads + g) * p.width;
    float* errors = p.errors + (static_cast<int64_t>(row) * kKvHeads + g) * p.width;
    const int end = min(first + kScoreBlocks, v.count);
#pragma unroll 1
    for (int b0 = first; b0 < end; b0 += 16) {
      const int ia = b0 + r, ib = b0 + r + 8;
      const int pa = ia < end ? __ldg(table + ia) : -1, pb = ib < end ? __ldg(table + ib) : -1;
      const bool oka = static_cast<unsigned>(pa) < static_cast<unsigned>(p.num_blocks), okb = static_cast<unsigned>(pb) < static_cast<unsigned>(p.num_blocks);
      const uint4* xa = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) + (static_cast<int64_t>(oka ? pa : 0) * 2 * kKvHeads + g) * kHeadDim) + c;
      const uint4* xb = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) + (static_cast<int64_t>(okb ? pb : 0) * 2 * kKvHeads + g) * kHeadDim) + c;
      uint4 a[8], b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // 0 .. 3 hi, 4 .. 7 lo
        const int at = (j >> 2) * (kRowValues / 8) + 4 * (j & 3);
        a[j] = oka ? __ldg(xa + at) : make_uint4(0, 0, 0, 0);
        b[j] = okb ? __ldg(xb + at) : make_uint4(0, 0, 0, 0);
      }
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
      float ea = max_nan(bf16_lo(ta), bf16_hi(ta)), eb = max_nan(bf16_lo(tb), bf16_hi(tb));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        sa = max_nan(sa, __shfl_xor_sync(0xffffffffu, sa, o));
        sb = max_nan(sb, __shfl_xor_sync(0xffffffffu, sb, o));
        ea = max_nan(ea, __shfl_xor_sync(0xffffffffu, ea, o));
        eb = max_nan(eb, __shfl_xor_sync(0xffffffffu, eb, o));
      }
      // a block outside the pool is no candidate: error -1
      if (c == 0 && ia < end) scores[ia] = sa, errors[ia] = oka ? kGamma * norm * ea : -1.f;
      if (c == 0 && ib < end) scores[ib] = sb, errors[ib] = okb ? kGamma * norm * eb : -1.f;
    }
  }
}

// ----------------------------------------------------------------- choice
// A block of threads per row and KV head. The MMA's scores decide all blocks but those within the error of the k-th
// largest; of these the score is formed again in two floats (products of bf16 are exact, sums are carried with their
// rounding errors: 2^-44 of the terms), and the larger ones, then the lower ones, fill what is left.
constexpr int kChooseThreads = 512;

// s + e += x, exactly but for e's own rounding.
__device__ __forceinline__ void add_exact(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// The score of block `at` for the 8 query heads at q, by one warp: as hi + lo, rounded into hi first; false if it is no
// number. Lane (h = lane >> 2, c = lane & 3) sums 32 of the 128 dims of head h.
__device__ __forceinline__ bool exact_score(const __nv_bfloat16* q, const __nv_bfloat16* bounds, int lane, float& hi, float& lo) {
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(q + (lane >> 2) * kHeadDim) + 16 * (lane & 3);
  const uint32_t* up = reinterpret_cast<const uint32_t*>(bounds) + 16 * (lane & 3);
  const uint32_t* down = up + kRowValues / 2;
  float s = 0.f, e = 0.f;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const uint32_t x = __ldg(qr + i), a = __ldg(up + i), b = __ldg(down + i);
    const float x0 = bf16_lo(x), x1 = bf16_hi(x);
    // of the two products one is 0 for any finite bounds; both count, so that 0 times an infinity shows
    add_exact(s, e, __fmul_rn(x0 > 0.f ? x0 : x0 * 0.f, bf16_lo(a)));
    add_exact(s, e, __fmul_rn(x0 < 0.f ? x0 : x0 * 0.f, bf16_lo(b)));
    add_exact(s, e, __fmul_rn(x1 > 0.f ? x1 : x1 * 0.f, bf16_hi(a)));
    add_exact(s, e, __fmul_rn(x1 < 0.f ? x1 : x1 * 0.f, bf16_hi(b)));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
    add_exact(s, e, s2);
    e = __fadd_rn(e, e2);
  }
  float t = __fadd_rn(s, e), z = __fsub_rn(t, s);
  float rest = __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(e, z));
  bool number = isfinite(t);  // a sum that overflows counts as none
  if (!number) rest = 0.f;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {  // the largest of the heads
    const float t2 = __shfl_xor_sync(0xffffffffu, t, o), r2 = __shfl_xor_sync(0xffffffffu, rest, o);
    number = __shfl_xor_sync(0xffffffffu, number ? 1 : 0, o) != 0 && number;
    if (t2 > t || (t2 == t && r2 > rest)) t = t2, rest = r2;
  }
  hi = t;
  lo = rest;
  return number;
}

__global__ void __launch_bounds__(kChooseThreads) gqa_block_choose_kernel(const BlockParams p) {
  __shared__ SelectSpace<kChooseThreads> sp;
  __shared__ float widest[kChooseThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t unit = blockIdx.x; unit < static_cast<int64_t>(p.rows) * kKvHeads; unit += gridDim.x) {
    const int row = static_cast<int>(unit / kKvHeads), g = static_cast<int>(unit % kKvHeads);
    const RowView v = row_view(p, row);
    const int* table = p.block_table + static_cast<int64_t>(max(v.req, 0)) * p.width;
    float* scores = p.scores + unit * p.width;
    float* errors = p.errors + unit * p.width;
    auto forced = [&](int i) { return i < p.keep_first || i >= v.count - p.keep_last; };
    // candidates; of those not forced the widest error
    int mine = 0, held = 0;
    float wide = 0.f;
    for (int i = tid; i < v.count; i += kChooseThreads) {
      const float e = errors[i];
      if (e == -1.f) continue;
      ++mine;
      if (forced(i)) ++held; else if (e < INFINITY) wide = fmaxf(wide, e);
    }
    const int count = block_sum(sp, mine), fixed = block_sum(sp, held);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    if (lane == 0) widest[warp] = wide;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) wide = fmaxf(wide, widest[w]);
    const int take = min(p.top, count) - fixed;  // of those not forced; fixed <= top
    const bool all = count <= p.top;
    float above_all = INFINITY, below_all = INFINITY;
    int ties = 0;
    uint64_t least = 0;
    bool settled = true;  // whether every block between the two limits is chosen
    auto open = [&](int i) { return errors[i] != -1.f && !forced(i); };  // errors of scores formed again stay above -1
    if (!all && take > 0) {
      int above = 0;
      const uint32_t kth = block_kth<kChooseThreads, uint32_t>(sp, v.count, take, open, [&](int i) { return ordered_bits(scores[i]); }, above);
      const float mark = __uint_as_float((kth & 0x80000000u) ? kth & 0x7fffffffu : ~kth);  // NaN if no number
      above_all = __fadd_ru(mark, __fmul_ru(2.f, wide));
      below_all = __fadd_rd(mark, __fmul_rd(-2.f, wide));
      if (!isfinite(mark)) above_all = INFINITY, below_all = -INFINITY;  // decide all of them again
    }
    // 2: chosen, 1: to be decided, 0: not chosen
    auto rough = [&](int i) {
      if (errors[i] == -1.f) return 0;
      if (all || forced(i)) return 2;
      if (take <= 0) return 0;
      const float s = scores[i];
      if (!(fabsf(s) < INFINITY) || !(errors[i] < INFINITY)) return 1;
      return s > above_all ? 2 : (s < below_all ? 0 : 1);
    };
    if (!all && take > 0) {
      int sure = 0, maybe = 0;
      for (int i = tid; i < v.count; i += kChooseThreads) {
        const int c = rough(i);
        sure += c == 2 && !forced(i);
        maybe += c == 1;
      }
      sure = block_sum(sp, sure);
      maybe = block_sum(sp, maybe);
      const int left = take - sure;
      settled = left >= maybe;
      if (!settled) {
        // form their scores again, a warp each; marked by an error of -2 while both floats are kept
        __syncthreads();
        for (int i0 = 32 * warp; i0 < v.count; i0 += kChooseThreads) {
          const int i = i0 + lane;
          const int page = i < v.count && rough(i) == 1 ? __ldg(table + i) : -1;
          for (unsigned m = __ballot_sync(0xffffffffu, page >= 0); m != 0; m &= m - 1) {
            const int src = __ffs(m) - 1;
            const int64_t block = __shfl_sync(0xffffffffu, page, src);
            float hi, lo;
            const bool number = exact_score(static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(row) * kQoHeads + g * kGroup) * kHeadDim,
                                            static_cast<const __nv_bfloat16*>(p.bounds) + (block * 2 * kKvHeads + g) * kHeadDim, lane, hi, lo);
            if (lane == 0) p.again[unit * p.width + i0 + src] = make_float2(number ? hi : INFINITY, number ? lo : 0.f);
          }
        }
        __syncthreads();
        int above = 0;
        least = block_kth<kChooseThreads, uint64_t>(
            sp, v.count, left, [&](int i) { return rough(i) == 1; },
            [&](int i) {
              const float2 x = p.again[unit * p.width + i];
              return (static_cast<uint64_t>(ordered_bits(x.x)) << 32) | ordered_bits(x.y);
            }, above);
        ties = left - above;
      }
    }
    int* out = p.blocks + unit * p.top;
    int at = 0;
    for (int i0 = 0; i0 < v.count; i0 += kChooseThreads) {
      const int i = i0 + tid;
      const int c = i < v.count ? rough(i) : 0;
      bool stay = c == 2 || (c == 1 && settled), tie = false;
      if (c == 1 && !settled) {
        const float2 x = p.again[unit * p.width + i];
        const uint64_t k = (static_cast<uint64_t>(ordered_bits(x.x)) << 32) | ordered_bits(x.y);
        tie = k == least;
        stay = k > least;
      }
      int tied, kept;
      const int tie_rank = block_rank(sp, tie, tied);
      stay = stay || (tie && tie_rank < ties);
      ties -= min(ties, tied);
      const int rank = block_rank(sp, stay, kept);
      if (stay && at + rank < p.top) out[at + rank] = i;
      at += kept;
    }
    for (int i = min(at, p.top) + tid; i < p.top; i += kChooseThreads) out[i] = -1;
    __syncthreads();
  }
}

cudaError_t launch_block_select(const BlockParams& p, cudaStream_t stream) {
  const dim3 grid((p.width + kScoreBlocks - 1) / kScoreBlocks, p.rows < 65535 ? p.rows : 65535);
  gqa_block_score_kernel<<<grid, 128, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(p.rows) * kKvHeads;
  gqa_block_choose_kernel<<<static_cast<int>(units < (1 << 20) ? units : (1 << 20)), kChooseThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ slots
__global__ void __launch_bounds__(256) gqa_block_slots_kernel(const BlockParams p) {
  pdl_launch_dependents();
  const int64_t per_row = static_cast<int64_t>(p.top) * p.page_size, total = p.rows * per_row;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; x < kKvHeads * total; x += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int g = static_cast<int>(x / total);
    const int64_t y = x - g * total;
    const int row = static_cast<int>(y / per_row), z = static_cast<int>(y - row * per_row);
    const int j = z / p.page_size, t = z - j * p.page_size;
    const RowView v = row_view(p, row);
    const int i = __ldg(p.blocks + (static_cast<int64_t>(row) * kKvHeads + g) * p.top + j);
    int slot = -1;
    if (i >= 0 && i < v.count && static_cast<int64_t>(i) * p.page_size + t < v.n) {
      const int block = __ldg(p.block_table + static_cast<int64_t>(v.req) * p.width + i);
      if (static_cast<unsigned>(block) < static_cast<unsigned>(p.num_blocks)) slot = block * p.page_size + t;
    }
    p.slots[x] = slot;
  }
}

cudaError_t launch_block_slots(const BlockParams& p, int sm_count, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(kKvHeads) * p.rows * p.top * p.page_size;
  int64_t grid = (n + 255) / 256;
  if (grid > 8 * sm_count) grid = 8 * sm_count;
  gqa_block_slots_kernel<<<static_cast<int>(grid), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
