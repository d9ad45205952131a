// Latent attention's absorbed form: the two projections around the latent
// decode. With W_h the head's 256 x 512 up-projection (rows 0..127 give its
// keys, rows 128..255 its values from a latent row c: k = W_k c, v = W_v c),
//   q . k = (q W_k) . c       absorb_q:   q_lat[n][h][0:512] = q[n][h][0:128] W_k[h]
//   sum p v = W_v (sum p c)   expand_out: out[n][h][0:128] = o_lat[n][h][0:512] W_v[h]^T
// so decode attends over the cached latents directly. absorb_q also appends
// the head's 64 rotary values (turned by the token's position if asked), which
// makes its output the 576-value query the latent decode reads.
//
// Both are one small matrix product per head: [tokens x K] x [K x N], bf16
// operands, fp32 accumulation, one rounding at the store. At the token counts
// of a decode step the head's weights (128 KB) are the larger operand, so the
// bound is the bytes of weights and rows.
//
// Up to 16 tokens, mma.sync: a CTA takes a head and 64 output columns and streams K in
// chunks of 64 through a cp.async ring; the results go through shared memory to 16-byte
// stores (a fragment's own are 4 bytes). Above, the tensor-memory MMA: 128 tokens (M) of a
// head and 256 (absorb_q) or 64 (expand_out) output columns a CTA, two CTAs an SM, operands
// and results by tensor copies, so that the loads of a whole CTA are in flight at once.
// Measured, 128 tokens x 128 heads: absorb_q 12.3 us (42 MB; 14.5 on mma.sync), expand_out
// 9.5 us (38 MB; 11.4 on mma.sync); 4 tokens x 16 heads: absorb_q 4.0 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_ptx.cuh"
#include "gqa_rope.cuh"
#include "gqa_tc.cuh"

namespace gqa {
namespace {

constexpr int kLat = 512, kNope = 128, kRope = 64, kHeadV = 128;
constexpr int kWRows = kNope + kHeadV;  // weight rows a head
constexpr int kBK = 64;                 // K chunk: 128-byte rows

// WM x WN warps, each MI x 16 rows by NI x 8 columns. BT: B is given [K][N]
// (absorb_q: N contiguous), else [N][K].
template <int WM, int WN, int MI, int NI, int STAGES, bool BT>
struct ProjTile {
  static constexpr int kThreads = WM * WN * 32;
  static constexpr int BM = WM * MI * 16, BN = WN * NI * 8;
  static constexpr int kABytes = BM * kBK * 2, kBBytes = BN * kBK * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kSmem = STAGES * kStage;
  static_assert(kSmem >= BM * BN * 2, "the results are staged in the ring");
};

// 16-byte chunk c of row r of a tile of 128-byte rows, XOR-swizzled.
__device__ __forceinline__ uint32_t sw(uint32_t base, int r, int c) { return base + r * 128 + ((c ^ (r & 7)) << 4); }

// The 64 rotary values of tokens [m0, m1), head h, by `threads` threads (whole warps, `tid` counting them, that meet at
// named barrier `bar`): an item is four pairs of a token, eight items' loads a thread in flight before the first store
// (loads after stores wait for them, as far as the compiler knows: 6 us for 64 tokens).
__device__ __forceinline__ void rotary_tail(const MlaProjParams& p, int m0, int m1, int h, int tid, int threads, int bar) {
  __shared__ unsigned long long turns[kRope / 2];
  constexpr int kItems = 8;
  const bool half = p.layout != kRopeInterleaved;
  // two words of two values each: half layout the pairs' first and their second elements, else two pairs each
  const int j = (tid & 7) * 4;  // pairs j .. j + 3 (threads is a multiple of 8)
  const int e1 = half ? j : 2 * j, e2 = half ? j + kRope / 2 : 2 * j + 4;
  const int step = threads / 8;
  if (p.inv_freq != nullptr && tid < kRope / 2) turns[tid] = rope_turn(__ldg(p.inv_freq + tid));
  bool filled = p.inv_freq == nullptr;
  for (int mb = m0 + tid / 8; mb < m1 || !filled; mb += kItems * step) {
    uint2 a[kItems], b[kItems];
    int pos[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int m = mb + i * step;
      if (m >= m1) break;
      const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + m * p.x_token_stride + h * p.x_head_stride + kNope;
      a[i] = __ldg(reinterpret_cast<const uint2*>(x + e1));
      b[i] = __ldg(reinterpret_cast<const uint2*>(x + e2));
      pos[i] = p.inv_freq != nullptr ? __ldg(p.positions + m) : 0;
    }
    if (!filled) asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
    filled = true;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int m = mb + i * step;
      if (m >= m1) break;
      if (p.inv_freq != nullptr) {
        float v[8] = {__uint_as_float(a[i].x << 16), __uint_as_float(a[i].x & 0xffff0000u), __uint_as_float(a[i].y << 16),
                      __uint_as_float(a[i].y & 0xffff0000u), __uint_as_float(b[i].x << 16), __uint_as_float(b[i].x & 0xffff0000u),
                      __uint_as_float(b[i].y << 16), __uint_as_float(b[i].y & 0xffff0000u)};
        float y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = rope_cos_sin(pos[i], turns[j + k], p.scale);
          const float x1 = half ? v[k] : v[2 * k], x2 = half ? v[4 + k] : v[2 * k + 1];
          const float y1 = x1 * c.x - x2 * c.y, y2 = x2 * c.x + x1 * c.y;
          if (half) {
            y[k] = y1;
            y[4 + k] = y2;
          } else {
            y[2 * k] = y1;
            y[2 * k + 1] = y2;
          }
        }
        a[i] = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        b[i] = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(m) * p.num_heads + h) * p.out_width + kLat;
      *reinterpret_cast<uint2*>(o + e1) = a[i];
      *reinterpret_cast<uint2*>(o + e2) = b[i];
    }
  }
}

template <int WM, int WN, int MI, int NI, int STAGES, bool BT>
__global__ void __launch_bounds__(WM* WN * 32) gqa_mla_proj_kernel(const MlaProjParams p) {
  using T = ProjTile<WM, WN, MI, NI, STAGES, BT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / WN, wn = warp % WN;
  const int n0 = blockIdx.x * T::BN, h = blockIdx.y, m0 = blockIdx.z * T::BM;
  if (BT && n0 >= kLat) {
    rotary_tail(p, m0, min(m0 + T::BM, p.num_tokens), h, tid, T::kThreads, 0);  // a CTA of its own
    return;
  }
  constexpr int K = BT ? kNope : kLat;
  constexpr int kChunks = K / kBK;
  const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.x) + h * p.x_head_stride;
  const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(p.w) + (static_cast<int64_t>(h) * kWRows + (BT ? 0 : kNope)) * kLat;

  auto load = [&](int chunk) {
    const uint32_t as = sb + (chunk % STAGES) * T::kStage, bs = as + T::kABytes;
    const int k0 = chunk * kBK;
    for (int i = tid; i < T::BM * 8; i += T::kThreads) {
      const int r = i >> 3, c = i & 7, m = m0 + r;
      const bool in = m < p.num_tokens;
      cp_async_16(sw(as, r, c), a + (in ? m : 0) * p.x_token_stride + k0 + c * 8, in ? 16u : 0u);
    }
    if (BT) {  // [64 k][BN n]: BN / 64 blocks of 64 rows x 128 bytes
      for (int i = tid; i < kBK * (T::BN / 8); i += T::kThreads) {
        const int r = i / (T::BN / 8), c = i % (T::BN / 8);
        cp_async_16(sw(bs + (c >> 3) * (kBK * 128), r, c & 7), b + static_cast<int64_t>(k0 + r) * kLat + n0 + c * 8, 16u);
      }
    } else {
      for (int i = tid; i < T::BN * 8; i += T::kThreads) {
        const int r = i >> 3, c = i & 7;
        cp_async_16(sw(bs, r, c), b + static_cast<int64_t>(n0 + r) * kLat + k0 + c * 8, 16u);
      }
    }
  };

  float acc[MI][NI][4] = {};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (s < kChunks) load(s);
    cp_async_commit();
  }
  for (int ck = 0; ck < kChunks; ++ck) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();
    if (ck + STAGES - 1 < kChunks) load(ck + STAGES - 1);
    cp_async_commit();
    const uint32_t as = sb + (ck % STAGES) * T::kStage, bs = as + T::kABytes;
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      uint32_t af[MI][4];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        ldsm_x4(sw(as, (wm * MI + mi) * 16 + (lane & 15), 2 * kk + (lane >> 4)), af[mi][0], af[mi][1], af[mi][2],
                af[mi][3]);
#pragma unroll
      for (int nj = 0; nj < NI; nj += 2) {
        uint32_t b0, b1, b2, b3;
        const int n = (wn * NI + nj) * 8;
        if (BT) {
          const int c = (n >> 3) + (lane >> 4);
          ldsm_x4_trans(sw(bs + (c >> 3) * (kBK * 128), kk * 16 + (lane & 15), c & 7), b0, b1, b2, b3);
        } else {
          ldsm_x4(sw(bs, n + ((lane >> 4) << 3) + (lane & 7), 2 * kk + ((lane >> 3) & 1)), b0, b1, b2, b3);
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          mma_bf16_16816(acc[mi][nj], af[mi][0], af[mi][1], af[mi][2], af[mi][3], b0, b1);
          mma_bf16_16816(acc[mi][nj + 1], af[mi][0], af[mi][1], af[mi][2], af[mi][3], b2, b3);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring becomes the staging of the results: BM rows, BN / 64 blocks of 128 bytes a row

#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = (wm * MI + mi) * 16 + (lane >> 2) + 8 * half;
#pragma unroll
      for (int nj = 0; nj < NI; ++nj) {
        const int c = wn * NI + nj;  // 16-byte chunk of the row
        const uint32_t at = sw(sb + (c >> 3) * (T::BM * 128), r, c & 7) + 4 * (lane & 3);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pack_bf16(acc[mi][nj][2 * half], acc[mi][nj][2 * half + 1]))
                     : "memory");
      }
    }
  __syncthreads();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + h * p.out_width;
  const int64_t row = static_cast<int64_t>(p.num_heads) * p.out_width;
  for (int i = tid; i < T::BM * (T::BN / 8); i += T::kThreads) {
    const int r = i / (T::BN / 8), c = i % (T::BN / 8), m = m0 + r;
    if (m >= p.num_tokens) break;
    uint4 v;
    ld_shared_u4(sw(sb + (c >> 3) * (T::BM * 128), r, c & 7), v.x, v.y, v.z, v.w);
    *reinterpret_cast<uint4*>(out + m * row + n0 + c * 8) = v;
  }
}

// ------------------------------------------------------------ tensor memory
// Stages of A (128 tokens x 64 of K) and B. absorb_q: K = 128 in two stages of A, and B, all 128 weight rows of 256
// columns (N contiguous: four regions of 128 x 64), with the first. expand_out: K = 512 in eight chunks through four
// stages, B being 64 weight rows x 64 values (K contiguous).
template <bool ABSORB>
struct TcTile {
  static constexpr int BN = ABSORB ? 256 : 64, K = ABSORB ? kNope : kLat, kChunks = K / 64;
  static constexpr int kA = 128 * 128;                             // 128 tokens x 64 values
  static constexpr int kB = ABSORB ? 4 * kA : 64 * 128;            // all of B, or a chunk's
  static constexpr int kStages = ABSORB ? 2 : 4;
  static constexpr int kBOff = kStages * kA;
  static constexpr int kBytes = kBOff + (ABSORB ? kB : kStages * kB);  // the results are staged over the operands
  static constexpr int kBars = kBytes, kSlot = kBars + (2 * kStages + 1) * 8, kSmem = kSlot + 8 + 1024;
  static constexpr uint32_t kCols = BN;
  static_assert(kBytes >= 128 * BN * 2 && 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(!ABSORB || kLat / BN == 2, "each of a head's two CTAs takes half of the rotary values");
};

struct ProjMaps {
  CUtensorMap x, w, out;  // boxes of 64 values x 1 head x 128 tokens; of 64 x 128 (64) weight rows
};

constexpr uint64_t kDrainNs = kDefaultWaitLimitNs;

template <bool ABSORB>
__global__ void __launch_bounds__(128) gqa_mla_proj_tc_kernel(const MlaProjParams p, const __grid_constant__ ProjMaps maps) {
  using T = TcTile<ABSORB>;
  extern __shared__ uint8_t smem_raw[];
  const int n0 = blockIdx.x * T::BN, h = blockIdx.y, m0 = blockIdx.z * 128;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ volatile int abort_s;
  auto full = [&](int s) { return base + T::kBars + 8u * s; };
  auto freed = [&](int s) { return base + T::kBars + 8u * (T::kStages + s); };
  const uint32_t done = base + T::kBars + 8u * (2 * T::kStages);
  if (tid == 0) {
    for (int i = 0; i < 2 * T::kStages + 1; ++i) mbar_init(base + T::kBars + 8u * i, 1);
    abort_s = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) tc_alloc(base + T::kSlot, T::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + T::kSlot);
  auto wait = [&](uint32_t bar, uint32_t parity, int bit) {
    return __all_sync(0xffffffffu, tc_wait_limited(bar, parity, &abort_s, p.err, bit, p.wait_limit_ns));
  };

  int c = 0;
  if (warp == 1) {  // copies
    for (; c < T::kChunks; ++c) {
      const int s = c % T::kStages;
      if (c >= T::kStages && !wait(freed(s), ((c / T::kStages) - 1) & 1, kErrTimeoutEmpty)) break;
      const uint32_t bytes = T::kA + (ABSORB ? (c == 0 ? T::kB : 0) : T::kB);
      tma_load_3d_warp(base + s * T::kA, &maps.x, 64 * c, h, m0, full(s), bytes);
      if (!ABSORB)
        tma_load_2d_warp(base + T::kBOff + s * T::kB, &maps.w, 64 * c, h * kWRows + kNope + n0, full(s));
      else if (c == 0)
        for (int r = 0; r < 4; ++r)
          tma_load_2d_warp(base + T::kBOff + r * T::kA, &maps.w, n0 + 64 * r, h * kWRows, full(s));
    }
  } else if (warp == 0) {  // MMAs: the whole warp walks, one elected lane issues
    constexpr uint32_t idesc = tc_idesc_bf16(128, T::BN, false, ABSORB);
    const uint64_t da0 = tc_sdesc(base, 16, 1024, kSwizzle128B);
    // absorb_q's B: N in regions of 64 columns (LBO), K in 8-row groups (SBO); expand_out's: K-major rows
    const uint64_t db0 = tc_sdesc(base + T::kBOff, ABSORB ? T::kA : 16, 1024, kSwizzle128B);
    for (; c < T::kChunks; ++c) {
      const int s = c % T::kStages;
      if (!wait(full(s), (c / T::kStages) & 1, kErrTimeoutFull)) break;
      const uint64_t da = da0 + s * (T::kA >> 4), db = db0 + (ABSORB ? c * ((64 * 128) >> 4) : s * (T::kB >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        tc_mma_bf16_warp(tmem, da + ((kk * 32) >> 4), db + ((kk * (ABSORB ? 2048 : 32)) >> 4), idesc, (c | kk) ? 1u : 0u);
      if (!ABSORB) tc_commit_warp(freed(s));
    }
    tc_commit_warp(done);
    __syncwarp();
  } else if (ABSORB) {  // meanwhile: the rotary values of this CTA's half of the tokens
    const int t0 = m0 + 64 * blockIdx.x;
    rotary_tail(p, t0, min(t0 + 64, p.num_tokens), h, tid - 64, 64, 1);
    __syncwarp();
  }
  // every warp takes its 32 rows of the result
  const bool good = wait(done, 0, kErrTimeoutFull) && (warp > 1 || c == T::kChunks);
  __syncwarp();
  tc_fence_after();
  if (__syncthreads_and(good && !abort_s)) {  // the operands have been read: their place takes the results
    const int row = 32 * warp + lane;
#pragma unroll 1
    for (int r = 0; r < T::BN / 64; ++r) {
      uint32_t v[64];
      tc_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 64 * r, v);
      tc_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 64 * r + 32, v + 32);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_bf16(__uint_as_float(v[8 * c + 2 * e]), __uint_as_float(v[8 * c + 2 * e + 1]));
        st_shared_u4(sw(base + r * T::kA, row, c), o[0], o[1], o[2], o[3]);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      for (int r = 0; r < T::BN / 64; ++r) tma_store_3d(&maps.out, n0 + 64 * r, h, m0, base + r * T::kA);
      bulk_commit();
      bulk_wait_read<0>();
    }
  } else if (warp < 2 && lane == 0) {
    // gave up: no copy may still be writing shared memory, and no MMA reading it or writing tensor memory, when the CTA
    // leaves (bounded, and deaf to the abort flag)
    const uint64_t t0 = global_timer_ns();
    auto drain = [&](uint32_t bar, uint32_t parity) {
      while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kDrainNs) {
      }
    };
    if (warp == 0) drain(done, 0);
    else
      for (int i = c > T::kStages ? c - T::kStages : 0; i < c; ++i) drain(full(i % T::kStages), (i / T::kStages) & 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tc_dealloc(tmem, T::kCols);
}

template <bool ABSORB>
cudaError_t launch_tc(const MlaProjParams& p, cudaStream_t stream) {
  using T = TcTile<ABSORB>;
  static std::atomic<int> configured[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(gqa_mla_proj_tc_kernel<ABSORB>);
  const cudaError_t e = set_smem_limit_once(configured, fn, T::kSmem);
  if (e != cudaSuccess) return e;
  ProjMaps maps;
  const int64_t x_size[3] = {ABSORB ? kNope : kLat, p.num_heads, p.num_tokens}, x_pitch[2] = {2 * p.x_head_stride, 2 * p.x_token_stride};
  const int64_t o_size[3] = {p.out_width, p.num_heads, p.num_tokens}, o_pitch[2] = {2 * p.out_width, int64_t{2} * p.out_width * p.num_heads};
  const int box[3] = {64, 1, 128};
  constexpr CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!tc_encode(&maps.x, kBf, p.x, 3, x_size, x_pitch, box) || !tc_encode(&maps.out, kBf, p.out, 3, o_size, o_pitch, box) ||
      !tc_encode_2d(&maps.w, kBf, p.w, kLat, static_cast<int64_t>(p.num_heads) * kWRows, kLat * 2, 64, ABSORB ? 128 : 64))
    return cudaErrorInvalidValue;
  const dim3 grid((ABSORB ? kLat : kHeadV) / T::BN, p.num_heads, (p.num_tokens + 127) / 128);
  gqa_mla_proj_tc_kernel<ABSORB><<<grid, 128, T::kSmem, stream>>>(p, maps);
  return cudaGetLastError();
}

template <int WM, int WN, int MI, int NI, int STAGES, bool BT>
cudaError_t launch(const MlaProjParams& p, cudaStream_t stream) {
  using T = ProjTile<WM, WN, MI, NI, STAGES, BT>;
  static std::atomic<int> configured[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(gqa_mla_proj_kernel<WM, WN, MI, NI, STAGES, BT>);
  const cudaError_t e = set_smem_limit_once(configured, fn, T::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((BT ? kLat / T::BN + 1 : kHeadV / T::BN), p.num_heads, (p.num_tokens + T::BM - 1) / T::BM);
  gqa_mla_proj_kernel<WM, WN, MI, NI, STAGES, BT><<<grid, T::kThreads, T::kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// 16 tokens: the most that the mma.sync tile takes in one pass over the weights. Both forms in us a call, weights cold,
// absorb_q / expand_out (mma.sync; tensor memory). 128 heads: 16 tokens 5.9 / 5.5; 7.7 / 6.8, 32 tokens 7.8 / 8.3;
// 8.0 / 6.8, 64 tokens 11.8 / 12.0; 9.6 / 6.8, 128 tokens 19.8 / 19.4; 10.3 / 7.0. With few heads the crossover lies
// higher (16 heads: 16 tokens 2.5 / 3.8; 4.8 / 5.1, 64 tokens 3.0 / 3.8; 6.6 / 5.2, 128 tokens 4.5 / 4.3; 6.9 / 5.3),
// which the rule does not use.
cudaError_t launch_mla_absorb_q(const MlaProjParams& p, cudaStream_t stream) {
  return p.num_tokens <= 16 ? launch<1, 4, 1, 2, 3, true>(p, stream) : launch_tc<true>(p, stream);
}

cudaError_t launch_mla_expand_out(const MlaProjParams& p, cudaStream_t stream) {
  return p.num_tokens <= 16 ? launch<1, 4, 1, 2, 6, false>(p, stream) : launch_tc<false>(p, stream);
}

}  // namespace gqa
