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
// bound is the bytes of weights and rows; mma.sync keeps up with HBM there
// (2 * tokens FLOP per weight byte). A CTA takes a head, BN output columns and
// BM tokens (16, 64 or 128, so that up to 128 tokens read the weights once) and
// streams K in chunks of 64 through a cp.async ring, absorb_q's two chunks at
// once. The results go through shared memory to 16-byte stores: a fragment's own
// are 4 bytes. Measured, 128 tokens x 128 heads: absorb_q 14.5 us (42 MB), expand_out
// 11.4 us (38 MB); 4 tokens x 16 heads: absorb_q 4.3 us. One wave of CTAs: its
// latency, not bytes, is what is left.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_ptx.cuh"
#include "gqa_rope.cuh"

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

// The 64 rotary values of tokens [m0, m1), head h: a thread takes four pairs of a token (a CTA of its own: at the end
// of one of the products they took longer than the product).
__device__ __forceinline__ void rotary_tail(const MlaProjParams& p, int m0, int m1, int h, int threads) {
  __shared__ unsigned long long turns[kRope / 2];
  if (p.inv_freq != nullptr) {
    if (threadIdx.x < kRope / 2) turns[threadIdx.x] = rope_turn(__ldg(p.inv_freq + threadIdx.x));
    __syncthreads();
  }
  const bool half = p.layout != kRopeInterleaved;
#pragma unroll 4
  for (int i = threadIdx.x; i < (m1 - m0) * 8; i += threads) {
    const int m = m0 + (i >> 3), j = (i & 7) * 4;  // pairs j .. j + 3
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + m * p.x_token_stride + h * p.x_head_stride + kNope;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(m) * p.num_heads + h) * p.out_width + kLat;
    // two words of two values each: half layout the pairs' first and their second elements, else two pairs each
    const int e1 = half ? j : 2 * j, e2 = half ? j + kRope / 2 : 2 * j + 4;
    uint2 a = *reinterpret_cast<const uint2*>(x + e1), b = *reinterpret_cast<const uint2*>(x + e2);
    if (p.inv_freq != nullptr) {
      const int pos = __ldg(p.positions + m);
      float v[8] = {__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                    __uint_as_float(a.y & 0xffff0000u), __uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                    __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u)};
      float y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 c = rope_cos_sin(pos, turns[j + k], p.scale);
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
      a = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
      b = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    }
    *reinterpret_cast<uint2*>(o + e1) = a;
    *reinterpret_cast<uint2*>(o + e2) = b;
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
    rotary_tail(p, m0, min(m0 + T::BM, p.num_tokens), h, T::kThreads);
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

cudaError_t launch_mla_absorb_q(const MlaProjParams& p, cudaStream_t stream) {
  if (p.num_tokens <= 16) return launch<1, 4, 1, 2, 3, true>(p, stream);   // 16 x 64
  if (p.num_tokens <= 64) return launch<2, 4, 2, 2, 3, true>(p, stream);   // 64 x 64
  return launch<4, 2, 2, 4, 3, true>(p, stream);                           // 128 x 64
}

cudaError_t launch_mla_expand_out(const MlaProjParams& p, cudaStream_t stream) {
  if (p.num_tokens <= 16) return launch<1, 4, 1, 2, 6, false>(p, stream);  // 16 x 64
  if (p.num_tokens <= 64) return launch<2, 4, 2, 2, 5, false>(p, stream);  // 64 x 64
  return launch<4, 2, 2, 4, 4, false>(p, stream);                          // 128 x 64
}

}  // namespace gqa
