// Rotary angles shared by the rotary, append and latent-projection kernels.
//
// The angle of a pair at position p is p * f radians, f a double. Far
// positions lose it in 32 bits (p = 10^6, f = 1: a float's step is 0.06), and
// 64-bit floating-point products are slow on this part. So f is turned once
// into a fixed-point fraction of a turn a position, u = frac(f / 2 pi) * 2^64,
// and the fraction of a turn at p is the integer p * u mod 2^64: exact in
// integer arithmetic at every 32-bit position, whole turns dropping off the
// top. The upper 32 bits, rounded (2^-33 of a turn), go to sincospif.
#pragma once

#include <cstdint>

namespace gqa {

enum : int { kRopeHalf = 0, kRopeInterleaved = 1 };

// Fraction of a turn a position, in units of 2^-64.
__device__ __forceinline__ unsigned long long rope_turn(double inv_freq) {
  const double t = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
  return __double2ull_rd((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of position `pos`'s angle, times `scale`.
__device__ __forceinline__ float2 rope_cos_sin(int pos, unsigned long long turn, float scale) {
  const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(pos)) * turn + 0x80000000ull;
  const float half_turns = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, s * scale);
}

}  // namespace gqa
