// Rotary angles shared by the rotary, append and latent-projection kernels.
//
// The angle of a pair at position p is p * f radians, f a double. Far
// positions lose it in 32 bits (p = 10^6, f = 1: a float's step is 0.06), and
// 64-bit floating-point arithmetic is slow on this part. So f is turned once
// into a fixed-point fraction of a turn a position, u = frac(f / 2 pi) * 2^64,
// and the fraction of a turn at p is the integer p * u mod 2^64, whole turns
// dropping off the top. u is off by little more than 1 (a double's f / 2 pi would not
// do: its rounding, times p = 2^31, is up to 2^-20 radians at f = 3.7), so p * u by
// 2^-33 of a turn at every 32-bit position. Its upper 32 bits, rounded (2^-33 more),
// go to sincospif as a float: 2^-25 of a half turn, the largest of the three.
#pragma once

#include <cstdint>

namespace gqa {

enum : int { kRopeHalf = 0, kRopeInterleaved = 1 };

// Fraction of a turn a position, in units of 2^-64. With f = m 2^e, m of 53 bits, it is m times the 128 bits of
// 2^(e + 64) / (2 pi) around the binary point (what lies above them are whole turns): Payne and Hanek's reduction. In
// integers, which cost a step's call 0.2 to 0.4 us less than two-part doubles. Below 2^-75 it is 0, and from 2^117 on,
// where a double's own step is 2^65 radians, taken as 0.
__device__ __forceinline__ unsigned long long rope_turn(double inv_freq) {
  constexpr unsigned long long k0 = 0x28be60db9391054aull, k1 = 0x7f09d5f47d4d3770ull, k2 = 0x36d8a5664f10e410ull;  // 1 / (2 pi)
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(inv_freq));
  const int exponent = static_cast<int>(bits >> 52) & 0x7ff, e = exponent - 1011;
  if (e <= -64 || e > 128) return 0;
  const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  unsigned long long whole = 0, part = k0 >> (-e & 63);  // of 2^(e + 64) / (2 pi): the 64 bits above the point and below it
  if (e >= 0) {
    const int r = e & 63;
    const unsigned long long w0 = e < 64 ? 0 : (e < 128 ? k0 : k1), w1 = e < 64 ? k0 : (e < 128 ? k1 : k2),
                             w2 = e < 64 ? k1 : (e < 128 ? k2 : 0);
    whole = (w0 << r) | ((w1 >> 1) >> (63 - r));
    part = (w1 << r) | ((w2 >> 1) >> (63 - r));
  }
  const unsigned long long u = m * whole + __umul64hi(m, part);
  return (bits >> 63) != 0 ? 0 - u : u;
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
