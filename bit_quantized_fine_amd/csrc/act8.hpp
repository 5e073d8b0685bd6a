// The 8-bit checkpoint of activations: blocks of 64 values along a row, one
// signed byte a value and one fp32 constant a block.
//
//   c = fl32(amax / 127), amax the block's largest magnitude
//   code = rint(fl32(x / c)), -127 .. 127 (ties to even); 0 where c = 0
//   value = bf16(fl32(code c))
// A block that holds a NaN or an infinity gets c = NaN and codes 0: all of it
// comes back as NaN, so an overflow does not pass for a number.
//
// A value is off by half a step of its block, amax / 254, and by the rounding of the
// product to bf16, half a step of bf16: up to 2^-8 of the value, so that the largest
// values of a block lose up to as much again (1.87 half steps of the block at most, where
// amax is 1.0625; exactly one where it is a power of two).  The constant is not itself
// rounded to fewer bits: a power of two would cost up to one bit of every code, against
// 6% of the bytes.
#pragma once

#include "device_common.hpp"

namespace qnf4 {

// One block's constant and what its values are multiplied with.
struct Act8Scale {
  float c;      // the stored constant
  float inv;    // RN(1 / c); 0 where c is 0 or NaN
  bool slow;    // 1 / c or the quotient's remainder could leave fp32's normal range
  bool bad;     // the block holds a NaN or an infinity
};

// amax_bits: the largest of the block's values' bits without their signs, as
// bf16 bits in the high half of a word (a NaN's bits are above infinity's).
__device__ __forceinline__ Act8Scale act8_scale(uint32_t amax_bits) {
  Act8Scale s;
  s.bad = amax_bits >= 0x7F800000u;
  s.c = s.bad ? __builtin_nanf("") : __builtin_bit_cast(float, amax_bits) / 127.f;
  s.slow = s.c < 0x1p-96f;   // (false for NaN)
  s.inv = (s.c > 0.f && !s.slow) ? 1.f / s.c : 0.f;
  return s;
}

// The code of x in the low byte of the result.  The quotient is correctly
// rounded: from RN(1 / c), one multiplication and Markstein's correction (q +
// RN(1 / c) (x - q c), the remainder exact in an fma), or a division where some
// lane's constant has a reciprocal outside the normal range.  Adding 1.5 2^23
// then rounds it to an integer, ties to even, in the low bits.  No clamp is
// needed: c is below amax / 127 by a factor of at most 1 - 2^-10 (its smallest
// is a subnormal of ten bits), so no quotient reaches 127.5.
template <bool DIVIDE>
__device__ __forceinline__ uint32_t act8_code(float x, const Act8Scale& s) {
  float q;
  if constexpr (DIVIDE) {
    q = s.c > 0.f ? x / s.c : 0.f;
  } else {
    q = x * s.inv;
    q = fmaf(fmaf(-q, s.c, x), s.inv, q);
  }
  return s.bad ? 0u : __builtin_bit_cast(uint32_t, q + 12582912.f);
}

template <bool DIVIDE>
__device__ __forceinline__ u32x2 act8_codes_by(u32x4 v, const Act8Scale& s) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    b[2 * i] = act8_code<DIVIDE>(bf16_lo_to_f32(w), s);
    b[2 * i + 1] = act8_code<DIVIDE>(bf16_hi_to_f32(w), s);
  }
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000C0Cu);
    r[i] = lo | hi;
  }
  return r;
}

// Eight values (four dwords of bf16 pairs) -> eight codes.
__device__ __forceinline__ u32x2 act8_codes(u32x4 v, const Act8Scale& s) {
  return __builtin_amdgcn_ballot_w64(s.slow) != 0 ? act8_codes_by<true>(v, s)
                                                  : act8_codes_by<false>(v, s);
}

// The largest magnitude's bits (in the high half) of eight bf16 values.
__device__ __forceinline__ uint32_t amax_bits8(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    m = max(m, max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
  }
  return m;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
  return max(v, o);
}
// Maximum over the four or eight lanes of a block (aligned groups of lanes).
__device__ __forceinline__ uint32_t max_over4(uint32_t v) {
  return dpp_max_u32<0x4E>(dpp_max_u32<0xB1>(v));   // quad_perm 1,0,3,2 and 2,3,0,1
}
__device__ __forceinline__ uint32_t max_over8(uint32_t v) {
  return dpp_max_u32<0x141>(max_over4(v));          // row_half_mirror
}

// Eight codes (two dwords) -> eight values as bf16 pairs.  With 128 added to a
// code (its sign bit flipped) one instruction makes a byte a float, and one fma
// takes 128 c off again: u c - 128 c is code c before its one rounding.  Where 128 c
// overflows (a block whose largest value is the largest of bf16), the codes are
// extended instead, an instruction more each.
__device__ __forceinline__ u32x4 act8_values(uint32_t a, uint32_t b, float c) {
  const float off = -128.f * c;
  if (__builtin_amdgcn_ballot_w64(off == -__builtin_inff()) != 0) {
    auto f = [&](uint32_t w, int i) {
      return static_cast<float>(static_cast<int8_t>(w >> (8 * i))) * c;
    };
    return u32x4{pack_bf16x2(f(a, 0), f(a, 1)), pack_bf16x2(f(a, 2), f(a, 3)),
                 pack_bf16x2(f(b, 0), f(b, 1)), pack_bf16x2(f(b, 2), f(b, 3))};
  }
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  auto f = [&](uint32_t w, int i) {
    return fmaf(static_cast<float>((w >> (8 * i)) & 0xFFu), c, off);
  };
  return u32x4{pack_bf16x2(f(a, 0), f(a, 1)), pack_bf16x2(f(a, 2), f(a, 3)),
               pack_bf16x2(f(b, 0), f(b, 1)), pack_bf16x2(f(b, 2), f(b, 3))};
}

}  // namespace qnf4
