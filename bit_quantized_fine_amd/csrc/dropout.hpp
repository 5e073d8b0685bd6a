// Adapter dropout: the keep mask of a tensor from a counter-based generator,
// regenerated wherever it is needed and never stored.
//
// Element i of a tensor (row-major index) belongs to piece i / 8.  The 128
// random bits of a piece are Philox4x32 with seven rounds (J. Salmon, M.
// Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC11: the fewest rounds that pass BigCrush) of the counter (piece, offset)
// under the key seed.  Element i takes 16-bit half i % 8, and is kept when
// that half is at least thr = min(round(65536 p), 65535); kept elements are
// scaled by 65536 / (65536 - thr), so the expectation is exact for the p that
// thr stands for.  Sixteen bits an element make one piece the eight bf16
// values of one 16-byte access: seven rounds are 14 multiplications (32 x 32
// -> 64) for eight elements, about half the time that reading and writing
// them takes.
#pragma once

#include "device_common.hpp"

namespace qnf4 {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The generator's key and counter offset, the same for every lane.
struct DropKey {
  uint32_t k0, k1, o0, o1;
  uint32_t thr;   // the threshold in both 16-bit halves
};
struct NoDropKey {};

// state: {seed, offset} in device memory, so a captured graph draws another
// mask on each replay when the caller advances the offset in between.
__device__ __forceinline__ DropKey load_drop_key(const uint64_t* state, uint32_t thr) {
  const uint64_t seed = state[0], off = state[1];
  DropKey k;
  k.k0 = static_cast<uint32_t>(seed);
  k.k1 = static_cast<uint32_t>(seed >> 32);
  k.o0 = static_cast<uint32_t>(off);
  k.o1 = static_cast<uint32_t>(off >> 32);
  k.thr = thr | (thr << 16);
  return k;
}

__device__ __forceinline__ u32x4 philox_piece(const DropKey& key, uint64_t piece) {
  uint32_t c0 = static_cast<uint32_t>(piece), c1 = static_cast<uint32_t>(piece >> 32);
  uint32_t c2 = key.o0, c3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Two 16-bit halves -> 0xFFFF where kept (half >= thr), 0 where dropped.
__device__ __forceinline__ uint32_t keep_bits(const DropKey& key, uint32_t w) {
  const u16x2 d = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, key.thr),
                                               __builtin_bit_cast(u16x2, w));
  const u16x2 one = {1, 1};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(d, one) - one);
}

// The 16-bit keep masks of the eight elements of a piece.
__device__ __forceinline__ u32x4 keep_piece(const DropKey& key, uint64_t piece) {
  const u32x4 w = philox_piece(key, piece);
  return u32x4{keep_bits(key, w.x), keep_bits(key, w.y), keep_bits(key, w.z),
               keep_bits(key, w.w)};
}

}  // namespace qnf4
