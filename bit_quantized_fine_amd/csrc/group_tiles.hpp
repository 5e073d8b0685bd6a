// Tiles of token rows grouped by expert.  The rows of expert e are
// [offsets[e], offsets[e + 1]); the offsets lie in device memory (the router
// wrote them), so the host only knows an upper bound of the tiles and every
// workgroup finds its own tile here.
//
// Offsets are clamped to [0, M] and a group that ends before it starts is
// empty, so offsets the caller got wrong cannot lead outside the buffers.
#pragma once

#include "device_common.hpp"

namespace qnf4 {

// Wave-uniform; rows fit 32 bits (M < 2^31).  The values come out of
// readfirstlane, so that the compiler sees them as uniform and keeps the buffer
// descriptors built from them in scalar registers.
struct GroupTile {
  int e;      // expert, or -1: past the last tile
  int row0;   // first row of the tile
  int end;    // end of the expert's rows
};

__device__ __forceinline__ void group_range(const int* offsets, int64_t M, int e, int64_t& lo,
                                            int64_t& hi) {
  const int64_t a = offsets[e], b = offsets[e + 1];
  lo = a < 0 ? 0 : (a > M ? M : a);
  hi = b < lo ? lo : (b > M ? M : b);
}

// Number of tiles of tq rows.  Every lane of the wave takes one expert of 64
// at a time; the result is wave-uniform.
__device__ __forceinline__ int group_tile_count(const int* offsets, int E, int64_t M, int tq) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    if (e0 + lane < E) {
      int64_t lo, hi;
      group_range(offsets, M, e0 + lane, lo, hi);
      n += static_cast<int>((hi - lo + tq - 1) / tq);
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
  return __builtin_amdgcn_readfirstlane(n);
}

// Tile `slot` (wave-uniform) in expert order, e = -1 past the last one.
__device__ __forceinline__ GroupTile group_tile(const int* offsets, int E, int64_t M, int tq,
                                                int slot) {
  const int lane = threadIdx.x & 63;
  int e = -1, row0 = 0, end = 0, base = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int64_t lo = 0, hi = 0;
    if (e0 + lane < E) group_range(offsets, M, e0 + lane, lo, hi);
    const int n = static_cast<int>((hi - lo + tq - 1) / tq);
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const unsigned long long past = __ballot(base + incl > slot);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int first = base + __builtin_amdgcn_readlane(incl - n, l);
      e = e0 + l;
      row0 = __builtin_amdgcn_readlane(static_cast<int>(lo), l) + (slot - first) * tq;
      end = __builtin_amdgcn_readlane(static_cast<int>(hi), l);
      break;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return GroupTile{__builtin_amdgcn_readfirstlane(e), __builtin_amdgcn_readfirstlane(row0),
                   __builtin_amdgcn_readfirstlane(end)};
}

// Most tiles of tq rows that M rows of E experts can make.
inline int64_t group_tile_bound(int64_t M, int E, int64_t tq) {
  const int64_t groups = E < M ? E : M;
  return groups + (M - groups) / tq;
}

}  // namespace qnf4
