// Tiles of token rows grouped by expert.  The rows of expert e are
// [offsets[e], offsets[e + 1]); the offsets lie in device memory (the router
// wrote them), so the host only knows an upper bound of the tiles and every
// workgroup finds its own tile here.
//
// Offsets are clamped to [0, M] and a group that ends before it starts has no
// tiles, so offsets the caller got wrong cannot lead outside the buffers.
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

// Rows of expert e.
__device__ __forceinline__ void group_range(const int* offsets, int64_t M, int e, int64_t& lo,
                                            int64_t& hi) {
  const int64_t a = offsets[e], b = offsets[e + 1];
  lo = a < 0 ? 0 : (a > M ? M : a);
  hi = b < lo ? lo : (b > M ? M : b);
}

// Inclusive sum of v over the lanes of the wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The tiles of tq rows, dealt out in expert order.  Every wave finds them by
// itself: a lane takes one expert of 64 at a time.  The first 64 experts'
// offsets are loaded at construction, so that a kernel can have them on their
// way while it does something else; with no more than 64 they are loaded once.
template <int TQ>
class GroupTiles {
 public:
  __device__ __forceinline__ GroupTiles(const int* offsets, int E, int64_t M)
      : offsets_(offsets), E_(E), M_(static_cast<int>(M)) {
    load(0);
  }

  // Number of tiles (wave-uniform).
  __device__ __forceinline__ int count() {
    incl_ = wave_scan(tiles());
    int n = __builtin_amdgcn_readlane(incl_, 63);
    for (int e0 = 64; e0 < E_; e0 += 64) {
      load(e0);
      n += __builtin_amdgcn_readlane(wave_scan(tiles()), 63);
    }
    if (E_ > 64) {
      load(0);
      incl_ = wave_scan(tiles());
    }
    return n;
  }

  // Tile `slot` (wave-uniform); after count().
  __device__ __forceinline__ GroupTile find(int slot) {
    int base = 0;
    for (int e0 = 0;; e0 += 64) {
      const unsigned long long past = __ballot(base + incl_ > slot);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int first = base + __builtin_amdgcn_readlane(incl_ - tiles(), l);
        const int row0 = __builtin_amdgcn_readlane(lo_, l) + (slot - first) * TQ;
        return GroupTile{__builtin_amdgcn_readfirstlane(e0 + l),
                         __builtin_amdgcn_readfirstlane(row0),
                         __builtin_amdgcn_readlane(hi_, l)};
      }
      if (e0 + 64 >= E_) return GroupTile{-1, 0, 0};
      base += __builtin_amdgcn_readlane(incl_, 63);
      load(e0 + 64);
      incl_ = wave_scan(tiles());
    }
  }

 private:
  __device__ __forceinline__ void load(int e0) {
    const int e = e0 + static_cast<int>(threadIdx.x & 63);
    lo_ = hi_ = 0;
    if (e < E_) {
      lo_ = min(max(offsets_[e], 0), M_);
      hi_ = min(max(offsets_[e + 1], lo_), M_);
    }
  }
  __device__ __forceinline__ int tiles() const { return (hi_ - lo_ + TQ - 1) / TQ; }

  const int* offsets_;
  int E_, M_;
  int lo_, hi_, incl_;
};

// Deals V token tiles x P weight tiles out to the eight XCDs (workgroup b runs on
// XCD b % 8).  Of token tile v, XCD x takes weight tiles floor((x P + v % 8) / 8)
// up to the next XCD's first, token tile after token tile: its workgroups share
// few token tiles at a time and much the same weight tiles throughout, and over
// every eight token tiles each XCD gets P tiles, full and partial ones mixed.
// (Contiguous runs of all tiles gave some XCDs only full token tiles: one round
// of workgroups more than the others.  All token tiles of one weight tile next
// to each other read each XCD's tokens from beyond L2: 8% slower.)
struct XcdTile {
  int v, pt;   // v >= V: no work
};
__device__ __forceinline__ XcdTile xcd_deal(int b, int P) {
  const int x = b & 7;
  int i = b >> 3;
  int v = 8 * (i / P);
  i -= v / 8 * P;
  for (int ph = 0;; ++ph) {
    const int first = (x * P + ph) >> 3, n = (((x + 1) * P + ph) >> 3) - first;
    if (i < n || ph == 7) return XcdTile{v + ph, first + i};
    i -= n;
  }
}
inline int64_t xcd_deal_grid(int64_t V, int64_t P) { return 8 * P * ((V + 7) / 8); }

// Most tiles of tq rows that M rows of E experts can make.
inline int64_t group_tile_bound(int64_t M, int E, int64_t tq) {
  const int64_t groups = E < M ? E : M;
  return groups + (M - groups) / tq;
}

}  // namespace qnf4
