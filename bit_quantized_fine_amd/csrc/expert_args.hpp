// Arguments of the kernels of the layer grouped by expert and the dealing out of
// their tiles.  (expert_dx.hip takes dY for X, G for T, A for B and dX for Y.)
#pragma once

#include "group_tiles.hpp"
#include "kernels.hpp"

namespace qnf4 {

constexpr uint32_t kOffNone = 0x80000000u;   // a buffer offset past the end of every buffer

struct ExpertArgs {
  const uint16_t* X;
  int64_t M;
  const int* offsets;
  int E;
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* absmax_scale;
  int64_t N, K;
  const float* T;     // [M][r], or (nz > 0) partial sums [nz][M][r] of it
  float* Tout;        // their sum goes here
  const uint16_t* B;
  uint16_t* Y;
  float* part;
  int nz, r;
  int ptiles, qtiles, splits, cps;
  // (last: fields used as vectors would take the ones behind them along into a
  // private array)
  float tscale;       // of T's partial sums
  float s;
  const uint64_t* state;   // dropout (dX only)
  uint32_t thr;
};

// The workgroup's tile: its token rows, weight row tile pt and split z of the
// reduction; e = -1 when there is no work for it.  Only the tiles that the
// groups have are dealt out (the grid holds the most that they could have).
template <int TQ>
__device__ __forceinline__ GroupTile expert_deal(const ExpertArgs& a, GroupTiles<TQ>& groups,
                                                 int& pt, int& z) {
  const int slots = min(a.qtiles, groups.count());
  const XcdTile t = xcd_deal(blockIdx.x, a.ptiles);
  pt = t.pt;
  z = 0;
  if (t.v >= slots * a.splits) return GroupTile{-1, 0, 0};
  z = t.v / slots;
  return groups.find(t.v - z * slots);
}

// The few-token form (expert_few.hip); fills in the tiles.
int64_t expert_few_threads(int64_t M, int E, int64_t N);
hipError_t launch_expert_few(ExpertArgs a, bool dq, const Nf4Tables& tb, hipStream_t stream);

// dX for many rows (expert_dx.hip), without a split reduction.
bool expert_dx_fits(int64_t M, int E, int64_t K);
int64_t expert_dx_threads(int64_t M, int E, int64_t K);
hipError_t launch_expert_dx(const uint16_t* dY, int64_t M, const int* offsets, int E,
                            const Nf4View& w, const float* G, const uint16_t* A, int r, float s,
                            uint16_t* dX, const Nf4Tables& tb, hipStream_t stream,
                            const Drop& d);

}  // namespace qnf4
