// Rank-r products of the layer grouped by expert: T = X . A_e and G = dY . B_e^T
// on each expert's rows, dB_e = s T_e^T dY_e and dA_e = s X_e^T G_e over them.
//
// T and G are tiled like the plain layer's (64 ranks x 128 tokens, reduction
// over K or N split so that about 256 workgroups run); a workgroup finds its
// expert's rows from the offsets, so a tile never straddles two experts.  dA
// and dB have one set of tiles per expert and reduce over that expert's rows
// only, in `splits` equal runs of its 64-row steps: an expert without rows
// writes zeros.  The partial sums of a split reduction are added in split
// order by a second launch (deterministic); without a split the result is
// written at once.
//
// With r = 64 and 8192 rows on 8 experts, T over 4096 columns takes 31 us, G and dB
// for 4096 columns 42 us and dA for 11008 columns 64 us (2.8 TB/s of X): bound by
// the traffic between L2 and the CUs, where the fp32 factor is read again by each
// of dA's column tiles, and by the largest expert's reductions.  (Largest experts
// first: 0.6% of the backward, less than the search cost other sizes; workgroups
// for two rounds instead of one: no change.)
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "group_tiles.hpp"
#include "kernels.hpp"
#include "rank_tiles.hpp"

namespace qnf4 {

namespace {

constexpr int RB_R = 64;     // tile of the rank dimension
constexpr int RB_X = 128;    // tile of the long dimension

template <int HL, class LP, class LQ>
constexpr int rank_lds() {
  return 2 * (LP::TILE + LQ::TILE + (HL == 0 ? 0 : (HL == 1 ? LP::TILE : LQ::TILE)));
}

template <int BP, int BQ>
__device__ __forceinline__ void scale_acc(Mma<BP, BQ>& mma, float scale) {
#pragma unroll
  for (int i = 0; i < Mma<BP, BQ>::TP; ++i)
#pragma unroll
    for (int j = 0; j < Mma<BP, BQ>::TQ; ++j) mma.acc[i][j] *= scale;
}

// C[m, j] = scale sum_k P_e[j, k] Q[m, k] on the rows m of every expert e.
struct RowsJob {
  OpParams po;        // P of expert 0
  int64_t pstride;    // elements from one expert's P to the next
  OpParams qo;        // Q [M][reduction]
  const int* offsets;
  int E;
  int64_t M;
  int r;
  int px, slots;      // rank tiles, token tiles at most
  int ntiles, tps;    // reduction tiles, and those of one split
  float* out;         // [splits][M][r]
  const uint64_t* state;
  uint32_t thr;
  // Applied here when there is one split.  Last in the structure: elsewhere the
  // compiler, which uses it as a vector, copies the fields behind it along into
  // a private array, moves that array to LDS and the workgroup past 64 KB with
  // it; workgroups then start so slowly that the gradient kernel of 8 experts
  // with 2 tokens each (4096 x 4096) took 17.2 us where it now takes 4.6.
  float scale;
};

template <class LP, class LQ>
__device__ __forceinline__ void rows_tile(const RowsJob& j, int x, int slot, int z, uint16_t* lds,
                                          int tid) {
  GroupTiles<RB_X> groups(j.offsets, j.E, j.M);
  groups.count();
  const GroupTile gt = groups.find(slot);
  if (gt.e < 0) return;
  const int64_t p0 = (int64_t)x * RB_R;
  const int kt0 = z * j.tps, kt1 = min(j.ntiles, kt0 + j.tps);
  Mma<RB_R, RB_X> mma;
  mma.zero();
  LP lp{j.po, p0};
  LQ lq{j.qo, gt.row0};
  lp.o.ptr = static_cast<const uint16_t*>(j.po.ptr) + gt.e * j.pstride;
  lq.o.nrows = gt.end;
  if constexpr (LQ::kDrop) lq.key = load_drop_key(j.state, j.thr);
  run_tiles<RB_R, RB_X, 0, 2>(lp, lq, kt0, kt1, mma, lds, tid);
  scale_acc(mma, j.scale);
  store_f32(mma, j.out + (int64_t)z * j.M * j.r, j.r, p0, gt.row0, j.r, gt.end, tid);
}

template <class LP, class LQ>
__global__ __launch_bounds__(NT) void k_group_rows(RowsJob j) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[rank_lds<0, LP, LQ>()];
  const int per = j.px * j.slots;
  const int z = blockIdx.x / per, t = blockIdx.x - z * per;
  rows_tile<LP, LQ>(j, t % j.px, t / j.px, z, lds, threadIdx.x);
}

// C_e[q, p] = scale sum_m P[m, p] Q[m, q] over the rows m of expert e; HL
// names the fp32 operand (1: P, 2: Q).
struct GradJob {
  OpParams po, qo;    // [M][P] and [M][Q], reduction-major
  const int* offsets;
  int E;
  int64_t M, P, Q;
  int px, qy, splits;
  uint16_t* out;      // [E][Q][P] bf16, one split
  float* ws;          // [splits][E][Q][P], more than one
  const uint64_t* state;
  uint32_t thr;
  float scale;        // last, as in RowsJob
};

template <int HL, int BP, int BQ, class LP, class LQ>
__device__ __forceinline__ void grad_tile(const GradJob& j, int blk, uint16_t* lds, int tid) {
  const int x = blk % j.px, y = (blk / j.px) % j.qy;
  const int ez = blk / (j.px * j.qy), e = ez % j.E, z = ez / j.E;
  int64_t lo, hi;
  group_range(j.offsets, j.M, e, lo, hi);
  const int ntiles = static_cast<int>((hi - lo + BK - 1) / BK);
  const int tps = (ntiles + j.splits - 1) / j.splits;
  const int kt0 = min(ntiles, z * tps), kt1 = min(ntiles, kt0 + tps);
  const int64_t p0 = (int64_t)x * BP, q0 = (int64_t)y * BQ;
  Mma<BP, BQ> mma;
  mma.zero();
  // the expert's rows of an operand of 2- or 4-byte elements
  auto rows = [&](const OpParams& o, int bytes) {
    return OpParams{static_cast<const char*>(o.ptr) + lo * o.ld * bytes, o.ld, o.nrows, hi - lo,
                    lo, o.scale};
  };
  LP lp{rows(j.po, HL == 1 ? 4 : 2), p0};
  LQ lq{rows(j.qo, HL == 2 ? 4 : 2), q0};
  if constexpr (LQ::kDrop) lq.key = load_drop_key(j.state, j.thr);
  run_tiles<BP, BQ, HL, 2>(lp, lq, kt0, kt1, mma, lds, tid);
  if (j.splits == 1) {
    scale_acc(mma, j.scale);
    store_bf16(mma, j.out + e * j.P * j.Q, j.P, p0, q0, j.P, j.Q, tid);
  } else {
    store_f32(mma, j.ws + ((int64_t)z * j.E + e) * j.P * j.Q, j.P, p0, q0, j.P, j.Q, tid);
  }
}

template <int HL, int BP, int BQ, class LP, class LQ>
__global__ __launch_bounds__(NT) void k_group_grad(GradJob j) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[rank_lds<HL, LP, LQ>()];
  grad_tile<HL, BP, BQ, LP, LQ>(j, blockIdx.x, lds, threadIdx.x);
}

// G's and dB's tiles in one launch (neither needs the other): workgroups
// [0, nrows) are G's, so that the two share the machine.
template <class LP, class LQ, int HL, int BP, int BQ, class LPG, class LQG>
__global__ __launch_bounds__(NT) void k_group_pair(RowsJob a, GradJob b, int nrows) {
  constexpr int LA = rank_lds<0, LP, LQ>(), LB = rank_lds<HL, LPG, LQG>();
  __shared__ __attribute__((aligned(16))) uint16_t lds[LA > LB ? LA : LB];
  const int blk = blockIdx.x;   // uniform: the branch is a scalar one
  if (blk < nrows) {
    const int per = a.px * a.slots;
    const int z = blk / per, t = blk - z * per;
    rows_tile<LP, LQ>(a, t % a.px, t / a.px, z, lds, threadIdx.x);
  } else {
    grad_tile<HL, BP, BQ, LPG, LQG>(b, blk - nrows, lds, threadIdx.x);
  }
}

// out[m][c] = scale sum_z part[z][m][c] on rows [offsets[0], offsets[E]);
// four columns a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void k_group_reduce(const float* part, int splits, int64_t M,
                                                      int64_t cols, float scale,
                                                      const int* offsets, int E, void* out) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  const int64_t count = M * cols;
  if (i >= count) return;
  const int64_t row = i / cols;
  if (row < offsets[0] || row >= offsets[E]) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int z = 0; z < splits; ++z)   // (unrolled: the loads go out together)
    s += *reinterpret_cast<const f32x4*>(part + (int64_t)z * count + i);
  s *= scale;
  if constexpr (BF16) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) =
        u32x2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = s;
  }
}

OpParams op(const void* p, int64_t ld, int64_t nrows, int64_t nred) {
  OpParams o{};
  o.ptr = p;
  o.ld = ld;
  o.nrows = nrows;
  o.nred = nred;
  o.scale = 1.f;
  return o;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct RowsPlan {
  int px, slots, ntiles, tps, splits;
};

// As the plain products: about one workgroup per CU, at least four reduction
// tiles a split.
RowsPlan plan_rows(int64_t M, int E, int64_t nred, int r) {
  RowsPlan p;
  p.px = static_cast<int>(cdiv(r, RB_R));
  p.slots = static_cast<int>(group_tile_bound(M, E, RB_X));
  p.ntiles = static_cast<int>(cdiv(nred, BK));
  const int64_t want = std::max<int64_t>(1, 256 / ((int64_t)p.px * p.slots));
  p.tps = static_cast<int>(std::max<int64_t>(4, cdiv(p.ntiles, want)));
  p.splits = static_cast<int>(cdiv(p.ntiles, p.tps));
  return p;
}

// Splits of an expert's rows for dA (len = K) or dB (len = N).
int grad_splits(int64_t M, int E, int64_t len, int r) {
  const int64_t tiles = cdiv(len, RB_X) * cdiv(r, RB_R) * E;
  const int64_t steps = cdiv(cdiv(M, E), BK);   // of an average expert
  return static_cast<int>(std::max<int64_t>(1, std::min(256 / tiles, steps / 4)));
}

RowsJob rows_job(const OpParams& po, int64_t pstride, const OpParams& qo, const int* offsets,
                 int E, int64_t M, int r, const RowsPlan& p, float scale, float* out,
                 const Drop& d) {
  RowsJob j{};
  j.po = po;
  j.pstride = pstride;
  j.qo = qo;
  j.offsets = offsets;
  j.E = E;
  j.M = M;
  j.r = r;
  j.px = p.px;
  j.slots = p.slots;
  j.ntiles = p.ntiles;
  j.tps = p.tps;
  j.scale = p.splits == 1 ? scale : 1.f;
  j.out = out;
  j.state = d.state;
  j.thr = d.thr;
  return j;
}

GradJob grad_job(const OpParams& po, const OpParams& qo, const int* offsets, int E, int64_t M,
                 int64_t P, int64_t Q, int bp, int bq, int splits, float scale, uint16_t* out,
                 float* ws, const Drop& d) {
  GradJob j{};
  j.po = po;
  j.qo = qo;
  j.offsets = offsets;
  j.E = E;
  j.M = M;
  j.P = P;
  j.Q = Q;
  j.px = static_cast<int>(cdiv(P, bp));
  j.qy = static_cast<int>(cdiv(Q, bq));
  j.splits = splits;
  j.scale = scale;
  j.out = out;
  j.ws = ws;
  j.state = d.state;
  j.thr = d.thr;
  return j;
}

}  // namespace

hipError_t launch_group_reduce(const float* part, int splits, int64_t M, int64_t cols, float scale,
                               const int* offsets, int E, float* f32, uint16_t* bf16,
                               hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(cdiv(M * cols / 4, 256)));
  if (f32)
    hipLaunchKernelGGL(k_group_reduce<false>, grid, dim3(256), 0, stream, part, splits, M, cols,
                       scale, offsets, E, f32);
  else
    hipLaunchKernelGGL(k_group_reduce<true>, grid, dim3(256), 0, stream, part, splits, M, cols,
                       scale, offsets, E, bf16);
  return hipGetLastError();
}

size_t grouped_down_ws_floats(int64_t M, int E, int64_t K, int r) {
  if (r <= 0 || M <= 0) return 0;
  const RowsPlan p = plan_rows(M, E, K, r);
  return p.splits > 1 ? (size_t)p.splits * M * r : 0;
}

size_t grouped_rank_ws_floats(int64_t M, int E, int64_t N, int64_t K, int r) {
  if (r <= 0 || M <= 0) return 0;
  const int sa = grad_splits(M, E, K, r), sb = grad_splits(M, E, N, r);
  size_t gb = grouped_down_ws_floats(M, E, N, r);   // G's, and dB's beside them
  if (sb > 1) gb += (size_t)sb * E * N * r;
  size_t f = std::max(grouped_down_ws_floats(M, E, K, r), gb);
  if (sa > 1) f = std::max<size_t>(f, (size_t)sa * E * K * r);
  return f;
}

int64_t grouped_rank_threads(int64_t M, int E, int64_t N, int64_t K, int r) {
  if (r <= 0 || M <= 0) return 0;
  auto rows = [&](int64_t nred) {
    const RowsPlan p = plan_rows(M, E, nred, r);
    return (int64_t)p.px * p.slots * p.splits;
  };
  auto grad = [&](int64_t len) {
    return cdiv(len, RB_X) * cdiv(r, RB_R) * E * grad_splits(M, E, len, r);
  };
  return NT * std::max(rows(K), std::max(rows(N) + grad(N), grad(K)));
}

hipError_t launch_grouped_down(const uint16_t* X, int64_t M, const int* offsets, int E, int64_t K,
                               const uint16_t* A, int r, float* T, float* ws, hipStream_t stream,
                               const Drop& d, int* nz) {
  const RowsPlan p = plan_rows(M, E, K, r);
  auto kern = d.on() ? k_group_rows<Bf16RedMajor<RB_R>, Bf16Nat<RB_X, true>>
                     : k_group_rows<Bf16RedMajor<RB_R>, Bf16Nat<RB_X>>;
  prof_begin(4, stream);
  hipLaunchKernelGGL(kern, dim3(p.px * p.slots * p.splits), dim3(NT), 0, stream,
                     rows_job(op(A, r, r, K), K * r, op(X, K, M, K), offsets, E, M, r, p,
                              d.scale(), p.splits > 1 ? ws : T, d));
  hipError_t e = hipGetLastError();
  if (nz)
    *nz = p.splits > 1 ? p.splits : 0;
  else if (e == hipSuccess && p.splits > 1)
    e = launch_group_reduce(ws, p.splits, M, r, d.scale(), offsets, E, T, nullptr, stream);
  prof_end(4, stream);
  return e;
}

hipError_t launch_grouped_grad_in_and_b(const uint16_t* dY, int64_t M, const int* offsets, int E,
                                        int64_t N, const uint16_t* B, const float* T, int r,
                                        float s, float* G, uint16_t* dB, float* ws,
                                        hipStream_t stream) {
  // G's partial sums, then dB's
  RowsPlan p{1, 0, 1, 1, 1};
  if (M > 0) p = plan_rows(M, E, N, r);
  const int nrows = p.px * p.slots * p.splits, sb = grad_splits(M, E, N, r);
  float* const wsb = ws + (p.splits > 1 ? (size_t)p.splits * M * r : 0);
  const RowsJob jg = rows_job(op(B, N, r, N), (int64_t)r * N, op(dY, N, M, N), offsets, E, M, r, p,
                              1.f, p.splits > 1 ? ws : G, {});
  const GradJob jb = grad_job(op(dY, N, N, M), op(T, r, r, M), offsets, E, M, N, r, RB_X, RB_R, sb,
                              s, dB, wsb, {});
  prof_begin(4, stream);
  hipLaunchKernelGGL((k_group_pair<Bf16Nat<RB_R>, Bf16Nat<RB_X>, 2, RB_X, RB_R,
                                   Bf16RedMajor<RB_X>, F32RedMajor<RB_R>>),
                     dim3(nrows + jb.px * jb.qy * E * sb), dim3(NT), 0, stream, jg, jb, nrows);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.splits > 1)
    e = launch_group_reduce(ws, p.splits, M, r, 1.f, offsets, E, G, nullptr, stream);
  if (e == hipSuccess && sb > 1)
    e = launch_split_reduce_bf16(wsb, sb, (int64_t)E * N * r, dB, stream, s);
  prof_end(4, stream);
  return e;
}

hipError_t launch_grouped_grad_a(const uint16_t* X, int64_t M, const int* offsets, int E,
                                 int64_t K, const float* G, int r, float s, uint16_t* dA,
                                 float* ws, hipStream_t stream, const Drop& d) {
  const int sa = grad_splits(M, E, K, r);
  const GradJob j = grad_job(op(G, r, r, M), op(X, K, K, M), offsets, E, M, r, K, RB_R, RB_X, sa,
                             s * d.scale(), dA, ws, d);
  auto kern = d.on()
      ? k_group_grad<1, RB_R, RB_X, F32RedMajor<RB_R>, Bf16RedMajor<RB_X, true>>
      : k_group_grad<1, RB_R, RB_X, F32RedMajor<RB_R>, Bf16RedMajor<RB_X>>;
  prof_begin(4, stream);
  hipLaunchKernelGGL(kern, dim3(j.px * j.qy * E * sa), dim3(NT), 0, stream, j);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && sa > 1)
    e = launch_split_reduce_bf16(ws, sa, (int64_t)E * K * r, dA, stream, s * d.scale());
  prof_end(4, stream);
  return e;
}

}  // namespace qnf4
