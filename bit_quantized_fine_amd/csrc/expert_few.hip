// Forward of the layer grouped by expert for few tokens (up to 16 rows an
// expert and tile): a stream over the weights of the experts that have rows.
//
// Workgroup = 8 waves on 32 weight rows of one expert; the waves split K in
// chunks of 128 (wave w takes chunks w, w + 8, ...), so that their 64-byte code
// segments are neighbours in memory, and each wave dequantizes its chunks
// straight into MFMA operands (k order as in expert_fwd.hip).  X is read from
// global memory: the rows a group does not have fall outside its buffer and
// move nothing, and with no X in LDS the loop has no barrier.  The LoRA update
// is added by wave w for ranks 32 w .. 32 w + 31, T's partial sums being added
// up on the way; then the waves' sums meet in LDS.  80 KB of LDS and 128
// registers put two workgroups on a CU, which hides the other's start: with
// three experts of 4096 x 4096 at one or two rows the calls' own latencies (the
// offsets, the first codes, T) are most of the time.
#include <type_traits>

#include "device_common.hpp"
#include "expert_args.hpp"
#include "group_tiles.hpp"
#include "kernels.hpp"
#include "rank_tiles.hpp"

namespace qnf4 {

namespace {

constexpr int FW = 8;            // waves, splitting K
constexpr int FT = 64 * FW;      // threads
constexpr int FF = 2;            // 16-row fragments
constexpr int FROWS = 16 * FF;   // weight rows
constexpr int FD = 2;            // chunks in flight a wave
constexpr int kFewLds = kRepTabBytes + 256 * FROWS * 2;   // level table, B's columns

// Weight rows 32 pt .. + 31 against the tile's tokens; with FOUR, of which there are
// 4 at most.
template <bool NODQ, bool FOUR>
__device__ __forceinline__ void few_tile(const ExpertArgs& a, uint8_t* dyn, const GroupTile& gt,
                                         int pt) {
  constexpr int XR = FOUR ? 1 : 4;   // X registers of 16 bytes a chunk
  uint16_t* const bst = reinterpret_cast<uint16_t*>(dyn + kRepTabBytes);   // B [r][FROWS]
  f32x4* const red = reinterpret_cast<f32x4*>(dyn);                        // [FW][FF][64]
  const int tid = threadIdx.x;
  const int wave = wave_id(), lane = tid & 63;
  const int li = lane & 15, g = lane >> 4;
  const int64_t N = a.N, K = a.K;
  const int K32 = static_cast<int>(K), KB = K32 / kBlock;
  const int64_t p0 = (int64_t)pt * FROWS, NW = N * a.E;
  const int rows = min(gt.end - gt.row0, 16);
  const int nchunks = (K32 + 127) / 128;

  const uint32_t nb = static_cast<uint32_t>(NW * K / kBlock);
  const BufRes rc = make_bufres(a.codes, static_cast<uint32_t>(NW * K / 2));
  const BufRes re = make_bufres(a.absmax_q, nb);
  const BufRes rd = make_bufres(a.absmax_scale, (NODQ ? nb : (nb + kGroup - 1) / kGroup) * 4u);
  const BufRes rx = make_bufres(a.X + (int64_t)gt.row0 * K, static_cast<uint32_t>(rows * K * 2));

  uint32_t cb[FF], eb[FF];
#pragma unroll
  for (int f = 0; f < FF; ++f) {
    const int64_t n = (int64_t)gt.e * N + p0 + 16 * f + li;
    cb[f] = static_cast<uint32_t>(n * (K / 2)) + 16u * g;   // + 64 c
    eb[f] = static_cast<uint32_t>(n * KB) + (g >> 1);       // + 2 c
  }
  // X: 16 bytes of step i of the lane's token li, + 256 c + 16 i.  Up to 4 tokens one
  // load a chunk fetches all steps: lane 4 i + t of a group takes step i of token t,
  // and step i's operand is shifted to lanes 0 .. 3 (the columns of the other lanes
  // are nobody's).  That is 7 vector memory instructions a chunk instead of 10: 21.0 -> 19.9
  // us at 4 rows of 8 experts of 4096 x 4096 on three of them, 33.9 -> 31.0 us for
  // 4096 x 11008.  (With three or four chunks in flight: 20.9 and 21.4 us.)
  const int xrow = FOUR ? li & 3 : li;
  const uint32_t xb =
      static_cast<uint32_t>(xrow * K32 + 32 * g + (FOUR ? 8 * (li >> 2) : 0)) * 2u;
  u32x4 cw[FD][FF], xw[FD][XR];
  uint32_t ce[FD][FF];
  float cd[FD][FF];
  auto load = [&](int c, int st) {
    const bool live = c < nchunks;
    const bool in = live && 2 * c + (g >> 1) < KB;   // (the second block of a half chunk: zeros)
#pragma unroll
    for (int f = 0; f < FF; ++f) {
      cw[st][f] = buf_load16(rc, live ? cb[f] + 64u * c : kOffNone);
      const uint32_t b = eb[f] + 2u * c;
      if constexpr (NODQ) {
        ce[st][f] = 1u;
        cd[st][f] = buf_load_f32(rd, in ? b * 4u : kOffNone);
      } else {
        ce[st][f] = buf_load_u8(re, in ? b : kOffNone);
        cd[st][f] = buf_load_f32(rd, in ? (b / kGroup) * 4u : kOffNone);
      }
    }
#pragma unroll
    for (int i = 0; i < XR; ++i)
      xw[st][i] = buf_load16(rx, in && xrow < rows ? xb + 256u * c + 16u * i : kOffNone);
  };
  auto operand = [&](int st, auto ic) {   // X of step i
    constexpr int I = decltype(ic)::value;
    if constexpr (!FOUR) {
      return xw[st][I];
    } else if constexpr (I == 0) {
      return xw[st][0];
    } else {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __builtin_amdgcn_update_dpp(0, static_cast<int>(xw[st][0][j]), 0x100 + 4 * I, 0xF,
                                           0xF, false);   // row_shl 4 I
      return v;
    }
  };
#pragma unroll
  for (int u = 0; u < FD; ++u) load(wave + FW * u, u);
  // B's columns: 16-byte piece tid (+ 512) is columns 8 (tid % 4) .. of rank tid / 4
  u32x4 bw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = tid / 4 + i * (FT / 4);
    const int64_t n = p0 + 8 * (tid % 4);
    bw[i] = j < a.r && n < N ? ld16(a.B + ((int64_t)gt.e * a.r + j) * N + n) : u32x4{0, 0, 0, 0};
  }

  f32x4 acc[FF];
#pragma unroll
  for (int f = 0; f < FF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t ta = rep_lane_base(lane);
  auto compute = [&](int st) {
    const u32x4 xo[4] = {operand(st, std::integral_constant<int, 0>{}),
                         operand(st, std::integral_constant<int, 1>{}),
                         operand(st, std::integral_constant<int, 2>{}),
                         operand(st, std::integral_constant<int, 3>{})};
#pragma unroll
    for (int f = 0; f < FF; ++f) {
      const float ch = NODQ ? cd[st][f] : static_cast<float>(ce[st][f]) * cd[st][f];
      f32x2 v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = cw[st][f][i];
        v[i][0] = rep_lookup<0>(ta, w);
        v[i][1] = rep_lookup<1>(ta, w);
        v[i][2] = rep_lookup<2>(ta, w);
        v[i][3] = rep_lookup<3>(ta, w);
      }
      __builtin_amdgcn_sched_barrier(0);   // all lookups before their first use
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u32x4 af;
#pragma unroll
        for (int b = 0; b < 4; ++b) af[b] = pack_bf16x2(v[i][b].x * ch, v[i][b].y * ch);
        acc[f] = mfma16(af, xo[i], acc[f]);
      }
    }
  };
  __syncthreads();   // the level table
  for (int c = wave; c < nchunks; c += FW * FD) {
#pragma unroll
    for (int u = 0; u < FD; ++u) {
      if (c + FW * u < nchunks) compute(u);
      load(c + FW * (u + FD), u);
    }
  }

  // LoRA update, ranks 32 wave + 8 g .. + 7 of token li
  const int j = 32 * wave + 8 * g;
  const bool mine = li < rows && j < a.r;
  f32x4 t0 = {0.f, 0.f, 0.f, 0.f}, t1 = t0;
  if (mine) {
    const int64_t at = (int64_t)(gt.row0 + li) * a.r + j, step = a.M * a.r;
    const float* src = a.T + at;
    if (a.nz > 0) {   // in split order
#pragma unroll 8
      for (int y = 0; y < a.nz; ++y, src += step) {
        t0 += *reinterpret_cast<const f32x4*>(src);
        t1 += *reinterpret_cast<const f32x4*>(src + 4);
      }
      t0 *= a.tscale;
      t1 *= a.tscale;
      if (pt == 0) {
        *reinterpret_cast<f32x4*>(a.Tout + at) = t0;
        *reinterpret_cast<f32x4*>(a.Tout + at + 4) = t1;
      }
    } else {
      t0 = *reinterpret_cast<const f32x4*>(src);
      t1 = *reinterpret_cast<const f32x4*>(src + 4);
    }
    t0 *= a.s;
    t1 *= a.s;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (tid / 4 + i * (FT / 4) < a.r) reinterpret_cast<u32x4*>(bst)[tid + i * FT] = bw[i];
  __syncthreads();   // B's columns; the table is no longer read
  if (32 * wave < a.r) {
    uint32_t hi[4], lo[4];
    split_bf16x2(t0.x, t0.y, hi[0], lo[0]);
    split_bf16x2(t0.z, t0.w, hi[1], lo[1]);
    split_bf16x2(t1.x, t1.y, hi[2], lo[2]);
    split_bf16x2(t1.z, t1.w, hi[3], lo[3]);
#pragma unroll
    for (int f = 0; f < FF; ++f) {
      u32x4 bf;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = j + 2 * i, col = 16 * f + li;
        const uint32_t b0 = k < a.r ? bst[k * FROWS + col] : 0u;
        const uint32_t b1 = k + 1 < a.r ? bst[(k + 1) * FROWS + col] : 0u;
        bf[i] = b0 | (b1 << 16);
      }
      acc[f] = mfma16(bf, u32x4{hi[0], hi[1], hi[2], hi[3]}, acc[f]);
      acc[f] = mfma16(bf, u32x4{lo[0], lo[1], lo[2], lo[3]}, acc[f]);
    }
  }
#pragma unroll
  for (int f = 0; f < FF; ++f) red[(wave * FF + f) * 64 + lane] = acc[f];
  __syncthreads();
  if (wave < FF) {   // fragment `wave`, its eight sums in order
    f32x4 v = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < FW; ++w) v += red[(w * FF + wave) * 64 + lane];
    const int64_t n = p0 + 16 * wave + 4 * g;
    if (li < rows && n < N)
      *reinterpret_cast<u32x2*>(a.Y + (int64_t)(gt.row0 + li) * N + n) =
          u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  }
}

}  // namespace

template <bool NODQ>
__global__ __launch_bounds__(FT, 4) void k_expert_few(ExpertArgs a, Nf4Tables tb) {
  // Dynamic LDS only: the level table sits at address 0; after the main loop
  // the waves' sums take its place.
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  GroupTiles<16> groups(a.offsets, a.E, a.M);
  build_rep_pair_table<FT>(reinterpret_cast<char*>(dyn), load_levels(tb), threadIdx.x);
  int pt, z;
  const GroupTile gt = expert_deal(a, groups, pt, z);
  if (gt.e < 0) return;
  if (gt.end - gt.row0 <= 4)
    few_tile<NODQ, true>(a, dyn, gt, pt);
  else
    few_tile<NODQ, false>(a, dyn, gt, pt);
}

namespace {

template <bool NODQ>
hipError_t launch_few(const ExpertArgs& a, const Nf4Tables& tb, hipStream_t stream) {
  static LdsLimit lds;
  const hipError_t attr = lds.raise(reinterpret_cast<const void*>(&k_expert_few<NODQ>), kFewLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_expert_few<NODQ>), dim3(static_cast<unsigned>(xcd_deal_grid(a.qtiles, a.ptiles))),
                     dim3(FT), kFewLds, stream, a, tb);
  return hipGetLastError();
}

}  // namespace

int64_t expert_few_threads(int64_t M, int E, int64_t N) {
  return FT * xcd_deal_grid(group_tile_bound(M, E, 16), (N + FROWS - 1) / FROWS);
}

hipError_t launch_expert_few(ExpertArgs a, bool dq, const Nf4Tables& tb, hipStream_t stream) {
  a.ptiles = static_cast<int>((a.N + FROWS - 1) / FROWS);
  a.qtiles = static_cast<int>(group_tile_bound(a.M, a.E, 16));
  a.splits = 1;
  a.part = nullptr;
  return dq ? launch_few<false>(a, tb, stream) : launch_few<true>(a, tb, stream);
}

}  // namespace qnf4
