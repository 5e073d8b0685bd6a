// Forward of the layer grouped by expert, Y = X . deq(W_e)^T + s . T . B_e on
// each expert's rows, on bf16 MFMA with the weights dequantized straight into
// MFMA operands.
//
// Workgroup = 8 waves, tile = 128 FR weight rows x 16 TB tokens of one expert.
// Wave w owns 16 FR rows and all tokens of the tile, so every weight is
// dequantized by exactly one wave and never passes through LDS: lane l = 16 g
// + i loads the 16 code bytes at 16 g of row i's 64-byte segment of a 128-k
// chunk, and dword t of them, dequantized, is the lane's share of the 16 x 32
// operand of step t (k = 32 g + 8 t .. + 7).  X is what the waves share: it is
// staged through LDS in the same k order, double-buffered, one barrier a chunk,
// its 16-byte pieces XOR-swizzled by row; with 192 tokens it fills the 160 KB of
// LDS together with the level table (half chunks, which need less, and two
// barriers a chunk: 2% slower).  The operands of the next step are dequantized
// while the MFMAs of the current one run.  X waits one or two chunks ahead in
// registers.
//
// Measured: 8 experts of 11008 x 4096, r = 64, 8192 rows: 765 to 785 us for the whole
// forward on most cards (740 on the best), 0.96 to 0.99 PFLOP/s where a large matrix
// product of the library reaches 1.38: bound by the chip's power.  Of the loop's
// time the lookups take 19%, scaling and packing 11%, X's reads 7% (timed without
// each).  96 rows on seven of the same experts: 57 us for this kernel, 2.8 TB/s of
// codes (67 us with T's two launches).
//
// The offsets are read on the GPU: the grid holds the most tiles the groups
// could make, a workgroup finds its expert and rows in them, and the last tile
// of a group runs the narrowest body that holds its rows.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "expert_args.hpp"
#include "group_tiles.hpp"
#include "kernels.hpp"
#include "rank_tiles.hpp"

namespace qnf4 {

namespace {

constexpr int EW = 8;            // waves
constexpr int ET = 64 * EW;      // threads

template <int FR, int TB>
struct ExpertTile {
  static constexpr int ROWS = 16 * FR * EW;       // weight rows
  static constexpr int TQ = 16 * TB;              // tokens
  static constexpr int PPR = 16;                  // 16-byte pieces of a token row's chunk
  static constexpr int XBUF = TQ * PPR * 8;       // elements of one X buffer
  static constexpr int PIECES = TQ * PPR;
  static constexpr int PP = (PIECES + ET - 1) / ET;   // pieces a thread stages
  static constexpr bool STREAM = FR == 1 && TB <= 2;   // bound by the stream of codes
  static constexpr int D = STREAM ? 4 : 2;        // code stages (128-k chunks)
  static constexpr int XST = TB > 8 ? 1 : 2;      // register stages of X
  static constexpr int MAIN = kRepTabBytes + 2 * XBUF * 2;
  static constexpr int TAIL = ROWS * 128 + TQ * 256;   // B tile, T hi and lo tiles
  static constexpr int YROW = ROWS + 8;                // a token row of the output tile
  static constexpr int OUT = TQ * YROW * 2;
  static constexpr int LDS = MAIN > TAIL ? (MAIN > OUT ? MAIN : OUT) : (TAIL > OUT ? TAIL : OUT);
};

// The narrower bodies a kernel of TB token subtiles holds (0: none): 12 -> 4,
// 8; 4 -> 1, 2; 2 -> 1.  Its LDS is that of the largest.
constexpr int narrow1(int tb) { return tb > 4 ? 4 : tb / 4; }
constexpr int narrow2(int tb) { return tb > 4 ? 8 : tb / 2; }
template <int FR, int TB>
constexpr int expert_lds() {
  int lds = ExpertTile<FR, TB>::LDS;
  if constexpr (narrow1(TB) > 0)
    lds = lds > ExpertTile<FR, narrow1(TB)>::LDS ? lds : ExpertTile<FR, narrow1(TB)>::LDS;
  if constexpr (narrow2(TB) > 0)
    lds = lds > ExpertTile<FR, narrow2(TB)>::LDS ? lds : ExpertTile<FR, narrow2(TB)>::LDS;
  return lds;
}

// Slot of 16-byte piece q of token row `row`.
template <int PPR>
__device__ __forceinline__ int xslot(int row, int q) {
  return PPR == 16 ? q ^ (row & 15) : q ^ ((row >> 1) & 7);
}

template <int FR, int TB, bool NODQ>
__device__ __forceinline__ void expert_tile(const ExpertArgs& a, uint8_t* dyn, int e, int64_t q0,
                                            int64_t mend, int pt, int z) {
  using Tile = ExpertTile<FR, TB>;
  constexpr int PPR = Tile::PPR, PP = Tile::PP;
  constexpr int XST = Tile::XST, D = Tile::D;
  constexpr int GB = TB >= 8 ? 2 : TB, NG = TB / GB;   // token subtiles a group, groups
  uint16_t* const Xs = reinterpret_cast<uint16_t*>(dyn + kRepTabBytes);
  const int tid = threadIdx.x;
  const int wave = wave_id(), lane = tid & 63;
  const int li = lane & 15, g = lane >> 4;
  const int64_t N = a.N, K = a.K;
  const int K32 = static_cast<int>(K), KB = K32 / kBlock;
  const int64_t p0 = (int64_t)pt * Tile::ROWS;
  const int64_t NW = N * a.E;
  const int c0 = z * a.cps;
  const int nchunks = min((K32 + 127) / 128, c0 + a.cps);   // end of this split's chunks

  // rows past W and tokens past the tile read as zero
  const uint32_t nb = static_cast<uint32_t>(NW * K / kBlock);
  const BufRes rc = make_bufres(a.codes, static_cast<uint32_t>(NW * K / 2));
  // (the windows below read whole aligned dwords of the 8-bit constants)
  constexpr bool WIN = Tile::STREAM && !NODQ;
  const uint32_t eoff =
      WIN ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.absmax_q)) & 3u : 0u;
  const BufRes re = make_bufres(a.absmax_q - eoff, WIN ? (eoff + nb + 3u) & ~3u : nb);
  const BufRes rd = make_bufres(a.absmax_scale, (NODQ ? nb : (nb + kGroup - 1) / kGroup) * 4u);
  const int64_t tile_rows = mend - q0 < Tile::TQ ? mend - q0 : Tile::TQ;
  const BufRes rx = make_bufres(a.X + q0 * K, static_cast<uint32_t>(tile_rows * K * 2));

  // codes and constants of the lane's FR rows, D chunks in flight
  uint32_t cb[FR], eb[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    const int64_t n = (int64_t)e * N + p0 + 16 * (FR * wave + f) + li;
    cb[f] = static_cast<uint32_t>(n * (K / 2)) + 16u * g;        // + 64 c
    eb[f] = static_cast<uint32_t>(n * KB) + (g >> 1);            // + 2 c
  }
  u32x4 cw[D][FR];
  uint32_t ce[D][FR];
  float cd[D][FR];
  auto load_codes = [&](int c, int st) {
    const bool live = c < nchunks;
    const bool blk = live && 2 * c + (g >> 1) < KB;   // the half chunk past K: constant 0
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      cw[st][f] = buf_load16(rc, live ? cb[f] + 64u * c : kOffNone);
      const uint32_t b = eb[f] + 2u * c;
      if constexpr (NODQ) {
        cd[st][f] = buf_load_f32(rd, blk ? b * 4u : kOffNone);
      } else if constexpr (!WIN) {
        ce[st][f] = buf_load_u8(re, blk ? b : kOffNone);
        cd[st][f] = buf_load_f32(rd, blk ? (b / kGroup) * 4u : kOffNone);
      }
    }
  };

  // Tiles of few tokens are bound by the code stream's vector memory instructions:
  // without those of the constants, two a chunk and fragment, 96 rows of 8 experts
  // of 11008 x 4096 took 61 us instead of 77.  So their constants come 16 chunks at
  // a time, in five loads: lane group g holds the 8-bit constants of blocks 8 g ..
  // + 7 of a window of 32 (three aligned dwords, shifted), every lane the window's
  // two possible second-level scales, and a chunk takes its constants from the
  // lanes that hold them: 67 us, and 65 with four chunks of codes in flight.  (With
  // more registers in use, the window's spill or cost more than they save: 39
  // against 38 us at 256 rows of 8 experts of 4096 x 4096.)
  uint32_t wraw[FR][3], wlo[FR], whi[FR];
  float dnext[FR][2], dlo[FR], dhi[FR];
  auto window_load = [&](int w) {
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      const uint32_t b = eb[f] - (g >> 1) + 2u * c0 + 32u * w;   // first block of the window
      const uint32_t at = (eoff + b + 8u * g) & ~3u;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        wraw[f][i] = __builtin_amdgcn_raw_buffer_load_b32(re, at + 4u * i, 0, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) dnext[f][i] = buf_load_f32(rd, (b / kGroup + i) * 4u);
    }
  };
  auto window_take = [&]() {
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      const uint32_t sh = (eoff + eb[f] - (g >> 1) + 2u * c0) & 3u;
      wlo[f] = __builtin_amdgcn_alignbyte(wraw[f][1], wraw[f][0], sh);
      whi[f] = __builtin_amdgcn_alignbyte(wraw[f][2], wraw[f][1], sh);
      dlo[f] = dnext[f][0];
      dhi[f] = dnext[f][1];
    }
  };

  // X piece idx = tid + 512 j: token row idx / 16, piece q = idx % 16.  Piece q = g
  // + 4 i is what lane group g takes at step i: k = 128 c + 8 (4 g + i) .. + 7.  In
  // this order a 16-byte read, which the LDS serves in groups of 16 lanes of two
  // g's, meets no bank twice; with q = 4 g + i it met every second one twice (784
  // instead of 822 us for the 8192 rows above).
  // (A thread's pieces are whole rows apart, so they share q and the swizzle.)
  static_assert(ET % PPR == 0 && (ET / PPR) % 16 == 0, "piece rows apart");
  const int xrow = tid / PPR, xq = tid % PPR;
  const int xcp = 4 * (xq & 3) + (xq >> 2);
  const uint32_t xsrc = static_cast<uint32_t>(xrow * K32 + 8 * xcp) * 2u;
  const uint32_t xstep = static_cast<uint32_t>(ET / PPR * K32) * 2u;
  uint16_t* const xdst = Xs + (xrow * PPR + xslot<PPR>(xrow, xq)) * 8;
  const bool xlive = Tile::PIECES % ET == 0 || tid < Tile::PIECES;
  u32x4 xw[XST][PP];
  auto load_x = [&](int c, int st) {
    const bool ok = xlive && c < nchunks && 128 * c + 8 * xcp < K32;
    const uint32_t o = ok ? xsrc + 256u * c : kOffNone;   // (+ j xstep < 2^31: stays past the end)
#pragma unroll
    for (int j = 0; j < PP; ++j) xw[st][j] = buf_load16(rx, o + j * xstep);
  };
  auto store_x = [&](int st, int buf) {
    if (xlive) {
#pragma unroll
      for (int j = 0; j < PP; ++j)
        *reinterpret_cast<u32x4*>(xdst + buf * Tile::XBUF + j * ET * 8) = xw[st][j];
    }
  };

  f32x4 acc[FR][TB];
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[f][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The level pairs of the 8 codes of step t, and bf16_rne(fl32(level * c)) of a
  // pair.
  struct Pairs {
    f32x2 v[4];
  };
  const uint32_t ta = rep_lane_base(lane);
  auto lookup = [&](int st, int f, int t) {
    const uint32_t w = cw[st][f][t];
    return Pairs{{rep_lookup<0>(ta, w), rep_lookup<1>(ta, w), rep_lookup<2>(ta, w),
                  rep_lookup<3>(ta, w)}};
  };
  // Constant of chunk c, codes in stage st, row fragment f (the half chunk past K:
  // 0).
  auto constant = [&](int c, int st, int f) {
    if constexpr (NODQ) {
      return cd[st][f];
    } else if constexpr (!WIN) {
      return static_cast<float>(ce[st][f]) * cd[st][f];
    } else {
      const int t = c - c0;
      const uint32_t b = eb[f] + 2u * c, b0 = eb[f] - (g >> 1) + 2u * (c0 + (t & ~15));
      const uint32_t lo = wlo[f], hi = whi[f];
      const uint32_t q =
          __builtin_amdgcn_ds_bpermute(4 * (li + 16 * ((t & 15) >> 2)), (t & 2) ? hi : lo);
      const float e = static_cast<float>((q >> (16 * (t & 1) + 8 * (g >> 1))) & 255u);
      const float d0 = dlo[f], d1 = dhi[f];
      return 2 * c + (g >> 1) < KB ? e * (b / kGroup == b0 / kGroup ? d0 : d1) : 0.f;
    }
  };
  auto scaled = [&](const Pairs& p, int t, float ch) {
    return pack_bf16x2(p.v[t].x * ch, p.v[t].y * ch);
  };
  // step i of the staging, token subtile b: token row 16 b + li, whose swizzle
  // is that of row li
  const uint16_t* const xsrow = Xs + li * PPR * 8;
  auto read_x = [&](int buf, int i, int b) {
    return *reinterpret_cast<const u32x4*>(xsrow + 8 * ((g + 4 * i) ^ li) + buf * Tile::XBUF +
                                           16 * b * PPR * 8);
  };

#pragma unroll
  for (int i = 0; i < D; ++i) load_codes(c0 + i, i);
  if constexpr (WIN) window_load(0);
  load_x(c0, 0);
  if constexpr (XST == 2) load_x(c0 + 1, 1);
  __syncthreads();   // the level table
  store_x(0, 0);
  load_x(c0 + XST, 0);
  if constexpr (WIN) {
    window_take();
    window_load(1);
  }
  u32x4 af[2][FR];   // operands of the current and the next step
  float ch[FR];      // constants of the codes that are next to be scaled
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    const Pairs p = lookup(0, f, 0);
    ch[f] = constant(c0, 0, f);
#pragma unroll
    for (int t = 0; t < 4; ++t) af[0][f][t] = scaled(p, t, ch[f]);
  }
  __syncthreads();
  // Chunk c, codes in stage ST.  A step's products run in groups of GB token
  // subtiles.  While a group's MFMAs run, the X operands of the next group and (at
  // a step's first group) the level pairs of the next step are on their way from
  // LDS; the pairs become operands one at a time between the later MFMAs, whose
  // pipe they leave busy.  The scheduling barriers keep that order: left alone,
  // the compiler issues a pair's two lookups next to their use and waits for each.
  // Groups of 2 subtiles against 4 and 3: 754, 770 and 764 us (192-token tiles, 8
  // experts of 11008 x 4096, 8192 rows); pairs scaled in one run behind a step's
  // last group: 761.  All of it is within a few percent because the chip is at its
  // power limit here: the main loop runs at 1.9 to 2.0 GHz, its MFMAs taking 62%
  // of the cycles.
  constexpr int SLOTS = TB * FR, PAIRS = 4 * FR, SLOT0 = SLOTS / 3;   // of a step
  auto chunk = [&](int c, auto stc) {
    constexpr int ST = decltype(stc)::value;
    constexpr int buf = ST & 1, xs = XST == 2 ? (ST + 1) & 1 : 0;
    u32x4 xf[2][GB];
#pragma unroll
    for (int b = 0; b < GB; ++b) xf[0][b] = read_x(buf, 0, b);
    Pairs pr[FR];
#pragma unroll
    for (int k = 0; k < 4 * NG; ++k) {
      const int i = k / NG;                      // step of the chunk
      const int nst = i < 3 ? ST : (ST + 1) % D;   // codes of the next step
      if (k % NG == 0) {
#pragma unroll
        for (int f = 0; f < FR; ++f) pr[f] = lookup(nst, f, (i + 1) % 4);
        if (i == 3) {
          if constexpr (WIN) {
            if (((c + 1 - c0) & 15) == 0) {
              window_take();
              window_load(((c + 1 - c0) >> 4) + 1);
            }
          }
#pragma unroll
          for (int f = 0; f < FR; ++f) ch[f] = constant(c + 1, nst, f);
        }
      }
      if (k + 1 < 4 * NG) {
#pragma unroll
        for (int b = 0; b < GB; ++b)
          xf[(k + 1) & 1][b] = read_x(buf, (k + 1) / NG, GB * ((k + 1) % NG) + b);
      }
      if (k == 0) {   // X of the next chunk, then the registers' next load
        store_x(xs, buf ^ 1);
        load_x(c + 1 + XST, xs);
      }
      if (k == 3 * NG) load_codes(c + D, ST);   // stage ST is used up
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < GB; ++b)
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          acc[f][GB * (k % NG) + b] =
              mfma16(af[i & 1][f], xf[k & 1][b], acc[f][GB * (k % NG) + b]);
          const int slot = (k % NG * GB + b) * FR + f;
#pragma unroll
          for (int u = 0; u < PAIRS; ++u)
            if (SLOT0 + u * (SLOTS - SLOT0) / PAIRS == slot)
              af[(i + 1) & 1][u / 4][u % 4] = scaled(pr[u / 4], u % 4, ch[u / 4]);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
  };
  // A chunk count that D does not divide adds passes over chunks past the end,
  // all zeros.
  for (int c = c0; c < nchunks; c += D) {
    chunk(c, std::integral_constant<int, 0>{});
    chunk(c + 1, std::integral_constant<int, 1>{});
    if constexpr (D == 4) {
      chunk(c + 2, std::integral_constant<int, 2>{});
      chunk(c + 3, std::integral_constant<int, 3>{});
    }
  }

  // LoRA update (the first split only): 64 ranks at a time, the B tile [64
  // ranks][ROWS] as it lies in memory, read with transposing loads, and s . T as
  // bf16 hi and lo tiles [TQ][64] in swizzled 128-byte rows.  (The two halves keep
  // 16 of the fp32 value's 24 bits, of which the bf16 result keeps 8.)
  if (a.r > 0 && z == 0) {
    uint16_t* const bt = reinterpret_cast<uint16_t*>(dyn);
    uint16_t* const th = bt + Tile::ROWS * 64;
    uint16_t* const tl = th + Tile::TQ * 64;
    const uint16_t* const Be = a.B + (int64_t)e * a.r * N;
    for (int j0 = 0; j0 < a.r; j0 += 64) {
      // (all loads of the step before the first store, so that one latency
      // serves them)
      constexpr int BP = Tile::ROWS * 8 / ET;   // 16-byte pieces of B a thread
      u32x4 bw[BP];
#pragma unroll
      for (int i = 0; i < BP; ++i) {
        const int idx = tid + ET * i, red = idx / (Tile::ROWS / 8), pc = idx % (Tile::ROWS / 8);
        const int64_t n = p0 + 8 * pc;
        bw[i] = j0 + red < a.r && n < N ? ld16(Be + (int64_t)(j0 + red) * N + n)
                                        : u32x4{0, 0, 0, 0};
      }
      constexpr int TP = (Tile::TQ * 16 + ET - 1) / ET;   // 4-rank pieces of T a thread
      f32x4 tw[TP];
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int idx = tid + ET * i, row = idx / 16, j = j0 + 4 * (idx % 16);
        tw[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (row < Tile::TQ && q0 + row < mend && j < a.r)
          tw[i] = *reinterpret_cast<const f32x4*>(a.T + (q0 + row) * a.r + j);
      }
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int idx = tid + ET * i, row = idx / 16, q = idx % 16;
        if (row < Tile::TQ) {
          const f32x4 v = tw[i] * a.s;
          uint32_t h0, h1, l0, l1;
          split_bf16x2(v.x, v.y, h0, l0);
          split_bf16x2(v.z, v.w, h1, l1);
          const int o = (row * 8 + xslot<8>(row, q >> 1)) * 8 + 4 * (q & 1);
          *reinterpret_cast<u32x2*>(th + o) = u32x2{h0, h1};
          *reinterpret_cast<u32x2*>(tl + o) = u32x2{l0, l1};
        }
      }
#pragma unroll
      for (int i = 0; i < BP; ++i) {
        const int idx = tid + ET * i, red = idx / (Tile::ROWS / 8), pc = idx % (Tile::ROWS / 8);
        st_lds16(bt + (pc / 16) * 64 * 128 + red * 128 + 8 * rm_slot<128>(red, pc % 16), bw[i]);
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 bf[FR];
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          const int col = 16 * (FR * wave + f);
          bf[f] = rm_frag<128>(bt + (col / 128) * 64 * 128, col % 128, ks, lane);
        }
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          const int row = 16 * b + li;
          const int o = (row * 8 + xslot<8>(row, 4 * ks + g)) * 8;
          const u32x4 hi = *reinterpret_cast<const u32x4*>(th + o);
          const u32x4 lo = *reinterpret_cast<const u32x4*>(tl + o);
#pragma unroll
          for (int f = 0; f < FR; ++f) {
            acc[f][b] = mfma16(bf[f], hi, acc[f][b]);
            acc[f][b] = mfma16(bf[f], lo, acc[f][b]);
          }
        }
      }
      __syncthreads();
    }
  }

  // This split's fp32 partial sums part[z][m][n..n+3] for the lane's 4
  // consecutive rows n of each subtile, or Y: the bf16 tile goes through LDS
  // (rows of ROWS + 8 values), so that a wave stores whole token rows of it
  // instead of 32-byte pieces of 16 rows.
  if (a.part) {
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      const int64_t n = p0 + 16 * (FR * wave + f) + 4 * g;
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int64_t m = q0 + 16 * b + li;
        if (m < mend && n < N)
          *reinterpret_cast<f32x4*>(a.part + ((int64_t)z * a.M + m) * N + n) = acc[f][b];
      }
    }
    return;
  }
  uint16_t* const ys = reinterpret_cast<uint16_t*>(dyn);
  if (a.r == 0) __syncthreads();   // (the LoRA step ends with a barrier)
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      const f32x4 v = acc[f][b];
      *reinterpret_cast<u32x2*>(ys + (16 * b + li) * Tile::YROW + 16 * (FR * wave + f) + 4 * g) =
          u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
    }
  __syncthreads();
  constexpr int YP = Tile::ROWS / 8;   // 16-byte pieces of a token row
#pragma unroll
  for (int i = 0; i < (Tile::TQ * YP + ET - 1) / ET; ++i) {
    const int idx = tid + ET * i, row = idx / YP, pc = idx % YP;
    const int64_t m = q0 + row, n = p0 + 8 * pc;
    if (row < Tile::TQ && m < mend && n < N)
      *reinterpret_cast<u32x4*>(a.Y + m * N + n) =
          *reinterpret_cast<const u32x4*>(ys + row * Tile::YROW + 8 * pc);
  }
}

}  // namespace

// (Up to 32 tokens two workgroups fit a CU: 80 KB of LDS, 128 registers.)
template <int FR, int TB, bool NODQ>
__global__ __launch_bounds__(ET, TB <= 2 ? 4 : 2) void k_expert_fwd(ExpertArgs a, Nf4Tables tb) {
  // Dynamic LDS only: the level table sits at address 0.
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  constexpr int TQ = 16 * TB;
  GroupTiles<TQ> groups(a.offsets, a.E, a.M);
  build_rep_pair_table<ET>(reinterpret_cast<char*>(dyn), load_levels(tb), threadIdx.x);
  int pt, z;
  const GroupTile gt = expert_deal(a, groups, pt, z);
  if (gt.e < 0) return;
  const int64_t rows = gt.end - gt.row0;
  constexpr int T1 = narrow1(TB), T2 = narrow2(TB);
  if constexpr (T1 > 0) {
    if (rows <= 16 * T1) {
      expert_tile<FR, T1, NODQ>(a, dyn, gt.e, gt.row0, gt.end, pt, z);
      return;
    }
  }
  if constexpr (T2 > 0) {
    if (rows <= 16 * T2) {
      expert_tile<FR, T2, NODQ>(a, dyn, gt.e, gt.row0, gt.end, pt, z);
      return;
    }
  }
  expert_tile<FR, TB, NODQ>(a, dyn, gt.e, gt.row0, gt.end, pt, z);
}

namespace {

template <int FR, int TB, bool NODQ>
hipError_t launch_variant(const ExpertArgs& a, const Nf4Tables& tb, hipStream_t stream) {
  constexpr int kLds = expert_lds<FR, TB>();
  static LdsLimit lds;
  const hipError_t attr =
      lds.raise(reinterpret_cast<const void*>(&k_expert_fwd<FR, TB, NODQ>), kLds);
  if (attr != hipSuccess) return attr;
  const dim3 grid(
      static_cast<unsigned>(xcd_deal_grid((int64_t)a.qtiles * a.splits, a.ptiles)));
  hipLaunchKernelGGL((k_expert_fwd<FR, TB, NODQ>), grid, dim3(ET), kLds, stream, a, tb);
  return hipGetLastError();
}

struct ExpertPlan {
  int fr, tb, ptiles, qtiles;   // tb = 0: the few-token kernel, which plans itself
  GemmSplit sp;
};

// Rows up to which the few-token kernel is used.  It streams the weights of few
// experts faster than k_expert_fwd: 8 experts of 4096 x 4096, r = 16, 4 rows on three
// of them 20 against 25 us, 16 rows on one 19 against 26, on three or four 22.6
// against 26.  With rows on all eight it is the slower one (31 against 30 us at 8
// rows, 32 against 30 at 16), but the host does not know how many have any.  At 32
// rows an expert can have more than one MFMA column tile, and it takes 36 against 31.
constexpr int64_t kFewRows = 16;
// Rows of an average expert above which a tile holds 64 tokens, and 192 (the
// narrower bodies take over in the last tile of a group).  Same experts, 32 /
// 64 / 192 tokens a tile: 35 / 37 / 39 us at 192 rows, 51 / 38 / 40 at 256, 51 /
// 40 / 40 at 320, 71 / 65 / 50 at 512; 32 experts of 1024 x 2048: 27 / 28 / 30 us
// at 768 rows, 35 / 29 / 30 at 1024, 45 / 44 / 36 at 1536.
constexpr int64_t kMidMean = 24, kWideMean = 40;

// Token subtiles by the rows of an average expert, 256 weight rows a workgroup
// if that leaves no CU idle (128 otherwise), and a split of K when there are
// fewer workgroups than the CUs hold, of at least four chunks each.
ExpertPlan plan_expert_fwd(int64_t M, int E, int64_t N, int64_t K) {
  ExpertPlan p;
  if (M <= kFewRows) return ExpertPlan{0, 0, 0, 0, GemmSplit{1, 0}};
  const int64_t mean = (M + E - 1) / E;
  p.tb = mean > kWideMean ? 12 : (mean > kMidMean ? 4 : 2);
  const int64_t room = p.tb == 2 ? 512 : 256;
  p.qtiles = static_cast<int>(group_tile_bound(M, E, 16 * p.tb));
  p.fr = 2;
  p.ptiles = static_cast<int>((N + 255) / 256);
  if (static_cast<int64_t>(p.ptiles) * p.qtiles < room) {
    p.fr = 1;
    p.ptiles = static_cast<int>((N + 127) / 128);
  }
  const int64_t tiles = static_cast<int64_t>(p.ptiles) * p.qtiles, chunks = (K + 127) / 128;
  const int64_t want = std::max<int64_t>(1, std::min(room / tiles, chunks / 4));
  p.sp.cps = static_cast<int>((chunks + want - 1) / want);
  p.sp.splits = static_cast<int>((chunks + p.sp.cps - 1) / p.sp.cps);
  return p;
}

}  // namespace

GemmSplit grouped_fwd_split(int64_t M, int E, int64_t N, int64_t K) {
  return plan_expert_fwd(M, E, N, K).sp;
}

int64_t grouped_fwd_threads(int64_t M, int E, int64_t N, int64_t K) {
  const ExpertPlan p = plan_expert_fwd(M, E, N, K);
  return p.tb == 0 ? expert_few_threads(M, E, N)
                   : ET * xcd_deal_grid((int64_t)p.qtiles * p.sp.splits, p.ptiles);
}

// The few-token kernel adds up T's partial sums itself: every workgroup reads
// those of its few rows.  With up to 32 tokens a tile that was 128 KB a
// workgroup, and a launch of its own cost less (96 rows, 8 experts of 11008 x
// 4096, r = 64: 80 against 85 us).
bool grouped_fwd_folds_t(int64_t M) { return M <= kFewRows; }

hipError_t launch_grouped_fwd_gemm(const uint16_t* X, int64_t M, const int* offsets, int E,
                                   const Nf4View& w, const float* T, int nz, float tscale,
                                   float* Tout, const uint16_t* B, int r, float s, uint16_t* Y,
                                   float* part, const Nf4Tables& tb, hipStream_t stream) {
  const int64_t N = w.N / E;
  const ExpertPlan p = plan_expert_fwd(M, E, N, w.K);
  if (p.sp.splits > 1 && !part) return hipErrorInvalidValue;
  const ExpertArgs a{X, M, offsets, E, w.codes, w.absmax_q, w.absmax_scale, N, w.K, T, Tout, B, Y,
                     p.sp.splits > 1 ? part : nullptr, nz, r, p.ptiles, p.qtiles, p.sp.splits,
                     p.sp.cps, tscale, s, nullptr, 0};
  auto pick = [&](auto nodq) {
    constexpr bool ND = decltype(nodq)::value;
    if (p.fr == 2)
      return p.tb == 12 ? launch_variant<2, 12, ND> : (p.tb == 4 ? launch_variant<2, 4, ND>
                                                                 : launch_variant<2, 2, ND>);
    return p.tb == 12 ? launch_variant<1, 12, ND> : (p.tb == 4 ? launch_variant<1, 4, ND>
                                                               : launch_variant<1, 2, ND>);
  };
  auto launch = w.dq ? pick(std::false_type{}) : pick(std::true_type{});
  prof_begin(0, stream);
  hipError_t e = p.tb == 0 ? launch_expert_few(a, w.dq, tb, stream)
                           : launch(a, tb, stream);
  if (e == hipSuccess && p.sp.splits > 1)
    e = launch_group_reduce(part, p.sp.splits, M, N, 1.f, offsets, E, nullptr, Y, stream);
  prof_end(0, stream);
  return e;
}

}  // namespace qnf4
