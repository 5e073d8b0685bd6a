// Backward dX = dY . deq(W) + s . G . A^T on bf16 MFMA (list item (4) of
// "DL0087 QLoRA: 4-bit Quantized LoRA": gradients pass through the frozen
// 4-bit weights; the backward pass dequantizes again), with the dequantized
// weight tile staged in LDS.
//
// Here the reduction runs over the weight's rows n while its 64-blocks run
// along k, so the weight enters the MFMA "transposed".  Workgroup = 8 waves,
// tile = 128 output columns (k) x 256 tokens (m), reduction in chunks of 64
// rows n.  Every chunk the 512 threads dequantize the tile's 64 x 128
// weights once -- thread t takes 16 codes of row t/8 -- into one of two LDS
// buffers in their natural row-major order, and the waves read their A
// fragments (16 columns k x 32 rows n) with ds_read_b64_tr_b16, which
// transposes 4 x 16 blocks of 16-bit elements across each group of 16 lanes.
// dY is staged through LDS by coalesced loads.  Wave w owns tokens
// 64 (w % 4) .. +63, all 128 columns, and the 32-row half (w / 4) of every
// chunk; the two halves' accumulators are added through LDS at the end.
//
// LDS layouts: a weight row n holds its 128 k as sixteen 16-byte pieces,
// piece p at slot p ^ ((n % 2) ^ 2 (n % 4) ^ 8 ((n / 8) % 2)): the rows a
// transposing read touches use distinct 32-byte slot pairs, and the two rows
// of a 16-lane dequantizing store use opposite slot parities.  A dY token row
// holds its 64 n as eight pieces, piece q at slot q ^ ((m / 2) % 8).
//
// The LoRA term s . G . A^T is appended as extra reduction steps over the
// rank: A^T fragments come straight from A [K, r], s.G enters as bf16 hi and
// lo halves.
//
// kFormDense instantiates the same kernel over a bf16 weight [N, K] (the 16-bit
// LoRA baseline): each thread loads its 16 weights of row t/8 (32 bytes) and
// stores them where the dequantized values would go.  kFormNoDq reads one
// fp32 constant per block (codes without double quantization).
//
// kExperts instantiates it over token rows grouped by expert (as expert_fwd.hip is):
// the reduction runs over the rows of the tile's expert.  With kQ = 64
// a tile is 64 tokens and the four wave columns split the 128 output columns;
// kQ = 128 lies between.  It serves the calls of few tiles, whose reduction it can
// split; with enough tiles to fill the machine expert_dx.hip is faster.
//
// kDrop is the backward of the layer whose adapter input was dropped out:
// dX = dY . deq(W) + s . mask . (G . A^T), s holding the mask's scale.  The
// adapter's term then needs sums of its own, masked before they are added:
// each wave forms them after the exchange, for the subtiles it stores, over
// all ranks.  The mask is regenerated there.  A piece of the generator covers
// eight columns of a token, two lanes' outputs, so the lane pair computes one
// piece each for two subtiles and hands over the half the other needs: 32
// outputs a lane take 8 generator calls instead of 16.
#include <type_traits>

#include "device_common.hpp"
#include "dropout.hpp"
#include "expert_args.hpp"
#include "group_tiles.hpp"
#include "kernels.hpp"

namespace qnf4 {

namespace {

constexpr int XP = 128;          // output columns k per workgroup
constexpr int XN = 64;           // weight rows n per chunk
constexpr int XWC = 4;           // wave columns: kQ / 64 token groups x column groups
constexpr int XKS = 2;           // waves splitting a chunk's two 32-n steps
constexpr int XW = XWC * XKS;    // waves
constexpr int XT = 64 * XW;      // threads
constexpr int XAS = XP;          // LDS row stride of the weight tile (256 B, swizzled)
constexpr int XYS = XN;          // LDS row stride of the dY tile (128 B, swizzled)
constexpr int XTB = 4;           // 16-token subtiles per wave
constexpr int kXA = XN * XAS;    // elements of one weight tile buffer

// A tile of kQ tokens (256, 128 or 64).
template <int kQ>
struct DxTile {
  static constexpr int WT = kQ / 64;              // token groups
  static constexpr int WR = XWC / WT;             // column groups
  static constexpr int TA = XP / 16 / WR;         // 16-column subtiles per wave (8 or 2)
  static constexpr int YTILE = kQ * XYS;          // elements of one dY tile buffer
  static constexpr int YPT = kQ * XN / 8 / XT;    // 16-byte dY pieces a thread stages per chunk
  static constexpr int LDS = kRepTabBytes + 2 * kXA * 2 + 2 * YTILE * 2;
};

__device__ __forceinline__ int xcd_remap_dx(int b, int total) {
  const int n8 = total >> 3, rem = total & 7;
  const int x = b & 7, i = b >> 3;
  return x * n8 + min(x, rem) + i;
}

// Slot of 16-byte piece p of weight-tile row n.
__device__ __forceinline__ int wslot(int n, int p) {
  return p ^ ((n & 1) ^ (2 * (n & 3)) ^ (8 * ((n >> 3) & 1)));
}

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 LdsV4i16;

}  // namespace

struct DxArgs {
  const uint16_t* dY;
  int64_t M;
  const uint16_t* Wd;
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* absmax_scale;
  int64_t N, K;
  const float* G;
  const uint16_t* Al;
  int r;
  float s;
  uint16_t* dX;
  int ptiles, qtiles, splits, cps;
  float* part;
  const int* offsets;
  int E;
  const uint64_t* state;
  uint32_t thr;
};

// One tile: tokens q0 .. mend - 1 (kQ at most), columns 128 pt .., split z of
// the reduction over the weight rows n0 .. n0 + N - 1 of expert e.
template <int kForm, int kQ, bool kExperts, bool kDrop>
__device__ __forceinline__ void dx_tile(const DxArgs& args, uint8_t* dyn, int e, int64_t q0,
                                        int64_t mend, int pt, int z) {
  using Tile = DxTile<kQ>;
  constexpr int XQ = kQ, XTA = Tile::TA, kXY = Tile::YTILE, XYPT = Tile::YPT;
  const uint16_t* const __restrict__ dY = args.dY;
  const int64_t M = args.M, N = args.N, K = args.K;
  const float* const __restrict__ G = args.G;
  const int r = args.r, cps = args.cps;
  const float s = args.s;
  uint16_t* const __restrict__ dX = args.dX;
  float* const __restrict__ part = args.part;
  const uint16_t* const __restrict__ Al = args.Al + (kExperts ? (int64_t)e * K * r : 0);
  uint16_t* Ws = reinterpret_cast<uint16_t*>(dyn + kRepTabBytes);   // [2][XN][XAS]
  uint16_t* Ys = Ws + 2 * kXA;                                       // [2][XQ][XYS]

  const int tid = threadIdx.x;
  const int wave = wave_id(), lane = tid & 63;
  const int li = lane & 15, g = lane >> 4;
  const int wc = wave % XWC, ks = wave / XWC;
  const int wt = wc % Tile::WT, wr = wc / Tile::WT;
  const int64_t k0 = (int64_t)pt * XP;
  const int64_t n0 = kExperts ? (int64_t)e * N : 0;
  const int64_t NW = kExperts ? N * args.E : N;     // rows of W
  const int c0 = z * cps;
  // end of this split's row chunks
  const int nchunks = min(static_cast<int>((N + XN - 1) / XN), c0 + cps);
  const int KB = static_cast<int>(K / kBlock);

  // Buffer descriptors: rows past W and tokens past the tile read as zero.  A row
  // n >= N of an expert is the next one's: its dY columns read as zero, and the
  // constants' buffers end with the expert's (whole groups of them), as zero times
  // one that is not finite, or whose weight is not in bf16, would be NaN.
  const uint32_t nb = static_cast<uint32_t>((n0 + N) * KB);
  const BufRes rc = make_bufres(args.codes, static_cast<uint32_t>(NW * K / 2));
  const BufRes re = make_bufres(args.absmax_q, nb);
  // second-level scales, or one fp32 constant per block (kFormNoDq)
  const BufRes rd = make_bufres(
      args.absmax_scale, (kForm == kFormNoDq ? nb : (nb + kGroup - 1) / kGroup) * 4u);
  // the bf16 weight (kFormDense; N K 2 < 2^31 bytes)
  const BufRes rw = make_bufres(args.Wd, static_cast<uint32_t>(kForm == kFormDense ? N * K * 2 : 0));
  // dY is addressed from the tile's first token (its 256 rows span less
  // than 2^31 bytes for N <= 2^22).  (A plain conditional, not min(): the
  // 64-bit min is opaque to the compiler's uniformity analysis and would put
  // the descriptor in vector registers.)
  const int64_t tile_rows = mend - q0 < XQ ? mend - q0 : XQ;
  const BufRes ry = make_bufres(dY + q0 * N, static_cast<uint32_t>(tile_rows * N * 2));

  // Dequantization role: row dr of the chunk, columns k0 + 16 dp .. +15.
  // Columns past K (a half tile when K % 128 == 64) get a zero constant.
  const int dr = tid >> 3, dp = tid & 7;
  const bool dkok = k0 + 16 * dp < K;
  const uint32_t dcode = static_cast<uint32_t>((n0 + dr) * (K / 2) + k0 / 2 + 8 * dp);   // + c 64 K/2
  const uint32_t dblk = static_cast<uint32_t>((n0 + dr) * KB + (k0 + 16 * dp) / kBlock);   // + c 64 KB
  // kFormDense: the same 16 weights as bf16, byte offset (+ c 64 K 2)
  const uint32_t dw = static_cast<uint32_t>((dr * K + k0 + 16 * dp) * 2);
  u32x2 cw[2];
  uint32_t ce[2];
  float cd[2];
  u32x4 ww[2][2];
  auto load_codes = [&](int c, int st) {
    const bool live = c < nchunks && dkok;
    if constexpr (kForm == kFormDense) {
      const uint32_t o = dw + static_cast<uint32_t>(c * XN) * static_cast<uint32_t>(K * 2);
      ww[st][0] = buf_load16(rw, live ? o : 0x80000000u);
      ww[st][1] = buf_load16(rw, live ? o + 16u : 0x80000000u);
    } else {
      const uint32_t blk = dblk + static_cast<uint32_t>(c * XN * KB);
      cw[st] = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                     rc, live ? dcode + static_cast<uint32_t>(c * XN) * static_cast<uint32_t>(K / 2)
                              : 0x80000000u, 0, 0));
      if constexpr (kForm == kFormNoDq) {   // e = 1, d = the block's absmax
        ce[st] = 1u;
        cd[st] = buf_load_f32(rd, live ? blk * 4u : 0x80000000u);
      } else {
        ce[st] = buf_load_u8(re, live ? blk : 0x80000000u);
        cd[st] = buf_load_f32(rd, live ? (blk / kGroup) * 4u : 0x80000000u);
      }
    }
  };
  uint32_t ta[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) ta[b] = rep_lane_base(lane);
  auto dequant = [&](int st, int buf) {
    uint16_t* dst = Ws + buf * kXA + dr * XAS;
    if constexpr (kForm == kFormDense) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<u32x4*>(dst + 8 * wslot(dr, 2 * dp + i)) = ww[st][i];
      return;
    }
    const float chat = static_cast<float>(ce[st]) * cd[st];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = cw[st][i];
      const f32x2 v0 = rep_lookup<0>(ta[0], w);
      const f32x2 v1 = rep_lookup<1>(ta[1], w);
      const f32x2 v2 = rep_lookup<2>(ta[2], w);
      const f32x2 v3 = rep_lookup<3>(ta[3], w);
      *reinterpret_cast<u32x4*>(dst + 8 * wslot(dr, 2 * dp + i)) =
          u32x4{pack_bf16x2(v0.x * chat, v0.y * chat), pack_bf16x2(v1.x * chat, v1.y * chat),
                pack_bf16x2(v2.x * chat, v2.y * chat), pack_bf16x2(v3.x * chat, v3.y * chat)};
    }
  };

  // dY staging role: piece j of thread tid is token row yr + 64 j (yr = tid / 8)
  // of the tile, 16-byte piece tid % 8 of its 128-byte chunk row.
  const int yr = tid >> 3, yq = tid & 7;
  const uint32_t ysrc = static_cast<uint32_t>((yr * N + 8 * yq) * 2);   // + 128 c
  u32x4 yw[2][XYPT];
  auto load_y = [&](int c, int st) {
    const bool live = c < nchunks && c * XN + 8 * yq < N;
#pragma unroll
    for (int j = 0; j < XYPT; ++j)
      yw[st][j] = buf_load16(
          ry, live ? ysrc + static_cast<uint32_t>((64 * j * N + c * XN) * 2) : 0x80000000u);
  };
  auto store_y = [&](int st, int buf) {
#pragma unroll
    for (int j = 0; j < XYPT; ++j) {
      const int row = yr + 64 * j;
      *reinterpret_cast<u32x4*>(Ys + buf * kXY + row * XYS + 8 * (yq ^ ((row >> 1) & 7))) =
          yw[st][j];
    }
  };

  f32x4 acc[XTA][XTB];
#pragma unroll
  for (int a = 0; a < XTA; ++a)
#pragma unroll
    for (int b = 0; b < XTB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A fragment (columns 16 a + li, rows 32 ks + 8 g .. +7): two transposing
  // reads of rows nb4 + t/4, columns 16 a + 4 (t % 4) (t = li).
  // Operands of one 32-n step are read into registers first; the MFMAs then
  // touch no memory, so the compiler can interleave them with the staging
  // work of the next chunk.
  u32x4 af[XTA], bf[XTB];
  // Transposing-read address of rows 32 ks + 8 g + 4 e + li / 4, columns
  // 16 a + 4 (li % 4): rbase[e] + 16 (a ^ rsw[e]) + ... in elements, where
  // rsw[e] is the row's XOR on the 16-column group.
  int rbase[2], rsw[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int n = 32 * ks + 8 * g + 4 * e + (li >> 2);
    const int x = (n & 1) ^ (2 * (n & 3)) ^ (8 * ((n >> 3) & 1));   // slot XOR
    rbase[e] = n * XAS + 8 * (((li & 3) >> 1) ^ (x & 1)) + 4 * (li & 1);
    rsw[e] = x >> 1;
  }
  auto read_frags = [&](int buf) {
    const uint16_t* yt = Ys + buf * kXY + (64 * wt + li) * XYS + 8 * ((g + 4 * ks) ^ (li >> 1));
#pragma unroll
    for (int b = 0; b < XTB; ++b) bf[b] = *reinterpret_cast<const u32x4*>(yt + 16 * b * XYS);
    const uint16_t* wt0 = Ws + buf * kXA;
    // Recomputing the 16 addresses each chunk (one VALU op each) is cheaper
    // than holding them in registers across the loop.
    int sw[2] = {rsw[0], rsw[1]};
    asm volatile("" : "+v"(sw[0]), "+v"(sw[1]));
#pragma unroll
    for (int a = 0; a < XTA; ++a) {
      v4i16 h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint16_t* src = wt0 + rbase[e] + 16 * ((wr * XTA + a) ^ sw[e]);
        h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4i16*)(src));
      }
      const u32x2 h0 = __builtin_bit_cast(u32x2, h[0]), h1 = __builtin_bit_cast(u32x2, h[1]);
      af[a] = u32x4{h0[0], h0[1], h1[0], h1[1]};
    }
  };
  auto mma = [&]() {
#pragma unroll
    for (int a = 0; a < XTA; ++a)
#pragma unroll
      for (int b = 0; b < XTB; ++b) acc[a][b] = mfma16(af[a], bf[b], acc[a][b]);
  };

  load_codes(c0, 0);
  load_codes(c0 + 1, 1);
  load_y(c0, 0);
  load_y(c0 + 1, 1);
  __syncthreads();   // level table
  dequant(0, 0);
  store_y(0, 0);
  load_codes(c0 + 2, 0);
  load_y(c0 + 2, 0);
  __syncthreads();
  // iteration c: read the operands of chunk c from buffers c&1; stage chunk
  // c+1 into buffers (c+1)&1 -- dequantize its codes and store its dY, both
  // loaded two iterations ago -- and refill those register stages with chunk
  // c+3; multiply chunk c.
  auto iter = [&](int c, auto stc) {
    constexpr int ST = decltype(stc)::value;
    read_frags(ST);
    dequant(ST ^ 1, ST ^ 1);
    store_y(ST ^ 1, ST ^ 1);
    load_codes(c + 3, ST ^ 1);
    load_y(c + 3, ST ^ 1);
    mma();
    __syncthreads();
  };
  // Iterations run in pairs with no exit between them, so the compiler's
  // load counting sees one path and waits only for the stage it consumes.
  // An odd chunk count adds one pass over a chunk past the end, whose codes,
  // constants and activations all read as zero: it adds zeros.
  for (int c = c0; c < nchunks; c += 2) {
    iter(c, std::integral_constant<int, 0>{});
    iter(c + 1, std::integral_constant<int, 1>{});
  }

  // LoRA term of column subtiles A0 .. A0 + TN - 1 (the first split only):
  // extra steps over the rank, ranks j0, j0 + step, ... 32 at a time.
  auto lora = [&](auto a0c, auto tnc, f32x4 (*dst)[XTB], int j0, int step) {
    constexpr int A0 = decltype(a0c)::value, TN = decltype(tnc)::value;
    for (; z == 0 && j0 < r; j0 += step) {
      const int j = j0 + 8 * g;
      u32x4 gh[XTB], gl[XTB];
#pragma unroll
      for (int b = 0; b < XTB; ++b) {
        const int64_t m = q0 + 64 * wt + 16 * b + li;
        uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
        if (m < mend && j < r) {
          const f32x4 t0 = *reinterpret_cast<const f32x4*>(G + m * r + j);
          const f32x4 t1 = *reinterpret_cast<const f32x4*>(G + m * r + j + 4);
          const float v[8] = {t0.x * s, t0.y * s, t0.z * s, t0.w * s,
                              t1.x * s, t1.y * s, t1.z * s, t1.w * s};
#pragma unroll
          for (int e = 0; e < 4; ++e) split_bf16x2(v[2 * e], v[2 * e + 1], hi[e], lo[e]);
        }
        gh[b] = u32x4{hi[0], hi[1], hi[2], hi[3]};
        gl[b] = u32x4{lo[0], lo[1], lo[2], lo[3]};
      }
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        const int64_t k = k0 + 16 * (wr * XTA + A0 + a) + li;
        const u32x4 af = (k < K && j < r) ? *reinterpret_cast<const u32x4*>(Al + k * r + j)
                                          : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < XTB; ++b) {
          dst[a][b] = mfma16(af, gh[b], dst[a][b]);
          dst[a][b] = mfma16(af, gl[b], dst[a][b]);
        }
      }
    }
  };
  // Without dropout the two halves take the rank steps in turn, before their
  // accumulators are added.
  if constexpr (!kDrop)
    lora(std::integral_constant<int, 0>{}, std::integral_constant<int, XTA>{}, acc, 32 * ks, 64);

  // Add the two n halves: wave ks keeps half of its column subtiles and
  // receives them from its partner (the other ks, same wave column) through
  // LDS, in one round; each half then stores its own column subtiles.
  constexpr int TH = XTA / 2;
  f32x4* xch = reinterpret_cast<f32x4*>(dyn);   // [2][XWC][TH][XTB][64]
  auto hand = [&](auto kc) {
    constexpr int GIVE = 1 - decltype(kc)::value;
#pragma unroll
    for (int a = 0; a < TH; ++a)
#pragma unroll
      for (int b = 0; b < XTB; ++b)
        xch[(((GIVE * XWC + wc) * TH + a) * XTB + b) * 64 + lane] = acc[GIVE * TH + a][b];
  };
  // This split's fp32 partial sums part[z][m][k..k+3] for the lane's 4
  // consecutive columns k of each subtile, or dX: the bf16 tile goes through
  // LDS (rows of 128 + 8 values), so that a wave stores 256 bytes of a token row
  // at a time instead of 32.
  constexpr int kXRow = XP + 8;
  uint16_t* const xs = reinterpret_cast<uint16_t*>(dyn);
  auto finish = [&](auto kc) {
    constexpr int K0 = decltype(kc)::value;
#pragma unroll
    for (int a = 0; a < TH; ++a)
#pragma unroll
      for (int b = 0; b < XTB; ++b)
        acc[K0 * TH + a][b] += xch[(((K0 * XWC + wc) * TH + a) * XTB + b) * 64 + lane];
    if constexpr (kDrop) {
      if (z == 0 && r > 0) {
        f32x4 low[TH][XTB];
#pragma unroll
        for (int a = 0; a < TH; ++a)
#pragma unroll
          for (int b = 0; b < XTB; ++b) low[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        lora(std::integral_constant<int, K0 * TH>{}, std::integral_constant<int, TH>{}, low, 0,
             32);
        const uint32_t thr = args.thr;
        const DropKey key = load_drop_key(args.state, thr);
#pragma unroll
        for (int b = 0; b < XTB; ++b) {
          const int64_t m = q0 + 64 * wt + 16 * b + li;
          // first of the two pieces of a subtile's 16 columns
          const uint64_t p0 =
              static_cast<uint64_t>(m * K + k0 + 16 * (wr * XTA + K0 * TH)) / 8 + (g >> 1);
          auto add = [&](int a, uint32_t w0, uint32_t w1) {
            f32x4 v = low[a][b];
            v.x = (w0 & 0xFFFFu) >= thr ? v.x : 0.f;
            v.y = (w0 >> 16) >= thr ? v.y : 0.f;
            v.z = (w1 & 0xFFFFu) >= thr ? v.z : 0.f;
            v.w = (w1 >> 16) >= thr ? v.w : 0.f;
            acc[K0 * TH + a][b] += v;
          };
          if constexpr (TH == 1) {
            const u32x4 w = philox_piece(key, p0);
            add(0, (g & 1) ? w.z : w.x, (g & 1) ? w.w : w.y);
          } else {
#pragma unroll
            for (int a = 0; a < TH; a += 2) {
              // lanes of even g (columns 0-3 of a piece) compute the piece of
              // subtile a, lanes of odd g (columns 4-7) that of subtile a + 1
              const bool odd = g & 1;
              const u32x4 w = philox_piece(key, p0 + 2 * (a + (odd ? 1 : 0)));
              const uint32_t g0 = __shfl_xor(odd ? w.x : w.z, 16);
              const uint32_t g1 = __shfl_xor(odd ? w.y : w.w, 16);
              add(a, odd ? g0 : w.x, odd ? g1 : w.y);
              add(a + 1, odd ? w.z : g0, odd ? w.w : g1);
            }
          }
        }
      }
    }
    const int col = 16 * (wr * XTA + K0 * TH) + 4 * g;   // of subtile a: + 16 a
    if (part) {
#pragma unroll
      for (int a = 0; a < TH; ++a)
#pragma unroll
        for (int b = 0; b < XTB; ++b) {
          const int64_t m = q0 + 64 * wt + 16 * b + li;
          if (m < mend && k0 + col + 16 * a < K)
            *reinterpret_cast<f32x4*>(part + ((int64_t)z * M + m) * K + k0 + col + 16 * a) =
                acc[K0 * TH + a][b];
        }
      return;
    }
    __syncthreads();   // every wave has taken its sums
#pragma unroll
    for (int a = 0; a < TH; ++a)
#pragma unroll
      for (int b = 0; b < XTB; ++b) {
        const f32x4 v = acc[K0 * TH + a][b];
        *reinterpret_cast<u32x2*>(xs + (64 * wt + 16 * b + li) * kXRow + col + 16 * a) =
            u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < XQ * (XP / 8) / XT; ++i) {
      const int idx = tid + XT * i, row = idx / (XP / 8), pc = idx % (XP / 8);
      const int64_t m = q0 + row, k = k0 + 8 * pc;
      if (m < mend && k < K)
        *reinterpret_cast<u32x4*>(dX + m * K + k) =
            *reinterpret_cast<const u32x4*>(xs + row * kXRow + 8 * pc);
    }
  };
  if (ks == 0) hand(std::integral_constant<int, 0>{}); else hand(std::integral_constant<int, 1>{});
  __syncthreads();
  if (ks == 0) finish(std::integral_constant<int, 0>{}); else finish(std::integral_constant<int, 1>{});
}

// The largest body's LDS: that of kQ (the narrower bodies hold less).
template <int kForm, int kQ, bool kExperts, bool kDrop>
__global__ __launch_bounds__(XT) void k_dx_gemm(DxArgs args, Nf4Tables tb) {
  // Dynamic LDS only (the level table sits at address 0): the replicated
  // table, two weight tiles, two dY tiles; the table's bytes hold the
  // accumulator exchange after the main loop.
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  // (grouped rows: the offsets are on their way while the table is built)
  GroupTiles<kQ> groups(args.offsets, kExperts ? args.E : 0, args.M);
  if constexpr (kForm != kFormDense)
    build_rep_pair_table<XT>(reinterpret_cast<char*>(dyn), load_levels(tb), threadIdx.x);

  // With a split reduction (few tiles), a workgroup takes row chunks
  // [z cps, (z + 1) cps) of its tile and writes fp32 partial sums.
  if constexpr (kExperts) {   // only the tiles that the groups have
    const int slots = min(args.qtiles, groups.count());
    const XcdTile t = xcd_deal(blockIdx.x, args.ptiles);
    if (t.v >= slots * args.splits) return;
    const int z = t.v / slots, pt = t.pt;
    const GroupTile gt = groups.find(t.v - z * slots);
    if (gt.e < 0) return;
    // the last tile of a group runs the narrowest body that holds its rows
    // (a launch of 64-token tiles is no faster at any number of rows: a backward of 8
    // experts of 4096 x 4096, r = 64, takes 58 / 59 us at 16 and 128 rows, 112 / 74
    // at 512 uneven ones)
    const int rows = gt.end - gt.row0;
    if (rows <= 64)
      dx_tile<kForm, 64, true, kDrop>(args, dyn, gt.e, gt.row0, gt.end, pt, z);
    else if (rows <= 128)
      dx_tile<kForm, 128, true, kDrop>(args, dyn, gt.e, gt.row0, gt.end, pt, z);
    else
      dx_tile<kForm, kQ, true, kDrop>(args, dyn, gt.e, gt.row0, gt.end, pt, z);
  } else {
    const int ntiles = args.ptiles * args.qtiles;
    const int lin = xcd_remap_dx(blockIdx.x, static_cast<int>(gridDim.x));
    const int z = lin / ntiles, tile = lin - z * ntiles;
    const int qt = tile / args.ptiles, pt = tile - qt * args.ptiles;
    dx_tile<kForm, kQ, false, kDrop>(args, dyn, 0, (int64_t)qt * kQ, args.M, pt, z);
  }
}

namespace {

constexpr int kTileQ = 256;   // tokens a tile

template <int kForm, int kQ, bool kExperts, bool kDrop>
hipError_t launch_dx_tiles(const uint16_t* dY, int64_t M, const Nf4View& w, int64_t N,
                           const float* G, const uint16_t* A, int r, float s, uint16_t* dX,
                           float* part, const Nf4Tables& tb, hipStream_t stream, int qtiles,
                           const GemmSplit& sp, const int* offsets, int E, const Drop& d) {
  constexpr int kLds = DxTile<kQ>::LDS;
  static LdsLimit lds;
  const hipError_t attr = lds.raise(
      reinterpret_cast<const void*>(&k_dx_gemm<kForm, kQ, kExperts, kDrop>), kLds);
  if (attr != hipSuccess) return attr;
  if (sp.splits > 1 && !part) return hipErrorInvalidValue;
  const int ptiles = static_cast<int>((w.K + XP - 1) / XP);
  const DxArgs args{dY,  M, w.dense, w.codes, w.absmax_q, w.absmax_scale, N, w.K,
                    G,   A, r,       kDrop ? s * d.scale() : s, dX, ptiles, qtiles, sp.splits, sp.cps,
                    sp.splits > 1 ? part : nullptr, offsets, E, d.state, d.thr};
  const dim3 grid(kExperts ? static_cast<unsigned>(
                                 xcd_deal_grid((int64_t)qtiles * sp.splits, ptiles))
                           : ptiles * qtiles * sp.splits);
  hipLaunchKernelGGL((k_dx_gemm<kForm, kQ, kExperts, kDrop>), grid, dim3(XT), kLds, stream, args,
                     tb);
  return hipGetLastError();
}

}  // namespace

GemmSplit dx_gemm_split(int64_t M, int64_t N, int64_t K) {
  return gemm_split((K + XP - 1) / XP * ((M + kTileQ - 1) / kTileQ), (N + XN - 1) / XN);
}

hipError_t launch_dx_gemm(const uint16_t* dY, int64_t M, const Nf4View& w,
                          const float* G, const uint16_t* A, int r, float s,
                          uint16_t* dX, float* part, const Nf4Tables& tb, hipStream_t stream,
                          const Drop& d) {
  const int qtiles = static_cast<int>((M + kTileQ - 1) / kTileQ);
  const GemmSplit sp = dx_gemm_split(M, w.N, w.K);
  if (w.dense && d.on()) return hipErrorInvalidValue;
  auto launch = w.dense ? launch_dx_tiles<kFormDense, kTileQ, false, false>
                : d.on() ? (w.dq ? launch_dx_tiles<kFormDq, kTileQ, false, true>
                                 : launch_dx_tiles<kFormNoDq, kTileQ, false, true>)
                         : (w.dq ? launch_dx_tiles<kFormDq, kTileQ, false, false>
                                 : launch_dx_tiles<kFormNoDq, kTileQ, false, false>);
  prof_begin(1, stream);
  hipError_t e = launch(dY, M, w, w.N, G, A, r, s, dX, part, tb, stream, qtiles, sp, nullptr, 0, d);
  if (e == hipSuccess && sp.splits > 1)
    e = launch_split_reduce_bf16(part, sp.splits, M * w.K, dX, stream);
  prof_end(1, stream);
  return e;
}

GemmSplit grouped_dx_split(int64_t M, int E, int64_t N, int64_t K) {
  return gemm_split((K + XP - 1) / XP * group_tile_bound(M, E, kTileQ),
                    (N + XN - 1) / XN);
}

int64_t grouped_dx_threads(int64_t M, int E, int64_t N, int64_t K) {
  const GemmSplit sp = grouped_dx_split(M, E, N, K);
  if (sp.splits == 1 && expert_dx_fits(M, E, K)) return expert_dx_threads(M, E, K);
  return XT * xcd_deal_grid(group_tile_bound(M, E, kTileQ) * sp.splits, (K + XP - 1) / XP);
}

hipError_t launch_grouped_dx_gemm(const uint16_t* dY, int64_t M, const int* offsets, int E,
                                  const Nf4View& w, const float* G, const uint16_t* A, int r,
                                  float s, uint16_t* dX, float* part, const Nf4Tables& tb,
                                  hipStream_t stream, const Drop& d) {
  const int64_t N = w.N / E;
  const int qtiles = static_cast<int>(group_tile_bound(M, E, kTileQ));
  const GemmSplit sp = grouped_dx_split(M, E, N, w.K);
  auto launch = d.on() ? (w.dq ? launch_dx_tiles<kFormDq, kTileQ, true, true>
                               : launch_dx_tiles<kFormNoDq, kTileQ, true, true>)
                       : (w.dq ? launch_dx_tiles<kFormDq, kTileQ, true, false>
                               : launch_dx_tiles<kFormNoDq, kTileQ, true, false>);
  prof_begin(1, stream);
  hipError_t e =
      sp.splits == 1 && expert_dx_fits(M, E, w.K)
          ? launch_expert_dx(dY, M, offsets, E, w, G, A, r, s, dX, tb, stream, d)
          : launch(dY, M, w, N, G, A, r, s, dX, part, tb, stream, qtiles, sp, offsets, E, d);
  if (e == hipSuccess && sp.splits > 1)
    e = launch_group_reduce(part, sp.splits, M, w.K, 1.f, offsets, E, nullptr, dX, stream);
  prof_end(1, stream);
  return e;
}

}  // namespace qnf4
