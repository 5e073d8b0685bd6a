// dX of the layer grouped by expert with many rows, dX = dY . deq(W_e) + s . G .
// A_e^T, the weights dequantized straight into MFMA operands as in the forward
// (expert_fwd.hip).
//
// Here the reduction runs over the weight's rows n, so an operand (16 columns k
// x 32 rows n) takes from each lane 8 codes that lie in 8 rows.  The code bytes
// are transposed, not the weights: a chunk's 64 rows x 128 code bytes are staged
// in LDS, and one transposing 8-bit read gives lane l = 16 g + i the bytes of rows
// 8 g .. + 7 at byte column i of the wave's 16.  A byte's level pair belongs to
// columns 2 i and 2 i + 1, which become row i of two operands, each pair being
// scaled by its row's block constant (staged as fp32, read in runs of 8).
//
// Workgroup = 8 waves, tile = 256 columns k x 16 TB tokens of one expert; wave w
// owns columns 32 w .. + 31 and all tokens, so every weight is dequantized once.
// dY is staged through LDS like X in the forward.  Codes and constants are stored
// two chunks ahead (four buffers), so that the next chunk's first operands can
// be formed before the barrier; dY one chunk ahead.
//
// With DROP (the adapter's input was dropped out) the adapter's term has sums of
// its own and is masked before it is added, s holding the mask's scale: a lane's
// outputs of a token are 8 consecutive columns, one piece of the generator.
//
// Measured: 8 experts of 4096 x 11008, r = 64, 8192 rows, the whole backward: 903
// us against 1030 with the kernel that passes dequantized weights through LDS
// (gemm_dx.hip), 1003 against 1107 with dropout (whose second set of sums spills
// some addresses); 854 to 892 and 966 on other cards.  Bound by the chip's power and
// by its own instructions: for as many MFMAs as the forward the kernel is busy for
// 11% more cycles, with twice the scalar and 1.17 times the LDS instructions.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "dropout.hpp"
#include "expert_args.hpp"
#include "group_tiles.hpp"
#include "kernels.hpp"
#include "rank_tiles.hpp"

namespace qnf4 {

namespace {

constexpr int VW = 8;                 // waves
constexpr int VT = 64 * VW;           // threads
constexpr int VK = 32 * VW;           // columns k of a tile
constexpr int VN = 64;                // rows n of a chunk
constexpr int VCODES = VN * VK / 2;   // code bytes of a chunk
constexpr int VCONST = VN * VK / 64;  // its block constants
constexpr int VTB = 12;               // token subtiles (4 and 8 in narrower bodies)

template <int TB>
struct VTile {
  static constexpr int TQ = 16 * TB;
  static constexpr int XBUF = TQ * VN;                 // elements of one dY buffer
  static constexpr int PP = TQ * (VN / 8) / VT;        // 16-byte pieces a thread stages
  static constexpr int MAIN = kRepTabBytes + 2 * XBUF * 2 + 4 * (VCODES + VCONST * 4);
  static constexpr int TAIL = VK * 128 + TQ * 256;     // A tile, G hi and lo tiles
  static constexpr int YROW = VK + 8;                  // a token row of the output tile
  static constexpr int OUT = TQ * YROW * 2;
  static constexpr int LDS = MAIN > TAIL ? (MAIN > OUT ? MAIN : OUT) : (TAIL > OUT ? TAIL : OUT);
  static_assert(TQ * (VN / 8) % VT == 0, "whole rounds of pieces");
};

typedef int v2i32 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i32 LdsV2i32;

// Slot of 16-byte piece q of a 128-byte row.
__device__ __forceinline__ int vslot(int row, int q) { return q ^ ((row >> 1) & 7); }

template <int TB, bool NODQ, bool DROP>
__device__ __forceinline__ void dx_expert_tile(const ExpertArgs& a, uint8_t* dyn, int e, int64_t q0,
                                               int64_t mend, int pt) {
  using Tile = VTile<TB>;
  constexpr int PP = Tile::PP, GB = 2, NG = TB / GB;   // token subtiles a group, groups
  uint16_t* const Xs = reinterpret_cast<uint16_t*>(dyn + kRepTabBytes);
  uint8_t* const Cs = reinterpret_cast<uint8_t*>(Xs + 2 * Tile::XBUF);   // [4][VN][128]
  float* const Ks = reinterpret_cast<float*>(Cs + 4 * VCODES);           // [4][4][VN]
  const int tid = threadIdx.x;
  const int wave = wave_id(), lane = tid & 63;
  const int li = lane & 15, g = lane >> 4;
  const int64_t N = a.N, K = a.K;
  const int N32 = static_cast<int>(N), K32 = static_cast<int>(K), KB = K32 / kBlock;
  const int64_t k0 = (int64_t)pt * VK, NW = N * a.E, n0 = (int64_t)e * N;
  const int nchunks = (N32 + VN - 1) / VN;

  // rows past W and tokens past the tile read as zero
  const uint32_t nb = static_cast<uint32_t>(NW * K / kBlock);
  const BufRes rc = make_bufres(a.codes, static_cast<uint32_t>(NW * K / 2));
  const BufRes re = make_bufres(a.absmax_q, nb);
  const BufRes rd = make_bufres(a.absmax_scale, (NODQ ? nb : (nb + kGroup - 1) / kGroup) * 4u);
  const int64_t tile_rows = mend - q0 < Tile::TQ ? mend - q0 : Tile::TQ;
  const BufRes rx = make_bufres(a.X + q0 * N, static_cast<uint32_t>(tile_rows * N * 2));

  // Staging: piece tid % 8 of code row tid / 8; thread tid < 256 takes the constant
  // of row tid / 4, block tid % 4; piece tid % 8 of dY's rows tid / 8 + 64 j.
  const int srow = tid >> 3, sq = tid & 7;
  const uint32_t csrc = static_cast<uint32_t>((n0 + srow) * (K / 2) + k0 / 2) + 16u * sq;
  const uint32_t cstep = static_cast<uint32_t>(VN * (K32 / 2));
  uint8_t* const cdst = Cs + 128 * srow + 16 * vslot(srow, sq);
  const int krow = tid >> 2, kb = static_cast<int>(k0 / kBlock) + (tid & 3);
  const bool kown = tid < VCONST && kb < KB;
  const uint32_t ksrc = static_cast<uint32_t>((n0 + krow) * KB + kb);
  float* const kdst = Ks + VN * (tid & 3) + (krow & (VN - 1));
  const uint32_t xsrc = static_cast<uint32_t>(srow * N32 + 8 * sq) * 2u;
  const uint32_t xstep = static_cast<uint32_t>(64 * N32) * 2u;
  uint16_t* const xdst = Xs + srow * VN + 8 * vslot(srow, sq);
  u32x4 cw[2], xw[2][PP];
  uint32_t ce[2];
  float cd[2];
  auto load_codes = [&](int c, int st) {
    const bool live = c < nchunks;
    cw[st] = buf_load16(rc, live ? csrc + cstep * static_cast<uint32_t>(c) : kOffNone);
    // (rows past the expert's: constant 0)
    const bool own = kown && VN * c + krow < N32;
    const uint32_t b = ksrc + static_cast<uint32_t>(VN * c * KB);
    if constexpr (NODQ) {
      cd[st] = buf_load_f32(rd, own ? b * 4u : kOffNone);
    } else {
      ce[st] = buf_load_u8(re, own ? b : kOffNone);
      cd[st] = buf_load_f32(rd, own ? (b / kGroup) * 4u : kOffNone);
    }
  };
  auto store_codes = [&](int c, int st) {
    *reinterpret_cast<u32x4*>(cdst + VCODES * (c & 3)) = cw[st];
    if (tid < VCONST)
      kdst[VCONST * (c & 3)] = NODQ ? cd[st] : static_cast<float>(ce[st]) * cd[st];
  };
  auto load_x = [&](int c, int st) {
    const bool ok = VN * c + 8 * sq < N32;
    const uint32_t o = ok ? xsrc + 128u * c : kOffNone;   // (+ j xstep < 2^31: stays past the end)
#pragma unroll
    for (int j = 0; j < PP; ++j) xw[st][j] = buf_load16(rx, o + j * xstep);
  };
  auto store_x = [&](int st, int buf) {
#pragma unroll
    for (int j = 0; j < PP; ++j)
      *reinterpret_cast<u32x4*>(xdst + buf * Tile::XBUF + 64 * j * VN) = xw[st][j];
  };

  f32x4 acc[2][TB];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[f][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const uint32_t ta = rep_lane_base(lane);
  // the lane's 8 code bytes (rows 32 i + 8 g .. + 7) and their constants, step i of
  // chunk c
  auto read_codes = [&](int c, int i) {
    const int row = 32 * i + 8 * g + (li >> 1);
    const uint8_t* p = Cs + VCODES * (c & 3) + 128 * row + 16 * vslot(row, wave) + 8 * (li & 1);
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((LdsV2i32*)(p)));
  };
  struct Consts {
    f32x4 v[2];
  };
  auto read_consts = [&](int c, int i) {
    const f32x4* p = reinterpret_cast<const f32x4*>(Ks + VCONST * (c & 3) + VN * (wave >> 1) +
                                                    32 * i + 8 * g);
    return Consts{{p[0], p[1]}};
  };
  struct Pairs {
    f32x2 v[8];
  };
  auto lookup = [&](u32x2 q) {
    return Pairs{{rep_lookup<0>(ta, q.x), rep_lookup<1>(ta, q.x), rep_lookup<2>(ta, q.x),
                  rep_lookup<3>(ta, q.x), rep_lookup<0>(ta, q.y), rep_lookup<1>(ta, q.y),
                  rep_lookup<2>(ta, q.y), rep_lookup<3>(ta, q.y)}};
  };
  // dword t of operand f: rows 2 t and 2 t + 1, bf16_rne(fl32(level * c))
  auto scaled = [&](const Pairs& p, const Consts& c, int f, int t) {
    const f32x2 u = p.v[2 * t], v = p.v[2 * t + 1];
    const f32x4 h = c.v[t >> 1];
    const float c0 = (t & 1) ? h.z : h.x, c1 = (t & 1) ? h.w : h.y;
    return f == 0 ? pack_bf16x2(u.x * c0, v.x * c1) : pack_bf16x2(u.y * c0, v.y * c1);
  };
  const uint16_t* const xsrow = Xs + li * VN;
  auto read_x = [&](int buf, int i, int b) {
    return *reinterpret_cast<const u32x4*>(xsrow + 8 * ((4 * i + g) ^ (li >> 1)) +
                                           buf * Tile::XBUF + 16 * b * VN);
  };

  load_codes(0, 0);
  load_x(0, 0);
  load_codes(1, 1);
  load_x(1, 1);
  store_codes(0, 0);
  load_codes(2, 0);
  store_x(0, 0);
  load_x(2, 0);
  store_codes(1, 1);
  load_codes(3, 1);
  __syncthreads();   // (the level table too)
  u32x4 af[2][2];    // operands of the current and the next step
  {
    const Pairs p = lookup(read_codes(0, 0));
    const Consts k = read_consts(0, 0);
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int t = 0; t < 4; ++t) af[0][f][t] = scaled(p, k, f, t);
  }
  u32x2 code = read_codes(0, 1);   // of the step after the next operands'
  // Chunk c (parity ST).  As in the forward, a step's products run in groups of GB
  // token subtiles, the next step's level pairs are looked up at its first group
  // and scaled between the later MFMAs; the code bytes they are looked up by were
  // read a step before.
  constexpr int SLOTS = 2 * TB, SLOT0 = SLOTS / 3;
  auto chunk = [&](int c, auto stc) {
    constexpr int ST = decltype(stc)::value;
    u32x4 xf[2][GB];
#pragma unroll
    for (int b = 0; b < GB; ++b) xf[0][b] = read_x(ST, 0, b);
    Pairs pr;
    Consts kc;
#pragma unroll
    for (int k = 0; k < 2 * NG; ++k) {
      const int i = k / NG;   // step of the chunk
      if (k % NG == 0) {      // the next step's: step 1 of this chunk, 0 of the next
        pr = lookup(code);
        kc = read_consts(i == 0 ? c : c + 1, 1 - i);
        code = read_codes(c + 1, i);
      }
      if (k + 1 < 2 * NG) {
#pragma unroll
        for (int b = 0; b < GB; ++b)
          xf[(k + 1) & 1][b] = read_x(ST, (k + 1) / NG, GB * ((k + 1) % NG) + b);
      }
      if (k == 0) {   // dY of the next chunk, codes of the one after, the next loads
        store_x(ST ^ 1, ST ^ 1);
        load_x(c + 3, ST ^ 1);
        store_codes(c + 2, ST);
        load_codes(c + 4, ST);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < GB; ++b)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          acc[f][GB * (k % NG) + b] =
              mfma16(af[i][f], xf[k & 1][b], acc[f][GB * (k % NG) + b]);
          const int slot = (k % NG * GB + b) * 2 + f;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (SLOT0 + u * (SLOTS - SLOT0) / 8 == slot)
              af[1 - i][u & 1][u >> 1] = scaled(pr, kc, u & 1, u >> 1);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
  };
  // (An odd chunk count adds a pass over a chunk past the end, all zeros.)
  for (int c = 0; c < nchunks; c += 2) {
    chunk(c, std::integral_constant<int, 0>{});
    chunk(c + 1, std::integral_constant<int, 1>{});
  }

  // LoRA update: 64 ranks at a time, the A tile [VK][64] and s . G as bf16 hi and lo
  // tiles [TQ][64], all in swizzled 128-byte rows.  (The two halves keep 16 of the
  // fp32 value's 24 bits, of which the bf16 result keeps 8.)
  f32x4 low[DROP ? 2 : 1][DROP ? TB : 1];
  if constexpr (DROP) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int b = 0; b < TB; ++b) low[f][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (a.r > 0) {
    uint16_t* const at = reinterpret_cast<uint16_t*>(dyn);
    uint16_t* const th = at + VK * 64;
    uint16_t* const tl = th + Tile::TQ * 64;
    const uint16_t* const Ae = a.B + (int64_t)e * K * a.r;
    for (int j0 = 0; j0 < a.r; j0 += 64) {
      constexpr int AP = VK * 8 / VT;         // 16-byte pieces of A a thread
      u32x4 aw[AP];
#pragma unroll
      for (int i = 0; i < AP; ++i) {
        const int row = srow + 64 * i, j = j0 + 8 * sq;
        aw[i] = k0 + row < K && j < a.r ? ld16(Ae + (k0 + row) * a.r + j) : u32x4{0, 0, 0, 0};
      }
      constexpr int TP = Tile::TQ * 16 / VT;   // 4-rank pieces of G a thread
      f32x4 tw[TP];
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int idx = tid + VT * i, row = idx / 16, j = j0 + 4 * (idx % 16);
        tw[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (q0 + row < mend && j < a.r)
          tw[i] = *reinterpret_cast<const f32x4*>(a.T + (q0 + row) * a.r + j);
      }
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int idx = tid + VT * i, row = idx / 16, q = idx % 16;
        const f32x4 v = tw[i] * a.s;
        uint32_t h0, h1, l0, l1;
        split_bf16x2(v.x, v.y, h0, l0);
        split_bf16x2(v.z, v.w, h1, l1);
        const int o = row * 64 + 8 * vslot(row, q >> 1) + 4 * (q & 1);
        *reinterpret_cast<u32x2*>(th + o) = u32x2{h0, h1};
        *reinterpret_cast<u32x2*>(tl + o) = u32x2{l0, l1};
      }
#pragma unroll
      for (int i = 0; i < AP; ++i) {
        const int row = srow + 64 * i;
        st_lds16(at + row * 64 + 8 * vslot(row, sq), aw[i]);
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 bf[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int row = 32 * wave + 2 * li + f;
          bf[f] = *reinterpret_cast<const u32x4*>(at + row * 64 + 8 * vslot(row, 4 * ks + g));
        }
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          const int row = 16 * b + li;
          const int o = row * 64 + 8 * vslot(row, 4 * ks + g);
          const u32x4 hi = *reinterpret_cast<const u32x4*>(th + o);
          const u32x4 lo = *reinterpret_cast<const u32x4*>(tl + o);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            f32x4& sum = DROP ? low[DROP ? f : 0][DROP ? b : 0] : acc[f][b];
            sum = mfma16(bf[f], hi, sum);
            sum = mfma16(bf[f], lo, sum);
          }
        }
      }
      __syncthreads();
    }
  }
  if constexpr (DROP) {
    if (a.r > 0) {
      const DropKey key = load_drop_key(a.state, a.thr);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int64_t m = q0 + 16 * b + li;
        const u32x4 w =
            philox_piece(key, static_cast<uint64_t>(m * K + k0 + 32 * wave + 8 * g) / 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[0][b][i] += (w[i] & 0xFFFFu) >= a.thr ? low[0][b][i] : 0.f;
          acc[1][b][i] += (w[i] >> 16) >= a.thr ? low[1][b][i] : 0.f;
        }
      }
    }
  }

  // dX: the lane's 8 consecutive columns 32 wave + 8 g .. of token li of each
  // subtile, through LDS, so that a wave stores whole token rows of the tile.
  uint16_t* const ys = reinterpret_cast<uint16_t*>(dyn);   // (behind a barrier either way)
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    const f32x4 u = acc[0][b], v = acc[1][b];
    *reinterpret_cast<u32x4*>(ys + (16 * b + li) * Tile::YROW + 32 * wave + 8 * g) =
        u32x4{pack_bf16x2(u.x, v.x), pack_bf16x2(u.y, v.y), pack_bf16x2(u.z, v.z),
              pack_bf16x2(u.w, v.w)};
  }
  __syncthreads();
  constexpr int YP = VK / 8;   // 16-byte pieces of a token row
#pragma unroll
  for (int i = 0; i < Tile::TQ * YP / VT; ++i) {
    const int idx = tid + VT * i, row = idx / YP, pc = idx % YP;
    const int64_t m = q0 + row, k = k0 + 8 * pc;
    if (m < mend && k < K)
      *reinterpret_cast<u32x4*>(a.Y + m * K + k) =
          *reinterpret_cast<const u32x4*>(ys + row * Tile::YROW + 8 * pc);
  }
}

template <bool NODQ, bool DROP>
__global__ __launch_bounds__(VT, 2) void k_expert_dx(ExpertArgs a, Nf4Tables tb) {
  // Dynamic LDS only: the level table sits at address 0.
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  GroupTiles<16 * VTB> groups(a.offsets, a.E, a.M);
  build_rep_pair_table<VT>(reinterpret_cast<char*>(dyn), load_levels(tb), threadIdx.x);
  int pt, z;
  const GroupTile gt = expert_deal(a, groups, pt, z);
  if (gt.e < 0) return;
  const int rows = gt.end - gt.row0;
  if (rows <= 64)
    dx_expert_tile<4, NODQ, DROP>(a, dyn, gt.e, gt.row0, gt.end, pt);
  else if (rows <= 128)
    dx_expert_tile<8, NODQ, DROP>(a, dyn, gt.e, gt.row0, gt.end, pt);
  else
    dx_expert_tile<VTB, NODQ, DROP>(a, dyn, gt.e, gt.row0, gt.end, pt);
}

template <bool NODQ, bool DROP>
hipError_t launch_tiles(const ExpertArgs& a, const Nf4Tables& tb, hipStream_t stream) {
  constexpr int kLds = VTile<VTB>::LDS;
  static_assert(kLds >= VTile<8>::LDS && kLds >= VTile<4>::LDS, "the widest body's LDS");
  static LdsLimit lds;
  const hipError_t attr = lds.raise(reinterpret_cast<const void*>(&k_expert_dx<NODQ, DROP>), kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_expert_dx<NODQ, DROP>),
                     dim3(static_cast<unsigned>(xcd_deal_grid(a.qtiles, a.ptiles))), dim3(VT), kLds,
                     stream, a, tb);
  return hipGetLastError();
}

}  // namespace

// Whole backwards (r = 64) with this kernel / with the other, which has narrower tiles
// and can split its reduction: 8 experts of 4096 x 4096 with 1024 rows (208 tiles at
// most) 111 / 96 us, with 2048 rows (288 tiles) 126 / 157; 32 experts of 2048 x 1024
// with 4096 rows (212) 85 / 81, with 8192 rows (296) 96 / 128; 64 experts of 1024 x
// 2048 with 128 rows (512) 61 / 80.  With up to 4 experts next to all tiles are full ones, and
// the rounds that 256 CUs need for them count; a round of this kernel's takes 1.28
// times as long as one of the other's 128 columns x 256 tokens.  One expert of
// 11008 x 4096, 3900 rows of X (2 rounds of either): 528 / 442 us; 4096 x
// 11008, 2048 rows (2 rounds / 3): 233 / 269.
bool expert_dx_fits(int64_t M, int E, int64_t K) {
  const int64_t tiles = (K + VK - 1) / VK * group_tile_bound(M, E, 16 * VTB);
  if (tiles < 256 || E > 4) return tiles >= 256;
  const int64_t other = (K + 127) / 128 * group_tile_bound(M, E, 256);
  return 128 * ((tiles + 255) / 256) <= 100 * ((other + 255) / 256);
}

int64_t expert_dx_threads(int64_t M, int E, int64_t K) {
  return VT * xcd_deal_grid(group_tile_bound(M, E, 16 * VTB), (K + VK - 1) / VK);
}

hipError_t launch_expert_dx(const uint16_t* dY, int64_t M, const int* offsets, int E,
                            const Nf4View& w, const float* G, const uint16_t* A, int r, float s,
                            uint16_t* dX, const Nf4Tables& tb, hipStream_t stream,
                            const Drop& d) {
  const ExpertArgs a{dY, M, offsets, E, w.codes, w.absmax_q, w.absmax_scale, w.N / E, w.K, G,
                     nullptr, A, dX, nullptr, 0, r, static_cast<int>((w.K + VK - 1) / VK),
                     static_cast<int>(group_tile_bound(M, E, 16 * VTB)), 1, 0, 1.f,
                     s * d.scale(), d.state, d.thr};
  auto launch = d.on() ? (w.dq ? launch_tiles<false, true> : launch_tiles<true, true>)
                       : (w.dq ? launch_tiles<false, false> : launch_tiles<true, false>);
  return launch(a, tb, stream);
}

}  // namespace qnf4
