// Tile building blocks of the rank-r products (T = X.A, G = dY.B^T, dA, dB),
// shared by the plain layer's products (gemm.hip) and those grouped by expert
// (grouped.hip): operand loaders, the MFMA tile step, the double-buffered tile
// loop and the stores of a tile of C[q, p] = sum_k P[p, k] . Q[q, k].
#pragma once

#include <type_traits>

#include "device_common.hpp"
#include "dropout.hpp"

namespace qnf4 {

constexpr int BK = 64;              // reduction elements per tile
constexpr int LDS_STRIDE = BK + 8;  // bf16 per LDS row: 144 B, spreads rows over banks
constexpr int NT = 256;             // threads per workgroup (4 waves)

struct OpParams {
  const void* ptr;
  int64_t ld;      // leading dimension of the source array (elements)
  int64_t nrows;   // extent of the tile-row index
  int64_t nred;    // extent of the reduction index
  int64_t drow0;   // masked operands: row of the whole tensor that ptr points to
  float scale;     // fp32 sources: value = scale * src
};

__device__ __forceinline__ u32x4 ld16(const void* p) {
  return *reinterpret_cast<const u32x4*>(p);
}
__device__ __forceinline__ void st_lds16(uint16_t* p, u32x4 v) {
  *reinterpret_cast<u32x4*>(p) = v;
}

// ---------------------------------------------------------------------------
// Loaders.  load(kt) fetches reduction tile kt into registers; store(lds)
// writes the tile [ROWS][LDS_STRIDE] to LDS; elements outside the operand
// are zero.  With DROP the operand is X under the adapter's dropout mask: the
// mask of each 16-byte piece (a generator's piece: ld % 8 == 0) is formed while
// the piece is on its way and applied when it is stored.
// ---------------------------------------------------------------------------

template <int ROWS, bool DROP = false>
struct Bf16Nat {   // element (row, k) = src[row * ld + k]
  static constexpr bool kDrop = DROP;
  static constexpr int TILE = ROWS * LDS_STRIDE;
  __device__ static u32x4 frag(const uint16_t* tile, int c0, int ks, int lane) {
    return *reinterpret_cast<const u32x4*>(tile + (c0 + (lane & 15)) * LDS_STRIDE + 32 * ks +
                                           8 * (lane >> 4));
  }
  static constexpr int CH = ROWS * BK / 8;              // 16-byte chunks
  static constexpr int CPT = (CH + NT - 1) / NT;
  OpParams o;
  int64_t row0;
  u32x4 r[CPT];
  std::conditional_t<DROP, DropKey, NoDropKey> key;
  u32x4 mask[DROP ? CPT : 1];
  __device__ void load(int kt, int tid) {
    const uint16_t* src = static_cast<const uint16_t*>(o.ptr);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT;
      const int row = idx >> 3, kc = idx & 7;
      const int64_t gr = row0 + row, gk = (int64_t)kt * BK + kc * 8;
      r[c] = (idx < CH && gr < o.nrows && gk < o.nred) ? ld16(src + gr * o.ld + gk)
                                                        : u32x4{0, 0, 0, 0};
      if constexpr (DROP)
        mask[c] = keep_piece(key, static_cast<uint64_t>((o.drow0 + gr) * o.ld + gk) / 8);
    }
  }
  __device__ void store(uint16_t* lds, int tid) {
    if constexpr (DROP) {
#pragma unroll
      for (int c = 0; c < CPT; ++c) r[c] &= mask[c];
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT;
      if (idx < CH) st_lds16(lds + (idx >> 3) * LDS_STRIDE + (idx & 7) * 8, r[c]);
    }
  }
};

// ---------------------------------------------------------------------------
// Reduction-major operands (element (row, k) = src[k * ld + row]: X^T, dY^T,
// and the fp32 G^T, T^T of the adapter gradients).  The tile is stored as it
// lies in memory, [BK reduction rows][COLS] (coalesced 16-byte loads, no
// register transposes), and the MFMA fragment -- 8 consecutive reduction
// elements of one row per lane -- is read with ds_read_b64_tr_b16, which
// transposes 4 x 16 blocks of 16-bit elements across each 16-lane group.
// 16-byte pieces are XOR-swizzled in 32-byte units so the 8 tile rows of a
// half-wave transposing read (rows 8g + 4e + i, g = 0, 1) hit distinct banks.
// ---------------------------------------------------------------------------

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 LdsV4i16;

template <int COLS>
__device__ __forceinline__ int rm_slot(int row, int piece) {
  static_assert(COLS == 64 || COLS == 128, "tile width");
  const int f = COLS == 64 ? (((row >> 1) & 1) | (((row >> 3) & 1) << 1))   // 128-byte rows
                           : ((row & 3) | (((row >> 3) & 1) << 2));          // 256-byte rows
  return piece ^ (2 * f);
}

// Fragment of tile rows (columns) c0 .. c0+15, reduction step ks.
template <int COLS>
__device__ __forceinline__ u32x4 rm_frag(const uint16_t* tile, int c0, int ks, int lane) {
  const int li = lane & 15, g = lane >> 4;
  const int col = c0 + 4 * (li & 3);
  u32x2 h[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int red = 32 * ks + 8 * g + 4 * e + (li >> 2);
    const uint16_t* p = tile + red * COLS + 8 * rm_slot<COLS>(red, col >> 3) + (col & 7);
    h[e] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4i16*)(p)));
  }
  return u32x4{h[0][0], h[0][1], h[1][0], h[1][1]};
}

template <int COLS, bool DROP = false>
struct Bf16RedMajor {   // element (row, k) = src[k * ld + row], bf16
  static constexpr bool kDrop = DROP;
  static constexpr int TILE = BK * COLS;
  static constexpr int PCS = COLS / 8;                 // 16-byte pieces per tile row
  static constexpr int CPT = BK * PCS / NT;            // pieces a thread
  OpParams o;
  int64_t row0;
  u32x4 r[CPT];
  std::conditional_t<DROP, DropKey, NoDropKey> key;
  u32x4 mask[DROP ? CPT : 1];
  __device__ void load(int kt, int tid) {
    const uint16_t* src = static_cast<const uint16_t*>(o.ptr);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT, red = idx / PCS, pc = idx % PCS;
      const int64_t gk = (int64_t)kt * BK + red, gr = row0 + 8 * pc;
      r[c] = (gk < o.nred && gr < o.nrows) ? ld16(src + gk * o.ld + gr) : u32x4{0, 0, 0, 0};
      if constexpr (DROP)
        mask[c] = keep_piece(key, static_cast<uint64_t>((o.drow0 + gk) * o.ld + gr) / 8);
    }
  }
  __device__ void store(uint16_t* lds, int tid) {
    if constexpr (DROP) {
#pragma unroll
      for (int c = 0; c < CPT; ++c) r[c] &= mask[c];
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT, red = idx / PCS, pc = idx % PCS;
      st_lds16(lds + red * COLS + 8 * rm_slot<COLS>(red, pc), r[c]);
    }
  }
  __device__ static u32x4 frag(const uint16_t* tile, int c0, int ks, int lane) {
    return rm_frag<COLS>(tile, c0, ks, lane);
  }
};

template <int COLS>
struct F32RedMajor {    // element (row, k) = scale * src[k * ld + row], fp32 -> bf16 hi, lo
  static constexpr bool kDrop = false;
  static constexpr int TILE = BK * COLS;
  static constexpr int QCS = COLS / 4;                 // 4-float pieces per tile row
  static constexpr int CPT = BK * QCS / NT;
  OpParams o;
  int64_t row0;
  f32x4 r[CPT];
  __device__ void load(int kt, int tid) {
    const float* src = static_cast<const float*>(o.ptr);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT, red = idx / QCS, qc = idx % QCS;
      const int64_t gk = (int64_t)kt * BK + red, gr = row0 + 4 * qc;
      r[c] = (gk < o.nred && gr < o.nrows) ? *reinterpret_cast<const f32x4*>(src + gk * o.ld + gr)
                                           : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  __device__ void store2(uint16_t* hi, uint16_t* lo, int tid) {
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int idx = tid + c * NT, red = idx / QCS, qc = idx % QCS;
      uint32_t h0, l0, h1, l1;
      split_bf16x2(r[c].x * o.scale, r[c].y * o.scale, h0, l0);
      split_bf16x2(r[c].z * o.scale, r[c].w * o.scale, h1, l1);
      const int off = red * COLS + 8 * rm_slot<COLS>(red, qc >> 1) + 4 * (qc & 1);
      *reinterpret_cast<u32x2*>(hi + off) = u32x2{h0, h1};
      *reinterpret_cast<u32x2*>(lo + off) = u32x2{l0, l1};
    }
  }
  __device__ static u32x4 frag(const uint16_t* tile, int c0, int ks, int lane) {
    return rm_frag<COLS>(tile, c0, ks, lane);
  }
};

// ---------------------------------------------------------------------------
// MFMA tile step and the double-buffered tile loop
// ---------------------------------------------------------------------------

template <int BP, int BQ>
struct Mma {
  static constexpr int TP = BP / 32, TQ = BQ / 32;   // 16x16 tiles per wave
  f32x4 acc[TP][TQ];
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // FP, FQ: the operands' tile layouts (their loaders' frag readers)
  template <class FP, class FQ>
  __device__ void step(const uint16_t* ldsP, const uint16_t* ldsQ, int wave, int lane) {
    const int wp = (wave & 1) * (BP / 2), wq = (wave >> 1) * (BQ / 2);
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      u32x4 a[TP], b[TQ];
#pragma unroll
      for (int i = 0; i < TP; ++i) a[i] = FP::frag(ldsP, wp + 16 * i, ks, lane);
#pragma unroll
      for (int j = 0; j < TQ; ++j) b[j] = FQ::frag(ldsQ, wq + 16 * j, ks, lane);
#pragma unroll
      for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) acc[i][j] = mfma16(a[i], b[j], acc[i][j]);
    }
  }
};

// Runs reduction tiles [kt0, kt1) through two LDS buffers with a ring of D
// register stages (tiles are loaded D ahead; a depth of 4 measured no faster
// than 2 for these memory-light tiles).  HL selects
// an fp32 operand split into bf16 hi and lo halves (1: P, 2: Q): both halves
// are staged per tile and multiplied against the other operand, which is
// loaded once.  Buffer layout: [P or P_hi][Q or Q_hi][second half].
template <int BP, int BQ, int HL, int D, class LP, class LQ>
__device__ void run_tiles(const LP& lp0, const LQ& lq0, int kt0, int kt1, Mma<BP, BQ>& mma,
                          uint16_t* lds, int tid) {
  static_assert(D % 2 == 0, "the ring depth keeps the LDS buffer of a slot fixed");
  if (kt0 >= kt1) return;
  constexpr int XT = HL == 0 ? 0 : (HL == 1 ? LP::TILE : LQ::TILE);   // the extra (lo) tile
  constexpr int BUF = LP::TILE + LQ::TILE + XT;
  const int wave = wave_id(), lane = tid & 63;
  LP lp[D];
  LQ lq[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    lp[d] = lp0;
    lq[d] = lq0;
  }
  auto P = [&](int b) { return lds + b * BUF; };
  auto Q = [&](int b) { return lds + b * BUF + LP::TILE; };
  auto X = [&](int b) { return lds + b * BUF + LP::TILE + LQ::TILE; };
  auto load = [&](int t, int d) {
    if (t < kt1) {
      lp[d].load(t, tid);
      lq[d].load(t, tid);
    }
  };
  auto store = [&](int d, int b) {
    if constexpr (HL == 0) {
      lp[d].store(P(b), tid);
      lq[d].store(Q(b), tid);
    } else if constexpr (HL == 1) {
      lp[d].store2(P(b), X(b), tid);
      lq[d].store(Q(b), tid);
    } else {
      lp[d].store(P(b), tid);
      lq[d].store2(Q(b), X(b), tid);
    }
  };
  auto step = [&](int b) {
    mma.template step<LP, LQ>(P(b), Q(b), wave, lane);
    if constexpr (HL == 1) mma.template step<LP, LQ>(X(b), Q(b), wave, lane);
    if constexpr (HL == 2) mma.template step<LP, LQ>(P(b), X(b), wave, lane);
  };
  // tile t lives in register slot (t - kt0) % D and LDS buffer (t - kt0) % 2
#pragma unroll
  for (int d = 0; d < D; ++d) load(kt0 + d, d);
  store(0, 0);
  load(kt0 + D, 0);
  __syncthreads();
  for (int kt = kt0; kt < kt1; kt += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int t = kt + u;
      if (t < kt1) {
        step(u & 1);
        if (t + 1 < kt1) {
          store((u + 1) % D, (u & 1) ^ 1);
          load(t + 1 + D, (u + 1) % D);
        }
        __syncthreads();
      }
    }
  }
}

// Stores C[q, p] as bf16 (lane holds 4 consecutive p of one q per tile).
template <int BP, int BQ>
__device__ void store_bf16(const Mma<BP, BQ>& mma, uint16_t* out, int64_t ldo,
                           int64_t p0, int64_t q0, int64_t P, int64_t Q, int tid) {
  const int wave = wave_id(), lane = tid & 63;
  const int64_t wp = p0 + (wave & 1) * (BP / 2) + 4 * (lane >> 4);
  const int64_t wq = q0 + (wave >> 1) * (BQ / 2) + (lane & 15);
#pragma unroll
  for (int i = 0; i < Mma<BP, BQ>::TP; ++i)
#pragma unroll
    for (int j = 0; j < Mma<BP, BQ>::TQ; ++j) {
      const int64_t p = wp + 16 * i, q = wq + 16 * j;
      if (p < P && q < Q) {   // P % 4 == 0, so the 4 values are all in range
        const f32x4 v = mma.acc[i][j];
        *reinterpret_cast<u32x2*>(out + q * ldo + p) =
            u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      }
    }
}

template <int BP, int BQ>
__device__ void store_f32(const Mma<BP, BQ>& mma, float* out, int64_t ldo,
                          int64_t p0, int64_t q0, int64_t P, int64_t Q, int tid) {
  const int wave = wave_id(), lane = tid & 63;
  const int64_t wp = p0 + (wave & 1) * (BP / 2) + 4 * (lane >> 4);
  const int64_t wq = q0 + (wave >> 1) * (BQ / 2) + (lane & 15);
#pragma unroll
  for (int i = 0; i < Mma<BP, BQ>::TP; ++i)
#pragma unroll
    for (int j = 0; j < Mma<BP, BQ>::TQ; ++j) {
      const int64_t p = wp + 16 * i, q = wq + 16 * j;
      if (p < P && q < Q) *reinterpret_cast<f32x4*>(out + q * ldo + p) = mma.acc[i][j];
    }
}

}  // namespace qnf4
