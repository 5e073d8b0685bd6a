// Root-mean-square norm in front of a layer: the residual's addition, the norm,
// and the 8-bit checkpoint of its output in one pass; and its backward.
//
//   forward    h = bf16(x + residual),  rstd = (mean_k h^2 + eps)^-1/2,
//              y = bf16(h rstd g),  y8 = checkpoint of y
//   backward   n = h rstd,  c = mean_k(dy g n),
//              dx = bf16(dres + rstd (dy g - n c)),  dg = sum over rows of dy n
//
// A row stays in the registers of the threads that share it (64 to 1024 of them,
// each with up to eight 16-byte pieces, in the backward with two), so that every byte
// is read once; rows too long for that (65536 values, in the backward 16384) are read
// twice, and in the backward with dg a third time, by a launch of its own for the
// columns.  Squares, sums and everything up to the one rounding of an output are fp32.
// Bound by the bytes they move: with three sets of buffers in turn, 4096 x 6656 with
// residual and checkpoint takes 52 us (247 MB, 4.8 TB/s), without the checkpoint 45
// (4.8); the backward of 4096 x 8192 60 us (268 MB, 57 without dg), where a large copy
// reaches 5.0 (on one set, which the 256 MB cache holds in part, 45, 38 and 57).
// 4096 x 17920 take 114 us forward, 133 backward (read twice) and 189 with dg (three
// times; 587 MB would take 118).  A row of up to 512 values is a wave's, which leaves lanes of
// short ones idle: 131072 x 128 take 52 us forward and 68 backward (27 by their bytes),
// x 256 60 and 76 (54).  Loads and stores marked non-temporal gained nothing (45.9 and
// 43.1 us the forward, 58.1 and 57.2 the backward with dg, with and without).
//
// dg's sum runs over rows: each workgroup adds up the rows it takes (always the
// same ones) in registers and a second launch adds the workgroups' sums in
// order (4.5 us).  Few rows skip both: workgroups of the one launch add up whole
// columns, reading the rows again.
#include <algorithm>
#include <cmath>

#include "act8.hpp"
#include "device_common.hpp"
#include "kernels.hpp"
#include "qlora_nf4.h"

namespace qnf4 {

namespace {

// Workgroups lie in rows of this many along y (a launch holds fewer than 2^32
// threads along x).
constexpr int64_t kRowBlocks = int64_t(1) << 21;

struct NormFwd {
  const uint16_t* x;
  const uint16_t* residual;   // may be null: h is x
  const void* g;
  int64_t M, K;
  float eps;
  uint16_t* h;
  uint16_t* y;
  float* rstd;
  int8_t* codes;              // may be null: no checkpoint
  float* scales;
  int g_fp32;
};

struct NormBwd {
  const uint16_t* dy;
  const uint16_t* dres;       // may be null
  const uint16_t* h;
  const float* rstd;
  const void* g;
  int64_t M, K;
  uint16_t* dx;
  void* dg;                   // may be null
  float* part;                // sums of dy n that a second launch adds up, or null
  int64_t row_blocks;         // workgroups for rows, and for columns after them (a
  int64_t col_blocks;         // grid of several rows holds more than both)
  int64_t run_rows;           // rows of a run of those
  int g_fp32;
};

// Sum over the wave, in every lane, always in the same order.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);    // quad_perm 1,0,3,2
  v += dpp_f32<0x4E>(v);    // quad_perm 2,3,0,1
  v += dpp_f32<0x141>(v);   // row_half_mirror
  v += dpp_f32<0x140>(v);   // row_mirror
  const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 0));
  const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16));
  const float c = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 32));
  const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 48));
  return (a + b) + (c + d);
}

// Sum over the TPR threads of a row.  red: TPR / 64 floats that no thread still
// reads (alternate two of them between barriers).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) s += red[w];
  return s;
}

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack8(u32x4 w) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i];
    f.v[2 * i] = bf16_lo_to_f32(u);
    f.v[2 * i + 1] = bf16_hi_to_f32(u);
  }
  return f;
}
__device__ __forceinline__ u32x4 pack8(const F8& f) {
  return u32x4{pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
               pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7])};
}
__device__ __forceinline__ u32x4 ld8(const uint16_t* p) {
  return *reinterpret_cast<const u32x4*>(p);
}
__device__ __forceinline__ void st8(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4*>(p) = v; }

// Eight factors g from column c.
__device__ __forceinline__ F8 load_g(const void* g, int fp32, int64_t c) {
  if (!fp32) return unpack8(ld8(static_cast<const uint16_t*>(g) + c));
  F8 f;
  const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(g) + c);
  const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(g) + c + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[i] = a[i];
    f.v[4 + i] = b[i];
  }
  return f;
}

__device__ __forceinline__ u32x4 add_residual(u32x4 x, u32x4 r) {
  F8 a = unpack8(x);
  const F8 b = unpack8(r);
#pragma unroll
  for (int i = 0; i < 8; ++i) a.v[i] += b.v[i];
  return pack8(a);
}

__device__ __forceinline__ float square_sum(u32x4 h, float s) {
  const F8 f = unpack8(h);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f.v[i], f.v[i], s);
  return s;
}

// y and its checkpoint from eight values of h.
__device__ __forceinline__ void norm_out(const NormFwd& a, u32x4 h, float rstd, int64_t row,
                                         int64_t c) {
  F8 f = unpack8(h);
  const F8 g = load_g(a.g, a.g_fp32, c);
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = f.v[i] * rstd * g.v[i];
  const u32x4 y = pack8(f);
  st8(a.y + row * a.K + c, y);
  if (a.codes) {   // eight lanes hold a block
    const Act8Scale s = act8_scale(max_over8(amax_bits8(y)));
    *reinterpret_cast<u32x2*>(a.codes + row * a.K + c) = act8_codes(y, s);
    if ((threadIdx.x & 7) == 0) a.scales[(row * a.K + c) / 64] = s.c;
  }
}

template <int TPR>
constexpr int row_threads() {
  return TPR < 256 ? 256 : TPR;
}

__device__ __forceinline__ int64_t block_index() {
  return (int64_t)blockIdx.y * kRowBlocks + blockIdx.x;
}

}  // namespace

// TPR threads a row, P pieces each; P = 0: rows of any length, read twice.
template <int TPR, int P>
__global__ __launch_bounds__(row_threads<TPR>()) void k_rms_fwd(NormFwd a) {
  constexpr int RPB = row_threads<TPR>() / TPR;
  __shared__ float red[TPR / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = block_index() * RPB + threadIdx.x / TPR;
  if (row >= a.M) return;   // (uniform over the threads that meet at a barrier)
  const uint16_t* x = a.x + row * a.K;
  const uint16_t* res = a.residual ? a.residual + row * a.K : nullptr;
  float ss = 0.f;
  if constexpr (P > 0) {
    u32x4 h[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t c = 8 * (p * TPR + t);
      h[p] = c < a.K ? ld8(x + c) : u32x4{0, 0, 0, 0};
    }
    if (res) {
      u32x4 r[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t c = 8 * (p * TPR + t);
        r[p] = c < a.K ? ld8(res + c) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t c = 8 * (p * TPR + t);
        h[p] = add_residual(h[p], r[p]);
        if (c < a.K) st8(a.h + row * a.K + c, h[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) ss = square_sum(h[p], ss);
    const float rstd = 1.f / sqrtf(row_sum<TPR>(ss, red) / static_cast<float>(a.K) + a.eps);
    if (t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t c = 8 * (p * TPR + t);
      if (c < a.K) norm_out(a, h[p], rstd, row, c);
    }
  } else {
    for (int64_t c = 8 * t; c < a.K; c += 8 * TPR) {
      u32x4 h = ld8(x + c);
      if (res) {
        h = add_residual(h, ld8(res + c));
        st8(a.h + row * a.K + c, h);
      }
      ss = square_sum(h, ss);
    }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(ss, red) / static_cast<float>(a.K) + a.eps);
    if (t == 0) a.rstd[row] = rstd;
    const uint16_t* h = res ? a.h + row * a.K : x;   // (a thread reads what it wrote itself)
    for (int64_t c = 8 * t; c < a.K; c += 8 * TPR) norm_out(a, ld8(h + c), rstd, row, c);
  }
}

namespace {

// Sums of dy n down 128 columns, of the rows from a run's first on: 16 threads a
// row, THREADS / 16 rows at a time.  With more runs than one they go to part.
template <int THREADS>
__device__ __forceinline__ void dg_columns(const NormBwd& a, int64_t block, float* lds) {
  constexpr int segs = THREADS / 16;
  const int t = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int64_t ncols = (a.K + 127) / 128, run = block / ncols;
  block -= run * ncols;
  const int64_t r0 = run * a.run_rows, r1 = min(a.M, r0 + a.run_rows);
  const int64_t c = 128 * block + 8 * t;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.K) {
#pragma unroll 4
    for (int64_t row = r0 + seg; row < r1; row += segs) {
      const F8 d = unpack8(ld8(a.dy + row * a.K + c)), h = unpack8(ld8(a.h + row * a.K + c));
      const float rstd = a.rstd[row];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(d.v[i], h.v[i] * rstd, s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) lds[threadIdx.x * 9 + i] = s[i];   // (9: no bank conflicts)
  __syncthreads();
  const int64_t col = 128 * block + threadIdx.x;
  if (threadIdx.x < 128 && col < a.K) {
    float v = 0.f;
    for (int j = 0; j < segs; ++j)
      v += lds[(16 * j + (threadIdx.x >> 3)) * 9 + (threadIdx.x & 7)];
    if (a.part)
      a.part[run * a.K + col] = v;
    else if (a.g_fp32)
      static_cast<float*>(a.dg)[col] = v;
    else
      static_cast<uint16_t*>(a.dg)[col] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
  }
}

// Of eight columns: the gradient g dy - n c, and what it needs.
__device__ __forceinline__ float norm_dot(const F8& h, const F8& dy, const F8& g, float rstd,
                                          float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(dy.v[i] * g.v[i], h.v[i] * rstd, s);
  return s;
}
__device__ __forceinline__ u32x4 norm_dx(const F8& h, const F8& dy, const F8& g, float rstd,
                                         float c, const F8& dres) {
  F8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o.v[i] = fmaf(rstd, fmaf(-(h.v[i] * rstd), c, dy.v[i] * g.v[i]), dres.v[i]);
  return pack8(o);
}

}  // namespace

template <int TPR, int P>
__global__ __launch_bounds__(row_threads<TPR>()) void k_rms_bwd(NormBwd a) {
  constexpr int NTHR = row_threads<TPR>(), RPB = NTHR / TPR;
  __shared__ float red[2][TPR / 64];
  // for the sums of columns, or of the waves that take a row each
  constexpr int kWaveSums = RPB > 1 ? RPB * 512 * P : 0;
  __shared__ __attribute__((aligned(16))) float
      cols[P == 0 ? 1 : (kWaveSums > NTHR * 9 ? kWaveSums : NTHR * 9)];
  const int64_t block = block_index();
  if constexpr (P > 0) {
    if (block >= a.row_blocks) {   // uniform
      if (block - a.row_blocks < a.col_blocks) dg_columns<NTHR>(a, block - a.row_blocks, cols);
      return;
    }
  }
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const F8 zero{};
  if constexpr (P > 0) {
    float acc[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[p][i] = 0.f;
    // the next row's loads are on their way while this one is summed and written
    struct Row {
      u32x4 h[P], dy[P], dr[P];
      float rstd;
    };
    auto load = [&](Row& v, int64_t row) {
      v.rstd = a.rstd[row];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t c = 8 * (p * TPR + t), i = row * a.K + c;
        const bool in = c < a.K;
        v.h[p] = in ? ld8(a.h + i) : u32x4{0, 0, 0, 0};
        v.dy[p] = in ? ld8(a.dy + i) : u32x4{0, 0, 0, 0};
        v.dr[p] = in && a.dres ? ld8(a.dres + i) : u32x4{0, 0, 0, 0};
      }
    };
    const int64_t step = a.row_blocks * RPB;
    int64_t row = block * RPB + sub;
    Row now, next;
    if (row < a.M) load(now, row);
    for (int turn = 0; row < a.M; row += step, turn ^= 1) {
      if (row + step < a.M) load(next, row + step);
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t c = 8 * (p * TPR + t);
        if (c < a.K)
          s = norm_dot(unpack8(now.h[p]), unpack8(now.dy[p]), load_g(a.g, a.g_fp32, c), now.rstd, s);
      }
      const float mean = row_sum<TPR>(s, red[turn]) / static_cast<float>(a.K);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t c = 8 * (p * TPR + t);
        if (c >= a.K) continue;
        const F8 fh = unpack8(now.h[p]), fd = unpack8(now.dy[p]);
        st8(a.dx + row * a.K + c,
            norm_dx(fh, fd, load_g(a.g, a.g_fp32, c), now.rstd, mean, unpack8(now.dr[p])));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[p][i] = fmaf(fd.v[i], fh.v[i] * now.rstd, acc[p][i]);
      }
      now = next;
    }
    if (a.part) {
      float* out = a.part + block * a.K;
      if constexpr (RPB > 1) {   // the rows' waves, added up in order
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<f32x4*>(cols + 8 * (p * TPR + t) + i + sub * 512 * P) =
                f32x4{acc[p][i], acc[p][i + 1], acc[p][i + 2], acc[p][i + 3]};
        __syncthreads();
        for (int c = 4 * threadIdx.x; c < a.K; c += 4 * NTHR) {
          f32x4 v = *reinterpret_cast<const f32x4*>(cols + c);
#pragma unroll
          for (int w = 1; w < RPB; ++w) v += *reinterpret_cast<const f32x4*>(cols + c + w * 512 * P);
          *reinterpret_cast<f32x4*>(out + c) = v;
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int64_t c = 8 * (p * TPR + t);
          if (c >= a.K) continue;
          *reinterpret_cast<f32x4*>(out + c) = f32x4{acc[p][0], acc[p][1], acc[p][2], acc[p][3]};
          *reinterpret_cast<f32x4*>(out + c + 4) = f32x4{acc[p][4], acc[p][5], acc[p][6], acc[p][7]};
        }
      }
    }
  } else {
    const int64_t row = block;
    if (row >= a.M) return;
    const float rstd = a.rstd[row];
    const uint16_t *h = a.h + row * a.K, *dy = a.dy + row * a.K;
    float s = 0.f;
    for (int64_t c = 8 * t; c < a.K; c += 8 * TPR)
      s = norm_dot(unpack8(ld8(h + c)), unpack8(ld8(dy + c)), load_g(a.g, a.g_fp32, c), rstd, s);
    const float mean = row_sum<TPR>(s, red[0]) / static_cast<float>(a.K);
    for (int64_t c = 8 * t; c < a.K; c += 8 * TPR)
      st8(a.dx + row * a.K + c,
          norm_dx(unpack8(ld8(h + c)), unpack8(ld8(dy + c)), load_g(a.g, a.g_fp32, c), rstd, mean,
                  a.dres ? unpack8(ld8(a.dres + row * a.K + c)) : zero));
  }
}

// Whole columns alone, for rows too long for the kernel above to add them up.
__global__ __launch_bounds__(256) void k_rms_dg_columns(NormBwd a) {
  __shared__ float cols[256 * 9];
  if (block_index() < a.col_blocks) dg_columns<256>(a, block_index(), cols);
}

// dg[c] = sum_p part[p][c]: 64 columns a workgroup, 64 runs of the parts, four
// columns a thread.
__global__ __launch_bounds__(1024) void k_rms_dg(const float* part, int64_t parts, int64_t K,
                                                 void* dg, int g_fp32) {
  __shared__ f32x4 sums[64][17];
  const int t = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int64_t c = 64 * (int64_t)blockIdx.x + 4 * t;
  const int64_t per = (parts + 63) / 64, p0 = min(parts, seg * per), p1 = min(parts, p0 + per);
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < K) {
#pragma unroll 4
    for (int64_t p = p0; p < p1; ++p) s += *reinterpret_cast<const f32x4*>(part + p * K + c);
  }
  sums[seg][t] = s;
  __syncthreads();
  if (seg < 8) {
#pragma unroll
    for (int j = 8; j < 64; j += 8) s += sums[seg + j][t];
  }
  __syncthreads();
  if (seg < 8) sums[seg][t] = s;
  __syncthreads();
  if (seg == 0 && c < K) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sums[j][t];
    if (g_fp32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(dg) + c) = s;
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(dg) + c) =
          u32x2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
  }
}

namespace {

constexpr int64_t kMaxK = int64_t(1) << 22;
constexpr int64_t kMaxActs = int64_t(1) << 40;
constexpr int64_t kLongRow = 65536;     // more than this: read twice

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

dim3 grid_of(int64_t blocks) {
  return dim3(static_cast<unsigned>(std::min(blocks, kRowBlocks)),
              static_cast<unsigned>(cdiv(blocks, kRowBlocks)));
}

int check_norm(int64_t M, int64_t K) {
  if (K < 8 || K % 8 != 0 || K > kMaxK || M < 0 || M > kMaxActs / K) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

template <int TPR, int P>
void fwd(const NormFwd& a, hipStream_t st) {
  constexpr int n = row_threads<TPR>();
  hipLaunchKernelGGL((k_rms_fwd<TPR, P>), grid_of(cdiv(a.M, n / TPR)), dim3(n), 0, st, a);
}

// Of the backward: workgroups for rows; how many sums of rows a second launch adds
// up (0: none); the rows of a run down the columns (0: none).
struct BwdPlan {
  int64_t row_blocks, parts, run_rows;
};
constexpr int64_t kLongRowBwd = 16384;   // more than this: read twice
int bwd_threads(int64_t K) { return K <= 2048 ? 256 : (K <= 4096 ? 512 : 1024); }

BwdPlan plan_bwd(int64_t M, int64_t K, bool dg) {
  BwdPlan p{cdiv(M, K <= 1024 ? 4 : 1), 0, 0};
  if (!dg) return p;
  if (K > kLongRowBwd) {
    // columns in a launch of their own, in runs of rows that fill the GPU
    const int64_t runs = std::max<int64_t>(1, std::min(M / 64, 1024 / cdiv(K, 128)));
    p.run_rows = std::max<int64_t>(1, cdiv(M, runs));
    p.parts = runs > 1 ? cdiv(M, p.run_rows) : 0;
  } else if (M > 1024 || (M > 512 && M * K > (int64_t(1) << 22))) {
    // Adding up columns reads dy and h twice, where sums of the workgroups are written
    // and read and take a second launch (512 x 8192: columns 12.9 us, sums 16.0; 1024 x
    // 4096: 15.0 and 16.3; 1024 x 8192: 23.1 and 19.9).  16 waves a CU: enough loads in
    // flight, and the fewest sums (4096 x 8192: 57 us with 256 workgroups of 1024
    // threads, 63 with 512, 61 with 512 of 512).
    p.row_blocks = std::min<int64_t>(p.row_blocks, 256 * (1024 / bwd_threads(K)));
    p.parts = p.row_blocks;
  } else {
    p.run_rows = std::max<int64_t>(1, M);
  }
  return p;
}
size_t bwd_need(const BwdPlan& p, int64_t K) {
  return static_cast<size_t>(p.parts) * K * sizeof(float);
}

template <int TPR, int P>
hipError_t bwd(const NormBwd& a, int64_t blocks, hipStream_t st) {
  hipLaunchKernelGGL((k_rms_bwd<TPR, P>), grid_of(blocks), dim3(row_threads<TPR>()), 0, st, a);
  return hipGetLastError();
}

}  // namespace

}  // namespace qnf4

using namespace qnf4;

extern "C" {

int qlora_rms_norm_fwd(const uint16_t* x, const uint16_t* residual, const void* g, int g_fp32,
                       int64_t M, int64_t K, float eps, uint16_t* h, uint16_t* y, float* rstd,
                       const qlora_act8* y8, qlora_stream_t stream) {
  const int st = check_norm(M, K);
  if (st) return st;
  if (!(eps > 0.f) || std::isinf(eps) || (y8 && K % kBlock != 0)) return QLORA_ERR_SHAPE;
  if (!g || (M > 0 && (!x || !y || !rstd || (residual && !h) ||
                       (y8 && (!y8->codes || !y8->scales)))))
    return QLORA_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(g) || !aligned16(h) || !aligned16(y) ||
      !aligned4(rstd) || (y8 && (!aligned16(y8->codes) || !aligned4(y8->scales))))
    return QLORA_ERR_ALIGN;
  if (M == 0) return QLORA_OK;
  const NormFwd a{x, residual, g, M, K, eps, h, y, rstd, y8 ? y8->codes : nullptr,
                  y8 ? y8->scales : nullptr, g_fp32 != 0};
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (K <= 512) fwd<64, 1>(a, hs);
  else if (K <= 1024) fwd<64, 2>(a, hs);
  else if (K <= 2048) fwd<256, 1>(a, hs);
  else if (K <= 4096) fwd<256, 2>(a, hs);
  else if (K <= 8192) fwd<256, 4>(a, hs);
  else if (K <= 16384) fwd<256, 8>(a, hs);
  else if (K <= 32768) fwd<1024, 4>(a, hs);
  else if (K <= kLongRow) fwd<1024, 8>(a, hs);
  else fwd<1024, 0>(a, hs);
  return hip_status(hipGetLastError());
}

size_t qlora_rms_norm_bwd_workspace_bytes(int64_t M, int64_t K) {
  if (check_norm(M, K) || M == 0) return 0;
  return bwd_need(plan_bwd(M, K, true), K);
}

int qlora_rms_norm_bwd(const uint16_t* dy, const uint16_t* dres, const uint16_t* h,
                       const float* rstd, const void* g, int g_fp32, int64_t M, int64_t K,
                       uint16_t* dx, void* dg, void* workspace, size_t workspace_bytes,
                       qlora_stream_t stream) {
  const int st = check_norm(M, K);
  if (st) return st;
  if (!g || (M > 0 && (!dy || !h || !rstd || !dx))) return QLORA_ERR_NULL;
  if (!aligned16(dy) || !aligned16(dres) || !aligned16(h) || !aligned4(rstd) || !aligned16(g) ||
      !aligned16(dx) || !aligned16(dg))
    return QLORA_ERR_ALIGN;
  const BwdPlan p = plan_bwd(M, K, dg != nullptr);
  const size_t need = bwd_need(p, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return QLORA_ERR_ALIGN;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  const int64_t cols = p.run_rows > 0 ? cdiv(K, 128) * std::max<int64_t>(1, p.parts) : 0;
  const NormBwd a{dy, dres, h, rstd, g, M, K, dx, dg,
                  p.parts > 0 ? static_cast<float*>(workspace) : nullptr, p.row_blocks, cols,
                  p.run_rows, g_fp32 != 0};
  const bool wide = K > kLongRowBwd;
  const int64_t n = p.row_blocks + (wide ? 0 : cols);
  hipError_t e = hipSuccess;
  if (n > 0) {
    if (K <= 512) e = bwd<64, 1>(a, n, hs);
    else if (K <= 1024) e = bwd<64, 2>(a, n, hs);
    else if (K <= 2048) e = bwd<256, 1>(a, n, hs);
    else if (K <= 4096) e = bwd<512, 1>(a, n, hs);
    else if (K <= 8192) e = bwd<1024, 1>(a, n, hs);
    else if (!wide) e = bwd<1024, 2>(a, n, hs);
    else e = bwd<1024, 0>(a, n, hs);
  }
  if (e == hipSuccess && wide && cols > 0) {
    hipLaunchKernelGGL(k_rms_dg_columns, grid_of(cols), dim3(256), 0, hs, a);
    e = hipGetLastError();
  }
  if (e == hipSuccess && p.parts > 0) {
    hipLaunchKernelGGL(k_rms_dg, dim3(static_cast<unsigned>(cdiv(K, 64))), dim3(1024), 0, hs,
                       a.part, p.parts, K, dg, g_fp32 != 0);
    e = hipGetLastError();
  }
  return hip_status(e);
}

}  // extern "C"
