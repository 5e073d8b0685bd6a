// MFMA GEMMs of the QLoRA NF4 linear layer on gfx950.
//
// The rank-r products (T = X.A, G = dY.B^T, dA, dB) have the form C[q, p] = sum_k P[p, k] . Q[q, k]: the
// workgroup stages a P tile (BP rows x 64 reduction elements) and a Q tile
// (BQ x 64) in LDS, and four waves (2 x 2) accumulate their (BP/2 x BQ/2)
// share with v_mfma_f32_16x16x32_bf16.  Each loader fixes its tile's LDS
// layout and how a lane reads its 8 reduction elements from it:
//   Bf16Nat  bf16 rows, reduction contiguous (X and dY of T and G, B as [r,N])
//   Bf16RedMajor / F32RedMajor  reduction-major tiles kept as they lie in
//            memory and read with transposing LDS reads (A as [K,r]; X, dY,
//            G, T of dA and dB); fp32 sources are split into bf16 hi and lo
//            passes, so the fp32 factor keeps ~16 bits through the bf16 MFMA
// The weight-streaming GEMMs (forward and dX) have kernels of their own.
#include <type_traits>

#include "device_common.hpp"
#include "kernels.hpp"
#include "rank_tiles.hpp"

namespace qnf4 {

// ---------------------------------------------------------------------------
// Rank-r products with a split reduction: partial sums of C[q, p] for
// reduction tiles [z*tps, (z+1)*tps) go to ws[z][q][p]; a second kernel sums
// the partials in split order (deterministic) and writes the result.
// ---------------------------------------------------------------------------

// HL: 0 = both operands bf16; 1 = P is fp32 (hi/lo); 2 = Q is fp32 (hi/lo).
template <int BP, int BQ, class LP, class LQ, int HL>
struct RankKind {
  static constexpr int XT = HL == 0 ? 0 : (HL == 1 ? LP::TILE : LQ::TILE);
  static constexpr int LDS = 2 * (LP::TILE + LQ::TILE + XT);   // bf16 elements
};

// One product: tile (x, y) of C and reduction split z.
struct RankJob {
  OpParams po, qo;
  int ntiles, tps;
  float* ws;
  int64_t P, Q;
  int px, qy, nblk;   // tiles along P and Q; workgroups (px qy splits)
  const uint64_t* state;   // Q under the dropout mask: the generator's state
  uint32_t thr;            // and threshold
};

template <int BP, int BQ, class LP, class LQ, int HL>
__device__ __forceinline__ void rank_tile(const RankJob& j, int x, int y, int z, uint16_t* lds,
                                          int tid) {
  const int64_t p0 = (int64_t)x * BP, q0 = (int64_t)y * BQ;
  const int kt0 = z * j.tps, kt1 = min(j.ntiles, kt0 + j.tps);
  Mma<BP, BQ> mma;
  mma.zero();
  LP lp{j.po, p0};
  LQ lq{j.qo, q0};
  if constexpr (LQ::kDrop) lq.key = load_drop_key(j.state, j.thr);
  run_tiles<BP, BQ, HL, 2>(lp, lq, kt0, kt1, mma, lds, tid);
  store_f32(mma, j.ws + (int64_t)z * j.P * j.Q, j.P, p0, q0, j.P, j.Q, tid);
}

template <int BP, int BQ, class LP, class LQ, int HL>
__global__ __launch_bounds__(NT) void k_rank(RankJob j) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[RankKind<BP, BQ, LP, LQ, HL>::LDS];
  // (the long axis along x: y and z take 65536 workgroups only; all three in x cost
  // two divisions and 0.3 us a launch)
  rank_tile<BP, BQ, LP, LQ, HL>(j, blockIdx.y, blockIdx.x, blockIdx.z, lds, threadIdx.x);
}

// Two independent products in one launch (workgroups [0, a.nblk) run the
// first, the rest the second), so they share the machine instead of running
// one after the other.
template <int BPA, int BQA, class LPA, class LQA, int HLA, int BPB, int BQB, class LPB, class LQB,
          int HLB>
__global__ __launch_bounds__(NT) void k_rank_pair(RankJob a, RankJob b) {
  constexpr int LA = RankKind<BPA, BQA, LPA, LQA, HLA>::LDS;
  constexpr int LB = RankKind<BPB, BQB, LPB, LQB, HLB>::LDS;
  __shared__ __attribute__((aligned(16))) uint16_t lds[LA > LB ? LA : LB];
  int blk = blockIdx.x;   // uniform: the branch is a scalar one
  if (blk < a.nblk) {
    rank_tile<BPA, BQA, LPA, LQA, HLA>(a, blk % a.px, (blk / a.px) % a.qy, blk / (a.px * a.qy),
                                       lds, threadIdx.x);
  } else {
    blk -= a.nblk;
    rank_tile<BPB, BQB, LPB, LQB, HLB>(b, blk % b.px, (blk / b.px) % b.qy, blk / (b.px * b.qy),
                                       lds, threadIdx.x);
  }
}

// out[i] = scale * sum_z ws[z][i]; fp32 or bf16 output; 4 elements a thread.
template <bool BF16_OUT>
__global__ __launch_bounds__(256) void k_split_reduce(const float* ws, int splits,
                                                      int64_t count, float scale,
                                                      void* out) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= count) return;
  // four independent partial sums so the loads of several splits overlap;
  // the combination order is fixed, so results are deterministic
  f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0, s2 = s0, s3 = s0;
  int z = 0;
  for (; z + 4 <= splits; z += 4) {
    s0 += *reinterpret_cast<const f32x4*>(ws + (int64_t)(z + 0) * count + i);
    s1 += *reinterpret_cast<const f32x4*>(ws + (int64_t)(z + 1) * count + i);
    s2 += *reinterpret_cast<const f32x4*>(ws + (int64_t)(z + 2) * count + i);
    s3 += *reinterpret_cast<const f32x4*>(ws + (int64_t)(z + 3) * count + i);
  }
  for (; z < splits; ++z) s0 += *reinterpret_cast<const f32x4*>(ws + (int64_t)z * count + i);
  f32x4 s = (s0 + s1) + (s2 + s3);
  s *= scale;
  if constexpr (BF16_OUT) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) =
        u32x2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = s;
  }
}

// Two split reductions in one launch: blocks [0, ga) reduce the first.
struct ReduceJob {
  const float* ws;
  int splits;
  int64_t count;
  float scale;
  void* out;
  int64_t prow;   // elements per output row (a multiple of 4)
  int64_t ldo;    // output row stride (prow for a dense output)
};

template <bool BF16_A, bool BF16_B>
__global__ __launch_bounds__(256) void k_split_reduce_pair(ReduceJob a, ReduceJob b, int ga) {
  const bool first = static_cast<int>(blockIdx.x) < ga;
  const ReduceJob& j = first ? a : b;
  const int64_t i = 4 * ((int64_t)(first ? blockIdx.x : blockIdx.x - ga) * blockDim.x + threadIdx.x);
  if (i >= j.count) return;
  f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0, s2 = s0, s3 = s0;
  int z = 0;
  for (; z + 4 <= j.splits; z += 4) {
    s0 += *reinterpret_cast<const f32x4*>(j.ws + (int64_t)(z + 0) * j.count + i);
    s1 += *reinterpret_cast<const f32x4*>(j.ws + (int64_t)(z + 1) * j.count + i);
    s2 += *reinterpret_cast<const f32x4*>(j.ws + (int64_t)(z + 2) * j.count + i);
    s3 += *reinterpret_cast<const f32x4*>(j.ws + (int64_t)(z + 3) * j.count + i);
  }
  for (; z < j.splits; ++z) s0 += *reinterpret_cast<const f32x4*>(j.ws + (int64_t)z * j.count + i);
  f32x4 s = (s0 + s1) + (s2 + s3);
  s *= j.scale;
  const int64_t row = i / j.prow, o = row * j.ldo + (i - row * j.prow);
  if (first ? BF16_A : BF16_B) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(j.out) + o) =
        u32x2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(j.out) + o) = s;
  }
}

// ---------------------------------------------------------------------------
// LoRA down-projection for few tokens (M <= 16): workgroup z covers spw
// consecutive slices of 128 k; partial[z][m][j] = sum over them of
// X[m, k] A[k, j].  Each A slice is transposed through LDS in 8x8 patches
// (16 KB a slice, staged by the first 128 threads), 64 ranks at a time; wave
// w multiplies ranks 16w..16w+15 of the 64 against the token fragments,
// which come straight from global memory.  128-k slices give 64 workgroups
// at K = 8192 where 256-k slices gave 32; the kernel is a short latency
// chain, so more of them in parallel end sooner (about 0.3 us per call).
// ---------------------------------------------------------------------------

constexpr int LDS_K = 128;             // k per slice
constexpr int LDS_KS = LDS_K + 8;      // LDS row stride (elements)

// With DROP, X is under the dropout mask: a lane forms the masks of the pieces
// it multiplies while they are on their way, and the sums are scaled.
template <bool DROP>
__global__ __launch_bounds__(256) void k_lora_down_small(const uint16_t* __restrict__ X, int M,
                                                         int64_t K, const uint16_t* __restrict__ A,
                                                         int r, int spw, float* __restrict__ ws,
                                                         const uint64_t* __restrict__ state,
                                                         uint32_t thr, float scale) {
  __shared__ __attribute__((aligned(16))) uint16_t at[64 * LDS_KS];
  const int tid = threadIdx.x;
  const int wave = wave_id(), lane = tid & 63;
  const int li = lane & 15, g = lane >> 4;
  const bool m_ok = li < M;
  const int jp = tid & 7, kp = tid >> 3;   // A patch: ranks j0 + 8 jp .., k rows 8 kp ..
  const int K32 = static_cast<int>(K);     // K <= 2^22 and M K, K r < 2^30 here
  const BufRes rx = make_bufres(X, static_cast<uint32_t>(M * K32 * 2));
  const BufRes ra = make_bufres(A, static_cast<uint32_t>(K32 * r * 2));
  // Slices run as a two-stage pipeline: the loads of slice sub + 1 are in
  // flight while slice sub is transposed and multiplied.
  u32x4 xf[2][LDS_K / 32];   // token fragments for the k32 steps of a slice
  DropKey key{};
  if constexpr (DROP) key = load_drop_key(state, thr);
  u32x4 rows[2][8];   // this thread's 8x8 patch of the slice's A rows
  for (int j0 = 0; j0 < r; j0 += 64) {
    // (buffer loads with out-of-range offsets instead of branches, so the
    // compiler can wait for one stage while the other is in flight)
    auto load = [&](int sub, int b) {   // past the workgroup's slices: reads nothing
      const int k0 = sub < spw ? (blockIdx.x * spw + sub) * LDS_K : K32;
#pragma unroll
      for (int st = 0; st < LDS_K / 32; ++st) {
        const int k = k0 + 32 * st + 8 * g;
        xf[b][st] = buf_load16(rx, m_ok && k < K ? static_cast<uint32_t>((li * K32 + k) * 2)
                                                 : 0x80000000u);
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int k = k0 + kp * 8 + t;
        const int j = j0 + jp * 8;
        const bool ok = kp * 8 < LDS_K && k < K && j < r;   // 16 threads of rows a slice
        rows[b][t] = buf_load16(ra, ok ? static_cast<uint32_t>((k * r + j) * 2) : 0x80000000u);
      }
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](int sub, auto bc) {
      constexpr int b = decltype(bc)::value;
      if (sub >= spw) return;   // uniform
      load(sub + 1, b ^ 1);
      u32x4 cols[8];
      transpose8x8_b16(rows[b], cols);
      if (kp * 8 < LDS_K) {   // threads past the slice's rows hold zeros
#pragma unroll
        for (int t = 0; t < 8; ++t)
          *reinterpret_cast<u32x4*>(at + (jp * 8 + t) * LDS_KS + kp * 8) = cols[t];
      }
      __syncthreads();
#pragma unroll
      for (int st = 0; st < LDS_K / 32; ++st) {
        const u32x4 af =
            *reinterpret_cast<const u32x4*>(at + (16 * wave + li) * LDS_KS + 32 * st + 8 * g);
        u32x4 x = xf[b][st];
        if constexpr (DROP) {
          const int k = (blockIdx.x * spw + sub) * LDS_K + 32 * st + 8 * g;
          x &= keep_piece(key, static_cast<uint64_t>(li * K + k) / 8);
        }
        acc = mfma16(af, x, acc);
      }
      __syncthreads();
    };
    load(0, 0);
    for (int sub = 0; sub < spw; sub += 2) {
      step(sub, std::integral_constant<int, 0>{});
      step(sub + 1, std::integral_constant<int, 1>{});
    }
    const int j = j0 + 16 * wave + 4 * g;
    if constexpr (DROP) acc *= scale;
    if (m_ok && j < r)
      *reinterpret_cast<f32x4*>(ws + ((int64_t)blockIdx.x * M + li) * r + j) = acc;
  }
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------

namespace {

OpParams op(const void* p, int64_t ld, int64_t nrows, int64_t nred, float scale = 1.f) {
  OpParams o{};
  o.ptr = p;
  o.ld = ld;
  o.nrows = nrows;
  o.nred = nred;
  o.scale = scale;
  o.drow0 = 0;
  return o;
}

unsigned cdiv(int64_t a, int64_t b) { return static_cast<unsigned>((a + b - 1) / b); }

struct Split {
  int ntiles, tps, splits;
};

// Split the reduction so that the grid has about one workgroup per CU, with
// at least four reduction tiles per split (fewer, larger splits keep the fp32
// partial sums small next to the operands they reduce).
Split choose_split(int64_t nred, int64_t ptiles, int64_t qtiles) {
  Split s;
  s.ntiles = static_cast<int>((nred + BK - 1) / BK);
  const int64_t want = std::max<int64_t>(1, 256 / std::max<int64_t>(1, ptiles * qtiles));
  s.tps = static_cast<int>(std::max<int64_t>(4, (s.ntiles + want - 1) / want));
  s.splits = (s.ntiles + s.tps - 1) / s.tps;
  return s;
}

RankJob job(const OpParams& po, const OpParams& qo, const Split& sp, float* ws, int64_t P,
            int64_t Q, int64_t px, int64_t qy, const Drop& d = {}) {
  RankJob j;
  j.po = po;
  j.qo = qo;
  j.ntiles = sp.ntiles;
  j.tps = sp.tps;
  j.ws = ws;
  j.P = P;
  j.Q = Q;
  j.px = static_cast<int>(px);
  j.qy = static_cast<int>(qy);
  j.nblk = static_cast<int>(px * qy * sp.splits);
  j.state = d.state;
  j.thr = d.thr;
  return j;
}

template <bool BF16>
hipError_t reduce(const float* ws, int splits, int64_t count, float scale, void* out,
                  hipStream_t stream) {
  const unsigned grid = cdiv(count / 4, 256);
  hipLaunchKernelGGL(k_split_reduce<BF16>, dim3(grid), dim3(256), 0, stream, ws, splits,
                     count, scale, out);
  return hipGetLastError();
}

constexpr int RB_R = 64;     // tile of the rank dimension
constexpr int RB_X = 128;    // tile of the long dimension

}  // namespace

GemmSplit gemm_split(int64_t tiles, int64_t nchunks) {
  GemmSplit g{1, static_cast<int>(nchunks)};
  // Only when the tiles would fill under three quarters of the 256 CUs, and
  // with at least 8 chunks per split (the partials cost a pass of their own).
  if (tiles >= 192 || nchunks < 16) return g;
  const int64_t want = std::min<int64_t>(256 / tiles, nchunks / 8);
  if (want < 2) return g;
  int64_t cps = (nchunks + want - 1) / want;
  cps += cps & 1;   // whole pairs of chunks
  g.splits = static_cast<int>((nchunks + cps - 1) / cps);
  g.cps = static_cast<int>(cps);
  return g;
}

hipError_t launch_split_reduce_bf16(const float* part, int splits, int64_t count, uint16_t* out,
                                    hipStream_t stream, float scale) {
  return reduce<true>(part, splits, count, scale, out, stream);
}

size_t rank_ws_floats(int64_t M, int64_t N, int64_t K, int r) {
  if (r <= 0) return 0;
  if (M <= 16)
    return (size_t)lora_down_partial_count(K, kMaxDownPartials) * M * r +
           rank_ws_floats(17, N, K, r);
  const int64_t rt = (r + RB_R - 1) / RB_R;
  const Split t = choose_split(K, rt, (M + RB_X - 1) / RB_X);
  const Split g = choose_split(N, rt, (M + RB_X - 1) / RB_X);
  const Split a = choose_split(M, rt, (K + RB_X - 1) / RB_X);
  const Split b = choose_split(M, (N + RB_X - 1) / RB_X, rt);
  size_t m = 0;
  m = std::max<size_t>(m, (size_t)t.splits * M * r);
  m = std::max<size_t>(m, (size_t)g.splits * M * r + (size_t)b.splits * r * N);   // together
  m = std::max<size_t>(m, (size_t)a.splits * K * r);
  return m;
}

size_t lora_down_ws_floats(int64_t M, int64_t K, int r) {
  if (r <= 0) return 0;
  if (M <= 16) return (size_t)lora_down_partial_count(K, kMaxDownPartials) * M * r;
  const Split t = choose_split(K, (r + RB_R - 1) / RB_R, (M + RB_X - 1) / RB_X);
  return (size_t)t.splits * M * r;
}

int lora_down_partial_count(int64_t K, int maxp) {
  const int64_t slices = (K + LDS_K - 1) / LDS_K;
  const int64_t spw = (slices + maxp - 1) / maxp;
  return static_cast<int>((slices + spw - 1) / spw);
}

hipError_t launch_lora_down_partials(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A,
                                     int r, int maxp, float* ws, int* nz, hipStream_t stream,
                                     const Drop& d) {
  if (maxp < 1 || maxp > kMaxDownPartials) return hipErrorInvalidValue;
  const int64_t slices = (K + LDS_K - 1) / LDS_K;
  const int spw = static_cast<int>((slices + maxp - 1) / maxp);
  *nz = lora_down_partial_count(K, maxp);
  prof_begin(4, stream);
  hipLaunchKernelGGL(d.on() ? k_lora_down_small<true> : k_lora_down_small<false>, dim3(*nz),
                     dim3(256), 0, stream, X, (int)M, K, A, r, spw, ws, d.state, d.thr, d.scale());
  prof_end(4, stream);
  return hipGetLastError();
}

hipError_t launch_lora_down(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A,
                            int r, float* T, float* ws, hipStream_t stream, const Drop& d) {
  if (M <= 16) {
    int nz = 0;
    hipError_t e =
        launch_lora_down_partials(X, M, K, A, r, kMaxDownPartials / 2, ws, &nz, stream, d);
    if (e == hipSuccess) {
      prof_begin(4, stream);
      e = reduce<false>(ws, nz, M * r, 1.f, T, stream);
      prof_end(4, stream);
    }
    return e;
  }
  const int64_t pt = (r + RB_R - 1) / RB_R, qt = (M + RB_X - 1) / RB_X;
  const Split sp = choose_split(K, pt, qt);
  auto kern = d.on() ? k_rank<RB_R, RB_X, Bf16RedMajor<RB_R>, Bf16Nat<RB_X, true>, 0>
                     : k_rank<RB_R, RB_X, Bf16RedMajor<RB_R>, Bf16Nat<RB_X>, 0>;
  prof_begin(4, stream);
  hipLaunchKernelGGL(kern, dim3(qt, pt, sp.splits), dim3(NT), 0, stream,
                     job(op(A, r, r, K), op(X, K, M, K), sp, ws, r, M, pt, qt, d));
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = reduce<false>(ws, sp.splits, M * r, d.scale(), T, stream);
  prof_end(4, stream);
  return e;
}

hipError_t launch_grad_in_and_b(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* B,
                                const float* T, int r, float s, float* G, uint16_t* dB,
                                float* ws, hipStream_t stream, int64_t ldy, int64_t ldb,
                                int ldt) {
  if (ldy <= 0) ldy = N;
  if (ldb <= 0) ldb = N;
  if (ldt <= 0) ldt = r;
  // G = dY . B^T: tiles (ranks, tokens), split over N
  const int64_t gpt = (r + RB_R - 1) / RB_R, gqt = (M + RB_X - 1) / RB_X;
  const Split gs = choose_split(N, gpt, gqt);
  // dB partials: tiles (N, ranks), split over M; after G's partials in ws
  const int64_t bpt = (N + RB_X - 1) / RB_X, bqt = (r + RB_R - 1) / RB_R;
  const Split bs = choose_split(M, bpt, bqt);
  float* wsb = ws + (size_t)gs.splits * M * r;
  const RankJob jg = job(op(B, ldb, r, N), op(dY, ldy, M, N), gs, ws, r, M, gpt, gqt);
  const RankJob jb = job(op(dY, ldy, N, M), op(T, ldt, r, M), bs, wsb, N, r, bpt, bqt);
  prof_begin(4, stream);
  hipLaunchKernelGGL((k_rank_pair<RB_R, RB_X, Bf16Nat<RB_R>, Bf16Nat<RB_X>, 0, RB_X, RB_R,
                                  Bf16RedMajor<RB_X>, F32RedMajor<RB_R>, 2>),
                     dim3(jg.nblk + jb.nblk), dim3(NT), 0, stream, jg, jb);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) {
    const ReduceJob rg{ws, gs.splits, M * r, 1.f, G, r, ldt};
    const ReduceJob rb{wsb, bs.splits, r * N, s, dB, N, ldb};
    const unsigned ga = cdiv(rg.count / 4, 256), gb = cdiv(rb.count / 4, 256);
    hipLaunchKernelGGL((k_split_reduce_pair<false, true>), dim3(ga + gb), dim3(256), 0, stream,
                       rg, rb, static_cast<int>(ga));
    e = hipGetLastError();
  }
  prof_end(4, stream);
  return e;
}

hipError_t launch_grad_a(const uint16_t* X, int64_t M, int64_t K, const float* G,
                         int r, float s, uint16_t* dA, float* ws, hipStream_t stream,
                         const Drop& d) {
  const int64_t pt = (r + RB_R - 1) / RB_R, qt = (K + RB_X - 1) / RB_X;
  const Split sp = choose_split(M, pt, qt);
  auto kern = d.on() ? k_rank<RB_R, RB_X, F32RedMajor<RB_R>, Bf16RedMajor<RB_X, true>, 1>
                     : k_rank<RB_R, RB_X, F32RedMajor<RB_R>, Bf16RedMajor<RB_X>, 1>;
  prof_begin(4, stream);
  hipLaunchKernelGGL(kern, dim3(qt, pt, sp.splits), dim3(NT), 0, stream,
                     job(op(G, r, r, M), op(X, K, K, M), sp, ws, r, K, pt, qt, d));
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = reduce<true>(ws, sp.splits, K * r, s * d.scale(), dA, stream);
  prof_end(4, stream);
  return e;
}

}  // namespace qnf4
