// Host-callable launchers of the gfx950 kernels.  Every launcher enqueues on
// `stream`, allocates nothing and returns hipGetLastError() of its launches.
// Shapes are validated by the caller (the C ABI layer).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qnf4 {

struct Nf4Tables;

// dq: double-quantized constants (absmax_q [nb] bytes, absmax_scale one fp32
// per 256 blocks), else absmax_scale holds each block's fp32 absmax.
hipError_t launch_quantize(const float* W, int64_t N, int64_t K, uint8_t* codes,
                           uint8_t* absmax_q, float* absmax_scale,
                           const Nf4Tables& tb, hipStream_t stream, bool dq = true);

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* absmax_q,
                             const float* absmax_scale, int64_t N, int64_t K,
                             uint16_t* out, const Nf4Tables& tb, hipStream_t stream,
                             bool dq = true);

struct Nf4View {
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* absmax_scale;
  int64_t N, K;
  // When set, the GEMM launchers read this bf16 weight [N, K] instead of the
  // NF4 fields (the 16-bit LoRA baseline); N K 2 must stay below 2^31 bytes.
  const uint16_t* dense = nullptr;
  // false: fp32 block constants in absmax_scale [N K / 64], absmax_q unused.
  bool dq = true;
};

// Dropout of the adapter's input: the generator's state {seed, offset} in
// device memory and the threshold on its 16-bit values; thr = 0 drops nothing.
struct Drop {
  const uint64_t* state = nullptr;
  uint32_t thr = 0;
  bool on() const { return thr > 0; }
  float scale() const { return 65536.f / static_cast<float>(65536u - thr); }
};

// Activations [tokens, K] held as an 8-bit checkpoint (act8.hpp).  With an
// order, row i of the call's X is token order[i] / topk.
struct Act8View {
  const int8_t* codes;
  const float* scales;
  int64_t tokens;
  const int* order = nullptr;
  int topk = 1;
};

// Dynamic LDS past what a launch may use by default.  The limit belongs to a
// kernel on one device, so it is raised the first time a launcher runs with
// that device current (once each; a static of the launcher keeps the devices).
class LdsLimit {
 public:
  hipError_t raise(const void* kernel, int bytes) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;   // (no bit: each time)
    if (done_.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done_.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// Profiling hook: the launchers call these around the launches of one
// kernel family (no-ops unless profiling is enabled).
void prof_begin(int family, hipStream_t stream);
void prof_end(int family, hipStream_t stream);

// Split reduction of a dequantizing GEMM whose tiles would leave most of
// the CUs idle: `splits` workgroups per tile, each over `cps` consecutive
// chunks of the reduction, write fp32 partials that a second kernel adds up
// in split order (deterministic) and rounds to bf16.
struct GemmSplit {
  int splits, cps;
};
GemmSplit gemm_split(int64_t tiles, int64_t nchunks);
hipError_t launch_split_reduce_bf16(const float* part, int splits, int64_t count, uint16_t* out,
                                    hipStream_t stream, float scale = 1.f);

// Y[M,N] = bf16( X . deq(W)^T + s . T . B ), large-M MFMA path with the
// dequantized weight tiles staged in LDS.  T [M, r] fp32 (may be null when
// r == 0).  part: fwd_gemm_split(M, N, K).splits * M * N floats when that is
// above 1 (else unused).  Segments (seg_rows > 0, a multiple of 128): rows
// [j seg_rows, (j + 1) seg_rows) of W carry adapter j, whose T is columns
// [j r, (j + 1) r) of T (row stride ldt) and whose B is columns of the same
// rows of B [r, N]; by default one segment, ldt = r.
GemmSplit fwd_gemm_split(int64_t M, int64_t N, int64_t K);
hipError_t launch_fwd_gemm(const uint16_t* X, int64_t M, const Nf4View& w,
                           const float* T, const uint16_t* B, int r, float s,
                           uint16_t* Y, float* part, const Nf4Tables& tb, hipStream_t stream,
                           int ldt = 0, int64_t seg_rows = 0);

// Same result, small-M streaming path, for shapes with decode_fits(M, K).
// decode_folds_t(M, r): the kernel can add up T's partial sums itself.
bool decode_fits(int64_t M, int64_t K);
bool decode_folds_t(int64_t M, int r);
// With nz > 0, T holds nz partial sums [nz][M][r] of X . A which the kernel
// adds up itself (workgroup 0 also writes the total to Tout); with nz == 0, T
// is the final [M][r] with row stride ldt (default r) and Tout is unused.  B
// and Y have row strides ldb and ldy (default N).
hipError_t launch_fwd_decode(const uint16_t* X, int64_t M, const Nf4View& w,
                             const float* T, int nz, float* Tout, const uint16_t* B, int r,
                             float s, uint16_t* Y, const Nf4Tables& tb, hipStream_t stream,
                             int ldt = 0, int64_t ldb = 0, int64_t ldy = 0);

// dX[M,K] = bf16( dY . deq(W) + s . G . A^T ), MFMA path with the
// dequantized weight tiles staged in LDS and read back transposed.
GemmSplit dx_gemm_split(int64_t M, int64_t N, int64_t K);
hipError_t launch_dx_gemm(const uint16_t* dY, int64_t M, const Nf4View& w,
                          const float* G, const uint16_t* A, int r, float s,
                          uint16_t* dX, float* part, const Nf4Tables& tb, hipStream_t stream,
                          const Drop& d = {}, bool add_up = true);   // false: partials stay

// Rank-r products with a split reduction; partials go to `ws`.
size_t rank_ws_floats(int64_t M, int64_t N, int64_t K, int r);
// The partials of T = X . A alone (the forward's rank product).
size_t lora_down_ws_floats(int64_t M, int64_t K, int r);

// Few-token LoRA down-projection: nz <= maxp fp32 partial sums [nz][M][r]
// of T = X . A (with d on, scale . (mask X) . A) go to ws (nz returned);
// M <= 16, maxp <= kMaxDownPartials.
constexpr int kMaxDownPartials = 64;
int lora_down_partial_count(int64_t K, int maxp);
hipError_t launch_lora_down_partials(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A,
                                     int r, int maxp, float* ws, int* nz, hipStream_t stream,
                                     const Drop& d = {});

// T[M,r] = X . A (fp32 out); with d on, scale . (mask X) . A.
hipError_t launch_lora_down(const uint16_t* X, int64_t M, int64_t K,
                            const uint16_t* A, int r, float* T, float* ws,
                            hipStream_t stream, const Drop& d = {});
// G[M,r] = dY . B^T (fp32 out) and dB[r,N] = bf16( s . T^T . dY ), both
// products in one launch and both split reductions in one more.  Row strides
// (0 = dense): ldy of dY, ldb of B and of dB, ldt of T and of G.
hipError_t launch_grad_in_and_b(const uint16_t* dY, int64_t M, int64_t N, const uint16_t* B,
                                const float* T, int r, float s, float* G, uint16_t* dB,
                                float* ws, hipStream_t stream, int64_t ldy = 0, int64_t ldb = 0,
                                int ldt = 0);
// dA[K,r] = bf16( s . X^T . G ); with d on, bf16( s scale . (mask X)^T . G ).
hipError_t launch_grad_a(const uint16_t* X, int64_t M, int64_t K, const float* G,
                         int r, float s, uint16_t* dA, float* ws, hipStream_t stream,
                         const Drop& d = {});

// ---------------------------------------------------------------------------
// Layers grouped by expert: rows [offsets[e], offsets[e + 1]) of X belong to
// expert e (offsets int32 [E + 1] in device memory).  The weight view holds the
// E experts' weights of N = w.N / E rows one after the other, A is [E][K][r]
// and B [E][r][N].  Rows outside all groups are neither read nor written.
// ---------------------------------------------------------------------------

GemmSplit grouped_fwd_split(int64_t M, int E, int64_t N, int64_t K);
GemmSplit grouped_dx_split(int64_t M, int E, int64_t N, int64_t K);
// T is final (nz = 0), or nz partial sums [nz][M][r] that the kernel adds up,
// scales by tscale and writes to Tout (grouped_fwd_folds_t: with few rows).
bool grouped_fwd_folds_t(int64_t M);
hipError_t launch_grouped_fwd_gemm(const uint16_t* X, int64_t M, const int* offsets, int E,
                                   const Nf4View& w, const float* T, int nz, float tscale,
                                   float* Tout, const uint16_t* B, int r, float s, uint16_t* Y,
                                   float* part, const Nf4Tables& tb, hipStream_t stream);
hipError_t launch_grouped_dx_gemm(const uint16_t* dY, int64_t M, const int* offsets, int E,
                                  const Nf4View& w, const float* G, const uint16_t* A, int r,
                                  float s, uint16_t* dX, float* part, const Nf4Tables& tb,
                                  hipStream_t stream, const Drop& d);
// Threads of the largest launch: of the forward GEMM, of dX and of the rank products.
int64_t grouped_fwd_threads(int64_t M, int E, int64_t N, int64_t K);
int64_t grouped_dx_threads(int64_t M, int E, int64_t N, int64_t K);
int64_t grouped_rank_threads(int64_t M, int E, int64_t N, int64_t K, int r);
// out[m][i] = scale * sum_z part[z][m][i] for the rows of the groups; exactly
// one of f32 and bf16 is the output.
hipError_t launch_group_reduce(const float* part, int splits, int64_t M, int64_t cols, float scale,
                               const int* offsets, int E, float* f32, uint16_t* bf16,
                               hipStream_t stream);
// Floats of workspace of the four rank products, and those of T alone.
size_t grouped_rank_ws_floats(int64_t M, int E, int64_t N, int64_t K, int r);
size_t grouped_down_ws_floats(int64_t M, int E, int64_t K, int r);
// T = scale . (mask X) . A_e.  With nz, a split product's partial sums stay in
// ws and *nz is their number (0: T is final).
hipError_t launch_grouped_down(const uint16_t* X, int64_t M, const int* offsets, int E, int64_t K,
                               const uint16_t* A, int r, float* T, float* ws, hipStream_t stream,
                               const Drop& d, int* nz = nullptr);
hipError_t launch_grouped_grad_in_and_b(const uint16_t* dY, int64_t M, const int* offsets, int E,
                                        int64_t N, const uint16_t* B, const float* T, int r,
                                        float s, float* G, uint16_t* dB, float* ws,
                                        hipStream_t stream);
hipError_t launch_grouped_grad_a(const uint16_t* X, int64_t M, const int* offsets, int E,
                                 int64_t K, const float* G, int r, float s, uint16_t* dA,
                                 float* ws, hipStream_t stream, const Drop& d);

// T and dA with X held as an 8-bit checkpoint: as launch_lora_down and
// launch_grad_a (workspace of rank_ws_floats), and as the grouped ones above.
hipError_t launch_lora_down_act8(const Act8View& x8, int64_t M, int64_t K, const uint16_t* A,
                                 int r, float* T, float* ws, hipStream_t stream, const Drop& d);
hipError_t launch_grad_a_act8(const Act8View& x8, int64_t M, int64_t K, const float* G, int r,
                              float s, uint16_t* dA, float* ws, hipStream_t stream,
                              const Drop& d);
// With grad_a_act8_whole (dA in one split), dA and the sum of dX's partials
// (part [splits][count]) in one launch.
bool grad_a_act8_whole(int64_t M, int64_t K, int r);
hipError_t launch_grad_a_act8_and_sum(const Act8View& x8, int64_t M, int64_t K, const float* G,
                                      int r, float s, uint16_t* dA, const float* part, int splits,
                                      int64_t count, uint16_t* dX, hipStream_t stream,
                                      const Drop& d);
hipError_t launch_grouped_down_act8(const Act8View& x8, int64_t M, const int* offsets, int E,
                                    int64_t K, const uint16_t* A, int r, float* T, float* ws,
                                    hipStream_t stream, const Drop& d);
int64_t grouped_grad_a_act8_threads(int64_t M, int E, int64_t K, int r);
hipError_t launch_grouped_grad_a_act8(const Act8View& x8, int64_t M, const int* offsets, int E,
                                      int64_t K, const float* G, int r, float s, uint16_t* dA,
                                      float* ws, hipStream_t stream, const Drop& d);

// n bf16 values (n % 64 == 0, rows of whole blocks) to codes and constants, and back.
hipError_t launch_act8_pack(const uint16_t* x, int64_t n, int8_t* codes, float* scales,
                            hipStream_t stream);
hipError_t launch_act8_unpack(const int8_t* codes, const float* scales, int64_t n, uint16_t* x,
                              hipStream_t stream);

// y[i] = mask scale x[i] (bf16, n elements; y may be x).
hipError_t launch_dropout(const uint16_t* x, int64_t n, const Drop& d, uint16_t* y,
                          hipStream_t stream);

// One AdamW step over n parameters (bf16 p, g; fp32 m, v, device or
// device-visible pinned host memory, 16-byte aligned), bias corrections for
// step `step` (>= 1).
hipError_t launch_adamw(uint16_t* p, const uint16_t* g, float* m, float* v, int64_t n,
                        float lr, float beta1, float beta2, float eps, float weight_decay,
                        int64_t step, hipStream_t stream);

}  // namespace qnf4
