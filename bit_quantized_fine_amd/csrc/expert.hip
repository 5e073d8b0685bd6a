// The exchange around a layer grouped by expert: slots (token, choice) sorted
// by expert on the GPU, token rows copied into expert order, expert rows
// summed back into token order with the router's weights, and the gradients of
// that sum.
//
// Plan.  A stable counting sort.  The slots are cut into at most kMaxBlocks
// blocks; with more than one, a first launch counts each block's slots per
// expert.  In the placing launch every block adds up the counts of all blocks
// (and of those before it), scans them over the experts, and ranks its own
// slots 1024 at a time: inside a wave the lanes with the same expert find each
// other by one ballot per bit of the expert's number, the waves' counts meet in
// LDS.  Slots with an id outside 0 .. E - 1 get no row.
//
// Rows.  One workgroup per token: the token's row is read once and written to
// the rows of its slots, or the rows of its slots are read once and summed in
// choice order, so results do not depend on the order of anything.  These
// kernels are bound by the bytes they move: 8192 tokens of 4096 columns with 4
// choices each take 60 us out (336 MB, 5.6 TB/s), 55 us back (6.1 TB/s) and 128 us
// in the sum's backward (604 MB, 4.7 TB/s), where a large copy reaches 5.0 TB/s;
// their plan takes 5 + 5 us.
#include <algorithm>

#include "device_common.hpp"
#include "kernels.hpp"
#include "qlora_nf4.h"

namespace qnf4 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kMaxBlocks = 128;
constexpr int kMaxE = 1024;

// Slots of one block (a multiple of kPlanThreads) and the number of blocks.
int64_t plan_chunk(int64_t n) {
  const int64_t per = (n + kMaxBlocks - 1) / kMaxBlocks;
  return std::max<int64_t>(kPlanThreads, (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads);
}
int plan_blocks(int64_t n) {
  return static_cast<int>(std::max<int64_t>(1, (n + plan_chunk(n) - 1) / plan_chunk(n)));
}

constexpr int kRowThreads = 256;
constexpr int kMaxTopk = 64;
// A launch holds fewer than 2^32 threads along x: the tokens' workgroups lie in rows
// of kRowBlocks along y.  (Workgroups that stride over the tokens instead took 0.5%
// longer for 8192 tokens, there and back with the gradients.)
constexpr int64_t kRowBlocks = int64_t(1) << 23;

}  // namespace

// counts[b][e] = slots of block b with expert e
__global__ __launch_bounds__(kPlanThreads) void k_plan_count(const int* __restrict__ ids,
                                                             int64_t n, int E, int64_t chunk,
                                                             int* __restrict__ counts) {
  __shared__ int hist[kMaxE];
  const int tid = threadIdx.x;
  if (tid < E) hist[tid] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * chunk;
  for (int64_t i = tid; i < chunk && s0 + i < n; i += kPlanThreads) {
    const int e = ids[s0 + i];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  if (tid < E) counts[(int64_t)blockIdx.x * E + tid] = hist[tid];
}

// counts: [gridDim.x][E], or null with a single block, which counts its slots
// itself.
__global__ __launch_bounds__(kPlanThreads) void k_plan_place(
    const int* __restrict__ ids, int64_t n, int E, int64_t chunk, const int* __restrict__ counts,
    int* __restrict__ offsets, int* __restrict__ order, int* __restrict__ inverse) {
  __shared__ int total[kMaxE];    // of all blocks, then the block's next row of each expert
  __shared__ int before[kMaxE];   // of the blocks before this one
  __shared__ int wsum[kPlanWaves + 1];
  extern __shared__ int wcnt[];   // [kPlanWaves][E]
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t s0 = (int64_t)blockIdx.x * chunk;
  total[tid] = 0;
  before[tid] = 0;
  for (int i = tid; i < kPlanWaves * E; i += kPlanThreads) wcnt[i] = 0;
  __syncthreads();
  if (counts) {
    const int cells = static_cast<int>(gridDim.x) * E;
    for (int i = tid; i < cells; i += kPlanThreads) {
      const int b = i / E, e = i - b * E, c = counts[i];
      if (c) {
        atomicAdd(&total[e], c);
        if (b < static_cast<int>(blockIdx.x)) atomicAdd(&before[e], c);
      }
    }
  } else {
    for (int64_t i = tid; i < n; i += kPlanThreads) {
      const int e = ids[i];
      if (e >= 0 && e < E) atomicAdd(&total[e], 1);
    }
  }
  __syncthreads();
  // exclusive scan of the totals over the experts (one a thread)
  const int mine = total[tid];
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  if (tid == 0) {
    int run = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int v = wsum[w];
      wsum[w] = run;
      run += v;
    }
    wsum[kPlanWaves] = run;
  }
  __syncthreads();
  const int first = wsum[wave] + incl - mine;
  const int kept = wsum[kPlanWaves];
  total[tid] = first + before[tid];
  if (blockIdx.x == 0) {
    if (tid < E) offsets[tid] = first;
    if (tid == 0) offsets[E] = kept;
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(E);   // of the numbers 0 .. E
  for (int64_t i0 = 0; i0 < chunk && s0 + i0 < n; i0 += kPlanThreads) {
    const int64_t slot = s0 + i0 + tid;
    const bool in = slot < n;
    int e = in ? ids[slot] : E;
    if (e < 0 || e > E) e = E;   // no row
    unsigned long long peers = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      peers &= ((e >> b) & 1) ? m : ~m;
    }
    const unsigned long long lower = peers & ((1ull << lane) - 1);
    if (e < E && lower == 0) wcnt[wave * E + e] = __builtin_popcountll(peers);
    __syncthreads();
    if (in) {
      int row = -1;
      if (e < E) {
        row = total[e] + __builtin_popcountll(lower);
        for (int w = 0; w < wave; ++w) row += wcnt[w * E + e];
        order[row] = static_cast<int>(slot);
      }
      inverse[slot] = row;
      if (slot >= kept) order[slot] = -1;   // rows behind the last group
    }
    __syncthreads();
    if (tid < E) {
      int c = 0;
      for (int w = 0; w < kPlanWaves; ++w) {
        c += wcnt[w * E + tid];
        wcnt[w * E + tid] = 0;
      }
      total[tid] += c;
    }
    __syncthreads();
  }
}

// The workgroup's token, `tokens` or more: none.
__device__ __forceinline__ int64_t row_token() {
  return (int64_t)blockIdx.y * kRowBlocks + blockIdx.x;
}

// Xs[inverse[t][j]] = X[t]
__global__ __launch_bounds__(kRowThreads) void k_expert_gather(const uint16_t* __restrict__ X,
                                                               int64_t tokens, int topk, int64_t K,
                                                               const int* __restrict__ inverse,
                                                               uint16_t* __restrict__ Xs) {
  const int64_t t = row_token(), n = tokens * topk;
  if (t >= tokens) return;
  for (int64_t c = 8 * threadIdx.x; c < K; c += 8 * kRowThreads) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(X + t * K + c);
    for (int j = 0; j < topk; ++j) {
      const int64_t row = inverse[t * topk + j];
      if (row >= 0 && row < n) *reinterpret_cast<u32x4*>(Xs + row * K + c) = v;
    }
  }
}

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    f[2 * i] = bf16_lo_to_f32(w);
    f[2 * i + 1] = bf16_hi_to_f32(w);
  }
}
__device__ __forceinline__ u32x4 pack8(const float* f) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
               pack_bf16x2(f[6], f[7])};
}

// out[t] = sum_j w[t][j] Y[inverse[t][j]], in fp32, rounded once
__global__ __launch_bounds__(kRowThreads) void k_expert_combine(
    const uint16_t* __restrict__ Y, int64_t tokens, int topk, int64_t K,
    const int* __restrict__ inverse, const float* __restrict__ weights,
    uint16_t* __restrict__ out) {
  const int64_t t = row_token(), n = tokens * topk;
  if (t >= tokens) return;
  for (int64_t c = 8 * threadIdx.x; c < K; c += 8 * kRowThreads) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < topk; j0 += 4) {   // four rows' loads in flight
      u32x4 v[4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i;
        const int64_t row = j < topk ? inverse[t * topk + j] : -1;
        const bool in = row >= 0 && row < n;   // a slot without a row adds 0 times 0
        v[i] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(Y + row * K + c))
                  : u32x4{0, 0, 0, 0};
        w[i] = !in ? 0.f : (weights ? weights[t * topk + j] : 1.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[8];
        unpack8(v[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[i], y[k], acc[k]);
      }
    }
    *reinterpret_cast<u32x4*>(out + t * K + c) = pack8(acc);
  }
}

// dY[inverse[t][j]] = w[t][j] dOut[t];  dw[t][j] = dOut[t] . Y[inverse[t][j]]
__global__ __launch_bounds__(kRowThreads) void k_expert_combine_bwd(
    const uint16_t* __restrict__ dOut, const uint16_t* __restrict__ Y, int64_t tokens, int topk,
    int64_t K, const int* __restrict__ inverse, const float* __restrict__ weights,
    uint16_t* __restrict__ dY, float* __restrict__ dw) {
  __shared__ float dots[kMaxTopk][kRowThreads / 64];
  const int64_t t = row_token(), n = tokens * topk;
  if (t >= tokens) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int j = 0; j < topk; ++j) {
    const int64_t row = inverse[t * topk + j];
    float dot = 0.f;
    if (row >= 0 && row < n) {
      const float w = weights[t * topk + j];
      for (int64_t c = 8 * threadIdx.x; c < K; c += 8 * kRowThreads) {
        float d[8], y[8], o[8];
        unpack8(*reinterpret_cast<const u32x4*>(dOut + t * K + c), d);
        unpack8(*reinterpret_cast<const u32x4*>(Y + row * K + c), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = fmaf(d[i], y[i], dot);
          o[i] = w * d[i];
        }
        *reinterpret_cast<u32x4*>(dY + row * K + c) = pack8(o);
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) dots[j][wave] = dot;
  }
  __syncthreads();
  if (threadIdx.x < static_cast<unsigned>(topk)) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 64; ++w) s += dots[threadIdx.x][w];
    dw[t * topk + threadIdx.x] = s;
  }
}

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Shapes of the row calls: tokens rows of K, topk slots each.
int check_rows(int64_t tokens, int topk, int64_t K) {
  if (topk < 1 || topk > kMaxTopk) return QLORA_ERR_EXPERT;
  if (tokens < 0 || K < 8 || K % 8 != 0 || K > (int64_t(1) << 22) ||
      tokens > (int64_t(1) << 30) / topk)
    return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

dim3 row_grid(int64_t tokens) {
  return dim3(static_cast<unsigned>(std::min(tokens, kRowBlocks)),
              static_cast<unsigned>((tokens + kRowBlocks - 1) / kRowBlocks));
}

int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

}  // namespace

}  // namespace qnf4

using namespace qnf4;

extern "C" {

size_t qlora_expert_plan_workspace_bytes(int64_t n, int E) {
  if (n < 1 || E < 1 || E > kMaxE) return 0;
  const int nb = plan_blocks(n);
  return nb > 1 ? (static_cast<size_t>(nb) * E * sizeof(int32_t) + 255) / 256 * 256 : 0;
}

int qlora_expert_plan(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order,
                      int32_t* inverse, void* workspace, size_t workspace_bytes,
                      qlora_stream_t stream) {
  if (E < 1 || E > kMaxE) return QLORA_ERR_EXPERT;
  if (n < 0 || n > (int64_t(1) << 30)) return QLORA_ERR_SHAPE;
  if (!offsets || (n > 0 && (!ids || !order || !inverse))) return QLORA_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(inverse, 4))
    return QLORA_ERR_ALIGN;
  const size_t need = qlora_expert_plan_workspace_bytes(n, E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QLORA_ERR_ALIGN;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int nb = plan_blocks(n);
  const int64_t chunk = plan_chunk(n);
  int* counts = nb > 1 ? static_cast<int*>(workspace) : nullptr;
  if (counts) {
    hipLaunchKernelGGL(k_plan_count, dim3(nb), dim3(kPlanThreads), 0, st, ids, n, E, chunk,
                       counts);
    if (hipGetLastError() != hipSuccess) return QLORA_ERR_HIP;
  }
  // static and dynamic LDS together exceed the default limit for large E
  static LdsLimit lds;
  if (lds.raise(reinterpret_cast<const void*>(&k_plan_place), kPlanWaves * kMaxE * 4) !=
      hipSuccess)
    return QLORA_ERR_HIP;
  hipLaunchKernelGGL(k_plan_place, dim3(nb), dim3(kPlanThreads), kPlanWaves * E * sizeof(int), st,
                     ids, n, E, chunk, counts, offsets, order, inverse);
  return hip_status(hipGetLastError());
}

int qlora_expert_gather(const uint16_t* X, int64_t tokens, int topk, int64_t K,
                        const int32_t* inverse, uint16_t* Xs, qlora_stream_t stream) {
  const int st = check_rows(tokens, topk, K);
  if (st) return st;
  if (tokens == 0) return QLORA_OK;
  if (!X || !inverse || !Xs) return QLORA_ERR_NULL;
  if (!aligned(X, 16) || !aligned(Xs, 16) || !aligned(inverse, 4)) return QLORA_ERR_ALIGN;
  hipLaunchKernelGGL(k_expert_gather, row_grid(tokens), dim3(kRowThreads), 0,
                     static_cast<hipStream_t>(stream), X, tokens, topk, K, inverse, Xs);
  return hip_status(hipGetLastError());
}

int qlora_expert_combine(const uint16_t* Y, int64_t tokens, int topk, int64_t K,
                         const int32_t* inverse, const float* weights, uint16_t* out,
                         qlora_stream_t stream) {
  const int st = check_rows(tokens, topk, K);
  if (st) return st;
  if (tokens == 0) return QLORA_OK;
  if (!Y || !inverse || !out) return QLORA_ERR_NULL;
  if (!aligned(Y, 16) || !aligned(out, 16) || !aligned(inverse, 4) || !aligned(weights, 4))
    return QLORA_ERR_ALIGN;
  hipLaunchKernelGGL(k_expert_combine, row_grid(tokens), dim3(kRowThreads), 0,
                     static_cast<hipStream_t>(stream), Y, tokens, topk, K, inverse, weights, out);
  return hip_status(hipGetLastError());
}

int qlora_expert_combine_bwd(const uint16_t* dOut, const uint16_t* Y, int64_t tokens, int topk,
                             int64_t K, const int32_t* inverse, const float* weights,
                             uint16_t* dY, float* dweights, qlora_stream_t stream) {
  const int st = check_rows(tokens, topk, K);
  if (st) return st;
  if (tokens == 0) return QLORA_OK;
  if (!dOut || !Y || !inverse || !weights || !dY || !dweights) return QLORA_ERR_NULL;
  if (!aligned(dOut, 16) || !aligned(Y, 16) || !aligned(dY, 16) || !aligned(inverse, 4) ||
      !aligned(weights, 4) || !aligned(dweights, 4))
    return QLORA_ERR_ALIGN;
  hipLaunchKernelGGL(k_expert_combine_bwd, row_grid(tokens), dim3(kRowThreads), 0,
                     static_cast<hipStream_t>(stream), dOut, Y, tokens, topk, K, inverse, weights,
                     dY, dweights);
  return hip_status(hipGetLastError());
}

}  // extern "C"
