// Activations to their 8-bit checkpoint and back (act8.hpp).
//
// A thread takes 16 values: two 16-byte pieces one way, one 16-byte piece of
// codes the other, so the four lanes of an aligned quad hold a block and find
// its largest magnitude with two lane moves.  Both kernels are bound by the
// bytes they move (3.06 a value); a value costs about eight operations on its
// way out and three on its way back.  With three sets of buffers in turn, 4096 x 17920
// values take 42 us out (5.4 TB/s) and 45 us back (5.0; on one set, which the cache holds
// in part, 40 and 36).  Non-temporal accesses gained nothing out (38 against 35 to 41, its
// output in one buffer) and cost the way back (69 to 74 against 38).
#include "act8.hpp"
#include "kernels.hpp"
#include "qlora_nf4.h"

namespace qnf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;   // values a thread
// Workgroups lie in rows of this many along y (a launch holds fewer than 2^32
// threads along x).
constexpr int64_t kRowBlocks = int64_t(1) << 23;

__device__ __forceinline__ int64_t first_value() {
  return (((int64_t)blockIdx.y * kRowBlocks + blockIdx.x) * kThreads + threadIdx.x) * kPer;
}

dim3 grid_of(int64_t n) {
  const int64_t blocks = (n + kThreads * kPer - 1) / (kThreads * kPer);
  return dim3(static_cast<unsigned>(blocks < kRowBlocks ? blocks : kRowBlocks),
              static_cast<unsigned>((blocks + kRowBlocks - 1) / kRowBlocks));
}

}  // namespace

__global__ __launch_bounds__(kThreads) void k_act8_pack(const uint16_t* __restrict__ x, int64_t n,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  const int64_t i = first_value();
  if (i >= n) return;   // (n % 64 == 0: whole blocks)
  const u32x4 a = *reinterpret_cast<const u32x4*>(x + i);
  const u32x4 b = *reinterpret_cast<const u32x4*>(x + i + 8);
  const Act8Scale s = act8_scale(max_over4(max(amax_bits8(a), amax_bits8(b))));
  const u32x2 ca = act8_codes(a, s), cb = act8_codes(b, s);
  *reinterpret_cast<u32x4*>(codes + i) = u32x4{ca.x, ca.y, cb.x, cb.y};
  if ((threadIdx.x & 3) == 0) scales[i / 64] = s.c;
}

__global__ __launch_bounds__(kThreads) void k_act8_unpack(const int8_t* __restrict__ codes,
                                                          const float* __restrict__ scales,
                                                          int64_t n, uint16_t* __restrict__ x) {
  const int64_t i = first_value();
  if (i >= n) return;
  const u32x4 v = *reinterpret_cast<const u32x4*>(codes + i);
  const float c = scales[i / 64];
  *reinterpret_cast<u32x4*>(x + i) = act8_values(v.x, v.y, c);
  *reinterpret_cast<u32x4*>(x + i + 8) = act8_values(v.z, v.w, c);
}

hipError_t launch_act8_pack(const uint16_t* x, int64_t n, int8_t* codes, float* scales,
                            hipStream_t stream) {
  hipLaunchKernelGGL(k_act8_pack, grid_of(n), dim3(kThreads), 0, stream, x, n, codes, scales);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const int8_t* codes, const float* scales, int64_t n, uint16_t* x,
                              hipStream_t stream) {
  hipLaunchKernelGGL(k_act8_unpack, grid_of(n), dim3(kThreads), 0, stream, codes, scales, n, x);
  return hipGetLastError();
}

}  // namespace qnf4
