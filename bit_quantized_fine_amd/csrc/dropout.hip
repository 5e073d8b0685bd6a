// Standalone dropout y = mask . scale . x over a flat bf16 tensor, the mask
// regenerated from the counter-based generator (dropout.hpp); its backward is
// the same call on the gradient.
//
// Each thread takes 16-byte pieces of eight values, one generator call each.
// The kernel is bound by the bytes it moves (2 read and 2 written an element):
// a piece costs about 14 wide multiplications and 60 simple operations against
// 32 bytes.  4096 x 17920 values take 54.7 us call after call: 5.4 TB/s.
#include "dropout.hpp"
#include "kernels.hpp"

namespace qnf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;   // 16-byte pieces a thread, kThreads apart
// Workgroups lie in rows of this many along y (a launch holds fewer than 2^32
// threads along x).
constexpr int64_t kRowBlocks = int64_t(1) << 23;

__device__ __forceinline__ uint32_t drop_pair(uint32_t x, uint32_t keep, float scale) {
  return pack_bf16x2(bf16_lo_to_f32(x) * scale, bf16_hi_to_f32(x) * scale) & keep;
}

}  // namespace

__global__ __launch_bounds__(kThreads) void k_dropout(const uint16_t* x, int64_t n,
                                                      const uint64_t* state, uint32_t thr,
                                                      float scale, uint16_t* y) {
  DropKey key{};   // thr = 0 keeps everything, and state may be null
  if (thr > 0) key = load_drop_key(state, thr);
  const int64_t whole = n / 8;
  const int64_t p0 =
      ((int64_t)blockIdx.y * kRowBlocks + blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  u32x4 v[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t p = p0 + i * kThreads;
    v[i] = p < whole ? *reinterpret_cast<const u32x4*>(x + 8 * p) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t p = p0 + i * kThreads;
    if (p < whole) {
      const u32x4 k = keep_piece(key, static_cast<uint64_t>(p));
      *reinterpret_cast<u32x4*>(y + 8 * p) =
          u32x4{drop_pair(v[i].x, k.x, scale), drop_pair(v[i].y, k.y, scale),
                drop_pair(v[i].z, k.z, scale), drop_pair(v[i].w, k.w, scale)};
    } else if (p == whole) {   // the last n % 8 values
      const u32x4 w = philox_piece(key, static_cast<uint64_t>(p));
#pragma unroll
      for (int e = 0; e < 7; ++e) {
        if (8 * p + e < n) {
          const uint32_t pair = e < 2 ? w.x : (e < 4 ? w.y : (e < 6 ? w.z : w.w));
          const uint32_t h = (e & 1) ? pair >> 16 : pair & 0xFFFFu;
          const float f = bf16_lo_to_f32(x[8 * p + e]) * scale;
          y[8 * p + e] = h >= thr ? static_cast<uint16_t>(pack_bf16x2(f, 0.f)) : 0;
        }
      }
    }
  }
}

hipError_t launch_dropout(const uint16_t* x, int64_t n, const Drop& d, uint16_t* y,
                          hipStream_t stream) {
  const int64_t blocks = n / (8 * kThreads * kPieces) + 1;
  const dim3 grid(static_cast<unsigned>(blocks < kRowBlocks ? blocks : kRowBlocks),
                  static_cast<unsigned>((blocks + kRowBlocks - 1) / kRowBlocks));
  hipLaunchKernelGGL(k_dropout, grid, dim3(kThreads), 0, stream, x, n, d.state, d.thr, d.scale(),
                     y);
  return hipGetLastError();
}

}  // namespace qnf4
