// Routing of tokens to experts: scores, the choice of the topk best, their
// weights, and the gradient of the weights back to the logits.
//
// A wave takes one token; lane l holds experts l EPL .. l EPL + EPL - 1, so that
// among equal values the lowest lane's first one is the lowest index.  Values
// are compared as integers of the same order: the logits' 32 bits where no bias
// is given (a softmax or sigmoid keeps their order), else the 64 bits of p +
// bias, formed in 64 bits: the scores of 256 experts lie about 2^-8 apart, so in
// 32 bits about one token in 10^4 would get an order that depends on how its
// scores were rounded.  A round of the choice is the wave's largest value by six
// lane moves, and a ballot for its owner.
//   By sigmoid and bias 32 bits choose and the chosen ones' 64 bits prove it
// (choose_by_32).  Two tokens share a wave where the rules at the launches say so.  A
// token's choice and weights are the same on either way.
//
// 8192 tokens of 256 experts by sigmoid, bias and groups, topk 8, take 8.0 us back to
// back in a graph (8.4 MB would take 1.9; one token a wave 10.7, wholly in 64 bits 15).
// All four waves a SIMD are resident at once, so that time is a wave's chain of
// dependent steps: waves wait for half of their cycles, and the 650 vector instructions
// for two tokens would take 4.3 us.  32768 tokens (20.3 us, 7 by their bytes) are bound
// by those instructions, at least 17.3 us of them.  By the logit alone 8192 tokens of 64
// experts take 4.5 us; 32768 of 256 in bf16 13.2 (4 by their bytes), 12.4 of them the
// vector instructions of the sort and of eight rounds.
//   Smaller batches are a launch and the call (8 us).  The backward of 8192 tokens of 64
// experts takes 4.5 us, of 256 5.7 (a softmax that is not renormalised, one token a wave
// with an exponential for every expert, 5.6 and 8.6).
//
// Weights and gradients are formed in 64 bits too, where they cost one lane's
// work a slot: what is left of 1 - p where one expert takes nearly all would
// lose its bits in 32.
#include <algorithm>
#include <cmath>

#include "act8.hpp"
#include "device_common.hpp"
#include "kernels.hpp"
#include "qlora_nf4.h"

namespace qnf4 {

namespace {

constexpr int kWaves = 4;          // waves a workgroup
constexpr int kMaxE = 1024;
constexpr double kLeastSum = 1e-250;     // of sigmoids that are divided by their sum as
                                         // they are (below, every logit is under -575)
constexpr int64_t kPairTokens = 2048;      // from here on two tokens share a wave (in_pairs,
constexpr int64_t kPairTokensBack = 4096;  // back_in_pairs)
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;
// Workgroups lie in rows of this many along y (a launch holds fewer than 2^32
// threads along x).
constexpr int64_t kRowBlocks = int64_t(1) << 23;

typedef double f64x2 __attribute__((ext_vector_type(2)));

struct Router {
  const void* logits;
  int64_t tokens;
  int E;
  const float* bias;      // may be null
  int topk;
  int sigmoid, renorm;
  float scale;
  int choose_groups;      // 0: every group stays
  int groups, top_groups, group_top;
  int gs;                 // experts of a group
  uint32_t gs_mul;        // e / gs = e gs_mul >> 20
  int gshift;             // log2 of the lanes that look at one group
  int in_lanes;           // those lanes hold the whole group (at most 16)
  int* ids;
  float* weights;
  const float* dweights;
  void* dlogits;
};

__device__ __forceinline__ int read_lane(int v, int lane) {
  return __builtin_amdgcn_readlane(v, lane);
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Orders a wave's LDS accesses: what its lanes wrote before is there for the others.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Largest value over the wave (zero where no lane has a larger one).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](auto moved) { v = max(v, static_cast<uint32_t>(moved)); };
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x111, 0xF, 0xF, false));   // row_shr 1
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x112, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x114, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x118, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x142, 0xA, 0xF, false));   // row_bcast 15
  step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x143, 0xC, 0xF, false));   // row_bcast 31
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
// Largest value over the W lanes (32 or 64) that hold a token, in all of them.
template <int W>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = dpp_max_u32<0x140>(max_over8(v));   // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // rows 0 and 1, 2 and 3
  v = max(r[0], r[1]);
  if constexpr (W == 64) {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(h[0], h[1]);
  }
  return v;
}
// Whether a mask holds several lanes of one token (W lanes a token), and how many of this
// lane's token come before it there.
template <int W>
__device__ __forceinline__ bool several(uint64_t at) {
  if constexpr (W == 64) return (at & (at - 1)) != 0;
  const uint32_t l = static_cast<uint32_t>(at), h = static_cast<uint32_t>(at >> 32);
  return ((l & (l - 1)) | (h & (h - 1))) != 0;
}
template <int W>
__device__ __forceinline__ uint32_t lanes_before(uint64_t at) {
  const uint32_t l = static_cast<uint32_t>(at), h = static_cast<uint32_t>(at >> 32);
  const uint32_t low = __builtin_amdgcn_mbcnt_lo(l, 0u);
  if constexpr (W == 64) return __builtin_amdgcn_mbcnt_hi(h, low);
  return (threadIdx.x & 32) ? __builtin_amdgcn_mbcnt_hi(h, 0u) : low;
}
// v moved across lanes (zero where there is no lane to take it from).
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Sum over the wave, always in the same order.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0x111>(v);        // row_shr 1, 2, 4, 8
  v += dpp_f64<0x112>(v);
  v += dpp_f64<0x114>(v);
  v += dpp_f64<0x118>(v);
  v += dpp_f64<0x142, 0xA>(v);   // row_bcast 15, 31
  v += dpp_f64<0x143, 0xC>(v);
  return read_lane(v, 63);
}
// The same over the W lanes of a token (of 32 lanes: bit for bit the sum over a wave
// whose other half is zero).
template <int W>
__device__ __forceinline__ double lanes_sum(double v) {
  if constexpr (W == 64) return wave_sum(v);
  v += dpp_f64<0x111>(v);
  v += dpp_f64<0x112>(v);
  v += dpp_f64<0x114>(v);
  v += dpp_f64<0x118>(v);
  v += dpp_f64<0x142, 0xA>(v);
  const double a = read_lane(v, 31), b = read_lane(v, 63);
  return (threadIdx.x & 32) ? b : a;
}

// exp(x) for x <= 0, to about one unit in the last place of 64 bits: x = n ln 2 +
// r with |r| <= ln 2 / 2 (W. Cody, W. Waite, "Software Manual for the Elementary
// Functions": ln 2 as a part of 32 bits, whose product with n is exact, and the
// rest), and the series of exp(r) to r^13 / 13!, which leaves out less than 2^-57.
// The coefficients are held in scalar registers (the empty asm puts them there): a
// step is then one fma that reads its coefficient, where the compiler else copies
// each into vector registers first, three instructions a step.
struct Exp {
  double c[12];   // 1 / 13!, ..., 1 / 2!
  __device__ __forceinline__ Exp() {
    double f = 6227020800.0;
#pragma unroll
    for (int i = 0; i < 12; ++i) {
      c[i] = 1.0 / f;
      asm("" : "+s"(c[i]));
      f /= 13 - i;   // (exact)
    }
  }
  __device__ __forceinline__ double operator()(double x) const {
    x = max(x, -800.0);   // 0 from about -745 on (-inf too)
    const double n = __builtin_rint(x * 1.4426950408889634074);
    double r = fma(n, -0x1.62e42feep-1, x);
    r = fma(n, -0x1.a39ef35793c76p-33, r);
    double p = c[0];
#pragma unroll
    for (int i = 1; i < 12; ++i) p = fma(p, r, c[i]);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
  }
};

// Integers in the order of the values; 0 for an expert that is not to be
// chosen (-inf or NaN).  v + 0 makes -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  return v > -__builtin_inff() ? b ^ ((b >> 31) ? ~0u : 0x80000000u) : 0u;
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return v > -__builtin_inf() ? b ^ ((b >> 63) ? ~0ull : 1ull << 63) : 0ull;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, (k >> 31) ? k ^ 0x80000000u : ~k);
}

template <class L>
__device__ __forceinline__ float to_f32(L v) {
  if constexpr (sizeof(L) == 2)
    return bf16_lo_to_f32(v);
  else
    return v;
}

// sigma(x) = exp(min(x, 0)) / (1 + exp(-|x|))
__device__ __forceinline__ double sigmoid64(const Exp& exp_neg, double x) {
  const double t = exp_neg(-fabs(x));
  return (x > 0.0 ? 1.0 : t) / (1.0 + t);
}

// EPL values from element e0 on, `none` past E.  Where E is whole pieces of a lane,
// a piece is one load (of any alignment: a token's row starts anywhere).
template <int EPL, class L>
__device__ __forceinline__ void load_piece(const L* row, int e0, int E, float none, float* x) {
  if (E % EPL == 0) {
    L v[EPL];
    const int at = e0 < E ? e0 : 0;
    __builtin_memcpy(v, row + at, sizeof(v));
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = e0 < E ? to_f32(v[i]) : none;
  } else {
    L v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = row[e0 + i < E ? e0 + i : 0];
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = e0 + i < E ? to_f32(v[i]) : none;
  }
}

// A token's logits: lane l holds experts l EPL ...; -inf past E.
template <int EPL, class L>
struct Logits {
  float x[EPL];
  bool bad;     // a NaN or +inf among them
  // W lanes a token, `lane` of them from lane `base` of the wave on
  template <int W>
  __device__ void load(const L* row, int E, int lane, int base) {
    load_piece<EPL, L>(row, lane * EPL, E, -__builtin_inff(), x);
    uint64_t b = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)   // signalling and quiet NaN, +inf
      b |= __builtin_amdgcn_ballot_w64(__builtin_amdgcn_classf(x[i], 0x203));
    bad = W == 64 ? b != 0 : static_cast<uint32_t>(b >> base) != 0;
  }
  // the largest, -inf without any
  __device__ float top() const {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) k = max(k, order_key(x[i]));
    k = wave_max(k);
    return k ? key_value(k) : -__builtin_inff();
  }
  // sum over the experts of exp(x - top), which this lane's d[i] receive
  __device__ double exps(const Exp& exp_neg, float top, double* d) const {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      d[i] = x[i] > -__builtin_inff() ? exp_neg(static_cast<double>(x[i]) - static_cast<double>(top))
                                      : 0.0;
      s += d[i];
    }
    return wave_sum(s);
  }
};

// The lane with the wave's largest key, the lowest of several; -1 if all are 0.
// Where the high words of 64 bits decide (all but about one round in 10^4), the low
// ones are not looked at.
__device__ __forceinline__ int best_lane(uint32_t k) {
  const uint32_t m = wave_max(k);
  return m ? __builtin_ctzll(__builtin_amdgcn_ballot_w64(k == m)) : -1;
}
__device__ __forceinline__ int best_lane(uint64_t k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32), lo = static_cast<uint32_t>(k);
  const uint32_t m = wave_max(hi);
  if (m == 0) return -1;   // (a key that is not 0 has its high word)
  uint64_t at = __builtin_amdgcn_ballot_w64(hi == m);
  if (at & (at - 1)) {
    const uint32_t l = wave_max(hi == m ? lo : 0u);
    at = __builtin_amdgcn_ballot_w64(hi == m && lo == l);
  }
  return __builtin_ctzll(at);
}

// The topk largest keys in order: lane j gets the expert of slot j, -1 if none is
// left.  Up to eight keys a lane are sorted first, so that a round only moves the
// winner's up: neighbours change places where the second is larger, which
// leaves equal ones in their order.
template <int EPL, class Key>
__device__ __forceinline__ int choose(Key* k, int topk, int lane) {
  int id = -1;
  if constexpr (EPL <= 8) {
    int at[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) at[i] = lane * EPL + i;
#pragma unroll
    for (int n = 0; n < EPL; ++n)
#pragma unroll
      for (int i = n & 1; i + 1 < EPL; i += 2) {
        const bool swap = k[i] < k[i + 1];
        const Key hi = swap ? k[i + 1] : k[i], lo = swap ? k[i] : k[i + 1];
        const int ih = swap ? at[i + 1] : at[i], il = swap ? at[i] : at[i + 1];
        k[i] = hi;
        k[i + 1] = lo;
        at[i] = ih;
        at[i + 1] = il;
      }
    for (int j = 0; j < topk; ++j) {
      const int who = best_lane(k[0]);
      if (who < 0) break;   // uniform
      const int e = read_lane(at[0], who);
      if (lane == j) id = e;
      if (lane == who) {
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) {
          k[i] = k[i + 1];
          at[i] = at[i + 1];
        }
        k[EPL - 1] = 0;
      }
    }
  } else {
    Key cur = k[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) cur = max(cur, k[i]);
    for (int j = 0; j < topk; ++j) {
      const int who = best_lane(cur);
      if (who < 0) break;   // uniform
      int e = 0;
      if (lane == who) {
        const Key m = cur;
        bool found = false;
        cur = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (!found && k[i] == m) {
            found = true;
            e = lane * EPL + i;
            k[i] = 0;
          }
          cur = max(cur, k[i]);
        }
      }
      e = read_lane(e, who);
      if (lane == j) id = e;
    }
  }
  return id;
}

// The two largest of all values that the lanes of a group hold (groups of 1 << n
// lanes, n <= 4), in all of them.
template <int CTRL>
__device__ __forceinline__ void merge_two(double& t1, double& t2) {
  const double o1 = dpp_f64<CTRL>(t1), o2 = dpp_f64<CTRL>(t2);
  t2 = max(min(t1, o1), max(t2, o2));
  t1 = max(t1, o1);
}
template <int CTRL>
__device__ __forceinline__ void merge_two(uint32_t& t1, uint32_t& t2) {
  auto moved = [](uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
  };
  const uint32_t o1 = moved(t1), o2 = moved(t2);
  t2 = max(min(t1, o1), max(t2, o2));
  t1 = max(t1, o1);
}
template <class T>
__device__ __forceinline__ void two_best_of_lanes(T& t1, T& t2, int lanes) {
  if (lanes > 1) merge_two<0xB1>(t1, t2);    // quad_perm 1,0,3,2
  if (lanes > 2) merge_two<0x4E>(t1, t2);    // quad_perm 2,3,0,1
  if (lanes > 4) merge_two<0x141>(t1, t2);   // row_half_mirror
  if (lanes > 8) merge_two<0x140>(t1, t2);   // row_mirror
}

// Relative weights u of the chosen (0 for lanes without one), for the
// renormalised forms: exp(x - m), times 1 / (1 + exp(-|x|)) for a sigmoid, whose
// factor exp(min(x, 0)) is the one shifted by m.
template <int W>
__device__ __forceinline__ double relative_weight(const Router& a, const Exp& exp_neg, bool live,
                                                  float lx) {
  const float v = a.sigmoid ? min(lx, 0.f) : lx;
  const float m = key_value(lanes_max<W>(live ? order_key(v) : 0u));
  if (!live) return 0.0;
  const double u = exp_neg(static_cast<double>(v) - static_cast<double>(m));
  return a.sigmoid ? u / (1.0 + exp_neg(-fabs(static_cast<double>(lx)))) : u;
}

// sigma(x) in 32 bits, off by less than 2^-21: t = exp(-|x|) is off by 2.6 2^-24
// (the product's rounding times |x| t <= 0.37, the exponential's last place), and 1 +
// t, its reciprocal and the product by 4 2^-24 of the result.
__device__ __forceinline__ float sigmoid32(float x) {
  const float t = __builtin_amdgcn_exp2f(fabsf(x) * -1.442695041f);
  const float s = __builtin_amdgcn_rcpf(1.f + t);
  return x > 0.f ? s : t * s;
}

// Sorts N keys (a power of two), the largest first: K. Batcher's merges of odd and
// even places (D. Knuth, "The Art of Computer Programming" 3, 5.3.4).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t* k) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int i = d % p; i + d < N; ++i) {
        if ((i - d % p) / d % 2 != 0 || i / (2 * p) != (i + d) / (2 * p)) continue;
        const uint32_t hi = max(k[i], k[i + d]), lo = min(k[i], k[i + d]);
        k[i] = hi;
        k[i + d] = lo;
      }
}

// The choice by sigmoid and bias through 32 bits, with what it proves.  A key is the
// rank's 32 bits with the expert's place in its lane in the lowest ones, so that a
// lane's keys differ and sorting them moves nothing else; a rank r read from a key
// is off by less than kErr (1 + |r|) (2^-20 of it by score and sum, the rest by the
// bits given away, at most 7 or 15 of 2^-23 r).  As that keeps the order of the
// bounds, the nth largest rank is off by as much.
//   Groups are chosen by the keys.  If some at the border could change sides (one
// token in 10^3), each lane forms its best one or two ranks in 64 bits, which give
// the groups' scores, unless a lane's next key could be among a group's best.
//   Experts are chosen by the keys, one more than topk, each round's winner (the first
// of several lanes) leaving its expert in `slots` (LDS, one a lane).  Their ranks are
// then formed in 64 bits, one a lane, and order them.  The choice stands if every chosen
// rank is above the best key left by more than its error: then it is the one that 64
// bits make.
//   Else (about one token in 10^5 of 256 experts) false: the choice is made anew.
//   For tokens without NaN and +inf, and groups within lanes.  W lanes a token, this
// one's being `lane` of them from lane `base` of the wave on; id and p: of this lane's
// slot, p in 64 bits.
template <int W, int EPL, class L>
__device__ __forceinline__ bool choose_by_32(const Router& a, const Exp& exp_neg, const float* x,
                                             const L* row, int lane, int base, int* slots,
                                             int& id, double& p) {
  constexpr float kErr = EPL <= 8 ? 0x1p-19f : 0x1p-18f;
  constexpr uint32_t kPlace = EPL - 1, kNone = 0x00800000u;   // keys below it: -inf
  constexpr uint64_t kLanes = W == 64 ? ~0ull : 0xFFFFFFFFull;
  slots[lane] = -1;
  float b[EPL];
  load_piece<EPL, float>(a.bias, lane * EPL, a.E, 0.f, b);
  uint32_t k[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float r = sigmoid32(x[i]) + b[i];
    // (not for NaN; never -0)
    const float v = x[i] > -__builtin_inff() && r > -__builtin_inff() ? r : -__builtin_inff();
    const int32_t bits = __builtin_bit_cast(int32_t, v);
    const uint32_t key = static_cast<uint32_t>(bits) ^ (static_cast<uint32_t>(bits >> 31) | 0x80000000u);
    k[i] = (key & ~kPlace) | (kPlace - i);
  }
  sort_down<EPL>(k);
  auto expert = [&](uint32_t key) {   // of this lane
    return lane * EPL + static_cast<int>(kPlace - (key & kPlace));
  };
  auto score = [&](int e) { return sigmoid64(exp_neg, static_cast<double>(to_f32(row[e]))); };
  // above every rank whose key is this one or a lower one
  auto bound = [&](uint32_t key) {
    const double v = key_value(key);
    return v + static_cast<double>(kErr) * (1.0 + fabs(v));
  };
  uint64_t doubt = 0;   // lanes that see a reason against the choice
  if (a.choose_groups) {
    uint32_t t1 = k[0], t2 = EPL > 1 ? k[EPL > 1 ? 1 : 0] : 0u;
    // this lane's group, its place among the group's lanes, their number
    const int shift = W == 64 ? a.gshift : a.gshift - 1;
    const int lanes = 1 << shift, g = lane >> shift, sub = lane & (lanes - 1);
    two_best_of_lanes(t1, t2, lanes);
    const bool any = t1 >= kNone && g < a.groups, both = a.group_top == 2 && t2 >= kNone;
    const float v1 = key_value(t1), v2 = both ? key_value(t2) : 0.f;
    // twice the errors of the two ranks, for the additions here
    const float off = 2.f * kErr * (2.f + fabsf(v1) + fabsf(v2));
    const float hi = any ? v1 + v2 + off : -__builtin_inff();
    const float lo = any ? v1 + v2 - off : -__builtin_inff();
    // groups ahead of this lane's, its lanes looking at one each
    const int first = base + (g << shift);
    const uint32_t mine = (1u << lanes) - 1;   // (lanes <= 16)
    auto of_mine = [&](bool v) {
      return __builtin_popcount(
          static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(v) >> first) & mine);
    };
    int sure = 0, perhaps = 0;
    for (int q0 = 0; q0 < a.groups; q0 += lanes) {
      const int q = q0 + sub, at = base + (q << shift);
      const float oh = __shfl(hi, at), ol = __shfl(lo, at);
      const bool other = q < a.groups && q != g;
      sure += of_mine(other && ol > hi);
      perhaps += of_mine(other && !(oh < lo));
    }
    bool stays = any && perhaps < a.top_groups;
    const uint64_t border = __builtin_amdgcn_ballot_w64(any && !stays && sure < a.top_groups);
    if (border != 0) {   // uniform
      const bool two = EPL > 1 && a.group_top == 2, here = ((border >> base) & kLanes) != 0;
      const uint32_t k1 = two ? k[EPL > 1 ? 1 : 0] : 0u;
      const uint32_t k2 = two ? (EPL > 2 ? k[EPL > 2 ? 2 : 0] : 0u) : (EPL > 1 ? k[EPL > 1 ? 1 : 0] : 0u);
      double d1 = -__builtin_inf(), d2 = d1;
      if (k[0] >= kNone) d1 = score(expert(k[0])) + static_cast<double>(a.bias[expert(k[0])]);
      if (k1 >= kNone) d2 = score(expert(k1)) + static_cast<double>(a.bias[expert(k1)]);
      const double low = min(d1, d2);
      d1 = max(d1, d2);
      d2 = low;
      two_best_of_lanes(d1, d2, lanes);
      const bool unclear = here && k2 >= kNone && !(bound(k2) < (a.group_top == 2 ? d2 : d1));
      const double sum = a.group_top == 2 && d2 > -__builtin_inf() ? d1 + d2 : d1;
      int better = 0;
      for (int q0 = 0; q0 < a.groups; q0 += lanes) {
        const int q = q0 + sub;
        const double o = __shfl(sum, base + (q << shift));
        better += of_mine(q < a.groups && (o > sum || (o == sum && q < g)));
      }
      if (here) stays = any && better < a.top_groups;
      doubt = __builtin_amdgcn_ballot_w64(unclear);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) k[i] = stays ? k[i] : 0u;
  }
  const int rounds = a.topk < W ? a.topk + 1 : W;
  for (int j = 0; j < rounds; ++j) {
    const uint32_t best = lanes_max<W>(k[0]);
    bool won = k[0] == best && best >= kNone;
    const uint64_t at = __builtin_amdgcn_ballot_w64(won);
    if (several<W>(at)) won = won && lanes_before<W>(at) == 0;   // uniform; one token in 10^5
    if (won) {
      slots[j] = expert(best);
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) k[i] = k[i + 1];
      k[EPL - 1] = 0;
    }
  }
  const uint32_t left = lanes_max<W>(k[0]);
  wave_lds_fence();
  id = slots[lane];
  const bool live = id >= 0;
  p = 0.0;
  double rank = -__builtin_inf();
  if (live) {
    p = score(id);
    rank = p + static_cast<double>(a.bias[id]);
  }
  const double next = __shfl_down(rank, 1);
  const int next_id = __shfl_down(id, 1);
  const bool turned = lane < W - 1 && next_id >= 0 && !(rank > next || (rank == next && id < next_id));
  if (__builtin_amdgcn_ballot_w64(turned) != 0) {   // uniform
    int place = 0;
    for (int j = 0; j < rounds; ++j) {
      const double r = __shfl(rank, base + j);
      const int e = __shfl(id, base + j);
      place += e >= 0 && (r > rank || (r == rank && e < id));
    }
    wave_lds_fence();
    if (live) slots[place] = lane;   // (places of the live, which are the first lanes)
    wave_lds_fence();
    const int from = base + (live ? slots[lane] : lane);
    id = __shfl(id, from);
    p = __shfl(p, from);
    rank = __shfl(rank, from);
  }
  if (lane >= a.topk) {
    id = -1;
    p = 0.0;
  }
  doubt |= __builtin_amdgcn_ballot_w64(id >= 0 && left >= kNone && !(rank > bound(left)));
  return ((doubt >> base) & kLanes) == 0;
}

__device__ __forceinline__ int64_t wave_token() {
  return ((int64_t)blockIdx.y * kRowBlocks + blockIdx.x) * kWaves + wave_id();
}

__device__ __forceinline__ void store_slot(const Router& a, int64_t t, int slot, int id, bool bad,
                                           double w) {
  if (slot >= a.topk) return;
  a.ids[t * a.topk + slot] = id;
  a.weights[t * a.topk + slot] =
      bad && id >= 0 ? __builtin_nanf("") : static_cast<float>(static_cast<double>(a.scale) * w);
}

// Token t by a wave, every value that the choice needs in 64 bits; mine: LDS for E
// values where groups are chosen that do not lie within lanes.
template <int EPL, class L>
__device__ __forceinline__ void route(const Router& a, const Exp& exp_neg, const Logits<EPL, L>& l,
                                      int64_t t, bool in, double* mine) {
  const int lane = threadIdx.x & 63;
  float top = 0.f;
  double p[EPL], sum = 0.0;   // p: scores where they rank, exps otherwise unused
  const bool sums = a.choose_groups && a.group_top == 2;
  if (a.bias || sums) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] = sigmoid64(exp_neg, l.x[i]);
    } else {
      top = l.top();
      sum = l.exps(exp_neg, top, p);
      const double r = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] *= r;
    }
  }
  double rank[EPL];   // with a bias
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      rank[i] = e < a.E && l.x[i] > -__builtin_inff()
                    ? p[i] + static_cast<double>(a.bias[e]) : -__builtin_inf();
    }
  }
  bool mine_stay = true;   // this lane's group, where a lane holds one
  uint64_t keep = 0;       // else bit (group << gshift): the group stays
  if (a.choose_groups) {
    double v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = a.bias ? rank[i] : (sums ? p[i] : static_cast<double>(l.x[i]));
      if (!(l.x[i] > -__builtin_inff()) || !(v[i] > -__builtin_inf())) v[i] = -__builtin_inf();
    }
    double t1 = -__builtin_inf(), t2 = t1;
    auto add = [&](double u) {
      t2 = max(t2, min(t1, u));
      t1 = max(t1, u);
    };
    // this lane's group, its place among the group's lanes, their number
    const int lanes = 1 << a.gshift, g = lane >> a.gshift, sub = lane & (lanes - 1);
    if (a.in_lanes) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) add(v[i]);
      two_best_of_lanes(t1, t2, lanes);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane * EPL + i < a.E) mine[lane * EPL + i] = v[i];
      __syncthreads();   // (uniform over the workgroup)
      if (g < a.groups)
        for (int j = sub; j < a.gs; j += lanes) add(mine[g * a.gs + j]);
      for (int d = 1; d < lanes; d <<= 1) {
        const double o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
        t2 = max(min(t1, o1), max(t2, o2));
        t1 = max(t1, o1);
      }
    }
    const double score = a.group_top == 2 && t2 > -__builtin_inf() ? t1 + t2 : t1;
    int better = 0;   // groups ahead of this lane's
    if (lanes >= a.groups) {   // each of a group's lanes looks at one other group
      const double o = __shfl(score, sub << a.gshift);
      const uint64_t ahead = __builtin_amdgcn_ballot_w64(
          sub < a.groups && (o > score || (o == score && sub < g)));
      better = __builtin_popcountll((ahead >> (lane - sub)) & ((2ull << (lanes - 1)) - 1));
    } else {
      for (int q = 0; q < a.groups; ++q) {
        const double o = read_lane(score, q << a.gshift);
        better += o > score || (o == score && q < g);
      }
    }
    mine_stay = g < a.groups && t1 > -__builtin_inf() && better < a.top_groups;
    if (!a.in_lanes) keep = __builtin_amdgcn_ballot_w64(mine_stay && sub == 0);
  }
  auto stays = [&](int i) {
    if (!a.choose_groups || a.in_lanes) return mine_stay;
    const int e = lane * EPL + i;
    return e < a.E && ((keep >> (((e * a.gs_mul) >> 20) << a.gshift)) & 1) != 0;
  };
  int id;
  if (a.bias) {
    uint64_t k[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) k[i] = stays(i) ? order_key(rank[i]) : 0ull;
    id = choose<EPL, uint64_t>(k, a.topk, lane);
  } else {
    uint32_t k[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) k[i] = stays(i) ? order_key(l.x[i]) : 0u;
    id = choose<EPL, uint32_t>(k, a.topk, lane);
  }
  const float lx =
      id >= 0 ? to_f32(static_cast<const L*>(a.logits)[t * a.E + id]) : 0.f;
  const bool live = id >= 0;
  double w;
  if (a.sigmoid) {
    w = live ? sigmoid64(exp_neg, lx) : 0.0;
    double total = a.renorm ? wave_sum(w) : 1.0;
    if (!(total > kLeastSum)) {   // uniform
      w = relative_weight<64>(a, exp_neg, live, lx);
      total = wave_sum(w);
    }
    w = live ? w / total : 0.0;
  } else if (a.renorm) {
    w = relative_weight<64>(a, exp_neg, live, lx);
    const double total = wave_sum(w);
    w = live ? w / total : 0.0;
  } else {
    if (sum == 0.0) {
      top = l.top();
      sum = l.exps(exp_neg, top, p);
    }
    w = live ? exp_neg(static_cast<double>(lx) - static_cast<double>(top)) / sum : 0.0;
  }
  if (in) store_slot(a, t, lane, id, l.bad, w);
}

}  // namespace

template <int EPL, class L>
__global__ __launch_bounds__(64 * kWaves) void k_router_fwd(Router a) {
  extern __shared__ double lds[];   // [kWaves][E] where groups are chosen
  __shared__ int slots[kWaves][64];
  const int lane = threadIdx.x & 63;
  const int64_t token = wave_token();
  const bool in = token < a.tokens;
  // (a wave without a token repeats the last one, for the barriers)
  const int64_t t = in ? token : a.tokens - 1;
  const L* row = static_cast<const L*>(a.logits) + t * a.E;
  Logits<EPL, L> l;
  l.template load<64>(row, a.E, lane, 0);
  const Exp exp_neg;
  if (a.bias && a.sigmoid && !l.bad && (!a.choose_groups || a.in_lanes)) {   // uniform
    int id;
    double p;
    if (choose_by_32<64, EPL, L>(a, exp_neg, l.x, row, lane, 0, slots[wave_id()], id, p)) {
      const double total = a.renorm ? wave_sum(p) : 1.0;
      if (total > kLeastSum) {
        if (in) store_slot(a, t, lane, id, false, p / total);
        return;
      }
    }
  }
  route<EPL, L>(a, exp_neg, l, t, in, lds + (int64_t)wave_id() * a.E);
}

// By sigmoid and bias with two tokens a wave: the rounds of the choice, its
// proof and the weights take as many instructions for both.  A token whose choice is
// not proven gets the whole wave.  (EPL experts a lane of 32.)
template <int EPL, class L>
__global__ __launch_bounds__(64 * kWaves) void k_router_fwd_pairs(Router a) {
  __shared__ int slots[kWaves][64];
  const int half = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;
  const int64_t first = 2 * wave_token();
  const bool in = first + half < a.tokens;
  const int64_t t = in ? first + half : a.tokens - 1;
  const L* row = static_cast<const L*>(a.logits) + t * a.E;
  Logits<EPL, L> l;
  l.template load<32>(row, a.E, lane, 32 * half);
  const Exp exp_neg;
  int id;
  double p;
  bool ok = choose_by_32<32, EPL, L>(a, exp_neg, l.x, row, lane, 32 * half,
                                     slots[wave_id()] + 32 * half, id, p);
  const double total = a.renorm ? lanes_sum<32>(p) : 1.0;
  ok = ok && !l.bad && total > kLeastSum;
  const uint64_t no = __builtin_amdgcn_ballot_w64(!ok);
  const bool stands = (static_cast<uint32_t>(no >> (32 * half))) == 0;
  if (stands && in) store_slot(a, t, lane, id, false, p / total);
  if (no == 0) return;   // (uniform)
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    if (static_cast<uint32_t>(no >> (32 * h)) == 0 || first + h >= a.tokens) continue;   // uniform
    Logits<EPL / 2, L> l;
    l.template load<64>(static_cast<const L*>(a.logits) + (first + h) * a.E, a.E,
                        threadIdx.x & 63, 0);
    route<EPL / 2, L>(a, exp_neg, l, first + h, true, nullptr);
  }
}

// By the logits themselves, without a bias and groups, two tokens a wave.  A bf16
// logit's key has room for its expert (the lower index above); with fp32 ones the sort
// moves the experts along, neighbours changing where the second is larger, which leaves
// equal ones in their order.
template <int EPL, class L>
__global__ __launch_bounds__(64 * kWaves) void k_router_top_pairs(Router a) {
  __shared__ int slots[kWaves][64];
  const int half = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;
  const int64_t token = 2 * wave_token() + half;
  const bool in = token < a.tokens;
  const int64_t t = in ? token : a.tokens - 1;
  const L* row = static_cast<const L*>(a.logits) + t * a.E;
  int* const slot = slots[wave_id()] + 32 * half;
  Logits<EPL, L> l;
  l.template load<32>(row, a.E, lane, 32 * half);
  slot[lane] = -1;
  constexpr bool kInKey = sizeof(L) == 2;
  constexpr uint32_t kIds = 0xFF;
  uint32_t k[EPL];
  int at[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    k[i] = order_key(l.x[i]);
    at[i] = lane * EPL + i;
    if (kInKey && k[i] != 0) k[i] = (k[i] & ~kIds) | (kIds - at[i]);
  }
  if constexpr (kInKey) {
    sort_down<EPL>(k);
  } else {
#pragma unroll
    for (int n = 0; n < EPL; ++n)
#pragma unroll
      for (int i = n & 1; i + 1 < EPL; i += 2) {
        const bool swap = k[i] < k[i + 1];
        const uint32_t hi = swap ? k[i + 1] : k[i], lo = swap ? k[i] : k[i + 1];
        const int ih = swap ? at[i + 1] : at[i], il = swap ? at[i] : at[i + 1];
        k[i] = hi;
        k[i + 1] = lo;
        at[i] = ih;
        at[i + 1] = il;
      }
  }
  for (int j = 0; j < a.topk; ++j) {
    const uint32_t best = lanes_max<32>(k[0]);
    const bool among = k[0] == best && best != 0;
    uint32_t below = 0;
    if constexpr (!kInKey) {   // the lowest lane of equal ones
      below = lanes_before<32>(__builtin_amdgcn_ballot_w64(among));
    }
    if (among && below == 0) {
      slot[j] = kInKey ? static_cast<int>(kIds - (best & kIds)) : at[0];
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) {
        k[i] = k[i + 1];
        at[i] = at[i + 1];
      }
      k[EPL - 1] = 0;
    }
  }
  wave_lds_fence();
  const int id = slot[lane];
  const bool live = id >= 0;
  const float lx = live ? to_f32(row[id]) : 0.f;
  const Exp exp_neg;
  double w, total = 0.0;
  if (a.sigmoid) {
    w = live ? sigmoid64(exp_neg, lx) : 0.0;
    total = a.renorm ? lanes_sum<32>(w) : 1.0;
  }
  const bool tiny = !(total > kLeastSum);
  if (__builtin_amdgcn_ballot_w64(tiny) != 0) {   // uniform; with a softmax always
    const double u = relative_weight<32>(a, exp_neg, live, lx), sum = lanes_sum<32>(u);
    if (tiny) {
      w = u;
      total = sum;
    }
  }
  if (in) store_slot(a, t, lane, id, l.bad, live ? w / total : 0.0);
}

// dlogits, W lanes a token (32: two tokens a wave).  Lane j holds slot j; sums over the
// slots run in their order in every lane.  A slot's gradient finds its expert through
// LDS.  Nothing is formed as a difference of nearly equal sums: what an expert that takes
// nearly all leaves to the others keeps its digits.
template <int W, int EPL, class L>
__global__ __launch_bounds__(64 * kWaves) void k_router_bwd(Router a) {
  __shared__ __attribute__((aligned(16))) double grads[kWaves * 64 * EPL];   // [token][expert]
  __shared__ __attribute__((aligned(16))) f64x2 slots[kWaves * 64];
  constexpr int T = 64 / W;
  const int lane = threadIdx.x & (W - 1), base = threadIdx.x & 63 & ~(W - 1);
  const int place = threadIdx.x / W;   // of the token in the workgroup
  const int64_t token = T * wave_token() + base / W;
  const bool in = token < a.tokens;
  const int64_t t = in ? token : a.tokens - 1;
  const L* row = static_cast<const L*>(a.logits) + t * a.E;
  double* const grad = grads + place * W * EPL;
  f64x2* const slot = slots + place * W;
  Logits<EPL, L> l;
  l.template load<W>(row, a.E, lane, base);
#pragma unroll
  for (int i = 0; i < EPL; ++i) grad[lane * EPL + i] = 0.0;
  int id = -1;
  double dw = 0.0;
  float lx = 0.f;
  if (lane < a.topk) {
    id = a.ids[t * a.topk + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) {
      lx = to_f32(row[id]);
      if (!(lx > -__builtin_inff()) && lx == lx) id = -1;   // -inf: never chosen
    }
    if (id >= 0) dw = static_cast<double>(a.dweights[t * a.topk + lane]);
  }
  const bool live = id >= 0;
  // an expert's slot leaves its mark; of several the last one
  wave_lds_fence();
  if (live) grad[id] = lane + 1;
  wave_lds_fence();
  const uint64_t twice = __builtin_amdgcn_ballot_w64(live && grad[live ? id : 0] != lane + 1);
  const Exp exp_neg;
  double d = 0.0;       // of this slot's expert
  double rest[EPL];     // softmax without renorm: of the experts without a slot, -p sum_j p_j dw_j
  if (a.renorm) {
    const double u = relative_weight<W>(a, exp_neg, live, lx), total = lanes_sum<W>(u);
    const double q = live ? u / total : 0.0;
    slot[lane] = f64x2{q, dw};
    wave_lds_fence();
    // q_i sum_j q_j (dw_i - dw_j): no difference of nearly equal sums
    double v = 0.0;
    if (twice == 0) {   // uniform
      for (int j = 0; j < a.topk; ++j) v += slot[j].x * (dw - slot[j].y);
    } else {
      // the terms of one expert's slots cancel in their sum: left out (but for a slot's own,
      // so that a token beside this one gets the same, infinities too)
      for (int j = 0; j < a.topk; ++j)
        if (__shfl(id, base + j) != id || j == lane) v += slot[j].x * (dw - slot[j].y);
    }
    d = q * v;
    if (a.sigmoid) d *= sigmoid64(exp_neg, -static_cast<double>(lx));
  } else if (a.sigmoid) {
    d = live ? dw * sigmoid64(exp_neg, lx) * sigmoid64(exp_neg, -static_cast<double>(lx)) : 0.0;
  } else if constexpr (W == 64) {   // (its sum over the experts would run in another order)
    const float top = l.top();
    const double r = 1.0 / l.exps(exp_neg, top, rest);
    // p_e (dw_e - sum_j p_j dw_j) as p_e (sum_j p_j (dw_e - dw_j) + dw_e u), u what the
    // experts without a slot have: next to one expert that takes nearly all, the difference
    // itself would lose the digits of 1 - p
    bool first = live;
    if (twice != 0) {   // uniform: an expert's first slot takes the sum of its slots' dw
      slot[lane] = f64x2{static_cast<double>(id), dw};
      wave_lds_fence();
      double all = 0.0;
      for (int j = 0; j < a.topk; ++j) {
        if (!live || slot[j].x != id) continue;
        first = first && j >= lane;
        all += slot[j].y;
      }
      dw = all;
      wave_lds_fence();
    }
    double u = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (grad[lane * EPL + i] != 0.0) rest[i] = 0.0;
      u += rest[i];
    }
    u = wave_sum(u) * r;
    const double p =
        first ? exp_neg(static_cast<double>(lx) - static_cast<double>(top)) * r : 0.0;
    slot[lane] = f64x2{p, dw};
    wave_lds_fence();
    double v = dw * u, sum = 0.0;
    for (int j = 0; j < a.topk; ++j) {
      v += slot[j].x * (dw - slot[j].y);
      sum += slot[j].x * slot[j].y;
    }
    d = first ? p * v : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) rest[i] = l.x[i] > -__builtin_inff() ? -rest[i] * r * sum : 0.0;
  }
  // an expert named by several slots gets their sum
  wave_lds_fence();
  if (live) grad[id] = twice == 0 ? d : 0.0;
  wave_lds_fence();
  if (twice != 0) {   // uniform
    for (int j = 0; j < a.topk; ++j) {
      if (live && lane == j) grad[id] += d;
      wave_lds_fence();
    }
  }
  L out[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    double g = grad[lane * EPL + i];
    if constexpr (W == 64)
      if (!a.renorm && !a.sigmoid) g += rest[i];
    const float v = l.bad ? __builtin_nanf("")
                          : static_cast<float>(static_cast<double>(a.scale) * g);
    if constexpr (sizeof(L) == 2)
      out[i] = static_cast<L>(pack_bf16x2(v, 0.f));
    else
      out[i] = v;
  }
  if (!in) return;
  L* const dst = static_cast<L*>(a.dlogits) + t * a.E + lane * EPL;
  if (a.E % EPL == 0) {
    if (lane * EPL < a.E) __builtin_memcpy(dst, out, sizeof(out));
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i < a.E) dst[i] = out[i];
  }
}

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_router(int64_t tokens, int E, const qlora_router_config* c) {
  if (!c) return QLORA_ERR_NULL;
  if (E < 1 || E > kMaxE || c->topk < 1 || c->topk > kMaxTopk) return QLORA_ERR_EXPERT;
  if (c->groups < 1 || c->groups > kMaxGroups || E % c->groups != 0 || c->top_groups < 1 ||
      c->top_groups > c->groups || c->group_top < 1 || c->group_top > 2)
    return QLORA_ERR_EXPERT;
  if (c->topk > E / c->groups * c->top_groups) return QLORA_ERR_EXPERT;
  if ((c->score != QLORA_SCORE_SOFTMAX && c->score != QLORA_SCORE_SIGMOID) ||
      (c->renorm != 0 && c->renorm != 1))
    return QLORA_ERR_EXPERT;
  if (!std::isfinite(c->scale)) return QLORA_ERR_EXPERT;
  if (tokens < 0 || tokens > (int64_t(1) << 30) / c->topk) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

// Experts a lane holds: 1, 2, 4, 8 or 16.
int lane_experts(int E) {
  int n = 1;
  while (64 * n < E) n *= 2;
  return n;
}

Router router(const void* logits, int64_t tokens, int E, const qlora_router_config* c) {
  Router a{};
  a.logits = logits;
  a.tokens = tokens;
  a.E = E;
  a.topk = c->topk;
  a.sigmoid = c->score == QLORA_SCORE_SIGMOID;
  a.renorm = c->renorm;
  a.scale = c->scale;
  a.choose_groups = c->top_groups < c->groups;
  a.groups = c->groups;
  a.top_groups = c->top_groups;
  a.group_top = c->group_top;
  a.gs = E / c->groups;
  // (e < 1024 and gs < 1024: e gs < 2^20, so the quotient is exact)
  a.gs_mul = ((1u << 20) + a.gs - 1) / a.gs;
  // whole groups in 1, 2, 4, 8 or 16 lanes: no way through LDS
  const int per = lane_experts(E);
  for (int n = 0; n <= 4; ++n)
    if (a.gs == per << n) {
      a.in_lanes = 1;
      a.gshift = n;
    }
  if (!a.in_lanes)
    while ((c->groups << (a.gshift + 1)) <= 64) ++a.gshift;
  return a;
}

// Two tokens a wave, where their slots and groups lie within 32 lanes and there are
// enough of them: 256 experts, 8 groups, topk 8, sigmoid and bias, one and two a wave:
// 1024 tokens 5.4 and 5.8 us, 2048 5.4 and 5.3, 4096 7.3 and 6.5, 8192 10.7 and 8.0,
// 32768 27.9 and 20.3 (64 experts, topk 6: 18.8 and 12.0).
bool in_pairs(const Router& a) {
  return a.bias && a.sigmoid && a.tokens >= kPairTokens && a.E <= 256 && a.topk <= 32 &&
         (!a.choose_groups || (a.in_lanes && a.gshift > 0));
}
// By the logits alone (but for a softmax without renorm, whose sum over the experts would
// run in another order) at any number of tokens: the rounds are shorter than those of a
// wave a token (64 experts, topk 6: 8 tokens 3.2 us and one a wave 3.6, 8192 4.5 and
// 6.4, 32768 9.3 and 16.2; 256 experts, topk 8: 3.7 and 4.4, 5.8 and 8.7, 13.2 and
// 23.8).  With fp32 logits eight experts a lane are too many to sort with their indices
// (256 experts: 5.8 and 4.3).
bool top_in_pairs(const Router& a) {
  return !a.bias && !a.choose_groups && (a.sigmoid || a.renorm) && a.topk <= 32;
}

// In the backward wherever no sum over a token's experts is formed (its order would
// change): 256 experts, topk 8, softmax renormalised, one and two a wave: 2048 tokens
// 3.9 and 4.3 us, 4096 4.8 and 4.8, 8192 6.3 and 5.7, 32768 16.0 and 13.9 (64 experts,
// topk 6: 3.6 and 3.7, 4.2 and 3.9, 5.2 and 4.5, 12.5 and 8.7).
bool back_in_pairs(const Router& a) {
  return (a.sigmoid || a.renorm) && a.tokens >= kPairTokensBack && a.E <= 256 && a.topk <= 32;
}

dim3 grid_of(int64_t blocks) {
  return dim3(static_cast<unsigned>(std::min(blocks, kRowBlocks)),
              static_cast<unsigned>((blocks + kRowBlocks - 1) / kRowBlocks));
}

template <bool BACK, int EPL, class L>
hipError_t launch(const Router& a, hipStream_t st) {
  const dim3 one = grid_of((a.tokens + kWaves - 1) / kWaves);
  const dim3 two = grid_of((a.tokens + 2 * kWaves - 1) / (2 * kWaves));
  const dim3 block(64 * kWaves);
  if constexpr (EPL <= 4) {
    void (*pairs)(Router) = nullptr;
    if constexpr (BACK) {
      if (back_in_pairs(a)) pairs = k_router_bwd<32, 2 * EPL, L>;
    } else {
      if (in_pairs(a)) pairs = k_router_fwd_pairs<2 * EPL, L>;
      if constexpr (2 * EPL <= 4 || sizeof(L) == 2)
        if (top_in_pairs(a)) pairs = k_router_top_pairs<2 * EPL, L>;
    }
    if (pairs) {
      hipLaunchKernelGGL(pairs, two, block, 0, st, a);
      return hipGetLastError();
    }
  }
  if constexpr (BACK)
    hipLaunchKernelGGL((k_router_bwd<64, EPL, L>), one, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_router_fwd<EPL, L>), one, block,
                       a.choose_groups && !a.in_lanes ? kWaves * a.E * sizeof(double) : 0, st, a);
  return hipGetLastError();
}

template <bool BACK, class L>
int dispatch(const Router& a, hipStream_t st) {
  hipError_t e;
  switch (lane_experts(a.E)) {
    case 1: e = launch<BACK, 1, L>(a, st); break;
    case 2: e = launch<BACK, 2, L>(a, st); break;
    case 4: e = launch<BACK, 4, L>(a, st); break;
    case 8: e = launch<BACK, 8, L>(a, st); break;
    default: e = launch<BACK, 16, L>(a, st);
  }
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

}  // namespace

}  // namespace qnf4

using namespace qnf4;

extern "C" {

int qlora_router_fwd(const void* logits, int logits_fp32, int64_t tokens, int E,
                     const float* bias, const qlora_router_config* cfg, int32_t* ids,
                     float* weights, qlora_stream_t stream) {
  const int st = check_router(tokens, E, cfg);
  if (st) return st;
  if (tokens > 0 && (!logits || !ids || !weights)) return QLORA_ERR_NULL;
  if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return QLORA_ERR_ALIGN;
  if (tokens == 0) return QLORA_OK;
  Router a = router(logits, tokens, E, cfg);
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  return logits_fp32 ? dispatch<false, float>(a, hs) : dispatch<false, uint16_t>(a, hs);
}

int qlora_router_bwd(const float* dweights, const void* logits, int logits_fp32,
                     const int32_t* ids, int64_t tokens, int E, const qlora_router_config* cfg,
                     void* dlogits, qlora_stream_t stream) {
  const int st = check_router(tokens, E, cfg);
  if (st) return st;
  if (tokens > 0 && (!dweights || !logits || !ids || !dlogits)) return QLORA_ERR_NULL;
  const uintptr_t size = logits_fp32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(ids, 4) ||
      !aligned(dweights, 4))
    return QLORA_ERR_ALIGN;
  if (tokens == 0) return QLORA_OK;
  Router a = router(logits, tokens, E, cfg);
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  return logits_fp32 ? dispatch<true, float>(a, hs) : dispatch<true, uint16_t>(a, hs);
}

}  // extern "C"
