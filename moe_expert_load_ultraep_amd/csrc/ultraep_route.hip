// gfx950 kernels of the routing to experts and its gradients
// (include/ultraep_layer.h).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "ultraep_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr double kNone = -__builtin_huge_val();  // key of an expert that is never chosen

// A logit as the definition takes it: masked ones (-inf, NaN) are -inf, +inf is FLT_MAX.
__device__ __forceinline__ float clean_logit(float l) { return l != l ? -__builtin_huge_valf() : fminf(l, FLT_MAX); }

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
  return clean_logit(a.bf16 ? bf16_lo(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at]);
}

// The lanes of a wave see each other's LDS.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float f32_of(uint32_t bits) { return __builtin_bit_cast(float, bits); }

__device__ __forceinline__ bool masked(float l) { return l == -__builtin_huge_valf(); }

// Softmax: largest logit and 1 / sum.
struct Soft {
  double m, inv;
};

// Of one token's logits, by one wave.
__device__ __forceinline__ Soft soft_of(const RouteArgs& a, int64_t t) {
  float m = -__builtin_huge_valf();
  for (int32_t e = lane_id(); e < a.E; e += 64) m = fmaxf(m, load_logit(a, t * a.E + e));
  Soft s{wave_max_f64(static_cast<double>(m)), 0.0};
  double sum = 0.0;
  for (int32_t e = lane_id(); e < a.E; e += 64) {
    const float l = load_logit(a, t * a.E + e);
    if (!masked(l)) sum += exp(static_cast<double>(l) - s.m);
  }
  s.inv = 1.0 / wave_sum_f64(sum);
  return s;
}

__device__ __forceinline__ double score_of(bool sigmoid, float l, const Soft& s) {
  if (masked(l)) return 0.0;
  const double x = static_cast<double>(l);
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - s.m) * s.inv;
}

// Weights of the chosen experts, one a lane (some: this lane has one, of logit l and
// score s).  Renormalised sigmoids are taken over a common factor, so that their sum
// is never zero.
__device__ __forceinline__ double weight_of(const RouteArgs& a, bool some, float l, double s) {
  if (!a.renorm) return some ? a.scale * s : 0.0;
  const double x = static_cast<double>(l);
  double m = wave_max_f64(some ? x : kNone), t;
  if (a.sigmoid) {
    m = fmin(m, 0.0);
    t = x > 0.0 ? exp(-m) / (1.0 + exp(-x)) : exp(x - m) / (1.0 + exp(x));
  } else {
    t = exp(x - m);
  }
  if (!some) t = 0.0;
  const double sum = wave_sum_f64(t);
  return some ? a.scale * t / sum : 0.0;
}

// One token by one wave, all in fp64.  keys: E fp64 of the wave's own, expert e's written
// and read by lane e % 64 (but for the groups').
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* keys, int32_t* __restrict__ topk_idx,
                                            float* __restrict__ topk_w) {
  const int lane = lane_id();
  Soft soft{0.0, 0.0};
  if (!a.sigmoid) soft = soft_of(a, t);
  // logits (and biases) of four experts at once, as this is mostly waiting
  const bool sums = a.groups > 1 && a.group_top == 2;  // of scores, also where the keys are the logits
  for (int32_t e0 = lane; e0 < a.E; e0 += 256) {
    float l[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t e = min(e0 + 64 * i, a.E - 1);
      l[i] = load_logit(a, t * a.E + e);
      b[i] = a.bias != nullptr ? a.bias[e] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double key = static_cast<double>(l[i]);
      if (!masked(l[i]) && (sums || a.bias != nullptr)) key = score_of(a.sigmoid, l[i], soft) + static_cast<double>(b[i]);
      if (e0 + 64 * i < a.E) keys[e0 + 64 * i] = key == key ? key : kNone;
    }
  }
  if (a.groups > 1) {
    const int32_t per = a.E / a.groups;
    wave_sync();
    double first = kNone, second = kNone;
    if (lane < a.groups) {
#pragma unroll 8
      for (int i = 0; i < per; ++i) {
        const double x = keys[lane * per + i];
        second = fmax(second, fmin(first, x));
        first = fmax(first, x);
      }
    }
    const double worth = a.group_top == 2 && second != kNone ? first + second : first;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double x = readlane_f64(worth, g);
      rank += x > worth || (x == worth && g < lane);
    }
    const uint64_t taken = ballot(lane < a.groups && worth != kNone && rank < a.topk_groups);
    wave_sync();
    for (int32_t e = lane; e < a.E; e += 64) {
      if (sums && a.bias == nullptr && keys[e] != kNone) keys[e] = static_cast<double>(load_logit(a, t * a.E + e));
      if (!((taken >> (e / per)) & 1)) keys[e] = kNone;
    }
  }
  int32_t mine = -1;  // lane j: the j-th expert
  for (int j = 0; j < a.k; ++j) {
    double best = kNone;
    int32_t at = lane;
#pragma unroll 4
    for (int32_t e = lane; e < a.E; e += 64) {
      const double x = keys[e];
      if (x > best) {
        best = x;
        at = e;
      }
    }
    const double top = wave_max_f64(best);
    if (top == kNone) break;  // the same in every lane
    const int32_t win = static_cast<int32_t>(~wave_max(best == top ? ~static_cast<uint32_t>(at) : 0u));  // the lowest id
    if (lane == j) mine = win;
    if (lane == win % 64) keys[win] = kNone;
  }
  const bool some = mine >= 0;
  const float lj = some ? load_logit(a, t * a.E + mine) : 0.f;
  const double w = weight_of(a, some, lj, score_of(a.sigmoid, lj, soft));
  if (lane < a.k) {
    topk_idx[t * a.k + lane] = mine;
    topk_w[t * a.k + lane] = static_cast<float>(w);
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, int32_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_w) {
  extern __shared__ double s_keys[];
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; t < a.tokens; t += nwaves)
    route_token(a, t, s_keys + wv * a.E, topk_idx, topk_w);
}

// ---------------------------------------------------------------------------
// Many tokens a wave.  LPT lanes have a token, four experts of every 4 * LPT each, and
// find its experts by 32-bit keys: the fp32 key as a whole number of 24 (23) bits, above
// the expert's id (complemented, so that the lower id is the larger key).  One
// v_med3_u32 a place keeps a sorted list, lists are merged across the lanes, and
// nothing has to be looked up afterwards.  Where two keys that the choice or its order
// hangs on are nearer than their errors can be, these two are compared in fp64, and where
// that does not settle it the token is done again (route_token): the ids are always those
// of fp64.
// Errors in units of 2^-24 (of the keys' range, which is at least 1): v_exp_f32 and
// v_rcp_f32 are off by a step, so a sigmoid by 3.9, a softmax by 27 with its sum; bias,
// fma and the cut to whole numbers add 2.5.  Bound by instructions: 262144 tokens of 256
// experts in 8 groups, 285 MB, 102 us (55 at the rate of a large copy; 95 without any
// token done again), vector instructions at work in 80 % of the SIMDs' time, LDS in 14 %,
// its bank conflicts 6 %; 524288 of 128 without groups, 302 MB, 75 us.  One wave a token, all in
// fp64: 616 and 821.  Logits read a round ahead: 106 and 83, as the chosen ones, read
// again for their weights, have left the L2 by then.
template <int LPT, int NI>
struct Packed {
  static constexpr int kIdBits = LPT * NI * 4 <= 256 ? 8 : 9;
  static constexpr uint32_t kIds = (1u << kIdBits) - 1;
  static constexpr float kTop = static_cast<float>(1u << (32 - kIdBits));  // values are below
};

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// The whole part; 0 of NaN and of what is below 0 (which a C++ conversion does not promise).
__device__ __forceinline__ uint32_t whole(float x) {
  uint32_t r;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(r) : "v"(x));
  return r;
}

// x into the descending list a, of whose first FROM values all are at least x.
template <int FROM, int KL>
__device__ __forceinline__ void insert(uint32_t (&a)[KL], uint32_t x) {
#pragma unroll
  for (int i = KL - 1; i > FROM; --i) a[i] = med3(a[i - 1], a[i], x);
  a[FROM] = max(a[FROM], x);
}

template <int J, int KL>
__device__ __forceinline__ void insert_all(uint32_t (&a)[KL], const uint32_t (&b)[KL]) {
  if constexpr (J < KL) {
    insert<J>(a, b[J]);
    insert_all<J + 1>(a, b);
  }
}

// The LPT lanes of a token, step by step: each step's partner has another part.
template <int LPT, typename F>
__device__ __forceinline__ void across_lanes(F&& step) {
  step(std::integral_constant<int, 0xB1>{});                      // quad_perm [1,0,3,2]
  step(std::integral_constant<int, 0x4E>{});                      // quad_perm [2,3,0,1]
  if constexpr (LPT > 4) step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  if constexpr (LPT > 8) step(std::integral_constant<int, 0x140>{});  // row_mirror
}

template <int LPT>
__device__ __forceinline__ float token_max(float x) {
  across_lanes<LPT>([&](auto c) { x = fmaxf(x, dppf<decltype(c)::value>(x)); });
  return x;
}
template <int LPT>
__device__ __forceinline__ float token_min(float x) {
  across_lanes<LPT>([&](auto c) { x = fminf(x, dppf<decltype(c)::value>(x)); });
  return x;
}
template <int LPT>
__device__ __forceinline__ float token_sum(float x) {
  across_lanes<LPT>([&](auto c) { x += dppf<decltype(c)::value>(x); });
  return x;
}
template <int LPT>
__device__ __forceinline__ uint32_t token_or(uint32_t x) {
  across_lanes<LPT>([&](auto c) { x |= dpp<decltype(c)::value>(x); });
  return x;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFastGroups = 16;
constexpr float kLogitRange = 16.f;  // of a row's logits, from its largest down, that keys tell apart

__device__ __forceinline__ float fast_sigmoid(float l) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * l));
}

// Words of a token's row of keys in LDS: 16 more than a multiple of 64, so that the rows
// of neighbouring tokens start in different banks.
__host__ __device__ inline int32_t key_pitch(int32_t E) { return E + ((16 - E) & 63); }  // a multiple of 16

struct KeyUnits {
  float c;        // units of a score
  float one;      // units that a sum of two keys is above a single key of the same worth
  float fine;     // keys in fp64 nearer than this may be in another order by their own rounding
  bool exact;     // the bias spans too much for them, or is too large
};

// The bias in units of the keys, in LDS; absent experts' are NaN, which gives no key.
template <int LPT, int NI>
__device__ __forceinline__ KeyUnits bias_units(const RouteArgs& a, float* table) {
  __shared__ float s_lo[kRouteWaves], s_hi[kRouteWaves];
  constexpr int kAll = LPT * NI * 4;
  const int tid = threadIdx.x;
  float lo = __builtin_huge_valf(), hi = -__builtin_huge_valf();
  for (int e = tid; e < a.E; e += kRouteThreads) {
    const float b = a.bias[e];
    if (b > -__builtin_huge_valf()) {  // not NaN either
      lo = fminf(lo, b);
      hi = fmaxf(hi, b);
    }
  }
  lo = token_min<16>(lo);
  hi = token_max<16>(hi);
  lo = fminf(fminf(readlane_f(lo, 0), readlane_f(lo, 16)), fminf(readlane_f(lo, 32), readlane_f(lo, 48)));
  hi = fmaxf(fmaxf(readlane_f(hi, 0), readlane_f(hi, 16)), fmaxf(readlane_f(hi, 32), readlane_f(hi, 48)));
  if (lane_id() == 0) {
    s_lo[tid >> 6] = lo;
    s_hi[tid >> 6] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRouteWaves; ++i) {
    lo = fminf(lo, s_lo[i]);
    hi = fmaxf(hi, s_hi[i]);
  }
  const float span = hi - lo + 1.f;
  // Sums with a bias are rounded to 2^-53 of it, which below 2^20 is far less than a unit;
  // two sums of two of them, to 2^-50.
  const float size = fmaxf(-lo, hi);
  KeyUnits u{(Packed<LPT, NI>::kTop - 64.f) / span, 0.f, 0x1p-40f + size * 0x1p-49f, !(span < 1e4f && size < 0x1p20f)};
  u.one = 8.f - lo * u.c;
  for (int e = tid; e < kAll; e += kRouteThreads) {
    const float b = e < a.E ? a.bias[e] : __builtin_nanf("");
    table[e] = b > -__builtin_huge_valf() ? (b - lo) * u.c + 8.f : __builtin_nanf("");
  }
  __syncthreads();
  return u;
}

// Key of e0 less that of e1 in fp64, for the token whose logits start at `row`.  A softmax
// is taken by its sum in fp32 (inv, its inverse), off by less than 2^-19: where that could
// decide, the answer is not sure.
__device__ __forceinline__ double exact_difference(const RouteArgs& a, int64_t row, int32_t e0, int32_t e1, float top, float inv,
                                                   float fine, bool& sure) {
  const double l0 = static_cast<double>(load_logit(a, row + e0)), l1 = static_cast<double>(load_logit(a, row + e1));
  if (a.bias == nullptr) return l0 - l1;
  const double b = static_cast<double>(a.bias[e0]) - static_cast<double>(a.bias[e1]);
  if (a.sigmoid) {  // as the definition adds them, so that equal ones are equal
    const double k0 = score_of(true, static_cast<float>(l0), Soft{}) + static_cast<double>(a.bias[e0]);
    const double k1 = score_of(true, static_cast<float>(l1), Soft{}) + static_cast<double>(a.bias[e1]);
    return k0 - k1;
  }
  const double s = (exp(l0 - top) - exp(l1 - top)) * inv, d = s + b;
  sure = fabs(d) > fabs(s) * 0x1p-19 + fine;
  return d;
}

// Words of LDS a wave has for itself: keys and worths of its tokens' groups, or E fp64.
template <int LPT>
__host__ __device__ inline int32_t wave_words(const RouteArgs& a) {
  return a.groups > 1 ? 64 / LPT * (key_pitch(a.E) + kFastGroups) : 2 * a.E;
}

// Workgroups that fit a CU by the registers they are given.
template <int LPT, int NI>
constexpr int kRouteFit = NI > 10 ? 3 : 4;

template <int LPT, int NI, int KL>
__global__ __launch_bounds__(kRouteThreads, (kRouteFit<LPT, NI>)) void route_fast_kernel(RouteArgs a, int32_t* __restrict__ topk_idx,
                                                                   float* __restrict__ topk_w) {
  extern __shared__ __align__(16) char s_dyn[];
  using P = Packed<LPT, NI>;
  constexpr int kTokens = 64 / LPT, kAll = LPT * NI * 4, MM = (KL - 2 + LPT - 1) / LPT;  // KL: k + 2 or more
  constexpr float kHigh = P::kTop - 64.f, kPerLogit = kHigh / kLogitRange;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t per = a.E / a.groups, pitch = key_pitch(a.E);
  float* bias = reinterpret_cast<float*>(s_dyn);  // [kAll]
  uint32_t* keys = reinterpret_cast<uint32_t*>(s_dyn) + kAll + wv * wave_words<LPT>(a);
  float* worths = reinterpret_cast<float*>(keys + kTokens * pitch);
  const bool with_bias = a.bias != nullptr;
  const bool in_fours = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 8 == 0;  // bf16
  KeyUnits units{0.f, 0.f, 0.f, false};
  if (with_bias) units = bias_units<LPT, NI>(a, bias);
  // what two keys have to be apart for their order to be certain, in units
  const uint32_t margin = with_bias ? (a.sigmoid ? (P::kIdBits == 8 ? 13u : 9u) : (P::kIdBits == 8 ? 64u : 40u)) : a.bf16 ? 0u : 8u;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  float l[4 * NI];
  // A batch's logits through one resource: an address a lane, chunks at constant
  // distances; what is behind a row is the next one's, or zeros behind the last.
  const auto load = [&](int64_t batch, int lane, int32_t E) {
    const int q = lane % LPT, tl = lane / LPT, size = a.bf16 ? 2 : 4;
    const int64_t left = min(a.tokens - batch * kTokens, static_cast<int64_t>(kTokens));
    const __amdgpu_buffer_rsrc_t rows = row_rsrc(static_cast<const char*>(a.logits) + batch * kTokens * E * size,
                                                 left > 0 ? static_cast<uint32_t>(left * E * size) : 0u);
    const int from = (tl * E + 4 * q) * size;
    if (!a.bf16) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rows, from + i * LPT * 16, 0, 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) l[4 * i + c] = f32_of(v[c]);
      }
    } else if (in_fours) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rows, from + i * LPT * 8, 0, 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) l[4 * i + c] = c & 1 ? bf16_hi(v[c / 2]) : bf16_lo(v[c / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NI; ++i)
        l[i] = bf16_lo(__builtin_amdgcn_raw_buffer_load_b16(rows, from + (i / 4 * LPT * 4 + i % 4) * 2, 0, 0));
    }
  };
  int64_t batch = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv;
  for (; batch * kTokens < a.tokens; batch += step) {
    // Made anew in every round: what hangs on them is cheap, and kept in registers (a
    // few for every expert of the lane) would push the logits out.
    int lane = lane_id();
    int32_t E = a.E;
    asm volatile("" : "+v"(lane), "+s"(E));
    const int q = lane % LPT, tl = lane / LPT;
    const int64_t t = batch * kTokens + tl;
    // (Not a round ahead: the chosen ones are read again, and should be in the L2 still.)
    load(batch, lane, E);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if ((i + 1) * LPT * 4 > E) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((i * LPT + q) * 4 + c >= E) l[4 * i + c] = -__builtin_huge_valf();
      }
    float top = -__builtin_huge_valf(), inv = 0.f;
    bool again = units.exact;
    if (!(with_bias && a.sigmoid)) {
#pragma unroll
      for (int i = 0; i < 4 * NI; ++i) top = fmaxf(top, l[i]);
      top = token_max<LPT>(top);
      again |= top == __builtin_huge_valf();
    }
    if (!a.sigmoid && (with_bias || !a.renorm)) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4 * NI; ++i) sum[i % 4] += __builtin_amdgcn_exp2f((l[i] - top) * kLog2e);
      const float total = token_sum<LPT>((sum[0] + sum[1]) + (sum[2] + sum[3]));
      again |= total != total && top > -__builtin_huge_valf();  // a NaN among them
      inv = 1.f / total;
    }
    // Keys, of values that are numbers: into LDS where there are groups, else into the
    // lane's list.  Not everything at once, which would take more registers than there are.
    uint32_t list[KL];
#pragma unroll
    for (int j = 0; j < KL; ++j) list[j] = 0;
    const int ids = static_cast<int>(P::kIds) - 4 * q;
    const auto make_keys = [&](auto&& values) {  // of a chunk
      const auto chunk = [&](int i, uint32_t (&key)[4]) {
        float x[4];
        values(i, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) key[c] = (whole(x[c]) << P::kIdBits) | static_cast<uint32_t>(ids - (i * LPT * 4 + c));
        if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      };
      if (a.groups > 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint32_t key[4];
          chunk(i, key);
          if ((i * LPT + q) * 4 < E)
            *reinterpret_cast<u32x4*>(keys + tl * pitch + (i * LPT + q) * 4) = u32x4{key[0], key[1], key[2], key[3]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint32_t key[4];
          chunk(i, key);
#pragma unroll
          for (int c = 0; c < 4; ++c) insert<0>(list, key[c]);
        }
      }
    };
    const auto logit_value = [&](float x) { return __builtin_fmaf(x - top, kPerLogit, kHigh); };  // NaN or below 0: 0
    if (with_bias) {
      float low = l[0];
#pragma unroll
      for (int i = 1; i < 4 * NI; ++i) low = fminf(low, l[i]);
      if (ballot(low == -__builtin_huge_valf()) != 0) {  // a masked expert's score is 0, which would be a key
#pragma unroll
        for (int i = 0; i < 4 * NI; ++i) l[i] = masked(l[i]) ? __builtin_nanf("") : l[i];
      }
      const float* b = bias + 4 * q;
      if (a.sigmoid)
        make_keys([&](int i, float (&x)[4]) {
          const f32x4 add = *reinterpret_cast<const f32x4*>(b + i * LPT * 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = __builtin_fmaf(fast_sigmoid(l[4 * i + c]), units.c, add[c]);
        });
      else
        make_keys([&](int i, float (&x)[4]) {
          const f32x4 add = *reinterpret_cast<const f32x4*>(b + i * LPT * 4);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            x[c] = __builtin_fmaf(__builtin_amdgcn_exp2f((l[4 * i + c] - top) * kLog2e) * inv, units.c, add[c]);
        });
    } else if (a.bf16) {
      // the 16 bits themselves, in ascending order: nothing is lost
      make_keys([&](int i, float (&x)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float y = l[4 * i + c];
          uint32_t u = __builtin_bit_cast(uint32_t, y == 0.f ? 0.f : y);
          u ^= static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u;
          x[c] = y > -__builtin_huge_valf() ? static_cast<float>((u >> 16) + 1) : 0.f;
        }
      });
    } else {
      make_keys([&](int i, float (&x)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = logit_value(l[4 * i + c]);
      });
    }
    if (a.groups > 1) {
      wave_sync();
      constexpr int kOwn = (kFastGroups + LPT - 1) / LPT;
      constexpr float kNoWorth = -__builtin_huge_valf();  // of a group without an expert to choose
      float worth[kOwn];
      uint32_t alone = 0;  // is there a group with one expert to choose, where others may have two?
      const uint32_t* row = keys + tl * pitch;
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) {
        const int g = gi * LPT + q;
        worth[gi] = kNoWorth;
        if (gi * LPT < a.groups) {
          uint32_t first = 0, second = 0;
          if (g < a.groups) {
            const auto see = [&](uint32_t x) {
              second = med3(first, second, x);
              first = max(first, x);
            };
            if (per % 4 == 0) {
              for (int j = 0; j < per; j += 4) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(row + g * per + j);
                see(x[0]), see(x[1]), see(x[2]), see(x[3]);
              }
            } else {
              for (int j = 0; j < per; ++j) see(row[g * per + j]);
            }
          }
          first >>= P::kIdBits;
          second >>= P::kIdBits;
          if (first != 0) {
            if (a.group_top == 1) {
              worth[gi] = static_cast<float>(first);
            } else if (with_bias) {
              worth[gi] = static_cast<float>(first + second);
              if (second == 0 && per > 1) {
                worth[gi] += units.one;
                alone = 1;
              }
            } else {  // scores of the two logits, up to the softmax's common factor
              float s = 0.f;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t v = k == 0 ? first : second;
                float x;
                if (a.bf16) {
                  uint32_t u = (v - 1) << 16;
                  u ^= (static_cast<uint32_t>(~(static_cast<int32_t>(u) >> 31)) | 0x80000000u) & 0xFFFF0000u;
                  x = __builtin_bit_cast(float, u);
                } else {
                  x = top + (static_cast<float>(v) - kHigh) * (1.f / kPerLogit);
                }
                const float y = a.sigmoid ? fast_sigmoid(x) : __builtin_amdgcn_exp2f((x - top) * kLog2e);
                if (v != 0) s += y;
              }
              worth[gi] = s;
            }
          }
          if (g < a.groups) worths[tl * kFastGroups + g] = worth[gi];
        }
      }
      wave_sync();
      int rank[kOwn];
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) rank[gi] = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float x = worths[tl * kFastGroups + g];
#pragma unroll
        for (int gi = 0; gi < kOwn; ++gi)
          if (gi * LPT < a.groups) rank[gi] += x > worth[gi] || (x == worth[gi] && g < gi * LPT + q);
      }
      uint32_t taken = 0;
      float in = __builtin_huge_valf(), out = -__builtin_huge_valf();
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) {
        const bool mine = worth[gi] > kNoWorth, take = mine && rank[gi] < a.topk_groups;
        if (take) taken |= 1u << (gi * LPT + q);
        if (take) in = fminf(in, worth[gi]);
        if (mine && !take) out = fmaxf(out, worth[gi]);
      }
      taken = token_or<LPT>(taken);
      float apart = static_cast<float>(margin);
      if (a.group_top == 2 && with_bias) {
        apart = 2.f * apart + 4.f;
        if (token_or<LPT>(alone) != 0) apart += fabsf(units.one) * 0x1p-22f;  // it is rounded twice, its sum once
      }
      if (a.group_top == 2 && !with_bias) {
        apart = 1e-5f;
        if (!a.bf16) {  // logits below the keys' range have scores up to this
          if (a.sigmoid) apart += 2.f * fast_sigmoid(top - kLogitRange);
          out = fmaxf(out, 0.f);
        }
      }
      in = token_min<LPT>(in);
      out = token_max<LPT>(out);
      const bool unsure = in - out < apart && t < a.tokens;  // the last that stays and the first that goes
      if (ballot(unsure) != 0) {
        // These two in fp64, one by the token's first lane and one by its second, where no
        // third is close to them nor to the two experts that their keys are made of.
        float better = __builtin_huge_valf(), worse = -__builtin_huge_valf();
        uint32_t ids[2] = {0, 0};
#pragma unroll
        for (int gi = 0; gi < kOwn; ++gi) {
          if (worth[gi] == kNoWorth) continue;
          const int r = rank[gi] - a.topk_groups, g = gi * LPT + q;
          if (r == -2) better = worth[gi];
          if (r == 1) worse = worth[gi];
          if (r == -1) ids[0] = g + 1;
          if (r == 0) ids[1] = g + 1;
        }
        const int32_t g0 = static_cast<int32_t>(token_or<LPT>(ids[0])) - 1, g1 = static_cast<int32_t>(token_or<LPT>(ids[1])) - 1;
        bool sure = token_min<LPT>(better) - out >= apart && in - token_max<LPT>(worse) >= apart && g0 >= 0 && g1 >= 0 &&
                    (with_bias || a.bf16 || in >= apart);
        double s = 0.0, b = 0.0;
        float l0 = -__builtin_huge_valf(), l1 = l0;
        if (unsure && sure && q < 2) {
          uint32_t k[3] = {0, 0, 0};
          const uint32_t* group = row + (q == 0 ? g0 : g1) * per;
          for (int j = 0; j < per; ++j) insert<0>(k, group[j]);
          const int n = a.group_top;
          const uint32_t x = (n == 1 ? k[0] : k[1]) >> P::kIdBits, y = (n == 1 ? k[1] : k[2]) >> P::kIdBits;
          // (A key of 0 is no expert; of fp32 logits without a bias it may be one below the keys' range.)
          sure = per == 1 || (y == 0 && (with_bias || a.bf16)) || x - y >= margin;
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            const uint32_t key = i == 0 ? k[0] : k[1];
            if ((key >> P::kIdBits) == 0) continue;
            const int32_t e = static_cast<int32_t>(P::kIds - (key & P::kIds));
            const float l = load_logit(a, t * E + e);
            if (i == 0)
              l0 = l;
            else
              l1 = l;
            const double score = n == 1 && !with_bias ? static_cast<double>(l) : score_of(a.sigmoid, l, Soft{static_cast<double>(top), 1.0});
            const double add = with_bias ? static_cast<double>(a.bias[e]) : 0.0;
            s += a.sigmoid ? score + add : score;
            b += add;
          }
        }
        const int first = lane - q;
        const double s0 = __shfl(s, first), s1 = __shfl(s, first + 1), b0 = __shfl(b, first), b1 = __shfl(b, first + 1);
        sure = __shfl(static_cast<int>(sure), first) != 0 && __shfl(static_cast<int>(sure), first + 1) != 0;
        double d = s0 - s1;  // of a softmax without its common factor
        if (!a.sigmoid && with_bias) {
          const double scores = d * inv;
          d = scores + (b0 - b1);
          sure = sure && fabs(d) > fabs(scores) * 0x1p-19 + units.fine;
        } else if (!a.sigmoid && a.group_top == 2) {
          // (the common factor rounds the scores, so they need not be equal where d is 0)
          const bool same = __shfl(l0, first) == __shfl(l0, first + 1) && __shfl(l1, first) == __shfl(l1, first + 1);
          sure = sure && (same || fabs(d) > 0x1p-40);
        }
        if (unsure && sure && (d < 0.0 || (d == 0.0 && g1 < g0))) taken ^= (1u << g0) | (1u << g1);
        again |= unsure && !sure;
      }
      for (int s = 0; s < a.topk_groups; ++s) {
        const bool some = taken != 0;
        const int g = some ? __builtin_ctz(taken) : 0;
        taken &= taken - 1;
        if (per % 4 == 0) {
          for (int j = 4 * q; j < per; j += 4 * LPT) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(row + g * per + j);
#pragma unroll
            for (int c = 0; c < 4; ++c) insert<0>(list, some ? x[c] : 0u);
          }
        } else {
          for (int j = q; j < per; j += LPT) insert<0>(list, some ? row[g * per + j] : 0u);
        }
      }
    }
    across_lanes<LPT>([&](auto ctrl) {
      uint32_t other[KL];
#pragma unroll
      for (int j = 0; j < KL; ++j) other[j] = dpp<decltype(ctrl)::value>(list[j]);
      insert_all<0>(list, other);
    });
    // Is every order that counts certain?  One that is not is settled by the two keys in
    // fp64; more, or one whose lower is close to a third, are for route_token.
    uint32_t last = 0, close = 0, upper = 0, lower = 0;
    int place = 0;
    bool before = false;
#pragma unroll
    for (int j = 0; j < KL - 1; ++j) {
      if (j > a.k) continue;
      const uint32_t x = list[j] >> P::kIdBits, y = list[j + 1] >> P::kIdBits;
      const bool near = y != 0 && x - y < margin;
      again |= near && before;
      before = near;
      if (j == a.k) continue;
      last = x;
      if (near) {
        close += 1;
        place = j;
        upper = list[j];
        lower = list[j + 1];
      }
    }
    again |= close > 1;
    const bool settle = close == 1 && !again && t < a.tokens;
    if (ballot(settle) != 0) {
      const int32_t e0 = static_cast<int32_t>(P::kIds - (upper & P::kIds)), e1 = static_cast<int32_t>(P::kIds - (lower & P::kIds));
      bool sure = true;
      const double d = settle ? exact_difference(a, t * E, e0, e1, top, inv, units.fine, sure) : 0.0;
      again |= settle && !sure;
      const bool swap = settle && (d < 0.0 || (d == 0.0 && e1 < e0));
#pragma unroll
      for (int j = 0; j < KL - 1; ++j) {
        if (swap && j == place) {
          list[j] = lower;
          list[j + 1] = upper;
        }
      }
    }
    // fewer than k, though not all are masked: are there any below the keys' range?
    const bool few = !with_bias && last < margin && !masked(top) && t < a.tokens;
    if (ballot(few) != 0) {
      uint32_t unseen = 0;
      for (int e = q; e < E && few; e += LPT) {
        const float x = load_logit(a, t * E + e);
        unseen |= !masked(x) && logit_value(x) < static_cast<float>(margin);
      }
      again |= few && token_or<LPT>(unseen) != 0;
    }
    // weights
    int32_t e_j[MM];
    float l_j[MM], w[MM];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int mm = 0; mm < MM; ++mm) {
      uint32_t k_j = 0;
#pragma unroll
      for (int c = 0; c < LPT; ++c)
        if (mm * LPT + c < KL - 2) k_j = q == c ? list[mm * LPT + c < KL ? mm * LPT + c : 0] : k_j;
      const bool some = (k_j >> P::kIdBits) != 0 && mm * LPT + q < a.k && t < a.tokens;
      e_j[mm] = some ? static_cast<int32_t>(P::kIds - (k_j & P::kIds)) : -1;
      l_j[mm] = some ? load_logit(a, t * E + e_j[mm]) : 0.f;
      if (some) m = fmaxf(m, l_j[mm]);
    }
    m = token_max<LPT>(m);
    float sum = 0.f;
    if (a.sigmoid) m = a.renorm ? fminf(m, 0.f) : 0.f;
    else if (!a.renorm) m = top;
    const float over = a.sigmoid ? expf(-m) : 1.f;
#pragma unroll
    for (int mm = 0; mm < MM; ++mm) {
      const float x = l_j[mm], s = expf(x > 0.f && a.sigmoid ? -x : x - m);
      w[mm] = a.sigmoid ? (x > 0.f ? over / (1.f + s) : s / (1.f + expf(x))) : s;
      if (e_j[mm] < 0) w[mm] = 0.f;
      sum += w[mm];
    }
    const float factor = a.scale * (a.renorm ? 1.f / token_sum<LPT>(sum) : a.sigmoid ? 1.f : inv);
    const bool write = t < a.tokens && !again;
#pragma unroll
    for (int mm = 0; mm < MM; ++mm) {
      const int j = mm * LPT + q;
      if (write && j < a.k) {
        topk_idx[t * a.k + j] = e_j[mm];
        topk_w[t * a.k + j] = e_j[mm] < 0 ? 0.f : w[mm] * factor;
      }
    }
    wave_sync();
    for (uint64_t redo = ballot(again && q == 0 && t < a.tokens); redo != 0; redo &= redo - 1)
      route_token(a, batch * kTokens + __builtin_ctzll(redo) / LPT, reinterpret_cast<double*>(keys), topk_idx, topk_w);
    wave_sync();
  }
}

// ---------------------------------------------------------------------------
// Gradients.  LPT lanes have a token, lane q its chosen experts j = q, q + LPT, ...; the
// tokens' rows are put together in LDS and go out as one stream of whole lines.  Bound by
// HBM: 262144 tokens of 256 experts write 268 MB and read the lines of the eight chosen
// logits, two thirds of all: 83 us (one wave a token, rows in registers: 224).
template <int LPT>
__host__ __device__ inline int32_t grad_words(int32_t E) { return 64 / LPT * key_pitch(E); }

// Where the same id stands more than once in a row, the first takes all their gradients,
// added up in the order of the row, and the others none.
template <int LPT, int MM>
__device__ __forceinline__ void merge_same(int32_t (&e)[MM], float (&d)[MM]) {
  const int lane = lane_id(), q = lane % LPT, first = lane - q;
  float sum[MM];
  bool later[MM];
#pragma unroll
  for (int mm = 0; mm < MM; ++mm) sum[mm] = 0.f, later[mm] = false;
#pragma unroll
  for (int nn = 0; nn < MM; ++nn)
    for (int c = 0; c < LPT; ++c) {
      const int32_t other = __shfl(e[nn], first + c);
      const float x = __shfl(d[nn], first + c);
#pragma unroll
      for (int mm = 0; mm < MM; ++mm) {
        if (other != e[mm]) continue;
        sum[mm] += x;
        later[mm] |= nn * LPT + c < mm * LPT + q;
      }
    }
#pragma unroll
  for (int mm = 0; mm < MM; ++mm) {
    if (e[mm] >= 0) d[mm] = sum[mm];
    if (later[mm]) e[mm] = -1;
  }
}

template <int LPT, int MM>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a, const int32_t* __restrict__ topk_idx,
                                                                       const float* __restrict__ grad_w,
                                                                       void* __restrict__ grad_logits) {
  extern __shared__ __align__(16) float s_rows[];
  constexpr int kTokens = 64 / LPT;
  const int lane = lane_id(), q = lane % LPT, tl = lane / LPT;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t E = a.E, pitch = key_pitch(E), words = grad_words<LPT>(E);
  float* rows = s_rows + wv * words;
  float* row = rows + tl * pitch;
  const bool every = !a.sigmoid && !a.renorm;
  const bool in_fours = E % 4 == 0 && reinterpret_cast<uintptr_t>(grad_logits) % (a.bf16 ? 8 : 16) == 0;
  const bool logits_in_fours = E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (a.bf16 ? 8 : 16) == 0;
  const float per_row = 1.f / static_cast<float>(E);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  for (int64_t batch = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; batch * kTokens < a.tokens; batch += step) {
    const int64_t t = batch * kTokens + tl;
    const bool there = t < a.tokens;
    int32_t e[MM];
    float g[MM], l[MM];
#pragma unroll
    for (int mm = 0; mm < MM; ++mm) {
      const int j = mm * LPT + q;
      e[mm] = there && j < a.k ? topk_idx[t * a.k + j] : -1;
      g[mm] = there && j < a.k ? grad_w[t * a.k + j] : 0.f;
    }
#pragma unroll
    for (int mm = 0; mm < MM; ++mm) {
      if (e[mm] >= E) e[mm] = -1;
      l[mm] = e[mm] >= 0 ? load_logit(a, t * E + e[mm]) : 0.f;
      if (masked(l[mm])) e[mm] = -1;
    }
    // is an id there twice?  Each writes its place and looks whether it is still there.
#pragma unroll
    for (int mm = 0; mm < MM; ++mm)
      if (e[mm] >= 0) reinterpret_cast<int32_t*>(row)[e[mm]] = mm * LPT + q;
    wave_sync();
    bool twice = false;
#pragma unroll
    for (int mm = 0; mm < MM; ++mm)
      if (e[mm] >= 0) twice |= reinterpret_cast<int32_t*>(row)[e[mm]] != mm * LPT + q;
    wave_sync();
    // scores and weights
    float d[MM], total = 0.f, inv = 0.f;
    if (every) {
      float m = -__builtin_huge_valf(), sum = 0.f;
      for (int i = 4 * q; i < E; i += 4 * LPT) {
        f32x4 x;
        if (logits_in_fours) {
          if (a.bf16) {
            const u32x2 v = there ? *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.logits) + t * E + i) : u32x2{0, 0};
            x = f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
          } else {
            x = there ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.logits) + t * E + i) : f32x4{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = clean_logit(x[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = !there ? 0.f : i + c < E ? load_logit(a, t * E + i + c) : -__builtin_huge_valf();
        }
        *reinterpret_cast<f32x4*>(row + i) = x;
        m = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      }
      m = token_max<LPT>(m);
      if (masked(m)) m = 0.f;  // all of them
      for (int i = 4 * q; i < E; i += 4 * LPT) {
        f32x4 x = *reinterpret_cast<const f32x4*>(row + i);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = __builtin_amdgcn_exp2f((x[c] - m) * kLog2e);
        *reinterpret_cast<f32x4*>(row + i) = x;
        sum += (x[0] + x[1]) + (x[2] + x[3]);
      }
      sum = token_sum<LPT>(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
      wave_sync();
#pragma unroll
      for (int mm = 0; mm < MM; ++mm) {
        d[mm] = e[mm] >= 0 ? a.scale * (row[e[mm]] * inv) * g[mm] : 0.f;
        total += d[mm];
      }
      total = token_sum<LPT>(total);
      wave_sync();
      const float each = -inv * total;
      for (int i = 4 * q; i < E; i += 4 * LPT) *reinterpret_cast<f32x4*>(row + i) *= each;
    } else {
      float m = -__builtin_huge_valf(), sum = 0.f;
#pragma unroll
      for (int mm = 0; mm < MM; ++mm)
        if (e[mm] >= 0) m = fmaxf(m, l[mm]);
      m = token_max<LPT>(m);
      if (a.sigmoid) m = a.renorm ? fminf(m, 0.f) : 0.f;
      const float over = a.sigmoid ? expf(-m) : 1.f;
      float rest[MM], w[MM];
#pragma unroll
      for (int mm = 0; mm < MM; ++mm) {
        const float x = expf(a.sigmoid ? -fabsf(l[mm]) : l[mm] - m), big = 1.f / (1.f + x);
        rest[mm] = l[mm] > 0.f ? x * big : big;  // 1 - s
        w[mm] = a.sigmoid ? (l[mm] > 0.f ? over : expf(l[mm] - m)) * big : x;
        if (e[mm] < 0) w[mm] = 0.f;
        sum += w[mm];
      }
      const float factor = a.scale * (a.renorm ? 1.f / token_sum<LPT>(sum) : 1.f);
#pragma unroll
      for (int mm = 0; mm < MM; ++mm) {
        if (e[mm] < 0) continue;
        w[mm] *= factor;
        total += w[mm] * g[mm];
      }
      // the sum without the scale, which may be zero
      total = a.renorm ? token_sum<LPT>(total) : 0.f;
      const float back = a.renorm && a.scale != 0.f ? total / a.scale : 0.f;
#pragma unroll
      for (int mm = 0; mm < MM; ++mm) {
        d[mm] = w[mm] * (g[mm] - back);
        if (a.sigmoid) d[mm] *= rest[mm];
      }
      const u32x4 zero = {0, 0, 0, 0};
      for (int i = 4 * lane; i < words; i += 256) *reinterpret_cast<u32x4*>(rows + i) = zero;
    }
    if (__builtin_expect(ballot(twice) != 0, 0)) merge_same<LPT, MM>(e, d);
    wave_sync();
#pragma unroll
    for (int mm = 0; mm < MM; ++mm)
      if (e[mm] >= 0) row[e[mm]] = every ? row[e[mm]] + d[mm] : d[mm];
    wave_sync();
    // out, all rows of the wave as one range
    const int32_t values = static_cast<int32_t>(min(a.tokens - batch * kTokens, static_cast<int64_t>(kTokens))) * E;
    char* out = static_cast<char*>(grad_logits) + batch * kTokens * E * (a.bf16 ? 2 : 4);
    if (in_fours) {
      for (int i = 4 * lane; i < values; i += 256) {
        const int r = static_cast<int>((static_cast<float>(i) + 0.5f) * per_row);
        const f32x4 x = *reinterpret_cast<const f32x4*>(rows + i + r * (pitch - E));
        if (a.bf16) {
          const u32x2 y = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
          *reinterpret_cast<u32x2*>(out + 2 * i) = y;
        } else {
          *reinterpret_cast<f32x4*>(out + 4 * i) = x;
        }
      }
    } else {
      for (int i = lane; i < values; i += 64) {
        const int r = static_cast<int>((static_cast<float>(i) + 0.5f) * per_row);
        const float x = rows[i + r * (pitch - E)];
        if (a.bf16)
          reinterpret_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack_bf16(x, 0.f));
        else
          reinterpret_cast<float*>(out)[i] = x;
      }
    }
    wave_sync();
  }
}

uint32_t route_grid(int64_t tokens) {
  const int64_t want = (tokens + kRouteWaves - 1) / kRouteWaves;
  return static_cast<uint32_t>(want < (1 << 20) ? want : (1 << 20));
}

}  // namespace

namespace {

template <int LPT, int NI, int KL>
void launch_fast(const RouteArgs& a, int32_t* idx, float* w, hipStream_t st) {
  constexpr int kTokens = 64 / LPT;
  const size_t lds = 4 * (LPT * NI * 4 + kRouteWaves * wave_words<LPT>(a));
  // as many workgroups as fit the CUs at once, by registers (three or four) and by LDS
  const int64_t fit = kRouteFit<LPT, NI>, by_lds = (160 << 10) / static_cast<int64_t>(lds);
  const int64_t want = (a.tokens + kTokens * kRouteWaves - 1) / (kTokens * kRouteWaves), most = 256 * (fit < by_lds ? fit : by_lds);
  hipLaunchKernelGGL((route_fast_kernel<LPT, NI, KL>), dim3(static_cast<uint32_t>(want < most ? want : most)), dim3(kRouteThreads),
                     lds, st, a, idx, w);
}

template <int LPT, int NI>
void launch_fast_of(const RouteArgs& a, int32_t* idx, float* w, hipStream_t st) {
  (a.k <= 4 ? launch_fast<LPT, NI, 6> : a.k <= 8 ? launch_fast<LPT, NI, 10> : launch_fast<LPT, NI, 14>)(a, idx, w, st);
}

// Whether the kernel for many tokens a wave takes the call.
bool fast_route(const RouteArgs& a) { return a.k <= 12 && a.E <= 512 && a.groups <= kFastGroups; }

}  // namespace

hipError_t launch_route(const RouteArgs& args, int32_t* idx, float* w, hipStream_t st) {
  if (args.tokens == 0) return hipSuccess;
  RouteArgs a = args;
  if (a.topk_groups == a.groups) a.groups = a.topk_groups = 1;  // all of them stay
  if (fast_route(a)) {
    // Few tokens: more lanes for each, whose work is done sooner (1024 of 256 experts in
    // groups: 16 lanes 8.5 us, 8 9.3, 4 12.5; 8192: 16.8, 16.3, 19.6).  Many: fewer, which
    // merge less; but with groups of many experts their keys fill LDS, and smaller rounds let
    // more waves in (262144 tokens of 256 experts: 8 lanes 102 us, 4 105; 65536 of 144, 160,
    // 176, 192, 208, 240 and 256 in groups: 31, 30, 30, 30, 33, 34, 30 and 26, 26, 31, 30, 35,
    // 37, 30; of 144, 176, 224 and 256 without: 19, 20, 20, 20 and 13, 16, 18, 18).
    const int lanes = a.E > 256 ? 8 : a.tokens <= 4096 ? 16 : a.tokens <= 16384 || (a.groups > 1 && a.E > 160) ? 8 : 4;
    const auto go = lanes == 16  ? (a.E <= 128 ? launch_fast_of<16, 2> : launch_fast_of<16, 4>)
                    : lanes == 8 ? (a.E <= 128   ? launch_fast_of<8, 4>
                                    : a.E <= 256 ? launch_fast_of<8, 8>
                                    : a.E <= 384 ? launch_fast_of<8, 12>
                                                 : launch_fast_of<8, 16>)
                    : a.E <= 32  ? launch_fast_of<4, 2>
                    : a.E <= 64  ? launch_fast_of<4, 4>
                    : a.E <= 128 ? launch_fast_of<4, 8>
                    : a.E <= 160 ? launch_fast_of<4, 10>
                                 : launch_fast_of<4, 16>;
    go(a, idx, w, st);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(route_kernel, dim3(route_grid(a.tokens)), dim3(kRouteThreads), kRouteWaves * a.E * sizeof(double), st, a, idx, w);
  return hipGetLastError();
}

namespace {

template <int LPT, int MM>
void launch_backward_as(const RouteArgs& a, const int32_t* idx, const float* grad_w, void* grad_logits, hipStream_t st) {
  const size_t lds = kRouteWaves * grad_words<LPT>(a.E) * sizeof(float);
  const int64_t want = (a.tokens + 64 / LPT * kRouteWaves - 1) / (64 / LPT * kRouteWaves), most = 1024;
  hipLaunchKernelGGL((route_backward_kernel<LPT, MM>), dim3(static_cast<uint32_t>(want < most ? want : most)), dim3(kRouteThreads), lds, st,
                     a, idx, grad_w, grad_logits);
}

template <int LPT>
void launch_backward_of(const RouteArgs& a, const int32_t* idx, const float* grad_w, void* grad_logits, hipStream_t st) {
  const auto go = a.k <= LPT ? launch_backward_as<LPT, 1> : a.k <= 2 * LPT ? launch_backward_as<LPT, 2> : launch_backward_as<LPT, 64 / LPT>;
  go(a, idx, grad_w, grad_logits, st);
}

}  // namespace

hipError_t launch_route_backward(const RouteArgs& a, const int32_t* idx, const float* grad_w, void* grad_logits,
                                 hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const auto go = a.E <= 256 ? launch_backward_of<8> : launch_backward_of<16>;
  go(a, idx, grad_w, grad_logits, st);
  return hipGetLastError();
}

}  // namespace ultraep
