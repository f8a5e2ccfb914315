// gfx950 kernels of the routing to experts and its gradients
// (include/ultraep_layer.h).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "ultraep_device.h"
#include "ultraep_internal.h"

#ifndef ROUTE_V1
#define ROUTE_V1 1024
#endif
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

__device__ __forceinline__ bool masked(float l) { return l == -__builtin_huge_valf(); }

// Softmax: largest logit and 1 / sum over the wave's logits (V a lane).
struct Soft {
  double m, inv;
};

template <int V>
__device__ __forceinline__ Soft soft_of(const float (&l)[V]) {
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  Soft s{wave_max_f64(static_cast<double>(m)), 0.0};
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (!masked(l[v])) sum += exp(static_cast<double>(l[v]) - s.m);
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

// One token by one wave, expert e = lane + 64 v in lane e % 64, all in fp64.  keys: room
// for E fp64 of the wave's own where there are groups.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* keys, int32_t* __restrict__ topk_idx,
                                            float* __restrict__ topk_w) {
  const int lane = lane_id();
  const int32_t per = a.E / a.groups;
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    l[v] = e < a.E ? load_logit(a, t * a.E + e) : -__builtin_huge_valf();
  }
  Soft soft{0.0, 0.0};
  if (!a.sigmoid) soft = soft_of(l);
  double key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    key[v] = kNone;
    if (masked(l[v])) continue;
    if (a.bias == nullptr) {
      key[v] = static_cast<double>(l[v]);
    } else {
      const double x = score_of(a.sigmoid, l[v], soft) + static_cast<double>(a.bias[e]);
      key[v] = x == x ? x : kNone;
    }
  }
  if (a.groups > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (e < a.E)
        keys[e] = a.bias == nullptr && a.group_top == 2 && key[v] != kNone ? score_of(a.sigmoid, l[v], soft) : key[v];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    double first = kNone, second = kNone;
    if (lane < a.groups)
      for (int i = 0; i < per; ++i) {
        const double x = keys[lane * per + i];
        second = fmax(second, fmin(first, x));
        first = fmax(first, x);
      }
    const double worth = a.group_top == 2 && second != kNone ? first + second : first;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double x = readlane_f64(worth, g);
      rank += x > worth || (x == worth && g < lane);
    }
    const uint64_t taken = ballot(lane < a.groups && worth != kNone && rank < a.topk_groups);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (e < a.E && !((taken >> (e / per)) & 1)) key[v] = kNone;
    }
  }
  int32_t mine = -1;  // lane j: the j-th expert
  for (int j = 0; j < a.k; ++j) {
    double best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const double top = wave_max_f64(best);
    if (top == kNone) break;  // the same in every lane
    const uint32_t e = lane + 64 * at;
    const uint32_t win = ~wave_max(best == top ? ~e : 0u);  // the lowest id
    if (lane == j) mine = static_cast<int32_t>(win);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 64 * v == static_cast<int>(win)) key[v] = kNone;
  }
  const bool some = mine >= 0;
  const float lj = some ? load_logit(a, t * a.E + mine) : 0.f;
  const double w = weight_of(a, some, lj, score_of(a.sigmoid, lj, soft));
  if (lane < a.k) {
    topk_idx[t * a.k + lane] = mine;
    topk_w[t * a.k + lane] = static_cast<float>(w);
  }
}

template <int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, int32_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_w) {
  extern __shared__ double s_keys[];
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; t < a.tokens; t += nwaves)
    route_token<V>(a, t, s_keys + wv * a.E, topk_idx, topk_w);
}

// ---------------------------------------------------------------------------
// Many tokens a wave.  LPT lanes have a token, four experts of every 4 * LPT each, and
// find its experts by 32-bit keys: the fp32 key as a whole number of VB bits, above
// the expert's id (complemented, so that the lower id is the larger key).  One
// v_med3_u32 a place keeps a sorted list, lists are merged across the lanes, and
// nothing has to be looked up afterwards.  Where two keys that the choice or its order
// hangs on are nearer than their errors can be, the token is done again in fp64
// (route_token), so the ids are always those of fp64.
template <int LPT>
struct Packed {
  static constexpr int kIdBits = LPT == 4 ? 8 : 9;
  static constexpr uint32_t kIds = (1u << kIdBits) - 1;
  static constexpr float kTop = static_cast<float>(1u << (32 - kIdBits));  // values are below
};

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
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
__host__ __device__ inline int32_t key_pitch(int32_t E) { return E + ((16 - E) & 63); }

struct KeyUnits {
  float c;        // units of a score
  bool exact;     // the bias spans too much for them
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
  KeyUnits u{(Packed<LPT>::kTop - 64.f) / span, !(span < 1e4f)};
  for (int e = tid; e < kAll; e += kRouteThreads) {
    const float b = e < a.E ? a.bias[e] : __builtin_nanf("");
    table[e] = b > -__builtin_huge_valf() ? (b - lo) * u.c + 8.f : __builtin_nanf("");
  }
  __syncthreads();
  return u;
}

template <int LPT, int NI, int KL>
__global__ __launch_bounds__(kRouteThreads) void route_fast_kernel(RouteArgs a, int32_t* __restrict__ topk_idx,
                                                                   float* __restrict__ topk_w) {
  extern __shared__ __align__(16) char s_dyn[];
  using P = Packed<LPT>;
  constexpr int kTokens = 64 / LPT, kAll = LPT * NI * 4, V = (kAll + 63) / 64, MM = (KL - 1 + LPT - 1) / LPT;
  constexpr float kHigh = P::kTop - 64.f, kPerLogit = kHigh / kLogitRange;
  const int lane = lane_id(), q = lane % LPT, tl = lane / LPT;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t E = a.E, per = E / a.groups, pitch = key_pitch(E);
  float* bias = reinterpret_cast<float*>(s_dyn);  // [kAll]
  uint32_t* keys = reinterpret_cast<uint32_t*>(s_dyn) + kAll + wv * kTokens * (pitch + kFastGroups);
  float* worths = reinterpret_cast<float*>(keys + kTokens * pitch);
  const bool with_bias = a.bias != nullptr;
  KeyUnits units{0.f, false};
  if (with_bias) units = bias_units<LPT, NI>(a, bias);
  // what two keys have to be apart for their order to be certain, in units
  const uint32_t margin = with_bias ? (a.sigmoid ? 16u : 64u) : a.bf16 ? 0u : 8u;
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  for (int64_t batch = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; batch * kTokens < a.tokens; batch += nwaves) {
    const int64_t t = batch * kTokens + tl, tok = min(t, a.tokens - 1);
    // logits
    float l[4 * NI];
    const auto logit_chunk = [&](int i, float (&x)[4]) {
      const int e = (i * LPT + q) * 4, at = e < E ? e : 0;
      if (a.bf16) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.logits) + tok * E + at);
        x[0] = bf16_lo(v[0]), x[1] = bf16_hi(v[0]), x[2] = bf16_lo(v[1]), x[3] = bf16_hi(v[1]);
      } else {
        const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.logits) + tok * E + at);
        x[0] = v[0], x[1] = v[1], x[2] = v[2], x[3] = v[3];
      }
      if (e >= E) x[0] = x[1] = x[2] = x[3] = -__builtin_huge_valf();
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float x[4];
      logit_chunk(i, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) l[4 * i + c] = x[c];
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
    // Keys, four at a time into LDS (where there are groups) or into the lane's list.
    uint32_t list[KL];
#pragma unroll
    for (int j = 0; j < KL; ++j) list[j] = 0;
    int ids = static_cast<int>(P::kIds) - 4 * q;
    asm volatile("" : "+v"(ids));  // made anew for every key: kept in registers they would be 4 * NI
    const auto pack = [&](int i, int c, uint32_t value) {
      return (value << P::kIdBits) | static_cast<uint32_t>(ids - (i * LPT * 4 + c));
    };
    // the value of an fp32 logit without a bias (NaN and masked ones: 0)
    const auto logit_value = [&](float x) {
      return static_cast<uint32_t>(x == x ? fmaxf(__builtin_fmaf(x - top, kPerLogit, kHigh), 0.f) : 0.f);
    };
    const auto put = [&](int i, const uint32_t (&key)[4]) {
      const int e = (i * LPT + q) * 4;
      if (a.groups > 1) {
        if (e < E) *reinterpret_cast<u32x4*>(keys + tl * pitch + e) = u32x4{key[0], key[1], key[2], key[3]};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) insert<0>(list, key[c]);
      }
    };
    if (with_bias) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(bias + (i * LPT + q) * 4);
        uint32_t key[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float x = l[4 * i + c], s = a.sigmoid ? fast_sigmoid(x) : __builtin_amdgcn_exp2f((x - top) * kLog2e) * inv;
          key[c] = pack(i, c, static_cast<uint32_t>(__builtin_fmaf(s, units.c, b[c])));  // NaN: 0
        }
        // a masked logit's score is 0, which is a key; NaN is none already
        if (ballot(fminf(fminf(l[4 * i], l[4 * i + 1]), fminf(l[4 * i + 2], l[4 * i + 3])) == -__builtin_huge_valf()) != 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (masked(l[4 * i + c])) key[c] = 0;
        }
        put(i, key);
      }
    } else if (a.bf16) {
      // the 16 bits themselves, in ascending order: nothing is lost
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t key[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float x = l[4 * i + c];
          uint32_t u = __builtin_bit_cast(uint32_t, x == 0.f ? 0.f : x);
          u ^= static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u;
          key[c] = x > -__builtin_huge_valf() ? pack(i, c, (u >> 16) + 1) : 0u;
        }
        put(i, key);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t key[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) key[c] = pack(i, c, logit_value(l[4 * i + c]));
        put(i, key);
      }
    }
    if (a.groups > 1) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      constexpr int kOwn = kFastGroups / LPT;
      float worth[kOwn];
      const uint32_t* row = keys + tl * pitch;
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) {
        const int g = gi * LPT + q;
        worth[gi] = -1.f;
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
            } else {  // scores of the two logits, up to the softmax's common factor
              float s = 0.f;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t v = k == 0 ? first : second;
                float x;
                if (a.bf16) {
                  uint32_t u = (v - 1) << 16;
                  u ^= static_cast<uint32_t>(~(static_cast<int32_t>(u) >> 31)) | 0x80000000u;
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
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      int rank[kOwn];
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) rank[gi] = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float x = worths[tl * kFastGroups + g];
#pragma unroll
        for (int gi = 0; gi < kOwn; ++gi) rank[gi] += x > worth[gi] || (x == worth[gi] && g < gi * LPT + q);
      }
      uint32_t taken = 0;
      float in = __builtin_huge_valf(), out = -__builtin_huge_valf();
#pragma unroll
      for (int gi = 0; gi < kOwn; ++gi) {
        const bool mine = worth[gi] >= 0.f, take = mine && rank[gi] < a.topk_groups;
        if (take) taken |= 1u << (gi * LPT + q);
        if (take) in = fminf(in, worth[gi]);
        if (mine && !take) out = fmaxf(out, worth[gi]);
      }
      taken = token_or<LPT>(taken);
      float apart = static_cast<float>(margin);
      if (a.group_top == 2 && with_bias) apart = 2.f * apart + 4.f;
      if (a.group_top == 2 && !with_bias) {
        apart = 1e-5f;
        if (!a.bf16) {  // logits below the keys' range have scores up to this
          if (a.sigmoid) apart += 2.f * fast_sigmoid(top - kLogitRange);
          out = fmaxf(out, 0.f);
        }
      }
      const float gap = token_min<LPT>(in) - token_max<LPT>(out);  // infinite where there is no other
      again |= gap < apart;
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
    // is every order that counts certain?
    uint32_t last = 0;
#pragma unroll
    for (int j = 0; j < KL - 1; ++j) {
      if (j >= a.k) continue;
      const uint32_t x = list[j] >> P::kIdBits, y = list[j + 1] >> P::kIdBits;
      again |= y != 0 && x - y < margin;
      last = x;
    }
    if (!with_bias && !a.bf16 && ballot(last < margin) != 0) {
      // fewer experts than k, or logits below the keys' range: are there such?
      int unseen = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float x[4];
        logit_chunk(i, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) unseen |= x[c] > -__builtin_huge_valf() && logit_value(x[c]) < margin;
      }
      again |= last < margin && token_or<LPT>(unseen) != 0;
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
        if (mm * LPT + c < KL - 1) k_j = q == c ? list[mm * LPT + c < KL ? mm * LPT + c : 0] : k_j;
      const bool some = (k_j >> P::kIdBits) != 0 && mm * LPT + q < a.k;
      e_j[mm] = some ? static_cast<int32_t>(P::kIds - (k_j & P::kIds)) : -1;
      l_j[mm] = some ? load_logit(a, tok * E + e_j[mm]) : 0.f;
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
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (uint64_t redo = ballot(again && q == 0 && t < a.tokens); redo != 0; redo &= redo - 1)
      route_token<V>(a, batch * kTokens + __builtin_ctzll(redo) / LPT, reinterpret_cast<double*>(keys), topk_idx, topk_w);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// One wave a token: lane j < k has the j-th chosen expert's gradient, every lane the
// elements e = lane + 64 v of the row.
template <int V>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a, const int32_t* __restrict__ topk_idx,
                                                                       const float* __restrict__ grad_w,
                                                                       void* __restrict__ grad_logits) {
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  const bool every = !a.sigmoid && !a.renorm;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; t < a.tokens; t += nwaves) {
    float l[V];
    Soft soft{0.0, 0.0};
    if (every) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        l[v] = e < a.E ? load_logit(a, t * a.E + e) : -__builtin_huge_valf();
      }
      soft = soft_of(l);
    }
    int32_t e_j = lane < a.k ? topk_idx[t * a.k + lane] : -1;
    if (e_j < 0 || e_j >= a.E) e_j = -1;
    const float l_j = e_j >= 0 ? load_logit(a, t * a.E + e_j) : -__builtin_huge_valf();
    if (masked(l_j)) e_j = -1;
    const bool some = e_j >= 0;
    const double g = some ? static_cast<double>(grad_w[t * a.k + lane]) : 0.0;
    const double s = score_of(a.sigmoid, l_j, soft);
    const double w = weight_of(a, some, some ? l_j : 0.f, s);
    const double total = wave_sum_f64(w * g);
    double d = a.renorm ? w * (g - total / a.scale) : w * g;
    if (a.sigmoid) d *= 1.0 - s;
    if (!some) d = 0.0;
    const float df = static_cast<float>(d);
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = every && !masked(l[v]) ? static_cast<float>(-total * score_of(false, l[v], soft)) : 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int32_t e = static_cast<int32_t>(readlane(static_cast<uint32_t>(e_j), j));
      const float x = readlane_f(df, j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane + 64 * v == e) out[v] += x;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (e >= a.E) continue;
      if (a.bf16)
        static_cast<uint16_t*>(grad_logits)[t * a.E + e] = static_cast<uint16_t>(pack_bf16(out[v], 0.f));
      else
        static_cast<float*>(grad_logits)[t * a.E + e] = out[v];
    }
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
  const size_t lds = 4 * (LPT * NI * 4 + (a.groups > 1 ? kRouteWaves * kTokens * (key_pitch(a.E) + kFastGroups) : 0));
  const int64_t want = (a.tokens + kTokens * kRouteWaves - 1) / (kTokens * kRouteWaves), most = ROUTE_V1;
  hipLaunchKernelGGL((route_fast_kernel<LPT, NI, KL>), dim3(static_cast<uint32_t>(want < most ? want : most)), dim3(kRouteThreads),
                     lds, st, a, idx, w);
}

template <int LPT, int NI>
void launch_fast_of(const RouteArgs& a, int32_t* idx, float* w, hipStream_t st) {
  (a.k <= 4 ? launch_fast<LPT, NI, 5> : a.k <= 8 ? launch_fast<LPT, NI, 9> : launch_fast<LPT, NI, 13>)(a, idx, w, st);
}

// Whether the kernel for many tokens a wave takes the call.
bool fast_route(const RouteArgs& a) {
  const size_t unit = a.bf16 ? 8 : 16;
  return a.k <= 12 && a.E <= 512 && a.E % 4 == 0 && a.groups <= kFastGroups && reinterpret_cast<uintptr_t>(a.logits) % unit == 0;
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, int32_t* idx, float* w, hipStream_t st) {
  if (args.tokens == 0) return hipSuccess;
  RouteArgs a = args;
  if (a.topk_groups == a.groups) a.groups = a.topk_groups = 1;  // all of them stay
  if (fast_route(a)) {
    const auto go = a.E <= 32    ? launch_fast_of<4, 2>
                    : a.E <= 64  ? launch_fast_of<4, 4>
                    : a.E <= 128 ? launch_fast_of<4, 8>
                    : a.E <= 160 ? launch_fast_of<4, 10>
                    : a.E <= 192 ? launch_fast_of<4, 12>
                    : a.E <= 256 ? launch_fast_of<4, 16>
                    : a.E <= 384 ? launch_fast_of<8, 12>
                                 : launch_fast_of<8, 16>;
    go(a, idx, w, st);
    return hipGetLastError();
  }
  const size_t lds = a.groups > 1 ? kRouteWaves * a.E * sizeof(double) : 0;
  const dim3 grid(route_grid(a.tokens)), block(kRouteThreads);
  if (a.E <= 64)
    hipLaunchKernelGGL(route_kernel<1>, grid, block, lds, st, a, idx, w);
  else if (a.E <= 256)
    hipLaunchKernelGGL(route_kernel<4>, grid, block, lds, st, a, idx, w);
  else
    hipLaunchKernelGGL(route_kernel<16>, grid, block, lds, st, a, idx, w);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& a, const int32_t* idx, const float* grad_w, void* grad_logits,
                                 hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const dim3 grid(route_grid(a.tokens)), block(kRouteThreads);
  if (a.E <= 64)
    hipLaunchKernelGGL(route_backward_kernel<1>, grid, block, 0, st, a, idx, grad_w, grad_logits);
  else if (a.E <= 256)
    hipLaunchKernelGGL(route_backward_kernel<4>, grid, block, 0, st, a, idx, grad_w, grad_logits);
  else
    hipLaunchKernelGGL(route_backward_kernel<16>, grid, block, 0, st, a, idx, grad_w, grad_logits);
  return hipGetLastError();
}

}  // namespace ultraep
