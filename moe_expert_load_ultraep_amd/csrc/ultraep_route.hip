// gfx950 kernels of the routing to experts and its gradients
// (include/ultraep_layer.h).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

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

// One wave a token, expert e = lane + 64 v in lane e % 64, all in fp64.
template <int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, int32_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_w) {
  extern __shared__ double s_keys[];
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  const int32_t per = a.E / a.groups;
  double* keys = s_keys + wv * a.E;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wv; t < a.tokens; t += nwaves) {
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

hipError_t launch_route(const RouteArgs& a, int32_t* idx, float* w, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
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
