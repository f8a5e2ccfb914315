// gfx950 kernels of the gradients' global norm and clipping
// (include/ultraep_experts.h): sum of squares over many tensors, and scaling
// them.
//
// Both walk the tensors' chunks of kGradBytes: a workgroup scans the tensors'
// chunk counts into LDS once and takes every gridDim-th chunk, so tensors of any
// sizes spread evenly, neighbouring chunks are read at one time, and the order of
// every sum depends on the sizes alone.  Bound by HBM: 4e8 fp32 elements, read
// twice and written once (4.8 GB), take 905-915 us, 5.3 TB/s, the rate of a large
// copy.  One contiguous share a workgroup took 977 us, ordinary instead of
// non-temporal accesses 930, two vectors in flight 934, eight 1002 (fewer waves
// fit), half as many workgroups 967.  The squares are added in fp64, whose cost
// does not show, so no square overflows and long sums lose nothing.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_device.h"
#include "ultraep_experts.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;                                 // 16-byte vectors in flight per lane
constexpr int kGradBytes = kGradThreads * kGradVecs * 16;    // bytes of a chunk
constexpr int kGradBlocks = ULTRAEP_GRAD_WORKSPACE_BYTES / 8;  // partial sums

// Vectors at any alignment of their elements, in global memory (addresses from
// a table would otherwise be loaded as generic ones).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef __attribute__((address_space(1))) u32x4_any global_vec;
typedef __attribute__((address_space(1))) uint16_t global_u16;
typedef __attribute__((address_space(1))) float global_f32;

__device__ __forceinline__ u32x4 load_vec(uintptr_t p) {
  return __builtin_nontemporal_load(reinterpret_cast<const global_vec*>(p));
}
__device__ __forceinline__ void store_vec(uintptr_t p, const u32x4& v) {
  __builtin_nontemporal_store(v, reinterpret_cast<global_vec*>(p));
}

// The workgroup's walk over the chunks: first[t] is the number of chunks before
// tensor t (2^31 chunks would be 32 TiB), `total` the number of all.
struct Walk {
  const void* const* tensors;
  const int64_t* numels;
  int32_t n;
  const int32_t* first;
  int32_t total;
};

struct Chunk {
  uintptr_t p;     // its first element
  int64_t at;      // elements of the tensor before it
  int32_t len;     // elements
  int32_t tensor;
};

// Chunk c < total; its tensor is `from` or a later one.
__device__ __forceinline__ Chunk chunk_at(const Walk& w, int32_t c, int32_t from, int32_t per_chunk, int32_t size) {
  int32_t lo = from, step = 1;  // doubling steps, then halving ones
  while (lo + step < w.n && w.first[lo + step] <= c) {
    lo += step;
    step *= 2;
  }
  for (; step > 0; step >>= 1)
    if (lo + step < w.n && w.first[lo + step] <= c) lo += step;
  Chunk x;
  x.tensor = lo;
  x.at = static_cast<int64_t>(c - w.first[lo]) * per_chunk;
  x.len = static_cast<int32_t>(min(w.numels[lo] - x.at, static_cast<int64_t>(per_chunk)));
  x.p = reinterpret_cast<uintptr_t>(w.tensors[lo]) + x.at * size;
  return x;
}

__device__ Walk grad_walk(const void* const* tensors, const int64_t* numels, int32_t n, int32_t per_chunk, int32_t* first) {
  __shared__ int32_t s_wave[kGradThreads / 64];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
  const int32_t each = (n + kGradThreads - 1) / kGradThreads;
  const int32_t t0 = min(tid * each, n), t1 = min(t0 + each, n);
  int32_t sum = 0;
  for (int32_t t = t0; t < t1; ++t) {
    const int64_t m = numels[t];
    const bool some = tensors[t] != nullptr;  // both loads at once
    first[t] = sum;
    sum += some && m > 0 ? static_cast<int32_t>((m + per_chunk - 1) / per_chunk) : 0;
  }
  const int32_t upto = wave_inclusive_scan(sum);
  if (lane == 63) s_wave[wv] = upto;
  __syncthreads();
  int32_t before = upto - sum, total = 0;
#pragma unroll
  for (int i = 0; i < kGradThreads / 64; ++i) {
    if (i < wv) before += s_wave[i];
    total += s_wave[i];
  }
  for (int32_t t = t0; t < t1; ++t) first[t] += before;
  __syncthreads();
  return Walk{tensors, numels, n, first, total};
}

__device__ __forceinline__ float f32_of(uint32_t bits) { return __builtin_bit_cast(float, bits); }
__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }

__device__ __forceinline__ float scaled(double c, float v) { return static_cast<float>(c * static_cast<double>(v)); }

__device__ __forceinline__ double square(float v) { return static_cast<double>(v) * static_cast<double>(v); }

// Sum of the squares of one vector's values.
template <bool BF16>
__device__ __forceinline__ double squares(const u32x4& v) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      s += square(bf16_lo(v[i]));
      s += square(bf16_hi(v[i]));
    } else {
      s += square(f32_of(v[i]));
    }
  }
  return s;
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const u32x2 x = __builtin_bit_cast(u32x2, v);
  const u32x2 y = {dpp<CTRL>(x[0]), dpp<CTRL>(x[1])};
  return __builtin_bit_cast(double, y);
}

__device__ __forceinline__ double readlane_f64(double v, int l) {
  const u32x2 x = __builtin_bit_cast(u32x2, v);
  const u32x2 y = {readlane(x[0], l), readlane(x[1], l)};
  return __builtin_bit_cast(double, y);
}

__device__ __forceinline__ double wave_sum_f64(double x) {
  x += dpp_f64<0xB1>(x);
  x += dpp_f64<0x4E>(x);
  x += dpp_f64<0x141>(x);
  x += dpp_f64<0x140>(x);
  return ((readlane_f64(x, 0) + readlane_f64(x, 16)) + readlane_f64(x, 32)) + readlane_f64(x, 48);
}

// Sum over the workgroup, in thread 0.
__device__ double block_sum_f64(double x) {
  __shared__ double s_sum[kGradThreads / 64];
  x = wave_sum_f64(x);
  if (lane_id() == 0) s_sum[threadIdx.x >> 6] = x;
  __syncthreads();
  return ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
}

template <bool BF16>
__global__ __launch_bounds__(kGradThreads) void grad_sumsq_kernel(const void* const* __restrict__ tensors,
                                                                  const int64_t* __restrict__ numels, int32_t n,
                                                                  double* __restrict__ partial) {
  extern __shared__ int32_t s_first[];
  constexpr int kSize = BF16 ? 2 : 4, kVec = 16 / kSize, kChunk = kGradBytes / kSize;
  const Walk w = grad_walk(tensors, numels, n, kChunk, s_first);
  double acc = 0.0;
  Chunk x, next;
  const int32_t blocks = static_cast<int32_t>(gridDim.x);
  if (static_cast<int32_t>(blockIdx.x) < w.total) next = chunk_at(w, static_cast<int32_t>(blockIdx.x), 0, kChunk, kSize);
  for (int32_t c = static_cast<int32_t>(blockIdx.x); c < w.total; c += blocks) {
    x = next;
    u32x4 v[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int i = (u * kGradThreads + static_cast<int>(threadIdx.x)) * kVec;
      v[u] = u32x4{0, 0, 0, 0};
      if (i + kVec <= x.len) v[u] = load_vec(x.p + i * kSize);
    }
    if (c + blocks < w.total) next = chunk_at(w, c + blocks, x.tensor, kChunk, kSize);
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) acc += squares<BF16>(v[u]);
    const int rest = x.len % kVec;  // values behind the last whole vector
    if (static_cast<int>(threadIdx.x) < rest) {
      const int i = x.len - rest + static_cast<int>(threadIdx.x);
      acc += square(BF16 ? bf16_lo(reinterpret_cast<const global_u16*>(x.p)[i]) : reinterpret_cast<const global_f32*>(x.p)[i]);
    }
  }
  const double s = block_sum_f64(acc);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// m: kGradBlocks partial sums, or none.
__global__ __launch_bounds__(kGradThreads) void grad_total_kernel(const double* __restrict__ partial, int32_t m,
                                                                  double* __restrict__ sumsq, bool accumulate) {
  double part[kGradBlocks / kGradThreads], acc = 0.0;  // all loads at once
#pragma unroll
  for (int i = 0; i < kGradBlocks / kGradThreads; ++i)
    part[i] = m > 0 ? partial[i * kGradThreads + static_cast<int>(threadIdx.x)] : 0.0;
#pragma unroll
  for (int i = 0; i < kGradBlocks / kGradThreads; ++i) acc += part[i];
  const double s = block_sum_f64(acc);
  if (threadIdx.x == 0) *sumsq = accumulate ? *sumsq + s : s;
}

template <bool BF16>
__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(const void* const* __restrict__ tensors,
                                                                 const int64_t* __restrict__ numels, int32_t n,
                                                                 const double* __restrict__ sumsq, double max_norm,
                                                                 float* __restrict__ norm_out, void* const* __restrict__ out) {
  extern __shared__ int32_t s_first[];
  constexpr int kSize = BF16 ? 2 : 4, kVec = 16 / kSize, kChunk = kGradBytes / kSize;
  const double square_sum = *sumsq;
  const Walk w = grad_walk(tensors, numels, n, kChunk, s_first);
  const double norm = sqrt(square_sum), ratio = max_norm / (norm + 1e-6);
  const double coef = ratio >= 1.0 ? 1.0 : ratio;  // NaN stays NaN; fp64, since a huge norm's factor is below fp32's range
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out != nullptr) *norm_out = static_cast<float>(norm);
  if (coef == 1.0 && out == nullptr) return;
  Chunk x, next;
  const int32_t blocks = static_cast<int32_t>(gridDim.x);
  if (static_cast<int32_t>(blockIdx.x) < w.total) next = chunk_at(w, static_cast<int32_t>(blockIdx.x), 0, kChunk, kSize);
  for (int32_t c = static_cast<int32_t>(blockIdx.x); c < w.total; c += blocks) {
    x = next;
    u32x4 v[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int i = (u * kGradThreads + static_cast<int>(threadIdx.x)) * kVec;
      if (i + kVec <= x.len) v[u] = load_vec(x.p + i * kSize);
    }
    const uintptr_t to = out == nullptr ? 0 : reinterpret_cast<uintptr_t>(out[x.tensor]);
    const uintptr_t d = to == 0 ? x.p : to + x.at * kSize;
    if (c + blocks < w.total) next = chunk_at(w, c + blocks, x.tensor, kChunk, kSize);
    if (coef == 1.0 && d == x.p) continue;
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int i = (u * kGradThreads + static_cast<int>(threadIdx.x)) * kVec;
      if (i + kVec > x.len) continue;
      u32x4 y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = BF16 ? pack_bf16(scaled(coef, bf16_lo(v[u][j])), scaled(coef, bf16_hi(v[u][j])))
                    : bits_of(scaled(coef, f32_of(v[u][j])));
      store_vec(d + i * kSize, y);
    }
    const int rest = x.len % kVec;
    if (static_cast<int>(threadIdx.x) < rest) {
      const int i = x.len - rest + static_cast<int>(threadIdx.x);
      if (BF16)
        reinterpret_cast<global_u16*>(d)[i] =
            static_cast<uint16_t>(pack_bf16(scaled(coef, bf16_lo(reinterpret_cast<const global_u16*>(x.p)[i])), 0.f));
      else
        reinterpret_cast<global_f32*>(d)[i] = scaled(coef, reinterpret_cast<const global_f32*>(x.p)[i]);
    }
  }
}

}  // namespace

hipError_t launch_grad_sumsq(const void* const* tensors, const int64_t* numels, int32_t n, bool bf16,
                             double* sumsq, bool accumulate, double* partial, hipStream_t st) {
  const int32_t grid = n > 0 ? kGradBlocks : 0;
  if (grid > 0) {
    if (bf16)
      hipLaunchKernelGGL(grad_sumsq_kernel<true>, dim3(grid), dim3(kGradThreads), n * sizeof(int32_t), st, tensors, numels, n, partial);
    else
      hipLaunchKernelGGL(grad_sumsq_kernel<false>, dim3(grid), dim3(kGradThreads), n * sizeof(int32_t), st, tensors, numels, n, partial);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(grad_total_kernel, dim3(1), dim3(kGradThreads), 0, st, partial, grid, sumsq, accumulate);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const void* const* tensors, const int64_t* numels, int32_t n, bool bf16,
                            const double* sumsq, double max_norm, float* norm, void* const* out,
                            hipStream_t st) {
  const int32_t grid = n > 0 ? kGradBlocks : 1;
  if (bf16)
    hipLaunchKernelGGL(grad_clip_kernel<true>, dim3(grid), dim3(kGradThreads), n * sizeof(int32_t), st, tensors, numels, n, sumsq, max_norm, norm, out);
  else
    hipLaunchKernelGGL(grad_clip_kernel<false>, dim3(grid), dim3(kGradThreads), n * sizeof(int32_t), st, tensors, numels, n, sumsq, max_norm, norm, out);
  return hipGetLastError();
}

}  // namespace ultraep
