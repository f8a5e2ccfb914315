// gfx950 kernels of the residual addition with the root-mean-square norm and of its
// gradients (include/ultraep_layer.h).  Bound by HBM: a row is read once, held in
// registers and written in all its forms.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

enum Stream { kNoResidual = 0, kBf16Stream = 1, kF32Stream = 2 };

// (By value: a bit cast of a vector's element in place takes its first one.)
__device__ __forceinline__ float f32_of(uint32_t bits) { return __builtin_bit_cast(float, bits); }

__device__ __forceinline__ void widen(const u32x4& v, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_lo(v[i]);
    o[2 * i + 1] = bf16_hi(v[i]);
  }
}

__device__ __forceinline__ u32x4 narrow(const float (&x)[8]) {
  return u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

// Eight elements from byte-addressed rows of either type; zeros behind the row's end.
__device__ __forceinline__ void load8(const __amdgpu_buffer_rsrc_t& r, int i, bool bf16, float (&o)[8]) {
  if (bf16) {
    widen(__builtin_amdgcn_raw_buffer_load_b128(r, 16 * i, 0, 0), o);
  } else {
    const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(r, 32 * i, 0, 0);
    const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(r, 32 * i + 16, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = f32_of(a[j]);
      o[4 + j] = f32_of(b[j]);
    }
  }
}

__device__ __forceinline__ void store8(const __amdgpu_buffer_rsrc_t& r, int i, bool bf16, const float (&x)[8]) {
  if (bf16) {
    __builtin_amdgcn_raw_buffer_store_b128(narrow(x), r, 16 * i, 0, 0);
  } else {
    u32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __builtin_bit_cast(uint32_t, x[j]);
      b[j] = __builtin_bit_cast(uint32_t, x[4 + j]);
    }
    __builtin_amdgcn_raw_buffer_store_b128(a, r, 32 * i, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(b, r, 32 * i + 16, 0, 0);
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, int64_t row, int32_t H, bool bf16) {
  const uint32_t bytes = static_cast<uint32_t>(H) * (bf16 ? 2u : 4u);
  return row_rsrc(static_cast<const char*>(base) + row * bytes, bytes);
}

// Sum over the workgroup in every thread, in a fixed order.  `part` alternates between
// two sets, so one barrier a sum is enough.
template <int THREADS>
__device__ __forceinline__ float group_sum(float x, float (&part)[THREADS / 64]) {
  x = wave_sum_f32(x);
  if (lane_id() == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = part[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) s += part[i];
  return s;
}

template <int STREAM, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a, const uint16_t* x, const void* residual, float eps,
                                                       void* h_out, uint16_t* y, uint8_t* q, uint8_t* q_scale,
                                                       float* rstd) {
  __shared__ float s_part[2][THREADS / 64];
  const int tid = threadIdx.x;
  constexpr bool kBf16 = STREAM != kF32Stream;
  const int32_t H = a.H, Hp = q_pitch(H), Hs = s_pitch(H);
  const __amdgpu_buffer_rsrc_t wr = row_of(a.weight, 0, H, a.weight_bf16);
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) load8(wr, v * THREADS + tid, a.weight_bf16, w[v]);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float h[NV][8];
    const __amdgpu_buffer_rsrc_t xr = row_of(x, row, H, true);
#pragma unroll
    for (int v = 0; v < NV; ++v) load8(xr, v * THREADS + tid, true, h[v]);
    if (STREAM != kNoResidual) {
      const __amdgpu_buffer_rsrc_t rr = row_of(residual, row, H, kBf16);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float r[8];
        load8(rr, v * THREADS + tid, kBf16, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] += r[j];
        if (kBf16) widen(narrow(h[v]), h[v]);  // the norm is of what the stream holds
      }
      if (h_out != nullptr) {
        const __amdgpu_buffer_rsrc_t hr = row_of(h_out, row, H, kBf16);
#pragma unroll
        for (int v = 0; v < NV; ++v) store8(hr, v * THREADS + tid, kBf16, h[v]);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += h[v][j] * h[v][j];
    const float mean = group_sum<THREADS>(sum, s_part[turn]) / static_cast<float>(H);
    turn ^= 1;
    const float inv = 1.f / sqrtf(mean + eps);
    if (tid == 0 && rstd != nullptr) rstd[row] = inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * THREADS + tid;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = 8 * i < H ? h[v][j] * inv * w[v][j] : 0.f;
      if (y != nullptr) store8(row_of(y, row, H, true), i, true, h[v]);
      if (q != nullptr) {
        const int32_t e = block_exponent_f32(row16_amax(h[v]));
        __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(h[v], power_of_two(e)), row_rsrc(q + row * Hp, static_cast<uint32_t>(Hp)),
                                              8 * i, 0, 0);
        const uint32_t s = four_scales(e);
        if (lane_id() == 0)  // words behind the row's last are dropped
          __builtin_amdgcn_raw_buffer_store_b32(s, row_rsrc(q_scale + row * Hs, static_cast<uint32_t>(Hs)), i / 16, 0, 0);
      }
    }
  }
}

// Gradients: a workgroup's rows one after another, its part of grad_weight in registers.
template <int STREAM, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormArgs a, const uint16_t* grad_y, const void* h_in,
                                                                const float* rstd, const void* grad_in, void* grad_h,
                                                                uint16_t* grad_x, float* partial) {
  __shared__ float s_part[2][THREADS / 64];
  const int tid = threadIdx.x;
  constexpr bool kBf16 = STREAM != kF32Stream;
  const int32_t H = a.H;
  const __amdgpu_buffer_rsrc_t wr = row_of(a.weight, 0, H, a.weight_bf16);
  float w[NV][8], acc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    load8(wr, v * THREADS + tid, a.weight_bf16, w[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float n[NV][8], z[NV][8];
    const __amdgpu_buffer_rsrc_t hr = row_of(h_in, row, H, kBf16), gr = row_of(grad_y, row, H, true);
    const float inv = rstd[row];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * THREADS + tid;
      load8(hr, i, kBf16, n[v]);
      load8(gr, i, true, z[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[v][j] *= inv;
        acc[v][j] += z[v][j] * n[v][j];
        z[v][j] *= w[v][j];
        sum += z[v][j] * n[v][j];
      }
    }
    const float mean = group_sum<THREADS>(sum, s_part[turn]) / static_cast<float>(H);
    turn ^= 1;
    const __amdgpu_buffer_rsrc_t to = row_of(grad_h, row, H, kBf16);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * THREADS + tid;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
      if (grad_in != nullptr) load8(row_of(grad_in, row, H, kBf16), i, kBf16, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] += inv * (z[v][j] - n[v][j] * mean);
      store8(to, i, kBf16, d);
      if (!kBf16 && grad_x != nullptr) store8(row_of(grad_x, row, H, true), i, true, d);
    }
  }
  if (partial == nullptr) return;
  const __amdgpu_buffer_rsrc_t pr = row_of(partial, blockIdx.x, H, false);
#pragma unroll
  for (int v = 0; v < NV; ++v) store8(pr, v * THREADS + tid, false, acc[v]);
}

// grad_weight from the workgroups' parts: 64 columns a workgroup, four threads a
// column, summed in fp64.
__global__ __launch_bounds__(256) void norm_weight_kernel(const float* __restrict__ partial, int32_t parts, int32_t H,
                                                          float* __restrict__ grad_weight, bool accumulate) {
  __shared__ double s_sum[4][64];
  const int c = threadIdx.x & 63, s = threadIdx.x >> 6;
  const int32_t col = blockIdx.x * 64 + c;
  double x = 0.0;
  if (col < H)
    for (int32_t i = s; i < parts; i += 4) x += static_cast<double>(partial[static_cast<int64_t>(i) * H + col]);
  s_sum[s][c] = x;
  __syncthreads();
  if (s != 0 || col >= H) return;
  x = ((s_sum[0][c] + s_sum[1][c]) + s_sum[2][c]) + s_sum[3][c];
  grad_weight[col] = static_cast<float>(accumulate ? static_cast<double>(grad_weight[col]) + x : x);
}

// Workgroups of the backward pass, each with a part of grad_weight.
int32_t backward_blocks(int64_t rows) { return static_cast<int32_t>(rows < 1024 ? rows : 1024); }

template <int STREAM, int THREADS, int NV>
void launch_norm_as(const NormArgs& a, const uint16_t* x, const void* residual, float eps, void* h, uint16_t* y,
                    uint8_t* q, uint8_t* q_scale, float* rstd, hipStream_t st) {
  const uint32_t grid = static_cast<uint32_t>(a.rows < 2048 ? a.rows : 2048);
  hipLaunchKernelGGL((norm_kernel<STREAM, THREADS, NV>), dim3(grid), dim3(THREADS), 0, st, a, x, residual, eps, h, y, q,
                     q_scale, rstd);
}

template <int STREAM>
void launch_norm_of(const NormArgs& a, const uint16_t* x, const void* residual, float eps, void* h, uint16_t* y,
                    uint8_t* q, uint8_t* q_scale, float* rstd, hipStream_t st) {
  const auto go = a.H <= 2048    ? launch_norm_as<STREAM, 256, 1>
                  : a.H <= 4096  ? launch_norm_as<STREAM, 256, 2>
                  : a.H <= 8192  ? launch_norm_as<STREAM, 256, 4>
                  : a.H <= 16384 ? launch_norm_as<STREAM, 1024, 2>
                                 : launch_norm_as<STREAM, 1024, 4>;
  go(a, x, residual, eps, h, y, q, q_scale, rstd, st);
}

template <int STREAM, int THREADS, int NV>
void launch_backward_as(const NormArgs& a, const uint16_t* grad_y, const void* h, const float* rstd, const void* grad_in,
                        void* grad_h, uint16_t* grad_x, float* partial, hipStream_t st) {
  hipLaunchKernelGGL((norm_backward_kernel<STREAM, THREADS, NV>), dim3(backward_blocks(a.rows)), dim3(THREADS), 0, st, a,
                     grad_y, h, rstd, grad_in, grad_h, grad_x, partial);
}

template <int STREAM>
void launch_backward_of(const NormArgs& a, const uint16_t* grad_y, const void* h, const float* rstd, const void* grad_in,
                        void* grad_h, uint16_t* grad_x, float* partial, hipStream_t st) {
  const auto go = a.H <= 2048    ? launch_backward_as<STREAM, 256, 1>
                  : a.H <= 4096  ? launch_backward_as<STREAM, 256, 2>
                  : a.H <= 8192  ? launch_backward_as<STREAM, 256, 4>
                  : a.H <= 16384 ? launch_backward_as<STREAM, 1024, 2>
                                 : launch_backward_as<STREAM, 1024, 4>;
  go(a, grad_y, h, rstd, grad_in, grad_h, grad_x, partial, st);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, const uint16_t* x, const void* residual, bool stream_bf16, float eps,
                       void* h, uint16_t* y, uint8_t* q, uint8_t* q_scale, float* rstd, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const auto go = residual == nullptr ? launch_norm_of<kNoResidual> : stream_bf16 ? launch_norm_of<kBf16Stream> : launch_norm_of<kF32Stream>;
  go(a, x, residual, eps, h, y, q, q_scale, rstd, st);
  return hipGetLastError();
}

size_t norm_workspace_bytes(int64_t rows, int32_t H) { return sizeof(float) * static_cast<size_t>(backward_blocks(rows)) * H; }

hipError_t launch_norm_backward(const NormArgs& a, const uint16_t* grad_y, const void* h, bool stream_bf16,
                                const float* rstd, const void* grad_in, void* grad_h, uint16_t* grad_x,
                                float* grad_weight, bool accumulate, float* partial, hipStream_t st) {
  if (a.rows > 0) {
    const auto go = stream_bf16 ? launch_backward_of<kBf16Stream> : launch_backward_of<kF32Stream>;
    go(a, grad_y, h, rstd, grad_in, grad_h, grad_x, grad_weight == nullptr ? nullptr : partial, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (grad_weight == nullptr) return hipSuccess;
  hipLaunchKernelGGL(norm_weight_kernel, dim3((a.H + 63) / 64), dim3(256), 0, st, partial, backward_blocks(a.rows), a.H,
                     grad_weight, accumulate);
  return hipGetLastError();
}

}  // namespace ultraep
