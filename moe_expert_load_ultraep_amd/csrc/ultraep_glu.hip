// gfx950 kernels of the gated activation between the experts' two products and of its
// gradient rows, quantised on their way out (include/ultraep_layer.h).  Bound by HBM.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

constexpr int kGluThreads = 256;
constexpr int kGluWaves = kGluThreads / 64;
constexpr int kGluChunk = 512;  // columns of a wave: 64 lanes x 8

// The rows of a segment: h [.][2F], and for the gradients grad [.][F].
struct GluRows {
  const uint16_t* h;
  const uint16_t* grad;
  int32_t F;
};

// sigmoid(z(g)) of either activation, and dz/dg.  The gelu's square is bounded, as
// beyond it nothing changes and 0 * inf would.
template <bool GELU>
__device__ __forceinline__ float gate(float g, float& dz) {
  constexpr float kLog2e = 1.4426950408889634f, kC = 1.5957691216057308f, kC3 = kC * 0.044715f;
  float z = g;
  dz = 1.f;
  if (GELU) {
    const float g2 = fminf(g * g, 1e8f);
    z = g * (kC + kC3 * g2);
    dz = kC + 3.f * kC3 * g2;
  }
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

__device__ __forceinline__ float nothing_tiny(float x) { return fabsf(x) < 0x1p-100f ? 0.f : x; }

// Eight columns: of a = f(g) u, or of its gradients d f(g) (upper) and d u f'(g).
template <bool BACK, bool GELU>
__device__ __forceinline__ void glu8(const u32x4& g, const u32x4& u, const u32x4& d, bool upper, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = i & 1 ? bf16_hi(g[i / 2]) : bf16_lo(g[i / 2]);
    const float ui = i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
    const float di = i & 1 ? bf16_hi(d[i / 2]) : bf16_lo(d[i / 2]);
    float dz;
    const float p = gate<GELU>(gi, dz);
    const float f = gi * p;
    float x = f * ui;
    if (BACK) x = upper ? di * f : di * ui * (p + f * (1.f - p) * dz);
    o[i] = nothing_tiny(x);
  }
}

// Columns h0.. of row `row`, zeros where there are none.
template <bool BACK, bool GELU>
__device__ __forceinline__ void glu_load(const GluRows& in, int64_t row, int32_t h0, bool there, float (&o)[8]) {
  const bool upper = BACK && h0 >= in.F;
  const int32_t c = there ? (upper ? h0 - in.F : h0) : 0;
  const uint16_t* h = in.h + row * (2 * static_cast<int64_t>(in.F)) + c;
  u32x4 d = {0, 0, 0, 0};
  const u32x4 g = *reinterpret_cast<const u32x4*>(h);
  const u32x4 u = *reinterpret_cast<const u32x4*>(h + in.F);
  if (BACK) d = *reinterpret_cast<const u32x4*>(in.grad + row * in.F + c);
  glu8<BACK, GELU>(g, u, d, upper, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = there ? o[i] : 0.f;
}

// Rows form alone: one wave per (row, 512 columns), 16 lanes a block.
template <bool BACK, bool GELU>
__global__ __launch_bounds__(kGluThreads) void glu_rows_kernel(const int32_t* __restrict__ off, int32_t ne, GluRows in,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                               int64_t cap) {
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t W = BACK ? 2 * in.F : in.F, Wp = q_pitch(W), Ws = s_pitch(W), nch = Ws / 4;
  const int64_t rows = group_row(off, ne, cap);
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kGluWaves;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGluWaves + wv; item < rows * nch; item += nwaves) {
    const int64_t row = item / nch;
    const int32_t ch = static_cast<int32_t>(item - row * nch), h0 = ch * kGluChunk + lane * 8;
    float x[8];
    glu_load<BACK, GELU>(in, row, h0, h0 < W, x);
    const int32_t e = block_exponent_f32(row16_amax(x));
    const __amdgpu_buffer_rsrc_t dst = row_rsrc(q + row * Wp, static_cast<uint32_t>(Wp));
    __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(x, power_of_two(e)), dst, h0, 0, 0);
    const uint32_t s = four_scales(e);
    if (lane == 0) *reinterpret_cast<uint32_t*>(scale + row * Ws + 4 * ch) = s;
  }
}

// Columns form, and the rows form with it: one workgroup per 128 rows of one expert
// and 128 columns.
template <bool BACK, bool GELU, bool ROWS>
__global__ __launch_bounds__(kGluThreads) void glu_cols_kernel(const int32_t* __restrict__ off, int32_t ne, GluRows in,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                               uint8_t* __restrict__ qt, uint8_t* __restrict__ scale_t,
                                                               int64_t cap, int32_t nblk, int32_t ncol) {
  __shared__ __align__(16) uint8_t s_tile[kQBlock * kQBlock];
  __shared__ uint32_t s_max[16][kQBlock];
  __shared__ float s_scale[kQBlock];
  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4;
  const int32_t W = BACK ? 2 * in.F : in.F, Wp = q_pitch(W), Ws = s_pitch(W);
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(nblk) * ncol; item += gridDim.x) {
    const int32_t b = static_cast<int32_t>(item / ncol), cb = static_cast<int32_t>(item - static_cast<int64_t>(b) * ncol);
    const int32_t p = find_group(off, ne, cap, kQBlock, b);
    const int32_t o = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
    const int64_t row0 = o + static_cast<int64_t>(b - (o / kQBlock + p)) * kQBlock;
    const int32_t live = static_cast<int32_t>(min(static_cast<int64_t>(o1) - row0, static_cast<int64_t>(kQBlock)));
    if (live <= 0) continue;  // the same for the whole workgroup
    const int32_t h0 = cb * kQBlock + 8 * c;
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * g + i;
      glu_load<BACK, GELU>(in, row0 + min(r, live - 1), h0, r < live && h0 < W, x[i]);
    }
    if (ROWS) {
      const __amdgpu_buffer_rsrc_t to_q = row_rsrc(q + row0 * Wp, static_cast<uint32_t>(live) * static_cast<uint32_t>(Wp));
      const __amdgpu_buffer_rsrc_t to_s = row_rsrc(scale + row0 * Ws, static_cast<uint32_t>(live) * static_cast<uint32_t>(Ws));
      // one scale byte a row, and behind the last block the padding's
      const bool pad = c > 0 && cb == ncol - 1 && cb + c < Ws;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * g + i;
        const int32_t e = block_exponent_f32(row16_amax(x[i]));
        __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(x[i], power_of_two(e)), to_q, r * Wp + h0, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(c == 0 ? e + 127 : 127), to_s,
                                             c == 0 || pad ? r * Ws + cb + c : 0x7FFFFFFF, 0, 0);
      }
    }
    // column maxima: over the thread's rows, then over the 16 row groups
    __syncthreads();  // earlier readers are done
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(x[i][j]));
      s_max[g][8 * c + j] = m;
    }
    __syncthreads();
    if (tid < kQBlock) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, s_max[i][tid]);
      const int32_t e = block_exponent_f32(m);
      s_scale[tid] = power_of_two(e);
      const int32_t h = cb * kQBlock + tid;
      if (h < W) scale_t[static_cast<int64_t>(b) * W + h] = static_cast<uint8_t>(e + 127);
    }
    __syncthreads();
    u32x2 bt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = s_scale[8 * c + j];
      bt[j] = u32x2{to_e4m3(x[0][j], x[1][j], x[2][j], x[3][j], s), to_e4m3(x[4][j], x[5][j], x[6][j], x[7][j], s)};
    }
    put_column_bytes(s_tile, c, g, bt);
    __syncthreads();
    const int32_t cols = min(kQBlock, W - cb * kQBlock);
    u32x4* out = reinterpret_cast<u32x4*>(qt + (static_cast<int64_t>(b) * W + static_cast<int64_t>(cb) * kQBlock) * kQBlock);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid + i * kGluThreads, h = u >> 3, part = u & 7;
      if (h < cols) out[u] = get_column_bytes(s_tile, h, part);
    }
  }
}

uint32_t grid_of(int64_t want) { return static_cast<uint32_t>(want < (1 << 20) ? want : (1 << 20)); }

template <bool BACK, bool GELU>
hipError_t launch_glu_as(const int32_t* off, int32_t ne, const GluRows& in, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                         uint8_t* qt_scale, int64_t cap, hipStream_t st) {
  const int32_t W = BACK ? 2 * in.F : in.F;
  if (qt == nullptr) {
    const int64_t items = cap * (s_pitch(W) / 4);
    hipLaunchKernelGGL((glu_rows_kernel<BACK, GELU>), dim3(grid_of((items + kGluWaves - 1) / kGluWaves)), dim3(kGluThreads), 0,
                       st, off, ne, in, q, q_scale, cap);
    return hipGetLastError();
  }
  const int32_t nblk = static_cast<int32_t>(cap / kQBlock) + ne, ncol = ceil_div(W, kQBlock);
  const dim3 grid(grid_of(static_cast<int64_t>(nblk) * ncol));
  if (q != nullptr)
    hipLaunchKernelGGL((glu_cols_kernel<BACK, GELU, true>), grid, dim3(kGluThreads), 0, st, off, ne, in, q, q_scale, qt,
                       qt_scale, cap, nblk, ncol);
  else
    hipLaunchKernelGGL((glu_cols_kernel<BACK, GELU, false>), grid, dim3(kGluThreads), 0, st, off, ne, in, q, q_scale, qt,
                       qt_scale, cap, nblk, ncol);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glu_quant(const int32_t* off, int32_t ne, const uint16_t* h, const uint16_t* grad, int32_t F,
                            bool gelu, uint8_t* q, uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, int64_t cap,
                            hipStream_t st) {
  if (ne == 0 || cap == 0) return hipSuccess;
  const GluRows in{h, grad, F};
  const auto go = grad == nullptr ? (gelu ? launch_glu_as<false, true> : launch_glu_as<false, false>)
                                  : (gelu ? launch_glu_as<true, true> : launch_glu_as<true, false>);
  return go(off, ne, in, q, q_scale, qt, qt_scale, cap, st);
}

}  // namespace ultraep
