// gfx950 kernels of the residual addition with the root-mean-square norm and of its
// gradients (include/ultraep_layer.h).  Bound by HBM: a row is read once, held in
// registers and written in all its forms.  32771 rows of 7168, bf16 stream, with the
// 8-bit form, 2.12 GB: 365 us, 5.8 TB/s (a large copy reaches 5.2); gradients of 16411
// rows of 7168, fp32 stream, 1.88 GB: 320 us, 5.9 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

enum Stream { kNoResidual = 0, kBf16Stream = 1, kF32Stream = 2 };

// (By value: a bit cast of a vector's element in place takes its first one.)
__device__ __forceinline__ float f32_of(uint32_t bits) { return __builtin_bit_cast(float, bits); }

// A thread holds eight columns of a wave's 512, vector i = 64 * (wave's place) + lane:
// eight in a row, 16 bytes of bf16; or, where the stream is fp32 (QUADS), four in a
// row and the four 256 columns behind, 16 bytes of fp32 each, so that every access of
// a wave covers whole lines.
template <bool QUADS>
__device__ __forceinline__ int column(int i, int half) {
  return QUADS ? (i >> 6) * 512 + (i & 63) * 4 + half * 256 : 8 * i + 4 * half;
}

// Eight columns as they are in memory.  AUX: cache policy.
template <bool QUADS, bool BF16, int AUX>
struct Raw8 {
  u32x4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& r, int i) {
    if (!BF16) {
#pragma unroll
      for (int k = 0; k < 2; ++k) v[BF16 ? 0 : k] = __builtin_amdgcn_raw_buffer_load_b128(r, 4 * column<QUADS>(i, k), 0, AUX);
    } else if (QUADS) {
      const u32x2 lo = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * column<QUADS>(i, 0), 0, AUX);
      const u32x2 hi = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * column<QUADS>(i, 1), 0, AUX);
      v[0] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      v[0] = __builtin_amdgcn_raw_buffer_load_b128(r, 2 * column<QUADS>(i, 0), 0, AUX);
    }
  }
  __device__ __forceinline__ float at(int j) const {
    if (BF16) return j & 1 ? bf16_hi(v[0][j / 2]) : bf16_lo(v[0][j / 2]);
    return f32_of(v[BF16 ? 0 : j / 4][j % 4]);
  }
};

template <bool QUADS, bool BF16, int AUX>
__device__ __forceinline__ void store8(const __amdgpu_buffer_rsrc_t& r, int i, const float (&x)[8]) {
  if (!BF16) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = __builtin_bit_cast(uint32_t, x[4 * k + j]);
      __builtin_amdgcn_raw_buffer_store_b128(a, r, 4 * column<QUADS>(i, k), 0, AUX);
    }
    return;
  }
  const u32x4 p = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  if (QUADS) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{p[0], p[1]}, r, 2 * column<QUADS>(i, 0), 0, AUX);
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{p[2], p[3]}, r, 2 * column<QUADS>(i, 1), 0, AUX);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(p, r, 2 * column<QUADS>(i, 0), 0, AUX);
  }
}

__device__ __forceinline__ float to_bf16_and_back(float x) { return bf16_lo(pack_bf16(x, 0.f)); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, int64_t row, int32_t H, bool bf16) {
  const uint32_t bytes = static_cast<uint32_t>(H) * (bf16 ? 2u : 4u);
  return row_rsrc(static_cast<const char*>(base) + row * bytes, bytes);
}

// The weight's columns of a thread, of either type.
template <bool QUADS, int TEAM, int NV>
__device__ __forceinline__ void load_weight(const NormArgs& a, int tid, float (&w)[NV][8]) {
  const __amdgpu_buffer_rsrc_t r = row_of(a.weight, 0, a.H, a.weight_bf16);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * TEAM + tid;
    if (a.weight_bf16) {
      Raw8<QUADS, true, 0> x;
      x.load(r, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[v][j] = x.at(j);
    } else {
      Raw8<QUADS, false, 0> x;
      x.load(r, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[v][j] = x.at(j);
    }
  }
}

// The rows form of a thread's columns: a block is 16 lanes of eight, or 32 of four.
template <bool QUADS, int AUX>
__device__ __forceinline__ void store_rows_form(const float (&y)[8], int i, uint8_t* q, uint8_t* q_scale, int32_t Hp, int32_t Hs) {
  const __amdgpu_buffer_rsrc_t to = row_rsrc(q, static_cast<uint32_t>(Hp)), to_s = row_rsrc(q_scale, static_cast<uint32_t>(Hs));
  uint32_t s;
  if (!QUADS) {
    const int32_t e = block_exponent_f32(row16_amax(y));
    __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(y, power_of_two(e)), to, 8 * i, 0, AUX);
    s = four_scales(e);
  } else {
    uint32_t m[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[k] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m[k] = max(m[k], finite_magnitude(y[4 * k + j]));
      m[k] = row16_max(m[k]);
      m[k] = max(m[k], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[k]), 16)));
      const float scale = power_of_two(block_exponent_f32(m[k]));
      __builtin_amdgcn_raw_buffer_store_b32(to_e4m3(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3], scale), to,
                                            column<true>(i, k), 0, AUX);
    }
    s = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      s |= static_cast<uint32_t>(block_exponent_f32(readlane(m[b / 2], 32 * (b % 2))) + 127) << (8 * b);
  }
  if (lane_id() == 0)  // words behind the row's last are dropped
    __builtin_amdgcn_raw_buffer_store_b32(s, to_s, i / 16, 0, 0);
}

// A row belongs to a team of TEAM threads with NV vectors each: one of a workgroup's
// four waves, or a whole workgroup.
__host__ __device__ constexpr int teams(int team) { return team == 64 ? 4 : 1; }

// Sum over the team in every thread, in a fixed order.  `part` alternates between two
// sets, so one barrier a sum is enough.
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float (&part)[TEAM / 64]) {
  x = wave_sum_f32(x);
  if (TEAM == 64) return x;
  if (lane_id() == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = part[0];
#pragma unroll
  for (int i = 1; i < TEAM / 64; ++i) s += part[i];
  return s;
}

// The next row is under way while this one's sum goes round.
template <int STREAM, int TEAM, int NV, bool STREAMING>
__global__ __launch_bounds__(TEAM * teams(TEAM)) void norm_kernel(NormArgs a, const uint16_t* x, const void* residual, float eps,
                                                       void* h_out, uint16_t* y, uint8_t* q, uint8_t* q_scale,
                                                       float* rstd) {
  __shared__ float s_part[2][TEAM / 64];
  const int tid = static_cast<int>(threadIdx.x) % TEAM;
  const int team = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TEAM);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams(TEAM) + team, step = static_cast<int64_t>(gridDim.x) * teams(TEAM);
  constexpr bool kQuads = STREAM == kF32Stream, kBf16 = !kQuads;
  constexpr int kAux = STREAMING ? kNonTemporal : 0;
  const int32_t H = a.H, Hp = q_pitch(H), Hs = s_pitch(H);
  float w[NV][8];
  load_weight<kQuads, TEAM>(a, tid, w);
  Raw8<kQuads, true, kAux> rx[NV];
  Raw8<kQuads, kBf16, kAux> rr[NV];
  const auto load = [&](int64_t row) {
    const __amdgpu_buffer_rsrc_t from_x = row_of(x, row, H, true);
#pragma unroll
    for (int v = 0; v < NV; ++v) rx[v].load(from_x, v * TEAM + tid);
    if (STREAM == kNoResidual) return;
    const __amdgpu_buffer_rsrc_t from_r = row_of(residual, row, H, kBf16);
#pragma unroll
    for (int v = 0; v < NV; ++v) rr[v].load(from_r, v * TEAM + tid);
  };
  if (first < a.rows) load(first);
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    float h[NV][8];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[v][j] = rx[v].at(j);
        if (STREAM != kNoResidual) h[v][j] += rr[v].at(j);
        if (STREAM == kBf16Stream) h[v][j] = to_bf16_and_back(h[v][j]);  // the norm is of what the stream holds
        sum += h[v][j] * h[v][j];
      }
    }
    if (row + step < a.rows) load(row + step);
    if (STREAM != kNoResidual && h_out != nullptr) {
      const __amdgpu_buffer_rsrc_t to = row_of(h_out, row, H, kBf16);
#pragma unroll
      for (int v = 0; v < NV; ++v) store8<kQuads, kBf16, kAux>(to, v * TEAM + tid, h[v]);
    }
    const float mean = team_sum<TEAM>(sum, s_part[turn]) / static_cast<float>(H);
    turn ^= 1;
    const float inv = 1.f / sqrtf(mean + eps);
    if (tid == 0 && rstd != nullptr) rstd[row] = inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * TEAM + tid;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = column<kQuads>(i, j / 4) < H ? h[v][j] * inv * w[v][j] : 0.f;
      if (y != nullptr) store8<kQuads, true, kAux>(row_of(y, row, H, true), i, h[v]);
      if (q != nullptr) store_rows_form<kQuads, kAux>(h[v], i, q + row * Hp, q_scale + row * Hs, Hp, Hs);
    }
  }
}

// Gradients: a team's rows one after another, its part of grad_weight in registers.
// The next row of a bf16 stream is under way while this one's sum goes round.
template <int STREAM, int TEAM, int NV, bool STREAMING>
__global__ __launch_bounds__(TEAM * teams(TEAM)) void norm_backward_kernel(NormArgs a, const uint16_t* grad_y, const void* h_in,
                                                                const float* rstd, const void* grad_in, void* grad_h,
                                                                uint16_t* grad_x, float* partial) {
  __shared__ float s_part[2][TEAM / 64];
  const int tid = static_cast<int>(threadIdx.x) % TEAM;
  const int team = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TEAM);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams(TEAM) + team, step = static_cast<int64_t>(gridDim.x) * teams(TEAM);
  constexpr bool kQuads = STREAM == kF32Stream, kBf16 = !kQuads;
  constexpr int kAux = STREAMING ? kNonTemporal : 0;
  const int32_t H = a.H;
  float w[NV][8], acc[NV][8];
  load_weight<kQuads, TEAM>(a, tid, w);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.f;
  constexpr bool kAhead = kBf16;
  Raw8<kQuads, kBf16, kAux> h[NV], back[NV];
  Raw8<kQuads, true, kAux> g[NV];
  float inv = 0.f;
  const auto load = [&](int64_t row) {
    const __amdgpu_buffer_rsrc_t hr = row_of(h_in, row, H, kBf16), gr = row_of(grad_y, row, H, true);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v].load(hr, v * TEAM + tid);
      g[v].load(gr, v * TEAM + tid);
    }
    inv = rstd[row];
  };
  if (kAhead && first < a.rows) load(first);
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    if (!kAhead) load(row);
    if (grad_in != nullptr) {
      const __amdgpu_buffer_rsrc_t br = row_of(grad_in, row, H, kBf16);
#pragma unroll
      for (int v = 0; v < NV; ++v) back[v].load(br, v * TEAM + tid);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) back[v] = Raw8<kQuads, kBf16, kAux>{};
    }
    float n[NV][8], z[NV][8];
    const float scale = inv;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[v][j] = h[v].at(j) * scale;
        acc[v][j] += g[v].at(j) * n[v][j];
        z[v][j] = g[v].at(j) * w[v][j];
        sum += z[v][j] * n[v][j];
      }
    if (kAhead && row + step < a.rows) load(row + step);
    const float mean = team_sum<TEAM>(sum, s_part[turn]) / static_cast<float>(H);
    turn ^= 1;
    const __amdgpu_buffer_rsrc_t to = row_of(grad_h, row, H, kBf16);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * TEAM + tid;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = back[v].at(j) + scale * (z[v][j] - n[v][j] * mean);
      store8<kQuads, kBf16, kAux>(to, i, d);
      if (!kBf16 && grad_x != nullptr) store8<kQuads, true, kAux>(row_of(grad_x, row, H, true), i, d);
    }
  }
  if (partial == nullptr) return;
  if (TEAM == 64) {  // the other waves' parts to the first
    __shared__ float s_acc[teams(TEAM)][8][64];
#pragma unroll
    for (int j = 0; j < 8; ++j) s_acc[TEAM == 64 ? team : 0][j][tid & 63] = acc[0][j];
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int k = 1; k < teams(TEAM); ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[0][j] += s_acc[k][j][tid & 63];
  }
  const __amdgpu_buffer_rsrc_t pr = row_of(partial, blockIdx.x, H, false);
#pragma unroll
  for (int v = 0; v < NV; ++v) store8<kQuads, false, 0>(pr, v * TEAM + tid, acc[v]);
}

// grad_weight from the workgroups' parts: 64 columns a workgroup, each summed by
// kSlices threads in fp64, all loads of a thread at once.
constexpr int kSlices = 16;

__global__ __launch_bounds__(64 * kSlices) void norm_weight_kernel(const float* __restrict__ partial, int32_t parts, int32_t H,
                                                                   float* __restrict__ grad_weight, bool accumulate) {
  __shared__ double s_sum[kSlices][64];
  const int c = threadIdx.x & 63, s = threadIdx.x >> 6;
  const int32_t col = blockIdx.x * 64 + c;
  double x = 0.0;
  if (col < H) {
#pragma unroll 8
    for (int32_t i = s; i < parts; i += kSlices) x += static_cast<double>(partial[static_cast<int64_t>(i) * H + col]);
  }
  s_sum[s][c] = x;
  __syncthreads();
  if (s != 0 || col >= H) return;
  x = 0.0;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) x += s_sum[i][c];
  grad_weight[col] = static_cast<float>(accumulate ? static_cast<double>(grad_weight[col]) + x : x);
}

constexpr int32_t kTeamOfOne = 512;  // columns up to which a wave has a row of its own

// Workgroups of a pass.  Each reads a row ahead, so that few waves keep the memory busy,
// and more only stand in each other's way: 256 workgroups of eight waves take 365 us
// for 32771 rows of 7168, 512 408; below 4096 columns more are needed (16000 rows of
// 1024: 2048 workgroups 15.5 us, 512 28.5; of 2048: 512 51, 1024 55).
int32_t norm_blocks(int32_t H) { return H <= 1024 ? 2048 : H <= 4096 ? 512 : 256; }

// Of the backward pass, each with a part of grad_weight to write and to add up again:
// eight waves a CU (1021 rows of 4096: 256 workgroups 10.9 us, 512 13.2; 16000 rows of
// 1024: 1024 workgroups 25.9 us, 512 31.4, 2048 30.1).
int32_t backward_blocks(int64_t rows, int32_t H) {
  const int32_t most = H <= kTeamOfOne ? 512 : H <= 1024 ? 1024 : H <= 2048 ? 512 : 256;
  const int32_t at_once = H <= kTeamOfOne ? teams(64) : 1;
  return static_cast<int32_t>(rows < static_cast<int64_t>(most) * at_once ? (rows + at_once - 1) / at_once : most);
}

// Beyond the last-level cache's size a pass finds nothing of its rows there again, and
// goes round the caches (32768 rows of 7168 backwards: 300 us, 340 through them; 1021 rows
// of 4096, which stay there: 13.1 us, 10.9 through them).
constexpr int64_t kCacheBytes = 256 << 20;

template <int STREAM, int TEAM, int NV>
void launch_norm_as(const NormArgs& a, const uint16_t* x, const void* residual, float eps, void* h, uint16_t* y,
                    uint8_t* q, uint8_t* q_scale, float* rstd, hipStream_t st) {
  const int64_t want = (a.rows + teams(TEAM) - 1) / teams(TEAM);
  const dim3 grid(static_cast<uint32_t>(want < norm_blocks(a.H) ? want : norm_blocks(a.H))), block(TEAM * teams(TEAM));
  const int64_t bytes = a.rows * a.H * (4 + (STREAM == kF32Stream ? 8 : STREAM == kBf16Stream ? 4 : 0) + (q != nullptr ? 1 : 0));
  if (bytes > kCacheBytes)
    hipLaunchKernelGGL((norm_kernel<STREAM, TEAM, NV, true>), grid, block, 0, st, a, x, residual, eps, h, y, q,
                       q_scale, rstd);
  else
    hipLaunchKernelGGL((norm_kernel<STREAM, TEAM, NV, false>), grid, block, 0, st, a, x, residual, eps, h, y, q,
                       q_scale, rstd);
}

template <int STREAM>
void launch_norm_of(const NormArgs& a, const uint16_t* x, const void* residual, float eps, void* h, uint16_t* y,
                    uint8_t* q, uint8_t* q_scale, float* rstd, hipStream_t st) {
  const auto go = a.H <= kTeamOfOne ? launch_norm_as<STREAM, 64, 1>
                  : a.H <= 1024     ? launch_norm_as<STREAM, 128, 1>
                  : a.H <= 2048     ? launch_norm_as<STREAM, 256, 1>
                  : a.H <= 4096     ? launch_norm_as<STREAM, 512, 1>
                  : a.H <= 8192     ? launch_norm_as<STREAM, 512, 2>
                                    : launch_norm_as<STREAM, 1024, 2>;
  go(a, x, residual, eps, h, y, q, q_scale, rstd, st);
}

template <int STREAM, int TEAM, int NV>
void launch_backward_as(const NormArgs& a, const uint16_t* grad_y, const void* h, const float* rstd, const void* grad_in,
                        void* grad_h, uint16_t* grad_x, float* partial, hipStream_t st) {
  const dim3 grid(backward_blocks(a.rows, a.H)), block(TEAM * teams(TEAM));
  if (a.rows * a.H * (STREAM == kF32Stream ? 14 : 8) > kCacheBytes)
    hipLaunchKernelGGL((norm_backward_kernel<STREAM, TEAM, NV, true>), grid, block, 0, st, a, grad_y, h, rstd,
                       grad_in, grad_h, grad_x, partial);
  else
    hipLaunchKernelGGL((norm_backward_kernel<STREAM, TEAM, NV, false>), grid, block, 0, st, a, grad_y, h, rstd,
                       grad_in, grad_h, grad_x, partial);
}

template <int STREAM>
void launch_backward_of(const NormArgs& a, const uint16_t* grad_y, const void* h, const float* rstd, const void* grad_in,
                        void* grad_h, uint16_t* grad_x, float* partial, hipStream_t st) {
  const auto go = a.H <= kTeamOfOne ? launch_backward_as<STREAM, 64, 1>
                  : a.H <= 1024     ? launch_backward_as<STREAM, 128, 1>
                  : a.H <= 2048     ? launch_backward_as<STREAM, 256, 1>
                  : a.H <= 4096     ? launch_backward_as<STREAM, 512, 1>
                  : a.H <= 8192     ? launch_backward_as<STREAM, 512, 2>
                                    : launch_backward_as<STREAM, 1024, 2>;
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

size_t norm_workspace_bytes(int64_t rows, int32_t H) { return sizeof(float) * static_cast<size_t>(backward_blocks(rows, H)) * H; }

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
  hipLaunchKernelGGL(norm_weight_kernel, dim3((a.H + 63) / 64), dim3(64 * kSlices), 0, st, partial, backward_blocks(a.rows, a.H), a.H,
                     grad_weight, accumulate);
  return hipGetLastError();
}

}  // namespace ultraep
