// gfx950 kernels of the experts' 8-bit products (include/ultraep_experts.h):
// rows times weights for every physical expert of a segment, and the weight
// gradients.  Both are sums over blocks of 128,
//   C[i][j] = sum_b 2^(sa[i][b] + sb[j][b] - 254) * sum_{r < 128} A[i][b][r] * B[j][b][r],
// which is what one V_MFMA_SCALE_F32_16X16X128 does with a scale byte a row of
// either operand: the power-of-two scales cost no vector instruction.
//
// Its precision, measured on the card: of eight products that a lane adds
// together, every one is cut (towards zero) at 2^-13 of the largest one's power
// of two; their sums and the accumulator are fp32.  The cuts come to 1.5e-5 of
// the result on normal operands (2-norm), a hundredth of the bf16 rounding that
// the rows products end in, so those use it: it is twice as fast as bf16.  The
// weight gradients end in fp32 and may be added to for many steps: they widen
// the bytes to bf16, scale included, which is exact, and multiply in bf16,
// whose products and sums are fp32.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMmThreads = 256;
constexpr int kMmTile = 128;  // both ways

// One operand of a tile: 128 of its rows, row r at base + min(r, last) *
// row_pitch + b * block_pitch; its scale byte at scale + (min(r, last) >>
// row_shift) * scale_row + b * scale_block.
struct Operand {
  const uint8_t* base;
  const uint8_t* scale;
  int64_t row_pitch, block_pitch;
  int64_t scale_row, scale_block;
  int32_t last;
  int32_t row_shift;
};

// acc[i][j] of a wave: its 64 rows of A by its 64 rows of B as 4 x 4 products
// of 16 x 16.  LDS holds 128 bytes a row in eight 16-byte parts, part c at
// c ^ (row % 8), so that 16 lanes reading one part of 16 rows meet no bank twice
// more often than they must.
__device__ __forceinline__ bf16x8 widen(const i32x8& v, int g, float s) {
  bf16x8 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = static_cast<uint32_t>(v[2 * g + i / 2]);
    const bf16x2 b = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true)
                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
    y[2 * i] = b[0];
    y[2 * i + 1] = b[1];
  }
  return y;
}

__device__ __forceinline__ float scale_of(int byte) { return __builtin_bit_cast(float, static_cast<uint32_t>(byte) << 23); }

template <bool WIDE>
__device__ __forceinline__ void mm_tile(const Operand& a, const Operand& b, int32_t blocks, uint8_t* sa, uint8_t* sb,
                                        f32x4 (&acc)[4][4]) {
  const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6, wi = wv >> 1, wj = wv & 1;
  const int l16 = lane & 15, kg = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int32_t blk = 0; blk < blocks; ++blk) {
    u32x4 va[4], vb[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = tid + u * kMmThreads, r = x >> 3, c = x & 7;
      va[u] = *reinterpret_cast<const u32x4*>(a.base + min(r, a.last) * a.row_pitch + blk * a.block_pitch + c * 16);
      vb[u] = *reinterpret_cast<const u32x4*>(b.base + min(r, b.last) * b.row_pitch + blk * b.block_pitch + c * 16);
    }
    int xa[4], xb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = min(wi * 64 + i * 16 + l16, a.last), rb = min(wj * 64 + i * 16 + l16, b.last);
      xa[i] = a.scale[static_cast<int64_t>(ra >> a.row_shift) * a.scale_row + blk * a.scale_block];
      xb[i] = b.scale[static_cast<int64_t>(rb >> b.row_shift) * b.scale_row + blk * b.scale_block];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = tid + u * kMmThreads, r = x >> 3, c = x & 7;
      *reinterpret_cast<u32x4*>(sa + r * 128 + ((c ^ r) & 7) * 16) = va[u];
      *reinterpret_cast<u32x4*>(sb + r * 128 + ((c ^ r) & 7) * 16) = vb[u];
    }
    __syncthreads();
    i32x8 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = wi * 64 + i * 16 + l16, rb = wj * 64 + i * 16 + l16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(sa + ra * 128 + (((2 * kg + h) ^ ra) & 7) * 16);
        const i32x4 y = *reinterpret_cast<const i32x4*>(sb + rb * 128 + (((2 * kg + h) ^ rb) & 7) * 16);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          fa[i][4 * h + d] = x[d];
          fb[i][4 * h + d] = y[d];
        }
      }
    }
    if (WIDE) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        bf16x8 wa[4], wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wa[i] = widen(fa[i], g, scale_of(xa[i]));
          wb[i] = widen(fb[i], g, scale_of(xb[i]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[i], wb[j], acc[i][j], 0, 0, 0);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[i], fb[j], acc[i][j], 0, 0, 0, xa[i], 0, xb[j]);
  }
}

// out[row][n]: A is the weights (a lane's four accumulators are consecutive
// n), B the rows.
__global__ __launch_bounds__(kMmThreads) void expert_gemm_kernel(
    const int32_t* __restrict__ off, int32_t ne, const uint8_t* __restrict__ q, const uint8_t* __restrict__ q_scale,
    int32_t K, const uint8_t* const* __restrict__ w, const uint8_t* const* __restrict__ w_scale, int32_t N,
    uint16_t* __restrict__ out, int64_t cap, int64_t tiles, int32_t ntile) {
  __shared__ __align__(16) uint8_t s_a[kMmTile * 128], s_b[kMmTile * 128];
  const int32_t Kp = q_pitch(K), Ks = s_pitch(K);
  const int lane = lane_id(), wv = threadIdx.x >> 6, wi = wv >> 1, wj = wv & 1;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int32_t tm = static_cast<int32_t>(t / ntile), tn = static_cast<int32_t>(t - static_cast<int64_t>(tm) * ntile);
    const int32_t p = find_group(off, ne, cap, kMmTile, tm);
    const int32_t o = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
    const int64_t row0 = o + static_cast<int64_t>(tm - (o / kMmTile + p)) * kMmTile;
    if (row0 >= o1) continue;
    const uint8_t* wp = w[p];
    const uint8_t* ws = w_scale[p];
    if (wp == nullptr || ws == nullptr || (reinterpret_cast<uintptr_t>(wp) & 15) != 0 ||
        (reinterpret_cast<uintptr_t>(ws) & 3) != 0)
      continue;
    const int32_t n0 = tn * kMmTile;
    const int32_t rows = static_cast<int32_t>(min(static_cast<int64_t>(o1) - row0, static_cast<int64_t>(kMmTile)));
    const int32_t cols = min(N - n0, kMmTile);
    const Operand a{wp + static_cast<int64_t>(n0) * Kp, ws + static_cast<int64_t>(tn) * Ks, Kp, 128, Ks, 1, cols - 1, 7};
    const Operand b{q + row0 * Kp, q_scale + row0 * Ks, Kp, 128, Ks, 1, rows - 1, 0};
    f32x4 acc[4][4];
    mm_tile<false>(a, b, Kp / 128, s_a, s_b, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wj * 64 + j * 16 + (lane & 15), c = wi * 64 + i * 16 + 4 * (lane >> 4);
        if (r < rows && c < cols) {
          u32x2 y;
          y[0] = pack_bf16(acc[i][j][0], acc[i][j][1]);
          y[1] = pack_bf16(acc[i][j][2], acc[i][j][3]);
          *reinterpret_cast<u32x2*>(out + (row0 + r) * N + n0 + c) = y;
        }
      }
  }
}

// grads[p][n][k]: A is x (four consecutive k a lane), B is dy.
__global__ __launch_bounds__(kMmThreads) void expert_wgrad_kernel(
    const int32_t* __restrict__ off, int32_t ne, const uint8_t* __restrict__ dyt, const uint8_t* __restrict__ dyt_scale,
    int32_t N, const uint8_t* __restrict__ xt, const uint8_t* __restrict__ xt_scale, int32_t K, int64_t cap,
    float* const* __restrict__ grads, bool accumulate, int64_t tiles, int32_t ntile, int32_t ktile) {
  __shared__ __align__(16) uint8_t s_a[kMmTile * 128], s_b[kMmTile * 128];
  const int lane = lane_id(), wv = threadIdx.x >> 6, wi = wv >> 1, wj = wv & 1;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int32_t per = ntile * ktile;
    const int32_t p = static_cast<int32_t>(t / per), rest = static_cast<int32_t>(t - static_cast<int64_t>(p) * per);
    const int32_t tn = rest / ktile, tk = rest - tn * ktile;
    float* g = grads[p];
    if (g == nullptr) continue;
    const int32_t o = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
    const int32_t blocks = max(ceil_div(o1 - o, kQBlock), 0);
    if (blocks == 0 && accumulate) continue;
    const int64_t b0 = o / kQBlock + p;
    const int32_t n0 = tn * kMmTile, k0 = tk * kMmTile;
    const int32_t rows = min(N - n0, kMmTile), cols = min(K - k0, kMmTile);
    const Operand a{xt + (b0 * K + k0) * kQBlock, xt_scale + b0 * K + k0, 128, static_cast<int64_t>(K) * kQBlock, 1, K, cols - 1, 0};
    const Operand b{dyt + (b0 * N + n0) * kQBlock, dyt_scale + b0 * N + n0, 128, static_cast<int64_t>(N) * kQBlock, 1, N, rows - 1, 0};
    f32x4 acc[4][4];
    mm_tile<true>(a, b, blocks, s_a, s_b, acc);
    const bool vec = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wj * 64 + j * 16 + (lane & 15), c = wi * 64 + i * 16 + 4 * (lane >> 4);
        if (r < rows && c < cols) {
          float* d = g + static_cast<int64_t>(n0 + r) * K + k0 + c;
          f32x4 y = acc[i][j];
          if (vec) {
            if (accumulate) y += *reinterpret_cast<const f32x4*>(d);
            *reinterpret_cast<f32x4*>(d) = y;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = accumulate ? d[e] + y[e] : y[e];
          }
        }
      }
  }
}

uint32_t mm_grid(int64_t tiles) { return static_cast<uint32_t>(tiles < (1 << 20) ? tiles : (1 << 20)); }

}  // namespace

hipError_t launch_expert_gemm(const int32_t* off, int32_t ne, const uint8_t* q, const uint8_t* q_scale, int32_t K,
                              const uint8_t* const* w, const uint8_t* const* w_scale, int32_t N, uint16_t* out,
                              int64_t cap, hipStream_t st) {
  if (ne == 0 || cap == 0) return hipSuccess;
  const int32_t ntile = ceil_div(N, kMmTile);
  const int64_t tiles = (cap / kMmTile + ne) * ntile;
  hipLaunchKernelGGL(expert_gemm_kernel, dim3(mm_grid(tiles)), dim3(kMmThreads), 0, st, off, ne, q, q_scale, K, w,
                     w_scale, N, out, cap, tiles, ntile);
  return hipGetLastError();
}

hipError_t launch_expert_wgrad(const int32_t* off, int32_t ne, const uint8_t* dyt, const uint8_t* dyt_scale, int32_t N,
                               const uint8_t* xt, const uint8_t* xt_scale, int32_t K, int64_t cap, float* const* grads,
                               bool accumulate, hipStream_t st) {
  if (ne == 0) return hipSuccess;
  const int32_t ntile = ceil_div(N, kMmTile), ktile = ceil_div(K, kMmTile);
  const int64_t tiles = static_cast<int64_t>(ne) * ntile * ktile;
  hipLaunchKernelGGL(expert_wgrad_kernel, dim3(mm_grid(tiles)), dim3(kMmThreads), 0, st, off, ne, dyt, dyt_scale, N, xt,
                     xt_scale, K, cap, grads, accumulate, tiles, ntile, ktile);
  return hipGetLastError();
}

}  // namespace ultraep
