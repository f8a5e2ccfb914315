// gfx950 kernels that quantise rows and weights to e4m3 with a power-of-two
// scale for each block of 128 (include/ultraep_experts.h, "Format").
//
// Both directions of the format are made from one read.  All kernels are
// HBM-streaming: two bytes read and one (two with both forms) written a value.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWaves = kQuantThreads / 64;
constexpr int kRowChunk = 512;  // columns a wave quantises: 64 lanes x 8

// Where the segment's rows come from: hidden[inv[seg0 + i] / k], or hidden[i].
struct RowSource {
  const int32_t* inv;
  int32_t k;
  const uint16_t* hidden;
  int64_t hidden_rows;
};

__device__ __forceinline__ int64_t source_row(const RowSource& s, int32_t seg0, int64_t i) {
  if (s.inv == nullptr) return i < s.hidden_rows ? i : -1;
  const int32_t n = s.inv[static_cast<int64_t>(seg0) + i];
  const int32_t t = n >= 0 ? n / s.k : -1;
  return t < s.hidden_rows ? t : -1;
}

// Rows form alone: one wave per (row, 512 columns), 16 lanes a block, so a
// block's maximum is four DPP steps and its four scale bytes one store.  Bound by
// HBM: 32771 rows of 7168 gathered and quantised, 706 MB, 145 us (4.9 TB/s;
// 20700 distinct tokens, but the counters show every row read); ordinary instead of
// non-temporal stores 151.
__global__ __launch_bounds__(kQuantThreads) void quant_rows_kernel(
    const int32_t* __restrict__ off, int32_t ne, RowSource in, int32_t H, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale, int64_t cap) {
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t Hp = q_pitch(H), Hs = s_pitch(H), nch = Hs / 4;
  const int32_t seg0 = off[0];
  const int64_t rows = group_row(off, ne, cap);
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kQuantWaves;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kQuantWaves + wv; item < rows * nch; item += nwaves) {
    const int64_t row = item / nch;
    const int32_t ch = static_cast<int32_t>(item - row * nch);
    const int64_t t = source_row(in, seg0, row);
    const int32_t tlo = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(t));
    const __amdgpu_buffer_rsrc_t src = row_rsrc(in.hidden + static_cast<int64_t>(max(tlo, 0)) * H,
                                                tlo < 0 ? 0u : 2u * static_cast<uint32_t>(H));
    const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(src, ch * 2 * kRowChunk + lane * 16, 0, kNonTemporal);
    const int32_t e = block_exponent(row16_amax(x));
    const u32x2 y = to_e4m3(x, power_of_two(e));
    const __amdgpu_buffer_rsrc_t dst = row_rsrc(q + row * Hp, static_cast<uint32_t>(Hp));
    __builtin_amdgcn_raw_buffer_store_b64(y, dst, ch * kRowChunk + lane * 8, 0, kNonTemporal);
    uint32_t s = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) s |= (readlane(static_cast<uint32_t>(e), 16 * b) + 127u) << (8 * b);
    if (lane == 0) *reinterpret_cast<uint32_t*>(scale + row * Hs + 4 * ch) = s;
  }
}

// 128 x 128 tiles, transposed on their way out.  A thread holds 8 x 8 values:
// row group g = thread / 16 (rows 8g..8g+7), column group c = thread % 16.
// Bytes wait in LDS as [column][row] with the 8-byte row groups of a column
// exchanged by g ^ (column / 8), so that neither the stores (16 column groups
// at once) nor the reads have bank conflicts.
__device__ __forceinline__ void put_column_bytes(uint8_t* tile, int c, int g, const u32x2 (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<u32x2*>(tile + (8 * c + j) * kQBlock + ((g ^ c) & 15) * 8) = b[j];
}

// 16 rows (r0 = 16 * part) of column h.
__device__ __forceinline__ u32x4 get_column_bytes(const uint8_t* tile, int h, int part) {
  const int c = (h >> 3) & 15;
  const u32x4 v = *reinterpret_cast<const u32x4*>(tile + h * kQBlock + (((2 * part) ^ (c & 14)) * 8));
  return (c & 1) ? u32x4{v[2], v[3], v[0], v[1]} : v;
}

// 8 x 8 transpose of bytes: b[j] holds column j's rows from a's rows.
__device__ __forceinline__ void transpose_bytes(const u32x2 (&a)[8], u32x2 (&b)[8]) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {      // columns 4*half..4*half+3
#pragma unroll
    for (int quad = 0; quad < 2; ++quad) {    // rows 4*quad..4*quad+3
      const uint32_t r0 = a[4 * quad][half], r1 = a[4 * quad + 1][half], r2 = a[4 * quad + 2][half],
                     r3 = a[4 * quad + 3][half];
      const uint32_t lo01 = __builtin_amdgcn_perm(r1, r0, 0x05010400u);  // r0b0 r1b0 r0b1 r1b1
      const uint32_t hi01 = __builtin_amdgcn_perm(r1, r0, 0x07030602u);  // r0b2 r1b2 r0b3 r1b3
      const uint32_t lo23 = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
      const uint32_t hi23 = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
      b[4 * half + 0][quad] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
      b[4 * half + 1][quad] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
      b[4 * half + 2][quad] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
      b[4 * half + 3][quad] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
    }
  }
}

// Columns form, and the rows form with it: one workgroup per 128 rows of one
// expert and 128 columns, so that a column block is its own and the rows are
// read once for both.  16411 rows of 4096, both forms, 270 MB: 54 us, 5.0 TB/s.
template <bool ROWS>
__global__ __launch_bounds__(kQuantThreads) void quant_cols_kernel(
    const int32_t* __restrict__ off, int32_t ne, RowSource in, int32_t H, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale, uint8_t* __restrict__ qt, uint8_t* __restrict__ scale_t, int64_t cap,
    int32_t nblk, int32_t ncol) {
  __shared__ __align__(16) uint8_t s_tile[kQBlock * kQBlock];
  __shared__ u32x4 s_max[16][16];
  __shared__ float s_scale[kQBlock];
  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4;
  const int32_t seg0 = off[0];
  const int32_t Hp = q_pitch(H), Hs = s_pitch(H);
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(nblk) * ncol; item += gridDim.x) {
    const int32_t b = static_cast<int32_t>(item / ncol), cb = static_cast<int32_t>(item - static_cast<int64_t>(b) * ncol);
    const int32_t p = find_group(off, ne, cap, kQBlock, b);
    const int32_t o = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
    const int64_t row0 = o + static_cast<int64_t>(b - (o / kQBlock + p)) * kQBlock;
    const int32_t live = static_cast<int32_t>(min(static_cast<int64_t>(o1) - row0, static_cast<int64_t>(kQBlock)));
    if (live <= 0) continue;  // the same for the whole workgroup
    const int32_t h0 = cb * kQBlock + 8 * c, hc = min(h0, H - 8);
    // every lane loads (a row that is not there: row 0) and unwanted values are
    // cleared; stores go through resources that end with the block's rows
    u32x4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = u32x4{0, 0, 0, 0};
    if (in.hidden_rows > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * g + i;
        const int32_t tok = static_cast<int32_t>(source_row(in, seg0, row0 + min(r, live - 1)));
        x[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(in.hidden + static_cast<int64_t>(max(tok, 0)) * H + hc));
        const uint32_t keep = r < live && tok >= 0 && h0 < H ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] &= keep;
      }
    }
    if (ROWS) {
      const __amdgpu_buffer_rsrc_t to_q = row_rsrc(q + row0 * Hp, static_cast<uint32_t>(live) * static_cast<uint32_t>(Hp));
      const __amdgpu_buffer_rsrc_t to_s = row_rsrc(scale + row0 * Hs, static_cast<uint32_t>(live) * static_cast<uint32_t>(Hs));
      // one scale byte a row, and behind the last block the padding's
      const bool pad = c > 0 && cb == ncol - 1 && cb + c < Hs;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * g + i;
        const int32_t e = block_exponent(row16_amax(x[i]));
        __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(x[i], power_of_two(e)), to_q, r * Hp + h0, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(c == 0 ? e + 127 : 127), to_s,
                                             c == 0 || pad ? r * Hs + cb + c : 0x7FFFFFFF, 0, 0);
      }
    }
    // column maxima: over the thread's rows, then over the 16 row groups
    int32_t e = 0;
    const auto column_maxima = [&](auto finite) {
      u32x4 m = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = pair_max(m[j], magnitudes<decltype(finite)::value>(x[i][j]));
      __syncthreads();  // earlier readers are done
      s_max[g][c] = m;
      __syncthreads();
      uint32_t mm = 0;
      if (tid < kQBlock) {
        const uint16_t* col = reinterpret_cast<const uint16_t*>(s_max) + tid;
#pragma unroll
        for (int i = 0; i < 16; ++i) mm = max(mm, static_cast<uint32_t>(col[i * kQBlock]));
        e = block_exponent(mm);
        s_scale[tid] = power_of_two(e);
      }
      return __syncthreads_or(mm >= kNotFinite) != 0;
    };
    if (column_maxima(std::false_type{})) column_maxima(std::true_type{});
    if (tid < kQBlock) {
      const int32_t h = cb * kQBlock + tid;
      if (h < H) scale_t[static_cast<int64_t>(b) * H + h] = static_cast<uint8_t>(e + 127);
    }
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = s_scale[8 * c + j];
    // column j's rows in pairs, then in bytes
    u32x2 bt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
      uint32_t pair[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pair[i] = __builtin_amdgcn_perm(x[2 * i + 1][j / 2], x[2 * i][j / 2], sel);
      bt[j] = u32x2{to_e4m3(pair[0], pair[1], sc[j]), to_e4m3(pair[2], pair[3], sc[j])};
    }
    put_column_bytes(s_tile, c, g, bt);
    __syncthreads();
    const int32_t hcols = min(kQBlock, H - cb * kQBlock);
    u32x4* out = reinterpret_cast<u32x4*>(qt + (static_cast<int64_t>(b) * H + static_cast<int64_t>(cb) * kQBlock) * kQBlock);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid + i * kQuantThreads, h = u >> 3, part = u & 7;
      if (h < hcols) out[u] = get_column_bytes(s_tile, h, part);
    }
  }
}

// One workgroup per 128 x 128 block of one expert's weights, which has one scale
// and is written both ways from the same registers.  6 experts of 4096 x 7168,
// both orders, 705 MB: 136 us, 5.2 TB/s.
__global__ __launch_bounds__(kQuantThreads) void weight_quant_kernel(
    const uint16_t* const* __restrict__ weights, int32_t n, int32_t N, int32_t K, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale, uint8_t* __restrict__ qt, uint8_t* __restrict__ scale_t) {
  __shared__ __align__(16) uint8_t s_tile[kQBlock * kQBlock];
  __shared__ uint32_t s_max[kQuantWaves];
  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4;
  const int32_t nb = ceil_div(N, kQBlock), kb = ceil_div(K, kQBlock);
  const int64_t per = static_cast<int64_t>(nb) * kb;
  for (int64_t item = blockIdx.x; item < per * n; item += gridDim.x) {
    const int64_t ex = item / per;
    const int32_t rest = static_cast<int32_t>(item - ex * per), bn = rest / kb, bk = rest - bn * kb;
    const uint16_t* w = weights[ex];
    if (w == nullptr) continue;
    const int32_t n0 = bn * kQBlock + 8 * g, k0 = bk * kQBlock + 8 * c;
    const bool vec = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
    u32x4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = u32x4{0, 0, 0, 0};
      if (n0 + i < N && k0 < K) {
        const uint16_t* s = w + static_cast<int64_t>(n0 + i) * K + k0;
        if (vec) {
          x[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(s));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = s[2 * j] | (static_cast<uint32_t>(s[2 * j + 1]) << 16);
        }
      }
    }
    const auto block_amax = [&](auto finite) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, amax_of<decltype(finite)::value>(x[i]));
      m = wave_max(m);
      __syncthreads();  // earlier readers are done
      if ((tid & 63) == 0) s_max[tid >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kQuantWaves; ++i) m = max(m, s_max[i]);
      return m;
    };
    uint32_t m = block_amax(std::false_type{});
    if (m >= kNotFinite) m = block_amax(std::true_type{});  // the same for the whole workgroup
    const int32_t e = block_exponent(m);
    u32x2 a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = to_e4m3(x[i], power_of_two(e));
    if (q != nullptr) {
      const int32_t Kp = q_pitch(K), Ks = s_pitch(K);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n0 + i < N) *reinterpret_cast<u32x2*>(q + (ex * N + n0 + i) * Kp + k0) = a[i];
      uint8_t* s = scale + (ex * nb + bn) * Ks;
      if (tid == 0) s[bk] = static_cast<uint8_t>(e + 127);
      if (bk == kb - 1 && tid > 0 && bk + tid < Ks) s[bk + tid] = 127;
    }
    if (qt != nullptr) {
      u32x2 bt[8];
      transpose_bytes(a, bt);
      put_column_bytes(s_tile, c, g, bt);
      __syncthreads();
      const int32_t Np = q_pitch(N), Ns = s_pitch(N), kcols = min(kQBlock, K - bk * kQBlock);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = tid + i * kQuantThreads, h = u >> 3, part = u & 7;
        if (h < kcols)
          *reinterpret_cast<u32x4*>(qt + (ex * K + bk * kQBlock + h) * Np + bn * kQBlock + part * 16) =
              get_column_bytes(s_tile, h, part);
      }
      uint8_t* s = scale_t + (ex * kb + bk) * Ns;
      if (tid == 0) s[bn] = static_cast<uint8_t>(e + 127);
      if (bn == nb - 1 && tid > 0 && bn + tid < Ns) s[bn + tid] = 127;
    }
  }
}

uint32_t grid_of(int64_t want) { return static_cast<uint32_t>(want < (1 << 20) ? want : (1 << 20)); }

}  // namespace

hipError_t launch_permute_quant(const int32_t* off, int32_t ne, const int32_t* inv, int32_t k,
                                const uint16_t* hidden, int64_t hidden_rows, int32_t H, uint8_t* q,
                                uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, int64_t cap,
                                hipStream_t st) {
  if (ne == 0 || cap == 0) return hipSuccess;
  const RowSource in{inv, k, hidden, hidden_rows};
  if (qt == nullptr) {
    const int64_t items = cap * (s_pitch(H) / 4);
    hipLaunchKernelGGL(quant_rows_kernel, dim3(grid_of((items + kQuantWaves - 1) / kQuantWaves)), dim3(kQuantThreads),
                       0, st, off, ne, in, H, q, q_scale, cap);
    return hipGetLastError();
  }
  const int32_t nblk = static_cast<int32_t>(cap / kQBlock) + ne, ncol = ceil_div(H, kQBlock);
  const uint32_t grid = grid_of(static_cast<int64_t>(nblk) * ncol);
  if (q != nullptr)
    hipLaunchKernelGGL(quant_cols_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, off, ne, in, H, q, q_scale, qt,
                       qt_scale, cap, nblk, ncol);
  else
    hipLaunchKernelGGL(quant_cols_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, off, ne, in, H, q, q_scale, qt,
                       qt_scale, cap, nblk, ncol);
  return hipGetLastError();
}

hipError_t launch_weight_quant(const uint16_t* const* weights, int32_t n, int32_t N, int32_t K,
                               uint8_t* q, uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale,
                               hipStream_t st) {
  if (n == 0) return hipSuccess;
  const int64_t blocks = static_cast<int64_t>(n) * ceil_div(N, kQBlock) * ceil_div(K, kQBlock);
  hipLaunchKernelGGL(weight_quant_kernel, dim3(grid_of(blocks)), dim3(kQuantThreads), 0, st, weights, n, N, K, q,
                     q_scale, qt, qt_scale);
  return hipGetLastError();
}

}  // namespace ultraep
