// gfx950 kernels of the gated activation between the experts' two products and of its
// gradient rows, quantised on their way out (include/ultraep_layer.h).  Bound by HBM:
// 32771 rows of 2048, both forms, 403 MB: 72 us, 5.6 TB/s; their gradients, 671 MB:
// 152 us, 4.4 TB/s (the registers of two halves leave a CU one workgroup; 219 with every
// half read for itself), in rows alone 92 us, 5.9 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

__device__ __forceinline__ float half_of(const u32x4& v, int i) { return i & 1 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]); }

// Eight columns: of a = f(g) u, or of its gradients d u f'(g) and (upper) d f(g).
template <bool BACK, bool GELU>
__device__ __forceinline__ void glu8(const u32x4& g, const u32x4& u, const u32x4& d, bool upper, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float dz;
    const float gi = half_of(g, i), p = gate<GELU>(gi, dz), f = gi * p;
    float x = f * half_of(u, i);
    if (BACK) x = half_of(d, i) * (upper ? f : half_of(u, i) * (p + f * (1.f - p) * dz));
    o[i] = nothing_tiny(x);
  }
}

// Both gradients at once.
template <bool GELU>
__device__ __forceinline__ void glu8_both(const u32x4& g, const u32x4& u, const u32x4& d, float (&lower)[8], float (&upper)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float dz;
    const float gi = half_of(g, i), di = half_of(d, i), p = gate<GELU>(gi, dz), f = gi * p;
    lower[i] = nothing_tiny(di * (half_of(u, i) * (p + f * (1.f - p) * dz)));
    upper[i] = nothing_tiny(di * f);
  }
}

// Eight columns in memory, past the caches or through them.
template <bool STREAMING>
__device__ __forceinline__ u32x4 glu_read(const uint16_t* p) {
  const u32x4* v = reinterpret_cast<const u32x4*>(p);
  return STREAMING ? __builtin_nontemporal_load(v) : *v;
}

// Columns h0.. of row `row`, zeros where there are none.  (What gradients are made of is
// read twice here, so the caches are wanted for it.)
template <bool BACK, bool GELU, bool STREAMING>
__device__ __forceinline__ void glu_load(const GluRows& in, int64_t row, int32_t h0, bool there, float (&o)[8]) {
  const bool upper = BACK && h0 >= in.F;
  const int32_t c = there ? (upper ? h0 - in.F : h0) : 0;
  const uint16_t* h = in.h + row * (2 * static_cast<int64_t>(in.F)) + c;
  u32x4 d = {0, 0, 0, 0};
  const u32x4 g = glu_read<STREAMING && !BACK>(h), u = glu_read<STREAMING && !BACK>(h + in.F);
  if (BACK) d = glu_read<false>(in.grad + row * in.F + c);
  glu8<BACK, GELU>(g, u, d, upper, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = there ? o[i] : 0.f;
}

// Rows form of a wave's 512 columns from h0 - 8 * lane on, 16 lanes a block; a byte of
// scale from the first lane of each.
__device__ __forceinline__ void glu_store_row(const float (&x)[8], uint8_t* q, uint8_t* scale, int64_t row, int32_t W, int32_t h0) {
  const int32_t Wp = q_pitch(W), Ws = s_pitch(W), e = block_exponent_f32(row16_amax(x));
  __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(x, power_of_two(e)), row_rsrc(q + row * Wp, static_cast<uint32_t>(Wp)), h0, 0, 0);
  if (lane_id() % 16 == 0)
    __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(e + 127), row_rsrc(scale + row * Ws, static_cast<uint32_t>(Ws)),
                                         h0 / kQBlock, 0, 0);
}

// Rows form alone: one wave per (row, 512 columns); of gradients of whole blocks (PAIR)
// 512 columns of either half, so that what both are made of is read and activated once.
template <bool BACK, bool GELU, bool PAIR>
__global__ __launch_bounds__(kGluThreads) void glu_rows_kernel(const int32_t* __restrict__ off, int32_t ne, GluRows in,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                               int64_t cap, int32_t nch) {
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t F = in.F, W = BACK ? 2 * F : F;
  const int64_t rows = group_row(off, ne, cap);
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kGluWaves;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGluWaves + wv; item < rows * nch; item += nwaves) {
    const int64_t row = item / nch;
    const int32_t ch = static_cast<int32_t>(item - row * nch), h0 = ch * kGluChunk + lane * 8;
    float x[8];
    if constexpr (PAIR) {
      float y[8];
      const bool there = h0 < F;
      const uint16_t* h = in.h + row * (2 * static_cast<int64_t>(F)) + (there ? h0 : 0);
      const u32x4 gate = glu_read<true>(h), up = glu_read<true>(h + F);
      glu8_both<GELU>(gate, up, glu_read<true>(in.grad + row * F + (there ? h0 : 0)), x, y);
      // lanes behind the half store nothing; the last blocks' padding is 127
      const int32_t at = there ? h0 : 0x40000000;
      glu_store_row(x, q, scale, row, W, at);
      glu_store_row(y, q, scale, row, W, there ? F + h0 : at);
      const int32_t Ws = s_pitch(W);
      if (ch == 0 && lane < Ws - W / kQBlock) scale[row * Ws + W / kQBlock + lane] = 127;
    } else {
      glu_load<BACK, GELU, false>(in, row, h0, h0 < W, x);
      glu_store_row(x, q, scale, row, W, h0);
    }
  }
}

// 128 x 128 tiles: a thread has kTileRows x 8 values, rows kTileRows * g.. and columns
// 8 * c.. .
constexpr int kTileThreads = 512;
constexpr int kTileRows = 4;

// What the workgroup shares.  Bytes wait as [column][row], the 16-byte row groups of a
// column exchanged by its thread's c, so that neither the 4-byte stores nor the 16-byte
// reads meet in one bank more than twice.
struct GluShared {
  __align__(16) uint8_t tile[kQBlock * kQBlock];
  uint32_t max[kQBlock];  // zeros between tiles
  float scale[kQBlock];
};

struct GluOut {
  uint8_t* q;
  uint8_t* scale;
  uint8_t* qt;
  uint8_t* scale_t;
  int32_t W;  // columns of the results
};

// One tile of the results: live rows from row0 on, of one expert, in its block b, and the
// 128 columns from 128 * cb on; in both forms or in columns alone.
// Rows go past the caches too where a workgroup writes BOTH halves (152 us, 155 through
// them); else not (74 us, 72 through them).
template <bool ROWS, bool STREAMING, bool BOTH>
__device__ __forceinline__ void glu_tile(const GluOut& to, GluShared& s, const float (&x)[kTileRows][8], int64_t row0, int32_t live,
                                         int32_t b, int32_t cb) {
  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4;
  const int32_t W = to.W, Wp = q_pitch(W), Ws = s_pitch(W), h0 = cb * kQBlock + 8 * c;
  if (ROWS) {
    const __amdgpu_buffer_rsrc_t to_q = row_rsrc(to.q + row0 * Wp, static_cast<uint32_t>(live) * static_cast<uint32_t>(Wp));
    const __amdgpu_buffer_rsrc_t to_s = row_rsrc(to.scale + row0 * Ws, static_cast<uint32_t>(live) * static_cast<uint32_t>(Ws));
    // one scale byte a row, and behind the last block the padding's
    const bool pad = c > 0 && cb == ceil_div(W, kQBlock) - 1 && cb + c < Ws;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
      const int r = kTileRows * g + i;
      const int32_t e = block_exponent_f32(row16_amax(x[i]));
      __builtin_amdgcn_raw_buffer_store_b64(to_e4m3(x[i], power_of_two(e)), to_q, r * Wp + h0, 0, STREAMING && BOTH ? kNonTemporal : 0);
      __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(c == 0 ? e + 127 : 127), to_s,
                                           c == 0 || pad ? r * Ws + cb + c : 0x7FFFFFFF, 0, 0);
    }
  }
  // column maxima: over the thread's rows, then over the row groups
  const auto column_maxima = [&](auto finite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float column[kTileRows];
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) column[i] = x[i][j];
      atomicMax(&s.max[8 * c + j], amax_of<decltype(finite)::value>(column));
    }
    __syncthreads();
    uint32_t m = 0;
    if (tid < kQBlock) {
      m = s.max[tid];
      s.max[tid] = 0;
      const int32_t e = block_exponent_f32(m), h = cb * kQBlock + tid;
      s.scale[tid] = power_of_two(e);
      if (m < kNotFiniteF32 && h < W) to.scale_t[static_cast<int64_t>(b) * W + h] = static_cast<uint8_t>(e + 127);
    }
    return __syncthreads_or(m >= kNotFiniteF32) != 0;
  };
  if (column_maxima(std::false_type{})) column_maxima(std::true_type{});
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint8_t* at = s.tile + (8 * c + j) * kQBlock + (((kTileRows * g) >> 4) ^ (c & 7)) * 16 + ((kTileRows * g) & 15);
    *reinterpret_cast<uint32_t*>(at) = to_e4m3(x[0][j], x[1][j], x[2][j], x[3][j], s.scale[8 * c + j]);
  }
  __syncthreads();
  const int32_t cols = min(kQBlock, W - cb * kQBlock);
  u32x4* out = reinterpret_cast<u32x4*>(to.qt + (static_cast<int64_t>(b) * W + static_cast<int64_t>(cb) * kQBlock) * kQBlock);
#pragma unroll
  for (int i = 0; i < kQBlock * kQBlock / 16 / kTileThreads; ++i) {
    const int u = tid + i * kTileThreads, h = u >> 3, part = u & 7;
    if (h >= cols) continue;
    const u32x4 v = *reinterpret_cast<const u32x4*>(s.tile + h * kQBlock + (part ^ ((h >> 3) & 7)) * 16);
    if (STREAMING)
      __builtin_nontemporal_store(v, out + u);
    else
      out[u] = v;
  }
}

// Columns form, and the rows form with it: one workgroup per 128 rows of one expert and
// 128 columns; of gradients of whole blocks (PAIR) 128 columns of either half, so that
// what both are made of is read and activated once.
template <bool BACK, bool GELU, bool ROWS, bool PAIR, bool STREAMING>
__global__ __launch_bounds__(kTileThreads) void glu_cols_kernel(const int32_t* __restrict__ off, int32_t ne, GluRows in, GluOut to,
                                                                int64_t cap, int32_t nblk, int32_t ncol) {
  __shared__ GluShared s;
  if (threadIdx.x < kQBlock) s.max[threadIdx.x] = 0;
  __syncthreads();
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(nblk) * ncol; item += gridDim.x) {
    const int32_t b = static_cast<int32_t>(item / ncol), cb = static_cast<int32_t>(item - static_cast<int64_t>(b) * ncol);
    const int32_t p = find_group(off, ne, cap, kQBlock, b);
    const int32_t o = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
    const int64_t row0 = o + static_cast<int64_t>(b - (o / kQBlock + p)) * kQBlock;
    const int32_t live = static_cast<int32_t>(min(static_cast<int64_t>(o1) - row0, static_cast<int64_t>(kQBlock)));
    if (live <= 0) continue;  // the same for the whole workgroup
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // addresses made anew rather than kept
    const int c = tid & 15, g = tid >> 4;
    const int32_t h0 = cb * kQBlock + 8 * c;
    float x[kTileRows][8];
    if constexpr (PAIR) {
      float y[kTileRows][8];
      u32x4 gate[kTileRows], up[kTileRows], d[kTileRows];
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) {
        const int64_t row = row0 + min(kTileRows * g + i, live - 1);
        const uint16_t* h = in.h + row * (2 * static_cast<int64_t>(in.F)) + h0;
        gate[i] = glu_read<STREAMING>(h);
        up[i] = glu_read<STREAMING>(h + in.F);
        d[i] = glu_read<STREAMING>(in.grad + row * in.F + h0);
      }
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) {
        const uint32_t keep = kTileRows * g + i < live ? 0xFFFFFFFFu : 0u;  // no gradient, no result
#pragma unroll
        for (int k = 0; k < 4; ++k) d[i][k] &= keep;
#pragma unroll
        for (int k = 0; k < 4; ++k) gate[i][k] &= keep, up[i][k] &= keep;
        glu8_both<GELU>(gate[i], up[i], d[i], x[i], y[i]);
        __builtin_amdgcn_sched_barrier(0);  // a row's registers before the next one's
      }
      glu_tile<ROWS, STREAMING, PAIR>(to, s, x, row0, live, b, cb);
      glu_tile<ROWS, STREAMING, PAIR>(to, s, y, row0, live, b, cb + ncol);
    } else {
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) {
        const int r = kTileRows * g + i;
        glu_load<BACK, GELU, STREAMING>(in, row0 + min(r, live - 1), h0, r < live && h0 < to.W, x[i]);
      }
      glu_tile<ROWS, STREAMING, PAIR>(to, s, x, row0, live, b, cb);
    }
  }
}

uint32_t grid_of(int64_t want) { return static_cast<uint32_t>(want < (1 << 20) ? want : (1 << 20)); }

// Half the last-level cache's size: a longer pass finds little of its rows there again,
// and goes round the caches (32771 rows of 2048: 72 us, 80 through them; gradients of 8192
// rows: 48 us, 55 through them; of 2999 rows of 1000: 18.8 us, 16.9 through them).
constexpr int64_t kCacheBytes = 128 << 20;

template <typename F>
void with_flag(bool flag, F&& f) {
  if (flag)
    f(std::true_type{});
  else
    f(std::false_type{});
}

template <bool BACK, bool GELU>
hipError_t launch_glu_as(const int32_t* off, int32_t ne, const GluRows& in, uint8_t* q, uint8_t* q_scale, uint8_t* qt,
                         uint8_t* qt_scale, int64_t cap, hipStream_t st) {
  const int32_t W = BACK ? 2 * in.F : in.F;
  const bool pair = BACK && in.F % kQBlock == 0;
  const auto launch = [&](auto is_pair) {
    constexpr bool kPair = decltype(is_pair)::value;
    if (qt == nullptr) {
      const int32_t nch = ceil_div(kPair ? in.F : W, kGluChunk);
      const int64_t waves = cap * nch;
      hipLaunchKernelGGL((glu_rows_kernel<BACK, GELU, kPair>), dim3(grid_of((waves + kGluWaves - 1) / kGluWaves)), dim3(kGluThreads), 0, st,
                         off, ne, in, q, q_scale, cap, nch);
      return;
    }
    const GluOut to{q, q_scale, qt, qt_scale, W};
    const int32_t nblk = static_cast<int32_t>(cap / kQBlock) + ne, ncol = ceil_div(kPair ? in.F : W, kQBlock);
    const dim3 grid(grid_of(static_cast<int64_t>(nblk) * ncol));
    const int64_t bytes = cap * in.F * ((BACK ? 6 : 4) + (BACK ? 2 : 1) * (q != nullptr ? 2 : 1));
    with_flag(q != nullptr, [&](auto rows) {
      with_flag(bytes > kCacheBytes, [&](auto streaming) {
        hipLaunchKernelGGL((glu_cols_kernel<BACK, GELU, decltype(rows)::value, kPair, decltype(streaming)::value>), grid, dim3(kTileThreads), 0,
                           st, off, ne, in, to, cap, nblk, ncol);
      });
    });
  };
  if constexpr (BACK)
    with_flag(pair, launch);
  else
    launch(std::false_type{});
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
