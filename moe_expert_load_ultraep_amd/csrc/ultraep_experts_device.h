// Device helpers of the experts' kernels: the segment's groups and the
// 8-bit block format (include/ultraep_experts.h).  Internal.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_device.h"

namespace ultraep {
namespace {

constexpr int kQBlock = 128;  // values per scale

__host__ __device__ inline int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }
// Row pitch of the rows and weights forms, and of their scales.
__host__ __device__ inline int32_t q_pitch(int32_t H) { return ceil_div(H, kQBlock) * kQBlock; }
__host__ __device__ inline int32_t s_pitch(int32_t H) { return ceil_div(ceil_div(H, kQBlock), 4) * 4; }

// First row of the range's expert p, counted from the range's first row and
// never beyond the rows that are there.
__device__ __forceinline__ int32_t group_row(const int32_t* off, int32_t p, int64_t cap) {
  const int64_t o = static_cast<int64_t>(off[p]) - off[0];
  return static_cast<int32_t>(max(min(o, cap), int64_t{0}));
}

// Tiles of `unit` rows: expert p's start at first(p) = row(p) / unit + p, so
// first(p + 1) - first(p) >= ceil(rows of p / unit) without any prefix sum
// (at most one tile an expert stays empty).  The expert of tile t is the last
// p with first(p) <= t; every wave finds it by itself, 64 experts a step.
// Every lane must be active; the result is wave-uniform.
__device__ __forceinline__ int32_t find_group(const int32_t* off, int32_t ne, int64_t cap, int32_t unit,
                                              int32_t t) {
  int32_t n = 0;
  for (int32_t p0 = 0; p0 < ne; p0 += 64) {
    const int32_t p = p0 + lane_id();
    const bool before = p < ne && group_row(off, min(p, ne - 1), cap) / unit + p <= t;
    const int32_t got = static_cast<int32_t>(__builtin_popcountll(ballot(before)));
    n += got;
    if (got < 64) break;
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// The row tiles of a segment: each expert's rows in tiles of `unit`, no tile
// without rows.  The counts are added up by a wave scan, 64 experts at a time;
// every wave finds its tile by itself.  Every lane must be active; results are
// wave-uniform.
__device__ __forceinline__ int32_t tiles_upto(const int32_t* off, int32_t ne, int64_t cap, int32_t unit, int32_t p0) {
  const int32_t p = p0 + lane_id();
  const int32_t rows = p < ne ? group_row(off, p + 1, cap) - group_row(off, p, cap) : 0;
  return wave_inclusive_scan((max(rows, 0) + unit - 1) / unit);
}

__device__ __forceinline__ int32_t row_tiles(const int32_t* off, int32_t ne, int64_t cap, int32_t unit) {
  int32_t total = 0;
  for (int32_t p0 = 0; p0 < ne; p0 += 64)
    total += static_cast<int32_t>(readlane(static_cast<uint32_t>(tiles_upto(off, ne, cap, unit, p0)), 63));
  return total;
}

struct RowTile {
  int32_t p;     // expert
  int64_t row0;  // first row, of the segment
  int32_t rows;  // 1..unit
};

// Row tile m < row_tiles(...).
__device__ __forceinline__ RowTile find_row_tile(const int32_t* off, int32_t ne, int64_t cap, int32_t unit, int32_t m) {
  int32_t before = 0;
  for (int32_t p0 = 0;; p0 += 64) {
    const int32_t upto = tiles_upto(off, ne, cap, unit, p0);
    const int32_t all = static_cast<int32_t>(readlane(static_cast<uint32_t>(upto), 63));
    if (m - before >= all && p0 + 64 < ne) {
      before += all;
      continue;
    }
    const int32_t l = min(static_cast<int32_t>(__builtin_popcountll(ballot(upto <= m - before))), 63);
    const int32_t p = p0 + l;
    const int32_t first = l > 0 ? static_cast<int32_t>(readlane(static_cast<uint32_t>(upto), max(l - 1, 0))) : 0;
    const int32_t o0 = __builtin_amdgcn_readfirstlane(group_row(off, p, cap));
    const int32_t o1 = __builtin_amdgcn_readfirstlane(group_row(off, p + 1, cap));
    const int64_t row0 = o0 + static_cast<int64_t>(m - before - first) * unit;
    return RowTile{p, row0, static_cast<int32_t>(min(o1 - row0, static_cast<int64_t>(unit)))};
  }
}

// Exponent of a block whose largest finite magnitude has these bf16 bits: the
// smallest e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(8 + e), 0 for a block
// without a finite value other than zero.
__device__ __forceinline__ int32_t block_exponent(uint32_t amax) {
  const int32_t e = static_cast<int32_t>(amax >> 7) - 135 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
  return amax == 0 ? 0 : max(e, -126);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float power_of_two(int32_t e) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(127 + e) << 23);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Magnitudes order as their bits do.  A block's largest is taken over all of
// them, two at a time, and once more without the infinities and NaN where the
// first answer is one (kNotFinite and above).
constexpr uint32_t kNotFinite = 0x7F80;

__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <bool FINITE>
__device__ __forceinline__ uint32_t magnitudes(uint32_t v) {
  const uint32_t m = v & 0x7FFF7FFFu;
  if (!FINITE) return m;
  const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
  return (lo < kNotFinite ? lo : 0u) | (hi < kNotFinite ? hi << 16 : 0u);
}

// Largest magnitude of eight bf16, as bf16 bits.
template <bool FINITE>
__device__ __forceinline__ uint32_t amax_of(const u32x4& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = pair_max(m, magnitudes<FINITE>(x[i]));
  return max(m & 0xFFFFu, m >> 16);
}

// Largest of 16 lanes (one aligned row), in every lane.
__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
  x = max(x, dpp<0xB1>(x));
  x = max(x, dpp<0x4E>(x));
  x = max(x, dpp<0x141>(x));
  return max(x, dpp<0x140>(x));
}

// Largest finite magnitude of the 16 lanes' values, as bf16 bits, in every lane.
__device__ __forceinline__ uint32_t row16_amax(const u32x4& x) {
  const uint32_t m = row16_max(amax_of<false>(x));
  if (__builtin_expect(ballot(m >= kNotFinite) != 0, 0)) return row16_max(amax_of<true>(x));
  return m;
}

// Two pairs of bf16 over a power of two, rounded to nearest even e4m3: the
// conversion scales exactly (subnormals included), infinities and NaN give NaN
// and nothing else is above 448.
__device__ __forceinline__ uint32_t to_e4m3(uint32_t pair0, uint32_t pair1, float scale) {
  i16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, pair0), scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, pair1), scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ u32x2 to_e4m3(const u32x4& x, float scale) {
  return u32x2{to_e4m3(x[0], x[1], scale), to_e4m3(x[2], x[3], scale)};
}

// The same from fp32 values: magnitudes as fp32 bits.
constexpr uint32_t kNotFiniteF32 = 0x7F800000;

__device__ __forceinline__ uint32_t finite_magnitude(float v) {
  const uint32_t m = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  return m < kNotFiniteF32 ? m : 0u;
}

__device__ __forceinline__ int32_t block_exponent_f32(uint32_t amax) {
  const int32_t e = static_cast<int32_t>(amax >> 23) - 135 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 0 : max(e, -126);
}

// Largest magnitude of N values but for NaN, as fp32 bits; infinite
// ones are left out only where FINITE.
template <bool FINITE, int N>
__device__ __forceinline__ uint32_t amax_of(const float (&x)[N]) {
  if (!FINITE) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
    return __builtin_bit_cast(uint32_t, m);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, finite_magnitude(x[i]));
  return m;
}

// Largest finite magnitude of the 16 lanes' values, as fp32 bits, in every lane.
__device__ __forceinline__ uint32_t row16_amax(const float (&x)[8]) {
  const uint32_t m = row16_max(amax_of<false>(x));
  if (__builtin_expect(ballot(m >= kNotFiniteF32) != 0, 0)) return row16_max(amax_of<true>(x));
  return m;
}

__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d, float scale) {
  i16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ u32x2 to_e4m3(const float (&x)[8], float scale) {
  return u32x2{to_e4m3(x[0], x[1], x[2], x[3], scale), to_e4m3(x[4], x[5], x[6], x[7], scale)};
}

// The scale bytes of a wave's four 16-lane blocks, one word.
__device__ __forceinline__ uint32_t four_scales(int32_t e) {
  uint32_t s = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) s |= (readlane(static_cast<uint32_t>(e), 16 * b) + 127u) << (8 * b);
  return s;
}

}  // namespace
}  // namespace ultraep
