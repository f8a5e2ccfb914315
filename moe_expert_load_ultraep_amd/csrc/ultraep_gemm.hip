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

// Order of the tiles.  Workgroups go to the eight XCDs in turn; each XCD takes
// one contiguous eighth of a walk that goes through eight row tiles by all
// column tiles at a time, so that the workgroups that share an L2 at one time
// read a near-square set of rows and weights.
struct Tile2 {
  int32_t m, n;
};

__device__ __forceinline__ Tile2 tile_order(int64_t t, int64_t tiles, int32_t mtile, int32_t ntile) {
  constexpr int kGroup = 8;
  const int64_t full = tiles & ~int64_t{7};
  if (t < full) t = (t & 7) * (full >> 3) + (t >> 3);
  const int64_t per = static_cast<int64_t>(kGroup) * ntile;
  const int32_t g = static_cast<int32_t>(t / per);
  const int32_t r = static_cast<int32_t>(t - g * per);
  const int32_t width = min(kGroup, mtile - g * kGroup);
  return Tile2{g * kGroup + r % width, r / width};
}

// ------------------------------------------------------------------------
// The 256 x 256 tile
// ------------------------------------------------------------------------
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(1))) int global_int;

constexpr int kBigTile = 256;        // rows of either operand
constexpr int kHalfBytes = 128 * 128;  // half of an operand's block of 128, in LDS

// One operand of a tile: row r of block b at base + min(r, last) * row_pitch +
// b * block_pitch, 128 bytes.
struct BigOperand {
  const uint8_t* base;
  int64_t block_pitch;
  uint32_t row_pitch;
  int32_t last;
};

// A wave's 128 rows of A are read as 16-row fragments i = 0..7, fragment row m
// being row 32 * (m / 4) + 4 * i + m % 4, so that a lane's accumulators
// (fragment rows 4 * (l / 16) + r) are 32 consecutive rows: whole lines when
// they are stored.  B's fragment j holds rows 16 * j + m.
//
// Half H of an operand's block is what the two waves along it read as
// fragments 4H..4H+3, 64 rows each: row s of the half is this row of the tile.
template <bool A, int H>
__device__ __forceinline__ int half_row(int s) {
  return A ? 128 * (s >> 6) + 32 * ((s >> 4) & 3) + 16 * H + (s & 15) : 128 * (s >> 6) + 64 * H + (s & 63);
}

// In LDS a row is eight 16-byte parts, part c at c ^ key(row).  64 banks are two
// rows wide: an even and an odd row share a key, and the eight pairs of the
// sixteen rows that are read together have different ones.
template <bool A>
__device__ __forceinline__ int part_key(int s) {
  return A ? ((s >> 1) & 1) | (((s >> 4) & 3) << 1) : (s >> 1) & 7;
}

// Byte offsets of the four 16-byte parts that this lane loads of half H.
template <bool A, int H>
__device__ __forceinline__ void load_offsets(const BigOperand& op, uint32_t (&off)[4]) {
  const int lane = lane_id(), wv = threadIdx.x >> 6;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int s = wv * 32 + u * 8 + (lane >> 3);
    off[u] = static_cast<uint32_t>(min(half_row<A, H>(s), op.last)) * op.row_pitch +
             static_cast<uint32_t>(((lane & 7) ^ part_key<A>(s)) * 16);
  }
}

// Half a block of an operand into LDS, asynchronously: four loads a wave, 1 KiB
// (eight rows) each.  At and behind `blocks` the resource is empty and zeros
// arrive, so the loop over blocks has no branches.
struct HalfLoad {
  __amdgpu_buffer_rsrc_t src;
  lds_u8* dst;
  const uint32_t (&off)[4];

  __device__ __forceinline__ HalfLoad(const BigOperand& op, int32_t b, int32_t blocks, const uint32_t (&o)[4], uint8_t* lds)
      : src(row_rsrc(op.base + min(b, blocks - 1) * op.block_pitch, b < blocks ? 0x7FFFFFFFu : 0u)),
        dst((lds_u8*)lds + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)) * 4096),
        off(o) {}

  __device__ __forceinline__ void issue(int u) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, dst + u * 1024, 16, static_cast<int>(off[u]), 0, 0, 0);
  }
};

__device__ __forceinline__ void load_half(const BigOperand& op, int32_t b, int32_t blocks, const uint32_t (&off)[4],
                                          uint8_t* lds) {
  const HalfLoad load(op, b, blocks, off, lds);
#pragma unroll
  for (int u = 0; u < 4; ++u) load.issue(u);
}

// Every wave's LDS reads are done and all but its last LOADS loads have
// arrived; then the workgroup meets.
template <int LOADS>
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((LOADS & 15) | (7 << 4) | ((LOADS >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// acc += A B of one 16 x 16 x 128 with byte BYTE of the scale words.  Written as
// volatile asm for two reasons: the accumulator is updated where it is (with
// the builtin the compiler picks another destination and moves whole
// accumulators about, 460 moves in 256 products), and products and LDS reads
// stay in the order of the source.  The s_nop covers a scale word or fragment
// that a vector instruction wrote just before.
template <int BYTE>
__device__ __forceinline__ void product(f32x4& acc, const i32x8& a, const i32x8& b, int xa, int xb) {
  if constexpr (BYTE == 0)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(xa), "v"(xb));
  else if constexpr (BYTE == 1)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(xa), "v"(xb));
  else if constexpr (BYTE == 2)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[1,1,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(xa), "v"(xb));
  else
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(xa), "v"(xb));
}

// Behind the products: their results are there before a vector instruction, a
// copy the compiler makes included, reads them (19 wait states).  It stands in
// the loop's own block, since copies start where the loop ends.
__device__ __forceinline__ void products_done() { asm volatile("s_nop 15\n\ts_nop 3"); }

// Fragment i of a half in LDS; at[h]: this lane's part h.
template <int STRIDE>
__device__ __forceinline__ i32x8 read_fragment(const uint8_t* lds, const int (&at)[2], int i) {
  return __builtin_shufflevector(*reinterpret_cast<const i32x4*>(lds + at[0] + i * STRIDE),
                                 *reinterpret_cast<const i32x4*>(lds + at[1] + i * STRIDE), 0, 1, 2, 3, 4, 5, 6, 7);
}

constexpr int kStrideA = 4 * 128, kStrideB = 16 * 128;  // bytes from a fragment's rows to the next one's

// A quarter of the wave's products: fragments a[4] by b[4], with the reads of
// the four fragments f of half `lds` and the loads of another half among them: a
// load's issue takes long enough for the matrix unit to run dry when several
// follow each other.
template <int I0, int J0, int BYTE, int STRIDE>
__device__ __forceinline__ void quadrant(const i32x8 (&a)[4], const i32x8 (&b)[4], int xa, const int (&xb)[8],
                                         f32x4 (&acc)[8][8], const uint8_t* lds, const int (&at)[2], i32x8 (&f)[4], const HalfLoad& load) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      product<BYTE>(acc[I0 + i][J0 + j], a[i], b[j], xa, xb[J0 + j]);
      if (j == 0) f[i] = read_fragment<STRIDE>(lds, at, i);
      if (j == 2) load.issue(i);
    }
}

// Scale bytes of four blocks: one word for the wave's 128 rows of A, one a
// fragment row of B.
struct ScaleWords {
  int a;
  int b[8];
};

struct ScaleSource {
  const uint8_t* a;  // the wave's row of weight scales
  const uint8_t* b;  // the tile's first row of row scales
  int32_t pitch;     // bytes a row
  int32_t last;      // B's last row
};

__device__ __forceinline__ void load_scales(const ScaleSource& s, int32_t block, ScaleWords& w) {
  const int row0 = ((threadIdx.x >> 6) & 1) * 128 + (lane_id() & 15);
  w.a = *reinterpret_cast<const global_int*>(reinterpret_cast<uintptr_t>(s.a) + block);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w.b[j] = *reinterpret_cast<const int*>(s.b + static_cast<uint32_t>(min(row0 + 16 * j, s.last)) * s.pitch + block);
}

// Waits for the words here, and not at their first use in the loop.
__device__ __forceinline__ void settle(ScaleWords& w) {
  asm volatile("" : "+v"(w.a));
#pragma unroll
  for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(w.b[j]));
}

// LDS and registers of the pipeline.  Halves are indexed [block parity][half].
struct Offsets {
  uint32_t a[2][4], b[2][4];
  int read_a[2], read_b[2];
};

// One block of 128, the U-th of four: the wave's 8 x 8 products of 16 x 16 x 128
// in four quadrants, odd blocks walking B's halves the other way round.  Every
// half is read once, in the quadrant before its first use, and the barrier
// behind that quadrant frees it for the block after next: its loads have seven
// quadrants (about 3600 cycles of products) to arrive, and 112 of the 128 KiB
// are in flight or waiting at any time.
template <int U>
__device__ __forceinline__ void big_step(const BigOperand& a, const BigOperand& b, const Offsets& o, int32_t k,
                                         int32_t blocks, uint8_t* alo, uint8_t* ahi, uint8_t* bx, uint8_t* by,
                                         uint8_t* next_alo, uint8_t* next_by, i32x8 (&fal)[4], i32x8 (&fah)[4],
                                         i32x8 (&fbx)[4], i32x8 (&fby)[4], const ScaleSource& ss, ScaleWords& sw,
                                         ScaleWords& sn, f32x4 (&acc)[8][8]) {
  constexpr int X = U & 1, Y = 1 - X;
  meet<16>();
  quadrant<0, 4 * X, U, kStrideB>(fal, fbx, sw.a, sw.b, acc, by, o.read_b, fby, HalfLoad(a, k + 2, blocks, o.a[0], alo));
  quadrant<0, 4 * Y, U, kStrideA>(fal, fby, sw.a, sw.b, acc, ahi, o.read_a, fah, HalfLoad(b, k + 2, blocks, o.b[X], bx));
  meet<16>();
  if (U == 2) load_scales(ss, min(k + 2, blocks - 1) & ~3, sn);
  quadrant<4, 4 * Y, U, kStrideA>(fah, fby, sw.a, sw.b, acc, next_alo, o.read_a, fal,
                                  HalfLoad(b, k + 2, blocks, o.b[Y], by));
  quadrant<4, 4 * X, U, kStrideB>(fah, fbx, sw.a, sw.b, acc, next_by, o.read_b, fby,
                                  HalfLoad(a, k + 2, blocks, o.a[1], ahi));
  if (U == 3) {
    sw = sn;
    products_done();
  }
}

// What the products of one segment share.
struct GemmArgs {
  const int32_t* off;
  int32_t ne;
  const uint8_t* q;
  const uint8_t* q_scale;
  int32_t K;
  const uint8_t* const* w;
  const uint8_t* const* w_scale;
  int32_t N;
  uint16_t* out;
  int64_t cap;
};

// Whether expert p's weights are there to be used.
__device__ __forceinline__ bool usable(const uint8_t* w, const uint8_t* ws) {
  return w != nullptr && ws != nullptr && (reinterpret_cast<uintptr_t>(w) & 15) == 0 &&
         (reinterpret_cast<uintptr_t>(ws) & 3) == 0;
}

// out[row][n]: A is the weights (a lane holds 32 consecutive n of a row), B the
// rows; one 256 x 256 tile a workgroup, four waves of 128 x 128.
__global__ __launch_bounds__(kMmThreads, 1) void expert_gemm_big_kernel(GemmArgs g, int32_t ntile) {
  __shared__ __align__(16) uint8_t a00[kHalfBytes], a01[kHalfBytes], a10[kHalfBytes], a11[kHalfBytes];
  __shared__ __align__(16) uint8_t b00[kHalfBytes], b01[kHalfBytes], b10[kHalfBytes], b11[kHalfBytes];
  const int32_t Kp = q_pitch(g.K), Ks = s_pitch(g.K), blocks = Kp / 128;
  const int lane = lane_id(), l16 = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), wi = wv >> 1, wj = wv & 1;
  const int32_t mtile = row_tiles(g.off, g.ne, g.cap, kBigTile);
  const int64_t tiles = static_cast<int64_t>(mtile) * ntile;
  if (blockIdx.x >= tiles) return;
  const Tile2 at = tile_order(blockIdx.x, tiles, mtile, ntile);
  const RowTile rt = find_row_tile(g.off, g.ne, g.cap, kBigTile, at.m);
  const uint8_t* wp = g.w[rt.p];
  const uint8_t* ws = g.w_scale[rt.p];
  if (!usable(wp, ws)) return;
  const int32_t n0 = at.n * kBigTile, rows = rt.rows, cols = min(g.N - n0, kBigTile);
  const BigOperand a{wp + static_cast<int64_t>(n0) * Kp, 128, static_cast<uint32_t>(Kp), cols - 1};
  const BigOperand b{g.q + rt.row0 * Kp, 128, static_cast<uint32_t>(Kp), rows - 1};
  const int32_t sblock = min(n0 / 128 + wi, ceil_div(g.N, 128) - 1);
  const ScaleSource ss{ws + static_cast<int64_t>(sblock) * Ks, g.q_scale + rt.row0 * Ks, Ks, rows - 1};
  Offsets o;
  load_offsets<true, 0>(a, o.a[0]);
  load_offsets<true, 1>(a, o.a[1]);
  load_offsets<false, 0>(b, o.b[0]);
  load_offsets<false, 1>(b, o.b[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int part = ((2 * kg + h) ^ (l16 >> 1)) * 16;
    o.read_a[h] = (wi * 64 + 16 * (l16 >> 2) + (l16 & 3)) * 128 + part;
    o.read_b[h] = (wj * 64 + l16) * 128 + part;
  }
  ScaleWords sw, sn;
  load_scales(ss, 0, sw);
  settle(sw);
  load_half(a, 0, blocks, o.a[0], a00);
  load_half(b, 0, blocks, o.b[0], b00);
  load_half(b, 0, blocks, o.b[1], b01);
  load_half(a, 0, blocks, o.a[1], a01);
  load_half(a, 1, blocks, o.a[0], a10);
  load_half(b, 1, blocks, o.b[1], b11);
  load_half(b, 1, blocks, o.b[0], b10);
  load_half(a, 1, blocks, o.a[1], a11);
  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x8 fal[4], fah[4], fb0[4], fb1[4];
  meet<24>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fal[i] = read_fragment<kStrideA>(a00, o.read_a, i);
    fb0[i] = read_fragment<kStrideB>(b00, o.read_b, i);
  }
  for (int32_t k = 0; k < blocks; k += 4) {
    big_step<0>(a, b, o, k, blocks, a00, a01, b00, b01, a10, b11, fal, fah, fb0, fb1, ss, sw, sn, acc);
    big_step<1>(a, b, o, k + 1, blocks, a10, a11, b11, b10, a00, b00, fal, fah, fb1, fb0, ss, sw, sn, acc);
    big_step<2>(a, b, o, k + 2, blocks, a00, a01, b00, b01, a10, b11, fal, fah, fb0, fb1, ss, sw, sn, acc);
    big_step<3>(a, b, o, k + 3, blocks, a10, a11, b11, b10, a00, b00, fal, fah, fb1, fb0, ss, sw, sn, acc);
  }
  const int c = wi * 128 + 32 * kg;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = wj * 128 + 16 * j + l16;
    if (r < rows) {
      u32x4* d = reinterpret_cast<u32x4*>(g.out + (rt.row0 + r) * g.N + n0 + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + 8 * i < cols)
          d[i] = u32x4{pack_bf16(acc[2 * i][j][0], acc[2 * i][j][1]), pack_bf16(acc[2 * i][j][2], acc[2 * i][j][3]),
                       pack_bf16(acc[2 * i + 1][j][0], acc[2 * i + 1][j][1]),
                       pack_bf16(acc[2 * i + 1][j][2], acc[2 * i + 1][j][3])};
    }
  }
  meet<0>();  // no load outlives the workgroup's LDS
}

// ------------------------------------------------------------------------
// The weight gradients' 256 x 256 tile
// ------------------------------------------------------------------------
typedef int i32x2v __attribute__((ext_vector_type(2)));

// acc += A B of one 16 x 16 x 32 in bf16, in place (see product); nothing that
// it reads is written by the two vector instructions before it.
__device__ __forceinline__ void product_wide(f32x4& acc, const i32x4& a, const i32x4& b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// Values 4 * HALF..4 * HALF + 3 of eight e4m3 bytes, times their scale, as bf16.
template <int HALF>
__device__ __forceinline__ void widen_half(i32x4& y, const i32x2v& raw, float scale) {
  int lo, hi;
  asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2" : "=v"(lo) : "v"(raw[HALF]), "v"(scale));
  asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2 op_sel:[1,0,0]" : "=v"(hi) : "v"(raw[HALF]), "v"(scale));
  y[2 * HALF] = lo;
  y[2 * HALF + 1] = hi;
}

// A block of 128 is 32 steps n = 8 g + i: A's fragment i by B's eight, over the
// g-th eight of each lane's 32 values.  During step n the fragment of A for step
// n + 1 and fragment i of B for the next g are widened, an instruction or two
// behind each product, from bytes read from LDS four steps before.
struct WideState {
  i32x4 a[2];     // A's fragment of this step and of the next
  i32x4 b[2][8];  // B's of this g and of the next
  i32x2v raw_a[4], raw_b[4];
  float sa[8], sb[8];  // scales of the block being widened
  int na[8], nb[8];    // scale bytes of the next one
};

struct WideTile {
  BigOperand a, b;
  const uint8_t *scale_a, *scale_b;  // scale bytes of the tile's rows, block 0
  int32_t pitch_a, pitch_b;          // scale bytes a block
  int32_t row_a, row_b;              // this lane's row of fragment 0
  uint32_t off_a[2][4], off_b[2][4];
  int at_a[4], at_b[4];              // LDS offset of this lane's eight bytes g, in a half
};

// Eight bytes of fragment i; the fragments' rows lie in two halves.
template <int STRIDE>
__device__ __forceinline__ i32x2v read_raw(const uint8_t* lo, const uint8_t* hi, int at, int i) {
  return *reinterpret_cast<const i32x2v*>((i < 4 ? lo : hi) + at + (i & 3) * STRIDE);
}

__device__ __forceinline__ int scale_byte(const uint8_t* s, int32_t row, int32_t last) { return s[min(row, last)]; }

// Block k in LDS buffers [half] of its parity; n_*: the other parity's, where
// block k + 1 is or arrives.  B's halves are read up to step 19 and A's up to
// step 26; behind the barriers there the loads of block k + 2 go into them, 32
// steps (about 4100 cycles of products) before they are read.
__device__ __forceinline__ void wide_block(const WideTile& t, WideState& w, int32_t k, int32_t blocks, uint8_t* al,
                                           uint8_t* ah, uint8_t* bl, uint8_t* bh, uint8_t* nal, uint8_t* nah, uint8_t* nbl,
                                           uint8_t* nbh, f32x4 (&acc)[8][8]) {
  const HalfLoad load_al(t.a, k + 2, blocks, t.off_a[0], al), load_ah(t.a, k + 2, blocks, t.off_a[1], ah);
  const HalfLoad load_bl(t.b, k + 2, blocks, t.off_b[0], bl), load_bh(t.b, k + 2, blocks, t.off_b[1], bh);
  const int64_t next = min(k + 1, blocks - 1);
  const uint8_t* sa = t.scale_a + next * t.pitch_a;
  const uint8_t* sb = t.scale_b + next * t.pitch_b;
#pragma unroll
  for (int n = 0; n < 32; ++n) {
    const int g = n >> 3, i = n & 7;
    if (n == 20 || n == 27) meet<8>();
    if (n == 24) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w.sb[j] = scale_of(w.nb[j]);
    }
    if (n == 31) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w.sa[j] = scale_of(w.na[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      product_wide(acc[i][j], w.a[n & 1], w.b[g & 1][j]);
      if (j == 0) widen_half<0>(w.a[(n + 1) & 1], w.raw_a[(n + 1) & 3], w.sa[(n + 1) & 7]);
      if (j == 1) widen_half<1>(w.a[(n + 1) & 1], w.raw_a[(n + 1) & 3], w.sa[(n + 1) & 7]);
      if (j == 2) widen_half<0>(w.b[(g + 1) & 1][i], w.raw_b[n & 3], w.sb[i]);
      if (j == 3) widen_half<1>(w.b[(g + 1) & 1][i], w.raw_b[n & 3], w.sb[i]);
      if (j == 4) {
        const int m = n + 5;
        w.raw_a[m & 3] = m < 32 ? read_raw<kStrideA>(al, ah, t.at_a[(m >> 3) & 3], m & 7)
                                : read_raw<kStrideA>(nal, nah, t.at_a[0], m & 7);
      }
      if (j == 5) {
        const int m = n + 4;  // widened at step m for g + 1
        w.raw_b[m & 3] = m < 24 ? read_raw<kStrideB>(bl, bh, t.at_b[((m >> 3) + 1) & 3], m & 7)
                                : read_raw<kStrideB>(nbl, nbh, t.at_b[((m >> 3) + 1) & 3], m & 7);
      }
      if (j == 6 || j == 7) {
        if (n >= 2 && n < 10) {
          if (j == 6) w.na[n - 2] = scale_byte(sa, t.row_a + 4 * (n - 2), t.a.last);
          if (j == 7) w.nb[n - 2] = scale_byte(sb, t.row_b + 16 * (n - 2), t.b.last);
        }
        if (n >= 20 && n < 24) (j == 6 ? load_bl : load_bh).issue(n - 20);
        if (n >= 27 && n < 31) (j == 6 ? load_al : load_ah).issue(n - 27);
      }
    }
  }
}

// The expert with the rank-th most rows (ties: lower expert first) of at most
// 64; of more, the rank-th expert.
__device__ __forceinline__ int32_t expert_of_rank(const int32_t* off, int32_t ne, int64_t cap, int32_t rank) {
  if (ne > 64) return rank;
  const int32_t l = lane_id(), p = min(l, ne - 1);
  const int32_t rows = l < ne ? group_row(off, p + 1, cap) - group_row(off, p, cap) : -1;
  int32_t before = 0;
  for (int32_t q = 0; q < ne; ++q) {
    const int32_t other = static_cast<int32_t>(readlane(static_cast<uint32_t>(rows), q));
    before += other > rows || (other == rows && q < l) ? 1 : 0;
  }
  return __builtin_amdgcn_readfirstlane(lowest_lane(ballot(l < ne && before == rank)));
}

// grads[p][n][k]: A is x (a lane holds 32 consecutive k of a row n), B is dy.
__global__ __launch_bounds__(kMmThreads, 1) void expert_wgrad_big_kernel(
    const int32_t* off, int32_t ne, const uint8_t* dyt, const uint8_t* dyt_scale, int32_t N, const uint8_t* xt,
    const uint8_t* xt_scale, int32_t K, int64_t cap, float* const* grads, bool accumulate, int32_t ntile,
    int32_t ktile) {
  __shared__ __align__(16) uint8_t a00[kHalfBytes], a01[kHalfBytes], a10[kHalfBytes], a11[kHalfBytes];
  __shared__ __align__(16) uint8_t b00[kHalfBytes], b01[kHalfBytes], b10[kHalfBytes], b11[kHalfBytes];
  const int lane = lane_id(), l16 = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), wi = wv >> 1, wj = wv & 1;
  // every expert's tiles are dealt to all XCDs (experts differ in rows, so an
  // XCD must not get whole ones), the expert with the most rows first
  const int32_t per = ntile * ktile, turn = static_cast<int32_t>(blockIdx.x) / per;
  const Tile2 at = tile_order(blockIdx.x - turn * per, per, ntile, ktile);
  const int32_t p = expert_of_rank(off, ne, cap, turn), tn = at.m, tk = at.n;
  float* out = grads[p];
  if (out == nullptr) return;
  const int32_t o0 = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
  const int32_t blocks = max(ceil_div(o1 - o0, kQBlock), 0);
  if (blocks == 0 && accumulate) return;
  const int64_t first = o0 / kQBlock + p;
  const int32_t n0 = tn * kBigTile, k0 = tk * kBigTile, rows = min(N - n0, kBigTile), cols = min(K - k0, kBigTile);
  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (blocks > 0) {
    WideTile t;
    t.a = BigOperand{xt + (first * K + k0) * kQBlock, static_cast<int64_t>(K) * kQBlock, 128u, cols - 1};
    t.b = BigOperand{dyt + (first * N + n0) * kQBlock, static_cast<int64_t>(N) * kQBlock, 128u, rows - 1};
    t.scale_a = xt_scale + first * K + k0;
    t.scale_b = dyt_scale + first * N + n0;
    t.pitch_a = K;
    t.pitch_b = N;
    t.row_a = wi * 128 + 32 * (l16 >> 2) + (l16 & 3);
    t.row_b = wj * 128 + l16;
    load_offsets<true, 0>(t.a, t.off_a[0]);
    load_offsets<true, 1>(t.a, t.off_a[1]);
    load_offsets<false, 0>(t.b, t.off_b[0]);
    load_offsets<false, 1>(t.b, t.off_b[1]);
    // odd lanes of sixteen take the two eights of a part the other way round, so
    // that 32 lanes reading eight bytes meet all banks once
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int part = ((2 * kg + (g >> 1)) ^ (l16 >> 1)) * 16 + ((g ^ kg) & 1) * 8;
      t.at_a[g] = (wi * 64 + 16 * (l16 >> 2) + (l16 & 3)) * 128 + part;
      t.at_b[g] = (wj * 64 + l16) * 128 + part;
    }
    WideState w;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w.sa[j] = scale_of(scale_byte(t.scale_a, t.row_a + 4 * j, t.a.last));
      w.sb[j] = scale_of(scale_byte(t.scale_b, t.row_b + 16 * j, t.b.last));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(w.sa[j]), "+v"(w.sb[j]));
    load_half(t.b, 0, blocks, t.off_b[0], b00);
    load_half(t.b, 0, blocks, t.off_b[1], b01);
    load_half(t.a, 0, blocks, t.off_a[0], a00);
    load_half(t.a, 0, blocks, t.off_a[1], a01);
    load_half(t.b, 1, blocks, t.off_b[0], b10);
    load_half(t.b, 1, blocks, t.off_b[1], b11);
    load_half(t.a, 1, blocks, t.off_a[0], a10);
    load_half(t.a, 1, blocks, t.off_a[1], a11);
    meet<16>();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const i32x2v raw = read_raw<kStrideB>(b00, b01, t.at_b[0], j);
      widen_half<0>(w.b[0][j], raw, w.sb[j]);
      widen_half<1>(w.b[0][j], raw, w.sb[j]);
    }
    const i32x2v raw = read_raw<kStrideA>(a00, a01, t.at_a[0], 0);
    widen_half<0>(w.a[0], raw, w.sa[0]);
    widen_half<1>(w.a[0], raw, w.sa[0]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      w.raw_a[(m + 1) & 3] = read_raw<kStrideA>(a00, a01, t.at_a[0], m + 1);
      w.raw_b[m] = read_raw<kStrideB>(b00, b01, t.at_b[1], m);
    }
    asm volatile("s_nop 1");
    for (int32_t k = 0; k < blocks; k += 2) {
      wide_block(t, w, k, blocks, a00, a01, b00, b01, a10, a11, b10, b11, acc);
      wide_block(t, w, k + 1, blocks, a10, a11, b10, b11, a00, a01, b00, b01, acc);
      products_done();
    }
  }
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const int c = wi * 128 + 32 * kg;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = wj * 128 + 16 * j + l16;
    if (r >= rows) continue;
    float* d = out + static_cast<int64_t>(n0 + r) * K + k0 + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + 4 * i >= cols) continue;
      f32x4 y = acc[i][j];
      if (vec) {
        if (accumulate) y += *reinterpret_cast<const f32x4*>(d + 4 * i);
        *reinterpret_cast<f32x4*>(d + 4 * i) = y;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[4 * i + e] = accumulate ? d[4 * i + e] + y[e] : y[e];
      }
    }
  }
  meet<0>();  // no load outlives the workgroup's LDS
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
  if (cap / ne >= 64) {
    const int32_t ntile = ceil_div(N, kBigTile), mtile = static_cast<int32_t>(cap / kBigTile) + ne;
    const GemmArgs g{off, ne, q, q_scale, K, w, w_scale, N, out, cap};
    hipLaunchKernelGGL(expert_gemm_big_kernel, dim3(static_cast<uint32_t>(static_cast<int64_t>(mtile) * ntile)),
                       dim3(kMmThreads), 0, st, g, ntile);
    return hipGetLastError();
  }
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
  if (true) {
    const int32_t ntile = ceil_div(N, kBigTile), ktile = ceil_div(K, kBigTile);
    hipLaunchKernelGGL(expert_wgrad_big_kernel, dim3(static_cast<uint32_t>(ne * ntile * ktile)), dim3(kMmThreads), 0, st,
                       off, ne, dyt, dyt_scale, N, xt, xt_scale, K, cap, grads, accumulate, ntile, ktile);
    return hipGetLastError();
  }
  const int32_t ntile = ceil_div(N, kMmTile), ktile = ceil_div(K, kMmTile);
  const int64_t tiles = static_cast<int64_t>(ne) * ntile * ktile;
  hipLaunchKernelGGL(expert_wgrad_kernel, dim3(mm_grid(tiles)), dim3(kMmThreads), 0, st, off, ne, dyt, dyt_scale, N, xt,
                     xt_scale, K, cap, grads, accumulate, tiles, ntile, ktile);
  return hipGetLastError();
}

}  // namespace ultraep
