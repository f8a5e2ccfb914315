// gfx950 kernels of the experts' 8-bit products (include/ultraep_experts.h):
// rows times weights for every physical expert of a segment, and the weight
// gradients.  Both are sums over blocks of 128,
//   C[i][j] = sum_b sum_{r < 128} (2^(sa[i][b] - 127) * A[i][b][r]) * (2^(sb[j][b] - 127) * B[j][b][r]),
// and both widen the bytes, scale included, to bf16 in the one instruction that
// does it, which is exact, and multiply with V_MFMA_F32_16X16X32_BF16, whose
// products and sums are fp32.
//
// The matrix instructions that take the bytes themselves are twice as fast, but
// do not keep fp32 sums.  Measured on the card, V_MFMA_SCALE_F32_16X16X128_F8F6F4
// and V_MFMA_F32_16X16X32_FP8_FP8 alike: of the eight products that a lane adds
// together, every one is cut (towards zero) at 2^-13 of the largest one's power
// of two, so where large products cancel, the others beside them are lost.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ultraep_experts_device.h"
#include "ultraep_internal.h"

namespace ultraep {
namespace {


constexpr int kMmThreads = 256;

__device__ __forceinline__ float scale_of(int byte) { return __builtin_bit_cast(float, static_cast<uint32_t>(byte) << 23); }

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
constexpr int kComputeUnits = 256;
constexpr int kHalfBytes = 128 * 128;  // half of an operand's block of 128, in LDS

// Workgroup b's share of `tiles` tiles: tile t's rows skip..skip + rows - 1.  A last
// round that fills at most half of the CUs has two workgroups for each of its
// tiles, if they may be halved: tiles + kComputeUnits / 2 workgroups suffice, and
// those that have none get a t of `tiles` and more.
struct TileShare {
  int64_t t;
  int32_t skip, rows;
};

__device__ __forceinline__ TileShare share_tile(int64_t b, int64_t tiles, bool halves) {
  const int64_t left = tiles % kComputeUnits, whole = halves && left <= kComputeUnits / 2 ? tiles - left : tiles;
  if (b < whole) return TileShare{b, 0, kBigTile};
  return TileShare{whole + ((b - whole) >> 1), (b - whole) & 1 ? 128 : 0, 128};
}

// One operand of a tile: row r of block b at base + min(r, last) * row_pitch +
// b * block_pitch, 128 bytes.
struct BigOperand {
  const uint8_t* base;
  int64_t block_pitch;
  uint32_t row_pitch;
  int32_t last;
};

// A wave reads its rows as 16-row fragments, and a lane's four accumulators are
// rows 4 * (l / 16).. of A's.  So that four lanes hold 64 consecutive bytes of
// an output row, the fragments of A are laid two into 32 rows where the output is
// bf16 (PAIRS: fragment i, row m is row 32 * (i / 2) + 8 * (m / 4) + 4 * (i % 2) +
// m % 4 of the wave's 128: eight values a lane, four lanes side by side), and one
// into 16 where it is fp32.
//
// Half H of an operand's block is what the two waves along it read as fragments
// 4H..4H+3, 64 rows each: row s of the half is this row of the tile.
template <bool PAIRS, int H>
__device__ __forceinline__ int half_row(int s) {
  return PAIRS ? 128 * (s >> 6) + 64 * H + (s & 63) : 128 * H + s;
}

// LDS bytes from a half's fragment 0 to fragment i, and a lane's row of fragment 0.
template <bool PAIRS>
__device__ __forceinline__ constexpr int fragment_at(int i) {
  return PAIRS ? (i >> 1) * 4096 + (i & 1) * 512 : i * 2048;
}

template <bool PAIRS>
__device__ __forceinline__ int fragment_row(int m) {
  return PAIRS ? 8 * (m >> 2) + (m & 3) : m;
}

// Row m of fragment j of wave wj along an operand without pairs.
__device__ __forceinline__ int b_row(int wj, int j, int m) { return 128 * (j >> 2) + 64 * wj + 16 * (j & 3) + m; }

// In LDS a row is eight 16-byte parts, part c at c ^ key(row).  64 banks are two
// rows wide: an even and an odd row share a key, and the eight pairs of the
// sixteen rows that are read together have different ones.  Counted conflicts: 2 %
// of the cycles LDS is read in the rows products, 0.5 % in the weight gradients.
template <bool PAIRS>
__device__ __forceinline__ int part_key(int s) {
  return PAIRS ? ((s >> 1) & 1) | (((s >> 3) & 3) << 1) : (s >> 1) & 7;
}

// Byte offsets of the four 16-byte parts that this lane loads of half H.
template <bool PAIRS, int H>
__device__ __forceinline__ void load_offsets(const BigOperand& op, uint32_t (&off)[4]) {
  const int lane = lane_id(), wv = threadIdx.x >> 6;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int s = wv * 32 + u * 8 + (lane >> 3);
    off[u] = static_cast<uint32_t>(min(half_row<PAIRS, H>(s), op.last)) * op.row_pitch +
             static_cast<uint32_t>(((lane & 7) ^ part_key<PAIRS>(s)) * 16);
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

// Behind the products: their results are there before a vector instruction, a
// copy the compiler makes included, reads them (19 wait states).  It stands in
// the loop's own block, since copies start where the loop ends.
__device__ __forceinline__ void products_done() { asm volatile("s_nop 15\n\ts_nop 3"); }

typedef int i32x2v __attribute__((ext_vector_type(2)));

// acc += A B of one 16 x 16 x 32 in bf16.  Written as volatile asm for two
// reasons: the accumulator is updated where it is (with the builtin the compiler
// picks another destination and moves whole accumulators about, 460 moves in 256
// products), and products and LDS reads stay in the order of the source.  Nothing
// that it reads may be written in the two wait states before it; the source leaves
// them, and tests/test_wait_states.py counts them in what the compiler made of it (an
// s_nop 1 before every product, which would settle it here, costs 13 %: 1450 us
// instead of 1256 for the 32768 rows below).
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

// A block of 128 is 32 steps n = 8 g + i: A's fragment i by B's J (eight, or the
// four of its first half), over the g-th eight of each lane's 32 values.  During
// step n the fragment of A for step n + 1 and fragment i of B for the next g are
// widened, an instruction or two behind each product, from bytes read from LDS
// four steps before.
struct WideState {
  i32x4 a[2];     // A's fragment of this step and of the next
  i32x4 b[2][8];  // B's of this g and of the next
  i32x2v raw_a[4], raw_b[4];
  float sa[8], sb[8];  // scales of the block being widened
  int na[8], nb[8];    // scale bytes of the next one
};

// ROWS (the rows products): A's fragments lie in PAIRS, its scale is one byte a
// block for the wave's 128 rows, B's `scale_row` bytes a row; else (the weight
// gradients) both operands' scales are a byte a row.
struct WideTile {
  BigOperand a, b;
  const uint8_t *scale_a, *scale_b;  // scale bytes of the tile's rows (ROWS: A's of the wave's rows), block 0
  int32_t pitch_a, pitch_b;          // scale bytes from a block to the next
  int32_t scale_row;                 // ROWS: scale bytes from a row of B to the next
  int32_t wi, wj, l16;
  uint32_t off_a[2][4], off_b[2][4];
  int at_a[4], at_b[4];              // LDS offset of this lane's eight bytes g, in a half
};

// LDS offsets of the eights.  Odd lanes of sixteen take the two eights of a part
// the other way round, so that 32 lanes reading eight bytes meet all banks once.
template <bool PAIRS>
__device__ __forceinline__ void read_offsets(WideTile& t) {
  const int kg = lane_id() >> 4;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int part = ((2 * kg + (g >> 1)) ^ (t.l16 >> 1)) * 16 + ((g ^ kg) & 1) * 8;
    t.at_a[g] = (t.wi * 64 + fragment_row<PAIRS>(t.l16)) * 128 + part;
    t.at_b[g] = (t.wj * 64 + t.l16) * 128 + part;
  }
}

// Eight bytes of fragment i; the fragments' rows lie in two halves.
template <bool PAIRS>
__device__ __forceinline__ i32x2v read_raw(const uint8_t* lo, const uint8_t* hi, int at, int i) {
  return *reinterpret_cast<const i32x2v*>((i < 4 ? lo : hi) + at + fragment_at<PAIRS>(i & 3));
}

// Scale byte of this lane's row of fragment j, s the block's bytes (a resource, so
// that a row costs one register and not an address).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scales_of(const uint8_t* s) { return row_rsrc(s, 0x7FFFFFFFu); }
template <bool ROWS>
__device__ __forceinline__ int scale_a(const WideTile& t, __amdgpu_buffer_rsrc_t s, int j) {
  return __builtin_amdgcn_raw_buffer_load_b8(s, ROWS ? 0 : min(b_row(t.wi, j, t.l16), t.a.last), 0, 0);
}
template <bool ROWS>
__device__ __forceinline__ int scale_b(const WideTile& t, __amdgpu_buffer_rsrc_t s, int j) {
  const int32_t row = min(b_row(t.wj, j, t.l16), t.b.last);
  return __builtin_amdgcn_raw_buffer_load_b8(s, ROWS ? row * t.scale_row : row, 0, 0);
}

// Block k in LDS buffers [half] of its parity; n_*: the other parity's, where
// block k + 1 is or arrives.  B's halves are read up to step 19 and A's up to
// step 26; behind the barriers there the loads of block k + 2 go into them, 32
// steps (about 4100 cycles of products with J = 8) before they are read.
template <int J, bool ROWS>
__device__ __forceinline__ void wide_block(const WideTile& t, WideState& w, int32_t k, int32_t blocks, uint8_t* al,
                                           uint8_t* ah, uint8_t* bl, uint8_t* bh, uint8_t* nal, uint8_t* nah, uint8_t* nbl,
                                           uint8_t* nbh, f32x4 (&acc)[8][8]) {
  constexpr int kScalesA = ROWS ? 1 : 8;
  const HalfLoad load_al(t.a, k + 2, blocks, t.off_a[0], al), load_ah(t.a, k + 2, blocks, t.off_a[1], ah);
  const HalfLoad load_bl(t.b, k + 2, blocks, t.off_b[0], bl), load_bh(t.b, k + 2, blocks, t.off_b[1], bh);
  const int64_t next = min(k + 1, blocks - 1);
  const __amdgpu_buffer_rsrc_t sa = scales_of(t.scale_a + next * t.pitch_a), sb = scales_of(t.scale_b + next * t.pitch_b);
#pragma unroll
  for (int n = 0; n < 32; ++n) {
    const int g = n >> 3, i = n & 7;
    if (n == 20) meet<8>();
    if (n == 27) meet<J>();
    if (n == 24) {
#pragma unroll
      for (int j = 0; j < J; ++j) w.sb[j] = scale_of(w.nb[j]);
    }
    if (n == 31) {
#pragma unroll
      for (int j = 0; j < kScalesA; ++j) w.sa[j] = scale_of(w.na[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      product_wide(acc[i][j], w.a[n & 1], w.b[g & 1][j]);
      if (j == 0) widen_half<0>(w.a[(n + 1) & 1], w.raw_a[(n + 1) & 3], w.sa[(n + 1) & (kScalesA - 1)]);
      if (j == 1) widen_half<1>(w.a[(n + 1) & 1], w.raw_a[(n + 1) & 3], w.sa[(n + 1) & (kScalesA - 1)]);
      if (j == 2 && i < J) widen_half<0>(w.b[(g + 1) & 1][i], w.raw_b[n & 3], w.sb[i]);
      if (j == 3 && i < J) widen_half<1>(w.b[(g + 1) & 1][i], w.raw_b[n & 3], w.sb[i]);
      if (j == J / 2) {  // behind the last use of the bytes it replaces
        const int m = n + 5;
        w.raw_a[m & 3] = m < 32 ? read_raw<ROWS>(al, ah, t.at_a[(m >> 3) & 3], m & 7)
                                : read_raw<ROWS>(nal, nah, t.at_a[0], m & 7);
      }
      if (j == J / 2 + 1 && ((n + 4) & 7) < J) {
        const int m = n + 4;  // widened at step m for g + 1
        w.raw_b[m & 3] = m < 24 ? read_raw<false>(bl, bh, t.at_b[((m >> 3) + 1) & 3], m & 7)
                                : read_raw<false>(nbl, nbh, t.at_b[((m >> 3) + 1) & 3], m & 7);
      }
      if (j == J - 2) {
        if (n >= 2 && n < 2 + kScalesA) w.na[n - 2] = scale_a<ROWS>(t, sa, n - 2);
        if (n >= 20 && n < 24) load_bl.issue(n - 20);
        if (n >= 27 && n < 31) load_al.issue(n - 27);
      }
      if (j == J - 1) {
        if (n >= 2 && n < 2 + J) w.nb[n - 2] = scale_b<ROWS>(t, sb, n - 2);
        if (J == 8 && n >= 20 && n < 24) load_bh.issue(n - 20);
        if (n >= 27 && n < 31) load_ah.issue(n - 27);
      }
    }
  }
}

// All blocks of a tile; LDS buffers [block parity][half].
template <int J, bool ROWS>
__device__ __forceinline__ void wide_tile(const WideTile& t, int32_t blocks, uint8_t* a00, uint8_t* a01, uint8_t* a10,
                                          uint8_t* a11, uint8_t* b00, uint8_t* b01, uint8_t* b10, uint8_t* b11,
                                          f32x4 (&acc)[8][8]) {
  constexpr int kScalesA = ROWS ? 1 : 8;
  WideState w;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < kScalesA) w.sa[j] = scale_of(scale_a<ROWS>(t, scales_of(t.scale_a), j));
    if (j < J) w.sb[j] = scale_of(scale_b<ROWS>(t, scales_of(t.scale_b), j));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < kScalesA) asm volatile("" : "+v"(w.sa[j]));
    if (j < J) asm volatile("" : "+v"(w.sb[j]));
  }
  load_half(t.b, 0, blocks, t.off_b[0], b00);
  if (J == 8) load_half(t.b, 0, blocks, t.off_b[1], b01);
  load_half(t.a, 0, blocks, t.off_a[0], a00);
  load_half(t.a, 0, blocks, t.off_a[1], a01);
  load_half(t.b, 1, blocks, t.off_b[0], b10);
  if (J == 8) load_half(t.b, 1, blocks, t.off_b[1], b11);
  load_half(t.a, 1, blocks, t.off_a[0], a10);
  load_half(t.a, 1, blocks, t.off_a[1], a11);
  meet<8 + J>();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const i32x2v raw = read_raw<false>(b00, b01, t.at_b[0], j);
    widen_half<0>(w.b[0][j], raw, w.sb[j]);
    widen_half<1>(w.b[0][j], raw, w.sb[j]);
  }
  const i32x2v raw = read_raw<ROWS>(a00, a01, t.at_a[0], 0);
  widen_half<0>(w.a[0], raw, w.sa[0]);
  widen_half<1>(w.a[0], raw, w.sa[0]);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    w.raw_a[(m + 1) & 3] = read_raw<ROWS>(a00, a01, t.at_a[0], m + 1);
    w.raw_b[m] = read_raw<false>(b00, b01, t.at_b[1], m);
  }
  asm volatile("s_nop 1");
  for (int32_t k = 0; k < blocks; k += 2) {
    wide_block<J, ROWS>(t, w, k, blocks, a00, a01, b00, b01, a10, a11, b10, b11, acc);
    wide_block<J, ROWS>(t, w, k + 1, blocks, a10, a11, b10, b11, a00, a01, b00, b01, acc);
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
// rows; one tile of 256 columns and up to `unit` rows a workgroup, four waves of
// 128 x 128 (128 x 64 when the rows fit B's first half).
//
// Bound by the bf16 products at the clock they leave; larger tiles do not fit the
// registers.  32768 rows by 6 experts of 4096 x 7168: 1237-1256 us, 1.5 PFLOP/s;
// 8192 x 8192 x 8192: 655 us, 1.7 PFLOP/s (a library's plain bf16 product reaches
// 1.24 there).  The 8-bit products that do not keep fp32 sums (see above) took 746
// and 384 us in the same loop.  A tile of at most 128 rows is bound by issue: 192
// widening instructions and 128 products a block, 1.3 us of which the products are
// 0.9.  When the last round of tiles fills at most half of the CUs, two workgroups
// take the halves of each (32768 rows: 1261 -> 1237 us; 34000: 1287 -> 1272; 16500
// by 4 experts of 4096 x 1536: 174 -> 167).
__global__ __launch_bounds__(kMmThreads, 1) void expert_gemm_big_kernel(GemmArgs g, int32_t ntile,
                                                                        int32_t unit) {
  __shared__ __align__(16) uint8_t a00[kHalfBytes], a01[kHalfBytes], a10[kHalfBytes], a11[kHalfBytes];
  __shared__ __align__(16) uint8_t b00[kHalfBytes], b01[kHalfBytes], b10[kHalfBytes], b11[kHalfBytes];
  const int32_t Kp = q_pitch(g.K), Ks = s_pitch(g.K), blocks = Kp / 128;
  const int lane = lane_id(), l16 = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), wi = wv >> 1, wj = wv & 1;
  const int32_t mtile = row_tiles(g.off, g.ne, g.cap, unit);
  const int64_t tiles = static_cast<int64_t>(mtile) * ntile;
  const TileShare share = share_tile(blockIdx.x, tiles, unit == kBigTile);
  if (share.t >= tiles) return;
  const Tile2 at = tile_order(share.t, tiles, mtile, ntile);
  RowTile rt = find_row_tile(g.off, g.ne, g.cap, unit, at.m);
  rt.row0 += share.skip;
  rt.rows = min(rt.rows - share.skip, share.rows);
  if (rt.rows <= 0) return;
  const uint8_t* wp = g.w[rt.p];
  const uint8_t* ws = g.w_scale[rt.p];
  if (!usable(wp, ws)) return;
  const int32_t n0 = at.n * kBigTile, rows = rt.rows, cols = min(g.N - n0, kBigTile);
  WideTile t;
  t.a = BigOperand{wp + static_cast<int64_t>(n0) * Kp, 128, static_cast<uint32_t>(Kp), cols - 1};
  t.b = BigOperand{g.q + rt.row0 * Kp, 128, static_cast<uint32_t>(Kp), rows - 1};
  t.scale_a = ws + static_cast<int64_t>(min(n0 / 128 + wi, ceil_div(g.N, 128) - 1)) * Ks;
  t.scale_b = g.q_scale + rt.row0 * Ks;
  t.pitch_a = t.pitch_b = 1;
  t.scale_row = Ks;
  t.wi = wi;
  t.wj = wj;
  t.l16 = l16;
  load_offsets<true, 0>(t.a, t.off_a[0]);
  load_offsets<true, 1>(t.a, t.off_a[1]);
  load_offsets<false, 0>(t.b, t.off_b[0]);
  load_offsets<false, 1>(t.b, t.off_b[1]);
  read_offsets<true>(t);
  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A fragment of rows at a time through the wave's own piece of LDS, so that a
  // store covers 256 consecutive bytes of four rows and need not go by way of the
  // caches.
  uint8_t* const stage = wv == 0 ? a00 : wv == 1 ? a01 : wv == 2 ? a10 : a11;
  uint16_t* const out = g.out + rt.row0 * g.N + n0;
  const auto store = [&](int j0, int j1) {
    meet<0>();  // LDS is free: the last loads (zeros) have arrived, the reads are done
    const int c = wi * 128 + 8 * l16;
#pragma unroll
    for (int j = j0; j < j1; ++j) {
      // copied to the other registers here, and not all 256 at the loop's end
#pragma unroll
      for (int i = 0; i < 8; ++i) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4*>(stage + l16 * 272 + 64 * i + 16 * kg) =
            u32x4{pack_bf16(acc[2 * i][j][0], acc[2 * i][j][1]), pack_bf16(acc[2 * i][j][2], acc[2 * i][j][3]),
                  pack_bf16(acc[2 * i + 1][j][0], acc[2 * i + 1][j][1]),
                  pack_bf16(acc[2 * i + 1][j][2], acc[2 * i + 1][j][3])};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = b_row(wj, j, 4 * u + kg);
        const u32x4 y = *reinterpret_cast<const u32x4*>(stage + (4 * u + kg) * 272 + 16 * l16);
        if (r < rows && c < cols)
          __builtin_nontemporal_store(y, reinterpret_cast<u32x4*>(out + static_cast<uint32_t>(r * g.N + c)));
      }
    }
  };
  if (rows > 128) {
    wide_tile<8, true>(t, blocks, a00, a01, a10, a11, b00, b01, b10, b11, acc);
    store(0, 8);
  } else {
    wide_tile<4, true>(t, blocks, a00, a01, a10, a11, b00, b01, b10, b11, acc);
    store(0, 4);
  }
}

// ------------------------------------------------------------------------
// Few rows an expert: the weights are the traffic
// ------------------------------------------------------------------------
constexpr int kThinWaves = 4;
constexpr int kThinThreads = 64 * kThinWaves;
constexpr int kThinRows = 32, kThinCols = 32;

// Fragment of 16 rows: the lane's two 16-byte parts kg and kg + 4 of its row, so
// that one load covers 64 bytes of each row in order.  Both operands take the
// same parts, so the products pair the same k.
struct ThinFragment {
  i32x4 part[2];
};

__device__ __forceinline__ ThinFragment thin_fragment(const uint8_t* row) {
  return ThinFragment{{*reinterpret_cast<const i32x4*>(row), *reinterpret_cast<const i32x4*>(row + 64)}};
}

// Bytes 8 * s..8 * s + 7 of the fragment, times their scale, as bf16.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8 thin_widen(const ThinFragment& f, int s, float scale) {
  const uint32_t lo = static_cast<uint32_t>(f.part[s >> 1][2 * (s & 1)]), hi = static_cast<uint32_t>(f.part[s >> 1][2 * (s & 1) + 1]);
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// 32 weight rows by 16 or 32 rows.  The four waves split the blocks of 128
// (wave v takes v, v + 4, ...), every weight byte goes from memory to the
// registers of the one wave that uses it, the next block's while this one is
// multiplied, and the waves' sums meet in LDS and are added in wave order.
// Bound by HBM: 41 rows by 6 experts of 4096 x 7168 (177 MB) take 37 us, 4.8 TB/s.
// Tiles of 16 rows alone read an expert's weights twice as often: 96 rows 61 us
// instead of 52, 128 rows of one expert 43 instead of 31.  With 64 columns a tile 38
// us, 53 and 25, but one expert's 16 or 32 rows 20 and 25 instead of 14; with 16
// columns 43, 64, 44, and 11.5 and 15.
constexpr int kThinFrags = kThinCols / 16;
struct ThinSums {
  float v[kThinWaves][kThinRows][kThinCols + 4];
};

// One wave's part of a tile of up to 16 * FR rows.
template <int FR>
__device__ __forceinline__ void thin_tile(const GemmArgs& g, const RowTile& rt, const uint8_t* wp, const uint8_t* ws, int32_t n0,
                                          int32_t cols, int wv, ThinSums& sums) {
  constexpr int FN = kThinFrags;
  const int32_t Kp = q_pitch(g.K), Ks = s_pitch(g.K), blocks = Kp / 128;
  const int lane = lane_id(), l16 = lane & 15, kg = lane >> 4;
  const uint8_t *pa[FN], *pb[FR], *sb[FR];
#pragma unroll
  for (int i = 0; i < FN; ++i) pa[i] = wp + static_cast<int64_t>(n0 + min(16 * i + l16, cols - 1)) * Kp + kg * 16;
#pragma unroll
  for (int i = 0; i < FR; ++i) {
    const int64_t r = rt.row0 + min(16 * i + l16, rt.rows - 1);
    pb[i] = g.q + r * Kp + kg * 16;
    sb[i] = g.q_scale + r * Ks;
  }
  const uint8_t* sa = ws + static_cast<int64_t>(n0 / 128) * Ks;
  f32x4 acc[FN][FR];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  ThinFragment fa[FN], fb[FR];
  int xa, xb[FR];
  const auto load = [&](int32_t block) {
    const int32_t b = min(block, blocks - 1);
#pragma unroll
    for (int i = 0; i < FN; ++i) fa[i] = thin_fragment(pa[i] + b * 128);
#pragma unroll
    for (int i = 0; i < FR; ++i) fb[i] = thin_fragment(pb[i] + b * 128);
    xa = sa[b];
#pragma unroll
    for (int i = 0; i < FR; ++i) xb[i] = sb[i][b];
  };
  load(wv);
  for (int32_t b = wv; b < blocks; b += kThinWaves) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 wa[FN], wb[FR];
#pragma unroll
      for (int i = 0; i < FN; ++i) wa[i] = thin_widen(fa[i], s, scale_of(xa));
#pragma unroll
      for (int j = 0; j < FR; ++j) wb[j] = thin_widen(fb[j], s, scale_of(xb[j]));
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FR; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[i], wb[j], acc[i][j], 0, 0, 0);
    }
    load(b + kThinWaves);
  }
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j) *reinterpret_cast<f32x4*>(&sums.v[wv][16 * j + l16][16 * i + 4 * kg]) = acc[i][j];
}

__global__ __launch_bounds__(kThinThreads) void expert_gemm_thin_kernel(GemmArgs g, int32_t ntile, int32_t unit) {
  __shared__ __align__(16) ThinSums s_sum;
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t mtile = row_tiles(g.off, g.ne, g.cap, unit);
  const int64_t tiles = static_cast<int64_t>(mtile) * ntile;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t full = tiles & ~int64_t{7};
    const int64_t at = t < full ? (t & 7) * (full >> 3) + (t >> 3) : t;  // an XCD's tiles follow each other
    const int32_t tn = static_cast<int32_t>(at / mtile), tm = static_cast<int32_t>(at - static_cast<int64_t>(tn) * mtile);
    const RowTile rt = find_row_tile(g.off, g.ne, g.cap, unit, tm);
    const uint8_t* wp = g.w[rt.p];
    const uint8_t* ws = g.w_scale[rt.p];
    if (!usable(wp, ws)) continue;
    const int32_t n0 = tn * kThinCols, cols = min(g.N - n0, kThinCols);
    if (t >= gridDim.x) __syncthreads();  // the previous tile's sums have been read
    if (rt.rows <= 16)
      thin_tile<1>(g, rt, wp, ws, n0, cols, wv, s_sum);
    else
      thin_tile<2>(g, rt, wp, ws, n0, cols, wv, s_sum);
    __syncthreads();
    // two columns a thread
    for (int u = threadIdx.x; u < kThinRows * kThinCols / 2; u += kThinThreads) {
      const int row = u / (kThinCols / 2), c = 2 * (u % (kThinCols / 2));
      if (row >= rt.rows || c >= cols) continue;
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int v = 0; v < kThinWaves; ++v) {
        lo += s_sum.v[v][row][c];
        hi += s_sum.v[v][row][c + 1];
      }
      *reinterpret_cast<uint32_t*>(g.out + (rt.row0 + row) * g.N + n0 + c) = pack_bf16(lo, hi);
    }
  }
}

// ------------------------------------------------------------------------
// The weight gradients
// ------------------------------------------------------------------------
// Four consecutive values of a gradient; vec: its address allows 16-byte accesses.
__device__ __forceinline__ void put_gradient(float* d, f32x4 y, bool accumulate, bool vec) {
  if (vec) {
    if (accumulate) y += *reinterpret_cast<const f32x4*>(d);
    __builtin_nontemporal_store(y, reinterpret_cast<f32x4*>(d));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = accumulate ? d[e] + y[e] : y[e];
  }
}

// The expert with the rank-th most rows (ties: lower expert first) of at most
// 64, a lane each; of more, the rank-th expert.  The order leaves short tiles for
// the end (against none: 6 of 4096 x 7168 from 32768 rows 1291 and 1328 us, 8 of
// 1408 x 2048 from 9000 61 and 68, 64 of 1024 x 1024 from 30000 115 and 127).
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

// grads[p][n][k]: A is x (a lane holds four consecutive k of a row n), B is dy.
//
// Bound by the bf16 products at the clock they leave.  32768 rows, 6 experts of
// 4096 x 7168: 1267-1333 us, 1.5 PFLOP/s (a library's plain bf16 product reaches
// 1.24 at 8192 x 8192 x 8192); added to what is there 1553, the old values being
// read where nothing overlaps them.  Before the stores covered whole lines it took
// 1352 us, and against that: 1200 without the loads (a bound, not a result), 2260
// with the tiles dealt to the XCDs in one walk over all experts (an XCD got whole
// experts), 1404 with the widening spread over all eight products of a step.
// Tiles of at most 128 rows of dy, the halves of a last round's among them,
// multiply four fragments of B instead of eight (4 experts of 512 x 1024 from 3000
// rows: 34 -> 23 us; 8 of 1408 x 2048 from 9000: 67 -> 63-68).
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
  const int32_t per = ntile * ktile;
  const TileShare share = share_tile(blockIdx.x, static_cast<int64_t>(ne) * per, true);
  const int32_t turn = static_cast<int32_t>(share.t / per);
  if (turn >= ne) return;
  const Tile2 at = tile_order(share.t - static_cast<int64_t>(turn) * per, per, ntile, ktile);
  const int32_t p = expert_of_rank(off, ne, cap, turn), tn = at.m, tk = at.n;
  float* out = grads[p];
  if (out == nullptr) return;
  const int32_t o0 = group_row(off, p, cap), o1 = group_row(off, p + 1, cap);
  const int32_t blocks = max(ceil_div(o1 - o0, kQBlock), 0);
  if (blocks == 0 && accumulate) return;
  const int64_t first = o0 / kQBlock + p;
  const int32_t n0 = tn * kBigTile + share.skip, k0 = tk * kBigTile;
  const int32_t rows = min(N - n0, share.rows), cols = min(K - k0, kBigTile);
  if (rows <= 0) return;
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
    t.wi = wi;
    t.wj = wj;
    t.l16 = l16;
    load_offsets<false, 0>(t.a, t.off_a[0]);
    load_offsets<false, 1>(t.a, t.off_a[1]);
    load_offsets<false, 0>(t.b, t.off_b[0]);
    load_offsets<false, 1>(t.b, t.off_b[1]);
    read_offsets<false>(t);
    if (rows > 128)
      wide_tile<8, false>(t, blocks, a00, a01, a10, a11, b00, b01, b10, b11, acc);
    else
      wide_tile<4, false>(t, blocks, a00, a01, a10, a11, b00, b01, b10, b11, acc);
  }
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  // a fragment of rows at a time through the wave's own piece of LDS, so that a
  // store covers 256 consecutive bytes four times (4 experts of 1536 x 5120 from
  // 2999 rows: 65 us; straight from the registers, 64 bytes of sixteen rows, 76)
  uint8_t* const stage = wv == 0 ? a00 : wv == 1 ? a01 : wv == 2 ? a10 : a11;
  const int c = 128 * ((lane >> 4) & 1) + 64 * wi + 4 * l16;
  meet<0>();  // LDS is free: the last loads (zeros) have arrived, the reads are done
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (128 * (j >> 2) >= rows) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<f32x4*>(stage + l16 * 528 + 64 * i + 16 * kg) = acc[i][j];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int m = 2 * u + (lane >> 5), r = b_row(wj, j, m);
      const f32x4 y = *reinterpret_cast<const f32x4*>(stage + m * 528 + 16 * (lane & 31));
      if (r < rows && c < cols) put_gradient(out + static_cast<int64_t>(n0 + r) * K + k0 + c, y, accumulate, vec);
    }
  }
}

uint32_t mm_grid(int64_t tiles) { return static_cast<uint32_t>(tiles < (1 << 20) ? tiles : (1 << 20)); }

}  // namespace

hipError_t launch_expert_gemm(const int32_t* off, int32_t ne, const uint8_t* q, const uint8_t* q_scale, int32_t K,
                              const uint8_t* const* w, const uint8_t* const* w_scale, int32_t N, uint16_t* out,
                              int64_t cap, hipStream_t st) {
  if (ne == 0 || cap == 0) return hipSuccess;
  const GemmArgs g{off, ne, q, q_scale, K, w, w_scale, N, out, cap};
  const int32_t nbig = ceil_div(N, kBigTile);
  // Few rows.  Thin tiles take each row tile's weights from memory at 4.8 TB/s,
  // cap / 32 + ne / 2 or so row tiles; big ones 1.3 us a block of 128 of K and
  // more the more of them share the memory, whatever the rows.  Both grow with
  // K alike, which leaves a bound on rows and N; and up to eight rows an expert
  // nearly every thin tile is its expert's only one.  Thin / big, us: 6 experts of
  // 4096 x 7168 at 4, 16, 24, 33 rows an expert 34/81, 54/82, 65/82, 80/82; 24 of
  // 2048 x 5120 at 4, 8, 12, 16: 55/70, 67/72, 77/73, 84/74; 32 of 7168 x 2048 at 4,
  // 8: 83/111, 98/115; 4 of 1536 x 5120 at 16, 32, 70, 100: 14/55, 21/55, 29/55,
  // 34/55; one of 4096 x 7168 at 16, 64, 128, 200: 14/73, 19/74, 33/74, 59/74; 8 of
  // 1024 x 1024 at 32, 55, 100: 8.9/16, 10/16, 13/17; 2 of 7168 x 2048 at 16, 32,
  // 64: 12/26, 15/26, 25/26.
  if (cap <= 8 * static_cast<int64_t>(ne) || (cap + 8 * static_cast<int64_t>(ne)) * N <= 1000000) {
    const int32_t ntile = ceil_div(N, kThinCols);
    // 32 rows a tile, or 16 where that makes too few tiles to keep the memory
    // busy (32 rows of one expert of 4096 x 7168, 128 or 256 tiles: 18.0 and 14.3
    // us; 64 rows, 256 or 512: 18.4 and 23.4)
    const int32_t unit = (cap / kThinRows + ne / 2) * ntile < 192 ? 16 : kThinRows;
    const int64_t tiles = (cap / unit + ne) * ntile;
    hipLaunchKernelGGL(expert_gemm_thin_kernel, dim3(mm_grid(tiles)), dim3(kThinThreads), 0, st, g, ntile, unit);
    return hipGetLastError();
  }
  // Rows a tile, 256 or 128: a tile of 128 takes about 11/15 of the time of one of
  // 256 (77 and 101 us a round at K = 5120), so what counts is the rounds of 256
  // workgroups; an expert's last tile is half full on average.  64 rows for each of
  // 24 experts: 78 us in tiles of 128, 101 in tiles of 256; 200: 135 and 157; 500
  // for each of 6 experts of 4096 x 7168: 182 and 149; 5461: 1483 and 1257.
  const auto rounds = [&](int32_t u) { return ((cap / u + ne / 2 + 1) * nbig + 255) / 256; };
  const int32_t unit = 11 * rounds(128) < 15 * rounds(256) ? 128 : 256;
  const int64_t tiles = (cap / unit + ne) * nbig + (unit == kBigTile ? kComputeUnits / 2 : 0);
  hipLaunchKernelGGL(expert_gemm_big_kernel, dim3(static_cast<uint32_t>(tiles)), dim3(kMmThreads), 0, st, g, nbig, unit);
  return hipGetLastError();
}

hipError_t launch_expert_wgrad(const int32_t* off, int32_t ne, const uint8_t* dyt, const uint8_t* dyt_scale, int32_t N,
                               const uint8_t* xt, const uint8_t* xt_scale, int32_t K, int64_t cap, float* const* grads,
                               bool accumulate, hipStream_t st) {
  if (ne == 0) return hipSuccess;
  const int32_t ntile = ceil_div(N, kBigTile), ktile = ceil_div(K, kBigTile);
  hipLaunchKernelGGL(expert_wgrad_big_kernel, dim3(static_cast<uint32_t>(ne * ntile * ktile + kComputeUnits / 2)), dim3(kMmThreads), 0, st, off,
                     ne, dyt, dyt_scale, N, xt, xt_scale, K, cap, grads, accumulate, ntile, ktile);
  return hipGetLastError();
}

}  // namespace ultraep
