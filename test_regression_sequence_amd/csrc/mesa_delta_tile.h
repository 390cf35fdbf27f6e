// Device helpers of the chunked gated delta rule (gfx950 / CDNA4, wave64).
//
// Numbers that need fp32's precision enter the bf16 matrix instructions as sums
// of up to three bf16 "planes" (x = p0 + p1 + p2 to 2^-25 of x); bf16 inputs are
// one plane.  Products of planes a and b with a + b <= MAX are added, the smaller
// ones first: MAX = 2 keeps fp32's precision, MAX = 1 half a step of 2^-17.
//
// Index orders.  A 16x16x32 instruction takes 8 numbers along its inner index a
// lane.  Every inner index here runs over pairs of 16-wide tiles, lane group
// g = lane / 16 holding 4g..4g+3 of the first and 4g..4g+3 of the second: that is
// how a result leaves the instruction, so a result tile is the next product's
// operand as it is, and what ds_read_b64_tr_b16 gives of a row-major tile.
#pragma once

#include "mesa_common.h"
#include "mesa_delta.h"

namespace mesa {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int N>
struct Planes {
  bf16x8 p[N];
};

// The planes of x: each takes what the ones before left.  (Two numbers a conversion.)
template <int N>
__device__ __forceinline__ void split4(f32x4 x, bf16x4 (&p)[N]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x2 w;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * e], x[2 * e + 1]}, bf16x2));
      if (n + 1 < N) {
        x[2 * e] -= __uint_as_float(w[e] << 16);
        x[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
      }
    }
    p[n] = __builtin_bit_cast(bf16x4, w);
  }
}

__device__ __forceinline__ bf16x8 join(bf16x4 lo, bf16x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int N>
__device__ __forceinline__ Planes<N> split8(f32x4 lo, f32x4 hi) {
  bf16x4 a[N], b[N];
  split4<N>(lo, a);
  split4<N>(hi, b);
  Planes<N> r;
#pragma unroll
  for (int n = 0; n < N; ++n) r.p[n] = join(a[n], b[n]);
  return r;
}

template <int MAX, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Planes<NA>& a, const Planes<NB>& b, f32x4 c) {
#pragma unroll
  for (int sum = MAX; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (sum - i >= 0 && sum - i < NB) c = mfma_bf16(a.p[i], b.p[sum - i], c);
  return c;
}

// The compiler moves nothing across (ON: where registers hold what that keeps alive).
template <bool ON>
__device__ __forceinline__ void fence() {
  if constexpr (ON) __builtin_amdgcn_sched_barrier(0);
}

// acc[i] += a[i] b for four row tiles, their products in turn.
template <int MAX, int NA, int NB>
__device__ __forceinline__ void mma_tiles(const Planes<NA> (&a)[4], const Planes<NB>& b, f32x4 (&acc)[4]) {
#pragma unroll
  for (int sum = MAX; sum >= 0; --sum)
#pragma unroll
    for (int n = 0; n < NA; ++n)
      if (sum - n >= 0 && sum - n < NB)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = mfma_bf16(a[i].p[n], b.p[sum - n], acc[i]);
}

// The same with the operands exchanged: the transposed tiles.
template <int MAX, int NA, int NB>
__device__ __forceinline__ void mma_tiles_t(const Planes<NA>& a, const Planes<NB> (&b)[4], f32x4 (&acc)[4]) {
#pragma unroll
  for (int sum = MAX; sum >= 0; --sum)
#pragma unroll
    for (int n = 0; n < NA; ++n)
      if (sum - n >= 0 && sum - n < NB)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = mfma_bf16(a.p[n], b[i].p[sum - n], acc[i]);
}

// Byte of a row-major bf16 tile of W columns (a multiple of 8).  Units of 8 bytes
// are exchanged from row to row: lanes that read equal columns of 16 rows, or 4
// units of each of 4 rows (ds_read_b64_tr_b16), lie in different LDS banks, for 16
// lanes over 32 banks as for 32 lanes over 64.
template <int W>
__device__ __forceinline__ uint32_t tile_at(int row, int byte) {
  const int r0 = row & 1, r1 = (row >> 1) & 1, r2 = (row >> 2) & 1, r3 = (row >> 3) & 1;
  const int swap = W >= 128 ? (r0 << 2 | r1 << 3 | r2 | r3 << 1 | r2 << 4)
                   : W == 64 ? (r0 | r3 << 1 | (r0 ^ r2) << 2 | r1 << 3) : (r1 | r3 << 1 | (r1 ^ r2) << 2);
  return row * (2 * W) + (((byte >> 3) ^ swap) << 3);
}

// 16 bytes from byte `byte` (a multiple of 16) of a row on.
template <int W>
__device__ __forceinline__ void tile_put16(char* tile, int row, int byte, u32x4 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  *reinterpret_cast<u32x2*>(tile + tile_at<W>(row, byte)) = u32x2{v[0], v[1]};
  *reinterpret_cast<u32x2*>(tile + tile_at<W>(row, byte + 8)) = u32x2{v[2], v[3]};
}

// Rows row0 .. row0+15 (one a lane), columns of tiles 2 s and 2 s + 1: operand of
// a product over columns.  N planes, `plane` bytes apart.
template <int W, int N>
__device__ __forceinline__ Planes<N> rows_of(const char* tile, int plane, int row0, int s, int lane) {
  const int row = row0 + (lane & 15), g = lane >> 4;
  const uint32_t lo = tile_at<W>(row, 64 * s + 8 * g), hi = tile_at<W>(row, 64 * s + 32 + 8 * g);
  Planes<N> r;
#pragma unroll
  for (int n = 0; n < N; ++n)
    r.p[n] = join(*reinterpret_cast<const bf16x4*>(tile + n * plane + lo),
                  *reinterpret_cast<const bf16x4*>(tile + n * plane + hi));
  return r;
}

// A lane's places in a tile's first rows, computed once: the same operands as
// rows_of and columns_of from any multiple of 16 rows on.
template <int W>
struct TileRows {
  uint32_t at[W / 16];
  __device__ __forceinline__ explicit TileRows(int lane) {
#pragma unroll
    for (int j = 0; j < W / 16; ++j) at[j] = tile_at<W>(lane & 15, 32 * j + 8 * (lane >> 4));
  }
  template <int N>
  __device__ __forceinline__ Planes<N> planes(const char* tile, int plane, int row0, int s) const {
    Planes<N> r;
#pragma unroll
    for (int n = 0; n < N; ++n)
      r.p[n] = join(*reinterpret_cast<const bf16x4*>(tile + at[2 * s] + n * plane + row0 * 2 * W),
                    *reinterpret_cast<const bf16x4*>(tile + at[2 * s + 1] + n * plane + row0 * 2 * W));
    return r;
  }
  __device__ __forceinline__ Planes<1> operator()(const char* tile, int row0, int s) const {
    return planes<1>(tile, 0, row0, s);
  }
  // columns 16 col + 4 g .. +3 of a lane's row
  template <int N>
  __device__ __forceinline__ f32x4 values(const char* tile, int plane, int row0, int col) const {
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = N - 1; n >= 0; --n) {
      const bf16x4 v = *reinterpret_cast<const bf16x4*>(tile + at[col] + n * plane + row0 * 2 * W);
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] += (float)v[e];
    }
    return r;
  }
};
// COLS: 16-wide tiles of columns from `first` on.
template <int W, int COLS = W / 16>
struct TileColumns {
  uint32_t at[COLS];
  __device__ __forceinline__ explicit TileColumns(int lane, int first = 0) {
#pragma unroll
    for (int j = 0; j < COLS; ++j)
      at[j] = tile_at<W>(4 * (lane >> 4) + ((lane & 15) >> 2), 32 * (first + j) + 8 * (lane & 3));
  }
  __device__ __forceinline__ bf16x4 four(const char* tile, int row0, int col) const {
    const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(const_cast<char*>(tile + at[col] + row0 * 2 * W)));
    return __builtin_bit_cast(bf16x4, r);
  }
  template <int N>
  __device__ __forceinline__ Planes<N> planes(const char* tile, int plane, int row0, int col) const {
    Planes<N> r;
#pragma unroll
    for (int n = 0; n < N; ++n) r.p[n] = join(four(tile + n * plane, row0, col), four(tile + n * plane, row0 + 16, col));
    return r;
  }
  __device__ __forceinline__ Planes<1> operator()(const char* tile, int row0, int col) const {
    return planes<1>(tile, 0, row0, col);
  }
};

// Rows 4 g .. 4 g + 3 behind row0, of column 16 col + lane % 16.
template <int W>
__device__ __forceinline__ bf16x4 column4(const char* tile, int row0, int col, int lane) {
  const int i = lane & 15, row = row0 + 4 * (lane >> 4) + (i >> 2);
  const char* at = tile + tile_at<W>(row, 32 * col + 8 * (i & 3));
  const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(const_cast<char*>(at)));
  return __builtin_bit_cast(bf16x4, r);
}

// Columns 16 col .. +15 (one a lane), rows row0 .. row0+31: operand of a product over rows.
template <int W, int N>
__device__ __forceinline__ Planes<N> columns_of(const char* tile, int plane, int row0, int col, int lane) {
  Planes<N> r;
#pragma unroll
  for (int n = 0; n < N; ++n)
    r.p[n] = join(column4<W>(tile + n * plane, row0, col, lane), column4<W>(tile + n * plane, row0 + 16, col, lane));
  return r;
}

// The values of one result tile's layout: 4 of N planes added up.
template <int W, int N>
__device__ __forceinline__ f32x4 column_values(const char* tile, int plane, int row0, int col, int lane) {
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const bf16x4 v = column4<W>(tile + n * plane, row0, col, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] += (float)v[e];
  }
  return r;
}

// A uniform address as the memory unit's descriptor: a lane's load adds its 32-bit
// offset itself, and one from 2^31 on reads zeros and no memory.  So a tile's loads
// are one run of instructions without a branch or a 64-bit sum, whichever rows exist;
// with branches the compiler waited for the loads before each, four latencies a tile.
typedef __amdgpu_buffer_rsrc_t Window;
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ Window window_at(const void* at) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, 0x7fffffff, 0x00020000);
}
__device__ __forceinline__ u32x4 window_load(Window w, uint32_t lane_offset, uint32_t offset) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w, lane_offset, offset, 0));
}

// 4 numbers of a row
template <bool BF16>
__device__ __forceinline__ f32x4 window_row(Window w, uint32_t lane_offset, uint32_t offset) {
  if constexpr (BF16) {
    const u16x4 u = __builtin_bit_cast(u16x4, __builtin_amdgcn_raw_buffer_load_b64(w, lane_offset, offset, 0));
    return f32x4{bf16_to_f32(u[0]), bf16_to_f32(u[1]), bf16_to_f32(u[2]), bf16_to_f32(u[3])};
  } else {
    return __builtin_bit_cast(f32x4, window_load(w, lane_offset, offset));
  }
}

__device__ __forceinline__ float window_number(Window w, uint32_t lane_offset, uint32_t offset) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(w, lane_offset, offset, 0));
}

__device__ __forceinline__ void window_store(Window w, uint32_t lane_offset, uint32_t offset, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), w, lane_offset, offset, 0);
}
// 16 bytes: the offset goes to the lanes.  The hardware still reads such a store's data when
// the next instruction runs; the compiler keeps that one from writing the registers where
// the store has no scalar offset, and takes one with a scalar offset to be safe, which it is
// not: zeros arrived as the product that the next instruction formed in their register.
__device__ __forceinline__ void window_store(Window w, uint32_t lane_offset, uint32_t offset, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), w, lane_offset + offset, 0, 0);
}
// 4 numbers in the rows' type
template <bool BF16>
__device__ __forceinline__ void window_store_row(Window w, uint32_t lane_offset, uint32_t offset, f32x4 v) {
  if constexpr (BF16) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    bf16x4 p[1];
    split4<1>(v, p);
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, p[0]), w, lane_offset, offset, 0);
  } else {
    window_store(w, lane_offset, offset, v);
  }
}

// 64 rows of W elements on their way from memory to an LDS tile: 16-byte pieces
// in registers, rows at and behind `live` as zeros whatever they hold.
template <int W, bool BF16, int THREADS>
struct RowLoads {
  static constexpr int kPer = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;  // elements of a piece, bytes of an element
  static constexpr int kPieces = 64 * W / kPer, kN = (kPieces + THREADS - 1) / THREADS;
  static constexpr int kRows = THREADS * kPer / W;  // rows between a thread's pieces
  u32x4 r[kN];

  // cols: columns that exist (the others are zeros); stride <= 2^20
  __device__ __forceinline__ void load(const void* base, int64_t row0, int64_t stride, int live, int cols, int tid) {
    const Window from = window_at(static_cast<const char*>(base) + row0 * kSize);
    const int row = tid / (W / kPer), col = tid % (W / kPer) * kPer;
    const uint32_t off = (uint32_t)(row * (int)stride + col) * kSize, step = kRows * (uint32_t)stride * kSize;
    const int rows = col < cols ? live : 0;
#pragma unroll
    for (int n = 0; n < kN; ++n) r[n] = window_load(from, row + n * kRows < rows ? off : kNowhere, n * step);
  }

  // N planes (1 for bf16, 3 for fp32)
  __device__ __forceinline__ void store(char* tile, int plane, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int row = tid / (W / kPer) + n * kRows, col = tid % (W / kPer) * kPer;
      if (kPieces % THREADS != 0 && row >= 64) continue;
      if constexpr (BF16) {
        tile_put16<W>(tile, row, 2 * col, r[n]);
      } else {
        bf16x4 p[3];
        split4<3>(__builtin_bit_cast(f32x4, r[n]), p);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x4*>(tile + i * plane + tile_at<W>(row, 2 * col)) = p[i];
      }
    }
  }
};

// 64 rows of W fp32 numbers in planes, between their conversion and LDS.
template <int W, int THREADS>
struct RowPlanes {
  using Loads = RowLoads<W, false, THREADS>;
  bf16x4 x[Loads::kN][3];
  __device__ __forceinline__ explicit RowPlanes(const Loads& rows) {
#pragma unroll
    for (int n = 0; n < Loads::kN; ++n) split4<3>(__builtin_bit_cast(f32x4, rows.r[n]), x[n]);
  }
  __device__ __forceinline__ void store(char* tile, int plane, int tid) const {
#pragma unroll
    for (int n = 0; n < Loads::kN; ++n) {
      const int row = tid / (W / 4) + n * Loads::kRows, col = tid % (W / 4) * 4;
      if (Loads::kPieces % THREADS != 0 && row >= 64) continue;
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x4*>(tile + i * plane + tile_at<W>(row, 2 * col)) = x[n][i];
    }
  }
};

// `BYTES` bytes on their way from memory to LDS as they are.
template <int BYTES, int THREADS>
struct CopyLoads {
  static_assert(BYTES % 16 == 0, "16-byte pieces");
  static constexpr int kPieces = BYTES / 16, kN = (kPieces + THREADS - 1) / THREADS;
  u32x4 r[kN];

  __device__ __forceinline__ void load(const void* base, int tid) {
    const Window from = window_at(base);
#pragma unroll
    for (int n = 0; n < kN; ++n)
      r[n] = window_load(from, (n + 1) * THREADS <= kPieces || tid + n * THREADS < kPieces ? (uint32_t)tid * 16 : kNowhere,
                         n * THREADS * 16);
  }
  __device__ __forceinline__ void store(char* to, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n)
      if ((n + 1) * THREADS <= kPieces || tid + n * THREADS < kPieces)
        reinterpret_cast<u32x4*>(to + n * THREADS * 16)[tid] = r[n];
  }
};

// A triangular 64x64 matrix as operands: six blocks of 16 rows x 32 inner indices, 8
// numbers a lane, one after another; a plane is 6 KB.  Halves of a block beyond the
// diagonal are zeros.
constexpr int kBlocksBytes = 6 * 1024;
__device__ __forceinline__ constexpr int lower_block(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }  // s <= i / 2
__device__ __forceinline__ constexpr int upper_block(int i, int s) { return i < 2 ? 2 * i + s : 2 + i; }  // s >= i / 2

// In memory: the fp32 numbers of its ten tiles, each 64 lanes' four, in the order of the
// blocks' halves.
constexpr int kTriangleBytes = (int)kDeltaMatrixBytes / 2;
template <bool LOWER>
__device__ __forceinline__ constexpr int triangle_tile(int i, int j) {  // row tile i, column tile j
  const int half = 2 * (LOWER ? lower_block(i, j / 2) : upper_block(i, j / 2)) + (j & 1);
  return LOWER ? half - (half > 1) - (half > 7) : half - (half > 4) - (half > 10);
}
template <bool LOWER>
__device__ __forceinline__ constexpr int triangle_half(int tile) {
  return LOWER ? tile + (tile >= 1) + (tile >= 6) : tile + (tile >= 4) + (tile >= 9);
}

// Its way from there to N planes of blocks.
template <int N, bool LOWER, int THREADS>
struct TriangleLoads : CopyLoads<kTriangleBytes, THREADS> {
  using Loads = CopyLoads<kTriangleBytes, THREADS>;
  static __device__ __forceinline__ void put(char* blocks, int half, int lane, const bf16x4 (&x)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      *reinterpret_cast<bf16x4*>(blocks + n * kBlocksBytes + (half >> 1) * 1024 + (half & 1) * 8 + lane * 16) = x[n];
  }
  // the two halves beyond the diagonal, once
  static __device__ __forceinline__ void clear(char* blocks, int tid) {
    const bf16x4 none[N] = {};
    if (tid < 64) put(blocks, LOWER ? 1 : 4, tid, none);
    else if (tid < 128) put(blocks, LOWER ? 7 : 10, tid - 64, none);
  }
  bf16x4 x[Loads::kN][N];
  __device__ __forceinline__ void split() {
#pragma unroll
    for (int n = 0; n < Loads::kN; ++n) split4<N>(__builtin_bit_cast(f32x4, Loads::r[n]), x[n]);
  }
  __device__ __forceinline__ void put(char* blocks, int tid) const {
#pragma unroll
    for (int n = 0; n < Loads::kN; ++n)
      if ((n + 1) * THREADS <= Loads::kPieces || tid + n * THREADS < Loads::kPieces)
        put(blocks, triangle_half<LOWER>(__builtin_amdgcn_readfirstlane(tid >> 6) + n * (THREADS / 64)), tid & 63, x[n]);
  }
  __device__ __forceinline__ void store(char* blocks, int tid) {
    split();
    put(blocks, tid);
  }
};

template <int N>
__device__ __forceinline__ Planes<N> block_of(const char* blocks, int block, int lane) {
  Planes<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n)
    f.p[n] = *reinterpret_cast<const bf16x8*>(blocks + n * kBlocksBytes + block * 1024 + lane * 16);
  return f;
}

// acc += L b goes in three pairs of blocks whose row tiles differ, each pair's loads
// one ahead.  LOWER: L lower triangular, else upper.  SWAP: the transposed tiles.
// `first`: the first pair, loaded before.
template <bool LOWER>
__device__ __forceinline__ constexpr int pair_step(int n) { return LOWER ? n / 2 : (n + 1) / 2; }
template <bool LOWER>
__device__ __forceinline__ constexpr int pair_row(int n) { return LOWER ? (n == 0 ? 0 : 2) : (n == 2 ? 2 : 0); }

template <int NA>
struct BlockPair {
  Planes<NA> a[2];
};

template <bool LOWER, int NA>
__device__ __forceinline__ BlockPair<NA> pair_of(const char* blocks, int n, int lane) {
  BlockPair<NA> f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = pair_row<LOWER>(n) + e, s = pair_step<LOWER>(n);
    f.a[e] = block_of<NA>(blocks, LOWER ? lower_block(i, s) : upper_block(i, s), lane);
  }
  return f;
}

// acc += L b for pair n of L's blocks.
template <int MAX, bool LOWER, bool SWAP, int NA, int NB>
__device__ __forceinline__ void mma_pair(int n, const BlockPair<NA>& f, const Planes<NB> (&b)[2], f32x4 (&acc)[4]) {
#pragma unroll
  for (int sum = MAX; sum >= 0; --sum)
#pragma unroll
    for (int q = 0; q < NA; ++q)
      if (sum - q >= 0 && sum - q < NB)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bf16x8 x = f.a[e].p[q], y = b[pair_step<LOWER>(n)].p[sum - q];
          f32x4& to = acc[pair_row<LOWER>(n) + e];
          to = SWAP ? mfma_bf16(y, x, to) : mfma_bf16(x, y, to);
        }
}

template <int MAX, bool LOWER, bool SWAP, bool FENCED, int NA, int NB>
__device__ __forceinline__ void mma_triangle(const char* blocks, BlockPair<NA> first, const Planes<NB> (&b)[2],
                                             f32x4 (&acc)[4], int lane) {
  BlockPair<NA> f[2];
  f[0] = first;
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    if (n < 2) f[(n + 1) & 1] = pair_of<LOWER, NA>(blocks, n + 1, lane);
    fence<FENCED>();
    mma_pair<MAX, LOWER, SWAP>(n, f[n & 1], b, acc);
    fence<FENCED>();
  }
}

// The number of valid tokens of sequence b.
__device__ __forceinline__ int delta_length(const DeltaParams& p, int b) {
  if (!p.lengths) return p.T;
  return min(max(__builtin_amdgcn_readfirstlane(p.lengths[b]), 0), p.T);
}

// The address of token t's number.
__device__ __forceinline__ float* gate_at(const DeltaGate& x, int b, int h, int64_t t) {
  return x.at + (b * x.b + h * x.h + t * x.t);
}

// exp2 of a difference of two logarithms that are kept in 64 bits.
__device__ __forceinline__ float decay(double a, double b) { return __builtin_amdgcn_exp2f((float)(a - b)); }
// The same with fp32's precision for small results too: the whole part becomes an exponent, where rounding 20.3
// to fp32 alone costs 2^-20 of the result.
__device__ __forceinline__ float decay_exact(double a, double b) {
  const double x = a - b;
  const float whole = rintf((float)x);
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(x - (double)whole)), (int)whole);
}

// One workgroup's part of a walk: 64 columns of one head's state over one segment's chunks.
struct Part {
  int bh, b, h, seg, col0, cols, len, first, last;
};

// The workgroups of one head go to one XCD (workgroups are handed to the 8 XCDs in
// turn), whose L2 they share.  False: no part.
__device__ __forceinline__ bool part_of(const DeltaParams& p, uint32_t id, Part& x) {
  const uint32_t xcd = id & 7, n = id >> 3;
  x.bh = (int)(n / p.by_part) * 8 + (int)xcd;
  if (x.bh >= p.B * p.H) return false;
  const uint32_t rest = n % p.by_part;
  x.seg = (int)(rest / p.by_slices) + p.seg0;
  x.b = (uint32_t)x.bh / p.by_h;
  x.h = (uint32_t)x.bh % p.by_h;
  x.col0 = 64 * (int)(rest % p.by_slices);
  x.cols = min(64, p.dv - x.col0);
  x.len = delta_length(p, x.b);
  x.first = x.seg * p.L;
  x.last = max(min((x.len + 63) / 64, x.first + p.L), x.first);
  return true;
}
inline uint32_t walk_blocks(const DeltaParams& p) {
  return (uint32_t)((p.B * p.H + 7) / 8 * 8 * ((p.dv + 63) / 64) * p.segs);
}

// Where a walk's state [dv, dk] comes from and goes to (null: zeros, nowhere).  `edge`: the
// segment that starts the walk, or ends it.  Behind the join none starts from `given`, which
// may lie under what another one of the launch ends with.
__device__ __forceinline__ const float* walk_from(const DeltaParams& p, const Part& x, const float* given, int edge) {
  const int64_t size = (int64_t)p.dv * p.dk;
  if (p.NS > 1 && !p.open) return p.seg_start + ((int64_t)x.bh * p.NS + x.seg) * size;
  return given && x.seg == edge ? given + x.bh * size : nullptr;
}
__device__ __forceinline__ float* walk_to(const DeltaParams& p, const Part& x, float* wanted, int edge) {
  const int64_t size = (int64_t)p.dv * p.dk;
  if (p.open) return p.seg_add + ((int64_t)x.bh * p.NS + x.seg) * size;
  return wanted && x.seg == edge ? wanted + x.bh * size : nullptr;
}

template <typename T>
__device__ __forceinline__ void store_out4(void* base, int64_t at, f32x4 v);
template <>
__device__ __forceinline__ void store_out4<float>(void* base, int64_t at, f32x4 v) {
  *reinterpret_cast<f32x4*>(static_cast<float*>(base) + at) = v;
}
template <>
__device__ __forceinline__ void store_out4<__bf16>(void* base, int64_t at, f32x4 v) {
  bf16x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = (__bf16)v[e];
  *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(base) + at) = r;
}

}  // namespace mesa
