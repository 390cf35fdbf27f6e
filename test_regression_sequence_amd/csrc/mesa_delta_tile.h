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

// The planes of x: each takes what the ones before left.
template <int N>
__device__ __forceinline__ void split4(f32x4 x, bf16x4 (&p)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[n][e] = (__bf16)x[e];
      if (n + 1 < N) x[e] -= (float)p[n][e];
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

// Byte of a row-major bf16 tile of W columns, in units of 32 bytes that are
// exchanged from row to row so that 16 rows' equal columns lie in all LDS banks.
template <int W>
__device__ __forceinline__ uint32_t tile_at(int row, int byte) {
  constexpr int kShift = W >= 128 ? 0 : W == 64 ? 1 : 2, kMask = W / 16 - 1;
  return row * (2 * W) + ((((byte >> 5) ^ ((row >> kShift) & kMask)) << 5) | (byte & 31));
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

// Row row0 + lane % 16, columns 16 col + 4 g .. +3.
template <int W, int N>
__device__ __forceinline__ f32x4 row_values(const char* tile, int plane, int row0, int col, int lane) {
  const uint32_t at = tile_at<W>(row0 + (lane & 15), 32 * col + 8 * (lane >> 4));
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(tile + n * plane + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] += (float)v[e];
  }
  return r;
}

// 64 rows of W elements on their way from memory to an LDS tile: 16-byte pieces
// in registers, rows at and behind `live` as zeros whatever they hold.
template <int W, bool BF16, int THREADS>
struct RowLoads {
  static constexpr int kPer = BF16 ? 8 : 4;  // elements of a piece
  static constexpr int kPieces = 64 * W / kPer, kN = (kPieces + THREADS - 1) / THREADS;
  u32x4 r[kN];

  // cols: columns that exist (the others are zeros)
  __device__ __forceinline__ void load(const void* base, int64_t row0, int64_t stride, int live, int cols, int tid) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int piece = tid + n * THREADS, row = piece / (W / kPer), col = piece % (W / kPer) * kPer;
      u32x4 v = {0, 0, 0, 0};
      if ((kPieces % THREADS == 0 || piece < kPieces) && row < live && col < cols) {
        const int64_t at = row0 + row * stride + col;
        v = *reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + at * (BF16 ? 2 : 4));
      }
      r[n] = v;
    }
  }

  // N planes (1 for bf16, 3 for fp32)
  __device__ __forceinline__ void store(char* tile, int plane, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int piece = tid + n * THREADS, row = piece / (W / kPer), col = piece % (W / kPer) * kPer;
      if (kPieces % THREADS != 0 && piece >= kPieces) continue;
      if constexpr (BF16) {
        *reinterpret_cast<u32x4*>(tile + tile_at<W>(row, 2 * col)) = r[n];
      } else {
        bf16x4 p[3];
        split4<3>(__builtin_bit_cast(f32x4, r[n]), p);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x4*>(tile + i * plane + tile_at<W>(row, 2 * col)) = p[i];
      }
    }
  }
};

// The number of valid tokens of sequence b.
__device__ __forceinline__ int delta_length(const DeltaParams& p, int b) {
  if (!p.lengths) return p.T;
  return min(max(p.lengths[b], 0), p.T);
}

// The address of token t's number.
__device__ __forceinline__ float* gate_at(const DeltaGate& x, int b, int h, int64_t t) {
  return x.at + (b * x.b + h * x.h + t * x.t);
}

// exp2 of a difference of two logarithms that are kept in 64 bits.
__device__ __forceinline__ float decay(double a, double b) { return exp2f((float)(a - b)); }

// Unit `id` of `slices` workgroups for each (sequence, head): those of one head go
// to one XCD (workgroups are handed to the 8 XCDs in turn), whose L2 they share.
__device__ __forceinline__ bool delta_unit(uint32_t id, int slices, int BH, int& bh, int& slice) {
  const uint32_t xcd = id & 7, n = id >> 3;
  bh = (int)(n / slices) * 8 + (int)xcd;
  slice = (int)(n % slices);
  return bh < BH;
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
