// Eight consecutive channels of a token row, as one lane loads and stores them.
// A row may start at any multiple of its element size: gfx950 takes 16-byte
// global accesses at such addresses, so the vectors are declared with the
// element's alignment and rows of odd lengths need no path of their own.  The
// last, partial vector of a row is loaded as the row's last 8 channels and
// shifted into place when it is used, and stored in pieces of 4, 2 and 1: element
// by element, with up to 7 accesses for one lane, the norm of 32768 bf16 rows of
// 1007 took 78 us and its gradient 145, against 47 and 54.
#pragma once

#include "mesa_common.h"

namespace mesa {

typedef u16x8 __attribute__((aligned(2))) u16x8_any;
typedef u16x4 __attribute__((aligned(2))) u16x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef f32x2 __attribute__((aligned(4))) f32x2_any;
typedef uint32_t __attribute__((aligned(2))) u32_any;

template <bool BF16>
struct Raw8;  // as stored
template <>
struct Raw8<true> {
  u16x8 v;
  __device__ __forceinline__ float at(int e) const { return bf16_to_f32(v[e]); }
};
template <>
struct Raw8<false> {
  f32x4 a, b;
  __device__ __forceinline__ float at(int e) const { return e < 4 ? a[e] : b[e - 4]; }
};

// Channels elem .. elem+7.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void* base, size_t elem) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.v = *reinterpret_cast<const u16x8_any*>(static_cast<const uint16_t*>(base) + elem);
  } else {
    const float* q = static_cast<const float*>(base) + elem;
    r.a = reinterpret_cast<const f32x4_any*>(q)[0];
    r.b = reinterpret_cast<const f32x4_any*>(q)[1];
  }
  return r;
}

// Channels elem .. elem+7, of which the first n (any int) exist; the rest are 0.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_part8(const void* base, size_t elem, int n) {
  if (n >= 8) return load_raw8<BF16>(base, elem);
  Raw8<BF16> r{};
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(base) + elem;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    uint32_t pair = 0, last = 0;
    if (n > 0) {
      if (n & 4) r.v.lo = *reinterpret_cast<const u16x4_any*>(q);
      if (n & 2) pair = *reinterpret_cast<const u32_any*>(q + (n & 4));
      if (n & 1) last = q[n & 6];
    }
    u32x4 w = __builtin_bit_cast(u32x4, r.v);
    const uint32_t first = n & 2 ? pair : last, second = n & 2 ? last : 0;
    if (n > 0 && n & 4) {
      w[2] = first;
      w[3] = second;
    } else {
      w[0] = first;
      w[1] = second;
    }
    r.v = __builtin_bit_cast(u16x8, w);
  } else {
    const float* q = static_cast<const float*>(base) + elem;
    f32x2 pair = {0.f, 0.f};
    float last = 0.f;
    if (n > 0) {
      if (n & 4) r.a = *reinterpret_cast<const f32x4_any*>(q);
      if (n & 2) pair = *reinterpret_cast<const f32x2_any*>(q + (n & 4));
      if (n & 1) last = q[n & 6];
    }
    const f32x4 rest = n & 2 ? f32x4{pair[0], pair[1], last, 0.f} : f32x4{last, 0.f, 0.f, 0.f};
    if (n > 0 && n & 4) r.b = rest;
    else r.a = rest;
  }
  return r;
}

// How rows of D channels end: with a whole vector (D a multiple of 8), within a
// vector (D > 8), or before the first one does (D < 8).  A choice made at compile
// time: without the others' code the loads of whole vectors are 2 to 5 % faster.
enum class RowEnd { kWhole, kWithin, kShort };
__host__ __device__ constexpr RowEnd row_end(int D) {
  return D % 8 == 0 ? RowEnd::kWhole : D > 8 ? RowEnd::kWithin : RowEnd::kShort;
}

// Channels ch .. ch+7 of the row that starts at `row`, 0 behind it.  kWithin: the
// vector that the row ends within, and those behind it, are loaded as the row's
// last 8; own_channels() then has to put them into place.
template <bool BF16, RowEnd END>
__device__ __forceinline__ Raw8<BF16> load_row8(const void* base, size_t row, int ch, int D) {
  constexpr uint32_t ES = BF16 ? 2 : 4;
  if constexpr (END == RowEnd::kWithin) {  // (a uniform row and a 32-bit offset within it)
    return load_raw8<BF16>(static_cast<const char*>(base) + row * ES + (uint32_t)min(ch, D - 8) * ES, 0);
  } else if constexpr (END == RowEnd::kWhole) {
    Raw8<BF16> r{};
    if (ch < D) r = load_raw8<BF16>(base, row + ch);
    return r;
  } else {
    return load_part8<BF16>(base, row + ch, D - ch);
  }
}

// Has r's loads finished here.
__device__ __forceinline__ void hold(Raw8<true>& r) { asm volatile("" : "+v"(r.v)); }
__device__ __forceinline__ void hold(Raw8<false>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// What load_row8 loaded of channels behind the row becomes 0, the others move
// from the end of the vector to their places.
__device__ __forceinline__ void own_channels(Raw8<true>& r, int ch, int D) {
  if (ch + 8 <= D) return;
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 v = __builtin_bit_cast(u64x2, r.v);
  const int by = min(16 * (ch + 8 - D), 128);  // bits, at least 16
  u64x2 o;
  if (by >= 64) o = u64x2{by < 128 ? v.y >> (by & 63) : 0, 0};
  else o = u64x2{v.x >> by | v.y << (64 - by), v.y >> by};
  r.v = __builtin_bit_cast(u16x8, o);
}
__device__ __forceinline__ void own_channels(Raw8<false>& r, int ch, int D) {
  if (ch + 8 <= D) return;
  const int by = min(ch + 8 - D, 8);  // channels
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = by < 8 ? r.at(e) : 0.f;
#pragma unroll
  for (int step = 4; step; step /= 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = by & step ? (e + step < 8 ? v[e + step] : 0.f) : v[e];
  r.a = f32x4{v[0], v[1], v[2], v[3]};
  r.b = f32x4{v[4], v[5], v[6], v[7]};
}

// The first n (any int; !TAIL: 8 or none) of y[0..7] to channels elem .. , rounded
// to nearest even.
template <bool BF16, bool TAIL>
__device__ __forceinline__ void store_raw8(void* base, size_t elem, const float (&y)[8], int n) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(base) + elem;
    u16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __builtin_bit_cast(uint16_t, f32_to_bf16(y[e]));
    if (n >= 8) {
      *reinterpret_cast<u16x8_any*>(q) = o;
    } else if (TAIL && n > 0) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      const u32x4 w = __builtin_bit_cast(u32x4, o);
      const uint32_t pair = n & 4 ? w[2] : w[0];
      const uint32_t last = n & 2 ? (n & 4 ? w[3] : w[1]) : pair;
      if (n & 4) *reinterpret_cast<u16x4_any*>(q) = u16x4{o[0], o[1], o[2], o[3]};
      if (n & 2) *reinterpret_cast<u32_any*>(q + (n & 4)) = pair;
      if (n & 1) q[n & 6] = (uint16_t)last;
    }
  } else {
    float* q = static_cast<float*>(base) + elem;
    if (n >= 8) {
      reinterpret_cast<f32x4_any*>(q)[0] = f32x4{y[0], y[1], y[2], y[3]};
      reinterpret_cast<f32x4_any*>(q)[1] = f32x4{y[4], y[5], y[6], y[7]};
    } else if (TAIL && n > 0) {
      const f32x2 pair = n & 4 ? f32x2{y[4], y[5]} : f32x2{y[0], y[1]};
      const float last = n & 2 ? (n & 4 ? y[6] : y[2]) : pair[0];
      if (n & 4) *reinterpret_cast<f32x4_any*>(q) = f32x4{y[0], y[1], y[2], y[3]};
      if (n & 2) *reinterpret_cast<f32x2_any*>(q + (n & 4)) = pair;
      if (n & 1) q[n & 6] = last;
    }
  }
}

// Maximum over each aligned group of N lanes (N = 16 or 64), in every lane.
#define MESA_DPP_MAX(v, ctrl) \
  fmaxf((v), __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), (ctrl), 0xF, 0xF, false)))
template <int N>
__device__ __forceinline__ float group_max(float v) {
  static_assert(N == 16 || N == 64, "a 16-lane row or a wave");
  v = MESA_DPP_MAX(v, 0xB1);
  v = MESA_DPP_MAX(v, 0x4E);
  v = MESA_DPP_MAX(v, 0x141);
  v = MESA_DPP_MAX(v, 0x140);
  if constexpr (N == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
  }
  return v;
}

}  // namespace mesa
