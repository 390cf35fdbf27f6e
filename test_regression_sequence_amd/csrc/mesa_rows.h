// Eight consecutive channels of a token row, as one lane loads and stores them.
// A row may start at any multiple of its element size: gfx950 takes 16-byte
// global accesses at such addresses, so the vectors are declared with the
// element's alignment and rows of odd lengths need no path of their own.  Only
// the last, partial vector of a row goes element by element.
#pragma once

#include "mesa_common.h"

namespace mesa {

typedef u16x8 __attribute__((aligned(2))) u16x8_any;
typedef u16x4 __attribute__((aligned(2))) u16x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

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

// Channels elem .. elem+7, of which the first n (any int) are the row's; the rest are 0.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void* base, size_t elem, int n) {
  Raw8<BF16> r{};
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(base) + elem;
    if (n >= 8) {
      r.v = *reinterpret_cast<const u16x8_any*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) r.v[e] = q[e];
    }
  } else {
    const float* q = static_cast<const float*>(base) + elem;
    if (n >= 8) {
      r.a = reinterpret_cast<const f32x4_any*>(q)[0];
      r.b = reinterpret_cast<const f32x4_any*>(q)[1];
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) {
          if (e < 4) r.a[e & 3] = q[e];
          else r.b[e & 3] = q[e];
        }
    }
  }
  return r;
}

// The first n (any int) of y[0..7] to channels elem .. , rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ void store_raw8(void* base, size_t elem, const float (&y)[8], int n) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(base) + elem;
    u16x8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __builtin_bit_cast(uint16_t, f32_to_bf16(y[e]));
    if (n >= 8) {
      *reinterpret_cast<u16x8_any*>(q) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) q[e] = o[e];
    }
  } else {
    float* q = static_cast<float*>(base) + elem;
    if (n >= 8) {
      reinterpret_cast<f32x4_any*>(q)[0] = f32x4{y[0], y[1], y[2], y[3]};
      reinterpret_cast<f32x4_any*>(q)[1] = f32x4{y[4], y[5], y[6], y[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) q[e] = y[e];
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
