// Tiles of the gated linear recurrence, h_t = a_t h_{t-1} + u_t per channel, and
// the scan that joins them.
//
// A token range [t0, t1) maps the state before it to the state behind it by
// h -> A h + E with A = prod a_t and E the state that starts from zero; ranges
// join as (A1, E1), (A2, E2) -> (A1 A2, A2 E1 + E2).  A workgroup of NW waves
// holds a tile of 64 channels by L = 4 NW TW tokens in registers: a wave is 4
// rows of 16 lanes, a lane holds 4 neighbouring channels of TW tokens in turn,
// row r of wave w those from (4 w + r) TW on.  Each lane folds its tokens, the
// rows of a wave are joined by cross-row swaps, the waves through LDS, and the
// tiles of one sequence and slab through device memory, so that every input is
// read once.
#pragma once

#include <type_traits>

#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_rows.h"

namespace mesa {

constexpr int kLruSlab = 64;    // channels of a tile
constexpr int kLruGroup = 16;   // tiles whose joined pair is published as one

// Words of one chain (sequence and slab) of `tiles` tiles: a word per channel
// of each tile, then of each whole group.
inline __host__ __device__ size_t lru_chain_words(int tiles) {
  return (size_t)(tiles + tiles / kLruGroup) * kLruSlab;
}

struct Pair {  // h -> A h + E
  float A, E;
};
__device__ __forceinline__ Pair join(Pair first, Pair second) {
  return Pair{first.A * second.A, __builtin_fmaf(second.A, first.E, second.E)};
}
__device__ __forceinline__ float apply(Pair p, float h) { return __builtin_fmaf(p.A, h, p.E); }

// From each row's pair: the pair of the wave's rows before this one, and of all
// four (REV: rows run backwards in the scan, row 3 first).
template <bool REV>
__device__ __forceinline__ void join_rows(Pair own, int row, Pair& before, Pair& all) {
  auto swap16 = [](float v) { return __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false); };
  auto swap32 = [](float v) { return __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false); };
  const auto a16 = swap16(own.A), e16 = swap16(own.E);
  constexpr int F = REV ? 1 : 0, S = 1 - F;
  const Pair first{__uint_as_float(a16[F]), __uint_as_float(e16[F])};
  const Pair second{__uint_as_float(a16[S]), __uint_as_float(e16[S])};
  const Pair two = join(first, second);
  const bool later = ((row & 1) != 0) != REV;
  const Pair in_two{later ? first.A : 1.f, later ? first.E : 0.f};
  const auto a32 = swap32(two.A), e32 = swap32(two.E);
  const Pair lo{__uint_as_float(a32[F]), __uint_as_float(e32[F])};
  const Pair hi{__uint_as_float(a32[S]), __uint_as_float(e32[S])};
  all = join(lo, hi);
  const bool later2 = (row >= 2) != REV;
  const Pair both = join(lo, in_two);
  before = Pair{later2 ? both.A : in_two.A, later2 ? both.E : in_two.E};
}

// A published pair is one 64-bit word, so that a reader sees it whole or not at
// all and no ordering with other memory is needed.  kLruEmpty (written by
// lru_clear_kernel before the tiles run) marks a word not yet published; its
// low half is a NaN pattern that A is replaced in.
constexpr uint64_t kLruEmpty = ~0ull;

__device__ __forceinline__ void publish(uint64_t* word, Pair p) {
  uint32_t a = __float_as_uint(p.A);
  if (a == 0xFFFFFFFFu) a = 0x7FC00000u;
  __hip_atomic_store(word, ((uint64_t)__float_as_uint(p.E) << 32) | a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The N words at `word`, kLruSlab apart (one lane a channel), of which the
// first `count` are waited for; the rest read as the identity.
template <int N>
__device__ __forceinline__ void await(const uint64_t* word, int count, Pair (&p)[N]) {
  uint64_t v[N];
  bool missing;
  do {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = i < count ? __hip_atomic_load(word + (size_t)i * kLruSlab, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    missing = false;
#pragma unroll
    for (int i = 0; i < N; ++i) missing |= (uint32_t)v[i] == 0xFFFFFFFFu;
  } while (__any(missing));
#pragma unroll
  for (int i = 0; i < N; ++i)
    p[i] = i < count ? Pair{__uint_as_float((uint32_t)v[i]), __uint_as_float((uint32_t)(v[i] >> 32))} : Pair{1.f, 0.f};
}

// The state before tile j (of `tiles`, counted in the scan's direction) of one
// chain, from the state before tile 0, in a wave with one lane per channel.
// Publishes this tile's pair first, so nobody waits for this wave longer than
// for its own loads; then folds the pairs of whole groups of tiles and of the
// tiles before j in its own group, each in order.  Which words are folded in
// which order depends on j alone: the result has the same bits in every run.
// Every wait ends: tiles take tickets in order, so a tile that is waited for is
// already running, and it publishes before it waits; a group's pair is
// published by its last tile, which waits for tiles only.
__device__ __forceinline__ float lru_carry(uint64_t* words, int tiles, int j, int lane, Pair own, float h) {
  uint64_t* tile_words = words + lane;
  uint64_t* group_words = words + (size_t)tiles * kLruSlab + lane;
  publish(tile_words + (size_t)j * kLruSlab, own);
  const int g = j / kLruGroup, i = j % kLruGroup;
  constexpr int N = 8;
  static_assert(kLruGroup == 2 * N, "a group's earlier tiles are two batches");
  // the group's pair first: later groups wait for it
  Pair tile0[N], tile1[N];
  await<N>(tile_words + (size_t)g * kLruGroup * kLruSlab, i, tile0);
  await<N>(tile_words + ((size_t)g * kLruGroup + N) * kLruSlab, i - N, tile1);
  if (i == kLruGroup - 1) {
    Pair all = tile0[0];
#pragma unroll
    for (int k = 1; k < N; ++k) all = join(all, tile0[k]);
#pragma unroll
    for (int k = 0; k < N; ++k) all = join(all, tile1[k]);
    publish(group_words + (size_t)g * kLruSlab, join(all, own));
  }
  for (int g0 = 0; g0 < g; g0 += N) {
    Pair p[N];
    await<N>(group_words + (size_t)g0 * kLruSlab, g - g0, p);
#pragma unroll
    for (int k = 0; k < N; ++k) h = apply(p[k], h);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) h = apply(tile0[k], h);
#pragma unroll
  for (int k = 0; k < N; ++k) h = apply(tile1[k], h);
  return h;
}

// 4 neighbouring channels of a token.
template <bool BF16>
struct Raw4;
template <>
struct Raw4<true> {
  u16x4 v;
  __device__ __forceinline__ float at(int e) const { return bf16_to_f32(v[e]); }
};
template <>
struct Raw4<false> {
  f32x4 v;
  __device__ __forceinline__ float at(int e) const { return v[e]; }
};

// Channels off[t] .. off[t]+3 from `q` on of N rows, the first n of them the row's.
template <bool BF16, int N>
__device__ __forceinline__ void load_raw4(const void* q_, const uint32_t (&off)[N], int n, Raw4<BF16> (&r)[N]) {
  typedef typename std::conditional<BF16, uint16_t, float>::type T;
  typedef typename std::conditional<BF16, u16x4_any, f32x4_any>::type V;
  const T* q = static_cast<const T*>(q_);
  if (n >= 4) {
#pragma unroll
    for (int t = 0; t < N; ++t) r[t].v = *reinterpret_cast<const V*>(q + off[t]);
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[t].v[e] = e < n ? q[off[t] + e] : T(0);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_raw4(void* base, size_t elem, const float (&y)[4], int n) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(base) + elem;
    u16x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint16_t, f32_to_bf16(y[e]));
    if (n >= 4) {
      *reinterpret_cast<u16x4_any*>(q) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) q[e] = o[e];
    }
  } else {
    float* q = static_cast<float*>(base) + elem;
    if (n >= 4) {
      *reinterpret_cast<f32x4_any*>(q) = f32x4{y[0], y[1], y[2], y[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) q[e] = y[e];
    }
  }
}

}  // namespace mesa
