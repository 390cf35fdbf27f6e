// Gated delta rule, forward: what the segments of a split walk make of states.
//
// Over a segment the state's rows go S -> S P + Q.  The walk of mesa_delta_scan.hip,
// without outputs, over Q's columns, from zero, and over P's: the dk unit columns, whose
// values are zeros.  The first segment, which needs no start, runs whole beside it, and
// nothing follows the last.
//
// Nothing is formed beside the chain of states, so all eight waves are chains, 16
// columns each, two on a SIMD to fill one another's waits: 128 columns a workgroup, and
// with dv = dk = 64 both kinds in one.  A chunk's keys, inverse and gates go to LDS
// while the chunk before is in the works; so do values of two bytes, those of four, whose
// planes would not fit beside two chunks of keys, go to their lanes.
//
// B=1 H=16 T=32768 d=128: 4.8 to 5.3 us a chunk and 128 columns, of which a SIMD's matrix unit
// works 40 % and its vector unit 42 %, hardly at the same time (four chains of 16 columns as
// in the walk itself: 2.7 us for 64 columns).  The two waves of a SIMD half a chunk apart,
// so that conversions of one meet products of the other, took a tenth longer: the second
// barrier a chunk costs more.  The first segment's walk in the same launch: 9 segments in
// place of 8 on 256 CUs, 536 -> 493 us for both launches of the walk.
#pragma once

#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK, bool BF16>
struct ProbeLds {
  static constexpr int NP = BF16 ? 1 : 3, kPlane = 64 * DK * 2;
  static constexpr int kT = NP * kPlane, kGates = kT + 3 * kBlocksBytes, kV = kGates + (int)sizeof(DeltaGates),
                       kBuffer = kV + (BF16 ? 64 * 256 : 0);
};

// Workgroups of a head's segment, and of the segments between the first and the last.
inline uint32_t probe_slices(const DeltaParams& p) { return (uint32_t)(p.dv + p.dk + 127) / 128; }
inline uint32_t probe_blocks(const DeltaParams& p) {
  return (uint32_t)((p.B * p.H + 7) / 8 * 8) * probe_slices(p) * (uint32_t)(p.NS - 2);
}
inline Divisor probe_part(const DeltaParams& p) { return divisor(probe_slices(p) * (uint32_t)(p.NS > 2 ? p.NS - 2 : 1)); }

// Workgroup `id` of them (by_part: of a head, by_slices: of those the ones of a segment).
template <int DK, bool BF16>
__device__ __forceinline__ void probe_segment(const DeltaParams& p, uint32_t id, const Divisor& by_part,
                                              const Divisor& by_slices, char* all) {
  using L = ProbeLds<DK, BF16>;
  constexpr int NP = L::NP, MT = DK / 16, KS = DK / 32;
  char (*const lds)[L::kBuffer] = reinterpret_cast<char (*)[L::kBuffer]>(all);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, g = lane >> 4;
  // one head's workgroups on one XCD, whose L2 they share
  const uint32_t n = id >> 3, rest = n % by_part;
  const int bh = n / by_part * 8 + (id & 7), seg = 1 + rest / by_slices, slice = rest % by_slices;
  if (bh >= p.B * p.H) return;
  const int b = (uint32_t)bh / p.by_h, h = (uint32_t)bh % p.by_h, hk = (uint32_t)h / p.by_shared, len = delta_length(p, b);
  const int first = seg * p.L, last = max(min((len + 63) / 64, first + p.L), first);
  const int col0 = 128 * slice + 16 * wave;
  const bool unit_columns = col0 >= p.dv, mine = col0 < p.dv + DK;
  const int col = (unit_columns ? col0 - p.dv : col0) + r;
  const int64_t k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  f32x4 m[MT];  // rows 16 i + 4 g + e of the state's transpose, column `col`
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = zero;
    if (unit_columns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) m[i][e] = 16 * i + 4 * g + e == col ? 1.f : 0.f;
    }
  }
  const TileRows<DK> rows(lane);
  const TileColumns<DK> columns(lane);
  RowLoads<DK, BF16, 512> kl;
  CopyLoads<3 * kBlocksBytes, 512> tl;
  CopyLoads<sizeof(DeltaGates), 512> gl;
  RowLoads<128, true, 512> vl;
  f32x4 v[4], v_next[4];  // V's rows 16 i + 4 g + e, column `col`
  auto load = [&](int c) {
    const int live = min(len - 64 * c, 64);
    const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
    kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
    tl.load(p.matrices + unit * (int64_t)delta_matrix_bytes(BF16), tid);
    gl.load(p.gates + unit, tid);
    if constexpr (BF16) {
      vl.load(p.v.at, v0 + 128 * slice + t0 * p.v.t, p.v.t, live, p.dv - 128 * slice, tid);
    } else {
      const Window from = window_at(static_cast<const float*>(p.v.at) + v0 + t0 * p.v.t);
      const uint32_t at = (4 * g * (uint32_t)p.v.t + col) * 4, step = (uint32_t)p.v.t * 4;
      const int there = unit_columns ? 0 : live - 4 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v_next[i][e] = window_number(from, 16 * i + e < there ? at : kNowhere, (16 * i + e) * step);
    }
  };
  auto store = [&](int c) {
    char* to = lds[c & 1];
    kl.store(to, L::kPlane, tid);
    tl.store(to + L::kT, tid);
    gl.store(to + L::kGates, tid);
    if constexpr (BF16) vl.store(to + L::kV, 0, tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = v_next[i];
  };

  if (first < last) {
    load(first);
    store(first);
    __syncthreads();
  }
  for (int c = first; c < last; ++c) {
    const char* keys = lds[c & 1];
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(keys + L::kGates);
    load(min(c + 1, last - 1));  // (without a branch around the loads)
    if (mine) {
      f32x4 x[4] = {zero, zero, zero, zero}, y[4];
      Planes<3> mp[KS], px[2], ut[2];
      Planes<NP> f[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[0][i] = rows.template planes<NP>(keys, L::kPlane, 16 * i, 0);
#pragma unroll
      for (int s = 0; s < KS; ++s) mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
      BlockPair<3> t;
#pragma unroll
      for (int s = 0; s < KS; ++s) {  // K M
        if (s + 1 < KS) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows.template planes<NP>(keys, L::kPlane, 16 * i, s + 1);
        } else {
          t = pair_of<true, 3>(keys + L::kT, 0, lane);
          if constexpr (BF16)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = column_values<128, 1>(keys + L::kV, 0, 16 * i, wave, lane);
        }
        fence<BF16>();
        mma_tiles<2>(f[s & 1], mp[s], x);
        fence<BF16>();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = v[i] - *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) * x[i];
        x[i] = zero;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) px[s] = split8<3>(y[2 * s], y[2 * s + 1]);
      mma_triangle<2, true, false, BF16>(keys + L::kT, t, px, x, lane);  // W
      constexpr int G = MT < 4 ? MT : 4, NG = 2 * MT / G;  // K^T in groups of 4 tiles
      Planes<NP> kt[2][4];
      auto group = [&](int n) {
#pragma unroll
        for (int i = 0; i < G; ++i)
          kt[n & 1][i] = columns.template planes<NP>(keys, L::kPlane, 32 * (n * G / MT), n * G % MT + i);
      };
      group(0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] *= *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]) *
                *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
      const float whole = gates.c[63];
#pragma unroll
      for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) ut[s] = split8<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {  // M += K^T U
        if (n + 1 < NG) group(n + 1);
        fence<BF16>();
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int q = 0; q < NP; ++q)
            if (sum - q >= 0)
#pragma unroll
              for (int i = 0; i < G; ++i)
                m[n * G % MT + i] = mfma_bf16(kt[n & 1][i].p[q], ut[n * G / MT].p[sum - q], m[n * G % MT + i]);
        fence<BF16>();
      }
    }
    store(c + 1);
    __syncthreads();
  }
  if (mine) {
    const int64_t at = (int64_t)bh * p.NS + seg;
    float* const to = unit_columns ? p.seg_map + (at * DK + col) * DK : p.seg_add + (at * p.dv + col) * DK;
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + 16 * i + 4 * g) = m[i];
  }
}

}  // namespace

}  // namespace mesa
