// Gated delta rule, forward, fp32: the walk over a sequence's chunks.
//
// The walk of mesa_delta_scan.hip for rows that are themselves three bf16 planes: six
// products where bf16 rows take three.  Four waves hold the state; they form K M and Q M
// in turn, so that planes of only two parts of the state live at a time.  The LDS has room
// for one chunk's planes (161 KB at dk = 128): four more waves load the next chunk and
// split its rows in registers meanwhile, and between the two barriers only write them.
// The state's waves alone, with the splits between the barriers, took 5.7 us a chunk at
// dk = 64, so it takes 4.4, of which 216 products are 1.5 (B=5 H=6 T=777 dk=64 dv=96 in 4
// segments: 18 to 19 us for the first segment and the openings of the others, 17 for the rest).
#include <algorithm>

#include "mesa_delta_probe.h"

namespace mesa {

namespace {

template <int DK>
struct ScanLds {
  static constexpr int NP = 3;
  static constexpr int kPlane = 64 * DK * 2, kMatrices = (int)delta_matrix_bytes(false);
  static constexpr int kK = 0, kQ = kK + NP * kPlane, kV = kQ + NP * kPlane, kT = kV + NP * 64 * 128,
                       kA = kT + 3 * kBlocksBytes, kGates = kT + kMatrices, kBytes = kGates + sizeof(DeltaGates);
};

template <int DK, bool OUT>
__device__ __forceinline__ void walk_segment(const DeltaParams& p, uint32_t id, char* lds) {
  using L = ScanLds<DK>;
  constexpr int NP = L::NP, MT = DK / 16, KS = DK / 32;
  const int tid = threadIdx.x & 255, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15,
            g = lane >> 4;
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x) < 256;
  Part part;
  if (!part_of(p, id, part)) return;
  const int bh = part.bh, b = part.b, h = part.h, hk = (uint32_t)h / p.by_shared, len = part.len, first = part.first,
            last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const int col = col0 + 16 * wave + r;                 // this lane's column of the state
  const bool mine = 16 * wave < cols;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h + col0,
                o0 = b * p.o.b + h * p.o.h + col0 + 16 * wave;

  if (!chain) {
    RowLoads<DK, false, 256> kl, ql;
    RowLoads<64, false, 256> vl;
    CopyLoads<L::kMatrices, 256> ml;
    CopyLoads<sizeof(DeltaGates), 256> gl;
    auto load = [&](int c) {
      const int live = min(len - 64 * c, 64);
      const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
      kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
      if constexpr (OUT) ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live, DK, tid);
      vl.load(p.v.at, v0 + t0 * p.v.t, p.v.t, live, cols, tid);
      ml.load(p.matrices + unit * L::kMatrices, tid);
      gl.load(p.gates + unit, tid);
    };
    if (first < last) {
      load(first);
      kl.store(lds + L::kK, L::kPlane, tid);
      if constexpr (OUT) ql.store(lds + L::kQ, L::kPlane, tid);
      vl.store(lds + L::kV, 64 * 128, tid);
      ml.store(lds + L::kT, tid);
      gl.store(lds + L::kGates, tid);
    }
    __syncthreads();
    for (int c = first; c < last; ++c) {  // (no branch around the loads: the last chunk is loaded once more)
      load(min(c + 1, last - 1));
      const RowPlanes<DK, 256> kp(kl), qp(OUT ? ql : kl);
      const RowPlanes<64, 256> vp(vl);
      fence<true>();
      __syncthreads();
      kp.store(lds + L::kK, L::kPlane, tid);
      if constexpr (OUT) qp.store(lds + L::kQ, L::kPlane, tid);
      vp.store(lds + L::kV, 64 * 128, tid);
      ml.store(lds + L::kT, tid);
      gl.store(lds + L::kGates, tid);
      __syncthreads();
    }
    return;
  }

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 m[MT];  // rows 16 i + 4 g + e of M, column `col`
  const float* const from = walk_from(p, part, p.s0, 0);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = zero;
    if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
  }
  __syncthreads();
  for (int c = first; c < last; ++c) {
    const int64_t unit = (int64_t)bh * p.NC + c;
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates);
    f32x4 o[4] = {zero, zero, zero, zero};

    if (mine) {
      if (p.states) {
        const Window to = window_at(p.states + unit * p.dv * DK);
#pragma unroll
        for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
      }
      Planes<3> mp[2], u[2], ut[2], px[2];
      BlockPair<3> t;
      BlockPair<3> a;
      Planes<NP> f[2][4];
      f32x4 x[4] = {zero, zero, zero, zero}, y[4] = {zero, zero, zero, zero};
      constexpr int E = OUT ? 2 : 1;
      auto rows = [&](int n) {  // the keys' rows, and the queries', of a part of the state
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[n & 1][i] = rows_of<DK, NP>(lds + (n % E ? L::kQ : L::kK), L::kPlane, 16 * i, n / E, lane);
      };
      rows(0);
      mp[0] = split8<3>(m[0], m[1]);
#pragma unroll
      for (int n = 0; n < E * KS; ++n) {  // x = K M, and o's transpose, a lane has 4 columns of one token: first Q M
        if (n + 1 < E * KS) rows(n + 1);
        else t = pair_of<true, 3>(lds + L::kT, 0, lane);
        if (n == E * (KS - 1))
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = column_values<64, NP>(lds + L::kV, 64 * 128, 16 * i, wave, lane);
        const int s = n / E;
        if (n % E == 0 && s + 1 < KS) mp[(s + 1) & 1] = split8<3>(m[2 * s + 2], m[2 * s + 3]);
        if (n % E) mma_tiles_t<2>(mp[s & 1], f[n & 1], o);
        else mma_tiles<2>(f[n & 1], mp[s & 1], x);
        if (n == E * (KS - 1)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = y[i] - *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) * x[i];
          px[0] = split8<3>(x[0], x[1]);
          px[1] = split8<3>(x[2], x[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = zero;
      mma_triangle<2, true, false, false>(lds + L::kT, t, px, x, lane);  // W
      Planes<NP> kt[2][4];
      // K^T in groups of tiles (at dk = 128 four a group take 22 registers through scratch: 256 heads of
      // 1024 tokens 346 us, so 316)
      constexpr int G = DK == 64 ? 4 : 2, NG = 2 * MT / G;
      auto keys = [&](int n, Planes<NP> (&to)[4]) {
#pragma unroll
        for (int i = 0; i < G; ++i)
          to[i] = columns_of<DK, NP>(lds + L::kK, L::kPlane, 32 * (n * G / MT), n * G % MT + i, lane);
      };
      keys(0, kt[0]);
      if (p.w) {
        const Window to = window_at(p.w + unit * 64 * p.dv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) window_store(to, (4 * g * p.dv + col) * 4, (16 * i + e) * p.dv * 4, x[i][e]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]);
        y[i] = x[i] * *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
      }
      const float whole = gates.c[63];
#pragma unroll
      for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) ut[s] = split8<3>(y[2 * s], y[2 * s + 1]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {  // M += K^T U
        if (n + 1 < NG) keys(n + 1, kt[(n + 1) & 1]);
        else if constexpr (OUT) a = pair_of<true, 3>(lds + L::kA, 0, lane);
        if (OUT && n == NG - 1) {
#pragma unroll
          for (int s = 0; s < 2; ++s) u[s] = split8<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] *= gates.c[16 * i + r];
        }
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int q = 0; q < NP; ++q)
            if (sum - q >= 0)
#pragma unroll
              for (int i = 0; i < G; ++i)
                m[n * G % MT + i] = mfma_bf16(kt[n & 1][i].p[q], ut[n * G / MT].p[sum - q], m[n * G % MT + i]);
      }
      if constexpr (OUT) {
        mma_triangle<2, true, true, false>(lds + L::kA, a, u, o, lane);
      }
    }
    __syncthreads();
    if (OUT && mine) {
      const int live = len - 64 * c;
      const Window to = window_at(static_cast<float*>(p.o.at) + o0 + 64 * (int64_t)c * p.o.t);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        window_store(to, 16 * i + r < live ? ((16 * i + r) * (uint32_t)p.o.t + 4 * g) * 4 : kNowhere, 0, o[i]);
    }
    __syncthreads();
  }

  float* const to = walk_to(p, part, p.s_final, p.NS - 1);
  if (mine && to) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + col * DK + 16 * i + 4 * g) = m[i];
  }
  if (OUT && mine) {  // behind the sequence
    const int end = (int)min((int64_t)p.T, (int64_t)64 * (first + p.L));
    for (int64_t t = max(len, 64 * first) + r; t < end; t += 16) {
      store_out4<float>(p.o.at, o0 + t * p.o.t + 4 * g, zero);
    }
  }
}

template <int DK, bool OUT>
__global__ __launch_bounds__(512, 2) void delta_scan_f32_kernel(DeltaParams p) {
  __shared__ __attribute__((aligned(16))) char lds[ScanLds<DK>::kBytes];
  walk_segment<DK, OUT>(p, blockIdx.x, lds);
}

// The first segment whole, and what the others but the last make of states, side by side.
template <int DK, bool OUT>
__global__ __launch_bounds__(512, 2) void delta_open_f32_kernel(DeltaParams p, uint32_t probes, Divisor by_part,
                                                                Divisor by_slices) {
  __shared__ __attribute__((aligned(16))) char lds[std::max(ScanLds<DK>::kBytes, 2 * ProbeLds<DK, false>::kBuffer)];
  if (blockIdx.x < probes) probe_segment<DK, false>(p, blockIdx.x, by_part, by_slices, lds);
  else walk_segment<DK, OUT>(p, blockIdx.x - probes, lds);
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  if (p.o.at) delta_scan_f32_kernel<DK, true><<<walk_blocks(p), 512, 0, s>>>(p);
  else delta_scan_f32_kernel<DK, false><<<walk_blocks(p), 512, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK>
hipError_t open(const DeltaParams& p, hipStream_t s) {
  const uint32_t probes = probe_blocks(p), blocks = probes + walk_blocks(p);
  if (p.o.at) delta_open_f32_kernel<DK, true><<<blocks, 512, 0, s>>>(p, probes, probe_part(p), divisor(probe_slices(p)));
  else delta_open_f32_kernel<DK, false><<<blocks, 512, 0, s>>>(p, probes, probe_part(p), divisor(probe_slices(p)));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan_f32(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

hipError_t launch_delta_open_f32(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? open<128>(p, s) : p.dk == 64 ? open<64>(p, s) : open<32>(p, s);
}

}  // namespace mesa
