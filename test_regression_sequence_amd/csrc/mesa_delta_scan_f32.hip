// Gated delta rule, forward, fp32: the walk over a sequence's chunks.
//
// The walk of mesa_delta_scan.hip for rows that are themselves three bf16 planes: six
// products where bf16 rows take three, and planes of keys and queries that fill the
// LDS (161 KB at dk = 128), so the workgroup is the four waves that hold the state, and
// each forms its columns of o too.  A chunk takes 5.7 us at dk = 64: 216 products (1.5 us) and,
// between its barriers, the conversions of the next chunk's rows, which nothing hides
// (B=5 H=6 T=777 dk=64 dv=96: 73 us in one walk, in 4 segments 25 us and 26 to form them).
#include "mesa_delta_probe.h"

namespace mesa {

namespace {

template <int DK>
struct ScanLds {
  static constexpr int NP = 3, NA = 3;
  static constexpr int kPlane = 64 * DK * 2, kMatrices = (int)delta_matrix_bytes(NA);
  static constexpr int kK = 0, kQ = kK + NP * kPlane, kV = kQ + NP * kPlane, kT = kV + NP * 64 * 128,
                       kA = kT + 3 * kBlocksBytes, kGates = kT + kMatrices, kBytes = kGates + sizeof(DeltaGates);
};

template <int DK, bool OUT>
__global__ __launch_bounds__(256, 1) void delta_scan_f32_kernel(DeltaParams p) {
  using L = ScanLds<DK>;
  constexpr int NP = L::NP, NA = L::NA, MT = DK / 16, KS = DK / 32;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, g = lane >> 4;
  Part part;
  if (!part_of(p, blockIdx.x, part)) return;
  const int bh = part.bh, b = part.b, h = part.h, hk = (uint32_t)h / p.by_shared, len = part.len, first = part.first,
            last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const int col = col0 + 16 * wave + r;                 // this lane's column of the state
  const bool mine = 16 * wave < cols;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h + col0,
                o0 = b * p.o.b + h * p.o.h + col0 + 16 * wave;

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 m[MT];  // rows 16 i + 4 g + e of M, column `col`
  const float* const from = walk_from(p, part, p.s0, 0);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = zero;
    if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
  }
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
  auto store = [&]() {
    kl.store(lds + L::kK, L::kPlane, tid);
    if constexpr (OUT) ql.store(lds + L::kQ, L::kPlane, tid);
    vl.store(lds + L::kV, 64 * 128, tid);
    ml.store(lds + L::kT, tid);
    gl.store(lds + L::kGates, tid);
  };

  if (first < last) {
    load(first);
    store();
    __syncthreads();
  }
  for (int c = first; c < last; ++c) {
    const int64_t unit = (int64_t)bh * p.NC + c;
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates);
    if (c + 1 < last) load(c + 1);
    f32x4 o[4] = {zero, zero, zero, zero};

    if (mine) {
      if (p.states) {
        const Window to = window_at(p.states + unit * p.dv * DK);
#pragma unroll
        for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
      }
      Planes<3> mp[KS], u[2], ut[2], px[2];
      BlockPair<3> t;
      BlockPair<NA> a;
      Planes<NP> f[2][4];
      f32x4 x[4] = {zero, zero, zero, zero}, y[4] = {zero, zero, zero, zero};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[0][i] = rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * i, 0, lane);
      mp[0] = split8<3>(m[0], m[1]);
#pragma unroll
      for (int s = 0; s < KS; ++s) {  // x = K M
        if (s + 1 < KS) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * i, s + 1, lane);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = column_values<64, NP>(lds + L::kV, 64 * 128, 16 * i, wave, lane);
          if constexpr (OUT)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows_of<DK, NP>(lds + L::kQ, L::kPlane, 16 * i, 0, lane);
        }
        if (s + 1 < KS) mp[s + 1] = split8<3>(m[2 * s + 2], m[2 * s + 3]);
        mma_tiles<2>(f[s & 1], mp[s], x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = y[i] - *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) * x[i];
      px[0] = split8<3>(x[0], x[1]);
      px[1] = split8<3>(x[2], x[3]);
      if constexpr (OUT) {  // o's transpose, a lane has 4 columns of one token: first Q M
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (s + 1 < KS) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              f[(KS + s + 1) & 1][i] = rows_of<DK, NP>(lds + L::kQ, L::kPlane, 16 * i, s + 1, lane);
          } else {
            t = pair_of<true, 3>(lds + L::kT, 0, lane);
          }
          mma_tiles_t<2>(mp[s], f[(KS + s) & 1], o);
        }
      } else {
        t = pair_of<true, 3>(lds + L::kT, 0, lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = zero;
      mma_triangle<2, true, false, false>(lds + L::kT, t, px, x, lane);  // W
      Planes<NP> kt[2][4];
      constexpr int G = MT < 4 ? MT : 4, NG = 2 * MT / G;  // K^T in groups of 4 tiles
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
        else if constexpr (OUT) a = pair_of<true, NA>(lds + L::kA, 0, lane);
        if (OUT && n == 0) {
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
    if (c + 1 < last) store();  // (ahead of o's stores, which then have the next chunk's time)
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

template <int DK>
__global__ __launch_bounds__(512, 2) void delta_open_f32_kernel(DeltaParams p, Divisor by_part, Divisor by_slices) {
  __shared__ __attribute__((aligned(16))) char lds[2 * ProbeLds<DK, false>::kBuffer];
  probe_segment<DK, false>(p, blockIdx.x, 0, by_part, by_slices, lds);
}

template <int DK>
hipError_t open(const DeltaParams& p, hipStream_t s) {
  const uint32_t slices = probe_slices(p);
  delta_open_f32_kernel<DK><<<probe_blocks(p, 0), 512, 0, s>>>(p, divisor(slices * (p.NS - 1)), divisor(slices));
  return hipGetLastError();
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  if (p.o.at) delta_scan_f32_kernel<DK, true><<<walk_blocks(p), 256, 0, s>>>(p);
  else delta_scan_f32_kernel<DK, false><<<walk_blocks(p), 256, 0, s>>>(p);
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
