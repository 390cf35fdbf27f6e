// Gated delta rule, backward, fp32: the walk back over a sequence's chunks.
//
// The walk of mesa_delta_adjoint.hip for rows that are themselves three bf16 planes: six
// products where bf16 rows take three.  Four waves hold the state; the LDS has room for one
// chunk's planes (161 KB at dk = 128), so four more load the next chunk and split its rows
// in registers meanwhile, and between the two barriers only write them.  The state's waves
// alone, with the splits between the barriers, took 2 to 7 % more for all gradients: 16
// heads of 4096 tokens, dk = dv = 128, 501 us, so 469; 14 heads of 333, 32, 67 and 63.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK>
struct AdjointLds {
  static constexpr int NP = 3;
  static constexpr int kPlane = 64 * DK * 2;
  static constexpr int kK = 0, kQ = kK + NP * kPlane, kO = kQ + NP * kPlane, kT = kO + NP * 64 * 128,
                       kA = kT + 3 * kBlocksBytes, kGates = kA + 3 * kBlocksBytes, kBytes = kGates + sizeof(DeltaGates);
};

template <int DK>
__global__ __launch_bounds__(512, 2) void delta_adjoint_f32_kernel(DeltaParams p) {
  using L = AdjointLds<DK>;
  constexpr int NP = L::NP, MT = DK / 16, KS = DK / 32;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const int tid = threadIdx.x & 255, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15,
            g = lane >> 4;
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x) < 256;
  Part part;
  if (!part_of(p, blockIdx.x, part)) return;
  const bool keep = !p.open || part.seg == p.NS - 1;  // whole: N and E go to memory
  const int bh = part.bh, b = part.b, h = part.h, hk = (uint32_t)h / p.by_shared, len = part.len, first = part.first,
            last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const int col = col0 + 16 * wave + r;
  const bool mine = 16 * wave < cols;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, o0 = b * p.d_o.b + h * p.d_o.h + col0;

  if (!chain) {
    RowLoads<DK, false, 256> kl, ql;
    RowLoads<64, false, 256> ol;
    TriangleLoads<3, false, 256> tl, al;
    CopyLoads<sizeof(DeltaGates), 256> gl;
    auto load = [&](int c) {
      const int live = min(len - 64 * c, 64);
      const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
      kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
      ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live, DK, tid);
      ol.load(p.d_o.at, o0 + t0 * p.d_o.t, p.d_o.t, live, cols, tid);
      tl.load(p.matrices_t + unit * (2 * kTriangleBytes), tid);
      al.load(p.matrices_t + unit * (2 * kTriangleBytes) + kTriangleBytes, tid);
      gl.load(p.gates + unit, tid);
    };
    tl.clear(lds + L::kT, tid);
    al.clear(lds + L::kA, tid);
    if (first < last) {
      load(last - 1);
      kl.store(lds + L::kK, L::kPlane, tid);
      ql.store(lds + L::kQ, L::kPlane, tid);
      ol.store(lds + L::kO, 64 * 128, tid);
      tl.store(lds + L::kT, tid);
      al.store(lds + L::kA, tid);
      gl.store(lds + L::kGates, tid);
    }
    __syncthreads();
    for (int c = last - 1; c >= first; --c) {  // (no branch around the loads: the first chunk is loaded once more)
      load(max(c - 1, first));
      const RowPlanes<DK, 256> kp(kl), qp(ql);
      const RowPlanes<64, 256> op(ol);
      tl.split();
      al.split();
      fence<true>();
      __syncthreads();
      kp.store(lds + L::kK, L::kPlane, tid);
      qp.store(lds + L::kQ, L::kPlane, tid);
      op.store(lds + L::kO, 64 * 128, tid);
      tl.put(lds + L::kT, tid);
      al.put(lds + L::kA, tid);
      gl.store(lds + L::kGates, tid);
      __syncthreads();
    }
    return;
  }

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 m[MT];
  const float* const from = walk_from(p, part, p.d_sfinal, p.NS - 1);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = zero;
    if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
  }
  __syncthreads();
  for (int c = last - 1; c >= first; --c) {
    const int64_t unit = (int64_t)bh * p.NC + c;
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates);

    if (mine) {
      if (keep) {
        const Window to = window_at(p.dstates + unit * p.dv * DK);
#pragma unroll
        for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
      }
      constexpr bool AHEAD = DK < 128;  // (at 128 it takes 20 registers through scratch, and 470 us become 516)
      Planes<3> mp[2], px[2], py[2];
      Planes<NP> f[2][4], of[2];
      BlockPair<3> a, t;
      f32x4 x[4] = {zero, zero, zero, zero}, y[4];
      auto rows = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[s & 1][i] = rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * i, s, lane);
      };
      rows(0);
      mp[0] = split8<3>(m[0], m[1]);
#pragma unroll
      for (int s = 0; s < KS; ++s) {  // tail K N
        if (s + 1 < KS) {
          if (AHEAD) rows(s + 1);
          mp[(s + 1) & 1] = split8<3>(m[2 * s + 2], m[2 * s + 3]);
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n) of[n] = columns_of<64, NP>(lds + L::kO, 64 * 128, 32 * n, wave, lane);
          a = pair_of<false, 3>(lds + L::kA, 0, lane);
        }
        if (!AHEAD && s) rows(s);
        mma_tiles<2>(f[s & 1], mp[s & 1], x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
        y[i] = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) *
               column_values<64, NP>(lds + L::kO, 64 * 128, 16 * i, wave, lane);
      }
      mma_triangle<2, false, false, false>(lds + L::kA, a, of, x, lane);  // dU
      t = pair_of<false, 3>(lds + L::kT, 0, lane);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        px[s] = split8<3>(x[2 * s], x[2 * s + 1]);
        py[s] = split8<3>(y[2 * s], y[2 * s + 1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = zero;
      mma_triangle<2, false, false, false>(lds + L::kT, t, px, x, lane);  // E
      constexpr int G = DK == 64 ? 4 : 2, NG = 4 * MT / G;  // Q^T, then K^T, in groups of tiles, fewer where registers end
      Planes<NP> kt[2][G];
      auto group = [&](int n) {
        const int k = n % (NG / 2) * G;
#pragma unroll
        for (int i = 0; i < G; ++i)
          kt[n & 1][i] = columns_of<DK, NP>(lds + (n < NG / 2 ? L::kQ : L::kK), L::kPlane, 32 * (k / MT), k % MT + i, lane);
      };
      group(0);
      if (keep) {
        const Window to = window_at(p.e + unit * 64 * p.dv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) window_store(to, (4 * g * p.dv + col) * 4, (16 * i + e) * p.dv * 4, x[i][e]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] *= -(*reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) *
                  *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]));
      const float whole = gates.c[63];
#pragma unroll
      for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) px[s] = split8<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if (n + 1 < NG) group(n + 1);
        const int k = n % (NG / 2) * G;
        const Planes<3>& by = n < NG / 2 ? py[k / MT] : px[k / MT];
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int q = 0; q < NP; ++q)
            if (sum - q >= 0)
#pragma unroll
              for (int i = 0; i < G; ++i) m[k % MT + i] = mfma_bf16(kt[n & 1][i].p[q], by.p[sum - q], m[k % MT + i]);
      }
    }
    __syncthreads();  // (the next chunk's LDS)
    __syncthreads();
  }

  float* const to = walk_to(p, part, p.ds0, 0);
  if (mine && to) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + col * DK + 16 * i + 4 * g) = m[i];
  }
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  delta_adjoint_f32_kernel<DK><<<walk_blocks(p), 512, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_adjoint_f32(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

}  // namespace mesa
