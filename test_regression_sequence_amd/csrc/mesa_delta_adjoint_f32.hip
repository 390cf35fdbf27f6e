// Gated delta rule, backward, fp32: the walk back over a sequence's chunks.
//
// The walk of mesa_delta_adjoint.hip for rows that are themselves three bf16 planes: six
// products where bf16 rows take three, and planes of keys and queries that fill the LDS
// (161 KB at dk = 128), so the workgroup is the four waves that hold the state.  B=3 H=4
// T=1000 dk=32 dv=64 in 8 segments of 2 chunks: 13 us, and as much to form their starts.
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
__global__ __launch_bounds__(256, 1) void delta_adjoint_f32_kernel(DeltaParams p) {
  using L = AdjointLds<DK>;
  constexpr int NP = L::NP, MT = DK / 16, KS = DK / 32;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, g = lane >> 4;
  Part part;
  if (!part_of(p, blockIdx.x, part)) return;
  const bool keep = !p.open || part.seg == p.NS - 1;  // whole: N and E go to memory
  const int bh = part.bh, b = part.b, h = part.h, hk = (uint32_t)h / p.by_shared, len = part.len, first = part.first,
            last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const int col = col0 + 16 * wave + r;
  const bool mine = 16 * wave < cols;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, o0 = b * p.d_o.b + h * p.d_o.h + col0;

  f32x4 m[MT];
  const float* const from = walk_from(p, part, p.d_sfinal, p.NS - 1);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
  }
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
  auto store = [&]() {
    kl.store(lds + L::kK, L::kPlane, tid);
    ql.store(lds + L::kQ, L::kPlane, tid);
    ol.store(lds + L::kO, 64 * 128, tid);
    tl.store(lds + L::kT, tid);
    al.store(lds + L::kA, tid);
    gl.store(lds + L::kGates, tid);
  };

  tl.clear(lds + L::kT, tid);
  al.clear(lds + L::kA, tid);
  if (first < last) {
    load(last - 1);
    store();
    __syncthreads();
  }
  for (int c = last - 1; c >= first; --c) {
    const int64_t unit = (int64_t)bh * p.NC + c;
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates);
    if (c > first) load(c - 1);

    if (mine) {
      f32x4 x[4];  // tail K N
      if (keep) {
        const Window to = window_at(p.dstates + unit * p.dv * DK);
#pragma unroll
        for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
      }
      Planes<3> mp[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          acc = mma<2>(rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * i, s, lane), mp[s], acc);
        x[i] = acc * *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
      }
      Planes<NP> of[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) of[s] = columns_of<64, NP>(lds + L::kO, 64 * 128, 32 * s, wave, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = i / 2; s < 2; ++s) x[i] = mma<2>(block_of<3>(lds + L::kA, upper_block(i, s), lane), of[s], x[i]);
      const Planes<3> px[2] = {split8<3>(x[0], x[1]), split8<3>(x[2], x[3])};
      f32x4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = i / 2; s < 2; ++s) acc = mma<2>(block_of<3>(lds + L::kT, upper_block(i, s), lane), px[s], acc);
        x[i] = acc;
      }
      if (keep) {
        const Window to = window_at(p.e + unit * 64 * p.dv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) window_store(to, (4 * g * p.dv + col) * 4, (16 * i + e) * p.dv * 4, x[i][e]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 cc = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]);
        x[i] *= -cc * *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]);
        y[i] = cc * column_values<64, NP>(lds + L::kO, 64 * 128, 16 * i, wave, lane);
      }
      const float whole = gates.c[63];
#pragma unroll
      for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Planes<3> ye = split8<3>(x[2 * s], x[2 * s + 1]), yo = split8<3>(y[2 * s], y[2 * s + 1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          m[i] = mma<2>(columns_of<DK, NP>(lds + L::kQ, L::kPlane, 32 * s, i, lane), yo, m[i]);
          m[i] = mma<2>(columns_of<DK, NP>(lds + L::kK, L::kPlane, 32 * s, i, lane), ye, m[i]);
        }
      }
    }
    __syncthreads();
    if (c > first) store();
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
  delta_adjoint_f32_kernel<DK><<<walk_blocks(p), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_adjoint_f32(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

}  // namespace mesa
