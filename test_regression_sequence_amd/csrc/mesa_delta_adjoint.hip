// Gated delta rule, backward: the walk back over a sequence's chunks (bf16 rows).
//
// As in the forward walk a wave holds 16 columns (value dimensions) of the
// adjoint state's transpose N [dk, dv], the gradient at the state behind a chunk.
// From the last chunk to the first
//     dU = A^T dO + diag(c_C / c) K N,   E = T^T dU,
//     N <- c_C N + Q^T (c dO) - K^T (c beta E),
// T = (I + diag(beta) X)^-1, A = lower(D Q K^T), transposed by mesa_delta_chunk.hip.
// N behind each chunk and E (dv = beta E) go to memory for the gradients of the
// chunks, which are then independent.  All products in three bf16 planes: the gates'
// gradients are fp32.
//
// Four waves hold N; four more, one beside each on its SIMD, take what does not depend
// on N, and pass it through LDS:
//     first half:   chain K N, E, half of K^T E     others Q^T (c dO), loads
//     second half:  chain the rest, N, its planes   others A^T dO of the next chunk, loads
//
// Memory bounds it: at B=8 H=16 T=4096 d=128 312 to 319 us for 1.4 GB, 4.4 TB/s where a large copy
// reaches 4.9; the chain itself takes about 3 us a chunk.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK>
struct AdjointLds {
  static constexpr int kTile = 64 * DK * 2, kGate = sizeof(DeltaGates);
  static constexpr int kK = 0, kQ = kK + 2 * kTile, kO = kQ + kTile, kT = kO + 2 * 64 * 128, kA = kT + 3 * kBlocksBytes,
                       kGates = kA + 3 * kBlocksBytes, kU = kGates + 2 * kGate, kN = kU + 4 * 4096,
                       kBytes = kN + 4 * DK * 64;
};

template <int DK>
__global__ __launch_bounds__(512, 2) void delta_adjoint_kernel(DeltaParams p) {
  using L = AdjointLds<DK>;
  constexpr int MT = DK / 16, KS = DK / 32;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const int tid = threadIdx.x & 255, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15,
            g = lane >> 4;
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x) < 256;
  Part part;
  if (!part_of(p, blockIdx.x, part)) return;
  const bool keep = !p.open || part.seg == p.NS - 1;  // whole: N and E go to memory
  const int bh = part.bh, b = part.b, h = part.h, len = part.len, first = part.first, last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const bool mine = 16 * wave < cols;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  char* const u_at = lds + L::kU + wave * 4096 + lane * 16;     // A^T dO: four tiles
  char* const n_at = lds + L::kN + wave * DK * 64 + lane * 16;  // Q^T (c dO): DK / 16 tiles
  const TileColumns<DK> columns(lane);
  constexpr int G = MT < 4 ? MT : 4, NG = 2 * MT / G;  // columns of Q or K in groups of 4 tiles, tokens 32 .. 63 first

  if (chain) {
    const int col = col0 + 16 * wave + r;
    f32x4 m[MT];
    const float* const from = walk_from(p, part, p.d_sfinal, p.NS - 1);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      m[i] = zero;
      if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
    }
    const TileRows<DK> rows(lane);
    Planes<3> mp[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
    __builtin_amdgcn_s_setprio(2);
    __syncthreads();
    __syncthreads();
    for (int c = last - 1; c >= first; --c) {
      const char* keys = lds + L::kK + (c & 1) * L::kTile;
      const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
      const int64_t unit = (int64_t)bh * p.NC + c;
      f32x4 x[4] = {zero, zero, zero, zero}, y[4], cc[4], cb[4];
      Planes<3> px[2], pe[2];
      Planes<1> f[2][4], kt[2][4];
      BlockPair<3> t[2];
      auto group = [&](int n, Planes<1> (&to)[4]) {
#pragma unroll
        for (int i = 0; i < G; ++i) to[i] = columns(keys, 32 * (1 - n * G / MT), n * G % MT + i);
      };
      auto mma_group = [&](int n) {
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
          for (int i = 0; i < G; ++i)
            m[n * G % MT + i] = mfma_bf16(kt[n & 1][i].p[0], pe[1 - n * G / MT].p[q], m[n * G % MT + i]);
      };
      if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[0][i] = rows(keys, 16 * i, 0);
#pragma unroll
        for (int s = 0; s < KS; ++s) {  // x = K N
          if (s + 1 < KS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows(keys, 16 * i, s + 1);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[i] = *reinterpret_cast<const f32x4*>(u_at + i * 1024);
              cc[i] = *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
            }
            t[0] = pair_of<false, 3>(lds + L::kT, 2, lane);
          }
          fence<true>();
          mma_tiles<2>(f[s & 1], mp[s], x);
          fence<true>();
        }
        if (keep) {
          const Window to = window_at(p.dstates + unit * p.dv * DK);
#pragma unroll
          for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
        }
        t[1] = pair_of<false, 3>(lds + L::kT, 1, lane);
        auto total = [&](int s) {  // dU
#pragma unroll
          for (int i = 2 * s; i < 2 * s + 2; ++i) {
            y[i] += cc[i] * x[i];
            x[i] = zero;
          }
          px[s] = split8<3>(y[2 * s], y[2 * s + 1]);
        };
        auto scale_of = [&](int s) {
#pragma unroll
          for (int i = 2 * s; i < 2 * s + 2; ++i) {
            cc[i] = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]);
            cb[i] = *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]);
          }
        };
        auto scaled = [&](int s) {  // E, and -c beta E
          const Window to = window_at(p.e + unit * 64 * p.dv);
#pragma unroll
          for (int i = 2 * s; i < 2 * s + 2; ++i) {
            if (keep)
#pragma unroll
              for (int e = 0; e < 4; ++e) window_store(to, (4 * g * p.dv + col) * 4, (16 * i + e) * p.dv * 4, x[i][e]);
            y[i] = -(cc[i] * cb[i]) * x[i];
          }
          pe[s] = split8<3>(y[2 * s], y[2 * s + 1]);
        };
        total(1);
        fence<true>();
        total(0);
        mma_pair<2, false, false>(2, t[0], px, x);  // rows 32 .. 63 of E
        t[0] = pair_of<false, 3>(lds + L::kT, 0, lane);
        scale_of(1);
        group(0, kt[0]);
        const float whole = gates.c[63];
        fence<true>();
        scaled(1);
        mma_pair<2, false, false>(1, t[1], px, x);
        scale_of(0);
        fence<true>();
        mma_pair<2, false, false>(0, t[0], px, x);
#pragma unroll
        for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
        for (int n = 0; n < NG / 2; ++n) {
          group(n + 1, kt[(n + 1) & 1]);
          fence<true>();
          mma_group(n);
        }
        scaled(0);
      }
      __syncthreads();
      if (mine) {
        f32x4 add[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) add[i] = *reinterpret_cast<const f32x4*>(n_at + i * 1024);
#pragma unroll
        for (int n = NG / 2; n < NG; ++n) {
          if (n + 1 < NG) group(n + 1, kt[(n + 1) & 1]);
          fence<true>();
          mma_group(n);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) m[i] += add[i];
#pragma unroll
        for (int s = 0; s < KS; ++s) mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
      }
      __syncthreads();
    }
    float* const to = walk_to(p, part, p.ds0, 0);
    if (mine && to) {
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + col * DK + 16 * i + 4 * g) = m[i];
    }
    return;
  }

  const int hk = (uint32_t)h / p.by_shared;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, o0 = b * p.d_o.b + h * p.d_o.h + col0;
  RowLoads<DK, true, 256> kl, ql;
  RowLoads<64, true, 256> ol;
  TriangleLoads<3, false, 256> tl, al;
  CopyLoads<L::kGate, 256> gl;
  auto live = [&](int c) { return min(len - 64 * c, 64); };
  // what A^T dO takes of a chunk ...
  auto load_first = [&](int c) {
    ol.load(p.d_o.at, o0 + 64 * (int64_t)c * p.d_o.t, p.d_o.t, live(c), cols, tid);
    al.load(p.matrices_t + ((int64_t)bh * p.NC + c) * (2 * kTriangleBytes) + kTriangleBytes, tid);
  };
  auto store_first = [&](int c) {
    ol.store(lds + L::kO + (c & 1) * 64 * 128, 0, tid);
    al.store(lds + L::kA, tid);
  };
  // ... and the rest, in KS parts
  auto load_rest = [&](int c, int s) {
    const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
    if (s == 0) kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live(c), DK, tid);
    if (s == min(1, KS - 1)) ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live(c), DK, tid);
    if (s == min(2, KS - 1)) tl.load(p.matrices_t + unit * (2 * kTriangleBytes), tid);
    if (s == KS - 1) gl.load(p.gates + unit, tid);
  };
  auto store_rest = [&](int c) {
    kl.store(lds + L::kK + (c & 1) * L::kTile, 0, tid);
    ql.store(lds + L::kQ, 0, tid);
    tl.store(lds + L::kT, tid);
    gl.store(lds + L::kGates + (c & 1) * L::kGate, tid);
  };
  auto before_n = [&](int c) {  // A^T dO
    const char* rows = lds + L::kO + (c & 1) * 64 * 128;
    BlockPair<3> a[3];
#pragma unroll
    for (int n = 0; n < 3; ++n) a[n] = pair_of<false, 3>(lds + L::kA, n, lane);
    Planes<1> of[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) of[s] = columns_of<64, 1>(rows, 0, 32 * s, wave, lane);
    f32x4 u[4] = {zero, zero, zero, zero};
    fence<true>();
#pragma unroll
    for (int n = 0; n < 3; ++n) mma_pair<2, false, false>(n, a[n], of, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(u_at + i * 1024) = u[i];
  };
  tl.clear(lds + L::kT, tid);
  al.clear(lds + L::kA, tid);
  if (first < last) {
    load_first(last - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) load_rest(last - 1, s);
    store_first(last - 1);
    store_rest(last - 1);
    load_first(max(last - 2, first));
  }
  __syncthreads();
  if (first < last) before_n(last - 1);
  __syncthreads();
  for (int c = last - 1; c >= first; --c) {  // (no branch around the loads: the first chunk is loaded once more)
    const int next = max(c - 1, first);
    const char* rows = lds + L::kO + (c & 1) * 64 * 128;
    const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
    store_first(c - 1);
    Planes<3> po[2];
    {
      f32x4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) * column_values<64, 1>(rows, 0, 16 * i, wave, lane);
      po[0] = split8<3>(y[0], y[1]);
      po[1] = split8<3>(y[2], y[3]);
    }
    f32x4 d[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) d[i] = zero;
    Planes<1> qt[2][4];
    auto group = [&](int n, Planes<1> (&to)[4]) {
#pragma unroll
      for (int i = 0; i < G; ++i) to[i] = columns(lds + L::kQ, 32 * (n * G / MT), n * G % MT + i);
    };
    group(0, qt[0]);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (n + 1 < NG) group(n + 1, qt[(n + 1) & 1]);
      fence<true>();
      if (n < KS) load_rest(next, n);
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int i = 0; i < G; ++i)
          d[n * G % MT + i] = mfma_bf16(qt[n & 1][i].p[0], po[n * G / MT].p[q], d[n * G % MT + i]);
      fence<true>();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(n_at + i * 1024) = d[i];
    __syncthreads();
    before_n(c - 1);
    store_rest(c - 1);
    load_first(max(c - 2, first));
    __syncthreads();
  }
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  delta_adjoint_kernel<DK><<<walk_blocks(p), 512, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_adjoint(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

}  // namespace mesa
