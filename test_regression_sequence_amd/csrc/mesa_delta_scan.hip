// Gated delta rule, forward: the walk over a sequence's chunks (bf16 rows).
//
// A wave holds 16 columns (value dimensions) of the state's transpose M [dk, dv]
// as result tiles in registers, four waves of a workgroup 64 columns of one head:
// columns never meet, so the walk needs no exchange of states, and M goes into its
// products without passing LDS.  Per chunk of 64 tokens
//     W = T (V - c K M),  U = beta W,  M <- c_C M + K^T diag(c_C / c) U,
//     O = c Q M + A U,    T = (I + X diag(beta))^-1,  A = lower(D Q K^T),
// T and A from mesa_delta_chunk.hip.  Everything that a state depends on is
// multiplied in three bf16 planes (fp32's precision); o takes two, whose error is
// far below its own rounding.
//
// The chain from M to the next M bounds the walk, so four more waves, one beside
// each of the others on its SIMD, take what is not on it: they load the next
// chunk and form o from the planes of M and U that the first four leave in LDS.
//     first half:   chain K M, W, U            others Q M
//     second half:  chain K^T U, planes of M   others next chunk to LDS, A U, o
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK>
struct ScanLds {
  static constexpr int kTile = 64 * DK * 2, kMatrix = (int)delta_matrix_bytes(2), kGate = sizeof(DeltaGates);
  static constexpr int kMPlane = DK * 32, kUPlane = 64 * 32;  // one wave's columns
  static constexpr int kK = 0, kQ = kK + 2 * kTile, kV = kQ + kTile, kT = kV + 64 * 128, kA = kT + 3 * kBlocksBytes,
                       kGates = kA + 4 * kBlocksBytes, kM = kGates + 2 * kGate, kU = kM + 8 * kMPlane,
                       kBytes = kU + 8 * kUPlane;
};

template <int DK, bool OUT>
__global__ __launch_bounds__(512, 2) void delta_scan_kernel(DeltaParams p) {
  using L = ScanLds<DK>;
  constexpr int MT = DK / 16, KS = DK / 32;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const int tid = threadIdx.x & 255, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x) < 256;
  int bh, slice;
  if (!delta_unit(blockIdx.x, (p.dv + 63) / 64, p.B * p.H, bh, slice)) return;
  const int b = bh / p.H, h = bh % p.H, len = delta_length(p, b);
  const int nc = (len + 63) / 64, col0 = 64 * slice, cols = min(64, p.dv - col0);
  const bool mine = 16 * wave < cols;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  char* const m_planes = lds + L::kM + wave * 2 * L::kMPlane + lane * 16;
  char* const u_planes = lds + L::kU + wave * 2 * L::kUPlane + lane * 16;

  if (chain) {
    const int col = col0 + 16 * wave + r;  // this lane's column of the state
    const int64_t state_at = ((int64_t)bh * p.dv + col) * DK + 4 * g;
    f32x4 m[MT];  // rows 16 i + 4 g + e of M
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      m[i] = zero;
      if (mine && p.s0) m[i] = *reinterpret_cast<const f32x4*>(p.s0 + state_at + 16 * i);
    }
    Planes<3> mp[KS];
    auto planes = [&]() {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
        if constexpr (OUT)
#pragma unroll
          for (int n = 0; n < 2; ++n) *reinterpret_cast<bf16x8*>(m_planes + n * L::kMPlane + s * 1024) = mp[s].p[n];
      }
    };
    planes();
    __builtin_amdgcn_s_setprio(2);
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      const char* keys = lds + L::kK + (c & 1) * L::kTile;
      const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
      f32x4 x[4] = {zero, zero, zero, zero}, y[4];
      Planes<3> ut[2];
      if (mine) {
        // operands come from LDS one step ahead of the products that take them: the
        // fences keep their loads there
        Planes<1> f[2][4];
        Planes<3> px[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[0][i] = rows_of<DK, 1>(keys, 0, 16 * i, 0, lane);
        BlockPair<3> t;
#pragma unroll
        for (int s = 0; s < KS; ++s) {  // x = K M
          if (s + 1 < KS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows_of<DK, 1>(keys, 0, 16 * i, s + 1, lane);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = column_values<64, 1>(lds + L::kV, 0, 16 * i, wave, lane);
            t = pair_of<true, 3>(lds + L::kT, 0, lane);
          }
          fence<true>();
          mma_tiles<2>(f[s & 1], mp[s], x);
          fence<true>();
        }
        if (p.states) {
          float* to = p.states + ((int64_t)bh * p.NC + c) * p.dv * DK + (int64_t)col * DK + 4 * g;
#pragma unroll
          for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + 16 * i) = m[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] -= *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]) * x[i];
        px[0] = split8<3>(y[0], y[1]);
        px[1] = split8<3>(y[2], y[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = zero;
        mma_triangle<2, true, false, true>(lds + L::kT, t, px, x, lane);  // W
        if (p.w) {
          float* to = p.w + (((int64_t)bh * p.NC + c) * 64 + 4 * g) * p.dv + col;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) to[(int64_t)(16 * i + e) * p.dv] = x[i][e];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] *= *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]);
          y[i] = x[i] * *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
        }
        if constexpr (OUT) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const Planes<2> u = split8<2>(x[2 * s], x[2 * s + 1]);
#pragma unroll
            for (int n = 0; n < 2; ++n) *reinterpret_cast<bf16x8*>(u_planes + n * L::kUPlane + s * 1024) = u.p[n];
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) ut[s] = split8<3>(y[2 * s], y[2 * s + 1]);
        const float whole = gates.c[63];
#pragma unroll
        for (int i = 0; i < MT; ++i) m[i] *= whole;
      }
      __syncthreads();
      if (mine) {
        constexpr int G = MT < 4 ? MT : 4, NG = 2 * MT / G;  // K^T in groups of 4 tiles
        Planes<1> kt[2][4];
        auto group = [&](int n, Planes<1> (&to)[4]) {
#pragma unroll
          for (int i = 0; i < G; ++i) to[i] = columns_of<DK, 1>(keys, 0, 32 * (n * G / MT), n * G % MT + i, lane);
        };
        group(0, kt[0]);
#pragma unroll
        for (int n = 0; n < NG; ++n) {  // M += K^T U
          if (n + 1 < NG) group(n + 1, kt[(n + 1) & 1]);
          fence<true>();
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int i = 0; i < G; ++i)
              m[n * G % MT + i] = mfma_bf16(kt[n & 1][i].p[0], ut[n * G / MT].p[q], m[n * G % MT + i]);
          fence<true>();
        }
        planes();
      }
      __syncthreads();
    }
    if (mine && p.s_final) {
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(p.s_final + state_at + 16 * i) = m[i];
    }
    return;
  }

  const int hk = h / (p.H / p.Hk);
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h + col0,
                o0 = b * p.o.b + h * p.o.h + col0 + 16 * wave + 4 * g;
  RowLoads<DK, true, 256> kl, ql;
  RowLoads<64, true, 256> vl;
  CopyLoads<3 * kBlocksBytes, 256> tl;
  CopyLoads<2 * kBlocksBytes, 256> al;
  CopyLoads<L::kGate, 256> gl;
  auto load = [&](int c) {
    const int live = min(len - 64 * c, 64);
    const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
    const char* matrix = p.matrices + unit * L::kMatrix;
    kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
    vl.load(p.v.at, v0 + t0 * p.v.t, p.v.t, live, cols, tid);
    tl.load(matrix, tid);
    gl.load(p.gates + unit, tid);
    if constexpr (OUT) {
      ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live, DK, tid);
      al.load(matrix + 3 * kBlocksBytes, tid);
    }
  };
  auto store = [&](int c) {
    kl.store(lds + L::kK + (c & 1) * L::kTile, 0, tid);
    vl.store(lds + L::kV, 0, tid);
    tl.store(lds + L::kT, tid);
    gl.store(lds + L::kGates + (c & 1) * L::kGate, tid);
    if constexpr (OUT) {
      ql.store(lds + L::kQ, 0, tid);
      al.store(lds + L::kA + (c & 1) * 2 * kBlocksBytes, tid);
    }
  };
  if (nc > 0) {
    load(0);
    store(0);
    if (nc > 1) load(1);
  }
  __syncthreads();
  for (int c = 0; c < nc; ++c) {
    f32x4 o[4] = {zero, zero, zero, zero};  // o's transpose: a lane has 4 columns of one token
    if (OUT && mine) {
      Planes<1> f[2][4];
      Planes<2> mp[2];
      auto operands = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[s & 1][i] = rows_of<DK, 1>(lds + L::kQ, 0, 16 * i, s, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n) mp[s & 1].p[n] = *reinterpret_cast<const bf16x8*>(m_planes + n * L::kMPlane + s * 1024);
      };
      operands(0);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (s + 1 < KS) operands(s + 1);
        fence<true>();
        mma_tiles_t<1>(mp[s & 1], f[s & 1], o);
        fence<true>();
      }
      const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= gates.c[16 * i + r];
    }
    __syncthreads();
    if (c + 1 < nc) store(c + 1);
    if (c + 2 < nc) load(c + 2);
    if (OUT && mine) {
      Planes<2> u[2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n) u[s].p[n] = *reinterpret_cast<const bf16x8*>(u_planes + n * L::kUPlane + s * 1024);
      const char* a = lds + L::kA + (c & 1) * 2 * kBlocksBytes;
      mma_triangle<1, true, true, true>(a, pair_of<true, 2>(a, 0, lane), u, o, lane);
      const int live = len - 64 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 16 * i + r;
        if (at < live) store_out4<__bf16>(p.o.at, o0 + (64 * (int64_t)c + at) * p.o.t, o[i]);
      }
    }
    __syncthreads();
  }
  if (OUT && mine) {  // behind the sequence
    for (int64_t t = len + r; t < p.T; t += 16) store_out4<__bf16>(p.o.at, o0 + t * p.o.t, zero);
  }
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((p.B * p.H + 7) / 8 * 8 * ((p.dv + 63) / 64));
  if (p.o.at) delta_scan_kernel<DK, true><<<blocks, 512, 0, s>>>(p);
  else delta_scan_kernel<DK, false><<<blocks, 512, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

}  // namespace mesa
