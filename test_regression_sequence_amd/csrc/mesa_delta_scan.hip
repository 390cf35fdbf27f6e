// Gated delta rule, forward: the walk over a sequence's chunks (bf16 rows).
//
// A wave holds 16 columns (value dimensions) of the state's transpose M [dk, dv]
// as result tiles in registers, four waves of a workgroup 64 columns of one head:
// columns never meet, so the walk needs no exchange of states, and M goes into its
// products without passing LDS.  Per chunk of 64 tokens
//     W = T (V - c K M),  U = beta W,  M <- c_C M + K^T diag(c_C / c) U,
//     O = c Q M + A U,    T = (I + X diag(beta))^-1,  A = lower(D Q K^T),
// T and A from mesa_delta_chunk.hip.  Everything that a state or o depends on is
// multiplied in three bf16 planes (fp32's precision).  With two for o, whose error is far
// below its own rounding, one in 2000 of its numbers was not the nearest.
//
// The chain from M to the next M bounds the walk, so four more waves, one beside
// each of the others on its SIMD, take what is not on it: they load the next
// chunk and form o from the planes of M and U that the first four leave in LDS.
//     first half:   chain K M, W, U, half of K^T U       others Q M, the next chunk's loads
//     second half:  chain the rest of K^T U, planes of M  others A U, next chunk to LDS, o
//
// A chunk takes 3.4 us where few workgroups run, of which the chain's 132 products are 0.9
// and their operands' ways through conversions and LDS the rest, and 4.3 to 4.7 on all CUs
// (B=1 H=16 T=32768 d=128, 8 segments of 57 chunks side by side: 244 to 266 us, the matrix unit
// 38 %, the vector unit 36 % and LDS 43 % of them).  With states and W kept memory is next: at
// B=8 H=16 T=4096 d=128 388 to 400 us for 1.6 GB, 4.0 to 4.1 TB/s where a large copy reaches 4.9.
// (o's products in two planes took 220 to 237 and 356 to 371 us.  In three, with A U in the walk's
// first half as then, prefill calls of 128 heads of 2048 tokens took 212 us, so 189.)
#include <algorithm>

#include "mesa_delta_probe.h"

namespace mesa {

namespace {

template <int DK>
struct ScanLds {
  static constexpr int kTile = 64 * DK * 2, kMatrix = (int)delta_matrix_bytes(true), kGate = sizeof(DeltaGates);
  static constexpr int kMPlane = DK * 32;  // one wave's columns
  static constexpr int kK = 0, kQ = kK + 2 * kTile, kV = kQ + kTile, kT = kV + 64 * 128, kA = kT + 3 * kBlocksBytes,
                       kGates = kA + 3 * kBlocksBytes, kM = kGates + 2 * kGate, kU = kM + 12 * kMPlane,
                       kBytes = kU + 4 * 4096;
};

template <int DK, bool OUT>
__device__ __forceinline__ void walk_segment(const DeltaParams& p, uint32_t id, char* lds) {
  using L = ScanLds<DK>;
  constexpr int MT = DK / 16, KS = DK / 32;
  const int tid = threadIdx.x & 255, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, g = lane >> 4;
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x) < 256;
  Part part;
  if (!part_of(p, id, part)) return;
  const int bh = part.bh, b = part.b, h = part.h, len = part.len, first = part.first, last = part.last;
  const int col0 = part.col0, cols = part.cols;
  const bool mine = 16 * wave < cols;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  char* const m_planes = lds + L::kM + wave * 3 * L::kMPlane + lane * 16;
  char* const u_to = lds + L::kU + wave * 4096 + lane * 16;  // U's four tiles

  if (chain) {
    const int col = col0 + 16 * wave + r;  // this lane's column of the state
    f32x4 m[MT];  // rows 16 i + 4 g + e of M
    const float* const from = walk_from(p, part, p.s0, 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      m[i] = zero;
      if (mine && from) m[i] = *reinterpret_cast<const f32x4*>(from + col * DK + 16 * i + 4 * g);
    }
    const TileRows<DK> rows(lane);
    const TileColumns<DK> columns(lane);
    Planes<3> mp[KS];
    auto planes = [&](int first, int last) {
#pragma unroll
      for (int s = first; s < last; ++s) {
        mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
        if constexpr (OUT)
#pragma unroll
          for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(m_planes + n * L::kMPlane + s * 1024) = mp[s].p[n];
      }
    };
    planes(0, KS);
    __builtin_amdgcn_s_setprio(2);
    __syncthreads();
    for (int c = first; c < last; ++c) {
      const char* keys = lds + L::kK + (c & 1) * L::kTile;
      const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
      f32x4 x[4] = {zero, zero, zero, zero}, y[4];
      Planes<3> ut[2];
      constexpr int G = MT < 4 ? MT : 4, NG = 2 * MT / G;  // K^T in groups of 4 tiles
      Planes<1> kt[2][4];
      auto group = [&](int n, Planes<1> (&to)[4]) {
#pragma unroll
        for (int i = 0; i < G; ++i) to[i] = columns(keys, 32 * (n * G / MT), n * G % MT + i);
      };
      auto mma_group = [&](int n) {
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
          for (int i = 0; i < G; ++i)
            m[n * G % MT + i] = mfma_bf16(kt[n & 1][i].p[0], ut[n * G / MT].p[q], m[n * G % MT + i]);
      };
      if (mine) {
        // Operands come from LDS one step ahead of the products that take them (the fences
        // keep their loads there); between two fences products of one block and the
        // conversions for the next run side by side.
        Planes<1> f[2][4];
        Planes<3> px[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[0][i] = rows(keys, 16 * i, 0);
        BlockPair<3> t[2];
        f32x4 cc[4];
#pragma unroll
        for (int s = 0; s < KS; ++s) {  // x = K M
          if (s + 1 < KS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[(s + 1) & 1][i] = rows(keys, 16 * i, s + 1);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[i] = column_values<64, 1>(lds + L::kV, 0, 16 * i, wave, lane);
              cc[i] = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]);
            }
            t[0] = pair_of<true, 3>(lds + L::kT, 0, lane);
          }
          fence<true>();
          mma_tiles<2>(f[s & 1], mp[s], x);
          fence<true>();
        }
        if (p.states) {
          const Window to = window_at(p.states + ((int64_t)bh * p.NC + c) * p.dv * DK);
#pragma unroll
          for (int i = 0; i < MT; ++i) window_store(to, (col * DK + 4 * g) * 4, 64 * i, m[i]);
        }
        t[1] = pair_of<true, 3>(lds + L::kT, 1, lane);
        f32x4 beta[2], tail[2];
        auto gates_of = [&](int s) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            beta[i] = *reinterpret_cast<const f32x4*>(&gates.beta[32 * s + 16 * i + 4 * g]);
            tail[i] = *reinterpret_cast<const f32x4*>(&gates.tail[32 * s + 16 * i + 4 * g]);
          }
        };
        auto residual = [&](int s) {  // V - c K M
#pragma unroll
          for (int i = 2 * s; i < 2 * s + 2; ++i) {
            y[i] -= cc[i] * x[i];
            x[i] = zero;
          }
          px[s] = split8<3>(y[2 * s], y[2 * s + 1]);
        };
        auto scaled = [&](int s) {  // W to U and tail U
#pragma unroll
          for (int i = 2 * s; i < 2 * s + 2; ++i) {
            x[i] *= beta[i & 1];
            if constexpr (OUT) *reinterpret_cast<f32x4*>(u_to + i * 1024) = x[i];
            y[i] = x[i] * tail[i & 1];
          }
          ut[s] = split8<3>(y[2 * s], y[2 * s + 1]);
        };
        auto keep = [&](int s) {
          if (p.w) {
            const Window to = window_at(p.w + ((int64_t)bh * p.NC + c) * 64 * p.dv);
#pragma unroll
            for (int i = 2 * s; i < 2 * s + 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) window_store(to, (4 * g * p.dv + col) * 4, (16 * i + e) * p.dv * 4, x[i][e]);
          }
        };
        residual(0);
        fence<true>();
        residual(1);
        mma_pair<2, true, false>(0, t[0], px, x);
        t[0] = pair_of<true, 3>(lds + L::kT, 2, lane);
        gates_of(0);
        group(0, kt[0]);
        const float whole = gates.c[63];
        fence<true>();
        keep(0);
        scaled(0);
        mma_pair<2, true, false>(1, t[1], px, x);
        gates_of(1);
        fence<true>();
        mma_pair<2, true, false>(2, t[0], px, x);
#pragma unroll
        for (int i = 0; i < MT; ++i) m[i] *= whole;
#pragma unroll
        for (int n = 0; n < NG / 2; ++n) {  // M += K^T U, the first 32 tokens
          group(n + 1, kt[(n + 1) & 1]);
          fence<true>();
          mma_group(n);
        }
        keep(1);
        scaled(1);
      }
      __syncthreads();
      if (mine) {
#pragma unroll
        for (int n = NG / 2; n < NG; ++n) {  // the other 32
          if (n + 1 < NG) group(n + 1, kt[(n + 1) & 1]);
          fence<true>();
          if (n == NG - 1) planes(0, KS - G / 2);
          mma_group(n);
        }
        planes(KS - G / 2, KS);
      }
      __syncthreads();
    }
    float* const to = walk_to(p, part, p.s_final, p.NS - 1);
    if (mine && to) {
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + col * DK + 16 * i + 4 * g) = m[i];
    }
    return;
  }

  const int hk = (uint32_t)h / p.by_shared;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h + col0,
                o0 = b * p.o.b + h * p.o.h + col0 + 16 * wave;
  const TileRows<DK> rows(lane);
  RowLoads<DK, true, 256> kl, ql;
  RowLoads<64, true, 256> vl;
  CopyLoads<3 * kBlocksBytes, 256> tl;
  TriangleLoads<3, true, 256> al;
  CopyLoads<L::kGate, 256> gl;
  // part s of KS of a chunk's loads, so that they go out along the products with Q
  auto load = [&](int c, int s) {
    const int live = min(len - 64 * c, 64);
    const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
    const char* matrix = p.matrices + unit * L::kMatrix;
    if (s == 0) kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
    if (OUT && s == min(1, KS - 1)) ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live, DK, tid);
    if (s == min(2, KS - 1)) {
      vl.load(p.v.at, v0 + t0 * p.v.t, p.v.t, live, cols, tid);
      tl.load(matrix, tid);
    }
    if (s == KS - 1) {
      if constexpr (OUT) al.load(matrix + 3 * kBlocksBytes, tid);
      gl.load(p.gates + unit, tid);
    }
  };
  auto load_all = [&](int c) {
#pragma unroll
    for (int s = 0; s < KS; ++s) load(c, s);
  };
  auto store = [&](int c) {
    kl.store(lds + L::kK + (c & 1) * L::kTile, 0, tid);
    vl.store(lds + L::kV, 0, tid);
    tl.store(lds + L::kT, tid);
    gl.store(lds + L::kGates + (c & 1) * L::kGate, tid);
    if constexpr (OUT) {
      ql.store(lds + L::kQ, 0, tid);
      al.store(lds + L::kA, tid);
    }
  };
  if constexpr (OUT) al.clear(lds + L::kA, tid);
  if (first < last) {
    load_all(first);
    store(first);
  }
  __syncthreads();
  f32x4 o[4], u[4];  // o's transpose (a lane has 4 columns of one token) and U
  BlockPair<3> a[3];
  auto finish = [&](int c) {  // o of chunk c: A U added to c Q M
    const Planes<3> up[2] = {split8<3>(u[0], u[1]), split8<3>(u[2], u[3])};
#pragma unroll
    for (int n = 0; n < 3; ++n) mma_pair<2, true, true>(n, a[n], up, o);
    const int live = mine ? len - 64 * c : 0;
    const Window to = window_at(static_cast<__bf16*>(p.o.at) + o0 + 64 * (int64_t)c * p.o.t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      window_store_row<true>(to, 16 * i + r < live ? (r * (uint32_t)p.o.t + 4 * g) * 2 : kNowhere,
                             16 * i * (uint32_t)p.o.t * 2, o[i]);
  };
  // Without a branch around the loads (the last chunk is loaded once more), and with
  // products for columns that do not exist: where paths with and without loads in
  // flight meet, the compiler waits for them.
  for (int c = first; c < last; ++c) {
    const int next = min(c + 1, last - 1);
    if constexpr (OUT) {
      Planes<1> f[2][4];
      Planes<3> mp[2];
      auto operands = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[s & 1][i] = rows(lds + L::kQ, 16 * i, s);
#pragma unroll
        for (int n = 0; n < 3; ++n) mp[s & 1].p[n] = *reinterpret_cast<const bf16x8*>(m_planes + n * L::kMPlane + s * 1024);
      };
      operands(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = zero;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (s + 1 < KS) operands(s + 1);
        fence<true>();
        load(next, s);
        mma_tiles_t<2>(mp[s & 1], f[s & 1], o);
        fence<true>();
      }
      const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates + (c & 1) * L::kGate);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= gates.c[16 * i + r];
#pragma unroll
      for (int n = 0; n < 3; ++n) a[n] = pair_of<true, 3>(lds + L::kA, n, lane);
    } else {
      load_all(next);
    }
    __syncthreads();
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const f32x4*>(u_to + i * 1024);
    }
    store(c + 1);
    if constexpr (OUT) finish(c);
    __syncthreads();
  }
  if (OUT && mine) {  // behind the sequence
    const int end = (int)min((int64_t)p.T, (int64_t)64 * (first + p.L));
    for (int64_t t = max(len, 64 * first) + r; t < end; t += 16) store_out4<__bf16>(p.o.at, o0 + t * p.o.t + 4 * g, zero);
  }
}

template <int DK, bool OUT>
__global__ __launch_bounds__(512, 2) void delta_scan_kernel(DeltaParams p) {
  __shared__ __attribute__((aligned(16))) char lds[ScanLds<DK>::kBytes];
  walk_segment<DK, OUT>(p, blockIdx.x, lds);
}

// The first segment whole, and what the others but the last make of states, side by side.
template <int DK, bool OUT>
__global__ __launch_bounds__(512, 2) void delta_open_kernel(DeltaParams p, uint32_t probes, Divisor by_part,
                                                            Divisor by_slices) {
  __shared__ __attribute__((aligned(16))) char lds[std::max(ScanLds<DK>::kBytes, 2 * ProbeLds<DK, true>::kBuffer)];
  if (blockIdx.x < probes) probe_segment<DK, true>(p, blockIdx.x, by_part, by_slices, lds);
  else walk_segment<DK, OUT>(p, blockIdx.x - probes, lds);
}

template <int DK>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  if (p.o.at) delta_scan_kernel<DK, true><<<walk_blocks(p), 512, 0, s>>>(p);
  else delta_scan_kernel<DK, false><<<walk_blocks(p), 512, 0, s>>>(p);
  return hipGetLastError();
}

template <int DK>
hipError_t open(const DeltaParams& p, hipStream_t s) {
  const uint32_t probes = probe_blocks(p), blocks = probes + walk_blocks(p);
  if (p.o.at) delta_open_kernel<DK, true><<<blocks, 512, 0, s>>>(p, probes, probe_part(p), divisor(probe_slices(p)));
  else delta_open_kernel<DK, false><<<blocks, 512, 0, s>>>(p, probes, probe_part(p), divisor(probe_slices(p)));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(p, s) : p.dk == 64 ? launch<64>(p, s) : launch<32>(p, s);
}

hipError_t launch_delta_open(const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? open<128>(p, s) : p.dk == 64 ? open<64>(p, s) : open<32>(p, s);
}

}  // namespace mesa
