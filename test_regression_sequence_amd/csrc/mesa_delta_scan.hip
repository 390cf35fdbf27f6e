// Gated delta rule, forward: the walk over a sequence's chunks.
//
// A wave holds 16 columns (value dimensions) of the state's transpose M [dk, dv]
// as result tiles in registers, a workgroup's four waves 64 columns of one head:
// columns never meet, so the walk needs no exchange of states, and M goes into its
// products without passing LDS.  Per chunk of 64 tokens
//     W = T (V - c K M),  U = beta W,  O = c Q M + lower(D Q K^T) U,
//     M <- c_C M + K^T diag(c_C / c) U,
// T = (I + X diag(beta))^-1 from mesa_delta_chunk.hip.  Everything that a state
// depends on is multiplied in three bf16 planes (fp32's precision); a bf16 o takes
// two, whose error is far below its own rounding.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

// The place of the 16x32 operand block (row tile i, inner step s) of a lower
// triangular 64x64 matrix, 8 numbers a lane; (0, 1) and (1, 1) are zero.
__device__ __forceinline__ constexpr int lower_block(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }

template <int DK, bool BF16>
struct ScanLds {
  static constexpr int NP = BF16 ? 1 : 3, NA = BF16 ? 2 : 3;
  static constexpr int kPlane = 64 * DK * 2, kBlocks = 6 * 1024;
  static constexpr int kK = 0, kQ = kK + NP * kPlane, kV = kQ + NP * kPlane, kT = kV + NP * 64 * 128,
                       kA = kT + 3 * kBlocks, kGates = kA + NA * kBlocks, kBytes = kGates + sizeof(DeltaGates);
};

template <int DK, bool BF16>
__global__ __launch_bounds__(256, BF16 && DK < 128 ? 2 : 1) void delta_scan_kernel(DeltaParams p) {
  using L = ScanLds<DK, BF16>;
  constexpr int NP = L::NP, NA = L::NA, MT = DK / 16, KS = DK / 32, OMAX = BF16 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  const DeltaGates& gates = *reinterpret_cast<const DeltaGates*>(lds + L::kGates);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
  int bh, slice;
  if (!delta_unit(blockIdx.x, (p.dv + 63) / 64, p.B * p.H, bh, slice)) return;
  const int b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.Hk), len = delta_length(p, b);
  const int nc = (len + 63) / 64, col0 = 64 * slice, cols = min(64, p.dv - col0);
  const int col = col0 + 16 * wave + r;                 // this lane's column of the state
  const bool mine = 16 * wave < cols, out = p.o.at != nullptr;
  const int64_t state_at = ((int64_t)bh * p.dv + col) * DK;
  const int64_t q0 = b * p.q.b + hk * p.q.h, k0 = b * p.k.b + hk * p.k.h, v0 = b * p.v.b + h * p.v.h + col0,
                o0 = b * p.o.b + h * p.o.h + col0 + 16 * wave + 4 * g;

  f32x4 m[MT];  // rows 16 i + 4 g + e of M, column `col`
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (mine && p.s0) m[i] = *reinterpret_cast<const f32x4*>(p.s0 + state_at + 16 * i + 4 * g);
  }
  // the halves of diagonal blocks above the diagonal
  for (int n = 0; n < 3; ++n)
    if (tid < 128) *reinterpret_cast<u32x4*>(lds + L::kT + n * L::kBlocks + (tid < 64 ? 0 : 3) * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
  for (int n = 0; n < NA; ++n)
    if (tid < 128) *reinterpret_cast<u32x4*>(lds + L::kA + n * L::kBlocks + (tid < 64 ? 0 : 3) * 1024 + lane * 16) = u32x4{0, 0, 0, 0};

  RowLoads<DK, BF16, 256> kl, ql;
  RowLoads<64, BF16, 256> vl;
  f32x4 tl[3];
  u32x4 gl;
  auto load = [&](int c) {
    const int live = min(len - 64 * c, 64);
    const int64_t t0 = 64 * (int64_t)c, unit = (int64_t)bh * p.NC + c;
    kl.load(p.k.at, k0 + t0 * p.k.t, p.k.t, live, DK, tid);
    if (out) ql.load(p.q.at, q0 + t0 * p.q.t, p.q.t, live, DK, tid);
    vl.load(p.v.at, v0 + t0 * p.v.t, p.v.t, live, cols, tid);
    const float* inv = p.inverse + unit * kDeltaInverse;
#pragma unroll
    for (int n = 0; n < 3; ++n)
      if (tid + 256 * n < 640) tl[n] = *reinterpret_cast<const f32x4*>(inv + (tid + 256 * n) * 4);
    if (tid < (int)sizeof(DeltaGates) / 16) gl = reinterpret_cast<const u32x4*>(p.gates + unit)[tid];
  };
  auto store = [&]() {
    kl.store(lds + L::kK, L::kPlane, tid);
    if (out) ql.store(lds + L::kQ, L::kPlane, tid);
    vl.store(lds + L::kV, 64 * 128, tid);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      if (tid + 256 * n < 640) {
        const int block = wave + 4 * n, i = block >= 6 ? 3 : block >= 3 ? 2 : block >= 1 ? 1 : 0;
        const int j = block - i * (i + 1) / 2;
        bf16x4 t[3];
        split4<3>(tl[n], t);
#pragma unroll
        for (int a = 0; a < 3; ++a)
          *reinterpret_cast<bf16x4*>(lds + L::kT + a * L::kBlocks + lower_block(i, j >> 1) * 1024 + lane * 16 +
                                     (j & 1) * 8) = t[a];
      }
    if (tid < (int)sizeof(DeltaGates) / 16) *reinterpret_cast<u32x4*>(lds + L::kGates + tid * 16) = gl;
  };
  auto block_of = [&](int base, int i, int s, auto& f) {
#pragma unroll
    for (int n = 0; n < (int)(sizeof(f.p) / 16); ++n)
      f.p[n] = *reinterpret_cast<const bf16x8*>(lds + base + n * L::kBlocks + lower_block(i, s) * 1024 + lane * 16);
  };

  if (nc > 0) load(0);
  for (int c = 0; c < nc; ++c) {
    const int64_t unit = (int64_t)bh * p.NC + c;
    __syncthreads();
    store();
    if (c + 1 < nc) load(c + 1);
    __syncthreads();

    if (out) {  // wave w: row tile w of D Q K^T, below and on the diagonal
      Planes<NP> qf[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) qf[s] = rows_of<DK, NP>(lds + L::kQ, L::kPlane, 16 * wave, s, lane);
      const double gt = gates.g[16 * wave + r];
      for (int j = 0; j <= wave; ++j) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          acc = mma<2>(rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * j, s, lane), qf[s], acc);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = 16 * j + 4 * g + e;
          acc[e] = at <= 16 * wave + r ? acc[e] * decay(gt, gates.g[at]) : 0.f;
        }
        bf16x4 a[NA];
        split4<NA>(acc, a);
#pragma unroll
        for (int n = 0; n < NA; ++n)
          *reinterpret_cast<bf16x4*>(lds + L::kA + n * L::kBlocks + lower_block(wave, j >> 1) * 1024 + lane * 16 +
                                     (j & 1) * 8) = a[n];
      }
    }

    Planes<3> mp[KS], u[2], ut[2];
    if (mine) {
      if (p.states) {
        float* to = p.states + unit * p.dv * DK + (int64_t)col * DK + 4 * g;
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(to + 16 * i) = m[i];
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) mp[s] = split8<3>(m[2 * s], m[2 * s + 1]);
      f32x4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          acc = mma<2>(rows_of<DK, NP>(lds + L::kK, L::kPlane, 16 * i, s, lane), mp[s], acc);
        const f32x4 cc = *reinterpret_cast<const f32x4*>(&gates.c[16 * i + 4 * g]);
        x[i] = column_values<64, NP>(lds + L::kV, 64 * 128, 16 * i, wave, lane) - cc * acc;
      }
      const Planes<3> px[2] = {split8<3>(x[0], x[1]), split8<3>(x[2], x[3])};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s <= i / 2; ++s) {
          Planes<3> t;
          block_of(L::kT, i, s, t);
          acc = mma<2>(t, px[s], acc);
        }
        x[i] = acc;
      }
      if (p.w) {
        float* to = p.w + (unit * 64 + 4 * g) * p.dv + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(int64_t)(16 * i + e) * p.dv] = x[i][e];
      }
      f32x4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= *reinterpret_cast<const f32x4*>(&gates.beta[16 * i + 4 * g]);
        y[i] = x[i] * *reinterpret_cast<const f32x4*>(&gates.tail[16 * i + 4 * g]);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u[s] = split8<3>(x[2 * s], x[2 * s + 1]);
        ut[s] = split8<3>(y[2 * s], y[2 * s + 1]);
      }
    }
    if (out) __syncthreads();
    if (mine) {
      if (out) {  // o's transpose: a lane has 4 columns of one token
        const int live = len - 64 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s)
            acc = mma<OMAX>(mp[s], rows_of<DK, NP>(lds + L::kQ, L::kPlane, 16 * i, s, lane), acc);
          acc *= gates.c[16 * i + r];
#pragma unroll
          for (int s = 0; s <= i / 2; ++s) {
            Planes<NA> a;
            block_of(L::kA, i, s, a);
            acc = mma<OMAX>(u[s], a, acc);
          }
          const int t = 16 * i + r;
          if (t < live) {
            const int64_t at = o0 + (64 * (int64_t)c + t) * p.o.t;
            if constexpr (BF16) store_out4<__bf16>(p.o.at, at, acc);
            else store_out4<float>(p.o.at, at, acc);
          }
        }
      }
      const float whole = gates.c[63];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        m[i] *= whole;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          m[i] = mma<2>(columns_of<DK, NP>(lds + L::kK, L::kPlane, 32 * s, i, lane), ut[s], m[i]);
      }
    }
  }

  if (mine && p.s_final) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(p.s_final + state_at + 16 * i + 4 * g) = m[i];
  }
  if (mine && out) {  // behind the sequence
    for (int64_t t = len + r; t < p.T; t += 16) {
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      if constexpr (BF16) store_out4<__bf16>(p.o.at, o0 + t * p.o.t, zero);
      else store_out4<float>(p.o.at, o0 + t * p.o.t, zero);
    }
  }
}

template <int DK, bool BF16>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((p.B * p.H + 7) / 8 * 8 * ((p.dv + 63) / 64));
  delta_scan_kernel<DK, BF16><<<blocks, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(bool bf16, const DeltaParams& p, hipStream_t s) {
  if (p.dk == 128) return bf16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  if (p.dk == 64) return bf16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  return bf16 ? launch<32, true>(p, s) : launch<32, false>(p, s);
}

}  // namespace mesa
