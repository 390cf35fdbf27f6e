// Gated delta rule: what a chunk of 64 tokens needs of its keys and gates alone.
//
// With X_tj = (c_t / c_j) k_t.k_j below the diagonal, the forward pass needs
// (I + X diag(beta))^-1 and the backward pass the transpose of (I + diag(beta)
// X)^-1: unit lower triangular 64x64 inverses, kept as their ten 16x16 blocks in
// fp32.  The four diagonal blocks are inverted by forward substitution, a lane a
// column; a block s below the diagonal is -T_ii sum_m L_im T_mj, by fp32 matrix
// instructions (16 block products).  Substitution keeps its accuracy for keys that
// repeat, where the powers of a Neumann series grow to 10^18.
//
// One wave a chunk: there are B H T / 64 of them, all independent.  Logarithms of
// the forget factors are summed in 64 bits, so that a ratio c_t / c_j keeps fp32's
// precision however strong the decay before it.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

constexpr int kLd = 20;  // floats of a 16-wide row in LDS

constexpr int block_of(int i, int j) { return i * (i + 1) / 2 + j; }

template <int DK, bool BF16, bool TRANSPOSED>
__global__ __launch_bounds__(64) void delta_chunk_kernel(DeltaParams p) {
  constexpr int NP = BF16 ? 1 : 3, ES = BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float low[10][16 * kLd];
  __shared__ __attribute__((aligned(16))) float diag[4][16 * kLd];
  __shared__ double sg[kDeltaChunk];
  __shared__ float sbeta[kDeltaChunk];
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const uint32_t unit = blockIdx.x;
  const int c = unit % p.NC, bh = unit / p.NC, b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.Hk);
  const int live = min(delta_length(p, b) - c * kDeltaChunk, kDeltaChunk);
  if (live <= 0) return;

  // gates: one token a lane
  double lg = 0.0;
  float beta = 0.f;
  if (lane < live) {
    const int64_t t = c * kDeltaChunk + lane;
    lg = fmax(log2((double)*gate_at(p.gamma, b, h, t)), -16384.0);  // a factor of 0 ends what came before
    beta = *gate_at(p.beta, b, h, t);
  }
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const double before = __shfl_up(lg, off);
    if (lane >= off) lg += before;
  }
  sg[lane] = lg;
  sbeta[lane] = beta;
  if constexpr (!TRANSPOSED) {
    DeltaGates& out = p.gates[unit];
    out.g[lane] = lg;
    out.c[lane] = exp2f((float)lg);
    out.tail[lane] = decay(__shfl(lg, 63), lg);
    out.beta[lane] = beta;
  }
  __syncthreads();

  // keys, 16 rows of 8 columns a lane group at a time
  Planes<NP> k[4][DK / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * i + r;
    const char* at = static_cast<const char*>(p.k.at) +
                     (b * p.k.b + hk * p.k.h + (int64_t)(c * kDeltaChunk + min(row, live - 1)) * p.k.t) * ES;
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const u32x4* q = reinterpret_cast<const u32x4*>(at + (32 * s + 8 * g) * ES);
      if constexpr (BF16) {
        u32x4 v = q[0];
        if (row >= live) v = u32x4{0, 0, 0, 0};
        k[i][s].p[0] = __builtin_bit_cast(bf16x8, v);
      } else {
        f32x4 x = __builtin_bit_cast(f32x4, q[0]), y = __builtin_bit_cast(f32x4, q[1]);
        if (row >= live) x = y = f32x4{0.f, 0.f, 0.f, 0.f};
        k[i][s] = split8<NP>(x, y);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) acc = mma<2>(k[i][s], k[j][s], acc);
      const int col = 16 * j + r;
      const double gj = sg[col];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        const float x = acc[e] * decay(sg[t], gj) * (TRANSPOSED ? sbeta[t] : sbeta[col]);
        low[block_of(i, j)][(4 * g + e) * kLd + r] = col < t ? x : 0.f;
      }
    }
  __syncthreads();

  {  // lane group g inverts diagonal block g, lane r its column r
    const float* l = low[block_of(g, g)];
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.f : 0.f;
#pragma unroll
      for (int m4 = 0; m4 < i; m4 += 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(l + i * kLd + m4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m4 + e < i) s = fmaf(-a[e], x[m4 + e], s);
      }
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) diag[g][i * kLd + r] = x[i];
  }
  __syncthreads();

  f32x4 t[4][4];  // T_ij, rows 4 g + e, column r
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[i][i][e] = diag[i][(4 * g + e) * kLd + r];
#pragma unroll
  for (int s = 1; s < 4; ++s)
#pragma unroll
    for (int i = s; i < 4; ++i) {
      const int j = i - s;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f}, out = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m < j || m >= i) continue;
        const f32x4 a = *reinterpret_cast<const f32x4*>(&low[block_of(i, m)][r * kLd + 4 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma_f32(a[e], t[m][j][e], acc);
      }
      const f32x4 d = *reinterpret_cast<const f32x4*>(&diag[i][r * kLd + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) out = mfma_f32(d[e], acc[e], out);
      t[i][j] = -out;
    }

  // a lane's 4 numbers lie along the later product's inner index: rows of the
  // transposed inverse as they are, rows of the inverse by way of LDS
  float* to = (TRANSPOSED ? p.inverse_t : p.inverse) + (int64_t)unit * kDeltaInverse + lane * 4;
  if constexpr (TRANSPOSED) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j) *reinterpret_cast<f32x4*>(to + block_of(i, j) * 256) = t[i][j];
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) low[block_of(i, j)][(4 * g + e) * kLd + r] = t[i][j][e];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 10; ++n)
      *reinterpret_cast<f32x4*>(to + n * 256) = *reinterpret_cast<const f32x4*>(&low[n][r * kLd + 4 * g]);
  }
}

template <int DK, bool BF16>
hipError_t launch(bool transposed, const DeltaParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.B * p.H * p.NC));
  if (transposed) delta_chunk_kernel<DK, BF16, true><<<grid, 64, 0, s>>>(p);
  else delta_chunk_kernel<DK, BF16, false><<<grid, 64, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunks(bool bf16, bool transposed, const DeltaParams& p, hipStream_t s) {
  if (p.dk == 128) return bf16 ? launch<128, true>(transposed, p, s) : launch<128, false>(transposed, p, s);
  if (p.dk == 64) return bf16 ? launch<64, true>(transposed, p, s) : launch<64, false>(transposed, p, s);
  return bf16 ? launch<32, true>(transposed, p, s) : launch<32, false>(transposed, p, s);
}

}  // namespace mesa
