// Gated delta rule: what a chunk of 64 tokens needs of its keys, queries and gates alone.
//
// With X_tj = (c_t / c_j) k_t.k_j below the diagonal, the forward walk needs
// (I + X diag(beta))^-1 and the backward walk the transpose of (I + diag(beta)
// X)^-1: unit lower triangular 64x64 inverses, formed as their ten 16x16 blocks in
// fp32.  The four diagonal blocks are inverted by forward substitution, a lane a
// column; a block s below the diagonal is -T_ii sum_m L_im T_mj, by fp32 matrix
// instructions (16 block products).  Substitution keeps its accuracy for keys that
// repeat, where the powers of a Neumann series grow to 10^18.  Both walks need
// (c_t / c_j) q_t.k_j on and below the diagonal, the backward one its transpose.
//
// One wave a chunk: there are B H T / 64 of them, all independent, so what can be
// done here is taken off the walks, whose chunks follow one another.  The matrices
// leave as the walks' operands, in bf16 parts.  Logarithms of the forget factors
// are summed in 64 bits, so that a ratio c_t / c_j keeps fp32's precision however
// strong the decay before it.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

constexpr int kLd = 20;  // floats of a 16-wide row in LDS

constexpr int tile_of(int i, int j) { return i * (i + 1) / 2 + j; }

template <int DK, bool BF16, bool TRANSPOSED>
__global__ __launch_bounds__(64) void delta_chunk_kernel(DeltaParams p) {
  constexpr int NP = BF16 ? 1 : 3, ES = BF16 ? 2 : 4, NA = BF16 && !TRANSPOSED ? 2 : 3;
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
    out.c[lane] = decay(lg, 0.0);
    out.tail[lane] = decay(__shfl(lg, 63), lg);
    out.beta[lane] = beta;
  }
  __syncthreads();

  // 16 rows of 8 columns a lane group at a time
  auto rows = [&](const DeltaRows& x, int i, Planes<NP> (&f)[DK / 32]) {
    const int row = 16 * i + r;
    const char* at = static_cast<const char*>(x.at) +
                     (b * x.b + hk * x.h + (int64_t)(c * kDeltaChunk + min(row, live - 1)) * x.t) * ES;
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const u32x4* from = reinterpret_cast<const u32x4*>(at + (32 * s + 8 * g) * ES);
      if constexpr (BF16) {
        u32x4 v = from[0];
        if (row >= live) v = u32x4{0, 0, 0, 0};
        f[s].p[0] = __builtin_bit_cast(bf16x8, v);
      } else {
        f32x4 x0 = __builtin_bit_cast(f32x4, from[0]), x1 = __builtin_bit_cast(f32x4, from[1]);
        if (row >= live) x0 = x1 = f32x4{0.f, 0.f, 0.f, 0.f};
        f[s] = split8<NP>(x0, x1);
      }
    }
  };
  Planes<NP> k[4][DK / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows(p.k, i, k[i]);

  char* const to = (TRANSPOSED ? p.matrices_t : p.matrices) + (int64_t)unit * delta_matrix_bytes(NA) + lane * 16;
  // A block's two tiles, in parts, to its place
  auto put = [&](int matrix, int parts, int block, const f32x4& lo, const f32x4& hi) {
    const Planes<3> f = split8<3>(lo, hi);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      if (n < parts)
        *reinterpret_cast<bf16x8*>(to + (matrix * 3 + n) * kBlocksBytes + block * 1024) = f.p[n];
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 even[4] = {zero, zero, zero, zero};

  if (p.q.at) {  // queries and keys: a lane has one query and 4 keys of a tile, transposed the other way round
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      Planes<NP> q[DK / 32];
      rows(p.q, t, q);
      f32x4 a[4] = {zero, zero, zero, zero};
#pragma unroll
      for (int j = 0; j <= t; ++j) {
#pragma unroll
        for (int s = 0; s < DK / 32; ++s)
          a[j] = TRANSPOSED ? mma<2>(q[s], k[j][s], a[j]) : mma<2>(k[j][s], q[s], a[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at_t = 16 * t + (TRANSPOSED ? 4 * g + e : r), at_j = 16 * j + (TRANSPOSED ? r : 4 * g + e);
          a[j][e] = at_j <= at_t ? a[j][e] * decay(sg[at_t], sg[at_j]) : 0.f;
        }
      }
      if constexpr (!TRANSPOSED) {
#pragma unroll
        for (int s = 0; s <= t / 2; ++s) put(1, NA, lower_block(t, s), a[2 * s], a[2 * s + 1]);
      } else {
        // blocks of a transposed matrix pair up tiles of two queries
        if (t & 1) {
#pragma unroll
          for (int j = 0; j <= t; ++j) put(1, NA, upper_block(j, t / 2), j < t ? even[j] : zero, a[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) even[j] = a[j];
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
        low[tile_of(i, j)][(4 * g + e) * kLd + r] = col < t ? x : 0.f;
      }
    }
  __syncthreads();

  {  // lane group g inverts diagonal block g, lane r its column r
    const float* l = low[tile_of(g, g)];
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
        const f32x4 a = *reinterpret_cast<const f32x4*>(&low[tile_of(i, m)][r * kLd + 4 * g]);
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
  if constexpr (TRANSPOSED) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = j / 2; s < 2; ++s)
        put(0, 3, upper_block(j, s), 2 * s < j ? zero : t[2 * s][j], t[2 * s + 1][j]);
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) low[tile_of(i, j)][(4 * g + e) * kLd + r] = t[i][j][e];
    __syncthreads();
    auto row = [&](int i, int j) { return *reinterpret_cast<const f32x4*>(&low[tile_of(i, j)][r * kLd + 4 * g]); };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s <= i / 2; ++s) put(0, 3, lower_block(i, s), row(i, 2 * s), 2 * s + 1 <= i ? row(i, 2 * s + 1) : zero);
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
