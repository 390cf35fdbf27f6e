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
// There are B H T / 64 chunks, all independent, so what can be done here is taken
// off the walks, whose chunks follow one another.  Four waves a chunk: wave w forms row
// tile w of both products, inverts diagonal block w and then has the inverse's column
// of blocks w, which depends on no other column.  The forward walk's inverse leaves as its operands, in bf16 parts, and the backward walk's matrices in fp32, tile
// by tile in the operands' order: 10 KB in place of 18 for conversions that the waves beside
// that walk's chain have the time for (train step at B=8 H=16 T=4096 d=128: walk back 341
// -> 317 us; forward those waves form o, and with both matrices so the walk went from 232 to
// 258 us).  What the queries take goes in fp32 too where rows are bf16 (256 heads of 2048
// tokens of 64, whole call: 222 -> 205 us); fp32 walks' LDS takes both as they come.
// Logarithms of the forget factors are summed in 64 bits, so that a ratio c_t / c_j keeps
// fp32's precision however strong the decay before it.
//
// Memory bounds it where there are many chunks: at B=1 H=16 T=32768 d=128 bf16 99 to 107 us for
// 0.52 GB forward (4.8 to 5.2 TB/s; a large copy 4.9), at B=8 H=16 T=4096 168 to 174 us for 0.96 GB
// for both.  One round of chunks is a chain of 6.5 us (fp32 9): loads 1, logarithms 1, products and
// decays 2, the diagonal blocks 1, the others and the way out 1.5.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

constexpr int kLd = 20;  // floats of a 16-wide row in LDS

__host__ __device__ constexpr int tile_of(int i, int j) { return i * (i + 1) / 2 + j; }

// BOTH: the walk back's matrices too, by workgroups behind the others.  (In place of a launch of
// their own: 6 to 8 us less a training step of few chunks; B=8 H=16 T=4096 d=128 184 us and 197.
// The body is a lambda: as a function of the parameters it spilled 92 registers back.)
template <int DK, bool BF16, bool BOTH>
__global__ __launch_bounds__(256, BF16 || DK == 32 ? 4 : 2) void delta_chunk_kernel(DeltaParams p, uint32_t units) {
  auto form = [&](auto transposed, uint32_t unit) {
    constexpr bool TRANSPOSED = transposed();
    constexpr int ES = BF16 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float low[10][16 * kLd];
    __shared__ __attribute__((aligned(16))) float diag[4][16 * kLd];
    __shared__ double sg[kDeltaChunk];
    __shared__ float sbeta[kDeltaChunk];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const uint32_t bh = unit / p.by_nc;
    const int c = unit % p.by_nc, b = bh / p.by_h, h = bh % p.by_h, hk = (uint32_t)h / p.by_shared;
    const int live = min(delta_length(p, b) - c * kDeltaChunk, kDeltaChunk);
    if (live <= 0) return;

    // 16 rows of 8 columns a lane group at a time
    auto rows = [&](const DeltaRows& x, int i, u32x4 (&f)[DK / 32][BF16 ? 1 : 2]) {
      const int64_t first = b * x.b + hk * x.h + (int64_t)(c * kDeltaChunk) * x.t;
      const Window from = window_at(static_cast<const char*>(x.at) + first * ES);
      const uint32_t at = 16 * i + r < live ? ((16 * i + r) * (uint32_t)x.t + 8 * g) * ES : kNowhere;
#pragma unroll
      for (int s = 0; s < DK / 32; ++s)
#pragma unroll
        for (int n = 0; n < (BF16 ? 1 : 2); ++n) f[s][n] = window_load(from, at, 32 * s * ES + 16 * n);
    };
    auto planes = [&](const u32x4 (&f)[BF16 ? 1 : 2]) {
      if constexpr (BF16) {
        Planes<1> x;
        x.p[0] = __builtin_bit_cast(bf16x8, f[0]);
        return x;
      } else {
        return split8<3>(__builtin_bit_cast(f32x4, f[0]), __builtin_bit_cast(f32x4, f[1]));
      }
    };
    u32x4 k_raw[4][DK / 32][BF16 ? 1 : 2], q_raw[DK / 32][BF16 ? 1 : 2];
    rows(p.k, wave, k_raw[3]);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < wave) rows(p.k, j, k_raw[j]);
    rows(p.q, wave, q_raw);

    // gates: one token a lane, the same in every wave
    double lg = 0.0;
    float beta = 0.f;
    if (lane < live) {
      const int64_t t = c * kDeltaChunk + lane;
      lg = log2((double)*gate_at(p.gamma, b, h, t));
      if (lg < -16384.0) lg = -16384.0;  // a factor of 0 ends what came before; a NaN or a negative one's stays NaN
      beta = *gate_at(p.beta, b, h, t);
    }
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const double before = __shfl_up(lg, off);
      if (lane >= off) lg += before;
    }
    if (wave == 0) {
      sg[lane] = lg;
      sbeta[lane] = beta;
      if constexpr (!TRANSPOSED) {
        DeltaGates& out = p.gates[unit];
        out.g[lane] = lg;
        out.c[lane] = decay_exact(lg, 0.0);
        out.tail[lane] = decay_exact(__shfl(lg, 63), lg);
        out.beta[lane] = beta;
      }
    }
    __syncthreads();

    char* const to = (TRANSPOSED ? p.matrices_t + (int64_t)unit * (2 * kTriangleBytes)
                                 : p.matrices + (int64_t)unit * delta_matrix_bytes(BF16)) + lane * 16;
    auto put_tile = [&](int matrix, int i, int j, const f32x4& x) {
      *reinterpret_cast<f32x4*>(to + matrix * kTriangleBytes + triangle_tile<false>(i, j) * 1024) = x;
    };
    // A block's two tiles, in parts, to its place
    auto put = [&](int matrix, int block, const f32x4& lo, const f32x4& hi) {
      const Planes<3> f = split8<3>(lo, hi);
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *reinterpret_cast<bf16x8*>(to + (matrix * 3 + n) * kBlocksBytes + block * 1024) = f.p[n];
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    // Row tile `wave`: keys with keys, and queries with keys (a lane has one query and 4 keys of
    // a tile, transposed the other way round).
    f32x4 kk[4] = {zero, zero, zero, zero}, a[4] = {zero, zero, zero, zero};  // [3]: the diagonal tile
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const auto own = planes(k_raw[3][s]);
      const auto q = planes(q_raw[s]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < 3 && j >= wave) continue;
        const auto k = planes(k_raw[j][s]);
        kk[j] = mma<2>(own, k, kk[j]);
        a[j] = TRANSPOSED ? mma<2>(q, k, a[j]) : mma<2>(k, q, a[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < 3 && j >= wave) continue;
      const int tile = j < 3 ? j : wave, col = 16 * tile + r;
      const double gj = sg[col];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * wave + 4 * g + e;
        const float d = decay(sg[t], gj);
        const float x = kk[j][e] * d * (TRANSPOSED ? sbeta[t] : sbeta[col]);
        low[tile_of(wave, tile)][(4 * g + e) * kLd + r] = col < t ? x : 0.f;
        if constexpr (TRANSPOSED) {
          a[j][e] = col <= t ? a[j][e] * d : 0.f;
        } else {
          const int at_t = 16 * wave + r, at_j = 16 * tile + 4 * g + e;
          a[j][e] = at_j <= at_t ? a[j][e] * decay(sg[at_t], sg[at_j]) : 0.f;
        }
      }
    }
    if constexpr (!TRANSPOSED) {
      const f32x4 d = a[3];
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j == 3 || j < wave)
            *reinterpret_cast<f32x4*>(to + 3 * kBlocksBytes + triangle_tile<true>(wave, j < 3 ? j : wave) * 1024) = a[j];
      } else {
        if (wave == 0) put(1, lower_block(0, 0), d, zero);
        else put(1, lower_block(wave, 0), a[0], wave == 1 ? d : a[1]);
        if (wave >= 2) put(1, lower_block(wave, 1), wave == 2 ? d : a[2], wave == 2 ? zero : d);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < wave) put_tile(1, j, wave, a[j]);
      put_tile(1, wave, wave, a[3]);
    }
    __syncthreads();

    {  // diagonal block `wave`, lane r (of each lane group) its column r
      const float* l = low[tile_of(wave, wave)];
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == r ? 1.f : 0.f;
#pragma unroll
        for (int m4 = 0; m4 < i; m4 += 4) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(l + i * kLd + m4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m4 + e < i) s = fmaf(-v[e], x[m4 + e], s);
        }
        x[i] = s;
      }
      if (g == 0)
#pragma unroll
        for (int i = 0; i < 16; ++i) diag[wave][i * kLd + r] = x[i];
    }
    __syncthreads();

    f32x4 t[4];  // T_ij of column j = wave, rows 4 g + e, column r
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = zero;
      if (i < wave) continue;
      if (i == wave) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[i][e] = diag[i][(4 * g + e) * kLd + r];
        continue;
      }
      f32x4 acc = zero, out = zero;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m < wave || m >= i) continue;
        const f32x4 x = *reinterpret_cast<const f32x4*>(&low[tile_of(i, m)][r * kLd + 4 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma_f32(x[e], t[m][e], acc);
      }
      const f32x4 d = *reinterpret_cast<const f32x4*>(&diag[i][r * kLd + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) out = mfma_f32(d[e], acc[e], out);
      t[i] = -out;
    }

    // a lane's 4 numbers lie along the later product's inner index: rows of the
    // transposed inverse as they are, rows of the inverse by way of LDS
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i >= wave) put_tile(0, wave, i, t[i]);
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < wave) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) low[tile_of(i, wave)][(4 * g + e) * kLd + r] = t[i][e];
      }
      __syncthreads();
      auto row = [&](int j) { return *reinterpret_cast<const f32x4*>(&low[tile_of(wave, j)][r * kLd + 4 * g]); };
      put(0, lower_block(wave, 0), row(0), wave >= 1 ? row(1) : zero);
      if (wave >= 2) put(0, lower_block(wave, 1), row(2), wave == 3 ? row(3) : zero);
    }
  };
  if (!BOTH || blockIdx.x < units) form(std::false_type{}, blockIdx.x);
  else if constexpr (BOTH) form(std::true_type{}, blockIdx.x - units);
}

template <int DK, bool BF16>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  const uint32_t units = (uint32_t)((int64_t)p.B * p.H * p.NC);
  if (p.matrices_t) delta_chunk_kernel<DK, BF16, true><<<2 * units, 256, 0, s>>>(p, units);
  else delta_chunk_kernel<DK, BF16, false><<<units, 256, 0, s>>>(p, units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunks(bool bf16, const DeltaParams& p, hipStream_t s) {
  if (p.dk == 128) return bf16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  if (p.dk == 64) return bf16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  return bf16 ? launch<32, true>(p, s) : launch<32, false>(p, s);
}

}  // namespace mesa
