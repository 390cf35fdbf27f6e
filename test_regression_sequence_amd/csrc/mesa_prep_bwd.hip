// Gradient of the query/key preprocessing (MesaNet page, "architecture": queries
// and keys convolved with a small causal window and normalised),
//     y_t[j] = sum_{i < W} w[h][j][i] x_{t-i}[j],   out_t = y_t / max(||y_t||, eps):
//     e_t = (d_t - o <o, d_t>) / n  where n = ||y_t|| > eps, else d_t / eps,
//     dx_s = sum_i w_i e_{s+i},   dw[h][j][i] = sum_{b,t} e_t[j] x_{t-i}[j].
//
// Bound by HBM: raw rows and incoming gradients are read once, raw gradients
// written once.  As in the forward kernel a row is spread over D/8 lanes with 8
// channels each.  A lane group walks `Steps` consecutive tokens with the last W
// raw rows and the W open dx rows in registers: token t's e is formed from the
// window, added to the rows t-W+1 .. t, and the first of them is complete.  The
// first tokens a group walks are its own; the W-1 behind them are the next
// group's and only complete this group's rows, so (W-1)/Steps of the work is
// done twice.  Loads run one block of tokens ahead.  dw is summed per lane over its
// at most 29 to 32 tokens in fp32, per workgroup through LDS and over workgroups by a
// second kernel in 64 bits (in fp32 the error grew with the sequences: 480 half
// steps over 2^15 equal ones at d=16), all in a fixed order.  At B=8, H=16, T=4096,
// d=128, W=4, bf16: 222 us, 1.19 GB at 5.4 TB/s, of which 0.11 GB are rows that two
// groups read.
#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_prep_rows.h"
#include "mesa_rows.h"

namespace mesa {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 4;  // tokens loaded together

template <int D, int W, int STEPS>
struct PrepBwdShape {
  static constexpr int LPR = D / 8;             // lanes per token row
  static constexpr int NG = kThreads / LPR;     // lane groups of a workgroup
  static constexpr int S = STEPS - (W - 1);     // own tokens of a group
  static constexpr int TILE = NG * S;           // own tokens of a workgroup
  static_assert(STEPS % kBlock == 0 && S > 0, "whole blocks");
};

template <bool BF16, int D, int W, int STEPS>
__global__ __launch_bounds__(kThreads) void prep_bwd_kernel(PrepBwdParams p) {
  using Sh = PrepBwdShape<D, W, STEPS>;
  constexpr int LPR = Sh::LPR, S = Sh::S;
  __shared__ float sums[Sh::NG][D * W];
  const int which = blockIdx.z, bh = blockIdx.y, h = bh % p.H, T = p.T;
  const int group = threadIdx.x / LPR, c0 = 8 * (threadIdx.x % LPR);
  const int t0 = (blockIdx.x * Sh::NG + group) * S;
  float w[8][W], dw[8][W] = {};
  prep_taps8<W>(p.w[which], h, D, c0, w);

  if (t0 < T) {
    const size_t seq = (size_t)bh * T * D + c0;
    const void* hist = p.hist_in[which];
    Raw8<BF16> x[kBlock], win[W];  // win[m]: raw row t-(W-1)+m
    Raw8<false> d[kBlock];
    auto load = [&](int t) {  // rows behind the sequence read its last row and are not used
#pragma unroll
      for (int u = 0; u < kBlock; ++u) {
        const size_t e = seq + (size_t)min(t + u, T - 1) * D;
        x[u] = load_raw8<BF16>(p.x[which], e);
        d[u] = load_raw8<false>(p.d[which], e);
      }
    };
    load(t0);
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
      const int r = t0 - (W - 1) + m;
      if (r >= 0) win[m] = load_raw8<BF16>(p.x[which], seq + (size_t)r * D);
      else if (hist) win[m] = load_raw8<BF16>(hist, ((size_t)bh * (W - 1) + (W - 1 + r)) * D + c0);
      else win[m] = Raw8<BF16>{};
    }
    float acc[W][8] = {};  // acc[m]: dx of row t-(W-1)+m so far
    for (int t = t0; t < t0 + STEPS; t += kBlock) {
      Raw8<BF16> xc[kBlock];
      Raw8<false> dc[kBlock];
#pragma unroll
      for (int u = 0; u < kBlock; ++u) {
        xc[u] = x[u];
        dc[u] = d[u];
      }
      if (t + kBlock < t0 + STEPS) load(t + kBlock);
#pragma unroll
      for (int u = 0; u < kBlock; ++u) {
        const int tt = t + u;
        win[W - 1] = xc[u];
        float x8[W][8], y[8], e[8];
#pragma unroll
        for (int m = 0; m < W; ++m)
#pragma unroll
          for (int c = 0; c < 8; ++c) x8[m][c] = win[m].at(c);
        float ss = prep_conv8<W>(w, x8, y), dot = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) dot = __builtin_fmaf(y[c], dc[u].at(c), dot);
        ss = group_sum<LPR>(ss);
        dot = group_sum<LPR>(dot);
        const bool own = tt < t0 + S, some = tt < T;
        float scale = some ? prep_scale(ss, p.inv_eps) : 0.f;
        if (some && ss != ss) scale = ss;  // (the minimum in prep_scale loses a NaN: the row would count as below eps)
        const float k = scale < p.inv_eps ? dot * scale * scale : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          e[c] = some ? scale * __builtin_fmaf(-y[c], k, dc[u].at(c)) : 0.f;
#pragma unroll
          for (int i = 0; i < W; ++i) acc[W - 1 - i][c] = __builtin_fmaf(w[c][i], e[c], acc[W - 1 - i][c]);
        }
        if (own) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int i = 0; i < W; ++i) dw[c][i] = __builtin_fmaf(e[c], x8[W - 1 - i][c], dw[c][i]);
        }
        // row s is complete
        const int s = tt - (W - 1);
        if (s < T && (s >= t0 || (t0 == 0 && p.dhist[which]))) {
          const int q = s - (T - (W - 1));  // the row of the history output that row s is copied to
          if (q >= 0 && p.d_hist[which]) {
            const Raw8<BF16> v = load_raw8<BF16>(p.d_hist[which], ((size_t)bh * (W - 1) + q) * D + c0);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[0][c] += v.at(c);
          }
          if (s >= t0) store_raw8<BF16, false>(p.dx[which], seq + (size_t)s * D, acc[0], 8);
          else store_raw8<BF16, false>(p.dhist[which], ((size_t)bh * (W - 1) + (W - 1 + s)) * D + c0, acc[0], 8);
        }
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {
          win[m] = win[m + 1];
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[m][c] = acc[m + 1][c];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[W - 1][c] = 0.f;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int i = 0; i < W; ++i) sums[group][(c0 + c) * W + i] = dw[c][i];
  __syncthreads();
  float* part = p.part + (((size_t)which * p.BH + bh) * gridDim.x + blockIdx.x) * (D * W);
  for (int i = threadIdx.x; i < D * W; i += kThreads) {
    double v = 0.;
#pragma unroll 8
    for (int g = 0; g < Sh::NG; ++g) v += sums[g][i];
    part[i] = (float)v;
  }
}

// dw[h][j][i] from the partial sums [2, BH, tiles, n = D W] of the workgroups:
// 16 sums a workgroup, 16 threads a sum over the head's sequences and tiles.
__global__ __launch_bounds__(256) void prep_bwd_dw_kernel(PrepBwdParams p, int tiles, int n) {
  __shared__ double sums[16][16];
  const int k = threadIdx.x % 16, slice = threadIdx.x / 16, i = blockIdx.x * 16 + k, h = blockIdx.y, which = blockIdx.z;
  const int rows = p.BH / p.H * tiles;  // (n is a multiple of 16)
  double v = 0.;
#pragma unroll 4
  for (int r = slice; r < rows; r += 16) {
    const size_t bh = (size_t)(r / tiles) * p.H + h;
    v += p.part[(((size_t)which * p.BH + bh) * tiles + r % tiles) * n + i];
  }
  sums[slice][k] = v;
  __syncthreads();
  if (slice == 0) {
    for (int g = 1; g < 16; ++g) v += sums[g][k];
    p.dw[which][(size_t)h * n + i] = (float)v;
  }
}

// Without tokens the history's gradient is that of its copy.
template <bool BF16>
__global__ __launch_bounds__(256) void prep_bwd_empty_kernel(PrepBwdParams p, long long n) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int which = blockIdx.y;
  if (i >= n || !p.dhist[which]) return;
  if constexpr (BF16)
    static_cast<uint16_t*>(p.dhist[which])[i] = p.d_hist[which] ? static_cast<const uint16_t*>(p.d_hist[which])[i] : 0;
  else
    static_cast<float*>(p.dhist[which])[i] = p.d_hist[which] ? static_cast<const float*>(p.d_hist[which])[i] : 0.f;
}

// Tokens that a group walks.  A walk takes the time of its steps one after the
// other, so few rows are walked in short pieces, although then (W-1)/8 of the
// work is done twice.  Short against long walks in us, bf16, W = 4, d = 128, by
// the waves that long walks would take: 9.9 / 22.4 at 72, 22.8 / 25.6 at 576,
// 34.9 / 34.3 at 1136, 60.1 / 61.4 at 2272, 122.9 / 118.5 at 4544; the short
// ones also lose less where a workgroup's rows end behind the sequence (d = 16,
// T = 4096, fp32: 40.8 / 57.2 at 1064).
constexpr int kLong = 32, kShort = 8;

int prep_bwd_tiles(int T, int D, int W, int steps) {
  const long long tile = (long long)(kThreads / (D / 8)) * (steps - (W - 1));
  return (int)((T + tile - 1) / tile);
}

int prep_bwd_steps(int BH, int T, int D, int W) {
  const long long waves = 2LL * BH * ((T + kLong - W) / (kLong - W + 1)) * (D / 8) / 64;
  return waves < 4096 ? kShort : kLong;
}

template <bool BF16, int D, int W>
hipError_t launch_w(const PrepBwdParams& p, hipStream_t s) {
  const int steps = prep_bwd_steps(p.BH, p.T, D, W), tiles = p.T > 0 ? prep_bwd_tiles(p.T, D, W, steps) : 0;
  if (tiles > 0) {
    if (steps == kShort)
      hipLaunchKernelGGL((prep_bwd_kernel<BF16, D, W, kShort>), dim3(tiles, p.BH, 2), dim3(kThreads), 0, s, p);
    else
      hipLaunchKernelGGL((prep_bwd_kernel<BF16, D, W, kLong>), dim3(tiles, p.BH, 2), dim3(kThreads), 0, s, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  } else if (W > 1) {
    const long long n = (long long)p.BH * (W - 1) * D;
    hipLaunchKernelGGL((prep_bwd_empty_kernel<BF16>), dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, s, p, n);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(prep_bwd_dw_kernel, dim3(D * W / 16, p.H, 2), dim3(256), 0, s, p, tiles, D * W);
  return hipGetLastError();
}

template <bool BF16, int D>
hipError_t launch_d(const PrepBwdParams& p, hipStream_t s) {
  switch (p.W) {
    case 1: return launch_w<BF16, D, 1>(p, s);
    case 2: return launch_w<BF16, D, 2>(p, s);
    case 3: return launch_w<BF16, D, 3>(p, s);
    case 4: return launch_w<BF16, D, 4>(p, s);
    default: return hipErrorInvalidValue;
  }
}

template <bool BF16>
hipError_t launch_t(int D, const PrepBwdParams& p, hipStream_t s) {
  switch (D) {
    case 16: return launch_d<BF16, 16>(p, s);
    case 64: return launch_d<BF16, 64>(p, s);
    case 128: return launch_d<BF16, 128>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t qk_prep_bwd_scratch(int BH, int T, int D, int W) {
  return (size_t)2 * BH * prep_bwd_tiles(T, D, W, prep_bwd_steps(BH, T, D, W)) * D * W * sizeof(float);
}

hipError_t launch_qk_prep_bwd(bool bf16, int D, const PrepBwdParams& p, hipStream_t s) {
  return bf16 ? launch_t<true>(D, p, s) : launch_t<false>(D, p, s);
}

}  // namespace mesa
