// Gradient of the query/key preprocessing (MesaNet page, "architecture": queries
// and keys convolved with a small causal window and normalised),
//     y_t[j] = sum_{i < W} w[h][j][i] x_{t-i}[j],   out_t = y_t / max(||y_t||, eps):
//     e_t = (d_t - o <o, d_t>) / n  where n = ||y_t|| > eps, else d_t / eps,
//     dx_s = sum_i w_i e_{s+i},   dw[h][j][i] = sum_{b,t} e_t[j] x_{t-i}[j].
#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_prep_rows.h"

namespace mesa {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void store1(void* base, size_t idx, float v) {
  if constexpr (BF16) {
    static_cast<uint16_t*>(base)[idx] = __builtin_bit_cast(uint16_t, f32_to_bf16(v));
  } else {
    static_cast<float*>(base)[idx] = v;
  }
}

// Raw channel j of row r >= -(W-1) of sequence bh.
template <bool BF16>
__device__ __forceinline__ float raw_at(const PrepBwdParams& p, int which, int D, int bh, int r, int j) {
  if (r >= 0) return load1<BF16>(p.x[which], ((size_t)bh * p.T + r) * D + j);
  if (!p.hist_in[which]) return 0.f;
  return load1<BF16>(p.hist_in[which], ((size_t)bh * (p.W - 1) + (p.W - 1 + r)) * D + j);
}

// e_t, one lane per token, into part [2, BH, T, D].
template <bool BF16>
__global__ __launch_bounds__(kThreads) void prep_bwd_e_kernel(PrepBwdParams p, int D) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int which = blockIdx.y;
  if (i >= (long long)p.BH * p.T) return;
  const int bh = (int)(i / p.T), t = (int)(i % p.T), h = bh % p.H;
  auto conv = [&](int j) {
    float y = 0.f;
    for (int k = 0; k < p.W; ++k) y += p.w[which][((size_t)h * D + j) * p.W + k] * raw_at<BF16>(p, which, D, bh, t - k, j);
    return y;
  };
  const float* d = p.d[which] + (size_t)i * D;
  float ss = 0.f, dot = 0.f;
  for (int j = 0; j < D; ++j) {
    const float y = conv(j);
    ss += y * y;
    dot += y * d[j];
  }
  const float scale = prep_scale(ss, p.inv_eps);
  const float k = scale < p.inv_eps ? dot * scale * scale : 0.f;
  float* e = p.part + ((size_t)which * p.BH * p.T + i) * D;
  for (int j = 0; j < D; ++j) e[j] = scale * (d[j] - conv(j) * k);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void prep_bwd_dx_kernel(PrepBwdParams p, int D) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int which = blockIdx.y, rows = p.T + p.W - 1;
  if (i >= (long long)p.BH * rows * D) return;
  const int j = (int)(i % D), r = (int)((i / D) % rows) - (p.W - 1), bh = (int)(i / ((long long)D * rows)), h = bh % p.H;
  float v = 0.f;
  for (int k = 0; k < p.W; ++k)
    if (r + k >= 0 && r + k < p.T)
      v += p.w[which][((size_t)h * D + j) * p.W + k] * p.part[(((size_t)which * p.BH + bh) * p.T + r + k) * D + j];
  const int q = r - (p.T - (p.W - 1));  // row of the history output this is a copy in
  if (q >= 0 && p.d_hist[which]) v += load1<BF16>(p.d_hist[which], ((size_t)bh * (p.W - 1) + q) * D + j);
  if (r >= 0) store1<BF16>(p.dx[which], ((size_t)bh * p.T + r) * D + j, v);
  else if (p.dhist[which]) store1<BF16>(p.dhist[which], ((size_t)bh * (p.W - 1) + (p.W - 1 + r)) * D + j, v);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void prep_bwd_dw_kernel(PrepBwdParams p, int D) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int which = blockIdx.y;
  if (i >= p.H * D * p.W) return;
  const int k = i % p.W, j = (i / p.W) % D, h = i / (p.W * D);
  float s = 0.f;
  for (int bh = h; bh < p.BH; bh += p.H)
    for (int t = 0; t < p.T; ++t)
      s += p.part[(((size_t)which * p.BH + bh) * p.T + t) * D + j] * raw_at<BF16>(p, which, D, bh, t - k, j);
  p.dw[which][i] = s;
}

template <bool BF16>
hipError_t launch_t(int D, const PrepBwdParams& p, hipStream_t s) {
  auto grid = [](long long n) { return dim3((unsigned)((n + kThreads - 1) / kThreads), 2); };
  if (p.T > 0) {
    hipLaunchKernelGGL((prep_bwd_e_kernel<BF16>), grid((long long)p.BH * p.T), dim3(kThreads), 0, s, p, D);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (p.T + p.W > 1) {
    hipLaunchKernelGGL((prep_bwd_dx_kernel<BF16>), grid((long long)p.BH * (p.T + p.W - 1) * D), dim3(kThreads), 0, s, p, D);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((prep_bwd_dw_kernel<BF16>), grid((long long)p.H * D * p.W), dim3(kThreads), 0, s, p, D);
  return hipGetLastError();
}

}  // namespace

size_t qk_prep_bwd_scratch(int BH, int T, int D, int) { return (size_t)2 * BH * T * D * 4; }

hipError_t launch_qk_prep_bwd(bool bf16, int D, const PrepBwdParams& p, hipStream_t s) {
  return bf16 ? launch_t<true>(D, p, s) : launch_t<false>(D, p, s);
}

}  // namespace mesa
