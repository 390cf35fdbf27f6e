// Residual addition and RMS norm of token rows, with a plain or an e4m3 output,
// and its gradient (MesaNet page, "architecture": the residual blocks' norm).
//     s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = w s r
//     ds = r (g - n mean(g n)) + d_residual,  g = dy w,  n = s r,  dw = sum_rows dy n
#include "mesa_common.h"
#include "mesa_kernels.h"

namespace mesa {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-100f;
constexpr int kGroup = 128;

template <bool BF16>
__device__ __forceinline__ void store1(void* base, size_t idx, float v) {
  if constexpr (BF16) {
    static_cast<uint16_t*>(base)[idx] = __builtin_bit_cast(uint16_t, f32_to_bf16(v));
  } else {
    static_cast<float*>(base)[idx] = v;
  }
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  v = fminf(fmaxf(v, -kE4m3Max), kE4m3Max);
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false);
}

__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kThreads / 64; ++i) s += lds[i];
  return s;
}

// One workgroup per row, every pass over the row re-reading it.
template <bool BF16, bool RBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_kernel(NormParams p) {
  __shared__ float lds[kThreads];
  const size_t row = blockIdx.x;
  auto at = [&](int c) {
    float v = load1<BF16>(p.x, row * p.D + c);
    if (p.residual) v += load1<RBF16>(p.residual, row * p.D + c);
    return v;
  };
  float ss = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kThreads) ss = __builtin_fmaf(at(c), at(c), ss);
  const float r = 1.f / sqrtf(block_sum(ss, lds) / p.D + p.eps);
  const int group = p.group ? p.group : p.D;
  for (int g0 = 0; g0 < p.D; g0 += group) {
    const int g1 = min(g0 + group, p.D);
    float inv = 1.f;
    if (p.e4m3) {
      float m = 0.f;
      for (int c = g0 + threadIdx.x; c < g1; c += kThreads) m = fmaxf(m, fabsf(at(c) * r * p.w[c]));
      __syncthreads();
      lds[threadIdx.x] = m;
      __syncthreads();
      m = kAmaxFloor;
      for (int i = 0; i < kThreads; ++i) m = fmaxf(m, lds[i]);
      inv = kE4m3Max / m;
      if (threadIdx.x == 0) p.scale[row * ((p.D + group - 1) / group) + g0 / group] = m / kE4m3Max;
    }
    for (int c = g0 + threadIdx.x; c < g1; c += kThreads) {
      const float v = at(c), y = v * r * p.w[c];
      if (p.e4m3) static_cast<uint8_t*>(p.y)[row * p.D + c] = to_e4m3(y * inv);
      else store1<BF16>(p.y, row * p.D + c, y);
      if (p.residual_out) store1<RBF16>(p.residual_out, row * p.D + c, v);
    }
  }
}

template <bool BF16, bool RBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_bwd_kernel(NormParams p) {
  __shared__ float lds[kThreads];
  const size_t row = blockIdx.x;
  float ss = 0.f, gs = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const float v = load1<RBF16>(p.x, row * p.D + c);
    ss = __builtin_fmaf(v, v, ss);
    gs = __builtin_fmaf(load1<BF16>(p.dy, row * p.D + c) * p.w[c], v, gs);
  }
  const float r = 1.f / sqrtf(block_sum(ss, lds) / p.D + p.eps);
  const float k = block_sum(gs, lds) * r / p.D;  // mean(g n)
  if (threadIdx.x == 0) static_cast<float*>(p.part)[row] = r;
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    const size_t e = row * p.D + c;
    const float n = load1<RBF16>(p.x, e) * r;
    float v = r * (load1<BF16>(p.dy, e) * p.w[c] - n * k);
    if (p.residual) v += load1<RBF16>(p.residual, e);
    store1<RBF16>(p.y, e, v);
    if (p.residual_out) store1<BF16>(p.residual_out, e, v);
  }
}

template <bool BF16, bool RBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_dw_kernel(NormParams p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.D) return;
  float s = 0.f;
  for (int row = 0; row < p.R; ++row) {
    const size_t e = (size_t)row * p.D + c;
    s += load1<BF16>(p.dy, e) * load1<RBF16>(p.x, e) * static_cast<const float*>(p.part)[row];
  }
  p.dw[c] = s;
}

template <bool BF16, bool RBF16>
hipError_t launch_bwd_t(const NormParams& p, hipStream_t s) {
  if (p.R > 0) {
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, RBF16>), dim3(p.R), dim3(kThreads), 0, s, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((rmsnorm_dw_kernel<BF16, RBF16>), dim3((p.D + kThreads - 1) / kThreads), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_scratch(int R, int) { return (size_t)R * 4; }

hipError_t launch_rmsnorm(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  const dim3 grid(p.R), block(kThreads);
  if (!bf16) hipLaunchKernelGGL((rmsnorm_kernel<false, false>), grid, block, 0, s, p);
  else if (res_bf16) hipLaunchKernelGGL((rmsnorm_kernel<true, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((rmsnorm_kernel<true, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  if (!bf16) return launch_bwd_t<false, false>(p, s);
  return res_bf16 ? launch_bwd_t<true, true>(p, s) : launch_bwd_t<true, false>(p, s);
}

}  // namespace mesa
