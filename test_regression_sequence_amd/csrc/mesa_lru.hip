// Gated linear recurrence: h_t = a_t h_{t-1} + u_t per channel, with decay and
// input from the token's gates (mesa_lru_gate.h).
#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_lru_gate.h"

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

__device__ __forceinline__ int lru_length(const LruParams& p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// One lane per channel of a sequence, walking its tokens.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void lru_fwd_kernel(LruParams p) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)p.B * p.D) return;
  const int b = (int)(i / p.D), ch = (int)(i % p.D);
  const int n = lru_length(p, b);
  const float rate = lru_rate(p.lam[ch], p.c);
  float h = p.h0 ? p.h0[i] : 0.f;
  for (int t = 0; t < p.T; ++t) {
    if (t % kLruChunk == 0) p.states[((size_t)b * p.NC + t / kLruChunk) * p.D + ch] = h;
    float out = 0.f;
    if (t < n) {
      const size_t e = ((size_t)b * p.T + t) * p.ld + ch;
      float a, u;
      lru_cell(load1<BF16>(p.x, e), load1<BF16>(p.ga, e), load1<BF16>(p.gi, e), rate, a, u);
      h = __builtin_fmaf(a, h, u);
      out = h;
    }
    if (p.y) store1<BF16>(p.y, ((size_t)b * p.T + t) * p.D + ch, out);
  }
  if (p.h_final) p.h_final[i] = h;
}

// The same lanes, chunks backwards: each chunk's states are walked again from
// the state before it, then its gradients from the last token to the first.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void lru_bwd_kernel(LruParams p) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)p.B * p.D) return;
  const int b = (int)(i / p.D), ch = (int)(i % p.D);
  const int n = lru_length(p, b);
  const float rate = lru_rate(p.lam[ch], p.c);
  float g = p.d_hfinal ? p.d_hfinal[i] : 0.f;  // adjoint of the state behind the token
  float vsum = 0.f;
  float before[kLruChunk];
  for (int c = p.NC - 1; c >= 0; --c) {
    const int t0 = c * kLruChunk;
    float h = p.states[((size_t)b * p.NC + c) * p.D + ch];
    for (int s = 0; s < kLruChunk && t0 + s < n; ++s) {
      const size_t e = ((size_t)b * p.T + t0 + s) * p.ld + ch;
      float a, u;
      before[s] = h;
      lru_cell(load1<BF16>(p.x, e), load1<BF16>(p.ga, e), load1<BF16>(p.gi, e), rate, a, u);
      h = __builtin_fmaf(a, h, u);
    }
    for (int s = min(kLruChunk, p.T - t0) - 1; s >= 0; --s) {
      const size_t row = (size_t)b * p.T + t0 + s, eg = row * p.ld_grad + ch;
      float dx = 0.f, dga = 0.f, dgi = 0.f;
      if (t0 + s < n) {
        const size_t e = row * p.ld + ch;
        const LruGrad r = lru_cell_grad(load1<BF16>(p.x, e), load1<BF16>(p.ga, e), load1<BF16>(p.gi, e), rate);
        g += load1<BF16>(p.dy, row * p.D + ch);
        const float v = g * __builtin_fmaf(-r.v_a, before[s], r.v_u);
        vsum += v;
        dx = g * r.dx_g;
        dgi = g * r.dgi_g;
        dga = v * r.sr1;
        g *= r.a;
      }
      store1<BF16>(p.dx, eg, dx);
      store1<BF16>(p.dga, eg, dga);
      store1<BF16>(p.dgi, eg, dgi);
    }
  }
  if (p.lam_part) p.lam_part[i] = vsum;  // (no tokens, no workspace: nothing to add)
  if (p.dh0) p.dh0[i] = g;
}

// dlam[ch] from `rows` partial sums [rows, D] of dL / d log w.
__global__ __launch_bounds__(kThreads) void lru_dlam_kernel(const float* part, const float* lam, float* dlam, int rows,
                                                            int D) {
  const int ch = blockIdx.x * kThreads + threadIdx.x;
  if (ch >= D) return;
  float s = 0.f;
  for (int r = 0; r < rows; ++r) s += part[(size_t)r * D + ch];
  dlam[ch] = s * lru_rate_slope(lam[ch]);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void lru_step_kernel(LruParams p) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)p.B * p.D) return;
  const long long n = i / p.D;
  const int ch = (int)(i % p.D);
  const size_t e = (size_t)n * p.ld + ch;
  float a, u;
  lru_cell(load1<BF16>(p.x, e), load1<BF16>(p.ga, e), load1<BF16>(p.gi, e), lru_rate(p.lam[ch], p.c), a, u);
  const float h = __builtin_fmaf(a, p.h_final[i], u);
  p.h_final[i] = h;
  store1<BF16>(p.y, i, h);
}

unsigned blocks(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_lru_fwd(bool bf16, const LruParams& p, hipStream_t s) {
  const dim3 grid(blocks((long long)p.B * p.D));
  if (bf16) hipLaunchKernelGGL((lru_fwd_kernel<true>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((lru_fwd_kernel<false>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_lru_bwd(bool bf16, const LruParams& p, hipStream_t s) {
  const dim3 grid(blocks((long long)p.B * p.D));
  if (bf16) hipLaunchKernelGGL((lru_bwd_kernel<true>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((lru_bwd_kernel<false>), grid, dim3(kThreads), 0, s, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL(lru_dlam_kernel, dim3(blocks(p.D)), dim3(kThreads), 0, s, p.lam_part, p.lam, p.dlam,
                     p.lam_part ? p.B : 0, p.D);
  return hipGetLastError();
}

hipError_t launch_lru_step(bool bf16, const LruParams& p, hipStream_t s) {
  const dim3 grid(blocks((long long)p.B * p.D));
  if (bf16) hipLaunchKernelGGL((lru_step_kernel<true>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((lru_step_kernel<false>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace mesa
