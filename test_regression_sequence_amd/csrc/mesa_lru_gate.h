// The gates of the linear recurrence (MesaNet page, "architecture": the layer
// that alternates with the Mesa layer in the Hawk-Mesa hybrid), one channel of
// one token:
//     s_r = sigmoid(ga),  s_i = sigmoid(gi),  w = 2 c softplus(lam) s_r = -2 log a,
//     a = exp(-w/2),  m = sqrt(1 - a^2) = sqrt(1 - exp(-w)).
// Every kernel of the recurrence forms them with these helpers, in fp32.
#pragma once

#include "mesa_common.h"

namespace mesa {

constexpr float kLog2e = 1.44269504088896340736f;

// 2 c softplus(lam), in fp32: softplus(z) = max(z, 0) + log(1 + exp(-|z|)).
__device__ __forceinline__ float lru_rate(float lam, float c) {
  return 2.f * c * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));
}

// sigmoid(lam) / softplus(lam), the factor from dL/d log w to dL/dlam.  Below
// lam = -15 both are exp(lam) to within exp(-15) = 3e-7 of themselves, and
// their quotient is 1 - exp(lam)/2 to first order.
__device__ __forceinline__ float lru_rate_slope(float lam) {
  if (lam < -15.f) return 1.f - 0.5f * expf(lam);
  return 1.f / ((1.f + expf(-lam)) * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam)))));
}

__device__ __forceinline__ float lru_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// 1 - exp(-w) for w >= 0, given a = exp(-w/2).  Above w = 1/4, 1 - a^2 keeps
// all but two bits.  Below it the difference would cancel, so the alternating
// series w (1 - w/2 + w^2/6 - ...) is summed to w^5/720: the first term left
// out is below w^6/5040 = 5e-8 of the value.  Both are formed and one selected:
// marked unpredictable, or the compiler makes a branch of every element.
__device__ __forceinline__ float lru_one_minus_a2(float w, float a) {
  float p = __builtin_fmaf(w, -1.f / 720.f, 1.f / 120.f);
  p = __builtin_fmaf(w, p, -1.f / 24.f);
  p = __builtin_fmaf(w, p, 1.f / 6.f);
  p = __builtin_fmaf(w, p, -0.5f);
  p = __builtin_fmaf(w, p, 1.f);
  const float series = w * p, direct = __builtin_fmaf(-a, a, 1.f);
  return __builtin_unpredictable(w < 0.25f) ? series : direct;
}

// Decay a and input u of one token: h_t = a h_{t-1} + u.
__device__ __forceinline__ void lru_cell(float x, float ga, float gi, float rate, float& a, float& u) {
  const float w = rate * lru_sigmoid(ga);
  a = __builtin_amdgcn_exp2f((-0.5f * kLog2e) * w);
  u = __builtin_amdgcn_sqrtf(lru_one_minus_a2(w, a)) * lru_sigmoid(gi) * x;
}

// The same with what the gradients need.  With g the adjoint of h_t and h1 the
// state before the token:
//     dx = g dx_g,  dgi = dx q,  v = g (v_u - v_a h1),  dga = v sr1,
// q = x (1 - s_i), v = dL / d log w = (w/2) g ((a^2/m) s_i x - a h1); the input
// is u = dx_g x.
struct LruGrad {
  float a, dx_g, q, v_u, v_a, sr1;
};

// 1 - sigmoid comes as exp(-z) sigmoid(z), which keeps its bits for large z;
// the exponent is capped at 126 so that exp(-z) stays finite (there sigmoid is
// 2^-126 and its complement 1).  1/m is the reciprocal square root of 1 - a^2
// raised to the smallest normal float: at w = 0 every gradient through a is
// then w times a finite number, 0.
__device__ __forceinline__ LruGrad lru_cell_grad(float x, float ga, float gi, float rate) {
  LruGrad r;
  const float er = __builtin_amdgcn_exp2f(fminf(-kLog2e * ga, 126.f));
  const float ei = __builtin_amdgcn_exp2f(fminf(-kLog2e * gi, 126.f));
  const float sr = __builtin_amdgcn_rcpf(1.f + er), si = __builtin_amdgcn_rcpf(1.f + ei);
  const float w = rate * sr;
  r.a = __builtin_amdgcn_exp2f((-0.5f * kLog2e) * w);
  const float m2 = lru_one_minus_a2(w, r.a);
  const float rm = __builtin_amdgcn_rsqf(fmaxf(m2, 0x1p-126f));
  const float m = m2 * rm;
  r.sr1 = er * sr;
  r.dx_g = m * si;
  r.q = x * (ei * si);
  const float wa = 0.5f * w * r.a;
  r.v_a = wa;
  r.v_u = wa * r.a * rm * (si * x);
  return r;
}

}  // namespace mesa
