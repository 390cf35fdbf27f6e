// The gates of the linear recurrence (MesaNet page, "architecture": the layer
// that alternates with the Mesa layer in the Hawk-Mesa hybrid), one channel of
// one token:
//     s_r = sigmoid(ga),  s_i = sigmoid(gi),  t = c log2(e) softplus(lam) s_r,
//     a = 2^-t,  m = sqrt(1 - a^2).
// Every kernel of the recurrence forms them with these helpers, in fp32.
#pragma once

#include "mesa_common.h"

namespace mesa {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// softplus(z) = max(z, 0) + log(1 + e), e = exp(-|z|), good to a few units in the
// last place over its whole range at a sixth of the instructions of the library's
// expf and log1pf (every lane forms it for its channels).  e: the product
// |z| log2(e) is taken in two floats, its rounding error enters to first order.
// log(1 + e) = 2 artanh(q) = 2 (q + q^3/3 + q^5/5 + ..), q = e / (2 + e) <= 1/3:
// the first term left out, q^15/15, is below 2e-8 of the sum.  (fminf and fmaxf
// return the other operand of a NaN; the last term is a selection that keeps it.)
__device__ __forceinline__ float lru_softplus(float z) {
  const float y = fmaxf(-fabsf(z), -150.f), hi = y * kLog2e;  // (exp(-150) is 0 here; an infinite y would give NaN)
  const float lo = __builtin_fmaf(y, 1.92596303e-8f, __builtin_fmaf(y, kLog2e, -hi));  // log2(e) - kLog2e = 1.926e-8
  float e = __builtin_amdgcn_exp2f(hi);
  e = __builtin_fmaf(e, lo * kLn2, e);
  const float q = e * __builtin_amdgcn_rcpf(2.f + e), q2 = q * q;
  float p = __builtin_fmaf(q2, 1.f / 13.f, 1.f / 11.f);
  p = __builtin_fmaf(q2, p, 1.f / 9.f);
  p = __builtin_fmaf(q2, p, 1.f / 7.f);
  p = __builtin_fmaf(q2, p, 1.f / 5.f);
  p = __builtin_fmaf(q2, p, 1.f / 3.f);
  p = __builtin_fmaf(q2, p, 1.f);
  return __builtin_fmaf(2.f * q, p, z < 0.f ? 0.f : z);
}

// c log2(e) softplus(lam): a channel's decay in halvings per token with its gate
// open; finite, so that a closed gate or a decay of 0 leaves no 0 * inf.  (c is
// multiplied last: with log2(e) it may pass the largest float, and times a
// softplus of 0 that would be NaN.)
__device__ __forceinline__ float lru_rate(float lam, float c) {
  const float rate = c * (kLog2e * lru_softplus(lam));
  return rate > 0x1p126f ? 0x1p126f : rate;  // (a NaN stays one)
}

// sigmoid(lam) / softplus(lam), the factor from dL/d log t to dL/dlam.  Below
// lam = -15 both are exp(lam) to within exp(-15) = 3e-7 of themselves, and
// their quotient is 1 - exp(lam)/2 to first order.
__device__ __forceinline__ float lru_rate_slope(float lam) {
  if (lam < -15.f) return 1.f - 0.5f * expf(lam);
  return 1.f / ((1.f + expf(-lam)) * lru_softplus(lam));
}

__device__ __forceinline__ float lru_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// 1 - 2^-2t for t >= 0, given a = 2^-t.  With w = 2 ln2 t, 1 - a^2 keeps all but
// two bits above w = 1/4.  Below it the difference would cancel, so the
// alternating series w (1 - w/2 + w^2/6 - ...) is summed to w^5/720: the first
// term left out is below w^6/5040 = 5e-8 of the value.  Both are formed and one
// selected: marked unpredictable, or the compiler makes a branch of every
// element.
__device__ __forceinline__ float lru_one_minus_a2(float t, float a) {
  constexpr double k = 2 * 0.69314718055994530942;
  float p = __builtin_fmaf(t, (float)(-k * k * k * k * k * k / 720), (float)(k * k * k * k * k / 120));
  p = __builtin_fmaf(t, p, (float)(-k * k * k * k / 24));
  p = __builtin_fmaf(t, p, (float)(k * k * k / 6));
  p = __builtin_fmaf(t, p, (float)(-k * k / 2));
  p = __builtin_fmaf(t, p, (float)k);
  const float series = t * p, direct = __builtin_fmaf(-a, a, 1.f);
  return __builtin_unpredictable(t < (float)(0.25 / k)) ? series : direct;
}

// Decay a and input u of one token: h_t = a h_{t-1} + u_t.
__device__ __forceinline__ void lru_cell(float x, float ga, float gi, float rate, float& a, float& u) {
  const float t = rate * lru_sigmoid(ga);
  a = __builtin_amdgcn_exp2f(-t);
  u = __builtin_amdgcn_sqrtf(lru_one_minus_a2(t, a)) * lru_sigmoid(gi) * x;
}

// The same with what the gradients need.  With g the adjoint of h_t and h1 the
// state before the token:
//     dx = g dx_g,  dgi = dx q,  v = g (vu - va h1),  dga = v sr1,
// q = x (1 - s_i), va = ln2 t a, vu = va (a / m) s_i x, v = dL / d log t.
struct LruGrad {
  float a, u, dx_g, q, va, vu, sr1;
};

// 1 - sigmoid comes as exp(-z) sigmoid(z), which keeps its bits for large z.
// Where exp(-z) overflows that is inf * 0: for ga the product is clamped to
// [0, 1], which makes it 0 (there t, and with it v, is 0 anyway); for gi, where
// q has no such range, the factor exp(-z) is capped at 2^126 instead (behind the
// sigmoid, which keeps a NaN that the cap would lose; dx is 0 there).  1/m is formed of
// 1 - a^2 raised to the smallest normal float: where a = 1, m is 0 and 1/m finite.
// It is up to 2^63, so vu takes it with va (t / m is of the order of m): times
// s_i x it could pass the largest float where vu is small or 0.
__device__ __forceinline__ LruGrad lru_cell_grad(float x, float ga, float gi, float rate) {
  LruGrad r;
  const float er = __builtin_amdgcn_exp2f(-kLog2e * ga);
  const float ei = __builtin_amdgcn_exp2f(-kLog2e * gi);
  const float sr = __builtin_amdgcn_rcpf(1.f + er), si = __builtin_amdgcn_rcpf(1.f + ei);
  const float t = rate * sr;
  r.a = __builtin_amdgcn_exp2f(-t);
  const float m2 = lru_one_minus_a2(t, r.a), rm = __builtin_amdgcn_rsqf(fmaxf(m2, 0x1p-126f)), m = m2 * rm;
  const float six = si * x;
  r.sr1 = __builtin_amdgcn_fmed3f(er * sr, 0.f, 1.f);
  r.dx_g = m * si;
  r.u = m * six;
  r.q = fminf(ei, 0x1p126f) * six;
  r.va = kLn2 * t * r.a;
  r.vu = r.va * rm * (r.a * six);
  return r;
}

}  // namespace mesa
