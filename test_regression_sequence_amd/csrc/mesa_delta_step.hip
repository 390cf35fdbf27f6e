// Gated delta rule, one token of N sequences: every state is read and written once.
//
// Row i of a state S [dv, dk] stands alone: with a = S_i.k and b = S_i.q,
//     w = v_i - gamma a,  S_i <- gamma S_i + beta w k,  o_i = gamma b + beta w (k.q),
// so both dots are formed before the row changes and S passes through registers
// once.  A row lies in dk / 8 lanes of 8 numbers; a wave takes 512 / dk rows at a
// time and has all its U times as many rows' loads in flight.  Memory bounds it: 256 sequences
// of 16 heads of 128 take 102 us for 0.54 GB of states, 5.3 TB/s (a large copy 4.9), 80 us
// where the last step's states are in part still cached; one sequence of 8 heads 2.9 us.
#include "mesa_common.h"
#include "mesa_delta.h"

namespace mesa {

namespace {

template <int DK, bool BF16, int U>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
  constexpr int LR = DK / 8, RW = 64 / LR;  // lanes a row, rows a wave at a time
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane % LR, row0 = lane / LR;
  const uint32_t at_head = blockIdx.x / p.by_groups;
  const int64_t head = at_head, n = at_head / p.by_h;
  const int first = ((blockIdx.x % p.by_groups) * 4 + wave) * RW * U + row0;
  const int h = at_head % p.by_h, hk = (uint32_t)h / p.by_shared;
  float* s = p.state + head * p.dv * DK + 4 * lr;
  f32x4 a[U], b[U];
  float v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = min(first + u * RW, p.dv - 1);
    a[u] = *reinterpret_cast<const f32x4*>(s + (int64_t)row * DK);
    b[u] = *reinterpret_cast<const f32x4*>(s + (int64_t)row * DK + DK / 2);
    v[u] = load1<BF16>(p.v, n * p.vn + h * p.vh + row);
  }
  const int64_t q_at = n * p.qn + hk * p.qh + 4 * lr, k_at = n * p.kn + hk * p.kh + 4 * lr;
  const f32x4 qa = load4<BF16>(p.q, q_at), qb = load4<BF16>(p.q, q_at + DK / 2);
  const f32x4 ka = load4<BF16>(p.k, k_at), kb = load4<BF16>(p.k, k_at + DK / 2);
  const float gamma = p.gamma[n * p.gn + h * p.gh], beta = p.beta[n * p.bn + h * p.bh];
  float kq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) kq += ka[e] * qa[e] + kb[e] * qb[e];
  kq = group_sum<LR>(kq);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = first + u * RW;
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sk += a[u][e] * ka[e] + b[u][e] * kb[e];
      sq += a[u][e] * qa[e] + b[u][e] * qb[e];
    }
    sk = group_sum<LR>(sk);
    sq = group_sum<LR>(sq);
    const float x = beta * (v[u] - gamma * sk), o = gamma * sq + x * kq;
    if (row < p.dv) {
      *reinterpret_cast<f32x4*>(s + (int64_t)row * DK) = gamma * a[u] + x * ka;
      *reinterpret_cast<f32x4*>(s + (int64_t)row * DK + DK / 2) = gamma * b[u] + x * kb;
      if (lr == 0) {
        const int64_t at = n * p.on + h * p.oh + row;
        if constexpr (BF16) static_cast<__bf16*>(p.o)[at] = (__bf16)o;
        else static_cast<float*>(p.o)[at] = o;
      }
    }
  }
}

template <int DK, bool BF16>
hipError_t launch(DeltaStepParams p, hipStream_t s) {
  constexpr int rows = 128, U = rows / (4 * (512 / DK));  // of a workgroup, and of a lane group
  const uint32_t groups = (uint32_t)((p.dv + rows - 1) / rows);
  p.by_groups = divisor(groups);
  p.by_h = divisor((uint32_t)p.H);
  p.by_shared = divisor((uint32_t)(p.H / p.Hk));
  delta_step_kernel<DK, BF16, U><<<(uint32_t)((int64_t)p.N * p.H * groups), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(bool bf16, const DeltaStepParams& p, hipStream_t s) {
  if (p.dk == 128) return bf16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  if (p.dk == 64) return bf16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  return bf16 ? launch<32, true>(p, s) : launch<32, false>(p, s);
}

}  // namespace mesa
