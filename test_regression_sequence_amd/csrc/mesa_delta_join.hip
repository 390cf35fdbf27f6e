// Gated delta rule: the states that the segments of a split walk start from.
//
// Over a segment the state's rows go S -> S P + Q (P = seg_map, Q = seg_add: what
// the segment makes of unit rows and of zero), and its gradients back N -> N P^T + Q;
// the segment at the walk's start has the given state in its Q already.  From one
// segment to the next that is a 16 x dk by dk x dk product for each 16 rows,
// in fp32 matrix instructions: a workgroup has 16 rows in LDS, each of its waves a
// tile of the result's columns.  9 segments: 17 us at H=16 dk=128, 5: 7 us at 32 heads of 64; maps
// loaded one or three steps ahead change nothing.
#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK, bool BACK>
__global__ __launch_bounds__(4 * DK) void delta_join_kernel(DeltaParams p) {
  constexpr int NT = DK / 16, kThreads = 4 * DK;
  __shared__ __attribute__((aligned(16))) float rows[2][16][DK + 4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int groups = p.dv / 16, bh = blockIdx.x / groups, row0 = blockIdx.x % groups * 16;
  const int64_t edge = (int64_t)bh * p.NS + (BACK ? p.NS - 1 : 0), second = BACK ? edge - 1 : edge + 1;
  for (int i = tid; i < 16 * DK; i += kThreads)
    p.seg_start[(second * p.dv + row0) * DK + i] = rows[1][i / DK][i % DK] = p.seg_add[(edge * p.dv + row0) * DK + i];
  for (int n = 1; n + 1 < p.NS; ++n) {
    const int seg = BACK ? p.NS - 1 - n : n, next = BACK ? seg - 1 : seg + 1;
    const int64_t at = (int64_t)bh * p.NS + seg, to = (int64_t)bh * p.NS + next;
    const float *map = p.seg_map + at * DK * DK, *add = p.seg_add + (at * p.dv + row0) * DK;
    const int col = 16 * wave + r;
    f32x4 b[NT], acc;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      if constexpr (BACK) {
        b[k] = *reinterpret_cast<const f32x4*>(map + (int64_t)col * DK + 16 * k + 4 * g);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[k][e] = map[(int64_t)(16 * k + 4 * g + e) * DK + col];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = add[(int64_t)(4 * g + e) * DK + col];
    __syncthreads();
    const auto& from = rows[n & 1];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(&from[r][16 * k + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mfma_f32(a[e], b[k][e], acc);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rows[~n & 1][4 * g + e][col] = acc[e];
      p.seg_start[(to * p.dv + row0 + 4 * g + e) * DK + col] = acc[e];
    }
  }
}

template <int DK>
hipError_t launch(bool back, const DeltaParams& p, hipStream_t s) {
  const uint32_t blocks = (uint32_t)(p.B * p.H * (p.dv / 16));
  if (back) delta_join_kernel<DK, true><<<blocks, 4 * DK, 0, s>>>(p);
  else delta_join_kernel<DK, false><<<blocks, 4 * DK, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_join(bool back, const DeltaParams& p, hipStream_t s) {
  return p.dk == 128 ? launch<128>(back, p, s) : p.dk == 64 ? launch<64>(back, p, s) : launch<32>(back, p, s);
}

}  // namespace mesa
