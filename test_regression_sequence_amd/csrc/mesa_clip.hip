// Global norm of many gradients, and clipping: two passes at memory rate.
//
// The first adds the squares up, the second scales by min(1, max_norm / (norm +
// eps)).  Squares are formed and added in 64 bits (exact squares, no overflow
// before the root), in a fixed order: a lane along its pieces, then lanes in a tree
// and waves in turn; the workgroups' sums so too, 256 lanes along them.  Equal inputs give
// equal bits.  The sums of at most about 2048 workgroups are added up again by each workgroup of
// the second pass (16 KB from L2), which spares a launch in between.  The second
// pass takes the pieces in the opposite order: what was read last may still be in the
// last-level cache.  Tensors start at any multiple of their element size.
//
// 671 MB of gradients, mostly bf16: 152 us for the first pass (4.4 TB/s), 238 us for the
// second (5.6 TB/s read and written; a large copy 4.9).  51 MB in fp32: 11 and 20 us, the second
// at 5.0 TB/s; its L2s find none of what the first pass read.
#include "mesa_clip.h"
#include "mesa_rows.h"

namespace mesa {

namespace {

constexpr int kThreads = 256, kVectors = kClipPiece / (8 * kThreads);

// The tensor that holds piece `id`.
__device__ __forceinline__ int tensor_of(const ClipTable& t, int64_t id) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= id) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// All threads of the workgroup receive the sum, formed in one order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int off = 1; off < 64; off *= 2) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kThreads / 64; ++i) v += part[i];
  return v;
}

template <bool BF16>
__device__ __forceinline__ double squares(const void* grad, int64_t at, int64_t n, double sum) {
  Raw8<BF16> r[kVectors];
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    const int64_t from = at + (int64_t)(i * kThreads + threadIdx.x) * 8;
    r[i] = load_part8<BF16>(grad, from, (int)min(n - from, (int64_t)8));
  }
#pragma unroll
  for (int i = 0; i < kVectors; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double x = r[i].at(e);
      sum = fma(x, x, sum);
    }
  return sum;
}

__global__ __launch_bounds__(kThreads) void clip_squares_kernel(ClipTable t, double* sums) {
  double sum = 0.0;
  for (int64_t id = blockIdx.x; id < t.first[t.count]; id += gridDim.x) {
    const int i = tensor_of(t, id);
    const int64_t at = (id - t.first[i]) * kClipPiece;
    sum = t.bf16[i] ? squares<true>(t.grad[i], at, t.n[i], sum) : squares<false>(t.grad[i], at, t.n[i], sum);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

template <bool BF16>
__device__ __forceinline__ void scaled(const void* grad, void* out, int64_t at, int64_t n, float factor, int power) {
  Raw8<BF16> r[kVectors];
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    const int64_t from = at + (int64_t)(i * kThreads + threadIdx.x) * 8;
    r[i] = load_part8<BF16>(grad, from, (int)min(n - from, (int64_t)8));
  }
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    const int64_t from = at + (int64_t)(i * kThreads + threadIdx.x) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_ldexpf(r[i].at(e) * factor, power);
    store_raw8<BF16, true>(out, from, v, (int)min(n - from, (int64_t)8));
  }
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipTable t, const double* sums, int n_sums, double max_norm,
                                                              double eps, float* norm_out, float* scale_out) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n_sums; i += kThreads) sum += sums[i];
  const double norm = sqrt(block_sum(sum)), ratio = max_norm / (norm + eps);
  // no bound leaves infinite gradients too as they are; a NaN stays one
  const float scale = ratio >= 1.0 || (max_norm == INFINITY && norm == norm) ? 1.f : (float)ratio;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm_out) *norm_out = (float)norm;
    if (scale_out) *scale_out = scale;
  }
  // A scale below fp32's normal numbers has few bits left there: as a number from 1/2 on and a power of two
  int power = 0;
  const float factor = scale < 0x1p-126f ? (float)frexp(ratio, &power) : scale;
  const int64_t all = t.first[t.count];
  for (int64_t id = all - 1 - blockIdx.x; id >= 0; id -= gridDim.x) {
    const int i = tensor_of(t, id);
    if (!t.out[i] || (t.out[i] == t.grad[i] && scale == 1.f)) continue;
    const int64_t at = (id - t.first[i]) * kClipPiece;
    if (t.bf16[i]) scaled<true>(t.grad[i], t.out[i], at, t.n[i], factor, power);
    else scaled<false>(t.grad[i], t.out[i], at, t.n[i], factor, power);
  }
}

}  // namespace

hipError_t launch_clip_squares(const ClipTable& t, int blocks, double* sums, hipStream_t s) {
  clip_squares_kernel<<<blocks, kThreads, 0, s>>>(t, sums);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable& t, int blocks, const double* sums, int n_sums, double max_norm, double eps,
                             float* norm, float* scale, hipStream_t s) {
  clip_scale_kernel<<<blocks, kThreads, 0, s>>>(t, sums, n_sums, max_norm, eps, norm, scale);
  return hipGetLastError();
}

}  // namespace mesa
