// Residual addition and RMS norm of token rows, with a plain or an e4m3 output,
// and its gradient (MesaNet page, "architecture": the residual blocks' norm).
//     s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = w s r
//     ds = r (g - n mean(g n)) + d_residual,  g = dy w,  n = s r,  dw = sum_rows dy n
//
// Both are bound by HBM: every input is read once and every output written
// once.  A row is held in registers by TPR lanes of NV vectors of 8 channels
// each, from its loads to its stores, so nothing is read twice; the smallest
// (TPR, NV) that covers D is taken, which keeps lanes busy and, up to D = 2048,
// a row within one wave (its sums then need no LDS and no barrier).  Row groups
// walk rows a grid apart and load the next row before they work on this one;
// w, and the backward's sums for dw, stay in their registers meanwhile.
//
// At R = 32768, D = 2048, bf16 rows and stream: 86 us with e4m3 rows (5.5 TB/s),
// 101 us with bf16 rows (5.3), the gradient 107 with its sum for dw; a copy runs at
// 5.15 TB/s.  Rows over 8192 leave no room for w in the gradient's registers; it is
// read from LDS there (145 -> 118 us at R = 4096, D = 16384, bf16).  With fp32
// tensors the gradient's rows of 4 vectors a lane still hold more than the
// registers: one wave per SIMD at D of 1025 to 2048 and of 4097 to 8192 (R = 32768,
// D = 2048: 200 us fp32, 203 bf16 on an fp32 stream, both above a copy's rate all
// the same), spills above 8192 (R = 4096, D = 16384: 303 us fp32, 3.5 TB/s).
#include <type_traits>

#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_rows.h"

namespace mesa {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-100f;
constexpr int kCus = 256;

template <int TPR>
struct NormShape {
  static constexpr int kThreads = TPR <= 256 ? 256 : TPR;
  static constexpr int kRows = kThreads / TPR;  // rows a workgroup holds at a time
};

// The first row of this lane's group (uniform where a row takes whole waves).
template <int TPR>
__device__ __forceinline__ int first_row() {
  int group = threadIdx.x / TPR;
  if constexpr (TPR >= 64) group = __builtin_amdgcn_readfirstlane(group);
  return blockIdx.x * NormShape<TPR>::kRows + group;
}

// Sums (a, b) over the TPR lanes of a row; the same bits in every lane.  Rows
// wider than a wave go through LDS, two buffers in turn: one barrier a call.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2 (*lds)[8], int& turn) {
  if constexpr (TPR <= 64) {
    a = group_sum<TPR>(a);
    b = group_sum<TPR>(b);
  } else {
    a = wave_sum(a);
    b = wave_sum(b);
    if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = float2{a, b};
    __syncthreads();
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {
      a += lds[turn][i].x;
      b += lds[turn][i].y;
    }
    turn ^= 1;
  }
}

template <int TPR>
__device__ __forceinline__ float row_max(float v, float2 (*lds)[8], int& turn) {
  if constexpr (TPR <= 64) {
    return group_max<TPR>(v);
  } else {
    v = group_max<64>(v);
    if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6].x = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v = fmaxf(v, lds[turn][i].x);
    turn ^= 1;
    return v;
  }
}

// The first n of 8 channels as e4m3 bytes.  |y| / scale is at most 448 but for
// rounding, well inside the range that rounds to 448.
template <bool TAIL>
__device__ __forceinline__ void store_e4m3(void* base, size_t elem, const float (&y)[8], float inv, int n) {
  uint32_t lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * inv, y[5] * inv, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * inv, y[7] * inv, hi, true);
  uint8_t* q = static_cast<uint8_t*>(base) + elem;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef u32x2 __attribute__((aligned(1))) u32x2_any;
  if (n >= 8) {
    *reinterpret_cast<u32x2_any*>(q) = u32x2{lo, hi};
  } else if (TAIL && n > 0) {
    typedef uint32_t __attribute__((aligned(1))) u32_byte;
    typedef uint16_t __attribute__((aligned(1))) u16_byte;
    const uint32_t rest = n & 4 ? hi : lo;
    if (n & 4) *reinterpret_cast<u32_byte*>(q) = lo;
    if (n & 2) *reinterpret_cast<u16_byte*>(q + (n & 4)) = (uint16_t)rest;
    if (n & 1) q[n & 6] = (uint8_t)(n & 2 ? rest >> 16 : rest);
  }
}

template <bool BF16, bool RBF16, RowEnd END, int TPR, int NV>
__global__ __launch_bounds__(NormShape<TPR>::kThreads) void rmsnorm_kernel(NormParams p) {
  using Sh = NormShape<TPR>;
  __shared__ float2 lds[2][8];
  int turn = 0;
  const int lane = threadIdx.x % TPR, D = p.D;
  const int stride = gridDim.x * Sh::kRows;
  int row = first_row<TPR>();
  Raw8<BF16> rx[NV];
  Raw8<RBF16> rr[NV];
  auto load = [&](int at) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (lane + TPR * k);
      rx[k] = load_row8<BF16, END>(p.x, (size_t)at * D, c, D);
      if (p.residual) rr[k] = load_row8<RBF16, END>(p.residual, (size_t)at * D, c, D);
    }
  };
  if (row < p.R) load(row);
  float w[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (lane + TPR * k);
    Raw8<false> v = load_row8<false, END>(p.w, 0, c, D);
    if constexpr (END == RowEnd::kWithin) own_channels(v, c, D);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[k][e] = v.at(e);
  }
  const float inv_d = 1.f / (float)D;
  while (row < p.R) {
    float s[NV][8], ss = 0.f, unused = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (END == RowEnd::kWithin) own_channels(rx[k], 8 * (lane + TPR * k), D);
      if constexpr (END == RowEnd::kWithin) if (p.residual) own_channels(rr[k], 8 * (lane + TPR * k), D);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[k][e] = rx[k].at(e);
        if (p.residual) s[k][e] += rr[k].at(e);
        ss = __builtin_fmaf(s[k][e], s[k][e], ss);
      }
    }
    const int here = row;
    row += stride;
    if (row < p.R) load(row);
    auto store_stream = [&] {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = 8 * (lane + TPR * k);
        store_raw8<RBF16, END != RowEnd::kWhole>(p.residual_out, (size_t)here * D + c, s[k], D - c);
      }
    };
    // residual_out may be an input.  The row's last vector is loaded with channels
    // of its neighbour's, which may be another wave's: then all waves have their
    // loads before one stores.
    constexpr bool kStoreLate = END == RowEnd::kWithin && TPR > 64;
    if (!kStoreLate && p.residual_out) store_stream();
    row_sum2<TPR>(ss, unused, lds, turn);
    if (kStoreLate && p.residual_out) store_stream();
    // For e4m3 a row's factor r cancels but in the scales.  There values are formed
    // with the power of two below r, and rounded twice before their codes, not three
    // times: at R = 32768, D = 2048 19 instead of 34 of 67 M codes differ from those
    // of exact values.
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_d, p.eps));
    const float power = __uint_as_float(__float_as_uint(r) & 0x7F800000u);
    const float factor = p.e4m3 ? power : r;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[k][e] = s[k][e] * factor * w[k][e];  // (s r is of order 1; r w may leave fp32)
    if (!p.e4m3) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = 8 * (lane + TPR * k);
        store_raw8<BF16, END != RowEnd::kWhole>(p.y, (size_t)here * D + c, s[k], D - c);
      }
      continue;
    }
    const float rest = __uint_as_float(__float_as_uint(r) & 0x007FFFFFu | 0x3F800000u);  // r / power
    float m[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      m[k] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m[k] = fmaxf(m[k], fabsf(s[k][e]));
    }
    auto scale = [&](float m) { return fmaxf(rest * m, kAmaxFloor) / kE4m3Max; };
    if (p.group) {  // 128 channels are the same vector of 16 neighbouring lanes
      const int groups = (D + 127) / 128;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        m[k] = group_max<16>(m[k]);
        const int g = (lane + TPR * k) / 16;
        if (lane % 16 == 0 && g < groups) p.scale[(size_t)here * groups + g] = scale(m[k]);
      }
    } else {
#pragma unroll
      for (int k = 1; k < NV; ++k) m[0] = fmaxf(m[0], m[k]);
      m[0] = row_max<TPR>(m[0], lds, turn);
#pragma unroll
      for (int k = 1; k < NV; ++k) m[k] = m[0];
      if (lane == 0) p.scale[here] = scale(m[0]);
    }
    // (divided, not multiplied by a reciprocal: its error would be common to a row)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (lane + TPR * k);
      const float inv = rest * m[k] >= kAmaxFloor ? kE4m3Max / m[k] : rest * (kE4m3Max / kAmaxFloor);
      store_e4m3<END != RowEnd::kWhole>(p.y, (size_t)here * D + c, s[k], inv, D - c);
    }
  }
}

// The same rows; dw is summed per lane over the rows that a group walks, in fp32,
// then over the workgroup's groups through LDS, in 64 bits, into one partial row
// per workgroup.  A chain of fp32 additions loses bits as it grows (2^20 rows of
// 2500, all alike: up to 512 half steps of fp32, 17 as it is), so behind every
// kDwRun rows a lane's sums are added to 64-bit ones: in LDS, or where that holds
// the weights (TPR = 512) in the workspace.
constexpr int kDwRun = 64;

template <bool BF16, bool RBF16, RowEnd END, int TPR, int NV>
__global__ __launch_bounds__(NormShape<TPR>::kThreads) void rmsnorm_bwd_kernel(NormParams p) {
  using Sh = NormShape<TPR>;
  __shared__ float2 lds[2][8];
  __shared__ float sums[Sh::kRows][Sh::kRows > 1 ? TPR * 8 : 1];
  constexpr bool kInLds = TPR == 512;
  __shared__ Raw8<false> weights[kInLds ? TPR * NV : 1];
  int turn = 0;
  const int lane = threadIdx.x % TPR, D = p.D;
  const int stride = gridDim.x * Sh::kRows;
  int row = first_row<TPR>();
  Raw8<RBF16> rs[NV], rr[NV];
  Raw8<BF16> rd[NV];
  auto load = [&](int at) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (lane + TPR * k);
      rs[k] = load_row8<RBF16, END>(p.x, (size_t)at * D, c, D);
      rd[k] = load_row8<BF16, END>(p.dy, (size_t)at * D, c, D);
      if (p.residual) rr[k] = load_row8<RBF16, END>(p.residual, (size_t)at * D, c, D);
    }
  };
  if (row < p.R) load(row);
  Raw8<false> w[kInLds ? 1 : NV];
  float dw[NV][8] = {};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (lane + TPR * k);
    Raw8<false> v = load_row8<false, END>(p.w, 0, c, D);
    if constexpr (END == RowEnd::kWithin) own_channels(v, c, D);
    if constexpr (!kInLds) w[k] = v;
    else if (threadIdx.x < TPR) weights[lane + TPR * k] = v;
  }
  if constexpr (kInLds) __syncthreads();
  auto weight = [&](int k) {
    if constexpr (kInLds) return weights[lane + TPR * k];
    else return w[k];
  };
  const float inv_d = 1.f / (float)D;
  __shared__ double lds_acc[kInLds ? 1 : TPR * NV * 8];
  // (each thread adds to, and reads, what it wrote itself)
  double* acc = kInLds ? p.acc + (size_t)blockIdx.x * (TPR * NV * 8) : lds_acc;
  float* part = p.part + (size_t)blockIdx.x * D;
  // Rows are counted alike for all of a workgroup's groups.  (Where it has several, in
  // one loop: two nested ones take up to 36 registers more.  Where it has one, nested:
  // 4 to 24 less.)
  constexpr int kNest = Sh::kRows == 1 ? kDwRun : 1;
  const int first = blockIdx.x * Sh::kRows;
  bool fresh = true;
  int runs = 0;
  for (int start = first; start < p.R; start += kNest * stride) {
    for (int run = 0; run < kNest && row < p.R; ++run) {
      float ss = 0.f, gs = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if constexpr (END == RowEnd::kWithin) own_channels(rs[k], 8 * (lane + TPR * k), D);
        if constexpr (END == RowEnd::kWithin) own_channels(rd[k], 8 * (lane + TPR * k), D);
        if constexpr (END == RowEnd::kWithin) if (p.residual) {
          own_channels(rr[k], 8 * (lane + TPR * k), D);
          if constexpr (TPR > 64) hold(rr[k]);  // before the barrier: ds may be d_residual (as in the forward)
        }
        const Raw8<false> wk = weight(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = rs[k].at(e);
          ss = __builtin_fmaf(s, s, ss);
          gs = __builtin_fmaf(rd[k].at(e) * wk.at(e), s, gs);
        }
      }
      row_sum2<TPR>(ss, gs, lds, turn);
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_d, p.eps));
      const float kk = gs * inv_d * r * r;  // mean(g n) r: ds = r g - n (mean(g n) r)
      const int here = row;
      row += stride;
      float ds[NV][8];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const Raw8<false> wk = weight(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = rs[k].at(e) * r, d = rd[k].at(e);
          ds[k][e] = __builtin_fmaf(-n, kk, r * (d * wk.at(e)));
          if (p.residual) ds[k][e] += rr[k].at(e);
          dw[k][e] = __builtin_fmaf(d, n, dw[k][e]);
        }
      }
      if (row < p.R) load(row);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = 8 * (lane + TPR * k);
        store_raw8<RBF16, END != RowEnd::kWhole>(p.y, (size_t)here * D + c, ds[k], D - c);
        if (p.residual_out) store_raw8<BF16, END != RowEnd::kWhole>(p.residual_out, (size_t)here * D + c, ds[k], D - c);
      }
    }
    const bool last = start + kNest * stride >= p.R;
    if (kNest == 1 && ++runs < kDwRun && !last) continue;
    // The run's sums to the 64-bit ones, the last run's on to the partial row.  (The thread's
    // number is hidden, or what follows from it is formed ahead of the rows and held in
    // registers while they are walked.)
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (Sh::kRows == 1) {  // a lane's channels are its own
        if (!(fresh && last))
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            double* at = acc + (8 * k + e) * TPR + thread;
            const double v = (fresh ? 0. : *at) + dw[k][e];
            if (!last) *at = v;
            dw[k][e] = last ? (float)v : 0.f;
          }
        const int c = 8 * (thread + TPR * k);
        if (last) store_raw8<false, END != RowEnd::kWhole>(part, c, dw[k], D - c);
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sums[thread / TPR][8 * (thread % TPR) + e] = dw[k][e];
          dw[k][e] = 0.f;
        }
        __syncthreads();
        for (int i = thread; i < TPR * 8; i += Sh::kThreads) {
          const int c = TPR * 8 * k + i;
          if (c >= D) break;
          double v = fresh ? 0. : acc[c];
#pragma unroll
          for (int g = 0; g < Sh::kRows; ++g) v += sums[g][i];
          if (last) part[c] = (float)v;
          else acc[c] = v;
        }
      }
    }
    fresh = false;
    runs = 0;
  }
}

// dw from G partial rows [G, D], summed in 64 bits: 16 channels a workgroup, 16 threads a channel.
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* part, float* dw, int G, int D) {
  __shared__ double sums[16][16];
  const int j = threadIdx.x % 16, slice = threadIdx.x / 16, c = blockIdx.x * 16 + j;
  double v = 0.;
  if (c < D) {
#pragma unroll 8
    for (int g = slice; g < G; g += 16) v += part[(size_t)g * D + c];
  }
  sums[slice][j] = v;
  __syncthreads();
  if (slice == 0 && c < D) {
    for (int i = 1; i < 16; ++i) v += sums[i][j];
    dw[c] = (float)v;
  }
}

constexpr int kMaxD = 512 * 4 * 8;  // the widest row group's channels

// Calls fn(TPR, NV) as constants for the smallest row group that holds D channels.
template <RowEnd END, typename F>
auto norm_shape(int D, F&& fn) {
  using std::integral_constant;
  if constexpr (END != RowEnd::kShort) {
    if (D > 8192) return fn(integral_constant<int, 512>{}, integral_constant<int, 4>{});
    if (D > 4096) return fn(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    if (D > 2048) return fn(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (D > 1024) return fn(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (D > 512) return fn(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (D > 256) return fn(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (D > 128) return fn(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  }
  return fn(integral_constant<int, 16>{}, integral_constant<int, 1>{});
}

// Workgroups of a launch: as many as rows need, at most `per_cu` a CU.
int norm_groups(int R, int rows, int per_cu) {
  const long long need = ((long long)R + rows - 1) / rows;
  return (int)(need < (long long)kCus * per_cu ? need : (long long)kCus * per_cu);
}

constexpr int kFwdPerCu = 4, kBwdPerCu = 2;

template <bool BF16, bool RBF16, RowEnd END>
hipError_t launch_fwd_t(const NormParams& p, hipStream_t s) {
  return norm_shape<END>(p.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    using Sh = NormShape<TPR>;
    hipLaunchKernelGGL((rmsnorm_kernel<BF16, RBF16, END, TPR, NV>), dim3(norm_groups(p.R, Sh::kRows, kFwdPerCu)),
                       dim3(Sh::kThreads), 0, s, p);
    return hipGetLastError();
  });
}

int bwd_groups(int R, int D) {
  return norm_shape<RowEnd::kWhole>(D, [&](auto tpr, auto) {
    return norm_groups(R, NormShape<decltype(tpr)::value>::kRows, kBwdPerCu);
  });
}

// Bytes of the 64-bit sums that do not fit LDS.
size_t acc_bytes(int R, int D) {
  const bool in_lds = norm_shape<RowEnd::kWhole>(D, [](auto tpr, auto) { return decltype(tpr)::value < 512; });
  const int G = bwd_groups(R, D);  // (a row a workgroup)
  return in_lds || R <= kDwRun * G ? 0 : (size_t)G * kMaxD * sizeof(double);
}

template <bool BF16, bool RBF16, RowEnd END>
hipError_t launch_bwd_t(const NormParams& p, hipStream_t s) {
  const int G = p.R > 0 ? bwd_groups(p.R, p.D) : 0;
  if (G > 0) {
    const hipError_t e = norm_shape<END>(p.D, [&](auto tpr, auto nv) {
      constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
      hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, RBF16, END, TPR, NV>), dim3(G), dim3(NormShape<TPR>::kThreads), 0, s, p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((p.D + 15) / 16), dim3(256), 0, s, p.part, p.dw,
                     G, p.D);
  return hipGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_scratch(int R, int D) { return acc_bytes(R, D) + (size_t)bwd_groups(R, D) * D * sizeof(float); }

void rmsnorm_bwd_carve(NormParams& p, void* workspace) {
  p.acc = static_cast<double*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + (p.R > 0 ? acc_bytes(p.R, p.D) : 0));
}

template <RowEnd END>
static hipError_t launch_fwd(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  if (!bf16) return launch_fwd_t<false, false, END>(p, s);
  return res_bf16 ? launch_fwd_t<true, true, END>(p, s) : launch_fwd_t<true, false, END>(p, s);
}

template <RowEnd END>
static hipError_t launch_bwd(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  if (!bf16) return launch_bwd_t<false, false, END>(p, s);
  return res_bf16 ? launch_bwd_t<true, true, END>(p, s) : launch_bwd_t<true, false, END>(p, s);
}

hipError_t launch_rmsnorm(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  switch (row_end(p.D)) {
    case RowEnd::kWhole: return launch_fwd<RowEnd::kWhole>(bf16, res_bf16, p, s);
    case RowEnd::kWithin: return launch_fwd<RowEnd::kWithin>(bf16, res_bf16, p, s);
    default: return launch_fwd<RowEnd::kShort>(bf16, res_bf16, p, s);
  }
}

hipError_t launch_rmsnorm_bwd(bool bf16, bool res_bf16, const NormParams& p, hipStream_t s) {
  switch (row_end(p.D)) {
    case RowEnd::kWhole: return launch_bwd<RowEnd::kWhole>(bf16, res_bf16, p, s);
    case RowEnd::kWithin: return launch_bwd<RowEnd::kWithin>(bf16, res_bf16, p, s);
    default: return launch_bwd<RowEnd::kShort>(bf16, res_bf16, p, s);
  }
}

}  // namespace mesa
