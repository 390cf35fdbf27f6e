// Gated linear recurrence: h_t = a_t h_{t-1} + u_t per channel, with decay and
// input from the token's gates (mesa_lru_gate.h).
#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_lru_gate.h"
#include "mesa_lru_tile.h"

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

template <bool BF16>
struct FwdTile {  // 16 tokens a lane row in bf16, 8 in fp32 whose raw values take twice the registers
  static constexpr int TW = BF16 ? 8 : 4, NW = 8, L = 4 * NW * TW;
};

template <bool BF16>
__global__ __launch_bounds__(512, 4) void lru_fwd_kernel(LruParams p) {
  using Sh = FwdTile<BF16>;
  constexpr int TW = Sh::TW, NW = Sh::NW, L = Sh::L;
  __shared__ Pair waves[NW][kLruSlab];
  __shared__ float start[NW][kLruSlab], rates[kLruSlab];
  __shared__ unsigned ticket;
  const int slabs = (p.D + kLruSlab - 1) / kLruSlab, tiles = (p.T + L - 1) / L;
  const unsigned chains = (unsigned)p.B * slabs;
  unsigned at = blockIdx.x;
  if (tiles > 1) {
    if (threadIdx.x == 0) ticket = atomicAdd(p.ticket, 1u);
    __syncthreads();
    at = ticket;
  }
  const int j = at / chains, chain = at % chains, b = chain / slabs, c0 = (chain % slabs) * kLruSlab;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane >> 4;
  const int ch = c0 + 4 * (lane & 15), nch = p.D - ch;
  const int n = lru_length(p, b);
  const int t0 = j * L + (4 * wave + row) * TW;
  const size_t base = (size_t)b * p.T;

  if (j * L >= n) {  // behind the length: zeros; no tile with valid tokens waits for this one
    if (j == 0 && p.h_final && wave == 0 && c0 + lane < p.D) {
      const size_t e = (size_t)b * p.D + c0 + lane;
      p.h_final[e] = p.h0 ? p.h0[e] : 0.f;
    }
    if (p.y) {
      const float zero[4] = {};
#pragma unroll
      for (int s = 0; s < TW; ++s)
        if (t0 + s < p.T) store_raw4<BF16>(p.y, (base + t0 + s) * p.D + ch, zero, nch);
    }
    return;
  }

  float a[TW][4], u[TW][4];
  {
    Raw4<BF16> x[TW], ga[TW], gi[TW];
    uint32_t off[TW];
#pragma unroll
    for (int s = 0; s < TW; ++s) off[s] = (uint32_t)(min(t0 + s, n - 1) - j * L) * p.ld + ch;  // (rows behind n: not used)
    const size_t first = (base + j * L) * p.ld * (BF16 ? 2 : 4);
    load_raw4<BF16>(static_cast<const char*>(p.x) + first, off, nch, x);
    load_raw4<BF16>(static_cast<const char*>(p.ga) + first, off, nch, ga);
    load_raw4<BF16>(static_cast<const char*>(p.gi) + first, off, nch, gi);
    if (threadIdx.x < kLruSlab) rates[threadIdx.x] = c0 + lane < p.D ? lru_rate(p.lam[c0 + lane], p.c) : 0.f;
    __syncthreads();
    float rate[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) rate[e] = rates[4 * (lane & 15) + e];
#pragma unroll
    for (int s = 0; s < TW; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lru_cell(x[s].at(e), ga[s].at(e), gi[s].at(e), rate[e], a[s][e], u[s][e]);
        if (t0 + s >= n) {
          a[s][e] = 1.f;
          u[s][e] = 0.f;
        }
      }
  }
  Pair before[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    Pair own{a[0][e], u[0][e]}, all;
#pragma unroll
    for (int s = 1; s < TW; ++s) own = join(own, Pair{a[s][e], u[s][e]});
    join_rows<false>(own, row, before[e], all);
    if (row == 0) waves[wave][4 * lane + e] = all;
  }
  __syncthreads();
  if (wave == 0) {
    Pair pre[NW], all{1.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      pre[w] = all;
      all = join(all, waves[w][lane]);
    }
    const bool valid = c0 + lane < p.D;
    float h = p.h0 && valid ? p.h0[(size_t)b * p.D + c0 + lane] : 0.f;
    if (tiles > 1)
      h = lru_carry(p.words + (size_t)chain * lru_chain_words(tiles), tiles, j, lane, all, h);
#pragma unroll
    for (int w = 0; w < NW; ++w) start[w][lane] = apply(pre[w], h);
  }
  __syncthreads();
  float h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = apply(before[e], start[wave][4 * (lane & 15) + e]);
  if (t0 % kLruChunk == 0 && t0 < n)
    store_raw4<false>(p.states, ((size_t)b * p.NC + t0 / kLruChunk) * p.D + ch, h, nch);
#pragma unroll
  for (int s = 0; s < TW; ++s) {
    const int t = t0 + s;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __builtin_fmaf(a[s][e], h[e], u[s][e]);
    if (t == n - 1 && p.h_final) store_raw4<false>(p.h_final, (size_t)b * p.D + ch, h, nch);
    if (p.y && t < p.T) {
      const float y[4] = {t < n ? h[0] : 0.f, t < n ? h[1] : 0.f, t < n ? h[2] : 0.f, t < n ? h[3] : 0.f};
      store_raw4<BF16>(p.y, (base + t) * p.D + ch, y, nch);
    }
  }
}

// Marks every word as not published and the ticket as 0.
__global__ __launch_bounds__(kThreads) void lru_clear_kernel(uint64_t* words, size_t n, unsigned* ticket) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) words[i] = kLruEmpty;
  if (i == 0) *ticket = 0;
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

template <bool BF16>
static hipError_t launch_fwd_t(const LruParams& p, hipStream_t s) {
  constexpr int L = FwdTile<BF16>::L;
  const size_t chains = (size_t)p.B * ((p.D + kLruSlab - 1) / kLruSlab);
  const int tiles = p.T > 0 ? (p.T + L - 1) / L : 1;
  if (tiles > 1) {
    const size_t n = chains * lru_chain_words(tiles);
    hipLaunchKernelGGL(lru_clear_kernel, dim3(blocks(n)), dim3(kThreads), 0, s, p.words, n, p.ticket);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((lru_fwd_kernel<BF16>), dim3((unsigned)(chains * tiles)), dim3(64 * FwdTile<BF16>::NW), 0, s, p);
  return hipGetLastError();
}

size_t lru_word_bytes(int B, int T, int D) {
  const size_t chains = (size_t)B * ((D + kLruSlab - 1) / kLruSlab);
  constexpr int L = FwdTile<false>::L;  // the smaller tile: the most words
  return chains * lru_chain_words((T + L - 1) / L) * sizeof(uint64_t) + 256;  // and the ticket
}

hipError_t launch_lru_fwd(bool bf16, const LruParams& p, hipStream_t s) {
  return bf16 ? launch_fwd_t<true>(p, s) : launch_fwd_t<false>(p, s);
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
