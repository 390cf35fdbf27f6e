// Gated linear recurrence: h_t = a_t h_{t-1} + u_t per channel, with decay and
// input from the token's gates (mesa_lru_gate.h).  A tile reads x, ga and gi once,
// forms a and u in registers, gets its carry (mesa_lru_tile.h), walks its tokens
// again from it and writes y.  Bound by HBM: at D=2048, bf16, 111 us at B=1,
// T=32768 and 113 at B=8, T=4096, both 579 MB at 5.1 to 5.2 TB/s (a copy: 5.15).
#include <algorithm>

#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_lru_gate.h"
#include "mesa_lru_tile.h"

namespace mesa {

namespace {

constexpr int kThreads = 256;

// Tokens a lane, of a tile of 8 times as many.  128 tokens a tile: shorter lanes
// make more tiles to join, 123 to 131 us (TW = 12) and 120 to 127 (TW = 8) against
// 111 to 115 at B=1, T=32768, D=2048, bf16; longer ones (TW = 24: 110 to 112) leave
// more of a tile empty at the end of a sequence.  Workgroups of 8 waves were slower
// throughout.  Short sequences take the smallest of four tiles that holds one: 17,
// 29 and 56 us with 8, 32 and 64 tokens against 73 to 79 with 128 at B=256, T=8, 32
// and 64, D=2048, bf16.
constexpr int kNw = 4, kTw = 16, kTile = 2 * kNw * kTw;
static_assert(kNw >= 4, "three waves wait for other tiles, one folds this one's");

template <bool BF16, bool LINES, int TW>
__global__ __launch_bounds__(256, 4) void lru_fwd_kernel(LruParams p) {
  constexpr int NW = kNw, L = 2 * NW * TW;
  static_assert(TW % kLruChunk == 0 || kLruChunk % TW == 0, "kept states lie at a lane's first token");
  constexpr uint32_t ES = BF16 ? 2 : 4;
  __shared__ Pair waves[NW][kLruSlab], pre[NW][kLruSlab];
  __shared__ LruCarry carry;
  __shared__ unsigned ticket;
  const LruGrid grid(p.B, p.T, p.D, L);
  const int tiles = grid.tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane >> 5, c2 = 2 * (lane & 31);
  int j, chain;
  if (!grid.take<LINES>(p.tickets, &ticket, j, chain)) return;
  const int b = chain / grid.slabs, c0 = (chain % grid.slabs) * kLruSlab;
  const int ch = c0 + c2, nch = p.D - ch;
  const int n = lru_length(p, b);
  const int tw0 = (2 * wave + row) * TW, t0 = j * L + tw0;  // this lane's first token
  const size_t first = (size_t)b * p.T + (size_t)j * L;     // the tile's first row of the tensors
  char* y = p.y ? static_cast<char*>(p.y) + first * p.D * ES : nullptr;
  const uint32_t yrow = p.D * ES, yoff = tw0 * yrow + ch * ES;

  if (j * L >= n) {  // behind the length: zeros; no tile with valid tokens waits for this one
    if (j == 0 && p.h_final && wave == 0 && c0 + lane < p.D) {
      const size_t e = (size_t)b * p.D + c0 + lane;
      p.h_final[e] = p.h0 ? p.h0[e] : 0.f;
    }
    if (y) {
      const float zero[2] = {};
#pragma unroll
      for (int s = 0; s < TW; ++s)
        if (t0 + s < p.T) store_raw2<BF16, LINES>(y, yoff + s * yrow, zero, nch);
    }
    return;
  }
  const bool whole = (j + 1) * L <= n;

  float a[TW][2], u[TW][2];
  {
    Raw2<BF16> x[TW], ga[TW], gi[TW];
    uint32_t off[TW];
    const int lc = lru_load_channel(ch, p.D);
#pragma unroll
    for (int s = 0; s < TW; ++s) {  // rows behind n read row n - 1 and are not used
      const int t = whole ? tw0 + s : min(tw0 + s, n - 1 - j * L);
      off[s] = ((uint32_t)t * p.ld + lc) * ES;
    }
    const size_t in = first * p.ld * ES;
    float lam[2];
    load_lam(p, ch, lam);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.x) + in, off, x);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.ga) + in, off, ga);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.gi) + in, off, gi);
    to_own_channels(p.D, ch, x);
    to_own_channels(p.D, ch, ga);
    to_own_channels(p.D, ch, gi);
    const float rate[2] = {lru_rate(lam[0], p.c), lru_rate(lam[1], p.c)};
#pragma unroll
    for (int s = 0; s < TW; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) lru_cell(x[s].at(e), ga[s].at(e), gi[s].at(e), rate[e], a[s][e], u[s][e]);
    if (!whole) {
#pragma unroll
      for (int s = 0; s < TW; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[s][e] = __builtin_unpredictable(t0 + s >= n) ? 1.f : a[s][e];
          u[s][e] = __builtin_unpredictable(t0 + s >= n) ? 0.f : u[s][e];
        }
    }
  }
  Pair before[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    Pair own{a[0][e], u[0][e]}, all;
#pragma unroll
    for (int s = 1; s < TW; ++s) own = join(own, Pair{a[s][e], u[s][e]});
    join_rows<false>(own, row, before[e], all);
    settle(before[e].A);
    settle(before[e].E);
    if (row == 0) waves[wave][c2 + e] = all;
  }
  float h_in = 0.f;  // the state before tile 0
  if (wave == 1 && p.h0 && c0 + lane < p.D) h_in = p.h0[(size_t)b * p.D + c0 + lane];
  settle(h_in);
  __syncthreads();
  uint64_t* words = p.words + (size_t)chain * lru_chain_words(tiles);
  Pair tile{1.f, 0.f};
  if (wave == 0) {
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      pre[w][lane] = tile;
      tile = join(tile, waves[w][lane]);
    }
    if (tiles > 1) publish(words + (size_t)j * kLruSlab + lane, tile);
  } else if (wave == 1) {
    carry_groups(words, tiles, j, lane, h_in, carry.h);
  } else if (wave < 4) {
    carry_tiles(words, j, wave - 2, lane, wave == 2 ? carry.early : carry.late);
  }
  __syncthreads();
  if (wave == 0 && j % kLruGroup == kLruGroup - 1) publish_group(words, tiles, j, lane, carry, tile);
  float h[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    h[e] = apply(carry.late[c2 + e], apply(carry.early[c2 + e], carry.h[c2 + e]));
    h[e] = apply(before[e], apply(pre[wave][c2 + e], h[e]));
  }
  if (t0 < n && t0 % kLruChunk == 0)
    store_raw2<false, LINES>(p.states, (((size_t)b * p.NC + t0 / kLruChunk) * p.D + ch) * 4, h, nch);
#pragma unroll
  for (int s = 0; s < TW; ++s)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      h[e] = __builtin_fmaf(a[s][e], h[e], u[s][e]);
      u[s][e] = h[e];
    }
  // behind n the state stays: a lane's last one is the final state wherever n lies in its tokens
  if (p.h_final && t0 < n && n <= t0 + TW) store_raw2<false, LINES>(p.h_final, ((size_t)b * p.D + ch) * 4, h, nch);
  if (!y) return;
  if (whole && nch >= 2) {
#pragma unroll
    for (int s = 0; s < TW; ++s) store_raw2<BF16, LINES>(y, yoff + s * yrow, u[s], 2);
  } else {
#pragma unroll
    for (int s = 0; s < TW; ++s) {
#pragma unroll
      for (int e = 0; e < 2; ++e) u[s][e] = t0 + s < n ? u[s][e] : 0.f;
      if (t0 + s < p.T) store_raw2<BF16, LINES>(y, yoff + s * yrow, u[s], nch);
    }
  }
}

// Marks every word as not published and sets the tickets to 0.
__global__ __launch_bounds__(kThreads) void lru_ready_kernel(uint64_t* words, size_t n, unsigned* tickets) {
  const size_t first = (size_t)blockIdx.x * kThreads + threadIdx.x, stride = (size_t)gridDim.x * kThreads;
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));  // (n is even: a slab is 64 words)
  for (size_t i = first; i < n / 2; i += stride) reinterpret_cast<u64x2*>(words)[i] = u64x2{kLruEmpty, kLruEmpty};
  if (first < kLruClasses * kLruCounterStride) tickets[first] = 0;
}

// One token: 8 channels a lane, bound by HBM (x, ga, gi and the state in, the
// state and y out): 46 us at N=4096, D=4096, bf16 (5.7 TB/s), and by the latency
// of a launch for few tokens (2.3 us).
template <bool BF16>
__global__ __launch_bounds__(kThreads) void lru_step_kernel(LruParams p) {
  const int groups = (p.D + 7) / 8;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)p.B * groups) return;
  const size_t row = (size_t)(i / groups);
  const int ch = (int)(i % groups) * 8, n = p.D - ch;
  const size_t in = row * p.ld, out = row * p.D;
  // (loaded exactly: the state is updated in place, by other waves too)
  const Raw8<BF16> x = load_part8<BF16>(p.x, in + ch, n), ga = load_part8<BF16>(p.ga, in + ch, n),
                   gi = load_part8<BF16>(p.gi, in + ch, n);
  const Raw8<false> before = load_part8<false>(p.h_final, out + ch, n), lam = load_part8<false>(p.lam, ch, n);
  float h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float a, u;
    lru_cell(x.at(k), ga.at(k), gi.at(k), lru_rate(lam.at(k), p.c), a, u);
    h[k] = __builtin_fmaf(a, before.at(k), u);
  }
  store_raw8<false, true>(p.h_final, out + ch, h, n);
  store_raw8<BF16, true>(p.y, out + ch, h, n);
}

unsigned blocks(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_lru_ready(const LruParams& p, size_t words, hipStream_t s) {
  const unsigned need = blocks(std::max<size_t>(words / 2, kLruClasses * kLruCounterStride));
  hipLaunchKernelGGL(lru_ready_kernel, dim3(std::min(need, 1024u)), dim3(kThreads), 0, s, p.words, words, p.tickets);
  return hipGetLastError();
}

template <bool BF16, bool LINES, int TW>
static hipError_t launch_fwd_t(const LruParams& p, hipStream_t s) {
  const LruGrid grid(p.B, p.T, p.D, 2 * kNw * TW);
  if (grid.tiles > 1) {
    if (const hipError_t e = launch_lru_ready(p, grid.chains * lru_chain_words(grid.tiles), s); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((lru_fwd_kernel<BF16, LINES, TW>), dim3(grid.workgroups()), dim3(64 * kNw), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, bool LINES>
static hipError_t launch_fwd_tw(const LruParams& p, hipStream_t s) {
  if (p.T <= 2 * kNw) return launch_fwd_t<BF16, LINES, 1>(p, s);
  if (p.T <= 8 * kNw) return launch_fwd_t<BF16, LINES, 4>(p, s);
  if (p.T <= 16 * kNw) return launch_fwd_t<BF16, LINES, 8>(p, s);
  return launch_fwd_t<BF16, LINES, kTw>(p, s);
}

size_t lru_fwd_word_bytes(int B, int T, int D) {
  const LruGrid grid(B, T, D, kTile);
  return grid.chains * lru_chain_words(grid.tiles) * sizeof(uint64_t);
}

hipError_t launch_lru_fwd(bool bf16, const LruParams& p, hipStream_t s) {
  const bool lines = lru_whole_lines(bf16, {p.ld, p.D}, {p.x, p.ga, p.gi, p.y});
  if (bf16) return lines ? launch_fwd_tw<true, true>(p, s) : launch_fwd_tw<true, false>(p, s);
  return lines ? launch_fwd_tw<false, true>(p, s) : launch_fwd_tw<false, false>(p, s);
}

hipError_t launch_lru_step(bool bf16, const LruParams& p, hipStream_t s) {
  const dim3 grid(blocks((long long)p.B * ((p.D + 7) / 8)));
  if (bf16) hipLaunchKernelGGL((lru_step_kernel<true>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((lru_step_kernel<false>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace mesa
