// Backward pass of the gated linear recurrence (mesa_lru_gate.h: the cell and
// its gradients; mesa_lru_tile.h: tiles and their joining).
//
// With c_t the adjoint of the state behind token t, g_t = c_t + dy_t and
// c_{t-1} = a_t g_t: a scan of the maps c -> a_t c + a_t dy_t, last token first.
// A tile reads x, ga, gi and dy once, forms decays, inputs and gradient factors
// in registers, walks the states again from the forward's kept state before
// its chunk (they need no other tile), joins its adjoints with the tiles behind
// it, and writes dx, dga and dgi.  Bound by HBM with the vector units three quarters
// busy: 187 to 213 us at B=8, T=4096, D=2048, bf16, 1.01 GB at 4.7 to 5.4 TB/s.
#include <algorithm>

#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_lru_gate.h"
#include "mesa_lru_tile.h"

namespace mesa {

namespace {

constexpr int kThreads = 256;

// 64 tokens a tile, 16 elements a lane: with what the gradients need of them 3
// workgroups fit a CU, with 12 elements 4, with 8 elements 5; 191, 195 and 208 us
// at B=8, T=4096, D=2048, bf16, and 101 against 138 (12 elements, tiles of 48
// tokens) at B=256, T=64.
// A wave's tokens then start at a kept state.  Sequences of at most 8 or 32 tokens
// take one tile of as many (kShort), and the state before a wave's tokens from the
// waves before it: 26 and 54 us against 80 and 85 with 64 tokens at B=256, T=8 and
// 32, D=2048, bf16.
constexpr int kNw = 4, kTw = kLruChunk / 2, kTile = 2 * kNw * kTw;
static_assert(kNw >= 4, "three waves wait for other tiles, one folds this one's");

template <bool BF16, bool LINES, int TW>
__global__ __launch_bounds__(256, 3) void lru_bwd_kernel(LruParams p) {
  constexpr int NW = kNw, L = 2 * NW * TW;
  constexpr bool kShort = TW < kTw;
  constexpr uint32_t ES = BF16 ? 2 : 4;
  __shared__ Pair waves[NW][kLruSlab], pre[NW][kLruSlab];
  __shared__ LruCarry carry;
  __shared__ float sums[NW][kLruSlab];
  __shared__ unsigned ticket;
  const LruGrid grid(p.B, p.T, p.D, L);
  const int tiles = grid.tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane >> 5, c2 = 2 * (lane & 31);
  int i, chain;  // i: the tile's place in the scan
  if (!grid.take<LINES>(p.tickets, &ticket, i, chain)) return;
  const int b = chain / grid.slabs, c0 = (chain % grid.slabs) * kLruSlab;
  const int ch = c0 + c2, nch = p.D - ch;
  const int n = lru_length(p, b), live = (n + L - 1) / L;
  const int j = i < live ? live - 1 - i : i;             // the tiles with valid tokens, last first; then the others
  const int tw0 = (2 * wave + row) * TW, t0 = j * L + tw0;  // this lane's first token
  const size_t first = (size_t)b * p.T + (size_t)j * L;     // the tile's first row of the tensors
  const size_t grad = first * p.ld_grad * ES;
  const uint32_t grow = p.ld_grad * ES, goff = tw0 * grow + ch * ES;
  float* part = p.lam_part ? p.lam_part + ((size_t)b * tiles + j) * p.D + c0 + lane : nullptr;  // (none without tokens)
  const bool mine = c0 + lane < p.D;

  if (i >= live) {  // behind the length: zeros
    if (wave == 0 && mine) {
      const size_t e = (size_t)b * p.D + c0 + lane;
      if (part) *part = 0.f;
      if (i == 0 && p.dh0) p.dh0[e] = p.d_hfinal ? p.d_hfinal[e] : 0.f;
    }
    const float zero[2] = {};
#pragma unroll
    for (int s = 0; s < TW; ++s)
      if (t0 + s < p.T) {
        store_raw2<BF16, LINES>(static_cast<char*>(p.dx) + grad, goff + s * grow, zero, nch);
        store_raw2<BF16, LINES>(static_cast<char*>(p.dga) + grad, goff + s * grow, zero, nch);
        store_raw2<BF16, LINES>(static_cast<char*>(p.dgi) + grad, goff + s * grow, zero, nch);
      }
    return;
  }
  const bool whole = (j + 1) * L <= n;

  Raw2<BF16> dy[TW];
  float a[TW][2], u[TW][2], dxg[TW][2], q[TW][2], va[TW][2], vu[TW][2], sr1[TW][2], h[2];
  {
    Raw2<BF16> x[TW], ga[TW], gi[TW];
    uint32_t off[TW], doff[TW];
    const int lc = lru_load_channel(ch, p.D);
#pragma unroll
    for (int s = 0; s < TW; ++s) {  // rows behind n read row n - 1 and are not used
      const int t = whole ? tw0 + s : min(tw0 + s, n - 1 - j * L);
      off[s] = ((uint32_t)t * p.ld + lc) * ES;
      doff[s] = ((uint32_t)t * p.D + lc) * ES;
    }
    const size_t in = first * p.ld * ES;
    float lam[2];
    load_lam(p, ch, lam);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.ga) + in, off, ga);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.gi) + in, off, gi);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.x) + in, off, x);
    load_raw2<BF16, LINES>(static_cast<const char*>(p.dy) + first * p.D * ES, doff, dy);
    Raw2<false> state[1];  // before this wave's tokens, or the sequence
    const int chunk = kShort ? 0 : min(j * L + wave * kLruChunk, n - 1) / kLruChunk;
    const uint32_t none[1] = {0};
    load_raw2<false, LINES>(p.states + ((size_t)b * p.NC + chunk) * p.D + lc, none, state);
    to_own_channels(p.D, ch, x);
    to_own_channels(p.D, ch, ga);
    to_own_channels(p.D, ch, gi);
    to_own_channels(p.D, ch, dy);
    to_own_channels(p.D, ch, state);
#pragma unroll
    for (int e = 0; e < 2; ++e) h[e] = state[0].at(e);
    const float rate[2] = {lru_rate(lam[0], p.c), lru_rate(lam[1], p.c)};
#pragma unroll
    for (int s = 0; s < TW; ++s) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const LruGrad r = lru_cell_grad(x[s].at(e), ga[s].at(e), gi[s].at(e), rate[e]);
        a[s][e] = r.a;
        u[s][e] = r.u;
        dxg[s][e] = r.dx_g;
        q[s][e] = r.q;
        va[s][e] = r.va;
        vu[s][e] = r.vu;
        sr1[s][e] = r.sr1;
        settle(dxg[s][e]);
        settle(u[s][e]);
        settle(q[s][e]);
        settle(va[s][e]);
        settle(vu[s][e]);
        settle(sr1[s][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // behind n the state and the adjoint pass; what else is formed there comes from row
  // n - 1, which may hold infinities and NaN, so gradients are selected where they are
  // stored and summed
  if (!whole) {
#pragma unroll
    for (int s = 0; s < TW; ++s) {
      const bool off = t0 + s >= n;
      clear_if(off, dy[s]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        a[s][e] = __builtin_unpredictable(off) ? 1.f : a[s][e];
        u[s][e] = __builtin_unpredictable(off) ? 0.f : u[s][e];
      }
    }
  }
  // the states before this lane's tokens, and with them v / g = vu - va h
  Pair earlier[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    Pair on{a[0][e], u[0][e]}, all;
#pragma unroll
    for (int s = 1; s < TW; ++s) on = join(on, Pair{a[s][e], u[s][e]});
    join_rows<false>(on, row, earlier[e], all);
    if (kShort && row == 0) pre[wave][c2 + e] = all;
  }
  if constexpr (kShort) {
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW - 1; ++w)
      if (w < wave) {
#pragma unroll
        for (int e = 0; e < 2; ++e) h[e] = apply(pre[w][c2 + e], h[e]);
      }
    // (pre is written again behind the next barrier)
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    h[e] = apply(earlier[e], h[e]);
#pragma unroll
    for (int s = 0; s < TW; ++s) {
      vu[s][e] = __builtin_fmaf(-va[s][e], h[e], vu[s][e]);
      settle(vu[s][e]);
      h[e] = __builtin_fmaf(a[s][e], h[e], u[s][e]);
    }
  }
  Pair before[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    Pair back{a[TW - 1][e], a[TW - 1][e] * dy[TW - 1].at(e)}, all;
#pragma unroll
    for (int s = TW - 2; s >= 0; --s) back = join(back, Pair{a[s][e], a[s][e] * dy[s].at(e)});
    join_rows<true>(back, row, before[e], all);
    settle(before[e].A);
    settle(before[e].E);
    if (row == 0) waves[wave][c2 + e] = all;
  }
  float c_in = 0.f;  // the adjoint behind the last token
  if (wave == 1 && p.d_hfinal && mine) c_in = p.d_hfinal[(size_t)b * p.D + c0 + lane];
  settle(c_in);
  __syncthreads();
  uint64_t* words = p.words + (size_t)chain * lru_chain_words(tiles);
  Pair tile{1.f, 0.f};
  if (wave == 0) {
#pragma unroll
    for (int w = NW - 1; w >= 0; --w) {
      pre[w][lane] = tile;
      tile = join(tile, waves[w][lane]);
    }
    if (tiles > 1) publish(words + (size_t)i * kLruSlab + lane, tile);
  } else if (wave == 1) {
    carry_groups(words, tiles, i, lane, c_in, carry.h);
  } else if (wave < 4) {
    carry_tiles(words, i, wave - 2, lane, wave == 2 ? carry.early : carry.late);
  }
  __syncthreads();
  if (wave == 0 && i % kLruGroup == kLruGroup - 1) publish_group(words, tiles, i, lane, carry, tile);

#pragma unroll
  for (int s = 0; s < TW; ++s) repack(dy[s]);
  float c[2], vsum[2] = {};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = apply(carry.late[c2 + e], apply(carry.early[c2 + e], carry.h[c2 + e]));
    c[e] = apply(before[e], apply(pre[wave][c2 + e], c[e]));
  }
  auto token = [&](int s, int valid, bool live) {
    float dx[2], dga[2], dgi[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float g = c[e] + dy[s].at(e), v = live ? g * vu[s][e] : 0.f;
      vsum[e] += v;
      dx[e] = live ? g * dxg[s][e] : 0.f;
      dgi[e] = live ? dx[e] * q[s][e] : 0.f;
      dga[e] = live ? v * sr1[s][e] : 0.f;
      c[e] = a[s][e] * g;
    }
    store_raw2<BF16, LINES>(static_cast<char*>(p.dx) + grad, goff + s * grow, dx, valid);
    store_raw2<BF16, LINES>(static_cast<char*>(p.dga) + grad, goff + s * grow, dga, valid);
    store_raw2<BF16, LINES>(static_cast<char*>(p.dgi) + grad, goff + s * grow, dgi, valid);
  };
  if (whole && nch >= 2) {
#pragma unroll
    for (int s = TW - 1; s >= 0; --s) token(s, 2, true);
  } else {
#pragma unroll
    for (int s = TW - 1; s >= 0; --s) token(s, t0 + s < p.T ? nch : 0, t0 + s < n);
  }
  if (p.dh0 && t0 == 0) store_raw2<false, LINES>(p.dh0, ((size_t)b * p.D + ch) * 4, c, nch);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    vsum[e] = add_rows(vsum[e]);
    if (row == 0) sums[wave][c2 + e] = vsum[e];
  }
  __syncthreads();
  if (wave == 0 && mine) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += sums[w][lane];
    *part = v;
  }
}

// dlam from `rows` partial sums [rows, D] of dL / d log t: 16 channels a
// workgroup, 16 threads a channel.  A tile's sum has 64 tokens in fp32 (14 roundings);
// the tiles are summed in 64 bits: in fp32 the error grew with their number, 2200 half
// steps over 2^14 equal sequences of 200 tokens.
__global__ __launch_bounds__(kThreads) void lru_dlam_kernel(const float* part, const float* lam, float* dlam, int rows,
                                                            int D) {
  __shared__ double sums[16][16];
  const int k = threadIdx.x % 16, slice = threadIdx.x / 16, ch = blockIdx.x * 16 + k;
  double v = 0.;
  if (ch < D) {
#pragma unroll 8
    for (int r = slice; r < rows; r += 16) v += part[(size_t)r * D + ch];
  }
  sums[slice][k] = v;
  __syncthreads();
  if (slice == 0 && ch < D) {
    for (int i = 1; i < 16; ++i) v += sums[i][k];
    dlam[ch] = (float)(v * lru_rate_slope(lam[ch]));
  }
}

template <bool BF16, bool LINES, int TW>
hipError_t launch_t(const LruParams& p, hipStream_t s) {
  const LruGrid grid(p.B, p.T, p.D, 2 * kNw * TW);
  if (grid.tiles > 1) {
    if (const hipError_t e = launch_lru_ready(p, grid.chains * lru_chain_words(grid.tiles), s); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((lru_bwd_kernel<BF16, LINES, TW>), dim3(grid.workgroups()), dim3(64 * kNw), 0, s, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL(lru_dlam_kernel, dim3((p.D + 15) / 16), dim3(kThreads), 0, s, p.lam_part, p.lam, p.dlam,
                     p.T > 0 ? p.B * grid.tiles : 0, p.D);
  return hipGetLastError();
}

template <bool BF16, bool LINES>
hipError_t launch_tw(const LruParams& p, hipStream_t s) {
  if (p.T <= 2 * kNw) return launch_t<BF16, LINES, 1>(p, s);
  if (p.T <= 8 * kNw) return launch_t<BF16, LINES, 4>(p, s);
  return launch_t<BF16, LINES, kTw>(p, s);
}

}  // namespace

size_t lru_bwd_word_bytes(int B, int T, int D) {
  const LruGrid grid(B, T, D, kTile);
  return grid.chains * lru_chain_words(grid.tiles) * sizeof(uint64_t);
}

size_t lru_bwd_part_bytes(int B, int T, int D) {
  const LruGrid grid(B, T, D, kTile);
  return (size_t)B * grid.tiles * D * sizeof(float);
}

hipError_t launch_lru_bwd(bool bf16, const LruParams& p, hipStream_t s) {
  const bool lines = lru_whole_lines(bf16, {p.ld, p.D, p.ld_grad}, {p.x, p.ga, p.gi, p.dy, p.dx, p.dga, p.dgi});
  if (bf16) return lines ? launch_tw<true, true>(p, s) : launch_tw<true, false>(p, s);
  return lines ? launch_tw<false, true>(p, s) : launch_tw<false, false>(p, s);
}

}  // namespace mesa
