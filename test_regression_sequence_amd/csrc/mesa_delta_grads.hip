// Gated delta rule, backward: the gradients of one chunk's tokens.
//
// With S0 the state before the chunk, dS the gradient at the state behind it, W
// from the forward walk, U = beta W and E from the walk back,
//     Z = lower(dO U^T D),   Y = -strict_lower(E U^T D) diag(beta on rows),
//     dQ = c dO S0 + Z K,    dV = beta E,    dbeta = E . W,
//     dK = tail U dS - c beta E S0 + Z^T Q + (Y + Y^T) K,
// and the logarithm of token i's forget factor acts on every pair t >= i > j, on
// what tokens t >= i read of S0, on what tokens j < i leave behind, and on S0 -> S'.
// Each of these terms has the factor itself as a factor, so their sum over it is the
// gradient at it; for factors below 2^-64, 0 among them, the terms are added up once more
// with the factor left out, as the products with it leave fp32's range.
//
// One workgroup a (sequence, head, chunk): a wave owns 16 tokens and half of the
// key dimension (and of Z and Y one), a lane one token in every result tile, so
// that rows are scaled by lane constants and leave in pieces of 4 columns.  The first part
// runs over the value dimension in slices of 32 (S0, dS and U through LDS, the next slice's
// loads in flight), the second over the chunk's pairs.  All products keep fp32's precision (three bf16 planes).
//
// At B=8 H=16 T=4096 d=128 bf16 it moves 2.45 GB in 691 to 718 us, 3.4 to 3.6 TB/s, 70 %
// of a large copy's rate.  The vector unit works 33 % of the time (a third of it on planes),
// the matrix unit 23 % and LDS 26 %, hardly at once: registers leave room for two waves a SIMD,
// which the barriers keep in step.  A workgroup that goes from chunk to chunk, its loads ahead
// across the second part, took the same time.  Sums for the gates by eight lanes a token in
// place of one wave's scans cost more in LDS than they saved (730 -> 805 us).
#include <algorithm>

#include "mesa_delta_tile.h"

namespace mesa {

namespace {

template <int DK, bool BF16>
struct GradLds {
  static constexpr int NP = BF16 ? 1 : 3, NZ = 3;
  static constexpr int kState = 32 * DK * 2, kU = 64 * 64, kPlane = 64 * DK * 2, kZ = 64 * 128;
  static constexpr int kS = 0, kD = 3 * kState, kUAt = 6 * kState, kEAt = kUAt + 3 * kU, kOAt = kEAt + 3 * kU,
                       kSlice = kOAt + NP * kU;
  // Two workgroups a CU hide one another's waits where 128 registers a lane do (keys and
  // queries then wait for the slices' end): 50 -> 41 us at B=4 H=8 T=2048 d=64 (44 with three
  // planes for Z and Y).  Else two slices in LDS where they fit: one is converted beside the
  // products of the other, a barrier a slice (750 -> 730 us at B=8 H=16 T=4096 d=128 bf16).
  static constexpr bool kPair = BF16 && DK <= 64, kTwo = !kPair && (BF16 || DK < 128);
  static constexpr int kFirst = (kTwo ? 2 : 1) * kSlice;
  static constexpr int kK = 0, kQ = NP * kPlane, kZAt = 2 * NP * kPlane, kYAt = kZAt + NZ * kZ,
                       kSmall = kYAt + NZ * kZ, kSecond = kSmall + 12 * 64 * 4;
  static constexpr int kBytes = kFirst > kSecond ? kFirst : kSecond;
};

// Forget factors below this have their gradient from terms without them.
constexpr float kSmallGate = 0x1p-64f;

template <int DK, bool BF16>
__global__ __launch_bounds__(512, BF16 && DK <= 64 ? 4 : 2) void delta_grads_kernel(DeltaParams p) {
  using L = GradLds<DK, BF16>;
  using Out = std::conditional_t<BF16, __bf16, float>;
  constexpr int NP = L::NP, NZ = L::NZ, MH = DK / 32, KS = DK / 32;
  constexpr bool PAIR = L::kPair;
  constexpr int kPieces = 8 * DK, NS = (kPieces + 511) / 512;  // 16-byte pieces of a state's slice
  __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
  __shared__ __attribute__((aligned(16))) DeltaGates gates;
  __shared__ float cols[8][64], rest[2][64], diag[2][64], part[2][64], behind[2][64], dbetas[64], gammas[64], red[8];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, g = lane >> 4;
  // waves w and w + 4 share a SIMD: tiles 0 .. 3 have 1 .. 4 tiles of pairs
  const int half = wave >> 2, tile = half ? 7 - wave : wave;
  const int own = 16 * tile + r;  // this lane's token
  // a thread's pieces of a slice: 4 columns of a row of the states, and of a token (row `from`) of W, E and dO
  const int from = tid >> 3, at4 = (tid & 7) * 4;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  cols[wave][lane] = 0.f;
  const TileRows<DK> rows(lane);
  const TileRows<32> slice_rows(lane);
  const TileRows<64> pair_rows(lane);
  const TileColumns<DK, MH> columns(lane, MH * half);
  const TileColumns<64, 1> pair_columns(lane, tile);

  const int64_t unit = blockIdx.x;
  const uint32_t bh = blockIdx.x / p.by_nc;
  const int c = blockIdx.x % p.by_nc, b = bh / p.by_h, h = bh % p.by_h, hk = (uint32_t)h / p.by_shared;
  const int64_t t0 = 64 * (int64_t)c;
  const int live = min(delta_length(p, b) - (int)t0, 64), here = min(p.T - (int)t0, 64);
  const bool there = own < here, valid = own < live;
  const uint32_t w_at = (from * p.dv + at4) * 4, do_at = (from * (uint32_t)p.d_o.t + at4) * sizeof(Out),
                 dv_at = (from * (uint32_t)p.dv_.t + at4) * sizeof(Out);
  auto rows_at = [&](const DeltaRows& x, int head) {
    return window_at(static_cast<const char*>(x.at) + (b * x.b + head * x.h + t0 * x.t) * sizeof(Out));
  };
  f32x4 sl[NS], dl[NS], wl, el, ol;
  const Window states = window_at(p.states + unit * p.dv * DK), dstates = window_at(p.dstates + unit * p.dv * DK),
               ws = window_at(p.w + unit * 64 * p.dv), es = window_at(p.e + unit * 64 * p.dv),
               dos = rows_at(p.d_o, h), dvs = rows_at(p.dv_, h);
  auto load = [&](int d0) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int piece = tid + 512 * n, row = piece / (DK / 4);
      const uint32_t at = row < min(32, p.dv - d0) ? piece * 16 : kNowhere;
      sl[n] = __builtin_bit_cast(f32x4, window_load(states, at, d0 * DK * 4));
      dl[n] = __builtin_bit_cast(f32x4, window_load(dstates, at, d0 * DK * 4));
    }
    const bool there = at4 < p.dv - d0;
    wl = __builtin_bit_cast(f32x4, window_load(ws, there ? w_at : kNowhere, d0 * 4));
    el = __builtin_bit_cast(f32x4, window_load(es, there ? w_at : kNowhere, d0 * 4));
    ol = window_row<BF16>(dos, there && from < live ? do_at : kNowhere, d0 * sizeof(Out));
  };
  RowLoads<DK, BF16, 512> kl, ql;
  CopyLoads<sizeof(DeltaGates), 512> gl;

  const bool heads = p.dq_heads != nullptr;
  const int at_key = 16 * MH * half + 4 * g;
  const int64_t heads_at = ((int64_t)bh * p.T + t0) * DK;
  const Window dqs = heads ? window_at(p.dq_heads + heads_at) : rows_at(p.dq, hk),
               dks = heads ? window_at(p.dk_heads + heads_at) : rows_at(p.dk_, hk);
  auto put = [&](const f32x4 (&dq)[MH], const f32x4 (&dk)[MH]) {
#pragma unroll
    for (int i = 0; i < MH; ++i) {
      if (heads) {
        const uint32_t to = there ? (own * DK + at_key) * 4 : kNowhere;
        window_store(dqs, to, 64 * i, dq[i]);
        window_store(dks, to, 64 * i, dk[i]);
      } else {
        window_store_row<BF16>(dqs, there ? (own * (uint32_t)p.dq.t + at_key) * sizeof(Out) : kNowhere,
                               16 * i * sizeof(Out), dq[i]);
        window_store_row<BF16>(dks, there ? (own * (uint32_t)p.dk_.t + at_key) * sizeof(Out) : kNowhere,
                               16 * i * sizeof(Out), dk[i]);
      }
    }
  };

  f32x4 aq[MH], ak[MH], ad[MH];  // dO S0, E S0, U dS: columns 16 (MH half + i) + 4 g + e
#pragma unroll
  for (int i = 0; i < MH; ++i) aq[i] = ak[i] = ad[i] = zero;
  if (live <= 0) {  // behind the sequence
    put(aq, ak);
    for (int d0 = 0; d0 < p.dv; d0 += 32)
      window_store_row<BF16>(dvs, from < here && at4 < p.dv - d0 ? dv_at : kNowhere, d0 * sizeof(Out), zero);
    if (tid < here) *gate_at(p.dgamma, b, h, t0 + tid) = *gate_at(p.dbeta, b, h, t0 + tid) = 0.f;
    return;
  }

  f32x4 zy[4] = {zero, zero, zero, zero};  // rows j, a lane's token t: U dO^T (half 0) or U E^T (half 1)
  float dbeta = 0.f, along = 0.f;
  const float beta_from = p.gates[unit].beta[from];
  load(0);
  auto load_rest = [&]() {
    kl.load(p.k.at, b * p.k.b + hk * p.k.h + t0 * p.k.t, p.k.t, live, DK, tid);
    ql.load(p.q.at, b * p.q.b + hk * p.q.h + t0 * p.q.t, p.q.t, live, DK, tid);
    gl.load(p.gates + unit, tid);
  };
  if constexpr (!PAIR) load_rest();
  if (tid < 64) gammas[tid] = tid < live ? *gate_at(p.gamma, b, h, t0 + tid) : 1.f;
  // the slice in registers to LDS, in planes
  auto stage = [&](int d0, char* to) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int piece = tid + 512 * n, row = piece / (DK / 4), col = piece % (DK / 4) * 4;
      if (kPieces % 512 != 0 && row >= 32) continue;
      bf16x4 a[3], d[3];
      split4<3>(sl[n], a);
      split4<3>(dl[n], d);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        *reinterpret_cast<bf16x4*>(to + L::kS + i * L::kState + tile_at<DK>(row, 2 * col)) = a[i];
        *reinterpret_cast<bf16x4*>(to + L::kD + i * L::kState + tile_at<DK>(row, 2 * col)) = d[i];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) along = fmaf(sl[n][e], dl[n][e], along);
    }
    const uint32_t at = tile_at<32>(from, 2 * at4);
    bf16x4 uu[3], x[3], o[NP];
    split4<3>(wl * beta_from, uu);
    split4<3>(el, x);
    split4<NP>(ol, o);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      *reinterpret_cast<bf16x4*>(to + L::kUAt + i * L::kU + at) = uu[i];
      *reinterpret_cast<bf16x4*>(to + L::kEAt + i * L::kU + at) = x[i];
      if (i < NP) *reinterpret_cast<bf16x4*>(to + L::kOAt + i * L::kU + at) = o[i];
    }
    window_store_row<BF16>(dvs, from < here && at4 < p.dv - d0 ? dv_at : kNowhere, d0 * sizeof(Out), el * beta_from);
#pragma unroll
    for (int n = 0; n < 4; ++n) dbeta = fmaf(el[n], wl[n], dbeta);
  };
  auto products = [&](const char* slice) {
    {
      const Planes<NP> of = slice_rows.template planes<NP>(slice + L::kOAt, L::kU, 16 * tile, 0);
      const Planes<3> ef = slice_rows.template planes<3>(slice + L::kEAt, L::kU, 16 * tile, 0);
#pragma unroll
      for (int i = 0; i < MH; ++i) {
        const Planes<3> s = columns.template planes<3>(slice + L::kS, L::kState, 0, i);
        aq[i] = mma<2>(s, of, aq[i]);
        ak[i] = mma<2>(s, ef, ak[i]);
        fence<PAIR>();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= tile) {
          const Planes<3> x = slice_rows.template planes<3>(slice + L::kUAt, L::kU, 16 * j, 0);
          zy[j] = half ? mma<2>(x, ef, zy[j]) : mma<2>(x, of, zy[j]);
        }
    }
    fence<PAIR>();
    const Planes<3> uf = slice_rows.template planes<3>(slice + L::kUAt, L::kU, 16 * tile, 0);
#pragma unroll
    for (int i = 0; i < MH; ++i) ad[i] = mma<2>(columns.template planes<3>(slice + L::kD, L::kState, 0, i), uf, ad[i]);
  };
  // (Loads behind the last slice give zeros; with a branch around them the compiler waits, 767 -> 835 us.)
  if constexpr (L::kTwo) {
    stage(0, lds);
    load(32);
    for (int d0 = 0; d0 < p.dv; d0 += 32) {
      char *now = lds + (d0 >> 5 & 1) * L::kSlice, *next = lds + (~d0 >> 5 & 1) * L::kSlice;
      __syncthreads();
      products(now);
      stage(d0 + 32, next);
      load(d0 + 64);
    }
  } else {
    for (int d0 = 0; d0 < p.dv; d0 += 32) {
      __syncthreads();
      stage(d0, lds);
      load(d0 + 32);
      __syncthreads();
      products(lds);
    }
  }

  if constexpr (PAIR) load_rest();
  __syncthreads();
  kl.store(lds + L::kK, L::kPlane, tid);
  ql.store(lds + L::kQ, L::kPlane, tid);
  gl.store(reinterpret_cast<char*>(&gates), tid);
  __syncthreads();

  // The tokens with small factors; for each of these, what a wave's pairs across it give, and what any token reads
  // of S0 and leaves behind, all without its factor
  const uint64_t small = __ballot(gammas[lane] < kSmallGate), zeros = __ballot(gammas[lane] == 0.f);
  float(*const across)[64] = reinterpret_cast<float(*)[64]>(lds + L::kSmall), (*const reads)[64] = across + 8,
                             (*const leaves)[64] = across + 10;
  if (small) across[wave][lane] = 0.f;
  auto own_log = [&](int i) { return gates.g[i] - (i ? gates.g[i - 1] : 0.0); };

  float sum = 0.f, earlier = 0.f;
  const float beta_own = gates.beta[own];
  char* const pairs = lds + (half ? L::kYAt : L::kZAt);
  {
    Planes<NP> f[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) f[s] = rows.template planes<NP>(lds + (half ? L::kK : L::kQ), L::kPlane, 16 * tile, s);
    const double gt = gates.g[own];
    const float weight = half ? -beta_own : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4 x = zero;
      if (j <= tile) {
        f32x4 dot = zero;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          dot = mma<2>(rows.template planes<NP>(lds + L::kK, L::kPlane, 16 * j, s), f[s], dot);
        const int at = 16 * j + 4 * g;
        // (factors of 0 that every pair of these tiles lies across)
        const uint64_t between = zeros & ((2ull << (16 * tile)) - 1) & ~((1ull << (16 * j + 15) << 1) - 1);
        for (uint64_t left = small; left; left &= left - 1) {
          const int i = __builtin_ctzll(left);
          if (i <= 16 * j || i >= 16 * tile + 16 || (between & ~(1ull << i))) continue;
          const double without = gt - own_log(i);
          float pairs = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pairs += at + e < i && i <= own ? zy[j][e] * weight * dot[e] * decay_exact(without, gates.g[at + e]) : 0.f;
          pairs = wave_sum(pairs);
          if (lane == 0) across[wave][i] += pairs;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = zy[j][e] * decay_exact(gt, gates.g[at + e]) * weight;
        if (j < tile) {  // pairs with tokens of earlier tiles: sums over them, and over the tile's tokens
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            earlier += x[e] * dot[e];
            const float column = group_sum<16>(x[e] * dot[e]);
            if (r == 0) cols[wave][at + e] = column;
          }
        } else {  // pairs within the tile, for each token i those with t >= i > j
          const int last = own - half;  // Y has no diagonal
          float before[4], run = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = at + e <= last ? x[e] : 0.f;
            before[e] = run;
            run += at + e <= last ? x[e] * dot[e] : 0.f;
          }
          float front = 0.f;
#pragma unroll
          for (int n = 1; n < 4; ++n) {
            const float of_group = __shfl_up(run, 16 * n);
            if (g >= n) front += of_group;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float column = group_sum<16>(at + e <= own ? front + before[e] : 0.f);
            if (r == 0) diag[half][at + e] = column;
          }
        }
      }
      if (j <= (tile | 1)) {
        bf16x4 a[NZ];
        split4<NZ>(x, a);
#pragma unroll
        for (int n = 0; n < NZ; ++n)
          *reinterpret_cast<bf16x4*>(pairs + n * L::kZ + tile_at<64>(own, 32 * j + 8 * g)) = a[n];
      }
    }
  }
  const float cc = gates.c[own], tail = gates.tail[own], cb = cc * beta_own;
  float left = 0.f;  // what this token leaves behind the chunk
  auto own_values = [&](const char* plane, int i) {
    return half ? rows.template values<NP>(plane, L::kPlane, 16 * tile, MH + i)
                : rows.template values<NP>(plane, L::kPlane, 16 * tile, i);
  };
  if (small) {
    float of_state = 0.f, behind_it = 0.f;
#pragma unroll
    for (int i = 0; i < MH; ++i) {
      const f32x4 q = own_values(lds + L::kQ, i), k = own_values(lds + L::kK, i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        of_state += q[e] * aq[i][e] - beta_own * k[e] * ak[i][e];
        behind_it += k[e] * ad[i][e];
      }
    }
    of_state = sum_lane_groups(of_state);
    behind_it = sum_lane_groups(behind_it);
    if (g == 0) {
      reads[half][own] = of_state;
      leaves[half][own] = behind_it;
    }
  }
#pragma unroll
  for (int i = 0; i < MH; ++i) {
    const f32x4 q = own_values(lds + L::kQ, i), k = own_values(lds + L::kK, i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum += cc * q[e] * aq[i][e] - cb * k[e] * ak[i][e];
      left += tail * k[e] * ad[i][e];
    }
    aq[i] *= cc;
    ak[i] = tail * ad[i] - cb * ak[i];
  }
  sum = sum_lane_groups(sum);
  left = sum_lane_groups(left);
  earlier = sum_lane_groups(earlier);
  dbeta = group_sum<8>(dbeta);
  along = wave_sum(along);
  if (g == 0) {
    part[half][own] = sum;
    behind[half][own] = left;
    rest[half][own] = earlier;
  }
  if ((tid & 7) == 0) dbetas[from] = dbeta;
  if (lane == 0) red[wave] = along;
  __syncthreads();

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (2 * s <= tile) {
      const Planes<NZ> zf = pair_rows.template planes<NZ>(lds + L::kZAt, L::kZ, 16 * tile, s);
      const Planes<NZ> yf = pair_rows.template planes<NZ>(lds + L::kYAt, L::kZ, 16 * tile, s);
#pragma unroll
      for (int i = 0; i < MH; ++i) {
        const Planes<NP> k = columns.template planes<NP>(lds + L::kK, L::kPlane, 32 * s, i);
        aq[i] = mma<2>(k, zf, aq[i]);
        ak[i] = mma<2>(k, yf, ak[i]);
      }
    }
    if (2 * s + 1 >= tile) {
      const Planes<NZ> zf = pair_columns.template planes<NZ>(lds + L::kZAt, L::kZ, 32 * s, 0);
      const Planes<NZ> yf = pair_columns.template planes<NZ>(lds + L::kYAt, L::kZ, 32 * s, 0);
#pragma unroll
      for (int i = 0; i < MH; ++i) {
        ak[i] = mma<2>(columns.template planes<NP>(lds + L::kQ, L::kPlane, 32 * s, i), zf, ak[i]);
        ak[i] = mma<2>(columns.template planes<NP>(lds + L::kK, L::kPlane, 32 * s, i), yf, ak[i]);
      }
    }
  }
  if (!valid) {
#pragma unroll
    for (int i = 0; i < MH; ++i) aq[i] = ak[i] = zero;
  }
  put(aq, ak);

  // The gradient at log gamma_i, each term added up where it counts and nowhere taken away again:
  // what tokens t >= i read of S0, what tokens j < i leave behind, S0 -> S', and the pairs t >= i > j:
  // those within i's tile, those of t >= i in it with earlier tiles, those of later tiles with j < i.
  if (wave == 0) {
    const int in = lane >> 4;
    double x = (double)part[0][lane] + part[1][lane], y = (double)behind[0][lane] + behind[1][lane], whole = 0.0;
    float tiles = rest[0][lane] + rest[1][lane], later[3];
#pragma unroll
    for (int t = 1; t < 4; ++t) later[t - 1] = lane < 16 * t ? cols[t][lane] + cols[7 - t][lane] : 0.f;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const double after = __shfl_down(x, off), before = __shfl_up(y, off);
      if (lane + off < 64) x += after;
      if (lane >= off) y += before;
      if (off < 16) {
        const float below = __shfl_down(tiles, off);
        if (r + off < 16) tiles += below;
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const float above = __shfl_up(later[t], off);
        if (lane >= off) later[t] += above;
      }
    }
    y = __shfl_up(y, 1);
    if (lane > 0) x += y;
#pragma unroll
    for (int t = 1; t < 4; ++t) {
      const float above = __shfl_up(later[t - 1], 1);
      if (lane > 0 && in < t) x += above;
    }
    x += (double)tiles + diag[0][lane] + diag[1][lane];
#pragma unroll
    for (int n = 0; n < 8; ++n) whole += red[n];
    x = (x + gates.c[63] * whole) / (double)gammas[lane];
    for (uint64_t left = small; left; left &= left - 1) {
      const int i = __builtin_ctzll(left);
      const double without = own_log(i), all = gates.g[63] - without;
      double sum = lane >= i ? ((double)reads[0][lane] + reads[1][lane]) * decay_exact(gates.g[lane], without)
                             : ((double)leaves[0][lane] + leaves[1][lane]) * decay_exact(all, gates.g[lane]);
#pragma unroll
      for (int off = 1; off < 64; off *= 2) sum += __shfl_xor(sum, off);
      sum += decay_exact(all, 0.0) * whole;
#pragma unroll
      for (int n = 0; n < 8; ++n) sum += across[n][i];
      if (lane == i) x = sum;
    }
    if (lane < here) {
      *gate_at(p.dgamma, b, h, t0 + lane) = lane < live ? (float)x : 0.f;
      *gate_at(p.dbeta, b, h, t0 + lane) = lane < live ? dbetas[lane] : 0.f;
    }
  }
}

// Sums over the heads that share keys, in their order: 4 columns of a token a thread, 256 threads a
// piece of a head.  At memory's rate (B=4 H=8 Hk=4 T=2048 d=64: 7 us for 42 MB).
template <int DK, bool BF16>
__global__ __launch_bounds__(256) void delta_heads_kernel(DeltaParams p, uint32_t all, Divisor by_pieces) {
  using Out = std::conditional_t<BF16, __bf16, float>;
  const int R = p.H / p.Hk;
  for (uint32_t piece = blockIdx.x; piece < all; piece += gridDim.x) {
    const uint32_t bhk = piece / by_pieces, b = bhk / (uint32_t)p.Hk, hk = bhk - b * p.Hk;
    const int64_t at = (int64_t)(piece % by_pieces) * 256 + threadIdx.x, t = at / (DK / 4);
    const int col = (int)(at % (DK / 4)) * 4;
    if (t >= p.T) continue;
    f32x4 q = {0.f, 0.f, 0.f, 0.f}, k = q;
    for (int i = 0; i < R; ++i) {
      const int64_t from = ((((int64_t)b * p.H + (int64_t)hk * R + i) * p.T) + t) * DK + col;
      q += *reinterpret_cast<const f32x4*>(p.dq_heads + from);
      k += *reinterpret_cast<const f32x4*>(p.dk_heads + from);
    }
    store_out4<Out>(p.dq.at, b * p.dq.b + hk * p.dq.h + t * p.dq.t + col, q);
    store_out4<Out>(p.dk_.at, b * p.dk_.b + hk * p.dk_.h + t * p.dk_.t + col, k);
  }
}

template <int DK, bool BF16>
hipError_t launch(const DeltaParams& p, hipStream_t s) {
  delta_grads_kernel<DK, BF16><<<(uint32_t)((int64_t)p.B * p.H * p.NC), 512, 0, s>>>(p);
  if (p.dq_heads) {
    const uint32_t pieces = (uint32_t)(((int64_t)p.T * (DK / 4) + 255) / 256), all = (uint32_t)(p.B * p.Hk) * pieces;
    delta_heads_kernel<DK, BF16><<<std::min(all, 1u << 20), 256, 0, s>>>(p, all, divisor(pieces));
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(bool bf16, const DeltaParams& p, hipStream_t s) {
  if (p.dk == 128) return bf16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  if (p.dk == 64) return bf16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  return bf16 ? launch<32, true>(p, s) : launch<32, false>(p, s);
}

}  // namespace mesa
