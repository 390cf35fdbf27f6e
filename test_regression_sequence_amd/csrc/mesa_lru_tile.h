// Tiles of the gated linear recurrence, h_t = a_t h_{t-1} + u_t per channel, and
// the scan that joins them.
//
// A token range [t0, t1) maps the state before it to the state behind it by
// h -> A h + E with A = prod a_t and E the state that starts from zero; ranges
// join as (A1, E1), (A2, E2) -> (A1 A2, A2 E1 + E2).  A workgroup of NW waves
// holds a tile of 64 channels by L = 2 NW TW tokens in registers: a wave is 2
// rows of 32 lanes, a lane holds 2 neighbouring channels of TW tokens in turn,
// row r of wave w those from (2 w + r) TW on.  Each lane folds its tokens, the
// rows of a wave are joined by a cross-row swap, the waves through LDS, and the
// tiles of one sequence and slab through device memory, so that every input is
// read once.  Two channels a lane, not four in four rows of 16 lanes: the loads
// are half as wide, but joining four rows took 22 instructions a channel, more
// than a quarter of what a token's gradients take (6 % of the forward's time and
// 5 % of the backward's at B=8, T=4096, D=2048, bf16).
#pragma once

#include <initializer_list>
#include <type_traits>

#include "mesa_common.h"
#include "mesa_kernels.h"
#include "mesa_lru_gate.h"
#include "mesa_rows.h"

namespace mesa {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kLruSlab = 64;    // channels of a tile
constexpr int kLruGroup = 16;   // tiles whose joined pair is published as one
constexpr int kLruSpan = 16;    // groups behind which the state is published

// Words of one chain (sequence and slab) of `tiles` tiles: a word per channel
// of each tile, then of each whole group, then of each whole span of groups.
inline __host__ __device__ size_t lru_chain_words(int tiles) {
  return (size_t)(tiles + tiles / kLruGroup + tiles / (kLruGroup * kLruSpan)) * kLruSlab;
}

struct Pair {  // h -> A h + E
  float A, E;
};
__device__ __forceinline__ Pair join(Pair first, Pair second) {
  return Pair{first.A * second.A, __builtin_fmaf(second.A, first.E, second.E)};
}
__device__ __forceinline__ float apply(Pair p, float h) { return __builtin_fmaf(p.A, h, p.E); }

// From the pairs of a wave's two rows: that of the row before this one (the
// identity for the first) and of both.  REV: row 1 comes first.
template <bool REV>
__device__ __forceinline__ void join_rows(Pair own, int row, Pair& before, Pair& all) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(own.A), __float_as_uint(own.A), false, false);
  const auto e = __builtin_amdgcn_permlane32_swap(__float_as_uint(own.E), __float_as_uint(own.E), false, false);
  constexpr int F = REV ? 1 : 0, S = 1 - F;
  const Pair first{__uint_as_float(a[F]), __uint_as_float(e[F])}, second{__uint_as_float(a[S]), __uint_as_float(e[S])};
  all = join(first, second);
  const bool later = (row != 0) != REV;
  before = Pair{later ? first.A : 1.f, later ? first.E : 0.f};
}

// The sum over a wave's two rows, in every lane.
__device__ __forceinline__ float add_rows(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Tiles of different chains need no order, so chains are dealt to at most 16
// classes of neighbouring slabs, each with a ticket counter on a cache line of
// its own: one counter for all hands out a ticket every 14 ns, which takes longer
// than the tiles (156 against 111 us forward, 290 against 195 backward at B=8,
// T=4096, D=2048, bf16).  A class's tickets run over its chains, then over time.
// Workgroups go round the 8 XCDs, each with a cache of its own.  Where slabs are
// whole cache lines nothing is shared, and by the eighths (workgroup i takes
// class i / 8) every XCD serves every class: with two neighbouring classes each
// an XCD reads the same columns of every row, which takes 124 to 133 against 113
// to 121 us at B=1, T=32768, D=2048, bf16.  Where slabs share lines, neighbours
// on one XCD read them once: 75 against 83 us forward, 136 against 163 backward
// at B=8, T=4096, D=1000, bf16.
constexpr int kLruClasses = 16, kLruCounterStride = 16;  // (in 4-byte words)

struct LruGrid {
  int slabs, tiles, chains, classes;
  __host__ __device__ LruGrid(int B, int T, int D, int L)
      : slabs((D + kLruSlab - 1) / kLruSlab), tiles(T > L ? (T + L - 1) / L : 1), chains(B * slabs),
        classes(chains < kLruClasses ? chains : kLruClasses) {}
  __host__ unsigned workgroups() const {  // 8 at a time, as many for each class as the largest has tiles
    return tiles > 1 ? 8u * classes * (((chains + classes - 1) / classes * tiles + 7) / 8) : (unsigned)chains;
  }
  __device__ int first_chain(int q) const { return (int)((long long)q * chains / classes); }
  // This workgroup's tile (in the scan's order) and chain; false if its class has none left.
  template <bool LINES>
  __device__ bool take(unsigned* tickets, unsigned* lds, int& j, int& chain) const {
    if (tiles == 1) {
      j = 0;
      chain = blockIdx.x;
      return true;
    }
    int q = blockIdx.x / 8 % classes;
    if constexpr (!LINES) q = classes == 16 ? blockIdx.x % 8 * 2 + blockIdx.x / 8 % 2 : blockIdx.x % classes;
    const int at = first_chain(q), m = first_chain(q + 1) - at;
    if (threadIdx.x == 0) *lds = atomicAdd(tickets + q * kLruCounterStride, 1u);
    __syncthreads();
    const unsigned t = __builtin_amdgcn_readfirstlane(*lds);
    j = t / m;
    chain = at + (int)(t % m);
    return j < tiles;
  }
};

// A published pair is one 64-bit word, so that a reader sees it whole or not at
// all and no ordering with other memory is needed.  kLruEmpty (written by
// lru_ready_kernel before the tiles run) marks a word not yet published; its
// low half is a NaN pattern that A is replaced in.
constexpr uint64_t kLruEmpty = ~0ull;

__device__ __forceinline__ void publish(uint64_t* word, Pair p) {
  uint32_t a = __float_as_uint(p.A);
  if (a == 0xFFFFFFFFu) a = 0x7FC00000u;
  __hip_atomic_store(word, ((uint64_t)__float_as_uint(p.E) << 32) | a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The N words at `word`, kLruSlab apart (one lane a channel), of which the
// first `count` are waited for; the rest read as the identity.
template <int N>
__device__ __forceinline__ void await(const uint64_t* word, int count, Pair (&p)[N]) {
  uint64_t v[N];
  bool missing;
  do {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = i < count ? __hip_atomic_load(word + (size_t)i * kLruSlab, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    missing = false;
#pragma unroll
    for (int i = 0; i < N; ++i) missing |= (uint32_t)v[i] == 0xFFFFFFFFu;
  } while (__any(missing));
#pragma unroll
  for (int i = 0; i < N; ++i)
    p[i] = i < count ? Pair{__uint_as_float((uint32_t)v[i]), __uint_as_float((uint32_t)(v[i] >> 32))} : Pair{1.f, 0.f};
}

// How tile j of a chain gets the state before it, from the state before tile 0:
// the pairs of the whole groups before its own are folded in order, then those
// of the earlier tiles of its group.  The fold over groups starts behind the last
// whole span, whose last tile publishes the state that the fold gives there.  (The
// tiles of a chain would otherwise read words as the square of their number: 7.1
// and 29.4 ms against 3.2 and 6.2, forward and backward, at B=1, T=2^20, D=2048,
// bf16; a state behind every group would make one chain of waits of them all.)
// Which words are folded in which order depends on j alone, so the result has the
// same bits in every run.  The tile
// reads the state before tile 0 before it publishes anything (so that the last
// tile, which has waited for all, may overwrite it), and publishes its own pair
// before it waits for any; the last tile of a group also
// publishes the group's, once it has the others.  Every wait ends: a class's
// tiles are handed out by tickets in the scan's order, so the first tile of a
// class that is not finished belongs to a workgroup that is running, and all
// that it waits for is published.
constexpr int kLruBatch = kLruGroup / 2;  // words one wave waits for at a time

// Three waves share the waiting, one lane per channel; each leaves its part of
// the fold in LDS.
struct LruCarry {
  Pair early[kLruSlab], late[kLruSlab];  // the group's earlier tiles, in two batches
  float h[kLruSlab];                     // the state behind the last whole group
};

template <int N>
__device__ __forceinline__ Pair fold(const Pair (&p)[N]) {
  Pair all = p[0];
#pragma unroll
  for (int k = 1; k < N; ++k) all = join(all, p[k]);
  return all;
}

__device__ __forceinline__ void carry_tiles(const uint64_t* words, int j, int part, int lane, Pair* to) {
  const int g = j / kLruGroup, i = j % kLruGroup - part * kLruBatch;
  Pair p[kLruBatch];
  await<kLruBatch>(words + (size_t)(g * kLruGroup + part * kLruBatch) * kLruSlab + lane, i, p);
  to[lane] = fold(p);
}

__device__ __forceinline__ void carry_groups(const uint64_t* words, int tiles, int j, int lane, float h, float* to) {
  const int g = j / kLruGroup, span = g / kLruSpan;
  const uint64_t* group = words + (size_t)tiles * kLruSlab + lane;
  if (span > 0) {
    Pair state[1];
    await<1>(group + (size_t)(tiles / kLruGroup + span - 1) * kLruSlab, 1, state);
    h = state[0].E;
  }
  for (int g0 = span * kLruSpan; g0 < g; g0 += kLruBatch) {
    Pair p[kLruBatch];
    await<kLruBatch>(group + (size_t)g0 * kLruSlab, g - g0, p);
#pragma unroll
    for (int k = 0; k < kLruBatch; ++k) h = apply(p[k], h);
  }
  to[lane] = h;
}

// What the last tile of a group publishes once it has its carry.
__device__ __forceinline__ void publish_group(uint64_t* words, int tiles, int j, int lane, const LruCarry& carry, Pair tile) {
  const int g = j / kLruGroup;
  const Pair group = join(join(carry.early[lane], carry.late[lane]), tile);
  uint64_t* to = words + (size_t)tiles * kLruSlab + lane;
  publish(to + (size_t)g * kLruSlab, group);
  if (g % kLruSpan == kLruSpan - 1)
    publish(to + (size_t)(tiles / kLruGroup + g / kLruSpan) * kLruSlab, Pair{0.f, apply(group, carry.h[lane])});
}

// A lane's channels of a token as stored (bf16: both in a word, so that the
// compiler keeps them packed).
template <bool BF16>
struct Raw2;
template <>
struct Raw2<true> {
  uint32_t v;
  __device__ __forceinline__ float at(int e) const { return __uint_as_float(e & 1 ? v & 0xFFFF0000u : v << 16); }
};
template <>
struct Raw2<false> {
  f32x2 v;
  __device__ __forceinline__ float at(int e) const { return v[e]; }
};
__device__ __forceinline__ void clear_if(bool off, Raw2<true>& r) { r.v = __builtin_unpredictable(off) ? 0 : r.v; }
__device__ __forceinline__ void clear_if(bool off, Raw2<false>& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i) r.v[i] = __builtin_unpredictable(off) ? 0 : r.v[i];
}

// Has v formed here.  The compiler otherwise moves work whose result is needed
// late behind the barriers, with all of its operands held until then.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// Hides that r is still what was loaded, so that a later use unpacks it again
// instead of holding its floats in registers meanwhile.
__device__ __forceinline__ void repack(Raw2<true>& r) { asm volatile("" : "+v"(r.v)); }
__device__ __forceinline__ void repack(Raw2<false>&) {}

// Where every row starts a cache line (128 bytes; a slab is then whole lines),
// the tensors are streamed: loads and stores carry the nontemporal hint, which
// takes 111 instead of 117 us forward and 191 instead of 204 backward at B=8,
// T=4096, D=2048, bf16.  Otherwise neighbouring slabs share lines, which have to
// stay in the caches until both are done: with the hint 109 instead of 81 us
// and 224 instead of 159 at B=8, T=4096, D=1000, bf16.
inline bool lru_whole_lines(bool bf16, std::initializer_list<int> strides, std::initializer_list<const void*> tensors) {
  size_t bits = 0;
  for (const int ld : strides) bits |= (size_t)ld * (bf16 ? 2 : 4);
  for (const void* q : tensors) bits |= reinterpret_cast<size_t>(q);
  return bits % 128 == 0;
}

// The first channel that a lane loads: its own, or where the row ends before it
// has two, the row's last two.  So loads are never predicated: a branch around
// them, even one that no lane of most slabs takes, had the compiler wait for all
// of them before the first use (6 % at B=1, T=32768, D=2048, bf16).
__device__ __forceinline__ int lru_load_channel(int ch, int D) { return min(ch, D - 2); }

// The two channels at `base` (uniform) + off[t] bytes of N rows.
template <bool BF16, bool LINES, int N>
__device__ __forceinline__ void load_raw2(const void* base, const uint32_t (&off)[N], Raw2<BF16> (&r)[N]) {
  typedef typename std::conditional<BF16, u32_any, f32x2_any>::type V;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const V* q = reinterpret_cast<const V*>(static_cast<const char*>(base) + off[t]);
    if constexpr (LINES) r[t].v = __builtin_nontemporal_load(q);
    else r[t].v = *q;
  }
}

// Where a lane's first channel is the row's last one, it was loaded second.
// (Lanes behind the row hold its last channels; nothing of theirs is stored.)
template <int N>
__device__ __forceinline__ void to_own_channels(int D, int ch, Raw2<true> (&r)[N]) {
  if (D & 1) {
    const int by = ch == D - 1 ? 16 : 0;
#pragma unroll
    for (int t = 0; t < N; ++t) r[t].v >>= by;
  }
}
template <int N>
__device__ __forceinline__ void to_own_channels(int D, int ch, Raw2<false> (&r)[N]) {
  if (D & 1) {
#pragma unroll
    for (int t = 0; t < N; ++t) r[t].v[0] = __builtin_unpredictable(ch == D - 1) ? r[t].v[1] : r[t].v[0];
  }
}

// The first n of a lane's channels to `base` + off bytes, rounded to nearest even.
template <bool BF16, bool LINES>
__device__ __forceinline__ void store_raw2(void* base, size_t off, const float (&y)[2], int n) {
  typedef typename std::conditional<BF16, uint32_t, f32x2>::type V;
  typedef typename std::conditional<BF16, u32_any, f32x2_any>::type VAny;
  char* q = static_cast<char*>(base) + off;
  V o;
  if constexpr (BF16) o = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{y[0], y[1]}, bf16x2));
  else o = f32x2{y[0], y[1]};
  if (n >= 2) {
    if constexpr (LINES) __builtin_nontemporal_store(o, reinterpret_cast<VAny*>(q));
    else *reinterpret_cast<VAny*>(q) = o;
  } else if (n > 0) {
    if constexpr (BF16) *reinterpret_cast<uint16_t*>(q) = (uint16_t)o;
    else *reinterpret_cast<float*>(q) = y[0];
  }
}

__device__ __forceinline__ int lru_length(const LruParams& p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// A lane's channels of lam.
__device__ __forceinline__ void load_lam(const LruParams& p, int ch, float (&lam)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) lam[e] = p.lam[min(ch + e, p.D - 1)];
}

}  // namespace mesa
