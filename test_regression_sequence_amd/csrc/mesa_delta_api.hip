// C ABI of the gated delta rule and of gradient clipping: argument validation,
// workspace carving, kernel launches.  Every check runs before the first launch,
// so a failing call writes nothing.
#include <algorithm>
#include <cmath>

#include "../../include/mesa.h"
#include "mesa_check.h"
#include "mesa_clip.h"
#include "mesa_delta.h"

using namespace mesa;

namespace {

struct Dim {
  int64_t size, stride;
};

// The dimensions of `heads` heads' rows that have more than one index, from the
// smallest stride to the largest; their number.
int dims_of(const mesa_delta_desc* d, int heads, const mesa_rows& r, Dim (&dims)[3]) {
  int n = 0;
  for (const Dim& x : {Dim{d->B, r.b}, Dim{heads, r.h}, Dim{d->T, r.t}})
    if (x.size > 1) dims[n++] = x;
  std::sort(dims, dims + n, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  return n;
}

// Whether no two rows of `width` elements share one (each dimension steps over all smaller ones).
bool apart(const mesa_delta_desc* d, int heads, int width, const mesa_rows& r) {
  if (d->T == 0) return true;
  Dim dims[3];
  const int n = dims_of(d, heads, r, dims);
  int64_t extent = width;
  for (int i = 0; i < n; ++i) {
    if (dims[i].stride < extent) return false;
    extent += dims[i].stride * (dims[i].size - 1);
  }
  return true;
}

// What such rows of `width` elements of `bytes` bytes fill; where rows share elements or lie
// between one another, all from the first element to the last.
Blocks blocks_of(const mesa_delta_desc* d, int heads, int width, size_t bytes, const mesa_rows& r, const void* at) {
  Dim dims[3];
  const int n = dims_of(d, heads, r, dims);
  if (d->T == 0) return {at, 0};
  int64_t piece = width, extent = width;
  bool nested = true;
  int i = 0;
  while (i < n && dims[i].stride == piece) piece *= dims[i++].size;
  Blocks x{at, piece * bytes};
  for (int64_t reach = piece; i < n; ++i) {
    nested = nested && dims[i].stride >= reach;
    reach += dims[i].stride * (dims[i].size - 1);
    x.step[x.dims++] = {(size_t)dims[i].size, dims[i].stride * bytes};
  }
  if (nested) return x;
  for (i = 0; i < n; ++i) extent += dims[i].stride * (dims[i].size - 1);
  return {at, extent * bytes};
}

// Gates are read one by one.
template <size_t N>
bool floats_aligned(const float* const (&ptrs)[N]) {
  for (const float* ptr : ptrs)
    if (reinterpret_cast<uintptr_t>(ptr) & 3u) return false;
  return true;
}

// (with B H <= 2^22 and T <= 2^28, checked below, no offset in bytes passes 2^62)
constexpr int64_t kMaxStride = (int64_t)1 << 36, kMaxTokenStride = 1 << 20;

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }
bool strides_ok(const mesa_rows& r) { return stride_ok(r.b) && stride_ok(r.h) && stride_ok(r.t); }

// Rows start at multiples of 16 bytes (a stride that no index uses does not matter).
bool rows_aligned(const mesa_delta_desc* d, int heads, const mesa_rows& r) {
  const int64_t e = d->dtype == MESA_BF16 ? 8 : 4;
  return d->T == 0 || ((d->B == 1 || r.b % e == 0) && (heads == 1 || r.h % e == 0) && (d->T == 1 || r.t % e == 0));
}

int chunks_of(const mesa_delta_desc* d) { return (int)(((int64_t)d->T + kDeltaChunk - 1) / kDeltaChunk); }

mesa_status check_delta(const mesa_delta_desc* d) {
  if (!d || d->B < 1 || d->H < 1 || d->Hk < 1 || d->T < 0 || d->H % d->Hk != 0 || !dtype_ok(d->dtype) || d->dk < 1 ||
      d->dv < 1)
    return MESA_ERR_INVALID_ARG;
  for (const mesa_rows* r : {&d->q, &d->k, &d->v, &d->o, &d->gamma, &d->beta})
    if (!strides_ok(*r)) return MESA_ERR_INVALID_ARG;
  if ((d->dk != 32 && d->dk != 64 && d->dk != 128) || d->dv % 16 != 0 || d->dv > 1024) return MESA_ERR_UNSUPPORTED;
  // offsets within a chunk of tokens have 32 bits
  for (const mesa_rows* r : {&d->q, &d->k, &d->v, &d->o, &d->gamma, &d->beta})
    if (d->T > 1 && r->t > kMaxTokenStride) return MESA_ERR_UNSUPPORTED;
  // launches of at most 2^32 threads
  if ((double)d->B * d->H * std::max(chunks_of(d), (d->dv + 63) / 64) > (double)(1 << 22)) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

// In how many segments a walk goes.  A walk of one workgroup a head and 64 columns takes
// its chunks one after the other; with fewer of those than the 256 CUs, segments of it run
// side by side, after a launch that finds what each makes of unit rows and of zero (128 of
// dv + dk columns a workgroup; the first segment runs with it) and one that joins them.  In
// times of one chunk (of 128: 3.4 us, in fp32 5.6), the two launches take about 3 and
// half a chunk a segment; half of that in fp32, as when its chunk took twice a bf16 one's time.
// Measured, one sequence, calls in segments and in one walk, forward and gradients on kept
// states: 1024 tokens and 4 heads of 64, 38 and 57 us, 42 and 62, in fp32 44 and 76, 51 and 87;
// 4 heads of 128, 52 and 70, 67 and 87, in fp32 68 and 110, 86 and 140; 4096 tokens and 16
// heads of 128, 109 and 244, 194 and 337, in fp32 162 and 398, 273 and 564.
constexpr int kMaxSegments = 32;

int64_t values_of(const mesa_delta_desc* d) { return (d->dv + 63) / 64; }
int64_t both_of(const mesa_delta_desc* d) { return (d->dv + d->dk + 127) / 128; }

// Bounds of heads and of heads times segments where a walk goes in segments (of all B and T).  Where the
// openings take no fewer workgroups than the walk the rule itself gives them (128 and 472 workgroups of
// 64 columns); else they bind it, to at most a tenth more by its own reckoning, as 31 short segments that
// take many rounds would save no more and hold 8184 workgroups' states.
int64_t most_heads(const mesa_delta_desc* d) { return (both_of(d) < values_of(d) ? 341 : 128) / values_of(d); }
int64_t most_segments(const mesa_delta_desc* d) { return (both_of(d) < values_of(d) ? 1024 : 472) / values_of(d); }

int segments_of(const mesa_delta_desc* d) {
  const int64_t heads = (int64_t)d->B * d->H, values = values_of(d), both = both_of(d);
  const int chunks = chunks_of(d);
  if (heads > most_heads(d)) return 1;
  const double more = d->dtype == MESA_BF16 ? 1.0 : 0.5;
  const auto rounds = [](int64_t blocks) { return (double)((blocks + 255) / 256); };
  int best = 1;
  double least = 0.9 * chunks * rounds(heads * values);
  for (int n = 2; n <= kMaxSegments && n * 2 <= chunks && n * heads <= most_segments(d); ++n) {
    const int per = (chunks + n - 1) / n;
    if ((chunks + per - 1) / per != n) continue;  // (no segment stays empty)
    const double time =
        per * (rounds(heads * (values + (n - 2) * both)) + rounds(heads * (n - 1) * values)) + more * (3 + 0.5 * n);
    if (time < least) {
      best = n;
      least = time;
    }
  }
  return best;
}

struct Carve {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(size_t bytes) {
    char* here = base ? base + at : nullptr;
    at += pad256(bytes);
    return reinterpret_cast<T*>(here);
  }
};

// Places the workspace's parts for that many heads, `segments` segments of them all; returns its size.
size_t place(const mesa_delta_desc* d, size_t heads, size_t segments, bool keep, void* workspace, DeltaParams& p) {
  Carve w{static_cast<char*>(workspace)};
  const size_t units = heads * chunks_of(d), state = (size_t)d->dv * d->dk * 4;
  p.gates = w.take<DeltaGates>(units * sizeof(DeltaGates));
  p.seg_map = w.take<float>(segments * d->dk * d->dk * 4);
  p.seg_add = w.take<float>(segments * state);
  p.seg_start = w.take<float>(segments * state);
  p.matrices = w.take<char>(units * delta_matrix_bytes(d->dtype == MESA_BF16));
  if (keep) {
    p.states = w.take<float>(units * state);
    p.w = w.take<float>(units * kDeltaChunk * d->dv * 4);
    p.matrices_t = w.take<char>(units * kDeltaMatrixBytes);
    p.dstates = w.take<float>(units * state);
    p.e = w.take<float>(units * kDeltaChunk * d->dv * 4);
    if (d->H != d->Hk) {
      const size_t rows = heads * d->T * d->dk * 4;
      p.dq_heads = w.take<float>(rows);
      p.dk_heads = w.take<float>(rows);
    }
  }
  return w.at;
}

void carve(const mesa_delta_desc* d, bool keep, void* workspace, DeltaParams& p) {
  const size_t heads = (size_t)d->B * d->H;
  p.NS = segments_of(d);
  p.L = (chunks_of(d) + p.NS - 1) / p.NS;
  place(d, heads, p.NS > 1 ? heads * p.NS : 0, keep, workspace, p);
}

// Room for what carve() places here and for any smaller B and T: without segments, or with as many as
// so many heads and chunks may be given.
size_t room(const mesa_delta_desc* d, bool keep) {
  DeltaParams p{};
  const size_t heads = (size_t)d->B * d->H, few = std::min(heads, (size_t)most_heads(d)),
               segments = std::min(few * std::min(kMaxSegments, chunks_of(d) / 2), (size_t)most_segments(d));
  return std::max(place(d, heads, 0, keep, nullptr, p), place(d, few, segments, keep, nullptr, p));
}

// (a token stride that no index uses may be any: kernels step by it to rows that they then leave out)
DeltaRows rows(const mesa_delta_desc* d, const void* at, const mesa_rows& r) {
  return {const_cast<void*>(at), r.b, r.h, d->T > 1 ? r.t : 0};
}

DeltaGate gate(const float* at, const mesa_rows& r) { return {const_cast<float*>(at), r.b, r.h, r.t}; }

DeltaParams delta_params(const mesa_delta_desc* d, const void* q, const void* k, const void* v, const float* gamma,
                         const float* beta, const float* s0, const int32_t* lengths) {
  DeltaParams p{};
  p.q = rows(d, q, d->q); p.k = rows(d, k, d->k); p.v = rows(d, v, d->v); p.gamma = gate(gamma, d->gamma);
  p.beta = gate(beta, d->beta); p.s0 = s0; p.lengths = lengths;
  p.B = d->B; p.H = d->H; p.Hk = d->Hk; p.T = d->T; p.dk = d->dk; p.dv = d->dv; p.NC = chunks_of(d);
  p.by_h = divisor((uint32_t)d->H); p.by_shared = divisor((uint32_t)(d->H / d->Hk));
  p.by_nc = divisor((uint32_t)std::max(p.NC, 1));
  return p;
}

// The launches of a walk in segments: `first` for what the others start from (with segments
// opened .. opened + openings - 1) and, behind the join, segments seg0 .. seg0 + segs - 1.
// With one segment the second alone.
template <typename First, typename Walk>
hipError_t in_segments(const DeltaParams& p, bool back, int opened, int openings, int seg0, int segs, hipStream_t s,
                       First&& first, Walk&& walk) {
  DeltaParams x = p;
  const auto range = [&](int from, int count) {
    const uint32_t slices = (uint32_t)(p.dv + 63) / 64;
    x.seg0 = from;
    x.segs = count;
    x.by_slices = divisor(slices);
    x.by_part = divisor(slices * (uint32_t)count);
  };
  if (p.NS > 1) {
    range(opened, openings);
    x.open = 1;
    hipError_t e = first(x);
    if (e == hipSuccess) e = launch_delta_join(back, p, s);
    if (e != hipSuccess) return e;
    x.open = 0;
  }
  range(p.NS > 1 ? seg0 : 0, p.NS > 1 ? segs : 1);
  return walk(x);
}

// A walk forward: the first segment runs beside the launch that opens the others.
hipError_t scan(bool bf16, const DeltaParams& p, hipStream_t s) {
  return in_segments(
      p, false, 0, 1, 1, p.NS - 1, s,
      [&](const DeltaParams& x) { return bf16 ? launch_delta_open(x, s) : launch_delta_open_f32(x, s); },
      [&](const DeltaParams& x) { return bf16 ? launch_delta_scan(x, s) : launch_delta_scan_f32(x, s); });
}

// A walk back; the segments' maps are those of the walk forward, and the last segment, which
// starts it, runs whole beside those that start from zero.
hipError_t adjoint(bool bf16, const DeltaParams& p, hipStream_t s) {
  const auto walk = [&](const DeltaParams& x) {
    return bf16 ? launch_delta_adjoint(x, s) : launch_delta_adjoint_f32(x, s);
  };
  return in_segments(p, true, 1, p.NS - 1, 0, p.NS - 1, s, walk, walk);
}

mesa_status launched(hipError_t e) { return e == hipSuccess ? MESA_OK : MESA_ERR_HIP; }

}  // namespace

extern "C" {

size_t mesa_delta_workspace_bytes(const mesa_delta_desc* d, int32_t keep_states) {
  if (check_delta(d) != MESA_OK || (keep_states != 0 && keep_states != 1)) return 0;
  return room(d, keep_states == 1);
}

mesa_status mesa_delta_fwd(const mesa_delta_desc* d, const void* q, const void* k, const void* v, const float* gamma,
                           const float* beta, const float* s0, const int32_t* lengths, void* o, float* s_final,
                           int32_t keep_states, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_delta(d);
  if (st != MESA_OK) return st;
  if (keep_states != 0 && keep_states != 1) return MESA_ERR_INVALID_ARG;
  if (d->T > 0 && (!q || !k || !v || !gamma || !beta || !o)) return MESA_ERR_INVALID_ARG;
  if (!apart(d, d->H, d->dv, d->o)) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({q, k, v, s0, lengths, o, s_final, workspace}) || !floats_aligned({gamma, beta}) ||
      !rows_aligned(d, d->Hk, d->q) || !rows_aligned(d, d->Hk, d->k) || !rows_aligned(d, d->H, d->v) ||
      !rows_aligned(d, d->H, d->o))
    return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_delta_workspace_bytes(d, keep_states);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const size_t e = dtype_bytes(d->dtype), state = (size_t)d->B * d->H * d->dv * d->dk * 4;
  const Blocks ins[] = {blocks_of(d, d->Hk, d->dk, e, d->q, q), blocks_of(d, d->Hk, d->dk, e, d->k, k),
                      blocks_of(d, d->H, d->dv, e, d->v, v), blocks_of(d, d->H, 1, 4, d->gamma, gamma),
                      blocks_of(d, d->H, 1, 4, d->beta, beta), {lengths, (size_t)d->B * 4}};
  const Blocks outs[] = {blocks_of(d, d->H, d->dv, e, d->o, o), {workspace, need}, {s_final, state}}, start{s0, state};
  // s_final may be s0, and nothing else may lie over s0
  if (overlap(outs, ins) || overlap(outs) || overlap<Blocks>({outs[0], outs[1]}, {start}) ||
      (s_final != s0 && overlap<Blocks>({outs[2]}, {start})))
    return MESA_ERR_INVALID_ARG;
  DeltaParams p = delta_params(d, q, k, v, gamma, beta, s0, lengths);
  carve(d, keep_states == 1, workspace, p);
  p.o = rows(d, o, d->o); p.s_final = s_final;
  const bool bf16 = d->dtype == MESA_BF16;
  if (d->T > 0 && launch_delta_chunks(bf16, p, stream) != hipSuccess) return MESA_ERR_HIP;
  if (d->T == 0) p.o.at = nullptr;
  return launched(scan(bf16, p, stream));
}

mesa_status mesa_delta_bwd(const mesa_delta_desc* d, const mesa_delta_grad_rows* gr, const void* q, const void* k,
                           const void* v, const float* gamma, const float* beta, const float* s0,
                           const int32_t* lengths, const void* d_o, const float* d_sfinal, void* dq, void* dk, void* dv,
                           float* dgamma, float* dbeta, float* ds0, int32_t states_in_workspace, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_delta(d);
  if (st != MESA_OK) return st;
  if (!gr || (states_in_workspace != 0 && states_in_workspace != 1)) return MESA_ERR_INVALID_ARG;
  for (const mesa_rows* r : {&gr->d_o, &gr->dq, &gr->dk, &gr->dv, &gr->dgamma, &gr->dbeta})
    if (!strides_ok(*r)) return MESA_ERR_INVALID_ARG;
  for (const mesa_rows* r : {&gr->d_o, &gr->dq, &gr->dk, &gr->dv, &gr->dgamma, &gr->dbeta})
    if (d->T > 1 && r->t > kMaxTokenStride) return MESA_ERR_UNSUPPORTED;
  if (d->T > 0 && (!q || !k || !v || !gamma || !beta || !d_o || !dq || !dk || !dv || !dgamma || !dbeta))
    return MESA_ERR_INVALID_ARG;
  if (!apart(d, d->Hk, d->dk, gr->dq) || !apart(d, d->Hk, d->dk, gr->dk) || !apart(d, d->H, d->dv, gr->dv) ||
      !apart(d, d->H, 1, gr->dgamma) || !apart(d, d->H, 1, gr->dbeta))
    return MESA_ERR_INVALID_ARG;
  if (!all_aligned({q, k, v, s0, lengths, d_o, d_sfinal, dq, dk, dv, ds0, workspace}) ||
      !floats_aligned({gamma, beta, dgamma, dbeta}) || !rows_aligned(d, d->Hk, d->q) ||
      !rows_aligned(d, d->Hk, d->k) || !rows_aligned(d, d->H, d->v) || !rows_aligned(d, d->H, gr->d_o) ||
      !rows_aligned(d, d->Hk, gr->dq) || !rows_aligned(d, d->Hk, gr->dk) || !rows_aligned(d, d->H, gr->dv))
    return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_delta_workspace_bytes(d, 1);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const size_t e = dtype_bytes(d->dtype), state = (size_t)d->B * d->H * d->dv * d->dk * 4;
  const Blocks ins[] = {blocks_of(d, d->Hk, d->dk, e, d->q, q), blocks_of(d, d->Hk, d->dk, e, d->k, k),
                      blocks_of(d, d->H, d->dv, e, d->v, v), blocks_of(d, d->H, 1, 4, d->gamma, gamma),
                      blocks_of(d, d->H, 1, 4, d->beta, beta), {lengths, (size_t)d->B * 4}, {s0, state},
                      blocks_of(d, d->H, d->dv, e, gr->d_o, d_o)};
  const Blocks outs[] = {blocks_of(d, d->Hk, d->dk, e, gr->dq, dq), blocks_of(d, d->Hk, d->dk, e, gr->dk, dk),
                       blocks_of(d, d->H, d->dv, e, gr->dv, dv), blocks_of(d, d->H, 1, 4, gr->dgamma, dgamma),
                       blocks_of(d, d->H, 1, 4, gr->dbeta, dbeta), {workspace, need}, {ds0, state}};
  const Blocks last{d_sfinal, state};
  // ds0 may be d_sfinal, and nothing else may lie over d_sfinal
  if (overlap(outs, ins) || overlap(outs) ||
      overlap<Blocks>({outs[0], outs[1], outs[2], outs[3], outs[4], outs[5]}, {last}) ||
      (ds0 != d_sfinal && overlap<Blocks>({outs[6]}, {last})))
    return MESA_ERR_INVALID_ARG;
  DeltaParams p = delta_params(d, q, k, v, gamma, beta, s0, lengths);
  carve(d, true, workspace, p);
  const bool bf16 = d->dtype == MESA_BF16;
  if (d->T > 0) {
    // (the walk forward here has no outputs)
    if (!states_in_workspace &&
        (launch_delta_chunks(bf16, p, stream) != hipSuccess || scan(bf16, p, stream) != hipSuccess))
      return MESA_ERR_HIP;
  }
  p.d_o = rows(d, d_o, gr->d_o); p.dq = rows(d, dq, gr->dq); p.dk_ = rows(d, dk, gr->dk); p.dv_ = rows(d, dv, gr->dv);
  p.dgamma = gate(dgamma, gr->dgamma); p.dbeta = gate(dbeta, gr->dbeta); p.d_sfinal = d_sfinal; p.ds0 = ds0;
  if (adjoint(bf16, p, stream) != hipSuccess) return MESA_ERR_HIP;
  return d->T > 0 ? launched(launch_delta_grads(bf16, p, stream)) : MESA_OK;
}

mesa_status mesa_delta_step(const mesa_delta_desc* d, const void* q, const void* k, const void* v, const float* gamma,
                            const float* beta, float* s_state, void* o, hipStream_t stream) {
  const mesa_status st = check_delta(d);
  if (st != MESA_OK) return st;
  if (d->T != 1 || !q || !k || !v || !gamma || !beta || !s_state || !o) return MESA_ERR_INVALID_ARG;
  if (!apart(d, d->H, d->dv, d->o)) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({q, k, v, s_state, o}) || !floats_aligned({gamma, beta}) || !rows_aligned(d, d->Hk, d->q) ||
      !rows_aligned(d, d->Hk, d->k) || !rows_aligned(d, d->H, d->v) || !rows_aligned(d, d->H, d->o))
    return MESA_ERR_ALIGNMENT;
  const size_t e = dtype_bytes(d->dtype), state = (size_t)d->B * d->H * d->dv * d->dk * 4;
  const Blocks ins[] = {blocks_of(d, d->Hk, d->dk, e, d->q, q), blocks_of(d, d->Hk, d->dk, e, d->k, k),
                      blocks_of(d, d->H, d->dv, e, d->v, v), blocks_of(d, d->H, 1, 4, d->gamma, gamma),
                      blocks_of(d, d->H, 1, 4, d->beta, beta)};
  const Blocks outs[] = {blocks_of(d, d->H, d->dv, e, d->o, o), {s_state, state}};
  if (overlap(outs, ins) || overlap(outs)) return MESA_ERR_INVALID_ARG;
  DeltaStepParams p{};
  p.q = q; p.k = k; p.v = v; p.gamma = gamma; p.beta = beta; p.state = s_state; p.o = o;
  p.qn = d->q.b; p.qh = d->q.h; p.kn = d->k.b; p.kh = d->k.h; p.vn = d->v.b; p.vh = d->v.h;
  p.gn = d->gamma.b; p.gh = d->gamma.h; p.bn = d->beta.b; p.bh = d->beta.h; p.on = d->o.b; p.oh = d->o.h;
  p.N = d->B; p.H = d->H; p.Hk = d->Hk; p.dk = d->dk; p.dv = d->dv;
  return launched(launch_delta_step(d->dtype == MESA_BF16, p, stream));
}

}  // extern "C"

// ---- global gradient norm and clipping ---------------------------------------

namespace {

int64_t pieces_of(int64_t n) { return (n + kClipPiece - 1) / kClipPiece; }

// The workgroups of one launch: its share of kClipBlocks, one at least, no more than it has pieces.
int blocks_of(int64_t own, int64_t all) {
  if (own == 0) return 1;
  const double share = std::max(1.0, std::floor((double)kClipBlocks * (double)own / (double)all));
  return (int)std::min((double)own, share);
}

constexpr size_t kClipSums = kClipBlocks + kClipMaxTensors / kClipTensors + 2;

mesa_status check_clip(int32_t count, const void* const* grads, void* const* outs, bool need_outs,
                       const int64_t* sizes, const mesa_dtype* dtypes) {
  if (count < 0 || (count > 0 && (!grads || !sizes || !dtypes || (need_outs && !outs)))) return MESA_ERR_INVALID_ARG;
  if (count > kClipMaxTensors) return MESA_ERR_UNSUPPORTED;
  double all = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || !dtype_ok(dtypes[i])) return MESA_ERR_INVALID_ARG;
    if (sizes[i] > 0 && (!grads[i] || (need_outs && !outs[i]))) return MESA_ERR_INVALID_ARG;
    all += (double)sizes[i];
  }
  if (all > 0x1p44) return MESA_ERR_UNSUPPORTED;
  for (int i = 0; i < count; ++i) {
    const uintptr_t mask = dtype_bytes(dtypes[i]) - 1;
    if (sizes[i] > 0 && ((reinterpret_cast<uintptr_t>(grads[i]) & mask) ||
                         (outs && (reinterpret_cast<uintptr_t>(outs[i]) & mask))))
      return MESA_ERR_ALIGNMENT;
  }
  return MESA_OK;
}

// Whether an output shares memory with anything but, whole, its own gradient: all
// arrays in the order of their starts, each against the furthest end before it.
bool clip_overlap(int32_t count, const void* const* grads, void* const* outs, const int64_t* sizes,
                  const mesa_dtype* dtypes, const Span (&more)[3]) {
  constexpr int kMost = 2 * kClipMaxTensors + 3;
  uint16_t order[kMost];
  int n = 0;
  // 2 i: gradient i, 2 i + 1: output i, behind them the other outputs
  const auto start = [&](int id) {
    const int i = id >> 1;
    if (i >= count) return reinterpret_cast<uintptr_t>(more[id - 2 * count].at);
    return reinterpret_cast<uintptr_t>(id & 1 ? outs[i] : grads[i]);
  };
  const auto bytes = [&](int id) {
    return (id >> 1) >= count ? more[id - 2 * count].bytes : (size_t)sizes[id >> 1] * dtype_bytes(dtypes[id >> 1]);
  };
  for (int i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    if (!outs || outs[i] != grads[i]) order[n++] = (uint16_t)(2 * i);
    if (outs && outs[i]) order[n++] = (uint16_t)(2 * i + 1);
  }
  for (int i = 0; i < 3; ++i)
    if (more[i].at && more[i].bytes) order[n++] = (uint16_t)(2 * count + i);
  std::sort(order, order + n, [&](uint16_t x, uint16_t y) { return start(x) < start(y); });
  uintptr_t end_in = 0, end_out = 0;  // the furthest ends of gradients and of outputs so far
  for (int i = 0; i < n; ++i) {
    const int id = order[i];
    const bool out = id >= 2 * count || (id & 1);
    const uintptr_t from = start(id), to = from + bytes(id);
    if (from < end_out || (out && from < end_in)) return true;
    if (out) end_out = std::max(end_out, to);
    else end_in = std::max(end_in, to);
  }
  return false;
}

// Calls f(table, its workgroups, the sums before it) for each launch's tensors; false at the first failure.
template <typename F>
bool each_table(int32_t count, const void* const* grads, void* const* outs, const int64_t* sizes,
                const mesa_dtype* dtypes, F&& f) {
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += pieces_of(sizes[i]);
  ClipTable t;
  int at = 0, i = 0;
  do {
    t.count = 0;
    t.first[0] = 0;
    for (; i < count && t.count < kClipTensors; ++i) {
      if (sizes[i] == 0) continue;
      t.grad[t.count] = grads[i];
      t.out[t.count] = outs ? outs[i] : nullptr;
      t.n[t.count] = sizes[i];
      t.bf16[t.count] = dtypes[i] == MESA_BF16;
      t.first[t.count + 1] = t.first[t.count] + pieces_of(sizes[i]);
      ++t.count;
    }
    const int blocks = blocks_of(t.first[t.count], all);
    if (!f(t, blocks, at)) return false;
    at += blocks;
  } while (i < count);
  return true;
}

mesa_status clip(int32_t count, const void* const* grads, void* const* outs, bool need_outs, const int64_t* sizes,
                 const mesa_dtype* dtypes, double max_norm, double eps, float* norm, float* scale, void* workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_clip(count, grads, outs, need_outs, sizes, dtypes);
  if (st != MESA_OK) return st;
  if (!all_aligned({workspace}) || !floats_aligned({norm, scale})) return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_grad_clip_workspace_bytes();
  if (!workspace || workspace_bytes < need) return MESA_ERR_WORKSPACE;
  if (clip_overlap(count, grads, outs, sizes, dtypes, {{norm, 4}, {scale, 4}, {workspace, need}}))
    return MESA_ERR_INVALID_ARG;
  double* sums = static_cast<double*>(workspace);
  int n_sums = 0;
  if (!each_table(count, grads, outs, sizes, dtypes, [&](const ClipTable& t, int blocks, int at) {
        n_sums = at + blocks;
        return launch_clip_squares(t, blocks, sums + at, stream) == hipSuccess;
      }))
    return MESA_ERR_HIP;
  if (!outs) {  // the norm alone
    ClipTable none;
    none.count = 0;
    none.first[0] = 0;
    return launched(launch_clip_scale(none, 1, sums, n_sums, max_norm, eps, norm, scale, stream));
  }
  return each_table(count, grads, outs, sizes, dtypes, [&](const ClipTable& t, int blocks, int at) {
           return launch_clip_scale(t, blocks, sums, n_sums, max_norm, eps, at ? nullptr : norm, at ? nullptr : scale,
                                    stream) == hipSuccess;
         })
             ? MESA_OK
             : MESA_ERR_HIP;
}

}  // namespace

extern "C" {

size_t mesa_grad_clip_workspace_bytes(void) { return pad256(kClipSums * sizeof(double)); }

mesa_status mesa_grad_norm(int32_t count, const void* const* grads, const int64_t* sizes, const mesa_dtype* dtypes,
                           float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!norm) return MESA_ERR_INVALID_ARG;
  return clip(count, grads, nullptr, false, sizes, dtypes, 1.0, 1.0, norm, nullptr, workspace, workspace_bytes, stream);
}

mesa_status mesa_grad_clip(int32_t count, const void* const* grads, void* const* outs, const int64_t* sizes,
                           const mesa_dtype* dtypes, double max_norm, double eps, float* norm, float* scale,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!norm || !(max_norm >= 0.0) || !(eps >= 0x1p-126) || std::isinf(eps)) return MESA_ERR_INVALID_ARG;
  return clip(count, grads, outs, true, sizes, dtypes, max_norm, eps, norm, scale, workspace, workspace_bytes, stream);
}

}  // extern "C"
