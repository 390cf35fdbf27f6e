// C ABI of the operators around the Mesa layer: argument validation, workspace
// carving, kernel launches.  Every check runs before the first launch, so a
// failing call writes nothing.
#include <algorithm>
#include <cmath>

#include "../../include/mesa.h"
#include "mesa_kernels.h"

namespace {

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return false;
  return true;
}

bool dtype_ok(mesa_dtype t) { return t == MESA_F32 || t == MESA_BF16; }

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// `rows` pieces of `bytes` bytes, `stride` bytes apart: a dense array is one piece.
struct Span {
  const void* at;
  size_t bytes, rows = 1, stride = 0;
};

// Whether any byte belongs to both.  Rows at one stride (slices of one wider
// tensor) may interleave; rows at different strides count as filling their range.
bool share(const Span& x, const Span& y) {
  if (!x.at || !y.at || x.bytes == 0 || y.bytes == 0 || x.rows == 0 || y.rows == 0) return false;
  const bool in_order = reinterpret_cast<uintptr_t>(x.at) < reinterpret_cast<uintptr_t>(y.at);
  const Span &a = in_order ? x : y, &b = in_order ? y : x;  // a starts first
  const size_t by = reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at);
  if (by >= (a.rows - 1) * a.stride + a.bytes) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  // each of b's rows starts `in` bytes behind the start of a row of a (the first behind row `row`)
  const size_t stride = a.rows > 1 ? a.stride : b.stride, row = by / stride, in = by % stride;
  return in < a.bytes || (row + 1 < a.rows && stride - in < b.bytes);
}

// Whether an output shares memory with an input.
template <size_t N, size_t M>
bool overlap(const Span (&outs)[N], const Span (&ins)[M]) {
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (share(o, i)) return true;
  return false;
}

// Whether two outputs share memory.
template <size_t N>
bool overlap(const Span (&outs)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (share(outs[i], outs[j])) return true;
  return false;
}

size_t dtype_bytes(mesa_dtype t) { return t == MESA_BF16 ? 2 : 4; }

// ---- gated linear recurrence ----------------------------------------------

// The token rows at stride ld.
Span lru_rows(const mesa_lru_desc* d, const void* at, int32_t ld) {
  const size_t e = dtype_bytes(d->dtype);
  return {at, d->D * e, (size_t)d->B * d->T, ld * e};
}

constexpr int kLruMaxStride = 1 << 20;

mesa_status check_lru(const mesa_lru_desc* d) {
  if (!d || d->B < 1 || d->T < 0 || d->D < 1 || d->ld < d->D || !dtype_ok(d->dtype)) return MESA_ERR_INVALID_ARG;
  if (!(d->c > 0.f) || std::isinf(d->c)) return MESA_ERR_INVALID_ARG;
  // lanes load two channels; offsets within a tile of tokens are 32-bit; a launch has at most 2^32 threads
  if (d->D < 2 || d->ld > kLruMaxStride) return MESA_ERR_UNSUPPORTED;
  const double tiles = (double)d->B * (d->T > 64 ? ((long long)d->T + 63) / 64 : 1) * ((d->D + 63) / 64);
  if (tiles > 8388608.0) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

int lru_chunks(const mesa_lru_desc* d) { return (d->T + mesa::kLruChunk - 1) / mesa::kLruChunk; }

size_t lru_state_bytes(const mesa_lru_desc* d) { return pad256((size_t)d->B * lru_chunks(d) * d->D * 4); }

size_t lru_word_bytes(const mesa_lru_desc* d) {
  return std::max(mesa::lru_fwd_word_bytes(d->B, d->T, d->D), mesa::lru_bwd_word_bytes(d->B, d->T, d->D));
}

mesa::LruParams lru_params(const mesa_lru_desc* d, const void* x, const void* ga, const void* gi, const float* lam,
                           const float* h0, const int32_t* lengths, void* workspace) {
  mesa::LruParams p{};
  p.x = x; p.ga = ga; p.gi = gi; p.lam = lam; p.h0 = h0; p.lengths = lengths;
  p.states = static_cast<float*>(workspace);
  char* at = static_cast<char*>(workspace) + lru_state_bytes(d);
  p.tickets = reinterpret_cast<unsigned*>(at);
  p.words = reinterpret_cast<uint64_t*>(at += mesa::kLruTicketBytes);
  p.lam_part = reinterpret_cast<float*>(at += lru_word_bytes(d));
  p.B = d->B; p.T = d->T; p.D = d->D; p.ld = d->ld; p.NC = lru_chunks(d); p.c = d->c;
  return p;
}

}  // namespace

extern "C" {

size_t mesa_lru_workspace_bytes(const mesa_lru_desc* d) {
  if (check_lru(d) != MESA_OK || d->T == 0) return 0;
  return lru_state_bytes(d) + mesa::kLruTicketBytes +
         lru_word_bytes(d) + pad256(mesa::lru_bwd_part_bytes(d->B, d->T, d->D));
}

mesa_status mesa_lru_fwd(const mesa_lru_desc* d, const void* x, const void* ga, const void* gi, const float* lam,
                         const float* h0, const int32_t* lengths, void* y, float* h_final, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_lru(d);
  if (st != MESA_OK) return st;
  if (!lam || (d->T > 0 && (!x || !ga || !gi || !y))) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({x, ga, gi, lam, h0, lengths, y, h_final, workspace})) return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_lru_workspace_bytes(d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const size_t per_channel = (size_t)d->D * 4, state = d->B * per_channel;
  const Span ins[] = {lru_rows(d, x, d->ld), lru_rows(d, ga, d->ld), lru_rows(d, gi, d->ld), {lam, per_channel},
                      {lengths, (size_t)d->B * 4}};
  const Span outs[] = {lru_rows(d, y, d->D), {workspace, need}, {h_final, state}}, start{h0, state};
  // h_final may be h0, and nothing else may lie over h0
  if (overlap(outs, ins) || overlap(outs) || overlap({outs[0], outs[1]}, {start}) ||
      (h_final != h0 && overlap({outs[2]}, {start})))
    return MESA_ERR_INVALID_ARG;
  mesa::LruParams p = lru_params(d, x, ga, gi, lam, h0, lengths, workspace);
  p.y = y; p.h_final = h_final;
  return mesa::launch_lru_fwd(d->dtype == MESA_BF16, p, stream) == hipSuccess ? MESA_OK : MESA_ERR_HIP;
}

mesa_status mesa_lru_bwd(const mesa_lru_desc* d, const void* x, const void* ga, const void* gi, const float* lam,
                         const float* h0, const int32_t* lengths, const void* dy, const float* d_hfinal, void* dx,
                         void* dga, void* dgi, int32_t ld_grad, float* dlam, float* dh0, int32_t states_in_workspace,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_lru(d);
  if (st != MESA_OK) return st;
  if (ld_grad < d->D || (states_in_workspace != 0 && states_in_workspace != 1)) return MESA_ERR_INVALID_ARG;
  if (ld_grad > kLruMaxStride) return MESA_ERR_UNSUPPORTED;
  if (!lam || !dlam || (d->T > 0 && (!x || !ga || !gi || !dy || !dx || !dga || !dgi))) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({x, ga, gi, lam, h0, lengths, dy, d_hfinal, dx, dga, dgi, dlam, dh0, workspace}))
    return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_lru_workspace_bytes(d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const bool bf16 = d->dtype == MESA_BF16;
  const size_t per_channel = (size_t)d->D * 4, state = d->B * per_channel;
  const Span ins[] = {lru_rows(d, x, d->ld), lru_rows(d, ga, d->ld), lru_rows(d, gi, d->ld), {lam, per_channel},
                      {h0, state}, {lengths, (size_t)d->B * 4}, lru_rows(d, dy, d->D)};
  const Span outs[] = {lru_rows(d, dx, ld_grad), lru_rows(d, dga, ld_grad), lru_rows(d, dgi, ld_grad),
                       {dlam, per_channel}, {workspace, need}, {dh0, state}};
  const Span last{d_hfinal, state};
  // dh0 may be d_hfinal, and nothing else may lie over d_hfinal
  if (overlap(outs, ins) || overlap(outs) || overlap({outs[0], outs[1], outs[2], outs[3], outs[4]}, {last}) ||
      (dh0 != d_hfinal && overlap({outs[5]}, {last})))
    return MESA_ERR_INVALID_ARG;
  mesa::LruParams p = lru_params(d, x, ga, gi, lam, h0, lengths, workspace);
  if (d->T > 0 && !states_in_workspace && mesa::launch_lru_fwd(bf16, p, stream) != hipSuccess) return MESA_ERR_HIP;
  if (d->T == 0) p.lam_part = nullptr;
  p.dy = dy; p.d_hfinal = d_hfinal;
  p.dx = dx; p.dga = dga; p.dgi = dgi; p.ld_grad = ld_grad; p.dlam = dlam; p.dh0 = dh0;
  return mesa::launch_lru_bwd(bf16, p, stream) == hipSuccess ? MESA_OK : MESA_ERR_HIP;
}

mesa_status mesa_lru_step(int32_t N, int32_t D, int32_t ld, float c, mesa_dtype dtype, const void* x, const void* ga,
                          const void* gi, const float* lam, float* h_state, void* y, hipStream_t stream) {
  if (N < 0) return MESA_ERR_INVALID_ARG;
  const mesa_lru_desc d{N > 0 ? N : 1, 1, D, ld, c, dtype};
  const mesa_status st = check_lru(&d);
  if (st != MESA_OK || N == 0) return st;
  if (!x || !ga || !gi || !lam || !h_state || !y) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({x, ga, gi, lam, h_state, y})) return MESA_ERR_ALIGNMENT;
  const mesa_lru_desc all{N, 1, D, ld, c, dtype};
  const size_t per_channel = (size_t)D * 4, state = N * per_channel;
  const Span ins[] = {lru_rows(&all, x, ld), lru_rows(&all, ga, ld), lru_rows(&all, gi, ld), {lam, per_channel}};
  const Span outs[] = {lru_rows(&all, y, D), {h_state, state}};
  if (overlap(outs, ins) || overlap(outs)) return MESA_ERR_INVALID_ARG;
  mesa::LruParams p = lru_params(&d, x, ga, gi, lam, nullptr, nullptr, nullptr);
  p.h_final = h_state; p.y = y;
  return mesa::launch_lru_step(dtype == MESA_BF16, p, stream) == hipSuccess ? MESA_OK : MESA_ERR_HIP;
}

}  // extern "C"

// ---- residual RMS norm ------------------------------------------------------

namespace {

mesa_status check_norm(int32_t R, int32_t D, mesa_dtype dtype, mesa_dtype res_dtype, float eps) {
  if (R < 0 || D < 1 || !dtype_ok(dtype) || !dtype_ok(res_dtype)) return MESA_ERR_INVALID_ARG;
  if (!(eps >= 0x1p-126f) || std::isinf(eps)) return MESA_ERR_INVALID_ARG;
  if (D > 16384 || R > (1 << 30) || (double)R * D > (double)(1LL << 40)) return MESA_ERR_UNSUPPORTED;
  if (dtype == MESA_F32 && res_dtype == MESA_BF16) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

}  // namespace

extern "C" {

mesa_status mesa_rmsnorm(int32_t R, int32_t D, mesa_dtype dtype, mesa_dtype res_dtype, const void* x,
                         const void* residual, const float* w, float eps, mesa_norm_out out, int32_t group, void* y,
                         float* scale, void* residual_out, hipStream_t stream) {
  const mesa_status st = check_norm(R, D, dtype, res_dtype, eps);
  if (st != MESA_OK) return st;
  if (out != MESA_NORM_OUT_DTYPE && out != MESA_NORM_OUT_E4M3) return MESA_ERR_INVALID_ARG;
  const bool e4m3 = out == MESA_NORM_OUT_E4M3;
  if (e4m3 && group < 0) return MESA_ERR_INVALID_ARG;
  if (e4m3 && group != 0 && group != 128) return MESA_ERR_UNSUPPORTED;
  if (R == 0) return MESA_OK;
  if (!x || !w || !y || (e4m3 && !scale)) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({x, residual, w, y, scale, residual_out})) return MESA_ERR_ALIGNMENT;
  const size_t n = (size_t)R * D, rows = n * dtype_bytes(dtype), stream_rows = n * dtype_bytes(res_dtype);
  const size_t groups = group ? (D + 127) / 128 : 1, weights = (size_t)D * 4;
  const Span outs[] = {{y, e4m3 ? n : rows}, {scale, e4m3 ? R * groups * 4 : 0}};
  if (overlap(outs, {{x, rows}, {residual, stream_rows}, {w, weights}, {residual_out, stream_rows}}) || overlap(outs) ||
      overlap({{residual_out, stream_rows}},
              {{residual_out == x && dtype == res_dtype ? nullptr : x, rows},
               {residual_out == residual ? nullptr : residual, stream_rows}, {w, weights}}))
    return MESA_ERR_INVALID_ARG;
  mesa::NormParams p{};
  p.x = x; p.residual = residual; p.w = w; p.y = y; p.scale = scale; p.residual_out = residual_out;
  p.R = R; p.D = D; p.eps = eps; p.e4m3 = e4m3 ? 1 : 0; p.group = e4m3 ? group : 0;
  return mesa::launch_rmsnorm(dtype == MESA_BF16, res_dtype == MESA_BF16, p, stream) == hipSuccess ? MESA_OK
                                                                                                   : MESA_ERR_HIP;
}

size_t mesa_rmsnorm_bwd_workspace_bytes(int32_t R, int32_t D) {
  if (check_norm(R, D, MESA_F32, MESA_F32, 1.f) != MESA_OK || R == 0) return 0;
  return mesa::rmsnorm_bwd_scratch(R, D);
}

mesa_status mesa_rmsnorm_bwd(int32_t R, int32_t D, mesa_dtype dtype, mesa_dtype res_dtype, const void* s,
                             const float* w, const void* dy, const void* d_residual, float eps, void* ds, void* dx,
                             float* dw, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_norm(R, D, dtype, res_dtype, eps);
  if (st != MESA_OK) return st;
  if (!dw || (R > 0 && (!s || !w || !dy || !ds))) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({s, w, dy, d_residual, ds, dx, dw, workspace})) return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_rmsnorm_bwd_workspace_bytes(R, D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const size_t n = (size_t)R * D, rows = n * dtype_bytes(dtype), stream_rows = n * dtype_bytes(res_dtype);
  const size_t weights = (size_t)D * 4;
  const Span ins[] = {{s, stream_rows}, {w, weights}, {dy, rows}};
  const Span outs[] = {{dx, rows}, {dw, weights}, {workspace, need}, {ds, stream_rows}}, along{d_residual, stream_rows};
  // ds may be d_residual, and nothing else may lie over d_residual
  if (overlap(outs, ins) || overlap(outs) || overlap({outs[0], outs[1], outs[2]}, {along}) ||
      (ds != d_residual && overlap({outs[3]}, {along})))
    return MESA_ERR_INVALID_ARG;
  mesa::NormParams p{};
  p.x = s; p.residual = d_residual; p.w = w; p.dy = dy; p.y = ds; p.residual_out = dx; p.dw = dw;
  p.R = R; p.D = D; p.eps = eps;
  mesa::rmsnorm_bwd_carve(p, workspace);
  return mesa::launch_rmsnorm_bwd(dtype == MESA_BF16, res_dtype == MESA_BF16, p, stream) == hipSuccess ? MESA_OK
                                                                                                       : MESA_ERR_HIP;
}

}  // extern "C"

// ---- gradient of the query/key preprocessing -----------------------------------

namespace {

mesa_status check_prep(int32_t B, int32_t H, int32_t T, int32_t d, int32_t window, mesa_dtype dtype) {
  if (B < 1 || H < 1 || T < 0 || window < 1 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
  if ((d != 16 && d != 64 && d != 128) || window > 4) return MESA_ERR_UNSUPPORTED;
  if ((long long)B * H > 65535 || T > (1 << 30)) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

}  // namespace

extern "C" {

size_t mesa_qk_preprocess_bwd_workspace_bytes(int32_t B, int32_t H, int32_t T, int32_t d, int32_t window,
                                              mesa_dtype dtype) {
  if (check_prep(B, H, T, d, window, dtype) != MESA_OK || T == 0) return 0;
  return mesa::qk_prep_bwd_scratch(B * H, T, d, window);
}

mesa_status mesa_qk_preprocess_bwd(int32_t B, int32_t H, int32_t T, int32_t d, int32_t window, mesa_dtype dtype,
                                   const void* q_raw, const void* k_raw, const float* w_q, const float* w_k,
                                   const void* q_hist, const void* k_hist, float eps, const float* d_q,
                                   const float* d_k, const void* d_q_hist_out, const void* d_k_hist_out,
                                   void* dq_raw, void* dk_raw, float* dw_q, float* dw_k, void* dq_hist, void* dk_hist,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mesa_status st = check_prep(B, H, T, d, window, dtype);
  if (st != MESA_OK) return st;
  // the forward's rule: finite and at least 2^-63
  if (!(eps >= 0x1p-63f) || std::isinf(eps)) return MESA_ERR_INVALID_ARG;
  if (!w_q || !w_k || !dw_q || !dw_k) return MESA_ERR_INVALID_ARG;
  if (T > 0 && (!q_raw || !k_raw || !d_q || !d_k || !dq_raw || !dk_raw)) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({q_raw, k_raw, w_q, w_k, q_hist, k_hist, d_q, d_k, d_q_hist_out, d_k_hist_out, dq_raw, dk_raw, dw_q,
                    dw_k, dq_hist, dk_hist, workspace}))
    return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_qk_preprocess_bwd_workspace_bytes(B, H, T, d, window, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  // every input row is read by up to `window` output rows
  const size_t n = (size_t)B * H * T * d, seq = n * dtype_bytes(dtype);
  const size_t hist = (size_t)B * H * (window - 1) * d * dtype_bytes(dtype), taps = (size_t)H * d * window * 4;
  const Span outs[] = {{dq_raw, seq}, {dk_raw, seq}, {dq_hist, hist}, {dk_hist, hist}, {dw_q, taps}, {dw_k, taps},
                       {workspace, need}};
  if (overlap(outs) ||
      overlap(outs,
              {{q_raw, seq}, {k_raw, seq}, {w_q, taps}, {w_k, taps}, {d_q, n * 4}, {d_k, n * 4}, {q_hist, hist},
               {k_hist, hist}, {d_q_hist_out, hist}, {d_k_hist_out, hist}}))
    return MESA_ERR_INVALID_ARG;

  mesa::PrepBwdParams p{};
  p.x[0] = q_raw; p.x[1] = k_raw; p.w[0] = w_q; p.w[1] = w_k; p.hist_in[0] = q_hist; p.hist_in[1] = k_hist;
  p.d[0] = d_q; p.d[1] = d_k; p.d_hist[0] = d_q_hist_out; p.d_hist[1] = d_k_hist_out;
  p.dx[0] = dq_raw; p.dx[1] = dk_raw; p.dw[0] = dw_q; p.dw[1] = dw_k; p.dhist[0] = dq_hist; p.dhist[1] = dk_hist;
  p.part = static_cast<float*>(workspace);
  p.BH = B * H; p.H = H; p.T = T; p.W = window; p.inv_eps = 1.0f / eps;
  return mesa::launch_qk_prep_bwd(dtype == MESA_BF16, d, p, stream) == hipSuccess ? MESA_OK : MESA_ERR_HIP;
}

}  // extern "C"
