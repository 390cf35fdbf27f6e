// C ABI of the operators around the Mesa layer: argument validation, workspace
// carving, kernel launches.  Every check runs before the first launch, so a
// failing call writes nothing.
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

// ---- gated linear recurrence ----------------------------------------------

mesa_status check_lru(const mesa_lru_desc* d) {
  if (!d || d->B < 1 || d->T < 0 || d->D < 1 || d->ld < d->D || !dtype_ok(d->dtype)) return MESA_ERR_INVALID_ARG;
  if (!(d->c > 0.f) || std::isinf(d->c)) return MESA_ERR_INVALID_ARG;
  if ((double)d->B * d->T * d->ld > (double)(1LL << 40)) return MESA_ERR_UNSUPPORTED;
  const double tiles = (double)d->B * ((d->T + 63) / 64) * ((d->D + 63) / 64);
  if (tiles >= 2147483648.0) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

int lru_chunks(const mesa_lru_desc* d) { return (d->T + mesa::kLruChunk - 1) / mesa::kLruChunk; }

size_t lru_state_bytes(const mesa_lru_desc* d) { return pad256((size_t)d->B * lru_chunks(d) * d->D * 4); }

size_t lru_part_bytes(const mesa_lru_desc* d) { return pad256((size_t)d->B * d->D * 4); }

mesa::LruParams lru_params(const mesa_lru_desc* d, const void* x, const void* ga, const void* gi, const float* lam,
                           const float* h0, const int32_t* lengths, void* workspace) {
  mesa::LruParams p{};
  p.x = x; p.ga = ga; p.gi = gi; p.lam = lam; p.h0 = h0; p.lengths = lengths;
  p.states = static_cast<float*>(workspace);
  p.B = d->B; p.T = d->T; p.D = d->D; p.ld = d->ld; p.NC = lru_chunks(d); p.c = d->c;
  return p;
}

}  // namespace

extern "C" {

size_t mesa_lru_workspace_bytes(const mesa_lru_desc* d) {
  if (check_lru(d) != MESA_OK || d->T == 0) return 0;
  return lru_state_bytes(d) + lru_part_bytes(d);
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
  if ((double)d->B * d->T * ld_grad > (double)(1LL << 40)) return MESA_ERR_UNSUPPORTED;
  if (!lam || !dlam || (d->T > 0 && (!x || !ga || !gi || !dy || !dx || !dga || !dgi))) return MESA_ERR_INVALID_ARG;
  if (!all_aligned({x, ga, gi, lam, h0, lengths, dy, d_hfinal, dx, dga, dgi, dlam, dh0, workspace}))
    return MESA_ERR_ALIGNMENT;
  const size_t need = mesa_lru_workspace_bytes(d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MESA_ERR_WORKSPACE;
  const bool bf16 = d->dtype == MESA_BF16;
  mesa::LruParams p = lru_params(d, x, ga, gi, lam, h0, lengths, workspace);
  if (d->T > 0) {
    if (!states_in_workspace && mesa::launch_lru_fwd(bf16, p, stream) != hipSuccess) return MESA_ERR_HIP;
    p.lam_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + lru_state_bytes(d));
  }
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
  mesa::LruParams p = lru_params(&d, x, ga, gi, lam, nullptr, nullptr, nullptr);
  p.h_final = h_state; p.y = y;
  return mesa::launch_lru_step(dtype == MESA_BF16, p, stream) == hipSuccess ? MESA_OK : MESA_ERR_HIP;
}

}  // extern "C"
