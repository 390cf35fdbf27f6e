// Parameters and launches of the gated delta rule.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

constexpr int kDeltaChunk = 64;  // tokens that are taken together

// Quotients of numbers below 2^30 by d, without a division: floor(n m / 2^shift).  m is 2^shift / d
// rounded up and shift 31 + floor(log2 d), so n m / 2^shift exceeds n / d by less than n / d 2^-30 < 1 / d.
// (A workgroup's place took four divisions of 200 cycles each.)
struct Divisor {
  uint32_t d, m, shift;
};
inline Divisor divisor(uint32_t d) {
  uint32_t log = 0;
  while (d >> (log + 1)) ++log;
  return {d, (uint32_t)((((uint64_t)1 << (31 + log)) + d - 1) / d), 31 + log};
}
__host__ __device__ inline uint32_t operator/(uint32_t n, const Divisor& x) {
  return (uint32_t)(((uint64_t)n * x.m) >> x.shift);
}
__host__ __device__ inline uint32_t operator%(uint32_t n, const Divisor& x) { return n - n / x * x.d; }

// Vectors of B x heads x T tokens; strides in elements, the last index contiguous.
struct DeltaRows {
  void* at;
  int64_t b, h, t;
};

// A number for each of B x heads x T tokens.
struct DeltaGate {
  float* at;
  int64_t b, h, t;
};

// What every kernel needs of a chunk's gates.
struct DeltaGates {
  double g[kDeltaChunk];    // log2 of the product of the chunk's forget factors up to and with token t
  float c[kDeltaChunk];     // that product
  float tail[kDeltaChunk];  // the product of those behind token t
  float beta[kDeltaChunk];  // 0 behind the sequence
};

// Bytes of a chunk's two triangular 64x64 matrices for the walk forward: the inverse as operands in three
// bf16 parts, and the products of its queries and keys in fp32, ten tiles (bf16 rows), or as operands too.
constexpr size_t delta_matrix_bytes(bool bf16) { return (3 * 6 + (bf16 ? 10 : 3 * 6)) * 1024; }
// ... and for the walk back in fp32: ten tiles each.
constexpr size_t kDeltaMatrixBytes = 2 * 10 * 1024;

struct DeltaParams {
  DeltaRows q, k, v, o;             // o.at null: the states alone
  DeltaGate gamma, beta;
  const float *s0;                  // [B, H, dv, dk] or null
  float* s_final;                   // [B, H, dv, dk] or null
  const int32_t* lengths;           // [B] or null
  int B, H, Hk, T, dk, dv, NC;      // NC chunks a (padded) sequence
  Divisor by_h, by_shared, by_nc;   // H, H / Hk, NC
  // A walk in NS segments of L chunks (NS = 1: whole).  seg_map: [B H, NS, dk, dk], row j what
  // an inner segment makes of the state whose row is unit vector j; seg_add: [B H, NS, dv, dk], what
  // it makes of a zero state (the segment at the walk's start: of the given one);
  // seg_start: [B H, NS, dv, dk], the states that segments start from behind the join (all but the walk's first)
  int NS, L;
  int seg0, segs;                   // the segments of a launch of a walk
  Divisor by_part, by_slices;       // its workgroups of a head, and of those the ones of a segment
  float *seg_map, *seg_add, *seg_start;
  int open;                         // 1: the launch before the join: ends go to seg_add, and a segment
                                    // that does not start the walk starts from zero
  DeltaGates* gates;                // [B H, NC]
  char* matrices;                   // [B H, NC, delta_matrix_bytes]
  float* states;                    // [B H, NC, dv, dk] before each chunk, or null
  float* w;                         // [B H, NC, 64, dv]: v_t - gamma_t S_{t-1} k_t, or null
  // backward
  DeltaRows d_o, dq, dk_, dv_;
  DeltaGate dgamma, dbeta;
  const float* d_sfinal;
  float* ds0;
  char* matrices_t;                 // [B H, NC, kDeltaMatrixBytes]: the backward pass's, or null
  float* dstates;                   // [B H, NC, dv, dk]: the gradient behind each chunk
  float* e;                         // [B H, NC, 64, dv]: dv_t / beta_t
  float *dq_heads, *dk_heads;       // [B, H, T, dk] where heads share keys
};

// Each returns hipSuccess or the launch error.
// Every chunk's gates and the matrices of the walk forward, and where matrices_t is there of the walk back.
hipError_t launch_delta_chunks(bool bf16, const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_scan(const DeltaParams& p, hipStream_t s);  // bf16 rows
hipError_t launch_delta_scan_f32(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_adjoint(const DeltaParams& p, hipStream_t s);  // bf16 rows
hipError_t launch_delta_adjoint_f32(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_grads(bool bf16, const DeltaParams& p, hipStream_t s);

// seg_map and seg_add of a walk forward, and its first segment whole.
hipError_t launch_delta_open(const DeltaParams& p, hipStream_t s);  // bf16 rows
hipError_t launch_delta_open_f32(const DeltaParams& p, hipStream_t s);
// seg_start from seg_map and seg_add; `back`: from the last segment to the first.
hipError_t launch_delta_join(bool back, const DeltaParams& p, hipStream_t s);

struct DeltaStepParams {
  const void *q, *k, *v;
  int64_t qn, qh, kn, kh, vn, vh, gn, gh, bn, bh, on, oh;  // strides of a sequence and of a head (elements)
  const float *gamma, *beta;
  float* state;
  void* o;
  int N, H, Hk, dk, dv;
  Divisor by_groups, by_h, by_shared;  // workgroups of a head, H, H / Hk
};
hipError_t launch_delta_step(bool bf16, const DeltaStepParams& p, hipStream_t s);

}  // namespace mesa
