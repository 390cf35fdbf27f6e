// Parameters and launches of the global gradient norm and clipping.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

constexpr int kClipTensors = 96;      // tensors of one launch: their table travels as its argument
constexpr int kClipPiece = 8192;      // elements that a workgroup takes at a time
constexpr int kClipBlocks = 2048;     // workgroups of all launches together, but one a launch at least
constexpr int kClipMaxTensors = 4096;

struct ClipTable {
  const void* grad[kClipTensors];
  void* out[kClipTensors];            // null: left alone
  int64_t n[kClipTensors];
  int64_t first[kClipTensors + 1];    // the tensor's first piece, and all pieces
  uint8_t bf16[kClipTensors];
  int count;
};

// Sums of squares of one launch's tensors, one a workgroup, to sums[0 .. blocks).
hipError_t launch_clip_squares(const ClipTable& t, int blocks, double* sums, hipStream_t s);
// norm = sqrt of all sums, scale = min(1, max_norm / (norm + eps)), outputs scaled.
// norm, scale: written by the first workgroup where not null.
hipError_t launch_clip_scale(const ClipTable& t, int blocks, const double* sums, int n_sums, double max_norm, double eps,
                             float* norm, float* scale, hipStream_t s);

}  // namespace mesa
