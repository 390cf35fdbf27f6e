// What the entry points check of their arguments: alignment, types, and which
// buffers share memory.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/mesa.h"

namespace mesa {

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return false;
  return true;
}

inline bool dtype_ok(mesa_dtype t) { return t == MESA_F32 || t == MESA_BF16; }

inline size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// `rows` pieces of `bytes` bytes, `stride` bytes apart: a dense array is one piece.
struct Span {
  const void* at;
  size_t bytes, rows = 1, stride = 0;
};

// Whether any byte belongs to both.  Rows at one stride (slices of one wider
// tensor) may interleave; rows at different strides count as filling their range.
inline bool share(const Span& x, const Span& y) {
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

inline size_t dtype_bytes(mesa_dtype t) { return t == MESA_BF16 ? 2 : 4; }

}  // namespace mesa
