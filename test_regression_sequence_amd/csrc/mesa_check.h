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

// `bytes` bytes, repeated along up to three dimensions, from the inner one to the outer one: each
// steps over all that its inner ones reach.
struct Blocks {
  struct Step {
    size_t count, stride;
  };
  const void* at;
  size_t bytes;
  int dims = 0;
  Step step[3] = {};

  size_t reach(int n) const {  // of the n inner dimensions
    size_t r = bytes;
    for (int i = 0; i < n; ++i) r += (step[i].count - 1) * step[i].stride;
    return r;
  }
};

// Whether any byte belongs to both, x's first nx dimensions from address a on and y's first ny from b on.
inline bool share(const Blocks& x, int nx, uintptr_t a, const Blocks& y, int ny, uintptr_t b) {
  const size_t of_x = x.reach(nx), of_y = y.reach(ny);
  if (a + of_x <= b || b + of_y <= a) return false;
  if (nx == 0 && ny == 0) return true;
  const size_t sx = nx ? x.step[nx - 1].stride : 0, sy = ny ? y.step[ny - 1].stride : 0;
  if (sx < sy || (sx == sy && b < a)) return share(y, ny, b, x, nx, a);
  const size_t count = x.step[nx - 1].count;
  if (sx == sy) {  // y's first row lies behind the start of x's row `row`; all other rows alike
    const size_t row = (b - a) / sx, in = (b - a) % sx;
    return (row < count && share(x, nx - 1, 0, y, ny - 1, in)) || (row + 1 < count && share(x, nx - 1, sx, y, ny - 1, in));
  }
  // x's rows that y reaches.  A dense y covers any between two of them; many of a y with gaps count as filled.
  const size_t row = x.reach(nx - 1), first = b >= a + row ? (b - a - row) / sx + 1 : 0,
               last = (b + of_y - 1 - a) / sx < count ? (b + of_y - 1 - a) / sx : count - 1;
  if (last >= first + (ny ? 16 : 2)) return true;
  for (size_t i = first; i <= last; ++i)
    if (share(x, nx - 1, a + i * sx, y, ny, b)) return true;
  return false;
}
inline bool share(const Blocks& x, const Blocks& y) {
  return x.at && y.at && x.bytes && y.bytes &&
         share(x, x.dims, reinterpret_cast<uintptr_t>(x.at), y, y.dims, reinterpret_cast<uintptr_t>(y.at));
}

// Whether an output shares memory with an input (Span or Blocks).
template <typename S = Span, size_t N, size_t M>
bool overlap(const S (&outs)[N], const S (&ins)[M]) {
  for (const S& o : outs)
    for (const S& i : ins)
      if (share(o, i)) return true;
  return false;
}

// Whether two outputs share memory.
template <typename S = Span, size_t N>
bool overlap(const S (&outs)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (share(outs[i], outs[j])) return true;
  return false;
}

inline size_t dtype_bytes(mesa_dtype t) { return t == MESA_BF16 ? 2 : 4; }

}  // namespace mesa
