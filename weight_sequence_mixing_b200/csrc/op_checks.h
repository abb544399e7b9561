// Host checks of the operators' tensors (ttt_ops.h): which elements a strided
// tensor covers, whether a written tensor overlaps itself, and whether two
// tensors share elements.  Plain C++, no CUDA types; nothing here throws.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/ttt_ops.h"

namespace ttt {

// A tensor of rows: up to three counted dimensions with a stride each, in
// elements, and `width` contiguous elements a row.
struct RowTensor {
  const void* ptr;
  int elem;  // bytes per element
  int64_t width;
  int64_t n[3], stride[3];
  RowTensor(const void* p, int elem_bytes, int64_t w, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1,
            int64_t s2 = 0)
      : ptr(p), elem(elem_bytes), width(w), n{n0, n1, n2}, stride{s0, s1, s2} {}

  bool empty() const { return width == 0 || n[0] == 0 || n[1] == 0 || n[2] == 0; }

  // elements from the first to the one after the last, or -1 above 2^60
  int64_t span() const {
    if (empty()) return 0;
    __int128 s = width;
    for (int i = 0; i < 3; ++i) s += __int128(n[i] - 1) * stride[i];
    return s > (__int128(1) << 60) ? -1 : int64_t(s);
  }

  // usable as an input: there, aligned to its elements, no negative stride
  bool readable() const {
    if (empty()) return true;
    if (!ptr || reinterpret_cast<uintptr_t>(ptr) % elem) return false;
    for (int i = 0; i < 3; ++i)
      if (n[i] < 0 || stride[i] < 0) return false;
    return span() >= 0;
  }

  // usable as an output: no element has two places.  With the dimensions in the
  // order of their strides, each step must clear all that lies inside it.
  bool writable() const {
    if (!readable()) return false;
    if (empty()) return true;
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (stride[order[j]] > stride[order[j + 1]]) {
          const int t = order[j];
          order[j] = order[j + 1];
          order[j + 1] = t;
        }
    __int128 inner = width;
    for (int k = 0; k < 3; ++k) {
      const int i = order[k];
      if (n[i] <= 1) continue;
      if (stride[i] < inner) return false;
      inner += __int128(n[i] - 1) * stride[i];
    }
    return true;
  }
};

inline bool same_tensor(const RowTensor& a, const RowTensor& b) {
  if (a.ptr != b.ptr || a.width != b.width) return false;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return true;
}

// Whether the tensors may share bytes.  Exact for tensors that do not interleave;
// for two of the same shape and strides whose rows interleave (two column ranges of
// one buffer), rows start at fixed remainders modulo the smallest stride, which
// keeps them apart when the remainders do.  Dimensions that lie densely behind one
// another (the heads of a token) count as one row.  Anything else that interleaves
// counts as sharing.
inline bool may_share(const RowTensor& a, const RowTensor& b) {
  if (a.empty() || b.empty()) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.ptr), b0 = reinterpret_cast<uintptr_t>(b.ptr);
  if (a0 + uintptr_t(a.span()) * a.elem <= b0 || b0 + uintptr_t(b.span()) * b.elem <= a0) return false;
  if (a.elem != b.elem || a.width != b.width) return true;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.stride[i] != b.stride[i])) return true;
  int64_t width = a.width;
  bool folded[3] = {a.n[0] <= 1, a.n[1] <= 1, a.n[2] <= 1};
  for (int pass = 0; pass < 3; ++pass)
    for (int i = 0; i < 3; ++i)
      if (!folded[i] && a.stride[i] == width) {
        width *= a.n[i];  // at most the span
        folded[i] = true;
      }
  int64_t step = 0;
  for (int i = 0; i < 3; ++i)
    if (!folded[i] && (step == 0 || a.stride[i] < step)) step = a.stride[i];
  if (step == 0) return true;
  for (int i = 0; i < 3; ++i)
    if (!folded[i] && a.stride[i] % step) return true;
  const uint64_t gap = a0 < b0 ? b0 - a0 : a0 - b0;
  if (gap % a.elem) return true;
  const int64_t r = int64_t(gap / a.elem % uint64_t(step));
  return r < width || step - r < width;
}

// whether every row of the tensor starts on a multiple of `bytes`
inline bool rows_aligned(const RowTensor& t, int bytes) {
  if (t.empty()) return true;
  if (reinterpret_cast<uintptr_t>(t.ptr) % bytes) return false;
  for (int i = 0; i < 3; ++i)
    if (t.n[i] > 1 && (__int128(t.stride[i]) * t.elem) % bytes) return false;
  return true;
}

inline bool is_aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace ttt
