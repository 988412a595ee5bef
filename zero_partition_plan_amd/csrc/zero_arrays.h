// The checks of a call's arrays that the block boundaries' and the token losses' entry points share.
#pragma once

#include <stdint.h>

#include "zero_internal.h"

namespace zero {

// A matrix of a call, or an array as a matrix of one row.
struct Arr {
  const char* name;
  const void* p;
  uint64_t rows, cols, ld;
  uint32_t bytes;  // of an element
  bool written;
  uint64_t size() const { return rows && cols ? ((rows - 1) * ld + cols) * bytes : 0; }
};

// Leading dimensions and alignment of every array, and overlaps of the written ones; arr[x0] may be arr[y0] itself.
inline zero_status check_arrays(const char* fn, const Arr* arr, int n, int x0 = -1, int y0 = -1) {
  for (int i = 0; i < n; ++i) {
    const Arr& a = arr[i];
    if (!a.p) continue;
    if (a.rows > 1 && a.ld < a.cols) return fail(ZERO_E_INVAL, "%s: %s: a leading dimension below the columns", fn, a.name);
    if (a.rows && a.ld >= (1ull << 63) / 4 / a.rows)
      return fail(ZERO_E_OVERFLOW, "%s: %s: a byte count does not fit in 63 bits", fn, a.name);
    if (a.size() && reinterpret_cast<uintptr_t>(a.p) % a.bytes)
      return fail(ZERO_E_INVAL, "%s: %s is not aligned to its element size", fn, a.name);
  }
  // Column slices of one buffer with the same leading dimension do not overlap, though their ranges do.
  auto apart = [](const Arr& x, const Arr& y) {
    const uint64_t lb = x.ld * x.bytes;
    if (x.rows < 2 || y.rows < 2 || lb != y.ld * y.bytes) return false;
    const uintptr_t p = reinterpret_cast<uintptr_t>(x.p), q = reinterpret_cast<uintptr_t>(y.p);
    const uint64_t gap = p < q ? (q - p) % lb : (p - q) % lb;  // of the one behind, from the other's rows
    const uint64_t front = (p < q ? x.cols * x.bytes : y.cols * y.bytes), back = (p < q ? y.cols * y.bytes : x.cols * x.bytes);
    return gap >= front && gap + back <= lb;
  };
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (!arr[i].written || i == j || !arr[i].p || !arr[j].p) continue;
      if (i == x0 && j == y0 && arr[i].p == arr[j].p && (arr[i].ld == arr[j].ld || arr[i].rows < 2)) continue;
      if (overlaps(arr[i].p, arr[i].size(), arr[j].p, arr[j].size()) && !apart(arr[i], arr[j]))
        return fail(ZERO_E_INVAL, "%s: %s overlaps %s", fn, arr[i].name, arr[j].name);
    }
  return ZERO_OK;
}

}  // namespace zero
