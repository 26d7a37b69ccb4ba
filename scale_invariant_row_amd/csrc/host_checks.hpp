// Host-side helpers of the C ABI's entry points: argument checks, overlap
// tests, the grid cap and launches in pieces.
#pragma once

#include "ds_rows.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <map>
#include <mutex>

namespace dsh {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Output buffer may be exactly the input buffer, or disjoint from it.
inline bool same_or_disjoint(const void* out, const void* in, size_t n) {
  return in == nullptr || out == in || !overlaps(out, n, in, n);
}

inline bool finite_nonneg(float v) { return std::isfinite(v) && v >= 0.f; }

// rows x cols elements of `esize` bytes; cols a multiple of `mult`.
inline int check_matrix(int64_t rows, int64_t cols, int64_t mult, int64_t esize) {
  if (rows < 0 || cols < mult || cols > DS_MAX_COLS || cols % mult != 0) return DS_ERR_SHAPE;
  if (rows > (INT64_MAX / 8) / (cols * esize)) return DS_ERR_SHAPE;
  return DS_OK;
}

// Compute units of the current device, cached per device.
inline int device_cus(int* cus) {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return DS_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(dev);
  if (it == cache.end()) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      return DS_ERR_DEVICE;
    it = cache.emplace(dev, n).first;
  }
  *cus = it->second;
  return DS_OK;
}

// Workgroups for `units` row groups (or items): one each, up to 64 per
// compute unit in a launch, well above what the chip holds at once.  Past
// that the ragged kernels loop (grid-stride) and the row kernels run as
// several launches (launch_in_pieces).  A cap of 2^20 workgroups measured
// the same (GPT-2's 768-wide linears, 18,432 items: 89.6-89.9 against
// 89.8-90.3 us forward).  DS_ROWS_TEST_MAX_GROUPS lowers the cap: a test
// hook that runs the several-launch and grid-stride paths at small sizes.
inline int64_t max_launch_groups(int cus) {
  const int64_t cap = (int64_t)cus * 64;
  const char* e = std::getenv("DS_ROWS_TEST_MAX_GROUPS");
  if (e != nullptr) {
    const long long v = std::atoll(e);
    if (v >= 1 && v < cap) return v;
  }
  return cap;
}

inline int grid_for(int64_t units, int cus) {
  return (int)std::max<int64_t>(1, std::min(units, max_launch_groups(cus)));
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? DS_OK : DS_ERR_LAUNCH; }

// For kernels that take one row group per workgroup, with no grid-stride
// loop: launch(r0, n) over rows [r0, r0 + n), in pieces of at most the grid
// cap of row groups (rows_per_group rows each).
template <class F>
hipError_t launch_in_pieces(int64_t rows, int rows_per_group, int cus, F&& launch) {
  const int64_t piece = max_launch_groups(cus) * rows_per_group;
  for (int64_t r0 = 0; r0 < rows; r0 += piece) {
    const hipError_t e = launch(r0, std::min<int64_t>(piece, rows - r0));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Bytes a strided [rows, width] bf16 view spans.
inline size_t span_bytes(int64_t rows, int64_t ld, int64_t width) {
  return rows == 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * 2;
}

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - ((a % b != 0) && ((a < 0) != (b < 0))); }

// Two [rows, wa] and [rows, wb] bf16 views at a and b share an element.  With
// one row stride ld (>= wa, wb) the test is exact: element (ra, ca) of a is
// element (rb, cb) of b when (ra - rb) ld = de + cb - ca, de = (b - a) / 2,
// so some multiple k ld with |k| < rows must lie in (de - wa, de + wb).
// Otherwise it compares the spans.
inline bool views_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb,
                   int64_t rows) {
  if (rows == 0 || wa == 0 || wb == 0 || a == nullptr || b == nullptr) return false;
  const intptr_t d = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a);
  if (lda != ldb || d % 2 != 0)
    return overlaps(a, span_bytes(rows, lda, wa), b, span_bytes(rows, ldb, wb));
  const int64_t de = d / 2, ld = lda;
  const int64_t k_lo = std::max<int64_t>(floor_div(de - wa, ld) + 1, -(rows - 1));
  const int64_t k_hi = std::min<int64_t>(floor_div(de + wb - 1, ld), rows - 1);
  for (int64_t k = k_lo; k <= k_hi; ++k) {
    const int64_t t = k * ld;          // t in [de - wa + 1, de + wb - 1] by construction
    if (t > de - wa && t < de + wb) return true;
  }
  return false;
}

}  // namespace dsh
