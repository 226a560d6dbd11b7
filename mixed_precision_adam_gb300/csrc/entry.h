// entry.h -- what the C entry points next to the step share: checks of
// pointers, sizes and types, and the guard that keeps exceptions inside.
#pragma once

#include <cmath>
#include <new>
#include <string>
#include <utility>

#include "dopt_internal.h"

namespace dopt {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t dtype_bytes(int32_t dtype) { return dtype == DOPT_F32 ? 4 : 2; }
inline bool known_dtype(int32_t dtype) { return dtype == DOPT_F32 || dtype == DOPT_BF16 || dtype == DOPT_F16; }

constexpr int64_t kMaxSide = int64_t(1) << 31;  // rows and columns stay below it
constexpr int64_t kMaxLd = int64_t(1) << 40;    // elements from row to row, so that byte distances fit 64 bits

// The distance of rows of values.
inline int check_ld(int64_t ld, int64_t cols, const std::string& who) {
  if (ld < cols) return fail(DOPT_E_INVALID, who + "ld below cols");
  if (ld > kMaxLd) return fail(DOPT_E_SIZE, who + "ld too large");
  return DOPT_OK;
}

// Sizes of a matrix.
inline int check_sides(int64_t rows, int64_t cols, const std::string& who) {
  if (rows < 0 || cols < 0) return fail(DOPT_E_INVALID, who + "negative size");
  if (rows >= kMaxSide || cols >= kMaxSide) return fail(DOPT_E_SIZE, who + "a size of 2^31 or more");
  return DOPT_OK;
}

// An 8-bit matrix with elements: its codes, scales and row distance.
inline int check_matrix8(const dopt_matrix8& m, const std::string& who) {
  if (!m.codes || !m.scales) return fail(DOPT_E_INVALID, who + "NULL codes or scales");
  if (!aligned_to(m.codes, 16) || !aligned_to(m.scales, 16))
    return fail(DOPT_E_ALIGN, who + "codes or scales not 16-byte aligned");
  if (m.ld < m.cols) return fail(DOPT_E_INVALID, who + "ld below cols");
  if (m.ld % 16) return fail(DOPT_E_ALIGN, who + "ld of the codes not a multiple of 16");
  if (m.ld >= kMaxSide * 2) return fail(DOPT_E_SIZE, who + "ld too large");
  return DOPT_OK;
}

// The drop threshold T of a dropout.
inline int check_drop(const dopt_drop& d, uint32_t* threshold, const std::string& who) {
  *threshold = 0;
  if (!(d.p >= 0.0 && d.p < 1.0)) return fail(DOPT_E_INVALID, who + "the dropout's p is not in [0, 1)");
  const double t = std::nearbyint(d.p * 65536.0);
  if (t > 65535.0) return fail(DOPT_E_INVALID, who + "the dropout's p is too near to 1");
  if (!aligned_to(d.d_step, 8)) return fail(DOPT_E_ALIGN, who + "d_step not 8-byte aligned");
  *threshold = (uint32_t)t;
  return DOPT_OK;
}

// What the rows of two arrays (`ld` elements apart, of `cols` elements of
// `elem` bytes) have in common: nothing, all of them row by row, or some
// elements at different places.  Rows of different distances that begin at
// different places count as apart: whether they meet is not looked for.
enum class Shared { none, same, some };
inline Shared shared_elements(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols, size_t elem) {
  if (!a || !b || rows <= 0 || cols <= 0) return Shared::none;
  if (a == b) return rows == 1 || lda == ldb ? Shared::same : Shared::some;
  if (reinterpret_cast<uintptr_t>(a) > reinterpret_cast<uintptr_t>(b)) {
    std::swap(a, b);
    std::swap(lda, ldb);
  }
  const uint64_t apart = reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a), width = (uint64_t)cols * elem;
  if (rows == 1) return apart < width ? Shared::some : Shared::none;
  if (lda != ldb) return Shared::none;
  // a row of b begins q rows and r bytes after a row of a
  const uint64_t pitch = (uint64_t)lda * elem, q = apart / pitch, r = apart % pitch;
  return (r < width && q < (uint64_t)rows) || (pitch - r < width && q + 1 < (uint64_t)rows) ? Shared::some : Shared::none;
}
// Of two arrays one of which is written: two outputs share nothing; an output
// and an input nothing, or the same rows.
inline int check_shared(Shared s, bool both_written, const char* a, const char* b, const std::string& fn) {
  if (s == Shared::some) return fail(DOPT_E_INVALID, fn + a + " and " + b + " share elements at different places");
  if (s == Shared::same && both_written) return fail(DOPT_E_INVALID, fn + a + " and " + b + " are one array");
  return DOPT_OK;
}

// Runs an entry point's body: a host allocation that fails (an error
// message's, say) is a status, not an exception through the C boundary.
template <typename F>
int guard_entry(F&& body) noexcept {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return DOPT_E_NOMEM;
  } catch (...) {
    return DOPT_E_INVALID;
  }
}

}  // namespace dopt
