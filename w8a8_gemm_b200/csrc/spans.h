// spans.h -- do two buffers of a call share a byte?  Host arithmetic without CUDA.
#pragma once
#include <stdint.h>

namespace sq {

// `rows` rows of `bytes` bytes, `pitch` bytes from one to the next (pitch >= bytes).
struct Span {
  uintptr_t at = 0;
  int64_t rows = 0, bytes = 0, pitch = 0;
  Span(const void *p, int64_t n, int64_t row_bytes, int64_t row_pitch)
      : at(reinterpret_cast<uintptr_t>(p)), rows(n), bytes(row_bytes), pitch(row_pitch) {
    if (rows > 1 && pitch == bytes) bytes *= rows, rows = 1;  // one run of bytes
  }
  Span(const void *p, int64_t run) : Span(p, 1, run, run) {}
  bool none() const { return at == 0 || rows < 1 || bytes < 1; }
  uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * pitch + bytes); }
};

// Exact where one of the two is a single run of bytes or both have the same
// pitch (columns of one wider buffer); two buffers of rows at different pitches are
// not looked into further than their ends.
inline bool overlap(const Span &a, const Span &b) {
  if (a.none() || b.none() || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows == 1 || b.rows == 1) {
    const Span &run = a.rows == 1 ? a : b, &s = a.rows == 1 ? b : a;
    // the first row that ends behind the run's beginning
    const int64_t before = static_cast<int64_t>(run.at - s.at) - s.bytes;
    const int64_t row = run.at < s.at || before < 0 ? 0 : before / s.pitch + 1;
    return row < s.rows && s.at + static_cast<uintptr_t>(row * s.pitch) < run.end();
  }
  if (a.pitch != b.pitch) return false;
  // b's row j lies m + (q + j - i) pitch bytes behind a's row i
  const int64_t d = static_cast<int64_t>(b.at - a.at), p = a.pitch;
  const int64_t q = d >= 0 ? d / p : -((-d + p - 1) / p), m = d - q * p;
  auto rows_differ_by = [&](int64_t k) { return k > -a.rows && k < b.rows; };
  return (m < a.bytes && rows_differ_by(-q)) || (p - m < b.bytes && rows_differ_by(-q - 1));
}

// Whether `out` overlaps any of the others.
template <typename... Others>
bool overlaps_any(const Span &out, const Others &...others) {
  return (overlap(out, others) || ...);
}

}  // namespace sq
