// Whether two arrays of spaced rows share a byte (host).
#pragma once
#include <cstdint>

namespace llm {

// Bytes [p + r ld, p + r ld + w) for r < n, w <= ld, against [q, q + len).
inline bool overlap(uintptr_t p, int64_t ld, int64_t w, int64_t n, uintptr_t q, int64_t len) {
  if (q + len <= p || q >= p + (n - 1) * ld + w) return false;
  if (q <= p) return true;
  const int64_t r = (int64_t)(q - p) / ld, in = (int64_t)(q - p) % ld;  // r < n
  return in < w || (r + 1 < n && in + len > ld);
}
// Two arrays of n rows of w bytes, ld and ld2 apart.
inline bool rows_overlap(const void *a, int64_t ld, const void *b, int64_t ld2, int64_t w, int64_t n) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  if (!overlap(p, (n - 1) * ld + w, (n - 1) * ld + w, 1, q, (n - 1) * ld2 + w)) return false;
  if (ld == ld2) {  // rows k apart start d - k ld apart: the two nearest
    const int64_t d = p < q ? (int64_t)(q - p) : (int64_t)(p - q), k = d / ld;
    return (k < n && d - k * ld < w) || (k + 1 < n && (k + 1) * ld - d < w);
  }
  for (int64_t r = 0; r < n; r++)
    if (overlap(p, ld, w, n, q + r * ld2, w)) return true;
  return false;
}

}  // namespace llm
