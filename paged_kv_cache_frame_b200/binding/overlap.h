// Whether two strided tensors of rows share memory: plain C++, shared by the
// binding and the host test.
#pragma once
#include <cstdint>
#include <utility>

namespace pkv {

// n x h rows of d bytes: row (t, i) starts at byte p + t * ts + i * hs.
// Strides are not negative.
struct RowSet {
  int64_t p, n, h, d, ts, hs;
};

// The same rows (at least one) in order of their address where they can be: dimensions
// without a step dropped, the larger stride first, neighbours run together.
inline RowSet in_order(RowSet a) {
  if (a.h == 1 || a.hs == 0) a.h = 1, a.hs = 0;
  if (a.n == 1 || a.ts == 0) a.n = 1, a.ts = 0;
  if (a.h == 1 || (a.n > 1 && a.ts < a.hs)) std::swap(a.n, a.h), std::swap(a.ts, a.hs);
  if (a.h > 1 && a.hs == a.d) a.d *= a.h, a.h = 1, a.hs = 0;
  if (a.h == 1 && a.n > 1 && a.ts == a.d) a.d *= a.n, a.n = 1, a.ts = 0;
  if (a.h == 1) std::swap(a.n, a.h), std::swap(a.ts, a.hs);
  return a;
}
// No row begins before the one in front of it has ended.
inline bool ordered(const RowSet& a) { return (a.h == 1 || a.hs >= a.d) && (a.n == 1 || a.ts >= (a.h - 1) * a.hs + a.d); }

// Whether any byte lies in both. Exact where one of the two is ordered, or
// both have the same rows and strides; else sets that reach into each other
// count as sharing.
inline bool share_memory(RowSet a, RowSet b) {
  if (a.n <= 0 || a.h <= 0 || a.d <= 0 || b.n <= 0 || b.h <= 0 || b.d <= 0) return false;
  a = in_order(a);
  b = in_order(b);
  auto end = [](const RowSet& x) { return x.p + (x.n - 1) * x.ts + (x.h - 1) * x.hs + x.d; };
  if (a.p >= end(b) || b.p >= end(a)) return false;
  const int64_t delta = b.p - a.p;
  if (a.n == b.n && a.h == b.h && a.d == b.d && a.ts == b.ts && a.hs == b.hs) {
    // delta = dt * ts + di * hs + less than a row, for some difference of two rows' places
    for (int64_t di = 1 - a.h; di < a.h; ++di) {
      const int64_t rest = delta - di * a.hs;
      int64_t dt = a.n > 1 ? rest / a.ts : 0;   // the nearest two multiples, whichever way this rounds
      for (int64_t k = dt - 1; k <= dt + 1; ++k) {
        const int64_t off = rest - k * a.ts;
        if (k > -a.n && k < a.n && off < a.d && off > -a.d) return true;
      }
    }
    return false;
  }
  if (!ordered(b) || (ordered(a) && a.n * a.h > b.n * b.h)) std::swap(a, b);
  if (!ordered(b)) return true;
  for (int64_t t = 0; t < a.n; ++t)
    for (int64_t i = 0; i < a.h; ++i) {
      const int64_t lo = a.p + t * a.ts + i * a.hs, last = lo + a.d - 1 - b.p;   // its last byte, from b's first
      if (last < 0) continue;
      // the last row of b that begins by then: the one that ends last
      int64_t bt = b.n > 1 ? last / b.ts : 0;
      if (bt >= b.n) bt = b.n - 1;
      int64_t bi = b.h > 1 ? (last - bt * b.ts) / b.hs : 0;
      if (bi >= b.h) bi = b.h - 1;
      if (b.p + bt * b.ts + bi * b.hs + b.d > lo) return true;
    }
  return false;
}

}  // namespace pkv
