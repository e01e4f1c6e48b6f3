// Host test of the binding's overlap rule: random sets of rows against their
// bytes. Exits non-zero on a failure.
#include <cstdio>
#include <random>
#include <set>

#include "overlap.h"

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return (int64_t)std::uniform_int_distribution<int>(lo, hi)(rng); };
  long long sharing = 0, apart = 0, over = 0;
  auto bytes = [](const pkv::RowSet& x) {
    std::set<int64_t> s;
    for (int64_t t = 0; t < x.n; ++t)
      for (int64_t i = 0; i < x.h; ++i)
        for (int64_t e = 0; e < x.d; ++e) s.insert(x.p + t * x.ts + i * x.hs + e);
    return s;
  };
  for (int round = 0; round < 400000; ++round) {
    auto draw = [&]() {
      pkv::RowSet x;
      x.p = 1000 + pick(0, 60);
      x.n = pick(0, 20) ? pick(1, 4) : 0;
      x.h = pick(1, 4);
      x.d = pick(1, 4);
      const int kind = (int)pick(0, 4);
      x.hs = kind == 0 ? pick(0, 12) : kind == 1 ? 0 : x.d + (pick(0, 1) ? pick(0, 3) : 0);
      x.ts = kind == 0 ? pick(0, 40) : kind == 2 ? 0 : x.h * x.hs + (pick(0, 1) ? pick(0, 20) : 0);
      if (pick(0, 3) == 0) std::swap(x.n, x.h), std::swap(x.ts, x.hs);
      return x;
    };
    const pkv::RowSet a = draw();
    pkv::RowSet b = draw();
    if (pick(0, 2) == 0) {   // the same rows elsewhere
      b = a;
      b.p += pick(-30, 30);
    }
    const auto sa = bytes(a), sb = bytes(b);
    bool want = false;
    for (int64_t x : sa) want = want || sb.count(x);
    const bool got = pkv::share_memory(a, b);
    const auto oa = pkv::in_order(a), ob = pkv::in_order(b);
    if ((!sa.empty() && bytes(oa) != sa) || (!sb.empty() && bytes(ob) != sb)) return std::printf("FAIL in_order, round %d\n", round), 1;
    const bool exact = pkv::ordered(oa) || pkv::ordered(ob);
    if (got != want && (exact || !got))
      return std::printf("FAIL round %d: [%d %d %d +%d +%d at %d] [%d %d %d +%d +%d at %d]: %d, expected %d\n", round, (int)a.n,
                         (int)a.h, (int)a.d, (int)a.ts, (int)a.hs, (int)a.p, (int)b.n, (int)b.h, (int)b.d, (int)b.ts, (int)b.hs,
                         (int)b.p, got, want),
             1;
    (want ? sharing : apart) += 1;
    over += got != want;
  }
  std::printf("ok %lld sharing, %lld apart, %lld taken for sharing\n", sharing, apart, over);
  return 0;
}
