// Host test of the page divisor: j / d as the kernels work it out, at every
// border of j and for divisors of all sizes. Exits non-zero on a failure.
#include <cstdio>

#include "page_divisor.h"

int main() {
  long long checked = 0;
  for (long long d = 1; d < (1LL << 31); d = d < 3000 ? d + 1 : d + d / 7 + 1) {
    uint32_t mul;
    int shift;
    pkv::page_divisor((int)d, &mul, &shift);
    auto div = [&](uint32_t j) { return mul ? (uint32_t)(((uint64_t)j * mul) >> 32) >> shift : j; };
    auto at = [&](long long j) {
      if (j < 0 || j >= (1LL << 31)) return true;
      ++checked;
      return div((uint32_t)j) == (uint32_t)(j / d);
    };
    const long long last = ((1LL << 31) - 1) / d * d;
    for (long long q = 0; q <= last; q += (last / 37 / d + 1) * d)
      for (int e = -1; e <= 1; ++e)
        if (!at(q + e)) return std::printf("FAIL %lld / %lld\n", q + e, d), 1;
    if (!at(last) || !at(last - 1) || !at((1LL << 31) - 1)) return std::printf("FAIL last / %lld\n", d), 1;
  }
  std::printf("ok %lld\n", checked);
  return 0;
}
