// Division of a token's index by the page size as a product: plain C++, shared
// by the launchers and the host tests.
#pragma once
#include <stdint.h>

namespace pkv {

// For 0 <= j < 2^31 and d > 1, with s = ceil(log2 d) and
// m = floor(2^(31 + s) / d) + 1: m d - 2^(31 + s) lies in (0, d] and d <= 2^s,
// so floor(j m / 2^(31 + s)) = floor(j / d), and m fits 32 bits. The kernels
// take the product's upper half and shift it by s - 1; mul 0 stands for d = 1.
inline void page_divisor(int page_size, uint32_t* mul, int* shift) {
  *mul = 0;
  *shift = 0;
  if (page_size == 1) return;
  int s = 0;
  while ((1LL << s) < page_size) ++s;
  *mul = (uint32_t)((1ULL << (31 + s)) / (uint32_t)page_size + 1);
  *shift = s - 1;
}

}  // namespace pkv
