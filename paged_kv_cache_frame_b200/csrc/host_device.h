// Index arithmetic that the kernels and the host tests share: compiled for
// both by nvcc, plain C++ elsewhere.
#pragma once
#include <stdint.h>

#if defined(__CUDACC__)
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

// An element of an index array that nobody writes while it is read.
PKV_HD int32_t index_at(const int32_t* p) {
#if defined(__CUDA_ARCH__)
  return __ldg(p);
#else
  return *p;
#endif
}

// A length as it stands, held to what a table can name.
template <typename Cache>
PKV_HD int held(const Cache& c, int n) {
  const int most = c.table_width * c.page_size;   // <= 2^30, checked by the host
  return n < 0 ? 0 : n > most ? most : n;
}

// Sequences of [0, n) that end at or before token t, all before the others:
// the sequence of token t (n where no sequence holds it).
PKV_HD int find_seq(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n;   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (cu[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

}  // namespace pkv
