// Shared by the token kernels: packed rows, type conversion, the page of a
// token.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "token_kernels.h"

namespace pkv {

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Bits of the cache's error word (kv_tokens_check).
constexpr uint32_t kErrIndex = 2u;

__device__ __forceinline__ void raise_error(uint32_t* word) { atomicOr(word, kErrIndex); }

// The length of sequence s, held to what its table can name.
__device__ __forceinline__ int seq_len(const TokenCache& c, int s) {
  const int n = __ldg(c.lens + s);
  const int most = c.table_width * c.page_size;   // <= INT32_MAX, checked by the host
  return n < 0 ? 0 : n > most ? most : n;
}
__device__ __forceinline__ bool seq_len_bad(const TokenCache& c, int s) {
  const int n = __ldg(c.lens + s);
  return n < 0 || n > c.table_width * c.page_size;
}

__device__ __forceinline__ int page_of(const TokenCache& c, int j) {
  return c.page_mul ? (int)(__umulhi((uint32_t)j, c.page_mul) >> c.page_shift) : j;
}

// K row of token j of sequence s in the pool's [max_pages * 2 * page_size]
// rows (its V row is page_size further), or -1 where the table holds no page
// of the pool. Rows fit 31 bits (checked by the host).
__device__ __forceinline__ int token_row(const TokenCache& c, int s, int j) {
  const int i = page_of(c, j);
  const int page = __ldg(c.tables + s * c.table_stride + i);
  if ((unsigned)page >= (unsigned)c.max_pages) return -1;
  return page * 2 * c.page_size + (j - i * c.page_size);
}

// Head h of token row `row`: offset in elements.
__device__ __forceinline__ long long row_offset(const TokenCache& c, int row, int h) {
  return ((long long)row * c.H + h) * c.D;
}

}  // namespace pkv
