// Shared by the token kernels: packed rows, type conversion, the page of a
// token.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "host_device.h"
#include "sm100.cuh"
#include "token_kernels.h"

namespace pkv {

template <typename T>
constexpr bool kIsFp16 = false;
template <>
constexpr bool kIsFp16<__half> = true;

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

// Two 16-bit values in a register (the first in the lower half), rounded to
// nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return kIsFp16<T> ? cvt_pack_f16(a, b) : cvt_pack_bf16(a, b);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// N values of T as they lie in memory, moved in one access: 32-bit words,
// each a float or two 16-bit values, or a single 16-bit value.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  static constexpr int kPerWord = 4 / sizeof(T);
  uint32_t w[N / kPerWord];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kPerWord == 1) return __uint_as_float(w[i]);
    else return i % 2 ? unpack2<T>(w[i / 2]).y : unpack2<T>(w[i / 2]).x;
  }
  // Values 2i and 2i + 1.
  __device__ __forceinline__ void set2(int i, float a, float b) {
    if constexpr (kPerWord == 1) {
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    } else {
      w[i] = pack2<T>(a, b);
    }
  }
};
template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void set(float a) { v = from_f32<T>(a); }
};

// Past the first-level cache: written by other CTAs of the launch.
__device__ __forceinline__ Pack<float, 2> load_cg(const Pack<float, 2>* p) {
  const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
  return {{x.x, x.y}};
}
__device__ __forceinline__ Pack<float, 4> load_cg(const Pack<float, 4>* p) {
  const uint4 x = __ldcg(reinterpret_cast<const uint4*>(p));
  return {{x.x, x.y, x.z, x.w}};
}

// Bits of the cache's error word (kv_tokens_check).
constexpr uint32_t kErrIndex = 2u;       // a page id, a length or cu_new out of range
constexpr uint32_t kErrWorkspace = 4u;   // a workspace that was not prepared

__device__ __forceinline__ void raise_error(uint32_t* word, uint32_t bit) { atomicOr(word, bit); }

// The length of sequence s, held to what its table can name.
__device__ __forceinline__ int seq_len(const TokenCache& c, int s) { return held(c, __ldg(c.lens + s)); }
__device__ __forceinline__ bool seq_len_bad(const TokenCache& c, int s) {
  const int n = __ldg(c.lens + s);
  return n < 0 || n > c.table_width * c.page_size;
}

// j / d for the divisor that page_divisor prepared.
__device__ __forceinline__ int divided(int j, uint32_t mul, int shift) {
  return mul ? (int)(__umulhi((uint32_t)j, mul) >> shift) : j;
}
__device__ __forceinline__ int page_of(const TokenCache& c, int j) { return divided(j, c.page_mul, c.page_shift); }

// K row of the sequence's token j, on page `page`, in the pool's
// [max_pages * 2 * page_size] rows (its V row is page_size further), or -1
// where that is no page of the pool. Rows fit 31 bits (checked by the host).
__device__ __forceinline__ int row_in(const TokenCache& c, int page, int j) {
  if ((unsigned)page >= (unsigned)c.max_pages) return -1;
  return page * 2 * c.page_size + (j - page_of(c, j) * c.page_size);
}

// Head h of token row `row`: offset in elements.
__device__ __forceinline__ long long row_offset(const TokenCache& c, int row, int h) {
  return ((long long)row * c.H + h) * c.D;
}

}  // namespace pkv
