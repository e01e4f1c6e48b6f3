// Rotary positions (kv_rotate): pair (a, b) of head values at position p
// becomes m (a cos - b sin, b cos + a sin) with the angle p * theta_i and the
// amplitude m; the gradient is the same with the negative angle.
//
// Bound by its bytes (each value read and written once). A thread keeps one
// unit of V pairs of a token, works its angles out once and goes through the
// token's heads with them, four heads' loads in flight; the threads of a
// block split heads and tokens. Sums of two products are in 32 bits, rounded
// once to the tensor's type.
#include "launch.cuh"
#include "rope_unit.cuh"

namespace pkv {

constexpr int kThreads = 256;
constexpr int kAhead = 4;   // heads in flight per thread

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a, int units,
                                                          int head_slots) {
  const int u = threadIdx.x % units;
  const int row = threadIdx.x / units;
  const int per_block = kThreads / units / head_slots;   // tokens
  const int token = (int)blockIdx.x * per_block + row / head_slots;
  const int h0 = row % head_slots;
  pdl_wait();
  pdl_trigger();
  if (row >= per_block * head_slots || token >= a.n_tokens) return;
  RopeUnit<T, V, kInter> unit;
  unit.place(u, a.head_dim, a.rope.rot);
  if (!unit.turns && !a.copy_rest) return;
  const T* x = static_cast<const T*>(a.x.p) + token * a.x.token_stride;
  T* y = static_cast<T*>(a.out.p) + token * a.out.token_stride;
  if (unit.turns) unit.angles(a.rope, u, __ldg(a.positions + token), a.inverse);
  for (int h = h0; h < a.n_heads; h += kAhead * head_slots) {
    Pack<T, V> x0[kAhead], x1[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int g = h + i * head_slots;
      if (g < a.n_heads) {
        const T* p = x + g * a.x.head_stride;
        x0[i] = *reinterpret_cast<const Pack<T, V>*>(p + unit.at0);
        if (unit.second) x1[i] = *reinterpret_cast<const Pack<T, V>*>(p + unit.at1);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int g = h + i * head_slots;
      if (g < a.n_heads) {
        T* p = y + g * a.out.head_stride;
        if (unit.turns) {
          Pack<T, V> y0, y1;
          unit.turn(x0[i], x1[i], u, a.rope.rot, y0, y1);
          x0[i] = y0;
          x1[i] = y1;
        }
        *reinterpret_cast<Pack<T, V>*>(p + unit.at0) = x0[i];
        if (unit.second) *reinterpret_cast<Pack<T, V>*>(p + unit.at1) = x1[i];
      }
    }
  }
}

template <typename T, int V, bool kInter>
static cudaError_t launch(const RotateArgs& a, cudaStream_t stream) {
  const int units = (a.head_dim + 2 * V - 1) / (2 * V);
  const int rows = kThreads / units;
  // Split a token's heads over just enough threads to fill the GPU (148 SMs of
  // 1024): every slot works the token's angles out again.
  int slots = 1;
  while (2 * slots <= rows && slots < a.n_heads && (long long)a.n_tokens * units * slots < 148 * 1024) slots *= 2;
  const int per_block = rows / slots;
  const int blocks = (a.n_tokens + per_block - 1) / per_block;
  return launch_pdl(rotate_kernel<T, V, kInter>, dim3(blocks), dim3(kThreads), 0, stream, a, units, slots);
}

// 16-byte packs where the rows and the rotated half allow them, else single
// values.
template <typename T>
static cudaError_t launch_typed(const RotateArgs& a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const bool inter = a.rope.interleaved;
  const bool wide = a.head_dim % (2 * V) == 0 && (inter || a.rope.rot % (2 * V) == 0) &&
                    (reinterpret_cast<uintptr_t>(a.x.p) | reinterpret_cast<uintptr_t>(a.out.p)) % 16 == 0 &&
                    (a.x.token_stride | a.x.head_stride | a.out.token_stride | a.out.head_stride) % V == 0;
  if (wide) return inter ? launch<T, V, true>(a, stream) : launch<T, V, false>(a, stream);
  return inter ? launch<T, 1, true>(a, stream) : launch<T, 1, false>(a, stream);
}

cudaError_t launch_rotate(const RotateArgs& a, int dtype, cudaStream_t stream) {
  if (a.n_tokens <= 0 || a.n_heads <= 0) return cudaSuccess;
  if (dtype == KV_BF16) return launch_typed<__nv_bfloat16>(a, stream);
  if (dtype == KV_FP16) return launch_typed<__half>(a, stream);
  return launch_typed<float>(a, stream);
}

}  // namespace pkv
