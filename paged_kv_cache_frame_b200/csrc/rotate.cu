// Rotary positions (kv_rotate): pair (a, b) of head values at position p
// becomes m (a cos - b sin, b cos + a sin) with the angle p * theta_i and the
// amplitude m; the gradient is the same with the negative angle.
//
// Bound by its bytes (each value read and written once). A block takes a few
// tokens with all of their heads; its threads go through the (token, head)
// rows with kAhead rows' loads in flight, each thread at its own unit of V
// pairs. Sums of two products are in 32 bits, rounded once to the tensor's
// type. 8192 tokens x 40 heads x 128 values of 16 bits, inputs not in cache:
// 29.7 us, 5.65 TB/s, 86% of a copy's rate (with the angles worked out by each
// thread for itself 48.8, with blocks of 256 threads 31.1, with four rows in
// flight and fewer blocks 30.6). 32-bit values, forward and gradient: 35.5 us
// for 201 MB, 87%. Pairs (i, i + rot / 2) with rot / 2 off the packs' grid go
// value by value: 77 us for the first of these with 120 of 128 values rotated,
// 42 for 8192 x 32 heads of 80 with 20 (84 MB).
#include "launch.cuh"
#include "rope_unit.cuh"

namespace pkv {

namespace {
constexpr int kThreads = 128;    // of a block; twice as many for heads of more units (KV_MAX_ROTATE_DIM in single values)
constexpr int kAhead = 2;        // rows in flight per thread
constexpr int kMaxTokens = 16;   // tokens of a block
}  // namespace

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(2 * kThreads, 4) rotate_kernel(const __grid_constant__ RotateArgs a, int units,
                                                          int per_block) {
  extern __shared__ __align__(16) float2 s_angle[];
  const int u = threadIdx.x % units;
  const int slot = threadIdx.x / units, slots = blockDim.x / units;   // at least one
  const int first = (int)blockIdx.x * per_block;
  const int tokens = min(per_block, a.n_tokens - first);
  const int rows = tokens * a.n_heads;
  const RopeUnit<T, V, kInter> unit(u, a.head_dim, a.rope.rot);
  const bool on = slot < slots && (unit.turns || a.copy_rest);
  pdl_wait();
  pdl_trigger();
  using P = Pack<T, V>;
  P x0[kAhead], x1[kAhead];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * slots;
      if (on && r < rows) {
        const int t = divided(r, a.head_mul, a.head_shift);
        const T* p = static_cast<const T*>(a.x.p) + (first + t) * a.x.token_stride + (r - t * a.n_heads) * a.x.head_stride;
        x0[i] = *reinterpret_cast<const P*>(p + unit.at0);
        if (unit.second) x1[i] = *reinterpret_cast<const P*>(p + unit.at1);
      }
    }
  };
  load(slot);   // on their way while the angles are worked out
  const int pairs = a.rope.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
    const int t = i / pairs, p = i - t * pairs;
    float c, s;
    rope_angle(a.rope.turn[p], __ldg(a.positions + first + t), a.rope.amplitude, c, s);
    s_angle[angle_at<V>(units, t, p)] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  for (int r0 = slot; r0 < rows; r0 += kAhead * slots) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * slots;
      if (on && r < rows) {
        const int t = divided(r, a.head_mul, a.head_shift);
        T* p = static_cast<T*>(a.out.p) + (first + t) * a.out.token_stride + (r - t * a.n_heads) * a.out.head_stride;
        if (unit.turns) unit.turn(x0[i], x1[i], s_angle, units, t, a.rope.rot);
        *reinterpret_cast<P*>(p + unit.at0) = x0[i];
        if (unit.second) *reinterpret_cast<P*>(p + unit.at1) = x1[i];
      }
    }
    load(r0 + kAhead * slots);
  }
}

template <typename T, int V, bool kInter>
static cudaError_t launch(const RotateArgs& a, cudaStream_t stream) {
  const int units = (a.head_dim + 2 * V - 1) / (2 * V);
  static_assert(KV_MAX_ROTATE_DIM / 2 <= 2 * kThreads, "a thread a unit");
  const int threads = units > kThreads ? 2 * kThreads : kThreads;
  const int per_block = rope_tokens_per_block(a.n_tokens, a.n_heads, units, threads, kMaxTokens);
  const int blocks = (a.n_tokens + per_block - 1) / per_block;
  return launch_pdl(rotate_kernel<T, V, kInter>, dim3(blocks), dim3(threads),
                    (size_t)per_block * units * V * sizeof(float2), stream, a, units, per_block);
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
