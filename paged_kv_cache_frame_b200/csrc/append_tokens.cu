// Appending tokens to a paged pool (kv_append_tokens): the keys rotated on the
// way, the values as they are, each row to the page and slot that the
// sequence's table gives for the token's index.
//
// Bound by its bytes. As in the rotation kernel a thread keeps one unit of V
// pairs of a token and goes through the heads with its angles; the values'
// packs 2u and 2u + 1 travel in the same thread. A warp finds the sequence of
// a token in cu_new with 32 probes at a time (two rounds for up to 1024
// sequences), once per token of the block.
#include "launch.cuh"
#include "rope_unit.cuh"

namespace pkv {

namespace {
constexpr int kThreads = 256;
constexpr int kAhead = 2;         // heads in flight per thread, keys and values
constexpr int kMaxTokens = 64;    // tokens a block takes

// Sequences s of [0, n) with cu[s + 1] <= t, all before the others: the
// sequence of token t (n where no sequence holds it). All lanes of a warp.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + (lane + 1) * step - 1;   // the last of the lane's stretch
    const bool below = probe < hi && __ldg(cu + probe + 1) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    lo = min(lo + k * step, hi);
    hi = min(lo + step - 1, hi);
  }
  return lo;
}
}  // namespace

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) append_tokens_kernel(const __grid_constant__ AppendTokensArgs a, int units,
                                                                 int head_slots) {
  __shared__ int s_row[kMaxTokens];   // pool row of the token's key, -1: not written
  __shared__ int s_pos[kMaxTokens];
  const int u = threadIdx.x % units;
  const int row = threadIdx.x / units;
  const int per_block = min(kMaxTokens, kThreads / units / head_slots);
  const int first = (int)blockIdx.x * per_block;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x / 32; i < per_block; i += kThreads / 32) {
    const int t = first + i;
    if (t >= a.n_tokens) break;
    int s = t, back = 1;   // the token is the back-th from the end of sequence s
    if (a.cu_new) {
      s = find_seq(a.cu_new, a.c.n_seqs, t);
      // Tokens behind the last sequence belong to none. A cu_new that does not
      // start at 0 or runs backwards can leave t outside of the sequence found.
      if (s < a.c.n_seqs) {
        back = __ldg(a.cu_new + s + 1) - t;
        if (t < __ldg(a.cu_new + s) || back < 1) {
          s = a.c.n_seqs;
          if (threadIdx.x % 32 == 0) raise_error(a.c.error);
        }
      }
    }
    int at = -1, pos = 0;
    if (s < a.c.n_seqs) {
      const int len = seq_len(a.c, s);
      const int j = len - back;
      bool bad = seq_len_bad(a.c, s);
      if (j >= 0) {
        at = token_row(a.c, s, j);
        bad |= at < 0;
      } else if (len > 0) {
        bad = true;   // more new tokens than the sequence holds (len 0: an unused row)
      }
      if (bad) {
        at = -1;
        if (threadIdx.x % 32 == 0) raise_error(a.c.error);
      }
      pos = a.positions ? __ldg(a.positions + t) : j;
    }
    if (threadIdx.x % 32 == 0) {
      s_row[i] = at;
      s_pos[i] = pos;
    }
  }
  __syncthreads();
  const int i = row / head_slots;
  const int t = first + i;
  if (i >= per_block || t >= a.n_tokens || s_row[i] < 0) return;
  RopeUnit<T, V, kInter> unit;
  unit.place(u, a.c.D, a.rope.rot);
  if (unit.turns) unit.angles(a.rope, u, s_pos[i], false);
  const T* k = static_cast<const T*>(a.k.p) + t * a.k.token_stride;
  const T* v = static_cast<const T*>(a.v.p) + t * a.v.token_stride;
  T* to = static_cast<T*>(a.c.pool) + row_offset(a.c, s_row[i], 0);
  const long long v_off = (long long)a.c.page_size * a.c.H * a.c.D;
  using P = Pack<T, V>;
  for (int h = row % head_slots; h < a.c.H; h += kAhead * head_slots) {
    P k0[kAhead], k1[kAhead], v0[kAhead], v1[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int g = h + n * head_slots;
      if (g < a.c.H) {
        const T* kp = k + g * a.k.head_stride;
        const T* vp = v + g * a.v.head_stride;
        k0[n] = *reinterpret_cast<const P*>(kp + unit.at0);
        k1[n] = *reinterpret_cast<const P*>(kp + unit.at1);
        v0[n] = *reinterpret_cast<const P*>(vp + 2 * u * V);
        v1[n] = *reinterpret_cast<const P*>(vp + 2 * u * V + V);
      }
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int g = h + n * head_slots;
      if (g < a.c.H) {
        if (unit.turns) {
          P y0, y1;
          unit.turn(k0[n], k1[n], u, a.rope.rot, y0, y1);
          k0[n] = y0;
          k1[n] = y1;
        }
        T* p = to + (long long)g * a.c.D;
        *reinterpret_cast<P*>(p + unit.at0) = k0[n];
        *reinterpret_cast<P*>(p + unit.at1) = k1[n];
        *reinterpret_cast<P*>(p + v_off + 2 * u * V) = v0[n];
        *reinterpret_cast<P*>(p + v_off + 2 * u * V + V) = v1[n];
      }
    }
  }
}

template <typename T, int V, bool kInter>
static cudaError_t launch(const AppendTokensArgs& a, cudaStream_t stream) {
  const int units = a.c.D / (2 * V);
  const int rows = kThreads / units;
  // As in the rotation: a token's heads over just enough threads to fill the
  // GPU.
  int slots = 1;
  while (2 * slots <= rows && slots < a.c.H && (long long)a.n_tokens * units * slots < 148 * 1024) slots *= 2;
  const int per_block = rows / slots < kMaxTokens ? rows / slots : kMaxTokens;
  const int blocks = (a.n_tokens + per_block - 1) / per_block;
  return launch_pdl(append_tokens_kernel<T, V, kInter>, dim3(blocks), dim3(kThreads), 0, stream, a, units, slots);
}

template <typename T>
static cudaError_t launch_typed(const AppendTokensArgs& a, cudaStream_t stream) {
  // Rows of the pool and of k and v are 16-byte aligned; only pairs (i,
  // i + rot / 2) with rot / 2 off the 8-value grid need single values.
  if (a.rope.interleaved) return launch<T, 8, true>(a, stream);
  return a.rope.rot % 16 == 0 ? launch<T, 8, false>(a, stream) : launch<T, 1, false>(a, stream);
}

cudaError_t launch_append_tokens(const AppendTokensArgs& a, int dtype, cudaStream_t stream) {
  if (a.n_tokens <= 0 || a.c.n_seqs <= 0) return cudaSuccess;
  return dtype == KV_FP16 ? launch_typed<__half>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace pkv
