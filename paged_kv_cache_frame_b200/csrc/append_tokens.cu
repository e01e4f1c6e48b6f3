// Appending tokens to a paged pool (kv_append_tokens): the keys rotated on the
// way, the values as they are, each row to the page and slot that the
// sequence's table gives for the token's index.
//
// Bound by its bytes. As in the rotation kernel a block takes a few tokens
// with all of their heads, and its threads go through the (token, head) rows,
// each at its own unit of V pairs; the values' packs 2u and 2u + 1 travel in
// the same thread. A warp finds the sequence of a token in cu_new with 32
// probes at a time (two rounds for up to 1024 sequences) while the first rows
// are on their way.
#include "launch.cuh"
#include "rope_unit.cuh"

namespace pkv {

namespace {
constexpr int kThreads = 256;
constexpr int kAhead = 2;         // rows in flight per thread, keys and values
constexpr int kMaxTokens = 8;     // tokens of a block: one per warp for the search

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
__global__ void __launch_bounds__(kThreads, 4) append_tokens_kernel(const __grid_constant__ AppendTokensArgs a, int units,
                                                                 int per_block) {
  extern __shared__ __align__(16) float2 s_angle[];
  __shared__ int s_row[kMaxTokens];   // pool row of the token's key, -1: not written
  const int u = threadIdx.x % units;
  const int slot = threadIdx.x / units, slots = kThreads / units;
  const int first = (int)blockIdx.x * per_block;
  const int tokens = min(per_block, a.n_tokens - first);
  const int rows = tokens * a.c.H;
  const RopeUnit<T, V, kInter> unit(u, a.c.D, a.rope.rot);
  pdl_wait();
  pdl_trigger();
  using P = Pack<T, V>;
  P k0[kAhead], k1[kAhead], v0[kAhead], v1[kAhead];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * slots;
      if (slot < slots && r < rows) {
        const int t = divided(r, a.head_mul, a.head_shift), h = r - t * a.c.H;
        const T* k = static_cast<const T*>(a.k.p) + (first + t) * a.k.token_stride + h * a.k.head_stride;
        const T* v = static_cast<const T*>(a.v.p) + (first + t) * a.v.token_stride + h * a.v.head_stride;
        k0[i] = *reinterpret_cast<const P*>(k + unit.at0);
        k1[i] = *reinterpret_cast<const P*>(k + unit.at1);
        v0[i] = *reinterpret_cast<const P*>(v + 2 * u * V);
        v1[i] = *reinterpret_cast<const P*>(v + 2 * u * V + V);
      }
    }
  };
  load(slot);   // on their way while places and angles are worked out
  // A warp a token: its row, then its angles.
  const int lane = threadIdx.x % 32;
  for (int i = threadIdx.x / 32; i < tokens; i += kThreads / 32) {
    const int t = first + i;
    int s = t, back = 1;   // the token is the back-th from the end of sequence s
    if (a.cu_new) {
      s = find_seq(a.cu_new, a.c.n_seqs, t);
      // Tokens behind the last sequence belong to none. A cu_new that does not
      // start at 0 or runs backwards can leave t outside of the sequence found.
      if (s < a.c.n_seqs) {
        back = __ldg(a.cu_new + s + 1) - t;
        if (t < __ldg(a.cu_new + s) || back < 1) {
          s = a.c.n_seqs;
          if (lane == 0) raise_error(a.c.error, kErrIndex);
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
        if (lane == 0) raise_error(a.c.error, kErrIndex);
      }
      pos = a.positions ? __ldg(a.positions + t) : j;
    }
    if (lane == 0) s_row[i] = at;
    for (int p = lane; p < a.rope.rot / 2; p += 32) {
      float c, sn;
      rope_angle(a.rope.turn[p], pos, a.rope.amplitude, c, sn);
      s_angle[angle_at<V>(units, i, p)] = make_float2(c, sn);
    }
  }
  __syncthreads();
  const long long v_off = (long long)a.c.page_size * a.c.H * a.c.D;
  for (int r0 = slot; r0 < rows; r0 += kAhead * slots) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * slots;
      if (slot < slots && r < rows) {
        const int t = divided(r, a.head_mul, a.head_shift), h = r - t * a.c.H;
        const int row = s_row[t];
        if (row >= 0) {
          if (unit.turns) unit.turn(k0[i], k1[i], s_angle, units, t, a.rope.rot);
          T* p = static_cast<T*>(a.c.pool) + row_offset(a.c, row, h);
          *reinterpret_cast<P*>(p + unit.at0) = k0[i];
          *reinterpret_cast<P*>(p + unit.at1) = k1[i];
          *reinterpret_cast<P*>(p + v_off + 2 * u * V) = v0[i];
          *reinterpret_cast<P*>(p + v_off + 2 * u * V + V) = v1[i];
        }
      }
    }
    load(r0 + kAhead * slots);
  }
}

template <typename T, int V, bool kInter>
static cudaError_t launch(const AppendTokensArgs& a, cudaStream_t stream) {
  const int units = a.c.D / (2 * V);
  const int per_block = rope_tokens_per_block(a.n_tokens, a.c.H, units, kThreads, kMaxTokens);
  const int blocks = (a.n_tokens + per_block - 1) / per_block;
  return launch_pdl(append_tokens_kernel<T, V, kInter>, dim3(blocks), dim3(kThreads),
                    (size_t)per_block * units * V * sizeof(float2), stream, a, units, per_block);
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
