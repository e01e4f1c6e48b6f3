// Appending tokens to a paged pool (kv_append_tokens): the keys rotated on the
// way, the values as they are, each row to the page and slot that the
// sequence's table gives for the token's index.
//
// Bound by its bytes and, short of some ten thousand tokens, by the chain of
// loads before a row's place is known. As in the rotation kernel a block takes
// a few tokens with all of their heads, and its threads go through the
// (token, head) rows, each at its own unit of V pairs; the values' packs 2u
// and 2u + 1 travel in the same thread. The first rows are on their way
// meanwhile; cu_new and the lengths are fetched together into shared memory,
// a thread a token searches there, and only its page is another load. Blocks
// are made large enough for all of them to run at once. Prompts of 9 sequences
// (6930 tokens x 8 heads x 128, 57 MB, nothing in cache): 14.3 us, of which
// the bytes need 8.7; with half as large blocks 15.5, with the search in
// global memory 17.4; value by value (120 of the 128 rotated) 30. One token of
// 64 sequences: 2.8 us, a launch.
#include "launch.cuh"
#include "rope_unit.cuh"

namespace pkv {

namespace {
constexpr int kThreads = 128;
constexpr int kCtasPerSm = 8;
constexpr int kAhead = 2;         // rows in flight per thread, keys and values
constexpr int kMaxTokens = 16;    // tokens of a block
constexpr int kMaxSeqs = 1024;    // sequences whose cu_new and lengths are kept in shared memory
}  // namespace

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_tokens_kernel(const __grid_constant__ AppendTokensArgs a, int units,
                                                                 int per_block) {
  extern __shared__ __align__(16) float2 s_angle[];
  __shared__ int s_row[kMaxTokens];   // pool row of the token's key, -1: not written
  __shared__ int s_pos[kMaxTokens];
  __shared__ int s_cu[kMaxSeqs + 1], s_len[kMaxSeqs];
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
  const int n = a.c.n_seqs;
  const bool kept = a.cu_new && n <= kMaxSeqs;
  if (kept) {
    for (int i = threadIdx.x; i <= n; i += kThreads) {
      s_cu[i] = __ldg(a.cu_new + i);
      if (i < n) s_len[i] = __ldg(a.c.lens + i);
    }
    __syncthreads();
  }
  int j = -1, page = -1;   // of the thread's token: its index in its sequence (-1: not written), and that page
  if (threadIdx.x < tokens) {
    const int i = threadIdx.x, t = first + i;
    const int32_t* cu = kept ? s_cu : a.cu_new;
    if (cu && t == 0 && cu[n] > a.n_tokens) raise_error(a.c.error, kErrIndex);   // tokens that the call does not bring
    int s = t, back = 1;   // the token is the back-th from the end of sequence s
    if (cu) {
      s = find_seq(cu, n, t);
      // Tokens behind the last sequence belong to none. A cu_new that does not
      // start at 0 or runs backwards can leave t outside of the sequence found.
      if (s < n) {
        back = cu[s + 1] - t;
        if (t < cu[s] || back < 1) {
          s = n;
          raise_error(a.c.error, kErrIndex);
        }
      }
    }
    int pos = 0;
    if (s < n) {
      const int raw = kept ? s_len[s] : __ldg(a.c.lens + s), len = held(a.c, raw);
      j = len - back;
      pos = a.positions ? __ldg(a.positions + t) : j;
      if (raw != len || (j < 0 && len > 0)) {   // more new tokens than the sequence holds (len 0: an unused row)
        raise_error(a.c.error, kErrIndex);
        j = -1;
      }
      if (j >= 0) page = __ldg(a.c.tables + s * a.c.table_stride + page_of(a.c, j));
    }
    s_pos[i] = pos;
  }
  __syncthreads();
  // The angles, while the pages are on their way.
  const int pairs = a.rope.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = divided(i, a.pair_mul, a.pair_shift), p = i - t * pairs;
    float c, sn;
    rope_angle(a.rope.turn[p], s_pos[t], a.rope.amplitude, c, sn);
    s_angle[angle_at<V>(units, t, p)] = make_float2(c, sn);
  }
  if (threadIdx.x < tokens) {
    const int at = j >= 0 ? row_in(a.c, page, j) : -1;
    if (j >= 0 && at < 0) raise_error(a.c.error, kErrIndex);
    s_row[threadIdx.x] = at;
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
  int per_block = (a.n_tokens + kSms * kCtasPerSm - 1) / (kSms * kCtasPerSm);   // all blocks at once
  if (per_block > kMaxTokens) per_block = kMaxTokens;
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
