// Attention of one new token per sequence over a paged pool (kv_decode), and
// the whole decode step (kv_decode_append): the query and the new key rotated,
// key and value written to the pool, then the attention.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,  j in [max(0, len - window), len)
//
// Bound by the bytes of K and V: each is read once for the whole group of
// query heads that shares it.
//
// Split. A unit is one (sequence, K/V head, group of at most `rows` query
// heads); its tokens are cut into tiles, all units' tiles stand in one line,
// and CTA c of G takes the c-th G-th of the line, whatever the sequences'
// lengths: no CTA waits for a long sequence. The lengths are read on the
// device, so a captured launch serves growing sequences. A unit that lies in
// one CTA is written to `out` by it; of the others every CTA leaves (max,
// sum, unnormalised O) in the workspace, and a second launch joins them in
// their order along the sequence, so results do not depend on timing.
//
// In a CTA each warp takes every kWarps-th step of kStep tokens and keeps a
// running max, sum and O of its own; no warp waits for another until the end
// of the unit. Token rows are gathered by 16-byte asynchronous copies into a
// ring per warp (rows past the end are zero-filled and masked, so what the
// pool holds there is never read).
//
// The products run transposed on mma.sync m16n8k16, the query heads on the
// N = 8 side: S^T = K Q^T (tokens x heads) and O^T += V^T P^T. K and V then
// fill the M = 16 side whatever the group's size, P moves from accumulator to
// operand layout by movmatrix, and a group of 8 costs one pass. At the
// measured 2 clk per mma and SM these take about a fifth of the time the
// bytes need. P is fed as a sum of two 16-bit values (its rounding and the
// rest): rounding P alone would add an error as large as the output's own.
#include <limits.h>

#include "launch.cuh"
#include "rope.cuh"
#include "sm100.cuh"
#include "token_access.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;

template <int D>
struct Shape {
  static constexpr int kM = D == 64 ? 2 : 1;            // 16-token blocks of a step
  static constexpr int kStep = 16 * kM;                 // tokens a warp takes at a time (8 KB of K and V)
  static constexpr int kTileTokens = kStep * kWarps;    // tokens of a tile of the split
  static constexpr int kStages = 3;
  static constexpr int kHalf = kStep * D * 2;           // K (or V) bytes of a stage
  static constexpr int kRing = kWarps * kStages * 2 * kHalf;
  static constexpr int kChunks = D / 8;                 // 16-byte chunks of a row
};

// (a, b) as packed 16-bit values and the packed remainders.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2<T>(a, b);
  const float2 h = unpack2<T>(hi);
  lo = pack2<T>(a - h.x, b - h.y);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;   // 0: the 16 bytes are zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// First token and number of tokens that sequence s's query sees.
__device__ __forceinline__ void span(const DecodeArgs& a, int s, int& first, int& len) {
  len = seq_len(a.c, s);
  first = a.window > 0 && len > a.window ? len - a.window : 0;
}
template <int kTileTokens>
__device__ __forceinline__ int seq_tiles(const DecodeArgs& a, int s) {
  int first, len;
  span(a, s, first, len);
  return (int)(((long long)(len - first) + kTileTokens - 1) / kTileTokens);
}

// Sum of v over the block (kThreads threads), and the inclusive sum up to the
// calling thread.
__device__ __forceinline__ long long block_scan(long long v, long long* scratch, long long& total) {
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) scratch[w] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) v += scratch[i];
    total += scratch[i];
  }
  __syncthreads();
  return v;
}

template <typename T, int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPad = D + 4;    // floats of a row of the warps' O: no two lanes in one bank
  static constexpr int kOffMl = kWarps * kRows * kPad * 4;            // within the ring: [warp][row][2]
  static constexpr int kOffQ = Shape<D>::kRing;                       // fused: rotated queries [rows][D] fp32
  static constexpr int kOffNew = kOffQ + kRows * D * 4;               // fused: new key and value [2][D]
  static constexpr int kFused = kOffNew + 2 * D * 2;
  static_assert(kOffMl + kWarps * kRows * 8 <= Shape<D>::kRing, "the warps' results fit the ring");
};

// Pair p (of D / 2) of a head in the rotation's order: its two elements, and
// whether they are rotated.
__device__ __forceinline__ bool rope_pair(const RopeTable& t, int p, int& e0, int& e1) {
  const bool on = p < t.rot / 2;
  if (t.interleaved || !on) {
    e0 = 2 * p;
    e1 = e0 + 1;
  } else {
    e0 = p;
    e1 = p + t.rot / 2;
  }
  return on;
}

}  // namespace

template <int D, typename T, int NT, bool kFused>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const __grid_constant__ DecodeArgs a) {
  using S = Shape<D>;
  using M = Smem<T, D, NT>;
  constexpr int kRows = M::kRows;
  constexpr bool kFP16 = kIsFp16<T>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_scan[kWarps];
  __shared__ long long s_base;
  __shared__ int s_seq;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int units = a.c.H * a.head_groups;   // of a sequence

  pdl_wait();      // the pool, the tables and the queries may come from earlier kernels
  pdl_trigger();

  // The line's length, and where this CTA's part starts.
  long long total = 0, mine = 0;
  bool bad = false;
  for (int s = tid; s < a.c.n_seqs; s += kThreads) {
    mine += (long long)seq_tiles<S::kTileTokens>(a, s) * units;
    bad |= seq_len_bad(a.c, s);
  }
  if (bad) raise_error(a.c.error);
  block_scan(mine, s_scan, total);
  T* out = static_cast<T*>(a.out);
  const int q_heads = a.c.H * a.group;
  for (int s = blockIdx.x; s < a.c.n_seqs; s += gridDim.x)   // sequences with nothing to see
    if (seq_len(a.c, s) == 0)
      for (int i = tid; i < q_heads * D; i += kThreads) out[(long long)s * q_heads * D + i] = from_f32<T>(0.f);
  const long long parts = total < a.grid ? total : a.grid;
  if (blockIdx.x >= parts) {
    if (tid == 0) a.part_meta[4 * blockIdx.x] = 0;
    return;
  }
  const long long start = blockIdx.x * total / parts, end = (blockIdx.x + 1) * total / parts;
  if (tid == 0) s_seq = a.c.n_seqs;
  long long before = 0;
  for (int s0 = 0; s0 < a.c.n_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    const long long n = s < a.c.n_seqs ? (long long)seq_tiles<S::kTileTokens>(a, s) * units : 0;
    long long sum;
    const long long upto = before + block_scan(n, s_scan, sum);
    if (n > 0 && start < upto && start >= upto - n) {
      s_seq = s;
      s_base = upto - n;
    }
    before += sum;
    if (before > start) break;
  }
  __syncthreads();
  int seq = s_seq;
  long long seq_base = s_base;

  uint8_t* ring = smem + warp * (S::kStages * 2 * S::kHalf);
  const uint32_t ring_u = smem_u32(ring);
  const T* pool = static_cast<const T*>(a.c.pool);
  const long long v_off = (long long)a.c.page_size * a.c.H * D;
  int starts_unit = 0;   // pieces of the unit that begins in this CTA and ends in a later one

  for (long long t = start; t < end && seq < a.c.n_seqs;) {
    int first, len;
    span(a, seq, first, len);
    const int tiles = seq_tiles<S::kTileTokens>(a, seq);
    if (tiles == 0) break;   // cannot be, unless the lengths change under the launch
    const int unit = (int)((t - seq_base) / tiles);
    const int tile0 = (int)((t - seq_base) % tiles);
    const int tile1 = (int)(tiles - tile0 < end - t ? tiles : tile0 + (end - t));
    const int h = unit / a.head_groups;
    const int head0 = unit % a.head_groups * kRows;                       // within the K/V head's group
    const int heads = a.group - head0 < kRows ? a.group - head0 : kRows;
    const int q0 = h * a.group + head0;
    const int tok0 = first + tile0 * S::kTileTokens;
    // tokens fit 31 bits; a tile past the end would not
    const int tok1 = tile1 == tiles ? len : first + tile1 * S::kTileTokens;
    const T* q = static_cast<const T*>(a.q.p) + seq * a.q.token_stride + q0 * a.q.head_stride;

    // The new token's row, where this piece holds it.
    const bool has_new = kFused && tile1 == tiles;
    bool new_ok = false;
    if (kFused) {
      float* sq = reinterpret_cast<float*>(smem + M::kOffQ);
      T* sn = reinterpret_cast<T*>(smem + M::kOffNew);
      const int pos = a.positions ? __ldg(a.positions + seq) : len - 1;
      int e0, e1;
      const int p = tid % (D / 2);
      const bool on = rope_pair(a.rope, p, e0, e1);
      float c = 1.f, s = 0.f;
      if (on) rope_angle(a.rope.turn[p], pos, a.rope.amplitude, c, s);
      for (int i = tid / (D / 2); i < kRows; i += kThreads / (D / 2)) {
        float x = 0.f, y = 0.f;
        if (i < heads) {
          x = to_f32(q[i * a.q.head_stride + e0]);
          y = to_f32(q[i * a.q.head_stride + e1]);
          if (on) rope_turn(x, y, c, s);
        }
        sq[i * D + e0] = x;
        sq[i * D + e1] = y;
      }
      if (has_new) {
        const int row = token_row(a.c, seq, len - 1);
        new_ok = row >= 0;
        if (!new_ok && tid == 0) raise_error(a.c.error);
        T* to = static_cast<T*>(a.c.pool) + row_offset(a.c, new_ok ? row : 0, h);
        const bool write = new_ok && head0 == 0;   // one of the head's groups writes it
        if (tid < D / 2) {
          const T* k = static_cast<const T*>(a.k.p) + seq * a.k.token_stride + h * a.k.head_stride;
          T kx = k[e0], ky = k[e1];
          if (on) {
            float x = to_f32(kx), y = to_f32(ky);
            rope_turn(x, y, c, s);
            kx = from_f32<T>(x);   // the cache's type: attended to as later tokens will read it
            ky = from_f32<T>(y);
          }
          sn[e0] = kx;
          sn[e1] = ky;
          if (write) {
            to[e0] = kx;
            to[e1] = ky;
          }
        }
        const T* v = static_cast<const T*>(a.v.p) + seq * a.v.token_stride + h * a.v.head_stride;
        for (int i = tid; i < D; i += kThreads) {
          const T x = v[i];
          sn[D + i] = x;
          if (write) to[v_off + i] = x;
        }
      }
      __syncthreads();
    }

    // Step i of this warp: tokens [base(i), base(i) + kStep). `valid` has bit
    // r set where row r is a token to attend to.
    const int warp0 = tok0 + warp * S::kStep;
    const int n_steps = warp0 < tok1 ? (tok1 - warp0 + S::kTileTokens - 1) / S::kTileTokens : 0;
    auto issue = [&](int i) -> uint32_t {
      if (i >= n_steps) return 0;
      const int base = warp0 + i * S::kTileTokens;
      int row = -1;
      bool ok = false;
      if (lane < S::kStep && lane < tok1 - base) {
        const int j = base + lane;
        if (has_new && j == len - 1) {
          ok = new_ok;   // comes from shared memory
        } else {
          row = token_row(a.c, seq, j);
          ok = row >= 0;
          if (!ok) raise_error(a.c.error);
        }
      }
      const uint32_t valid = __ballot_sync(0xffffffffu, ok);
      constexpr int kPerPass = 32 / S::kChunks;   // rows of a pass
      const int chunk = lane % S::kChunks;
      const uint32_t dst0 = ring_u + (i % S::kStages) * (2 * S::kHalf);
#pragma unroll
      for (int r0 = 0; r0 < S::kStep; r0 += kPerPass) {
        const int r = r0 + lane / S::kChunks;
        const int from = __shfl_sync(0xffffffffu, row, r);
        const T* src = pool + row_offset(a.c, from < 0 ? 0 : from, h) + chunk * 8;
        const uint32_t dst = dst0 + r * (D * 2) + ((chunk ^ (r & 7)) << 4);
        cp_async16(dst, src, from >= 0);
        cp_async16(dst + S::kHalf, src + v_off, from >= 0);
      }
      return valid;
    };

    uint32_t valid[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      valid[i] = issue(i);
      cp_async_commit();
    }

    // Queries as B operands: heads lane / 4 of each block of 8, values
    // 16 k + (lane % 4) * 2 and the next, and those 8 further.
    uint32_t qb[NT][D / 16][2], qlo[NT][kFused ? D / 16 : 1][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = n * 8 + lane / 4, d = k * 16 + e * 8 + lane % 4 * 2;
          if (kFused) {
            const float2 x = *reinterpret_cast<const float2*>(smem + M::kOffQ + (i * D + d) * 4);
            split2<T>(x.x, x.y, qb[n][k][e], qlo[n][k][e]);   // the rotated query is not rounded
          } else {
            qb[n][k][e] = i < heads ? *reinterpret_cast<const uint32_t*>(q + i * a.q.head_stride + d) : 0u;
          }
        }

    float o[NT][D / 16][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

    for (int i = 0; i < n_steps; ++i) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      valid[S::kStages - 1] = issue(i + S::kStages - 1);
      cp_async_commit();
      const uint32_t on = valid[0];
#pragma unroll
      for (int k = 0; k < S::kStages - 1; ++k) valid[k] = valid[k + 1];
      const uint32_t ks = ring_u + (i % S::kStages) * (2 * S::kHalf), vs = ks + S::kHalf;
      if (kFused && has_new) {
        const int r = len - 1 - (warp0 + i * S::kTileTokens);
        if (r >= 0 && r < S::kStep) {
          if (lane < 2 * S::kChunks) {
            const int chunk = lane % S::kChunks;
            const uint4 x = reinterpret_cast<const uint4*>(smem + M::kOffNew)[lane];
            *reinterpret_cast<uint4*>(ring + (i % S::kStages) * (2 * S::kHalf) + (lane / S::kChunks) * S::kHalf +
                                      r * (D * 2) + ((chunk ^ (r & 7)) << 4)) = x;
          }
          __syncwarp();
        }
      }

      // S^T: rows are tokens lane / 4 and lane / 4 + 8 of each block, columns
      // heads (lane % 4) * 2 and the next.
      float sc[S::kM][NT][4];
#pragma unroll
      for (int b = 0; b < S::kM; ++b) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[b][n][0] = sc[b][n][1] = sc[b][n][2] = sc[b][n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t x[4];
          const int r = b * 16 + lane % 16;
          ldsm_x4(ks + r * (D * 2) + (((2 * k + lane / 16) ^ (r & 7)) << 4), x);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816<kFP16>(sc[b][n], x, qb[n][k][0], qb[n][k][1]);
            if (kFused) mma_16816<kFP16>(sc[b][n], x, qlo[n][k][0], qlo[n][k][1]);
          }
        }
      }
      constexpr uint32_t kAll = S::kStep == 32 ? 0xffffffffu : (1u << S::kStep % 32) - 1;
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
        for (int b = 0; b < S::kM; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = b * 16 + lane / 4 + (e >> 1) * 8;
            const float x = sc[b][n][e] * a.scale_log2;
            sc[b][n][e] = on == kAll || (on >> r & 1) ? x : -INFINITY;
            top[n][e & 1] = fmaxf(top[n][e & 1], sc[b][n][e]);
          }
      }
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = top[n][c];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          top[n][c] = fmaxf(x, m[n][c]);
          grew |= top[n][c] > m[n][c];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = top[n][c] > m[n][c] ? ex2_approx(m[n][c] - top[n][c]) : 1.f;   // 0 from -inf
            m[n][c] = top[n][c];
            l[n][c] *= f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              o[n][k][c] *= f;
              o[n][k][c + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int b = 0; b < S::kM; ++b) {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];   // nothing valid so far: every p is 0
          const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = ex2_approx(sc[b][n][2 * e] - m0), p1 = ex2_approx(sc[b][n][2 * e + 1] - m1);
            l[n][0] += p0;
            l[n][1] += p1;
            uint32_t hi, lo;
            split2<T>(p0, p1, hi, lo);
            ph[n][e] = movmatrix_t(hi);
            pl[n][e] = movmatrix_t(lo);
          }
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t x[4];
          const int r = b * 16 + lane % 8 + lane / 16 * 8;
          ldsm_x4_t(vs + r * (D * 2) + (((2 * k + (lane / 8 & 1)) ^ (r & 7)) << 4), x);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816<kFP16>(o[n][k], x, ph[n][0], ph[n][1]);
            mma_16816<kFP16>(o[n][k], x, pl[n][0], pl[n][1]);
          }
        }
      }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);

    // Join the warps in shared memory.
    __syncthreads();   // every ring is drained
    float* wo = reinterpret_cast<float*>(smem);
    float* wml = reinterpret_cast<float*>(smem + M::kOffMl);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int i = warp * kRows + n * 8 + lane % 4 * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          wo[(i + (e & 1)) * M::kPad + k * 16 + lane / 4 + (e >> 1) * 8] = o[n][k][e];
      if (lane < 4) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          wml[2 * (i + c)] = m[n][c];
          wml[2 * (i + c) + 1] = l[n][c];
        }
      }
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == tiles;
    const bool opens = tile0 == 0 && !whole;
    const long long slot = 2 * blockIdx.x + (opens ? 1 : 0);
    for (int x = tid; x < heads * (D / 2); x += kThreads) {
      const int i = x / (D / 2), d = x % (D / 2) * 2;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wml[2 * (w * kRows + i)]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(wml[2 * (w * kRows + i)] - ref);
        const float2 y = *reinterpret_cast<const float2*>(wo + (w * kRows + i) * M::kPad + d);
        sum = fmaf(f, wml[2 * (w * kRows + i) + 1], sum);
        a0 = fmaf(f, y.x, a0);
        a1 = fmaf(f, y.y, a1);
      }
      if (whole) {
        const float r = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // no page of the table was valid: zeros
        *reinterpret_cast<uint32_t*>(out + ((long long)seq * q_heads + q0 + i) * D + d) = pack2<T>(a0 * r, a1 * r);
      } else {
        *reinterpret_cast<float2*>(a.part_o + (slot * kRows + i) * D + d) = make_float2(a0, a1);
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * kRows + i) * 2) = make_float2(top, sum);
      }
    }
    if (opens) {
      const long long last = seq_base + (long long)(unit + 1) * tiles - 1;   // the unit's last tile, and its CTA
      starts_unit = (int)(((last + 1) * parts - 1) / total) - blockIdx.x + 1;
      if (tid == 0) {
        a.part_meta[4 * blockIdx.x + 1] = seq;
        a.part_meta[4 * blockIdx.x + 2] = q0;
        a.part_meta[4 * blockIdx.x + 3] = heads;
      }
    }
    __syncthreads();   // the ring may be filled again
    t += tile1 - tile0;
    if (t >= seq_base + (long long)tiles * units && t < end) {
      seq_base += (long long)tiles * units;
      do ++seq;
      while (seq < a.c.n_seqs && seq_tiles<S::kTileTokens>(a, seq) == 0);
    }
  }
  if (tid == 0) a.part_meta[4 * blockIdx.x] = starts_unit;
}

// Joins the parts of the unit that CTA blockIdx.x of the attention launch
// began and a later one ended: O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,
// in the order of the parts. One query head per blockIdx.y; the warps take
// every kWarps-th part.
template <int D, typename T, int kRows>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int V = D / 32;
  __shared__ float s_o[kWarps][D];
  __shared__ float s_l[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const int4 meta = *reinterpret_cast<const int4*>(a.part_meta + 4 * c);   // parts, sequence, first head, heads
  const int n = meta.x, i = blockIdx.y;
  if (n == 0 || i >= meta.w) return;
  auto slot = [&](int p) { return (2LL * (c + p) + (p == 0 ? 1 : 0)) * kRows + i; };
  float top = -INFINITY;
  for (int p = lane; p < n; p += 32) top = fmaxf(top, a.part_ml[2 * slot(p)]);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (top == -INFINITY) top = 0.f;
  float acc[V] = {}, sum = 0.f;
#pragma unroll 4
  for (int p = warp; p < n; p += kWarps) {
    const long long s = slot(p);
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * s);
    const Pack<float, V> x = *reinterpret_cast<const Pack<float, V>*>(a.part_o + s * D + lane * V);
    const float f = ex2_approx(ml.x - top);
    sum = fmaf(f, ml.y, sum);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = fmaf(f, x.get(e), acc[e]);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
  if (lane == 0) s_l[warp] = sum;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  float y = 0.f;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    y += s_o[w][d];
    sum += s_l[w];
  }
  const float r = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  const int q_heads = a.c.H * a.group;
  static_cast<T*>(a.out)[((long long)meta.y * q_heads + meta.z + i) * D + d] = from_f32<T>(y * r);
}

int decode_rows(int group) { return group <= 8 ? 8 : 16; }

int decode_grid(int D, int group, int num_sms) {
  (void)D;
  (void)group;
  return num_sms * kCtasPerSm;
}

template <int D, typename T, int NT, bool kFused>
static cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  using M = Smem<T, D, NT>;
  static std::atomic<uint8_t> done[kMaxDevices];
  const int bytes = kFused ? M::kFused : Shape<D>::kRing;
  cudaError_t e = ensure_dynamic_smem(decode_kernel<D, T, NT, kFused>, bytes, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_kernel<D, T, NT, kFused>, dim3(a.grid), dim3(kThreads), bytes, stream, a);
  if (e != cudaSuccess) return e;
  const int heads = a.group < M::kRows ? a.group : M::kRows;
  return launch_pdl(decode_join_kernel<D, T, M::kRows>, dim3(a.grid, heads), dim3(kThreads), 0, stream, a);
}

template <int D, typename T>
static cudaError_t launch_shape(const DecodeArgs& a, bool fused, cudaStream_t stream) {
  if (decode_rows(a.group) == 8) return fused ? launch<D, T, 1, true>(a, stream) : launch<D, T, 1, false>(a, stream);
  return fused ? launch<D, T, 2, true>(a, stream) : launch<D, T, 2, false>(a, stream);
}

cudaError_t launch_decode(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream) {
  if (a.c.n_seqs <= 0) return cudaSuccess;
  if (a.c.D == 64)
    return dtype == KV_FP16 ? launch_shape<64, __half>(a, fused, stream)
                            : launch_shape<64, __nv_bfloat16>(a, fused, stream);
  return dtype == KV_FP16 ? launch_shape<128, __half>(a, fused, stream)
                          : launch_shape<128, __nv_bfloat16>(a, fused, stream);
}

}  // namespace pkv
