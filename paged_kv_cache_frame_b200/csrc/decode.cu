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
// sum, unnormalised O) in the workspace, and the CTA that arrives last joins
// them, in their order along the sequence whichever CTA that is: results do
// not depend on timing, and no CTA waits for another. More than kJoin parts
// are joined in two rounds, kGroup neighbours first.
//
// In a CTA each warp takes every kWarps-th step of kStep tokens and keeps a
// running max, sum and O of its own; no warp waits for another until the end
// of the unit. Token rows are gathered by 16-byte asynchronous copies into a
// ring per warp (rows past the end are zero-filled and masked, so what the
// pool holds there is never read). The ring runs on into the CTA's next unit
// while the warps of this one are joined.
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
constexpr int kJoin = 32;    // parts that one CTA joins at once (a lane each)
constexpr int kGroup = 16;   // parts joined in a first round where there are more

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

// Shared memory behind the rings. The rotated queries of a unit and the
// join's weights and sums take the place of the warps' O: never at once.
template <int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kOffO = Shape<D>::kRing;                        // [warp][8 heads][D] fp32, one block of 8 at a time
  static constexpr int kOffMl = kOffO + kWarps * 8 * D * 4;            // [warp][8 heads] (max, sum)
  static constexpr int kOffNew = kOffMl + kWarps * 8 * 8;              // fused: new key and value [2][D]
  static constexpr int kBytes = kOffNew + 2 * D * 2;
  static_assert(kRows * D * 4 <= kWarps * 8 * D * 4, "the queries fit the warps' O");
};

// Element d of row i of a warp's O block: row i shifted by 4 i floats, so
// that no two lanes of an accumulator's store share a bank.
template <int D>
__device__ __forceinline__ int o_at(int w, int i, int d) {
  return (w * 8 + i) * D + ((d + 4 * i) & (D - 1));
}

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

// A CTA's part of the line.
struct Line {
  long long t, end;   // tiles [t, end) of the line are left
  long long base;     // the line's index of sequence seq's first tile
  int seq;
};

// The tiles of one unit that the CTA takes.
struct Piece {
  int seq, first, len;      // tokens [first, len) are seen
  int unit, tiles;          // the unit in its sequence, and its tiles
  int tile0, tile1;
  long long unit_base;      // the line's index of its first tile
};

template <int kTileTokens>
__device__ __forceinline__ bool next_piece(const DecodeArgs& a, int units, Line& l, Piece& p) {
  if (l.t >= l.end) return false;
  for (; l.seq < a.c.n_seqs; ++l.seq) {
    p.tiles = seq_tiles<kTileTokens>(a, l.seq);
    const long long n = (long long)p.tiles * units;
    if (l.t < l.base + n) break;
    l.base += n;
  }
  if (l.seq >= a.c.n_seqs) return false;   // cannot be, unless the lengths change under the launch
  p.seq = l.seq;
  span(a, l.seq, p.first, p.len);
  p.unit = (int)((l.t - l.base) / p.tiles);
  p.unit_base = l.base + (long long)p.unit * p.tiles;
  p.tile0 = (int)(l.t - p.unit_base);
  p.tile1 = (int)(p.tiles - p.tile0 < l.end - l.t ? p.tiles : p.tile0 + (l.end - l.t));
  l.t += p.tile1 - p.tile0;
  return true;
}

// A part of a unit: CTA c0 + p's, in that CTA's second slot if it opened the
// unit, else in its first.
__device__ __forceinline__ long long part_slot(int c0, int p) { return 2LL * (c0 + p) + (p == 0 ? 1 : 0); }

// Adds one to a counter; the arrival that completes `of` sets it back to zero
// and returns true, with the others' writes visible. Called by one thread
// after a barrier behind the CTA's writes.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, int of) {
  fence_acq_rel_gpu();
  const bool last = atomicAdd(counter, 1u) == (uint32_t)(of - 1);
  if (last) {
    atomicExch(counter, 0u);
    fence_acq_rel_gpu();
  }
  return last;
}

// Joins parts p0, p0 + step, ... (n of at most 32) of the unit begun by CTA
// c0: O = sum_i 2^(m_i - M) O_i, l = sum_i 2^(m_i - M) l_i. The last round
// writes O / l to `out` (the unit's first query row), others the part in the
// first one's place. A lane per part works the weights out; the rows' 16-byte
// pieces are spread over the threads, several lanes of parts to a piece where
// there are threads to spare.
template <int D, typename T, int kRows>
__device__ __forceinline__ void join_parts(const DecodeArgs& a, float* smem, int c0, int p0, int step, int n, int heads,
                                           T* out) {
  constexpr int kPieces = D / 4;   // of a row
  constexpr int kPre = 8;          // parts requested before the weights are known
  float* s_f = smem;                                        // [part][row]
  float* s_l = s_f + 32 * kRows;                            // [row] sum
  float* s_m = s_l + kRows;                                 // [row] max
  float4* s_o = reinterpret_cast<float4*>(s_m + kRows);     // [lane of parts][piece]
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int items = heads * kPieces;
  const int lanes = items < kThreads ? kThreads / items : 1;
  const int r = lanes > 1 ? tid / items : 0;
  const int it0 = lanes > 1 ? tid % items : tid;
  auto row = [&](int p, int it) {
    return reinterpret_cast<const float4*>(a.part_o + part_slot(c0, p0 + p * step) * kRows * D) + it;
  };
  float4 pre[kPre];
#pragma unroll
  for (int k = 0; k < kPre; ++k) {
    const int p = r + k * lanes;
    pre[k] = r < lanes && it0 < items && p < n ? __ldcg(row(p, it0)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i = warp; i < heads; i += kWarps) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (part_slot(c0, p0 + lane * step) * kRows + i) * 2));
    float top = ml.x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = ex2_approx(ml.x - (top == -INFINITY ? 0.f : top));
    float sum = f * ml.y;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    s_f[lane * kRows + i] = f;
    if (lane == 0) {
      s_l[i] = sum;
      s_m[i] = top;
    }
  }
  __syncthreads();
  for (int it = it0; it < items; it += kThreads) {
    const int i = it / kPieces;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& x, int p) {
      const float f = s_f[p * kRows + i];
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    };
    if (r < lanes) {
      for (int p = r; p < n; p += kPre * lanes) {
        float4 x[kPre];
#pragma unroll
        for (int k = 0; k < kPre; ++k)
          if (p + k * lanes < n) x[k] = it == it0 && p == r ? pre[k] : __ldcg(row(p + k * lanes, it));
#pragma unroll
        for (int k = 0; k < kPre; ++k)
          if (p + k * lanes < n) add(x[k], p + k * lanes);
      }
    }
    if (lanes > 1) {   // uniform: every thread is here once
      s_o[tid] = acc;
      __syncthreads();
      if (r == 0) {
        for (int k = 1; k < lanes; ++k) {
          const float4 x = s_o[k * items + it];
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
        }
      }
    }
    if (r != 0) continue;
    if (out) {
      const float sum = s_l[i];
      const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // no page was valid: zeros
      *reinterpret_cast<uint2*>(out + it * 4) =
          make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    } else {
      *const_cast<float4*>(row(0, it)) = acc;
      if (it % kPieces == 0)
        *reinterpret_cast<float2*>(a.part_ml + (part_slot(c0, p0) * kRows + i) * 2) = make_float2(s_m[i], s_l[i]);
    }
  }
}

}  // namespace

template <int D, typename T, int NT, bool kFused>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const __grid_constant__ DecodeArgs a) {
  using S = Shape<D>;
  using M = Smem<D, NT>;
  constexpr int kRows = M::kRows;
  constexpr bool kFP16 = kIsFp16<T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps];
  __shared__ long long s_base;
  __shared__ int s_seq;
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int units = a.c.H * a.head_groups;   // of a sequence

  pdl_wait();      // the pool, the tables and the queries may come from earlier kernels
  pdl_trigger();

  // The line's length, and where this CTA's part starts.
  uint32_t magic = 0;
  if (tid == 0) magic = __ldcg(a.ws_magic);
  if (tid == 0) s_seq = a.c.n_seqs;
  auto tiles_at = [&](int s) { return s < a.c.n_seqs ? (long long)seq_tiles<S::kTileTokens>(a, s) * units : 0; };
  long long total = 0, mine = tiles_at(tid), upto;
  if (a.c.n_seqs > kThreads) {   // more than a round: the sum of all first
    long long sum = mine;
    for (int s = tid + kThreads; s < a.c.n_seqs; s += kThreads) sum += tiles_at(s);
    block_scan(sum, s_scan, total);
  }
  long long round;
  upto = block_scan(mine, s_scan, round);
  if (a.c.n_seqs <= kThreads) total = round;
  const long long parts = total < a.grid ? total : a.grid;
  Line work;
  work.t = parts ? blockIdx.x * total / parts : 0;
  work.end = blockIdx.x < parts ? (blockIdx.x + 1) * total / parts : work.t;
  for (int s0 = 0;;) {
    if (mine > 0 && work.t < upto && work.t >= upto - mine) {
      s_seq = s0 + tid;
      s_base = upto - mine;
    }
    s0 += kThreads;
    if (s0 >= a.c.n_seqs || work.t < round) break;
    mine = tiles_at(s0 + tid);
    const long long before = round;
    upto = before + block_scan(mine, s_scan, round);
    round += before;
  }
  T* out = static_cast<T*>(a.out);
  const int q_heads = a.c.H * a.group;
  for (int s = blockIdx.x; s < a.c.n_seqs; s += gridDim.x) {
    if (tid == 0 && seq_len_bad(a.c, s)) raise_error(a.c.error, kErrIndex);
    if (seq_len(a.c, s) == 0)   // nothing to see
      for (int i = tid; i < q_heads * D; i += kThreads) out[(long long)s * q_heads * D + i] = from_f32<T>(0.f);
  }
  if (work.t >= work.end) return;
  __syncthreads();
  work.seq = s_seq;
  work.base = s_base;

  uint8_t* ring = smem + warp * (S::kStages * 2 * S::kHalf);
  const uint32_t ring_u = smem_u32(ring);
  const T* pool = static_cast<const T*>(a.c.pool);
  const long long v_off = (long long)a.c.page_size * a.c.H * D;

  // The loads' side runs kStages - 1 steps ahead of the products', over the
  // ends of units. Step i of a warp in a piece: tokens
  // [tok0 + (i kWarps + warp) kStep, + kStep).
  Line ahead = work;
  int l_seq = 0, l_head = 0, l_len = 0, l_next = 0, l_end = 0, l_stage = 0;   // next token and end of this warp's steps
  // Requests the next step's rows; bit r of the result is set where row r is
  // a token to attend to.
  auto issue = [&]() -> uint32_t {
    while (l_next >= l_end) {
      Piece p;
      if (!next_piece<S::kTileTokens>(a, units, ahead, p)) return 0;
      l_seq = p.seq;
      l_head = p.unit / a.head_groups;
      l_len = p.len;
      l_end = p.tile1 == p.tiles ? p.len : p.first + p.tile1 * S::kTileTokens;
      // a piece's last tile may have no token for this warp
      const long long from = (long long)p.first + (long long)p.tile0 * S::kTileTokens + warp * S::kStep;
      l_next = from < l_end ? (int)from : l_end;
    }
    int row = -1;
    bool ok = false;
    if (lane < S::kStep && lane < l_end - l_next) {
      const int j = l_next + lane;
      row = token_row(a.c, l_seq, j);
      ok = row >= 0;
      if (!ok) raise_error(a.c.error, kErrIndex);
      if (kFused && j == l_len - 1) row = -1;   // the new token comes from shared memory
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, ok);
    constexpr int kPerPass = 32 / S::kChunks;   // rows of a pass
    const int chunk = lane % S::kChunks;
    const uint32_t dst0 = ring_u + l_stage * (2 * S::kHalf);
#pragma unroll
    for (int r0 = 0; r0 < S::kStep; r0 += kPerPass) {
      const int r = r0 + lane / S::kChunks;
      const int from = __shfl_sync(0xffffffffu, row, r);
      const T* src = pool + row_offset(a.c, from < 0 ? 0 : from, l_head) + chunk * 8;
      const uint32_t dst = dst0 + r * (D * 2) + ((chunk ^ (r & 7)) << 4);
      cp_async16(dst, src, from >= 0);
      cp_async16(dst + S::kHalf, src + v_off, from >= 0);
    }
    l_stage = l_stage + 1 == S::kStages ? 0 : l_stage + 1;
    l_next = l_end - l_next > S::kTileTokens ? l_next + S::kTileTokens : l_end;
    return valid;
  };
  uint32_t valid[S::kStages];
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) {
    valid[i] = issue();
    cp_async_commit();
  }

  int stage = 0;
  Piece p;
  while (next_piece<S::kTileTokens>(a, units, work, p)) {
    const int h = p.unit / a.head_groups;
    const int head0 = p.unit % a.head_groups * kRows;                     // within the K/V head's group
    const int heads = a.group - head0 < kRows ? a.group - head0 : kRows;
    const int q0 = h * a.group + head0;
    const int tok0 = p.first + p.tile0 * S::kTileTokens + warp * S::kStep;
    const int tok1 = p.tile1 == p.tiles ? p.len : p.first + p.tile1 * S::kTileTokens;
    const T* q = static_cast<const T*>(a.q.p) + p.seq * a.q.token_stride + q0 * a.q.head_stride;
    const bool has_new = kFused && p.tile1 == p.tiles;   // the new token's row lies in this piece

    if (kFused) {
      float* sq = reinterpret_cast<float*>(smem + M::kOffO);
      T* sn = reinterpret_cast<T*>(smem + M::kOffNew);
      const int pos = a.positions ? __ldg(a.positions + p.seq) : p.len - 1;
      int e0, e1;
      const int pair = tid % (D / 2);
      const bool on = rope_pair(a.rope, pair, e0, e1);
      float c = 1.f, s = 0.f;
      if (on) rope_angle(a.rope.turn[pair], pos, a.rope.amplitude, c, s);
      __syncthreads();   // the last unit's results have been read
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
        const int row = token_row(a.c, p.seq, p.len - 1);
        T* to = static_cast<T*>(a.c.pool) + row_offset(a.c, row < 0 ? 0 : row, h);
        const bool write = row >= 0 && head0 == 0;   // one of the head's groups writes it
        if (tid < D / 2) {
          const T* k = static_cast<const T*>(a.k.p) + p.seq * a.k.token_stride + h * a.k.head_stride;
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
        const T* v = static_cast<const T*>(a.v.p) + p.seq * a.v.token_stride + h * a.v.head_stride;
        for (int i = tid; i < D; i += kThreads) {
          const T x = v[i];
          sn[D + i] = x;
          if (write) to[v_off + i] = x;
        }
      }
      __syncthreads();
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
            const float2 x = *reinterpret_cast<const float2*>(smem + M::kOffO + (i * D + d) * 4);
            split2<T>(x.x, x.y, qb[n][k][e], qlo[n][k][e]);   // the rotated query is not rounded
          } else {
            qb[n][k][e] = i < heads ? *reinterpret_cast<const uint32_t*>(q + i * a.q.head_stride + d) : 0u;
          }
        }

    float o[NT][D / 16][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

    const int n_steps = tok0 < tok1 ? (tok1 - tok0 + S::kTileTokens - 1) / S::kTileTokens : 0;
    for (int i = 0; i < n_steps; ++i) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      valid[S::kStages - 1] = issue();
      cp_async_commit();
      const uint32_t on = valid[0];
#pragma unroll
      for (int k = 0; k < S::kStages - 1; ++k) valid[k] = valid[k + 1];
      const uint32_t ks = ring_u + stage * (2 * S::kHalf), vs = ks + S::kHalf;
      if (kFused && has_new) {
        const int r = p.len - 1 - (tok0 + i * S::kTileTokens);
        if (r >= 0 && r < S::kStep) {
          if (lane < 2 * S::kChunks) {
            const int chunk = lane % S::kChunks;
            const uint4 x = reinterpret_cast<const uint4*>(smem + M::kOffNew)[lane];
            *reinterpret_cast<uint4*>(ring + stage * (2 * S::kHalf) + (lane / S::kChunks) * S::kHalf + r * (D * 2) +
                                      ((chunk ^ (r & 7)) << 4)) = x;
          }
          __syncwarp();
        }
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;

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
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);

    // Join the warps in shared memory, a block of 8 heads at a time.
    float* wo = reinterpret_cast<float*>(smem + M::kOffO);
    float* wml = reinterpret_cast<float*>(smem + M::kOffMl);
    const bool whole = p.tile0 == 0 && p.tile1 == p.tiles;
    const int c0 = whole ? 0 : (int)(((p.unit_base + 1) * parts - 1) / total);   // the unit's first CTA
    const long long slot = part_slot(c0, blockIdx.x - c0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n > 0 && heads <= n * 8) break;
      __syncthreads();   // what stood here has been read
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          wo[o_at<D>(warp, lane % 4 * 2 + (e & 1), k * 16 + lane / 4 + (e >> 1) * 8)] = o[n][k][e];
      if (lane < 4) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<float2*>(wml + 2 * (warp * 8 + lane * 2 + c)) = make_float2(m[n][c], l[n][c]);
      }
      __syncthreads();
      const int block = heads - n * 8 < 8 ? heads - n * 8 : 8;
      for (int x = tid; x < block * (D / 2); x += kThreads) {
        const int i = x / (D / 2), d = x % (D / 2) * 2;
        float2 ml[kWarps];
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = *reinterpret_cast<const float2*>(wml + 2 * (w * 8 + i));
          top = fmaxf(top, ml[w].x);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2_approx(ml[w].x - ref);
          const float2 y = *reinterpret_cast<const float2*>(wo + o_at<D>(w, i, d));
          sum = fmaf(f, ml[w].y, sum);
          a0 = fmaf(f, y.x, a0);
          a1 = fmaf(f, y.y, a1);
        }
        const int row = n * 8 + i;
        if (whole) {
          const float r = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // no page was valid: zeros
          *reinterpret_cast<uint32_t*>(out + ((long long)p.seq * q_heads + q0 + row) * D + d) = pack2<T>(a0 * r, a1 * r);
        } else {
          *reinterpret_cast<float2*>(a.part_o + (slot * kRows + row) * D + d) = make_float2(a0, a1);
          if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * kRows + row) * 2) = make_float2(top, sum);
        }
      }
    }
    if (!whole) {
      // The parts of the unit, this CTA's among them; the last to arrive joins.
      const int n = (int)(((p.unit_base + p.tiles) * parts - 1) / total) - c0 + 1;
      const int me = blockIdx.x - c0;
      T* to = out + ((long long)p.seq * q_heads + q0) * D;
      const bool two = n > kJoin;
      const int g0 = two ? me / kGroup * kGroup : 0;
      const int of = two ? min(kGroup, n - g0) : n;
      __syncthreads();
      if (tid == 0) {
        if (magic != kWorkspaceMagic) raise_error(a.c.error, kErrWorkspace);
        s_last = magic == kWorkspaceMagic && arrive_last(a.counters + part_slot(c0, g0), of);
      }
      __syncthreads();
      if (s_last) {
        join_parts<D, T, kRows>(a, wo, c0, g0, 1, of, heads, two ? nullptr : to);
        if (two) {
          const int groups = (n + kGroup - 1) / kGroup;
          __syncthreads();
          if (tid == 0) s_last = arrive_last(a.counters + 2 * a.grid + part_slot(c0, 0), groups);
          __syncthreads();
          if (s_last) join_parts<D, T, kRows>(a, wo, c0, 0, kGroup, groups, heads, to);
        }
      }
    }
  }
  cp_async_wait<0>();
}

int decode_rows(int group) { return group <= 8 ? 8 : 16; }

int decode_grid(int num_sms) { return num_sms * kCtasPerSm; }

template <int D, typename T, int NT, bool kFused>
static cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  static std::atomic<uint8_t> done[kMaxDevices];
  constexpr int kBytes = Smem<D, NT>::kBytes;
  const cudaError_t e = ensure_dynamic_smem(decode_kernel<D, T, NT, kFused>, kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_kernel<D, T, NT, kFused>, dim3(a.grid), dim3(kThreads), kBytes, stream, a);
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
