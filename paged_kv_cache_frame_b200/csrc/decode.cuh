// Attention of one new token per sequence over a paged pool (kv_decode), and
// the whole decode step (kv_decode_append): the query and the new key rotated,
// key and value written to the pool, then the attention.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,  j in [max(0, len - window), len)
//
// Bound by the bytes of K and V: each is read once for the whole group of
// query heads that shares it.
//
// Split. A head unit is a K/V head with a group of at most `rows` of its query
// heads. A CTA has one head unit, and the CTAs with the same place in their
// units' rows ("a rank") take the same tokens: the heads of a token lie side
// by side in the pool, and read at the same time they cost the memory far
// less than one after the other (16 heads of 64, 1.28 GB: 192 us against 222
// with each head's tokens cut elsewhere). The sequences are cut into tiles.
// Every CTA works its own part of the split out from the lengths, which are
// read on the device, so a captured launch serves growing sequences:
//   - while cutting every sequence into parts of at most part_tiles tiles
//     gives no more parts than ranks, each part is a rank's: short sequences
//     stay whole, and nothing is joined that would not pay for it;
//   - else all sequences' tiles (and kSeqCost more each, for what a sequence
//     costs by itself) stand in one line, and rank r of R takes the r-th R-th
//     of it, whatever the sequences' lengths: none waits for a long one.
// A sequence that lies in one rank is written to `out` by it; of the others
// every rank leaves (max, sum, unnormalised O) in the workspace, and the one
// that arrives last joins them, in their order along the sequence whichever
// that is: results do not depend on timing, and no CTA waits for another.
// More than kJoin parts are joined in two rounds, kGroup neighbours first.
//
// In a CTA each of the W warps takes every W-th step of kStep tokens and keeps a
// running max, sum and O of its own; no warp waits for another until the end
// of the sequence. Token rows are gathered by 16-byte asynchronous copies into a
// ring per warp (rows past the end are zero-filled and masked, so what the
// pool holds there is never read). The ring runs on into the CTA's next
// sequence while the warps of this one are joined, and the next one's queries
// (and new key and value) are in registers by then.
//
// The products run transposed on mma.sync m16n8k16, the query heads on the
// N = 8 side: S^T = K Q^T (tokens x heads) and O^T += V^T P^T. K and V then
// fill the M = 16 side whatever the group's size, P moves from accumulator to
// operand layout by movmatrix, and a group of 8 costs one pass. At the
// measured 2 clk per mma and SM these take about a seventh of the time the
// bytes need (tcgen05 would add a trip of S and P through tensor memory to
// every step). P is fed as a sum of two 16-bit values, its rounding and the
// rest: rounding P alone would add an error as large as the output's own.
// fp16 has few values far below 1, so there P counts from kLift powers of two
// below the maximum: what is left of a weight is within 2^-38 of the largest
// one (2^-25 without), which matters where one key takes nearly all of it and
// its value is small.
// Groups of 9 to 16 take two blocks of heads in a pass (32 x 4 x 16 heads of
// 128 over 4096 tokens: 53 us, of which the bytes need 41; a batch that took 62
// us needed 71 as two units).
//
// Measured, inputs not in cache, of a copy's 6.54 TB/s:
//   4 x 16 heads of 64, 77928 tokens, pages of 999     186 us  105%
//   64 sequences of up to 8192, 8 x 4 heads of 128     146 us  100%
//   1 sequence of 262111, 4 x 8 heads of 128           88.6 us  93%
//   1 sequence of 20352, 16 heads of 64                20.2 us  63%
//   a step of 128 sequences, window 1500, 4 x 7 of 64  37.1 us  66%
//   16 heads of 300 tokens                              5.6 us
// The DRAM traffic is the algorithm's bytes. What is left in the shorter ones
// is the start (lengths, then pages, then rows: 2 to 3 us), the join (2 to 3
// us) and CTAs that end at different times.
#pragma once
#include <float.h>
#include <limits.h>

#include "decode_split.h"
#include "launch.cuh"
#include "rope.cuh"
#include "sm100.cuh"
#include "token_access.cuh"

namespace pkv {

namespace {

// In powers of two: how far the reference that P counts from lies below the
// scores' running maximum, and the growth of a score that it lets pass. P
// stays below 2^(kLift + kSlack): 2^15 in fp16, which ends at 2^16.
template <typename T>
constexpr float kLift = kIsFp16<T> ? 13.f : 0.f;
template <typename T>
constexpr float kSlack = kIsFp16<T> ? 2.f : 8.f;
// The maximum of tokens whose scores are all -inf, where that of no token is
// -inf: their sum is 0 as well, but their softmax has no value.
constexpr float kLowest = -FLT_MAX;

template <int D, int NT, bool kFused, int W>
struct Shape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kCtasPerSm = decode_ctas_per_sm(8 * NT, kFused, W);
  static constexpr int kStep = decode_step(D);
  static constexpr int kM = kStep / 16;                 // 16-token blocks of a step
  static constexpr int kStride = kStep * W;             // tokens of a step of all warps
  static constexpr int kStages = decode_stages(8 * NT, kFused, W);
  static constexpr int kHalf = kStep * D * 2;           // K (or V) bytes of a stage
  static constexpr int kRing = W * kStages * 2 * kHalf;
  static constexpr int kChunks = D / 8;                 // 16-byte chunks of a row
  static constexpr int kBlock = D == 128 && kCtasPerSm == 3 ? 4 : 8;   // heads whose O the warps join at a time
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

// Shared memory behind the rings. A piece's queries (as they come, and
// rotated) take the place of the warps' O: never at once.
template <int D, int NT, bool kFused, int W>
struct Smem {
  using S = Shape<D, NT, kFused, W>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kO = W * S::kBlock * D * 4;
  static constexpr int kOffO = S::kRing;                               // [warp][kBlock heads][D] fp32
  static constexpr int kOffMl = kOffO + kO;                            // [warp][kBlock heads] (max, sum)
  static constexpr int kOffNew = kOffMl + W * S::kBlock * 8;           // fused: new key and value [2][D]
  static constexpr int kBytes = kOffNew + 2 * D * 2;
  static constexpr int kOffTurned = kOffO + kRows * D * 2;             // queries [row][D] fp32, behind them as they came
  static_assert(kRows * D * 6 <= kO, "the queries fit the warps' O");
  // An SM has 228 KB, of which every CTA takes 1 KB and its static part besides.
  static_assert(S::kCtasPerSm * (kBytes + 1024 + 128) <= 228 * 1024, "the CTAs of an SM fit");
};

// A lane's remainders of the queries in one product.
template <int NT>
struct alignas(8 * NT) Low {
  uint32_t w[NT][2];
};

// Element d of row i of a warp's O block: row i shifted by 4 i floats, so
// that no two lanes of an accumulator's store share a bank.
template <int D, int kBlock>
__device__ __forceinline__ int o_at(int w, int i, int d) {
  return (w * kBlock + i) * D + ((d + 4 * i) & (D - 1));
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

// The rank's part of the split. Each warp works it out by itself, a lane for a
// stretch of the sequences.
__device__ __forceinline__ Split split(const DecodeArgs& a, uint32_t rank) {
  const int lane = threadIdx.x % 32;
  const int stretch = (a.c.n_seqs + 31) / 32;
  const int s0 = min(lane * stretch, a.c.n_seqs), s1 = min(s0 + stretch, a.c.n_seqs);
  unsigned long long mine = 0;   // places of the line below, parts above; both stay below 2^31
  for (int s = s0; s < s1; ++s) {
    const uint32_t tiles = tiles_of(a, seq_len(a.c, s));
    mine += (unsigned long long)parts_of(a, tiles) << 32 | (tiles ? tiles + kSeqCost : 0);
  }
  unsigned long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const unsigned long long total = __shfl_sync(0xffffffffu, upto, 31);
  Split l;
  split_range(a, rank, (uint32_t)(total >> 32), (uint32_t)total, l);
  const uint32_t last = l.by_parts ? (uint32_t)(upto >> 32) : (uint32_t)upto;
  const uint32_t size = l.by_parts ? (uint32_t)(mine >> 32) : (uint32_t)mine;
  const uint32_t here = __ballot_sync(0xffffffffu, l.t < last && l.t >= last - size);
  const int owner = here ? __ffs(here) - 1 : 31;
  // the stretch of place t: the sequence in front of it, and its first place
  seek(a, l, __shfl_sync(0xffffffffu, here ? s0 : a.c.n_seqs, owner) - 1, __shfl_sync(0xffffffffu, last - size, owner));
  return l;
}

// What an output is divided by, inverted: without a token seen (a sequence of
// pages that are none) it is zero, with scores of -inf alone not a number.
__device__ __forceinline__ float inverse_sum(float top, float sum) {
  return sum > 0.f ? 1.f / sum : top == -INFINITY ? 0.f : NAN;
}

// Adds one to a counter; true for the arrival that completes `of`, with the
// others' writes visible to it. Called by one thread, after a barrier behind
// the CTA's writes.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, int of) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  const bool last = old == (uint32_t)(of - 1);
  if (last) *counter = 0;   // for the next launch
  return last;
}

// Joins parts p0, p0 + step, ... (n of at most 32) of the sequence begun by
// rank r0: O = sum_i 2^(m_i - M) O_i, l = sum_i 2^(m_i - M) l_i. The last round
// writes O / l to `out` (the unit's first query row of the sequence), others
// the part in the first one's place. A warp takes a query head at a time (of
// fewer heads than warps, if they divide these, several warps some of its
// parts each, added up in `sums`): a lane a part's weight, then all lanes the
// parts' rows with kPre of them in flight, the first before the weights are
// known. All threads of the CTA.
template <int D, typename T, int kRows, int W>
__device__ __forceinline__ void join_parts(const DecodeArgs& a, float* sums, int r0, uint32_t unit, int p0, int step, int n,
                                           int heads, T* out) {
  constexpr int V = D / 32;    // values of a lane
  constexpr int kPre = D == 128 ? 4 : 8;   // 16 registers: more and three CTAs' share is spilled (short batches +15%)
  using P = Pack<float, V>;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int share = W % heads == 0 ? W / heads : 1;                      // warps of a head
  const int k1 = warp % share;                                           // this warp's parts: k1, k1 + share, ...
  auto slot = [&](int k) { return part_slot(a, r0, p0 + k * step, unit) * kRows; };
  for (int i = warp / share; i < heads; i += W / share) {
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + i;
    P* rows = reinterpret_cast<P*>(a.part_o) + i * 32 + lane;
    const float2 x = __ldcg(ml + slot(min(lane, n - 1)));
    float acc[V] = {};
    P y[kPre];
#pragma unroll
    for (int k = 0; k < kPre; ++k)
      if (k1 + k * share < n) y[k] = load_cg(rows + slot(k1 + k * share) * 32);
    const float m = lane < n ? x.x : -INFINITY;
    float top = m;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = ex2_approx(m - (top == -INFINITY ? 0.f : top));
    float sum = lane < n ? f * x.y : 0.f;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    for (int k0 = k1; k0 < n; k0 += kPre * share) {
#pragma unroll
      for (int k = 0; k < kPre; ++k) {
        const int at = k0 + k * share;
        const float w = __shfl_sync(0xffffffffu, f, at % 32);
        if (at < n)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(w, y[k].get(e), acc[e]);
      }
#pragma unroll
      for (int k = 0; k < kPre; ++k) {
        const int at = k0 + (kPre + k) * share;
        if (at < n) y[k] = load_cg(rows + slot(at) * 32);
      }
    }
    if (share > 1) {   // uniform: every warp is here once
      if (k1 > 0)
#pragma unroll
        for (int e = 0; e < V; ++e) sums[(warp * 32 + lane) * V + e] = acc[e];
      __syncthreads();
      if (k1 > 0) break;
      for (int k = 1; k < share; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += sums[((warp + k) * 32 + lane) * V + e];
    }
    if (out) {
      const float inv = inverse_sum(top, sum);
      uint32_t* to = reinterpret_cast<uint32_t*>(out + i * D + lane * V);
#pragma unroll
      for (int e = 0; e < V; e += 2) to[e / 2] = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
    } else {
      P r;
#pragma unroll
      for (int e = 0; e < V; e += 2) r.set2(e / 2, acc[e], acc[e + 1]);
      const long long at = slot(0);
      rows[at * 32] = r;
      if (lane == 0) reinterpret_cast<float2*>(a.part_ml)[at + i] = make_float2(top, sum);
    }
  }
}

}  // namespace

template <int D, typename T, int NT, bool kFused, int W>
__global__ void __launch_bounds__(Shape<D, NT, kFused, W>::kThreads, Shape<D, NT, kFused, W>::kCtasPerSm)
    decode_kernel(const __grid_constant__ DecodeArgs a) {
  using S = Shape<D, NT, kFused, W>;
  using M = Smem<D, NT, kFused, W>;
  constexpr int kThreads = S::kThreads;
  constexpr int kRows = M::kRows;
  constexpr bool kFP16 = kIsFp16<T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ bool s_last, s_more;
  __shared__ Piece s_piece[2];   // this one and the next
  __shared__ Split s_work;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t rank = blockIdx.x / a.units, unit = blockIdx.x - rank * a.units;
  const int h = unit / a.head_groups;                                   // its K/V head
  const int head0 = (unit - h * a.head_groups) * kRows;                 // and query heads, within the head's group
  const int heads = a.group - head0 < kRows ? a.group - head0 : kRows;
  const int q0 = h * a.group + head0;

  pdl_wait();      // the pool, the tables and the queries may come from earlier kernels
  pdl_trigger();

  uint32_t magic = 0;
  if (tid == 0) magic = __ldcg(a.ws_magic);
  Split ahead = split(a, rank);
  T* out = static_cast<T*>(a.out);
  const int q_heads = a.c.H * a.group;
  for (int s = blockIdx.x; s < a.c.n_seqs; s += gridDim.x) {
    if (tid == 0 && seq_len_bad(a.c, s)) raise_error(a.c.error, kErrIndex);
    if (seq_len(a.c, s) == 0)   // nothing to see
      for (int i = tid; i < q_heads * D; i += kThreads) out[(long long)s * q_heads * D + i] = from_f32<T>(0.f);
  }
  uint8_t* ring = smem + warp * (S::kStages * 2 * S::kHalf);
  const uint32_t ring_u = smem_u32(ring);
  const T* pool = static_cast<const T*>(a.c.pool);
  const long long v_off = (long long)a.c.page_size * a.c.H * D;

  // A piece's queries, and its new key and value where it holds the new
  // token: 16 bytes a thread and round, requested a piece ahead.
  constexpr int kQ = kRows * S::kChunks / kThreads > 0 ? kRows * S::kChunks / kThreads : 1;
  uint4 raw[kQ], raw_new = make_uint4(0, 0, 0, 0);
  int new_page = -1, new_pos = -1;
  auto request = [&](const Piece& p) {
    const T* q = static_cast<const T*>(a.q.p) + p.seq * a.q.token_stride + q0 * a.q.head_stride;
#pragma unroll
    for (int x = 0; x < kQ; ++x) {
      const int i = (x * kThreads + tid) / S::kChunks, chunk = tid % S::kChunks;
      raw[x] = i < heads ? *reinterpret_cast<const uint4*>(q + i * a.q.head_stride + chunk * 8)
                                                : make_uint4(0, 0, 0, 0);
    }
    if (kFused) {
      if (a.positions) new_pos = __ldg(a.positions + p.seq);
      if (p.tok1 == p.raw) {
        new_page = __ldg(a.c.tables + p.seq * a.c.table_stride + page_of(a.c, p.tok1 - 1));
        if (tid < 2 * S::kChunks) {
          const RowsIn& from = tid < S::kChunks ? a.k : a.v;
          raw_new = *reinterpret_cast<const uint4*>(static_cast<const T*>(from.p) + p.seq * from.token_stride +
                                                    h * from.head_stride + tid % S::kChunks * 8);
        }
      }
    }
  };

  // The CTA's pieces, one after the other, as its last warp finds them: what
  // the barriers below depend on is the same for all warps even if the lengths
  // change under the launch, which must not be but must not hang.
  if (tid == kThreads - 32) s_work = ahead;
  int which = 0;   // of s_piece
  auto find_next = [&](int to) {
    if (warp == W - 1) {
      __syncwarp();
      Split work = s_work;
      Piece next;
      const bool found = next_piece(a, rank, work, next);
      __syncwarp();
      if (lane == 0) {
        s_work = work;
        s_more = found;
        if (found) s_piece[to] = next;
      }
    }
  };
  find_next(0);

  // The loads' side runs kStages - 1 steps ahead of the products', over the
  // ends of units. Step i of a warp in a piece: tokens
  // [tok0 + (i W + warp) kStep, + kStep).
  constexpr int kPerPass = 32 / S::kChunks;   // rows of a pass
  const int chunk = lane % S::kChunks;
  const long long row_size = (long long)a.c.H * D;
  const T* const src0 = pool + h * D + chunk * 8;                 // the lane's chunk of the head in row 0
  int l_seq = 0, l_raw = 0, l_next = 0, l_end = 0, l_stage = 0;   // next token and end of this warp's steps
  int l_page = 0;                                                 // the lane's page of the next step, looked up ahead
  bool l_ok = false;                                              // (not looked at before it is needed)
  auto look_up = [&]() {   // goes on to the next piece where this one has no step left
    while (l_next >= l_end) {
      Piece p;
      if (!next_piece(a, rank, ahead, p)) {
        l_next = INT_MAX;
        return;
      }
      l_seq = p.seq;
      l_raw = p.raw;
      l_end = p.tok1;
      l_next = p.tok0 + warp * S::kStep;   // a piece may have no step for this warp
    }
    l_ok = lane < S::kStep && lane < l_end - l_next;
    if (l_ok) l_page = __ldg(a.c.tables + l_seq * a.c.table_stride + page_of(a.c, l_next + lane));
  };
  // Requests the next step's rows; bit r of the result is set where row r is
  // a token to attend to.
  auto issue = [&]() -> uint32_t {
    if (l_next == INT_MAX) return 0;
    int row = l_ok ? row_in(a.c, l_page, l_next + lane) : -1;
    if (l_ok && row < 0) raise_error(a.c.error, kErrIndex);
    const uint32_t valid = __ballot_sync(0xffffffffu, row >= 0);
    if (kFused && l_next + lane == l_raw - 1) row = -1;   // the new token comes from shared memory
    const uint32_t dst0 = ring_u + l_stage * (2 * S::kHalf);
#pragma unroll
    for (int r0 = 0; r0 < S::kStep; r0 += kPerPass) {
      const int r = r0 + lane / S::kChunks;
      const int from = __shfl_sync(0xffffffffu, row, r);
      const T* src = src0 + max(from, 0) * row_size;
      const uint32_t dst = dst0 + r * (D * 2) + ((chunk ^ (r & 7)) << 4);
      cp_async16(dst, src, from >= 0);
      cp_async16(dst + S::kHalf, src + v_off, from >= 0);
    }
    l_stage = l_stage + 1 == S::kStages ? 0 : l_stage + 1;
    l_next += S::kStride;
    look_up();
    return valid;
  };
  look_up();
  __syncthreads();
  if (!s_more) return;
  request(s_piece[0]);
  uint32_t valid[S::kStages] = {};   // of the steps under way, the next one first
#pragma unroll 1   // one copy of issue()
  for (int i = 0; i < S::kStages - 1; ++i) {
#pragma unroll
    for (int k = 0; k < S::kStages - 2; ++k) valid[k] = valid[k + 1];
    valid[S::kStages - 2] = issue();
    cp_async_commit();
  }

  // The thread's pair of a head's values, in every piece.
  int e0 = 0, e1 = 0;
  const bool on = kFused && rope_pair(a.rope, tid % (D / 2), e0, e1);
  const uint64_t turn = on ? a.rope.turn[tid % (D / 2)] : 0;

  int stage = 0;
  for (;;) {
    const Piece& p = s_piece[which];
    const int tok0 = p.tok0 + warp * S::kStep, tok1 = p.tok1;
    const bool has_new = kFused && tok1 == p.raw;   // the new token's row lies in this piece

    __syncthreads();   // the last piece's results, and where this one lies, have been read
    uint4* sq = reinterpret_cast<uint4*>(smem + M::kOffO);
    float* sf = reinterpret_cast<float*>(smem + M::kOffTurned);
    T* sn = reinterpret_cast<T*>(smem + M::kOffNew);
#pragma unroll
    for (int x = 0; x < kQ; ++x)
      if (x * kThreads + tid < kRows * S::kChunks) sq[x * kThreads + tid] = raw[x];
    const int row_of_new = row_in(a.c, new_page, tok1 - 1);
    const int pos = a.positions ? new_pos : held(a.c, p.raw) - 1;
    if (has_new && tid < 2 * S::kChunks) reinterpret_cast<uint4*>(sn)[tid] = raw_new;
    find_next(which ^ 1);
    if (kFused) {
      float c = 1.f, s = 0.f;
      if (on) rope_angle(turn, pos, a.rope.amplitude, c, s);
      __syncthreads();
      const T* raw_q = reinterpret_cast<const T*>(sq);
      for (int i = tid / (D / 2); i < kRows; i += kThreads / (D / 2)) {
        float x = to_f32(raw_q[i * D + e0]), y = to_f32(raw_q[i * D + e1]);
        if (on) rope_turn(x, y, c, s);
        if constexpr (kFP16) x *= a.q_down, y *= a.q_down;   // a power of two: into the range of the two values below
        sf[i * D + e0] = x;
        sf[i * D + e1] = y;
      }
      if (has_new && on && tid < D / 2) {
        float x = to_f32(sn[e0]), y = to_f32(sn[e1]);
        rope_turn(x, y, c, s);
        sn[e0] = from_f32<T>(x);   // the cache's type: attended to as later tokens will read it
        sn[e1] = from_f32<T>(y);
      }
    }
    __syncthreads();
    if (s_more) request(s_piece[which ^ 1]);
    if (has_new && tid < 2 * S::kChunks) {
      if (row_of_new < 0) {
        if (tid == 0) raise_error(a.c.error, kErrIndex);
      } else if (head0 == 0) {   // one of the head's groups writes it
        T* to = static_cast<T*>(a.c.pool) + row_offset(a.c, row_of_new, h) + (tid < S::kChunks ? 0 : v_off);
        reinterpret_cast<uint4*>(to)[tid % S::kChunks] = reinterpret_cast<const uint4*>(sn)[tid];
      }
    }

    // Queries as B operands: heads lane / 4 of each block of 8, values
    // 16 k + (lane % 4) * 2 and the next, and those 8 further.
    // Of two blocks the remainders stay in shared memory (where the queries
    // as they came were), a lane's of a product side by side: registers.
    constexpr bool kLowInSmem = kFused && NT == 2;
    Low<NT>* const low_at = reinterpret_cast<Low<NT>*>(sq);
    uint32_t qb[NT][D / 16][2], qlo[NT][kFused && !kLowInSmem ? D / 16 : 1][2];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = (n * 8 + lane / 4) * D + k * 16 + e * 8 + lane % 4 * 2;
          if constexpr (kFused) {
            const float2 x = *reinterpret_cast<const float2*>(sf + at);
            split2<T>(x.x, x.y, qb[n][k][e], lo[n][e]);   // the rotated query is not rounded
            if constexpr (!kLowInSmem) qlo[n][k][e] = lo[n][e];
          } else {
            qb[n][k][e] = reinterpret_cast<const uint32_t*>(sq)[at / 2];
          }
        }
      if constexpr (kLowInSmem)
        if (k % W == warp) {
          Low<NT> x;
#pragma unroll
          for (int n = 0; n < NT; ++n) x.w[n][0] = lo[n][0], x.w[n][1] = lo[n][1];
          low_at[k * 32 + lane] = x;
        }
    }
    if constexpr (kLowInSmem) __syncthreads();

    float o[NT][D / 16][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

    uint32_t any = 0;   // a token was seen
    const int n_steps = tok0 < tok1 ? (tok1 - tok0 + S::kStride - 1) / S::kStride : 0;
    for (int i = 0; i < n_steps; ++i) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      valid[S::kStages - 1] = issue();
      cp_async_commit();
      const uint32_t seen = valid[0];
      any |= seen;
#pragma unroll
      for (int k = 0; k < S::kStages - 1; ++k) valid[k] = valid[k + 1];
      const uint32_t ks = ring_u + stage * (2 * S::kHalf), vs = ks + S::kHalf;
      if (kFused && has_new && row_of_new >= 0) {   // a token without a page leaves its row zero
        const int r = tok1 - 1 - (tok0 + i * S::kStride);
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
      // heads (lane % 4) * 2 and the next. Even and odd products (and the
      // queries' remainders) in sums of their own: shorter chains.
      constexpr int kTurns = NT == 1 ? 2 : 1;         // even and odd apart, where a block of heads does not do
      constexpr int kSums = kFused ? 2 * kTurns : kTurns;
      float sc[S::kM][NT][4];
#pragma unroll
      for (int b = 0; b < S::kM; ++b) {
        float part[NT][kSums][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t x[4];
          const int r = b * 16 + lane % 16;
          ldsm_x4(ks + r * (D * 2) + (((2 * k + lane / 16) ^ (r & 7)) << 4), x);
          Low<NT> lows;
          if constexpr (kLowInSmem) lows = low_at[k * 32 + lane];
          auto low = [&](int n, int k, int e) {
            if constexpr (kLowInSmem) return lows.w[n][e];
            else return qlo[n][k][e];
          };
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816<kFP16>(part[n][k % kTurns], x, qb[n][k][0], qb[n][k][1]);
            if constexpr (kFused)
              mma_16816<kFP16>(part[n][kTurns + k % kTurns], x, low(n, k, 0), low(n, k, 1));
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = part[n][0][e];
#pragma unroll
            for (int t = 1; t < kSums; ++t) x += part[n][t][e];
            sc[b][n][e] = x * a.scale_log2;
          }
      }
      constexpr uint32_t kAll = S::kStep == 32 ? 0xffffffffu : (1u << S::kStep % 32) - 1;
      if (seen != kAll) {
#pragma unroll
        for (int b = 0; b < S::kM; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(seen >> (b * 16 + lane / 4 + (e >> 1) * 8) & 1)) sc[b][n][e] = -INFINITY;
      }
      // The reference m (kLift below the maximum) follows the scores only
      // when one exceeds it by kSlack more; O and l have the same factor.
      // Mostly a vote is all it takes.
      float top[NT][2];
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[n][c] = fmaxf(sc[0][n][c], sc[0][n][c + 2]);
          if constexpr (S::kM == 2) top[n][c] = fmaxf(top[n][c], fmaxf(sc[1][n][c], sc[1][n][c + 2]));
          grew |= top[n][c] > m[n][c] + (kLift<T> + kSlack<T>);
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = top[n][c];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            x -= kLift<T>;
            const float f = x > m[n][c] ? ex2_approx(m[n][c] - x) : 1.f;   // 0 from -inf
            m[n][c] = fmaxf(x, m[n][c]);
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
        // A few blocks of values at a time, first with P, then with its
        // remainder: no product waits for the one before it.
        constexpr int kBlocks = 4 / NT;
#pragma unroll
        for (int k0 = 0; k0 < D / 16; k0 += kBlocks) {
          uint32_t x[kBlocks][4];
          const int r = b * 16 + lane % 8 + lane / 16 * 8;
#pragma unroll
          for (int k = 0; k < kBlocks; ++k)
            ldsm_x4_t(vs + r * (D * 2) + (((2 * (k0 + k) + (lane / 8 & 1)) ^ (r & 7)) << 4), x[k]);
#pragma unroll
          for (int k = 0; k < kBlocks; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816<kFP16>(o[n][k0 + k], x[k], ph[n][0], ph[n][1]);
#pragma unroll
          for (int k = 0; k < kBlocks; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816<kFP16>(o[n][k0 + k], x[k], pl[n][0], pl[n][1]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
        if (any && m[n][c] == -INFINITY) m[n][c] = kLowest;
      }

    // Join the warps in shared memory, a block of heads at a time.
    float* wo = reinterpret_cast<float*>(smem + M::kOffO);
    float* wml = reinterpret_cast<float*>(smem + M::kOffMl);
    constexpr int kBlock = S::kBlock;
    const bool whole = p.parts == 1;
    const long long slot = part_slot(a, p.r0, rank - p.r0, unit);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int block = 0; block < 8; block += kBlock) {
        const int first = n * 8 + block;
        if (first > 0 && heads <= first) break;
        __syncthreads();   // what stood here has been read
        const int i0 = lane % 4 * 2 - block;   // the lane's two heads, in the block or not
        if (i0 >= 0 && i0 < kBlock) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              wo[o_at<D, kBlock>(warp, i0 + (e & 1), k * 16 + lane / 4 + (e >> 1) * 8)] = o[n][k][e];
          if (lane < 4) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<float2*>(wml + 2 * (warp * kBlock + i0 + c)) = make_float2(m[n][c], l[n][c]);
          }
        }
        __syncthreads();
        const int here = heads - first < kBlock ? heads - first : kBlock;
        for (int x = tid; x < here * (D / 2); x += kThreads) {
          const int i = x / (D / 2), d = x % (D / 2) * 2;
          float2 ml[W];
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            ml[w] = *reinterpret_cast<const float2*>(wml + 2 * (w * kBlock + i));
            top = fmaxf(top, ml[w].x);
          }
          const float ref = top == -INFINITY ? 0.f : top;
          float sum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float f = ex2_approx(ml[w].x - ref);
            const float2 y = *reinterpret_cast<const float2*>(wo + o_at<D, kBlock>(w, i, d));
            sum = fmaf(f, ml[w].y, sum);
            a0 = fmaf(f, y.x, a0);
            a1 = fmaf(f, y.y, a1);
          }
          const int row = first + i;
          if (whole) {
            const float r = inverse_sum(top, sum);
            *reinterpret_cast<uint32_t*>(out + ((long long)p.seq * q_heads + q0 + row) * D + d) =
                pack2<T>(a0 * r, a1 * r);
          } else {
            *reinterpret_cast<float2*>(a.part_o + (slot * kRows + row) * D + d) = make_float2(a0, a1);
            if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * kRows + row) * 2) = make_float2(top, sum);
          }
        }
      }
    }
    if (!whole) {
      // The sequence's parts, this CTA's among them; the last to arrive joins.
      T* to = out + ((long long)p.seq * q_heads + q0) * D;
      const Join j = join_of(rank - p.r0, p.parts);
      __syncthreads();
      if (tid == 0) {
        const bool ready = magic == kWorkspaceMagic;
        if (!ready) raise_error(a.c.error, kErrWorkspace);
        s_last = ready && arrive_last(a.counters + first_counter(a, p.r0, j, unit), j.of);
      }
      __syncthreads();
      bool last = s_last;
      if (last) join_parts<D, T, kRows, W>(a, wo, p.r0, unit, j.g0, 1, j.of, heads, j.two ? nullptr : to);
      if (last && j.two) {
        __syncthreads();
        if (tid == 0) s_last = arrive_last(a.counters + second_counter(a, p.r0, unit), j.groups);
        __syncthreads();
        last = s_last;
        if (last) join_parts<D, T, kRows, W>(a, wo, p.r0, unit, 0, kGroup, j.groups, heads, to);
      }
    }
    if (!s_more) break;
    which ^= 1;
  }
  cp_async_wait<0>();
}

template <int D, typename T, int NT, bool kFused, int W>
cudaError_t launch_decode_shape(const DecodeArgs& a, cudaStream_t stream) {
  static std::atomic<uint8_t> done[kMaxDevices];
  constexpr int kBytes = Smem<D, NT, kFused, W>::kBytes;
  const cudaError_t e = ensure_dynamic_smem(decode_kernel<D, T, NT, kFused, W>, kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_kernel<D, T, NT, kFused, W>, dim3(a.ranks * a.units), dim3(32 * W), kBytes, stream, a);
}

template <int D, typename T, int NT>
cudaError_t launch_decode_rows(const DecodeArgs& a, bool fused, cudaStream_t stream) {
  if (a.warps == 8)
    return fused ? launch_decode_shape<D, T, NT, true, 8>(a, stream) : launch_decode_shape<D, T, NT, false, 8>(a, stream);
  return fused ? launch_decode_shape<D, T, NT, true, 4>(a, stream) : launch_decode_shape<D, T, NT, false, 4>(a, stream);
}

template <int D>
cudaError_t launch_decode_dim(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream) {
  const bool one = decode_rows(a.group) == 8;
  if (dtype == KV_FP16)
    return one ? launch_decode_rows<D, __half, 1>(a, fused, stream) : launch_decode_rows<D, __half, 2>(a, fused, stream);
  return one ? launch_decode_rows<D, __nv_bfloat16, 1>(a, fused, stream)
             : launch_decode_rows<D, __nv_bfloat16, 2>(a, fused, stream);
}

}  // namespace pkv
