// Launch interfaces of the token operators (host side): rotary positions,
// appending tokens to a paged pool, attention of one new token per sequence.
// Every launcher returns the CUDA error of the launch; none allocates memory.
#pragma once
#include <cuda_runtime.h>

#include "../../include/kv.h"
#include "rope.h"

namespace pkv {

// [n, heads, head_dim] rows in elements of the tensor's type, the head's
// values next to each other.
struct RowsIn {
  const void* p;
  long long token_stride, head_stride;
};
struct RowsOut {
  void* p;
  long long token_stride, head_stride;
};

struct RotateArgs {
  RowsIn x;
  RowsOut out;
  const int32_t* positions;   // [n_tokens]
  int n_tokens, n_heads, head_dim;
  int inverse;
  int copy_rest;              // out is not x: the values behind rot_dim are copied
  uint32_t head_mul;          // n_heads as a divisor (page_divisor.h)
  int head_shift;
  RopeTable rope;
};

// The paged sequences of a call, as the kernels need them.
struct TokenCache {
  void* pool;                 // [max_pages, 2, page_size, H, D]
  const int32_t* tables;      // [n_seqs] rows of table_width page ids, table_stride apart
  const int32_t* lens;        // [n_seqs]
  uint32_t* error;
  long long table_stride;
  int max_pages, page_size, table_width;
  int H, D, n_seqs;
  uint32_t page_mul;          // j / page_size == umulhi(j, page_mul) >> page_shift for 0 <= j < 2^31
  int page_shift;
};

struct AppendTokensArgs {
  TokenCache c;
  RowsIn k, v;
  const int32_t* cu_new;      // [n_seqs + 1], or NULL: token s is sequence s's
  const int32_t* positions;   // [n_tokens], or NULL: the token's index in its sequence
  int n_tokens;
  uint32_t head_mul, pair_mul;     // c.H and rope.rot / 2 as divisors
  int head_shift, pair_shift;
  RopeTable rope;             // rot 0: none
};

constexpr uint32_t kWorkspaceMagic = 0xa5a5a5a5u;

struct DecodeArgs {
  TokenCache c;
  RowsIn q;
  void* out;                  // [n_seqs, q_heads, D] contiguous
  RowsIn k, v;                // the new tokens (fused append), else NULL
  const int32_t* positions;   // [n_seqs], or NULL: len - 1
  const uint32_t* ws_magic;   // kWorkspaceMagic where the workspace was prepared
  uint32_t* counters;         // [4 * CTAs] arrivals, zero between launches
  float* part_ml;             // [2 * CTAs][rows][2]
  float* part_o;              // [2 * CTAs][rows][D]
  int group;                  // query heads a K/V head serves
  int head_groups;            // groups of at most `rows` query heads a unit takes
  int window;                 // 0: the whole cache
  int units, ranks;           // CTAs: H * head_groups units, `ranks` of each
  int warps;                  // of a CTA (decode_shape.h)
  int tile_shift;             // log2 of a tile's tokens
  int part_tiles;             // tiles that are not worth a join
  float scale_log2;           // scale * log2(e) / q_down
  float q_down;               // power of two on a step's queries in fp16, 1 elsewhere
  RopeTable rope;
};

cudaError_t launch_rotate(const RotateArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_append_tokens(const AppendTokensArgs& a, int dtype, cudaStream_t stream);
// One launch of a.ranks * a.units CTAs; heads of 64 or of 128 values.
cudaError_t launch_decode_d64(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream);
cudaError_t launch_decode_d128(const DecodeArgs& a, int dtype, bool fused, cudaStream_t stream);

}  // namespace pkv
