// C entry points of the token operators (declared in include/kv.h): argument
// checks, workspace layout, launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/kv.h"
#include "api_error.h"
#include "decode_shape.h"
#include "launch.cuh"
#include "page_divisor.h"
#include "token_kernels.h"

namespace {

using pkv::api_cuda_fail;
using pkv::api_fail;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// No exception leaves a C entry: what the standard library may throw on the
// way (it allocates for error texts) becomes a status.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return KV_ERR_CAPACITY;
  }
}

// Checks the paged sequences and fills the kernels' view of them.
int view_cache(const kv_tokens* c, const std::string& who, pkv::TokenCache* out) {
  if (!c) return api_fail(KV_ERR_ARG, who + ": NULL sequences");
  if (c->head_dim != 64 && c->head_dim != 128) return api_fail(KV_ERR_UNSUPPORTED, who + ": head_dim must be 64 or 128");
  if (c->dtype != KV_BF16 && c->dtype != KV_FP16) return api_fail(KV_ERR_UNSUPPORTED, who + ": dtype must be KV_BF16 or KV_FP16");
  if (c->max_pages < 1 || c->page_size < 1 || c->num_heads < 1 ||
      c->num_heads > KV_MAX_Q_HEADS)
    return api_fail(KV_ERR_ARG, who + ": max_pages, page_size or num_heads out of range");
  if (c->n_seqs < 0 || c->n_seqs > KV_MAX_TOKEN_SEQS) return api_fail(KV_ERR_ARG, who + ": n_seqs out of range");
  if (c->table_width < 1 || c->table_stride < c->table_width) return api_fail(KV_ERR_ARG, who + ": table_width or table_stride out of range");
  // The kernels' token indices run up to a tile past a sequence's end, its
  // rows up to the pool's, both in 31 bits.
  if ((long long)c->table_width * c->page_size > (1LL << 30) || (long long)c->max_pages * 2 * c->page_size > INT_MAX)
    return api_fail(KV_ERR_ARG, who + ": more than 2^30 tokens a sequence or 2^31 - 1 rows a pool");
  if (!c->pool || !c->error) return api_fail(KV_ERR_ARG, who + ": NULL pool or error word");
  if (c->n_seqs > 0 && (!c->tables || !c->lens)) return api_fail(KV_ERR_ARG, who + ": NULL tables or lens");
  if (!aligned(c->pool, 16)) return api_fail(KV_ERR_ARG, who + ": pool not 16-byte aligned");
  if (!aligned(c->error, 4) || !aligned(c->tables, 4) || !aligned(c->lens, 4))
    return api_fail(KV_ERR_ARG, who + ": error, tables or lens not 4-byte aligned");
  std::memset(out, 0, sizeof(*out));
  out->pool = c->pool;
  out->tables = c->tables;
  out->lens = c->lens;
  out->error = c->error;
  out->table_stride = c->table_stride;
  out->max_pages = c->max_pages;
  out->page_size = c->page_size;
  out->table_width = c->table_width;
  out->H = c->num_heads;
  out->D = c->head_dim;
  out->n_seqs = c->n_seqs;
  pkv::page_divisor(c->page_size, &out->page_mul, &out->page_shift);
  return KV_OK;
}

// Rows that the kernels read in 16-byte pieces.
int view_rows(const kv_rows* r, const char* name, const std::string& who, pkv::RowsIn* out) {
  if (!r || !r->data) return api_fail(KV_ERR_ARG, who + ": NULL " + name);
  if (!aligned(r->data, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0)
    return api_fail(KV_ERR_ARG, who + ": rows of " + name + " not 16-byte aligned");
  out->p = r->data;
  out->token_stride = r->token_stride;
  out->head_stride = r->head_stride;
  return KV_OK;
}

int view_rope(const kv_rope_t* r, int head_dim, const std::string& who, pkv::RopeTable* out) {
  if (!r) {
    std::memset(out, 0, sizeof(*out));
    return KV_OK;
  }
  if (r->table.rot > head_dim) return api_fail(KV_ERR_ARG, who + ": rot_dim above head_dim");
  *out = r->table;
  return KV_OK;
}

// Tokens and heads of a call: the kernels' row counters run a block's rows
// past the last one in 31 bits.
constexpr int kMaxCount = 1 << 30;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// [magic | arrival counters | the parts' maxima and sums | their outputs], for
// the largest of the shapes that a launch may have; nothing is split where a
// unit has one CTA.
struct DecodeLayout {
  int units, rows, sms;
  size_t counters, off_counters, off_ml, off_o, total;
};

DecodeLayout decode_layout(const kv_tokens* c, int q_heads) {
  const int group = q_heads / c->num_heads;
  DecodeLayout l;
  l.rows = pkv::decode_rows(group);
  l.units = c->num_heads * ((group + l.rows - 1) / l.rows);
  l.sms = pkv::current_device_sms();
  size_t ctas = 0;
  for (int shape = 0; shape < 4; ++shape) {
    const int ranks = pkv::decode_ranks(l.units, l.rows, shape & 1, shape & 2 ? 8 : 4, l.sms);
    if (ranks > 1 && (size_t)ranks * l.units > ctas) ctas = (size_t)ranks * l.units;
  }
  l.counters = 4 * (size_t)pkv::decode_most_ctas(l.sms) * sizeof(uint32_t);   // in one place whatever the heads
  l.off_counters = 256;
  l.off_ml = align256(l.off_counters + l.counters);
  l.off_o = align256(l.off_ml + 2 * ctas * l.rows * 8);
  l.total = align256(l.off_o + 2 * ctas * l.rows * c->head_dim * 4);
  return l;
}

int check_group(const kv_tokens* c, int q_heads, const std::string& who) {
  if (q_heads < 1 || q_heads > KV_MAX_Q_HEADS || q_heads % c->num_heads != 0)
    return api_fail(KV_ERR_ARG, who + ": q_heads must be a multiple of the pool's heads, at most KV_MAX_Q_HEADS");
  return KV_OK;
}

int decode_impl(const kv_tokens* c, const kv_rows* q, int q_heads, const kv_rows* k, const kv_rows* v,
                const kv_rope_t* rope, const int32_t* positions, bool fused, float scale, int window, void* out,
                void* workspace, size_t workspace_bytes, void* stream, const char* name) {
  const std::string who(name);
  pkv::DecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc = view_cache(c, who, &a.c);
  if (rc != KV_OK) return rc;
  if ((rc = check_group(c, q_heads, who)) != KV_OK) return rc;
  const double s = scale != 0 ? (double)scale : 1 / std::sqrt((double)c->head_dim);
  if (!std::isfinite((float)(s * 1.4426950408889634)))   // the logits' own, in powers of two
    return api_fail(KV_ERR_ARG, who + ": scale is not finite, or too large");
  if (window < 0) return api_fail(KV_ERR_ARG, who + ": window < 0");
  if ((rc = view_rope(rope, c->head_dim, who, &a.rope)) != KV_OK) return rc;
  // A rotated query may be amplitude * sqrt(2) times as large as its type's
  // largest value. In fp16, which has no range to spare, the kernel takes it
  // down by the power of two that covers that, and the scale up.
  int down = 0;
  if (c->dtype == KV_FP16 && a.rope.rot > 0) std::frexp(a.rope.amplitude * 1.4142135623730951, &down);
  if (down < 0) down = 0;
  const float scale_log2 = (float)std::ldexp(s * 1.4426950408889634, down);
  if (!std::isfinite(scale_log2)) return api_fail(KV_ERR_ARG, who + ": scale is too large for the rotation's amplitude");
  if (!aligned(positions, 4)) return api_fail(KV_ERR_ARG, who + ": positions not 4-byte aligned");
  if (c->n_seqs == 0) return KV_OK;
  if ((rc = view_rows(q, "q", who, &a.q)) != KV_OK) return rc;
  if (fused && (rc = view_rows(k, "k", who, &a.k)) != KV_OK) return rc;
  if (fused && (rc = view_rows(v, "v", who, &a.v)) != KV_OK) return rc;
  if (!out || !aligned(out, 16)) return api_fail(KV_ERR_ARG, who + ": out NULL or not 16-byte aligned");
  a.group = q_heads / c->num_heads;
  const DecodeLayout l = decode_layout(c, q_heads);
  if (!workspace || !aligned(workspace, 16)) return api_fail(KV_ERR_ARG, who + ": workspace NULL or not 16-byte aligned");
  if (workspace_bytes < l.total) return api_fail(KV_ERR_CAPACITY, who + ": workspace smaller than kv_decode_workspace_bytes()");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.out = out;
  a.positions = positions;
  a.ws_magic = reinterpret_cast<const uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + l.off_counters);
  a.part_ml = reinterpret_cast<float*>(ws + l.off_ml);
  a.part_o = reinterpret_cast<float*>(ws + l.off_o);
  a.head_groups = l.units / c->num_heads;
  a.window = window;
  a.units = l.units;
  a.warps = pkv::decode_warps(c->n_seqs, l.units, l.sms);
  a.ranks = pkv::decode_ranks(l.units, l.rows, fused, a.warps, l.sms);
  a.tile_shift = pkv::decode_tile_shift(c->head_dim, a.warps, c->n_seqs, (long long)c->table_width * c->page_size);
  a.part_tiles = pkv::decode_part_tiles(a.warps);
  a.scale_log2 = scale_log2;
  a.q_down = (float)std::ldexp(1.0, -down);
  const cudaError_t e = c->head_dim == 64 ? pkv::launch_decode_d64(a, c->dtype, fused, (cudaStream_t)stream)
                                          : pkv::launch_decode_d128(a, c->dtype, fused, (cudaStream_t)stream);
  return e == cudaSuccess ? KV_OK : api_cuda_fail(e, (who + ": launch").c_str());
}

}  // namespace

extern "C" {

int kv_rope_init(kv_rope_t** out, int rot_dim, int layout, int scaling, double base, double factor,
                 double original_context, double low_turns, double high_turns, double amplitude) {
  return guarded([&] {
    if (!out) return api_fail(KV_ERR_ARG, "kv_rope_init: out is NULL");
    *out = nullptr;
    double theta[pkv::kMaxRot / 2], amp = 1;
    std::string why;
    const int rc = pkv::rope_frequencies({rot_dim, layout, scaling, base, factor, original_context, low_turns,
                                          high_turns, amplitude}, theta, &amp, &why);
    return rc == KV_OK ? kv_rope_init_frequencies(out, rot_dim, layout, theta, amp) : api_fail(rc, why);
  });
}

int kv_rope_init_frequencies(kv_rope_t** out, int rot_dim, int layout, const double* theta, double amplitude) {
  return guarded([&] {
    if (!out) return api_fail(KV_ERR_ARG, "kv_rope_init_frequencies: out is NULL");
    *out = nullptr;
    if (!theta) return api_fail(KV_ERR_ARG, "kv_rope_init_frequencies: NULL theta");
    kv_rope* r = new kv_rope();
    std::string why;
    const int rc = pkv::rope_table(rot_dim, layout, theta, amplitude, &r->table, &why);
    if (rc != KV_OK) {
      delete r;
      return api_fail(rc, why);
    }
    std::memcpy(r->theta, theta, sizeof(double) * (rot_dim / 2));
    r->amplitude = amplitude;
    r->layout = layout;
    *out = r;
    return (int)KV_OK;
  });
}

void kv_rope_free(kv_rope_t* rope) { delete rope; }

int kv_rope_get(const kv_rope_t* rope, int* rot_dim, int* layout, double* amplitude, double* theta, int cap) {
  return guarded([&] {
    if (!rope || !rot_dim || !layout || !amplitude || cap < 0 || (cap > 0 && !theta))
      return api_fail(KV_ERR_ARG, "kv_rope_get: bad argument");
    *rot_dim = rope->table.rot;
    *layout = rope->layout;
    *amplitude = rope->amplitude;
    for (int i = 0; i < rope->table.rot / 2 && i < cap; ++i) theta[i] = rope->theta[i];
    return (int)KV_OK;
  });
}

int kv_rotate(const kv_rope_t* rope, const kv_rows* x, const kv_rows* out, const int32_t* positions, int n_tokens,
              int n_heads, int head_dim, int dtype, int inverse, void* stream) {
  return guarded([&] {
    const std::string who("kv_rotate");
    if (!rope) return api_fail(KV_ERR_ARG, who + ": NULL rope");
    if (dtype != KV_BF16 && dtype != KV_FP16 && dtype != KV_FP32) return api_fail(KV_ERR_UNSUPPORTED, who + ": unknown dtype");
    if (n_tokens < 0 || n_heads < 0 || n_tokens > kMaxCount || n_heads > kMaxCount)
      return api_fail(KV_ERR_ARG, who + ": n_tokens or n_heads out of range");
    if (head_dim < 2 || head_dim > KV_MAX_ROTATE_DIM || head_dim % 2 != 0)
      return api_fail(KV_ERR_ARG, who + ": head_dim must be even, 2..512");
    pkv::RotateArgs a;
    std::memset(&a, 0, sizeof(a));
    const int rc = view_rope(rope, head_dim, who, &a.rope);
    if (rc != KV_OK) return rc;
    if (n_tokens == 0 || n_heads == 0) return (int)KV_OK;
    const size_t size = dtype == KV_FP32 ? 4 : 2;
    if (!x || !out || !x->data || !out->data) return api_fail(KV_ERR_ARG, who + ": NULL x or out");
    if (!aligned(x->data, size) || !aligned(out->data, size)) return api_fail(KV_ERR_ARG, who + ": x or out misaligned");
    if (!positions || !aligned(positions, 4)) return api_fail(KV_ERR_ARG, who + ": positions NULL or not 4-byte aligned");
    a.x = {x->data, x->token_stride, x->head_stride};
    a.out = {out->data, out->token_stride, out->head_stride};
    a.copy_rest = x->data != out->data;
    if (!a.copy_rest && (x->token_stride != out->token_stride || x->head_stride != out->head_stride))
      return api_fail(KV_ERR_ARG, who + ": in place with other strides");
    a.positions = positions;
    a.n_tokens = n_tokens;
    a.n_heads = n_heads;
    a.head_dim = head_dim;
    a.inverse = inverse != 0;
    pkv::page_divisor(n_heads, &a.head_mul, &a.head_shift);
    const cudaError_t e = pkv::launch_rotate(a, dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? (int)KV_OK : api_cuda_fail(e, "kv_rotate: launch");
  });
}

int kv_append_tokens(const kv_tokens* c, const kv_rows* k, const kv_rows* v, int n_tokens, const int32_t* cu_new,
                     const kv_rope_t* rope, const int32_t* positions, void* stream) {
  return guarded([&] {
    const std::string who("kv_append_tokens");
    pkv::AppendTokensArgs a;
    std::memset(&a, 0, sizeof(a));
    int rc = view_cache(c, who, &a.c);
    if (rc != KV_OK) return rc;
    if (n_tokens < 0 || n_tokens > kMaxCount) return api_fail(KV_ERR_ARG, who + ": n_tokens out of range");
    if (!cu_new && n_tokens != c->n_seqs)
      return api_fail(KV_ERR_ARG, who + ": without cu_new there is one token per sequence");
    if (!aligned(cu_new, 4) || !aligned(positions, 4)) return api_fail(KV_ERR_ARG, who + ": cu_new or positions not 4-byte aligned");
    if ((rc = view_rope(rope, c->head_dim, who, &a.rope)) != KV_OK) return rc;
    if (n_tokens == 0 || c->n_seqs == 0) return (int)KV_OK;
    if ((rc = view_rows(k, "k", who, &a.k)) != KV_OK) return rc;
    if ((rc = view_rows(v, "v", who, &a.v)) != KV_OK) return rc;
    a.cu_new = cu_new;
    a.positions = positions;
    a.n_tokens = n_tokens;
    pkv::page_divisor(c->num_heads, &a.head_mul, &a.head_shift);
    pkv::page_divisor(a.rope.rot > 0 ? a.rope.rot / 2 : 1, &a.pair_mul, &a.pair_shift);
    const cudaError_t e = pkv::launch_append_tokens(a, c->dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? (int)KV_OK : api_cuda_fail(e, "kv_append_tokens: launch");
  });
}

size_t kv_decode_workspace_bytes(const kv_tokens* c, int q_heads) {
  size_t n = 0;
  guarded([&] {
    pkv::TokenCache view;
    if (view_cache(c, "kv_decode_workspace_bytes", &view) != KV_OK) return 0;
    if (check_group(c, q_heads, "kv_decode_workspace_bytes") != KV_OK) return 0;
    n = decode_layout(c, q_heads).total;
    return 0;
  });
  return n;
}

int kv_decode_workspace_init(const kv_tokens* c, int q_heads, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    const std::string who("kv_decode_workspace_init");
    pkv::TokenCache view;
    int rc = view_cache(c, who, &view);
    if (rc != KV_OK) return rc;
    if ((rc = check_group(c, q_heads, who)) != KV_OK) return rc;
    const DecodeLayout l = decode_layout(c, q_heads);
    if (!workspace || !aligned(workspace, 16)) return api_fail(KV_ERR_ARG, who + ": workspace NULL or not 16-byte aligned");
    if (workspace_bytes < l.total) return api_fail(KV_ERR_CAPACITY, who + ": workspace smaller than kv_decode_workspace_bytes()");
    static_assert(pkv::kWorkspaceMagic == 0xa5a5a5a5u, "the magic is one byte over and over");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaError_t e = cudaMemsetAsync(ws + l.off_counters, 0, l.counters, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0xa5, 4, (cudaStream_t)stream);
    return e == cudaSuccess ? (int)KV_OK : api_cuda_fail(e, "kv_decode_workspace_init: memset");
  });
}

int kv_decode(const kv_tokens* c, const kv_rows* q, int q_heads, float scale, int window, void* out, void* workspace,
              size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return decode_impl(c, q, q_heads, nullptr, nullptr, nullptr, nullptr, false, scale, window, out, workspace,
                       workspace_bytes, stream, "kv_decode");
  });
}

int kv_decode_append(const kv_tokens* c, const kv_rows* k, const kv_rows* v, const kv_rows* q, int q_heads,
                     const kv_rope_t* rope, const int32_t* positions, float scale, int window, void* out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return decode_impl(c, q, q_heads, k, v, rope, positions, true, scale, window, out, workspace, workspace_bytes,
                       stream, "kv_decode_append");
  });
}

int kv_tokens_check(const kv_tokens* c, void* stream) {
  return guarded([&] {
    if (!c || !c->error) return api_fail(KV_ERR_ARG, "kv_tokens_check: NULL sequences or error word");
    uint32_t w = 0;
    cudaError_t e = cudaMemcpyAsync(&w, c->error, sizeof(w), cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return api_cuda_fail(e, "kv_tokens_check: read error word");
    if (!w) return (int)KV_OK;
    e = cudaMemsetAsync(c->error, 0, sizeof(w), (cudaStream_t)stream);
    if (e != cudaSuccess) return api_cuda_fail(e, "kv_tokens_check: clear error word");
    return api_fail(KV_ERR_DEVICE_CHECK, "kernel error word " + std::to_string(w));
  });
}

}  // extern "C"
