// Native binding of the token operators' Python objects: tensors checked and
// handed to the C entry points of include/kv.h without a detour through Python
// attributes, and the rotation as an autograd node. A call from Python costs
// its launch (2.4 us) and 2 us around it; through ctypes it was 7.
//
// Calls run on torch's current stream of the tensors' device. A status of the
// library becomes the package's KVError, a wrong argument a ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <sstream>
#include <string>
#include <utility>

#include "kv.h"
#include "overlap.h"

namespace {

PyObject* g_check = nullptr;   // check(status, where) of the package: raises KVError

struct LibraryError : std::runtime_error {
  int status;
  const char* where;
  LibraryError(int s, const char* w) : std::runtime_error(std::string(w) + ": " + kv_last_error()), status(s), where(w) {}
};

void check_status(int status, const char* where) {
  if (status != KV_OK) throw LibraryError(status, where);
}

// The sequence of sizes as Python shows them.
std::string shown(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  if (s.size() == 1) o << ",";
  o << ")";
  return o.str();
}

// Shape, type, device and layout of a tensor, before its address goes to the
// library. Not contiguous: the last dimension only has to be dense.
void check_tensor(const at::Tensor& x, const char* name, at::IntArrayRef shape, at::ScalarType dtype, at::Device device,
                  bool contiguous) {
  TORCH_CHECK_VALUE(x.sizes() == shape, name, ": shape ", shown(x.sizes()), ", expected ", shown(shape));
  TORCH_CHECK_VALUE(x.scalar_type() == dtype, name, ": dtype ", x.scalar_type(), ", expected ", dtype);
  TORCH_CHECK_VALUE(x.device() == device, name, ": on ", x.device(), ", expected ", device);
  TORCH_CHECK_VALUE(!x.is_neg(), name, ": its values are not the memory's (resolve_neg() first)");
  if (x.is_contiguous()) return;
  TORCH_CHECK_VALUE(!contiguous, name, ": must be contiguous");
  TORCH_CHECK_VALUE(x.stride(-1) == 1 || x.size(-1) <= 1 || x.numel() == 0, name, ": the last dimension must be contiguous");
}

void check_device(const at::Tensor& x, const char* name) {
  TORCH_CHECK_VALUE(x.is_cuda(), name, ": must be a CUDA tensor, not on ", x.device());
}

// No operator has a forward-mode derivative: a tangent is refused, not dropped.
void check_no_tangent(const at::Tensor& x, const char* name) {
  TORCH_CHECK_VALUE(!x._fw_grad(0).defined() || !c10::AutogradState::get_tls_state().get_fw_grad_mode(), name,
                    ": carries a tangent, and there is no forward-mode derivative (unpack_dual it)");
}

// The operators without a gradient refuse inputs that would want one.
void check_no_gradient(const at::Tensor& x, const char* name) {
  check_no_tangent(x, name);
  TORCH_CHECK_VALUE(!x.requires_grad() || !at::GradMode::is_enabled(), name,
                    ": requires a gradient, which this operator does not have (detach it or call under torch.no_grad)");
}

// A tensor that a call writes: apart from its own elements, and counted as
// changed, so that autograd notices where it was saved.
void check_written(const at::Tensor& x, const char* name) {
  check_no_gradient(x, name);
  TORCH_CHECK_VALUE(at::has_internal_overlap(x) != at::MemOverlap::Yes, name, ": its elements share memory (an expanded tensor)");
}
void written(const at::Tensor& x) {
  if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}

// A [n, heads, head_dim] tensor's rows; the stride of a dimension of one
// element says nothing and is 0.
kv_rows rows_of(const at::Tensor& x) {
  return {x.data_ptr(), x.size(0) > 1 ? x.stride(0) : 0, x.size(1) > 1 ? x.stride(1) : 0};
}

pkv::RowSet bytes_of(const at::Tensor& x, const kv_rows& r) {
  const int64_t size = x.element_size();
  return {reinterpret_cast<int64_t>(r.data), x.size(0), x.size(1), x.size(2) * size, r.token_stride * size, r.head_stride * size};
}
pkv::RowSet bytes_of(const at::Tensor& x) {   // contiguous
  return {reinterpret_cast<int64_t>(x.data_ptr()), 1, 1, (int64_t)x.nbytes(), 0, 0};
}

// What a call writes lies apart from what it reads.
void check_apart(const pkv::RowSet& x, const char* name, const pkv::RowSet& read, const char* other) {
  TORCH_CHECK_VALUE(!pkv::share_memory(x, read), name, ": shares memory with ", other, ", which the call reads");
}

const int32_t* index_of(const c10::optional<at::Tensor>& x, const char* name, int64_t n, at::Device device) {
  if (!x) return nullptr;
  check_tensor(*x, name, {n}, at::kInt, device, true);
  return x->data_ptr<int32_t>();
}

at::Tensor empty_rows(const at::Tensor& x) { return at::empty_like(x, x.options(), at::MemoryFormat::Contiguous); }

int dtype_code(at::ScalarType t) { return t == at::kBFloat16 ? KV_BF16 : t == at::kHalf ? KV_FP16 : t == at::kFloat ? KV_FP32 : -1; }

// ---------------------------------------------------------------- rotation
struct Rope : torch::CustomClassHolder {
  kv_rope_t* handle;
  explicit Rope(kv_rope_t* h) : handle(h) {}
  ~Rope() override { kv_rope_free(handle); }
};

at::Tensor rotate(const c10::intrusive_ptr<Rope>& rope, const at::Tensor& x, const at::Tensor& positions,
                  const c10::optional<at::Tensor>& given, bool inverse) {
  const int code = dtype_code(x.scalar_type());
  TORCH_CHECK_VALUE(code >= 0, "x: dtype ", x.scalar_type(), ", expected bfloat16, float16 or float32");
  TORCH_CHECK_VALUE(x.dim() == 3, "x: shape ", shown(x.sizes()), ", expected [tokens, heads, head_dim]");
  check_no_tangent(x, "x");
  check_device(x, "x");
  check_tensor(x, "x", x.sizes(), x.scalar_type(), x.device(), false);
  TORCH_CHECK_VALUE(x.size(0) <= INT32_MAX && x.size(1) <= INT32_MAX && x.size(2) <= INT32_MAX, "x: too large");
  check_tensor(positions, "positions", {x.size(0)}, at::kInt, x.device(), true);
  if (given) {
    check_tensor(*given, "out", x.sizes(), x.scalar_type(), x.device(), false);
    check_written(*given, "out");
  }
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  at::Tensor out = given ? *given : empty_rows(x);
  const kv_rows from = rows_of(x), to = rows_of(out);
  if (given && !(from.data == to.data && from.token_stride == to.token_stride && from.head_stride == to.head_stride))
    check_apart(bytes_of(out, to), "out", bytes_of(x, from), "x");
  check_status(kv_rotate(rope->handle, &from, &to, positions.data_ptr<int32_t>(), (int)x.size(0), (int)x.size(1),
                         (int)x.size(2), code, inverse, c10::cuda::getCurrentCUDAStream(x.device().index()).stream()),
               "kv_rotate");
  if (given) written(out);
  return out;
}

// y = rotation of x; dx = the inverse rotation of dy, itself differentiable.
struct Rotation : torch::autograd::Function<Rotation> {
  static at::Tensor forward(torch::autograd::AutogradContext* ctx, const at::Tensor& x, const at::Tensor& positions,
                            c10::intrusive_ptr<Rope> rope, bool inverse) {
    ctx->save_for_backward({positions});
    ctx->saved_data["inverse"] = inverse;
    at::Tensor y = rotate(rope, x, positions, c10::nullopt, inverse);
    ctx->saved_data["rope"] = c10::IValue::make_capsule(std::move(rope));
    return y;
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list g) {
    const at::Tensor positions = ctx->get_saved_variables()[0];
    at::Tensor dy = g[0];
    if (!dy.defined()) return {at::Tensor(), at::Tensor(), at::Tensor(), at::Tensor()};
    dy = dy.resolve_neg();   // a view whose values are not the memory's: not the user's to resolve
    if (dy.stride(-1) != 1) dy = dy.contiguous();
    auto rope = c10::static_intrusive_pointer_cast<Rope>(ctx->saved_data["rope"].toCapsule());
    const bool inverse = !ctx->saved_data["inverse"].toBool();
    at::Tensor dx = at::GradMode::is_enabled() ? Rotation::apply(dy, positions, std::move(rope), inverse)
                                               : rotate(rope, dy, positions, c10::nullopt, inverse);
    return {dx, at::Tensor(), at::Tensor(), at::Tensor()};
  }
};

// ---------------------------------------------------------------- paged sequences
struct Tokens {
  kv_tokens c;
  at::Tensor pool, tables, lens, error;   // what `c` points to
  bool read_only;                         // the pages belong to frame caches
  at::ScalarType dtype;
  at::Device device;
  std::map<std::pair<void*, int64_t>, at::Tensor> workspaces;   // of eager calls, by stream and query heads
  std::map<int64_t, size_t> bytes;                              // of a workspace, by query heads
};

cudaStream_t stream_of(const Tokens& t) { return c10::cuda::getCurrentCUDAStream(t.device.index()).stream(); }

size_t workspace_bytes(Tokens& t, int64_t heads) {
  const auto it = t.bytes.find(heads);
  if (it != t.bytes.end()) return it->second;
  const size_t n = heads > 0 && heads <= KV_MAX_Q_HEADS ? kv_decode_workspace_bytes(&t.c, (int)heads) : 0;
  return n ? t.bytes[heads] = n : 0;
}

at::Tensor new_workspace(Tokens& t, int64_t heads) {
  at::Tensor ws = at::empty({(int64_t)workspace_bytes(t, heads)}, at::TensorOptions().dtype(at::kByte).device(t.device));
  check_status(kv_decode_workspace_init(&t.c, (int)heads, ws.data_ptr(), (size_t)ws.numel(), stream_of(t)),
               "kv_decode_workspace_init");
  return ws;
}

// k and v [n, heads, head_dim] of new tokens.
void check_new(const Tokens& t, const at::Tensor& k, const at::Tensor& v, int64_t n) {
  TORCH_CHECK_VALUE(!t.read_only, "the tokens of a frame plan are read only: their pages and slots are the caches'");
  const int64_t shape[] = {n, t.c.num_heads, t.c.head_dim};
  check_tensor(k, "k", shape, t.dtype, t.device, false);
  check_tensor(v, "v", shape, t.dtype, t.device, false);
  check_no_gradient(k, "k");
  check_no_gradient(v, "v");
}

void append(Tokens& t, const at::Tensor& k, const at::Tensor& v, const c10::optional<at::Tensor>& cu_new, const Rope* rope,
            const c10::optional<at::Tensor>& positions) {
  const int64_t n = cu_new && k.dim() == 3 ? k.size(0) : t.c.n_seqs;
  check_new(t, k, v, n);
  check_written(t.pool, "pool");
  TORCH_CHECK_VALUE(n <= INT32_MAX, "k: too many tokens");
  const int32_t* cu = index_of(cu_new, "cu_new", (int64_t)t.c.n_seqs + 1, t.device);
  const int32_t* pos = index_of(positions, "positions", n, t.device);
  const c10::cuda::OptionalCUDAGuard guard(t.device);
  const kv_rows kr = rows_of(k), vr = rows_of(v);
  check_apart(bytes_of(t.pool), "pool", bytes_of(k, kr), "k");
  check_apart(bytes_of(t.pool), "pool", bytes_of(v, vr), "v");
  check_status(kv_append_tokens(&t.c, &kr, &vr, (int)n, cu, rope ? rope->handle : nullptr, pos, stream_of(t)),
               "kv_append_tokens");
  written(t.pool);
}

// decode, and decode_append where k and v are given.
at::Tensor decode(Tokens& t, const c10::optional<at::Tensor>& k, const c10::optional<at::Tensor>& v, const at::Tensor& q,
                  const Rope* rope, const c10::optional<at::Tensor>& positions, const c10::optional<at::Tensor>& given,
                  const c10::optional<double>& scale, int64_t window, const c10::optional<at::Tensor>& workspace) {
  TORCH_CHECK_VALUE(q.dim() == 3, "q: shape ", shown(q.sizes()), ", expected [n_seqs, q heads, head_dim]");
  if (k) check_new(t, *k, *v, t.c.n_seqs);
  check_no_gradient(t.pool, "pool");
  const int64_t heads = q.size(1);
  const int64_t shape[] = {t.c.n_seqs, heads, t.c.head_dim};
  check_tensor(q, "q", shape, t.dtype, t.device, false);
  check_no_gradient(q, "q");
  TORCH_CHECK_VALUE(heads >= 1 && heads % t.c.num_heads == 0, "q: ", heads, " heads, expected a multiple of the pool's ",
                    t.c.num_heads);
  if (given) {
    check_tensor(*given, "out", shape, t.dtype, t.device, true);
    check_written(*given, "out");
  }
  const float s = scale ? (float)*scale : 0.f;
  TORCH_CHECK_VALUE(!scale || s != 0, "scale: 0 would weigh all tokens alike");
  TORCH_CHECK_VALUE(window >= INT32_MIN && window <= INT32_MAX, "window: out of range");
  if (workspace)
    TORCH_CHECK_VALUE(workspace->device() == t.device && workspace->is_contiguous(),
                      "workspace: must be contiguous, on the pool's device");
  const int32_t* pos = index_of(positions, "positions", t.c.n_seqs, t.device);
  const c10::cuda::OptionalCUDAGuard guard(t.device);
  const cudaStream_t stream = stream_of(t);
  at::Tensor out = given ? *given : empty_rows(q), ws;
  if (workspace) {
    ws = *workspace;
  } else if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
    ws = new_workspace(t, heads);   // the graph's own, prepared by each replay
  } else {
    at::Tensor& kept = t.workspaces[{stream, heads}];
    if (!kept.defined()) kept = new_workspace(t, heads);
    ws = kept;
  }
  const kv_rows qr = rows_of(q);
  if (given) {
    const pkv::RowSet to = bytes_of(out);
    check_apart(to, "out", bytes_of(t.pool), "pool");
    if (!(out.data_ptr() == qr.data && q.is_contiguous())) check_apart(to, "out", bytes_of(q, qr), "q");
  }
  if (k) {
    const kv_rows kr = rows_of(*k), vr = rows_of(*v);
    const pkv::RowSet kb = bytes_of(*k, kr), vb = bytes_of(*v, vr), pool = bytes_of(t.pool);
    check_apart(pool, "pool", kb, "k");
    check_apart(pool, "pool", vb, "v");
    check_apart(pool, "pool", bytes_of(q, qr), "q");
    if (given) check_apart(bytes_of(out), "out", kb, "k"), check_apart(bytes_of(out), "out", vb, "v");
    check_status(kv_decode_append(&t.c, &kr, &vr, &qr, (int)heads, rope ? rope->handle : nullptr, pos, s, (int)window,
                                  out.data_ptr(), ws.data_ptr(), ws.nbytes(), stream),
                 "kv_decode_append");
    written(t.pool);
  } else {
    check_status(kv_decode(&t.c, &qr, (int)heads, s, (int)window, out.data_ptr(), ws.data_ptr(), ws.nbytes(), stream),
                 "kv_decode");
  }
  if (given) written(out);
  return out;
}

// ---------------------------------------------------------------- Python
constexpr const char* kRopeName = "paged_kv_cache_frame_b200.rope";
constexpr const char* kTokensName = "paged_kv_cache_frame_b200.tokens";

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
c10::optional<at::Tensor> optional_tensor(PyObject* o, const char* name) {
  return o == Py_None ? c10::nullopt : c10::optional<at::Tensor>(tensor(o, name));
}
c10::intrusive_ptr<Rope>* rope_slot(PyObject* o) {
  if (o == Py_None) return nullptr;
  auto* p = static_cast<c10::intrusive_ptr<Rope>*>(PyCapsule_GetPointer(o, kRopeName));
  if (!p) throw python_error();
  return p;
}
Tokens& tokens_of(PyObject* o) {
  auto* p = static_cast<Tokens*>(PyCapsule_GetPointer(o, kTokensName));
  if (!p) throw python_error();
  return *p;
}
int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

// Runs f, an error of the library as KVError.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const LibraryError& e) {
    PyObject* r = PyObject_CallFunction(g_check, "is", e.status, e.where);
    if (r) {   // check() raises
      Py_DECREF(r);
      PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* expect(Py_ssize_t got, Py_ssize_t want) {
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
  return nullptr;
}

PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (handle), which the capsule then owns
  if (n != 1) return expect(n, 1);
  return guarded([&]() -> PyObject* {
    void* h = PyLong_AsVoidPtr(a[0]);
    if (!h && PyErr_Occurred()) throw python_error();
    auto* p = new c10::intrusive_ptr<Rope>(c10::make_intrusive<Rope>(static_cast<kv_rope_t*>(h)));
    return PyCapsule_New(p, kRopeName, [](PyObject* o) {
      delete static_cast<c10::intrusive_ptr<Rope>*>(PyCapsule_GetPointer(o, kRopeName));
    });
  });
}

PyObject* py_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (rope, x, positions, out, inverse)
  if (n != 5) return expect(n, 5);
  return guarded([&]() -> PyObject* {
    const auto* slot = rope_slot(a[0]);
    TORCH_CHECK_TYPE(slot, "rope: None");
    const auto& rope = *slot;
    const at::Tensor& x = tensor(a[1], "x");
    const at::Tensor& positions = tensor(a[2], "positions");
    const auto out = optional_tensor(a[3], "out");
    const int inverse = PyObject_IsTrue(a[4]);
    if (inverse < 0) throw python_error();
    at::Tensor y;
    {
      pybind11::gil_scoped_release release;
      if (at::GradMode::is_enabled() && (x.requires_grad() || (out && out->requires_grad()))) {
        TORCH_CHECK_VALUE(!out, "rotate: out is not for a call that records a gradient");
        y = Rotation::apply(x, positions, rope, inverse != 0);
      } else {
        y = rotate(rope, x, positions, out, inverse != 0);
      }
    }
    return THPVariable_Wrap(std::move(y));
  });
}

PyObject* py_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (pool, tables, lens, read_only)
  if (n != 4) return expect(n, 4);
  return guarded([&]() -> PyObject* {
    const at::Tensor& pool = tensor(a[0], "pool");
    TORCH_CHECK_VALUE(pool.dim() == 5 && pool.size(1) == 2, "pool: shape ", shown(pool.sizes()),
                      ", expected [max_pages, 2, page_size, heads, head_dim]");
    TORCH_CHECK_VALUE(pool.scalar_type() == at::kBFloat16 || pool.scalar_type() == at::kHalf, "pool: dtype ",
                      pool.scalar_type(), ", expected bfloat16 or float16");
    check_device(pool, "pool");
    check_tensor(pool, "pool", pool.sizes(), pool.scalar_type(), pool.device(), true);
    const at::Tensor &tables = tensor(a[1], "tables"), &lens = tensor(a[2], "lens");
    TORCH_CHECK_VALUE(tables.dim() == 2, "tables: shape ", shown(tables.sizes()), ", expected [n_seqs, width]");
    const int64_t seqs = tables.size(0), width = tables.size(1);
    check_tensor(tables, "tables", tables.sizes(), at::kInt, pool.device(), false);
    check_tensor(lens, "lens", {seqs}, at::kInt, pool.device(), true);
    for (int64_t s : {pool.size(0), pool.size(2), pool.size(3), pool.size(4), seqs, width})
      TORCH_CHECK_VALUE(s <= INT32_MAX, "pool, tables: too large");
    const int read_only = PyObject_IsTrue(a[3]);
    if (read_only < 0) throw python_error();
    const c10::cuda::OptionalCUDAGuard guard(pool.device());
    at::Tensor error = at::zeros({1}, at::TensorOptions().dtype(at::kInt).device(pool.device()));
    kv_tokens c;
    c.pool = pool.data_ptr();
    c.tables = tables.data_ptr<int32_t>();
    c.lens = lens.data_ptr<int32_t>();
    c.error = reinterpret_cast<uint32_t*>(error.data_ptr<int32_t>());
    c.table_stride = seqs > 1 ? tables.stride(0) : width;
    c.max_pages = (int)pool.size(0);
    c.page_size = (int)pool.size(2);
    c.num_heads = (int)pool.size(3);
    c.head_dim = (int)pool.size(4);
    c.dtype = dtype_code(pool.scalar_type());
    c.table_width = (int)width;
    c.n_seqs = (int)seqs;
    auto* t = new Tokens{c, pool, tables, lens, error, read_only != 0, pool.scalar_type(), pool.device(), {}, {}};
    return PyCapsule_New(t, kTokensName,
                         [](PyObject* o) { delete static_cast<Tokens*>(PyCapsule_GetPointer(o, kTokensName)); });
  });
}

PyObject* py_address(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (tokens): of its kv_tokens
  if (n != 1) return expect(n, 1);
  return guarded([&]() -> PyObject* { return PyLong_FromVoidPtr(&tokens_of(a[0]).c); });
}

PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (tokens, k, v, cu_new, rope, positions)
  if (n != 6) return expect(n, 6);
  return guarded([&]() -> PyObject* {
    const auto* rope = rope_slot(a[4]);
    append(tokens_of(a[0]), tensor(a[1], "k"), tensor(a[2], "v"), optional_tensor(a[3], "cu_new"), rope ? rope->get() : nullptr,
           optional_tensor(a[5], "positions"));
    Py_RETURN_NONE;
  });
}

PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // (tokens, k, v, q, rope, positions, out, scale, window, workspace); k and v None: no append
  if (n != 10) return expect(n, 10);
  return guarded([&]() -> PyObject* {
    const auto* rope = rope_slot(a[4]);
    c10::optional<double> scale;
    if (a[7] != Py_None) {
      scale = PyFloat_AsDouble(a[7]);
      if (PyErr_Occurred()) throw python_error();
    }
    return THPVariable_Wrap(decode(tokens_of(a[0]), optional_tensor(a[1], "k"), optional_tensor(a[2], "v"), tensor(a[3], "q"),
                                   rope ? rope->get() : nullptr, optional_tensor(a[5], "positions"),
                                   optional_tensor(a[6], "out"), scale, integer(a[8]), optional_tensor(a[9], "workspace")));
  });
}

PyObject* py_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (tokens, q_heads)
  if (n != 2) return expect(n, 2);
  return guarded([&]() -> PyObject* {
    Tokens& t = tokens_of(a[0]);
    const c10::cuda::OptionalCUDAGuard guard(t.device);
    return THPVariable_Wrap(new_workspace(t, integer(a[1])));
  });
}

PyObject* py_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (tokens, q_heads)
  if (n != 2) return expect(n, 2);
  return guarded([&]() -> PyObject* {
    Tokens& t = tokens_of(a[0]);
    const c10::cuda::OptionalCUDAGuard guard(t.device);
    return PyLong_FromSize_t(workspace_bytes(t, integer(a[1])));
  });
}

PyObject* py_check(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (tokens): synchronises
  if (n != 1) return expect(n, 1);
  return guarded([&]() -> PyObject* {
    Tokens& t = tokens_of(a[0]);
    pybind11::gil_scoped_release release;
    const c10::cuda::OptionalCUDAGuard guard(t.device);
    check_status(kv_tokens_check(&t.c, stream_of(t)), "kv_tokens_check");
    Py_RETURN_NONE;
  });
}

PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {   // (check)
  if (n != 1) return expect(n, 1);
  Py_INCREF(a[0]);
  Py_XSETREF(g_check, a[0]);
  Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("init", py_init), FAST("rope", py_rope), FAST("rotate", py_rotate), FAST("tokens", py_tokens),
                         FAST("address", py_address), FAST("append", py_append), FAST("decode", py_decode),
                         FAST("workspace", py_workspace), FAST("workspace_bytes", py_workspace_bytes),
                         FAST("check", py_check), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tokens() { return PyModule_Create(&module); }
