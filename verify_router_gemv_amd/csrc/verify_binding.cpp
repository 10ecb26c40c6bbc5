// Python binding of the verify-round operators (module _verify_ops): argument checks and marshalling only.
//
// These calls come once or twice per layer of every round, with kernels of a few microseconds, so the
// checks of their eight to twelve tensors are done here, on the tensors' own records (about 3 us a call;
// the same checks and the packing of the argument struct took 11 us from Python).  Every argument is
// positional; verify_ops.py has the signatures and their documentation.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "verify_ops.h"

namespace {

PyObject* g_error = nullptr;  // binding.MoeRoundError(status, what, hip_error)

struct TypeFault { std::string what; };
struct ValueFault { std::string what; };
struct Raised {};  // a Python exception is set

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

enum Kind { kFloats = 1, kCache = 2, kI32 = 4, kI64 = 8, kF32 = 16 };

bool is_kind(at::ScalarType t, int kinds) {
  switch (t) {
    case at::kFloat: return kinds & (kFloats | kF32);
    case at::kBFloat16: case at::kHalf: return kinds & (kFloats | kCache);
    case at::kInt: return kinds & kI32;
    case at::kLong: return kinds & kI64;
    default: return false;
  }
}

int type_code(at::ScalarType t) { return t == at::kFloat ? VERIFY_F32 : t == at::kBFloat16 ? VERIFY_BF16 : VERIFY_F16; }

// The GPU that a call's tensors live on: the first tensor's.
struct Call {
  int device = -1;

  const at::Tensor& tensor(PyObject* o, const char* name, int kinds, int64_t ndim) {
    if (!THPVariable_Check(o)) throw TypeFault{std::string(name) + " must be a torch tensor"};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!is_kind(t.scalar_type(), kinds) || t.layout() != at::kStrided)
      throw TypeFault{std::string(name) + ": unsupported dtype or layout (" + c10::toString(t.scalar_type()) + ")"};
    if (t.dim() != ndim)
      throw ValueFault{std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, not " + std::to_string(ndim)};
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device))
      throw ValueFault{std::string(name) + " must live on the GPU, with the other tensors (" + t.device().str() + ")"};
    device = static_cast<int>(t.get_device());
    return t;
  }
  const at::Tensor& like(PyObject* o, const char* name, const at::Tensor& as, bool shape) {
    const at::Tensor& t = tensor(o, name, kFloats, as.dim());
    if (t.scalar_type() != as.scalar_type())
      throw TypeFault{std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + " != " + c10::toString(as.scalar_type())};
    if (shape) expect(t, name, as.sizes());
    return t;
  }
  static void expect(const at::Tensor& t, const char* name, at::IntArrayRef s) {
    if (t.sizes() != s) throw ValueFault{std::string(name) + ": shape " + shape_text(t.sizes()) + " != " + shape_text(s)};
  }
  template <typename P>
  P vector(PyObject* o, const char* name, int64_t length, int kind) {
    const at::Tensor& t = tensor(o, name, kind, 1);
    if (t.size(0) != length)
      throw ValueFault{std::string(name) + ": length " + std::to_string(t.size(0)) + " != " + std::to_string(length)};
    if (length > 1 && t.stride(0) != 1) throw ValueFault{std::string(name) + " must be contiguous"};
    return static_cast<P>(t.data_ptr());
  }
  template <typename P>
  P maybe(PyObject* o, const char* name, int64_t length, int kind) {
    return o == Py_None ? nullptr : vector<P>(o, name, length, kind);
  }
  at::Tensor empty(at::IntArrayRef s, at::ScalarType type) const {
    return at::empty(s, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

// Strides but the last dimension's, which must be contiguous. A dimension of one element has none of its
// own (torch may report any): 0.
void strides(const at::Tensor& t, const char* name, int64_t* a, int64_t* b, int64_t* c = nullptr) {
  const int64_t n = t.dim();
  if (t.size(n - 1) > 1 && t.stride(n - 1) != 1) throw ValueFault{std::string(name) + ": the last dimension must be contiguous"};
  int64_t* out[3] = {a, b, c};
  for (int64_t i = 0; i + 1 < n; ++i) *out[i] = t.size(i) > 1 ? t.stride(i) : 0;
}
int64_t row_stride(const at::Tensor& t, const char* name) {
  if (t.size(1) > 1 && t.stride(1) != 1) throw ValueFault{std::string(name) + ": the last dimension must be contiguous"};
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// A size for a 32-bit field.
int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) throw ValueFault{std::string(name) + ": " + std::to_string(n) + " is too many"};
  return static_cast<int32_t>(n);
}

int64_t number(PyObject* o, const char* name, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < lo || v > hi) throw ValueFault{std::string(name) + ": " + std::to_string(v) + " is out of range"};
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

void check(int64_t status, const char* what) {
  if (status >= 0) return;
  PyObject* e = PyObject_CallFunction(g_error, "isi", static_cast<int>(status), what,
                                      status == MOE_ERR_HIP ? verify_last_hip_error() : 0);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Makes the call's device current while it lives, if another one is.
struct On {
  c10::OptionalDeviceGuard guard;
  explicit On(const Call& c) {
    if (c.device != c10::hip::current_device())
      guard.reset_device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
  }
};

// A contiguous piece of a contiguous tensor, of the same type (what narrow and view give, without their
// dispatch: the small tensors of one call share one allocation).
at::Tensor piece(const at::Tensor& of, int64_t from, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(of.storage()), of.key_set(),
                                                          of.dtype());
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(of.storage_offset() + from);
  impl->set_sizes_contiguous(sizes);
  return t;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
// A new reference to `o`, or the tensor made in its place.
PyObject* given(PyObject* o, const at::Tensor& made) {
  if (made.defined()) return wrap(made);
  Py_INCREF(o);
  return o;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const TypeFault& e) {
    PyErr_SetString(PyExc_TypeError, e.what.c_str());
  } catch (const ValueFault& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Raised&) {
  } catch (...) {  // torch's own (an allocation that failed, for instance)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (cached, rows, table, free_pages, page_size, total_rows, parents, free_head, row_start, slots, positions,
//  masks, counts) -> the last five; None: made here (masks only with parents)
PyObject* round_slots(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c;
    verify_slots_args a{};
    a.struct_bytes = sizeof(a);
    const at::Tensor& table = c.tensor(o[2], "table", kI32, 2);
    const int64_t B = table.size(0), W = table.size(1), N = number(o[5], "total_rows", 0);
    a.cached = c.vector<int32_t*>(o[0], "cached", B, kI32);
    a.rows = c.vector<int32_t*>(o[1], "rows", B, kI32);
    a.table = static_cast<int32_t*>(table.data_ptr());
    a.table_stride = row_stride(table, "table");
    if (a.table_stride < W) throw ValueFault{"table: its rows overlap"};
    const at::Tensor& free_pages = c.tensor(o[3], "free_pages", kI32, 1);
    a.free_pages = c.vector<int32_t*>(o[3], "free_pages", free_pages.size(0), kI32);
    a.n_free = size32(free_pages.size(0), "free_pages");
    a.page_size = static_cast<int32_t>(number(o[4], "page_size"));
    a.free_head = c.maybe<int32_t*>(o[7], "free_head", 1, kI32);
    a.parents = c.maybe<int32_t*>(o[6], "parents", N, kI32);
    a.n_requests = size32(B, "requests");
    a.width = size32(W, "table columns");
    a.total_rows = static_cast<int32_t>(N);
    const bool tree = o[6] != Py_None;
    at::Tensor made[5];
    if (o[8] == Py_None) {
      const at::Tensor buf = c.empty({B + 3 + 2 * N}, at::kInt);
      made[1] = piece(buf, 0, {N});
      made[2] = piece(buf, N, {N});
      made[0] = piece(buf, 2 * N, {B + 1});
      made[4] = piece(buf, 2 * N + B + 1, {2});
      if (tree) made[3] = c.empty({N}, at::kLong);
      a.slots = static_cast<int32_t*>(buf.data_ptr());
      a.positions = a.slots + N;
      a.row_start = a.positions + N;
      a.counts = a.row_start + B + 1;
      a.masks = tree ? static_cast<int64_t*>(made[3].data_ptr()) : nullptr;
    } else {
      if ((o[11] != Py_None) != tree) throw ValueFault{"out.masks must be given exactly when parents are"};
      a.row_start = c.vector<int32_t*>(o[8], "out.row_start", B + 1, kI32);
      a.slots = c.vector<int32_t*>(o[9], "out.slots", N, kI32);
      a.positions = c.vector<int32_t*>(o[10], "out.positions", N, kI32);
      a.masks = c.maybe<int64_t*>(o[11], "out.masks", N, kI64);
      a.counts = c.vector<int32_t*>(o[12], "out.counts", 2, kI32);
    }
    {
      const On on(c);
      check(verify_round_slots(&a, c.stream()), "verify_round_slots");
    }
    PyObject* out = PyTuple_New(5);
    if (!out) return nullptr;
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(out, i, given(o[8 + i], made[i]));
    return out;
  });
}

// (q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out, q_weight, k_weight, eps, interleaved) -> q_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c;
    verify_rope_args a{};
    a.struct_bytes = sizeof(a);
    const at::Tensor& q = c.tensor(o[0], "q", kFloats, 3);
    const at::Tensor& k = c.like(o[1], "k", q, false);
    const at::Tensor& v = c.like(o[2], "v", q, false);
    const int64_t T = q.size(0), heads = q.size(1), D = q.size(2), kv = k.size(1);
    Call::expect(k, "k", {T, kv, D});
    Call::expect(v, "v", {T, kv, D});
    const at::Tensor& kc = c.tensor(o[6], "k_cache", kCache, 4);
    Call::expect(kc, "k_cache", {kc.size(0), kv, kc.size(2), D});
    const at::Tensor& vc = c.like(o[7], "v_cache", kc, true);
    if (q.scalar_type() != at::kFloat && q.scalar_type() != kc.scalar_type())
      throw TypeFault{"q, k, v: neither float32 nor the cache's dtype"};
    at::Tensor made;
    if (o[8] == Py_None) made = c.empty({T, heads, D}, kc.scalar_type());
    const at::Tensor& out = made.defined() ? made : c.tensor(o[8], "q_out", kCache, 3);
    if (out.scalar_type() != kc.scalar_type()) throw TypeFault{"q_out: not the cache's dtype"};
    Call::expect(out, "q_out", q.sizes());
    const at::Tensor& f = c.tensor(o[5], "inv_freq", kF32, 1);
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    a.v = v.data_ptr();
    a.q_out = out.data_ptr();
    a.k_cache = kc.data_ptr();
    a.v_cache = vc.data_ptr();
    a.positions = c.vector<int32_t*>(o[3], "positions", T, kI32);
    a.slots = c.vector<int32_t*>(o[4], "slots", T, kI32);
    a.inv_freq = c.vector<float*>(o[5], "inv_freq", f.size(0), kF32);
    a.q_weight = c.maybe<float*>(o[9], "q_weight", D, kF32);
    a.k_weight = c.maybe<float*>(o[10], "k_weight", D, kF32);
    strides(q, "q", &a.q_row, &a.q_head);
    strides(k, "k", &a.k_row, &a.k_head);
    strides(v, "v", &a.v_row, &a.v_head);
    strides(out, "q_out", &a.o_row, &a.o_head);
    strides(kc, "k_cache", &a.kc_page, &a.kc_head, &a.kc_token);
    strides(vc, "v_cache", &a.vc_page, &a.vc_head, &a.vc_token);
    a.n_pages = kc.size(0);
    a.n_rows = size32(T, "rows");
    a.heads = size32(heads, "heads");
    a.kv_heads = size32(kv, "kv_heads");
    a.dim = size32(D, "head size");
    a.page_size = size32(kc.size(2), "page size");
    a.n_freq = size32(f.size(0), "inv_freq");
    a.in_type = type_code(q.scalar_type());
    a.cache_type = type_code(kc.scalar_type());
    a.eps = real(o[11]);
    a.interleaved = PyObject_IsTrue(o[12]);
    if (a.interleaved < 0) return nullptr;
    {
      const On on(c);
      check(verify_qk_norm_rope(&a, c.stream()), "verify_qk_norm_rope");
    }
    return given(o[8], made);
  });
}

// (q, k_cache, v_cache, table, cached, row_start, out, masks, max_rows, scale) -> out
PyObject* tree_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    verify_attention_args a{};
    a.struct_bytes = sizeof(a);
    const at::Tensor& q = c.tensor(o[0], "q", kCache, 3);
    const int64_t T = q.size(0), heads = q.size(1), D = q.size(2);
    const at::Tensor& kc = c.tensor(o[1], "k_cache", kCache, 4);
    if (kc.scalar_type() != q.scalar_type()) throw TypeFault{"k_cache: not q's dtype"};
    Call::expect(kc, "k_cache", {kc.size(0), kc.size(1), kc.size(2), D});
    const at::Tensor& vc = c.like(o[2], "v_cache", kc, true);
    const at::Tensor& table = c.tensor(o[3], "table", kI32, 2);
    const int64_t B = table.size(0);
    at::Tensor made;
    if (o[6] == Py_None) made = c.empty({T, heads, D}, q.scalar_type()).zero_();
    const at::Tensor& out = made.defined() ? made : c.like(o[6], "out", q, true);
    a.q = q.data_ptr();
    a.k_cache = kc.data_ptr();
    a.v_cache = vc.data_ptr();
    a.table = static_cast<int32_t*>(table.data_ptr());
    a.table_stride = row_stride(table, "table");
    a.cached = c.vector<int32_t*>(o[4], "cached", B, kI32);
    a.row_start = c.vector<int32_t*>(o[5], "row_start", B + 1, kI32);
    a.masks = c.maybe<int64_t*>(o[7], "masks", T, kI64);
    a.out = out.data_ptr();
    strides(q, "q", &a.q_row, &a.q_head);
    strides(out, "out", &a.o_row, &a.o_head);
    strides(kc, "k_cache", &a.kc_page, &a.kc_head, &a.kc_token);
    strides(vc, "v_cache", &a.vc_page, &a.vc_head, &a.vc_token);
    a.n_pages = kc.size(0);
    a.n_rows = size32(T, "rows");
    a.n_requests = size32(B, "requests");
    a.heads = size32(heads, "heads");
    a.kv_heads = size32(kc.size(1), "kv_heads");
    a.dim = size32(D, "head size");
    a.page_size = size32(kc.size(2), "page size");
    a.width = size32(table.size(1), "table columns");
    a.max_rows = o[8] == Py_None ? static_cast<int32_t>(T < 1 ? 1 : T < VERIFY_MAX_TREE_ROWS ? T : VERIFY_MAX_TREE_ROWS)
                                 : static_cast<int32_t>(number(o[8], "max_rows"));
    a.type = type_code(q.scalar_type());
    a.scale = o[9] == Py_None ? static_cast<float>(1.0 / sqrt(static_cast<double>(D))) : real(o[9]);
    const int64_t need = verify_tree_attention_workspace(&a);
    check(need, "verify_tree_attention");
    at::Tensor work;
    if (need) work = c.empty({need}, at::kByte);
    {
      const On on(c);
      check(verify_tree_attention(&a, need ? work.data_ptr() : nullptr, need, c.stream()), "verify_tree_attention");
    }
    return given(o[6], made);
  });
}

// (logits, tokens, top) -> (logprobs, entropy, top_ids, top_logprobs)
PyObject* token_logprobs(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Call c;
    verify_logprobs_args a{};
    a.struct_bytes = sizeof(a);
    const at::Tensor& x = c.tensor(o[0], "logits", kFloats, 2);
    const int64_t T = x.size(0), V = x.size(1);
    a.logits = x.data_ptr();
    a.row_stride = row_stride(x, "logits");
    int64_t N = 0;
    if (o[1] != Py_None) {
      const at::Tensor& tokens = c.tensor(o[1], "tokens", kI32 | kI64, 2);
      N = tokens.size(1);
      Call::expect(tokens, "tokens", {T, N});
      if (!tokens.is_contiguous()) throw ValueFault{"tokens must be contiguous"};
      if (N) a.tokens = tokens.data_ptr();
      a.tokens_64 = N && tokens.scalar_type() == at::kLong;
    }
    const int64_t most = V < VERIFY_MAX_ALTERNATIVES ? V : VERIFY_MAX_ALTERNATIVES, top = number(o[2], "top");
    if (top < 0 || top > most) throw ValueFault{"top must be between 0 and " + std::to_string(most)};
    a.n_rows = size32(T, "rows");
    a.vocab = size32(V, "vocabulary");
    a.n_tokens = size32(N, "tokens");
    a.top = static_cast<int32_t>(top);
    a.type = type_code(x.scalar_type());
    const at::Tensor buf = c.empty({T * (N + 1 + top)}, at::kFloat);
    const at::Tensor ids = c.empty({T, top}, at::kInt);
    a.logprobs = N ? static_cast<float*>(buf.data_ptr()) : nullptr;
    a.entropy = static_cast<float*>(buf.data_ptr()) + T * N;
    a.top_logprobs = a.entropy + T;
    a.top_ids = static_cast<int32_t*>(ids.data_ptr());
    const int64_t need = verify_token_logprobs_workspace(&a);
    check(need, "verify_token_logprobs");
    at::Tensor work;
    if (need) work = c.empty({need}, at::kByte);
    {
      const On on(c);
      check(verify_token_logprobs(&a, need ? work.data_ptr() : nullptr, need, c.stream()), "verify_token_logprobs");
    }
    PyObject* out = PyTuple_New(4);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, wrap(piece(buf, 0, {T, N})));
    PyTuple_SET_ITEM(out, 1, wrap(piece(buf, T * N, {T})));
    PyTuple_SET_ITEM(out, 2, wrap(ids));
    PyTuple_SET_ITEM(out, 3, wrap(piece(buf, T * (N + 1), {T, top})));
    return out;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef methods[] = {
    {"round_slots", fast<round_slots>(), METH_FASTCALL, nullptr},
    {"qk_norm_rope", fast<qk_norm_rope>(), METH_FASTCALL, nullptr},
    {"tree_attention", fast<tree_attention>(), METH_FASTCALL, nullptr},
    {"token_logprobs", fast<token_logprobs>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_verify_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__verify_ops() { return PyModule_Create(&module); }
