// Python calls of the decoder-block operators (awq_block.h): one function per operator that
// checks its tensors, forms the argument structure and calls the C entry point on PyTorch's
// current stream. A decode step makes these calls for every layer, and their kernels take a
// few microseconds: checked and marshalled in Python, a call costs 9 to 13 us of host time,
// here 5 to 9 (MI355X host). block.py holds the signatures and the documentation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/awq_block.h"

namespace {

PyObject *g_stream = nullptr;     // device number -> the current stream's handle
PyObject *g_workspace = nullptr;  // (bytes, device number) -> tensor
PyObject *g_error = nullptr;      // AwqError(status, function)

struct Refused {};  // thrown with a Python error set

// A reference that ends with its scope
struct Owned {
  PyObject* object = nullptr;
  ~Owned() { Py_XDECREF(object); }
};

[[noreturn]] void refuse(PyObject* kind, const char* format, const char* name) {
  PyErr_Format(kind, format, name);
  throw Refused{};
}

// None is allowed and gives NULL where `optional`
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}

// What the tensors of one call share.
struct Call {
  int64_t device;
  at::ScalarType dtype;

  explicit Call(const at::Tensor& t, const char* name) : device(-1), dtype(t.scalar_type()) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a device tensor", name);
    device = t.get_device();
  }
  void on_device(const at::Tensor& t, const char* name) const {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a device tensor", name);
    if (t.get_device() != device) refuse(PyExc_ValueError, "%s is on another device than the other operands", name);
  }
  int32_t element_type(const char* name) const {
    if (dtype == at::kHalf) return AWQ_DT_F16;
    if (dtype == at::kBFloat16) return AWQ_DT_BF16;
    refuse(PyExc_TypeError, "%s must be float16 or bfloat16", name);
  }
  // a contiguous tensor of a type and shape (a dimension of -1 is not looked at)
  template <typename T>
  T* vector(const at::Tensor* t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    if (t == nullptr) return nullptr;
    on_device(*t, name);
    if (t->scalar_type() != type) refuse(PyExc_TypeError, "%s has the wrong type", name);
    bool same = t->dim() == static_cast<int64_t>(shape.size());
    for (size_t i = 0; same && i < shape.size(); ++i)
      same = shape.begin()[i] < 0 || t->size(static_cast<int64_t>(i)) == shape.begin()[i];
    if (!same) refuse(PyExc_ValueError, "%s has the wrong shape", name);
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T*>(t->data_ptr());
  }
  // a packed operand [tokens, heads, D]; a dimension of one has no stride that matters (one
  // token cut out of a long tensor keeps that tensor's)
  template <typename T>
  T* packed(const at::Tensor& t, const char* name, int64_t& token, int64_t& head) const {
    on_device(t, name);
    if (t.scalar_type() != dtype) refuse(PyExc_TypeError, "%s has another type than the other operands", name);
    if (t.dim() != 3) refuse(PyExc_ValueError, "%s must be [tokens, heads, head_dim]", name);
    if (t.stride(2) != 1) refuse(PyExc_ValueError, "the elements of a head of %s must be contiguous", name);
    head = t.size(1) > 1 ? t.stride(1) : t.size(2);
    token = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
    return static_cast<T*>(t.data_ptr());
  }
  // a paged cache [pages, kv_heads, page_size, D] of two tensors with one layout
  void cache(const at::Tensor& k, const at::Tensor& v, int64_t heads, int64_t d, int64_t& pages,
             int32_t& page_size, int64_t& page, int64_t& head, int64_t& slot) const {
    on_device(k, "k_cache");
    on_device(v, "v_cache");
    if (k.scalar_type() != dtype) refuse(PyExc_TypeError, "%s has another type than the other operands", "k_cache");
    if (v.scalar_type() != dtype) refuse(PyExc_TypeError, "%s has another type than the other operands", "v_cache");
    if (k.dim() != 4 || k.size(1) != heads || k.size(3) != d)
      refuse(PyExc_ValueError, "%s must be [pages, kv_heads, page_size, head_dim]", "k_cache");
    bool same = k.sizes() == v.sizes();
    for (int i = 0; same && i < 4; ++i) same = k.size(i) <= 1 || k.stride(i) == v.stride(i);
    if (!same) refuse(PyExc_ValueError, "%s must have k_cache's shape and layout", "v_cache");
    if (k.stride(3) != 1) refuse(PyExc_ValueError, "the elements of a slot of %s must be contiguous", "k_cache");
    if (k.size(2) > INT32_MAX) refuse(PyExc_ValueError, "%s has too large pages", "k_cache");
    pages = k.size(0);
    page_size = static_cast<int32_t>(k.size(2));
    page = pages > 1 ? k.stride(0) : 0;
    head = heads > 1 ? k.stride(1) : 0;
    slot = page_size > 1 ? k.stride(2) : d;
  }
  hipStream_t stream() const {
    PyObject* index = PyLong_FromLongLong(device);
    PyObject* handle = index == nullptr ? nullptr : PyObject_CallOneArg(g_stream, index);
    Py_XDECREF(index);
    if (handle == nullptr) throw Refused{};
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (p == nullptr && PyErr_Occurred()) throw Refused{};
    return static_cast<hipStream_t>(p);
  }
};

int32_t count(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(PyExc_ValueError, "%s has too large a dimension", name);
  return static_cast<int32_t>(n);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

template <typename F>
void run(const char* name, F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  if (rc != AWQ_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "is", rc, name);
    if (e != nullptr) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Refused{};
  }
}

// the given output (checked by the caller), or a new contiguous one like `ref`
at::Tensor output(PyObject* o, const char* name, const at::Tensor& ref) {
  if (o == Py_None) return at::empty(ref.sizes(), ref.options());
  const at::Tensor& t = *tensor(o, name);
  if (t.sizes() != ref.sizes()) refuse(PyExc_ValueError, "%s has the wrong shape", name);
  return t;
}

void want(Py_ssize_t got, Py_ssize_t n) {
  if (got != n) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw Refused{};
  }
}

// q, positions, inv_freq, k, v, k_cache, v_cache, slots, interleaved, inverse, scale, q_out, k_out
PyObject* rope(PyObject* const* in, Py_ssize_t n) {
  want(n, 13);
  const at::Tensor *q = tensor(in[0], "q", true), *k = tensor(in[3], "k", true), *v = tensor(in[4], "v", true);
  const at::Tensor *kc = tensor(in[5], "k_cache", true), *vc = tensor(in[6], "v_cache", true);
  const at::Tensor *positions = tensor(in[1], "positions"), *freq = tensor(in[2], "inv_freq");
  const at::Tensor* slots = tensor(in[7], "slots", true);
  if (q == nullptr && k == nullptr) refuse(PyExc_ValueError, "%s or k is required", "q");
  if ((kc == nullptr) != (vc == nullptr)) refuse(PyExc_ValueError, "%s and v_cache go together", "k_cache");
  if (k == nullptr && (kc != nullptr || in[12] != Py_None)) refuse(PyExc_ValueError, "a cache or k_out needs %s", "k");
  if (kc != nullptr && (v == nullptr || slots == nullptr)) refuse(PyExc_ValueError, "a cache needs v and %s", "slots");
  const at::Tensor& ref = q != nullptr ? *q : *k;
  const char* ref_name = q != nullptr ? "q" : "k";
  const Call call(ref, ref_name);
  awq_rope_args a{};
  a.dtype = call.element_type(ref_name);
  if (ref.dim() != 3) refuse(PyExc_ValueError, "%s must be [tokens, heads, head_dim]", ref_name);
  const int64_t d = ref.size(2);
  a.tokens = ref.size(0);
  a.head_dim = count(d, ref_name);
  a.positions = call.vector<int32_t>(positions, "positions", at::kInt, {a.tokens});
  a.inv_freq = call.vector<float>(freq, "inv_freq", at::kFloat, {-1});
  a.slots = call.vector<int64_t>(slots, "slots", at::kLong, {a.tokens});
  if (2 * freq->size(0) > d) refuse(PyExc_ValueError, "%s has more pairs than the head", "inv_freq");
  a.rot_dim = count(2 * freq->size(0), "inv_freq");
  a.interleaved = truth(in[8]);
  a.inverse = truth(in[9]);
  a.scale = static_cast<float>(number(in[10]));
  at::Tensor q_out, k_out;
  if (q != nullptr) {
    a.q = call.packed<void>(*q, "q", a.q_token, a.q_head);
    a.q_heads = count(q->size(1), "q");
    q_out = output(in[11], "q_out", *q);
    a.q_out = call.packed<void>(q_out, "q_out", a.qo_token, a.qo_head);
  }
  if (k != nullptr) {
    a.k = call.packed<void>(*k, "k", a.k_token, a.k_head);
    a.kv_heads = count(k->size(1), "k");
    if (k->size(0) != a.tokens || k->size(2) != d) refuse(PyExc_ValueError, "%s must have q's tokens and head size", "k");
    if (kc == nullptr || in[12] != Py_None) {
      k_out = output(in[12], "k_out", *k);
      a.k_out = call.packed<void>(k_out, "k_out", a.ko_token, a.ko_head);
    }
    if (kc != nullptr) {
      a.v = call.packed<void>(*v, "v", a.v_token, a.v_head);
      if (v->sizes() != k->sizes()) refuse(PyExc_ValueError, "%s must have k's shape", "v");
      call.cache(*kc, *vc, k->size(1), d, a.pages, a.page_size, a.cache_page, a.cache_head, a.cache_slot);
      a.k_cache = kc->data_ptr();
      a.v_cache = vc->data_ptr();
    }
  }
  const hipStream_t stream = call.stream();
  run("awq_rope", [&] { return awq_rope(&a, stream); });
  PyObject* both = PyTuple_New(2);
  if (both == nullptr) throw Refused{};
  auto put = [&](int i, const at::Tensor& t) {
    PyObject* o = Py_None;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
    } else {
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(both, i, o);
  };
  put(0, q_out);
  put(1, k_out);
  return both;
}

// q, k, v, cu_seqlens, scale, out
PyObject* attn_prompt(PyObject* const* in, Py_ssize_t n) {
  want(n, 6);
  const at::Tensor &q = *tensor(in[0], "q"), &k = *tensor(in[1], "k"), &v = *tensor(in[2], "v");
  const at::Tensor* cu = tensor(in[3], "cu_seqlens");
  const Call call(q, "q");
  awq_attn_prompt_args a{};
  a.dtype = call.element_type("q");
  a.q = call.packed<void>(q, "q", a.q_token, a.q_head);
  a.k = call.packed<void>(k, "k", a.k_token, a.k_head);
  a.v = call.packed<void>(v, "v", a.v_token, a.v_head);
  a.tokens = q.size(0);
  a.q_heads = count(q.size(1), "q");
  a.kv_heads = count(k.size(1), "k");
  a.head_dim = count(q.size(2), "q");
  if (k.size(0) != a.tokens || k.size(2) != q.size(2)) refuse(PyExc_ValueError, "%s must have q's tokens and head size", "k");
  if (v.sizes() != k.sizes()) refuse(PyExc_ValueError, "%s must have k's shape", "v");
  a.cu = call.vector<int32_t>(cu, "cu_seqlens", at::kInt, {-1});
  if (cu->size(0) < 1) refuse(PyExc_ValueError, "%s must be [seqs + 1]", "cu_seqlens");
  a.seqs = cu->size(0) - 1;
  a.scale = in[4] == Py_None ? 1.0f / std::sqrt(static_cast<float>(a.head_dim)) : static_cast<float>(number(in[4]));
  at::Tensor out = output(in[5], "out", q);
  a.out = call.packed<void>(out, "out", a.o_token, a.o_head);
  const hipStream_t stream = call.stream();
  run("awq_attn_prompt", [&] { return awq_attn_prompt(&a, stream); });
  return THPVariable_Wrap(out);
}

// q, k_cache, v_cache, block_table, ctx_lens, cu_q, max_q, mask, scale, out, ws
PyObject* attn_tree(PyObject* const* in, Py_ssize_t n) {
  want(n, 11);
  const at::Tensor &q = *tensor(in[0], "q"), &kc = *tensor(in[1], "k_cache"), &vc = *tensor(in[2], "v_cache");
  const at::Tensor *table = tensor(in[3], "block_table"), *ctx = tensor(in[4], "ctx_lens"), *cu = tensor(in[5], "cu_q");
  const at::Tensor *mask = tensor(in[7], "mask", true), *ws = tensor(in[10], "ws", true);
  const Call call(q, "q");
  awq_attn_tree_args a{};
  a.dtype = call.element_type("q");
  a.q = call.packed<void>(q, "q", a.q_token, a.q_head);
  a.tokens = q.size(0);
  a.q_heads = count(q.size(1), "q");
  a.head_dim = count(q.size(2), "q");
  if (kc.dim() != 4) refuse(PyExc_ValueError, "%s must be [pages, kv_heads, page_size, head_dim]", "k_cache");
  a.kv_heads = count(kc.size(1), "k_cache");
  call.cache(kc, vc, kc.size(1), q.size(2), a.pages, a.page_size, a.cache_page, a.cache_head, a.cache_slot);
  a.k_cache = kc.data_ptr();
  a.v_cache = vc.data_ptr();
  a.block_table = call.vector<int32_t>(table, "block_table", at::kInt, {-1, -1});
  a.seqs = table->size(0);
  a.table_width = table->size(1);
  a.ctx_lens = call.vector<int32_t>(ctx, "ctx_lens", at::kInt, {a.seqs});
  a.cu_q = call.vector<int32_t>(cu, "cu_q", at::kInt, {a.seqs + 1});
  a.mask = reinterpret_cast<const uint64_t*>(call.vector<int64_t>(mask, "mask", at::kLong, {a.tokens}));
  a.max_q = integer32(in[6], "max_q");
  a.scale = in[8] == Py_None ? 1.0f / std::sqrt(static_cast<float>(a.head_dim)) : static_cast<float>(number(in[8]));
  at::Tensor out = output(in[9], "out", q);
  a.out = call.packed<void>(out, "out", a.o_token, a.o_head);
  Owned made;  // until the launch: under capture nothing else holds it
  if (ws == nullptr) {
    const size_t need = awq_attn_tree_workspace_bytes(a.tokens, a.seqs, a.table_width, a.page_size, a.max_q,
                                                      a.q_heads, a.kv_heads, a.head_dim);
    if (need > 0) {
      made.object = PyObject_CallFunction(g_workspace, "nL", static_cast<Py_ssize_t>(need), static_cast<long long>(call.device));
      if (made.object == nullptr) throw Refused{};
      ws = &THPVariable_Unpack(made.object);
    }
  }
  if (ws != nullptr) {
    a.ws = call.vector<void>(ws, "ws", at::kByte, {-1});
    a.ws_bytes = static_cast<size_t>(ws->size(0));
  }
  const hipStream_t stream = call.stream();
  run("awq_attn_tree", [&] { return awq_attn_tree(&a, stream); });
  return THPVariable_Wrap(out);
}

// x, inv_s_c, packed, n, k, group, fmt, bias, act, mul, residual, y, ws
PyObject* gemm_fused(PyObject* const* in, Py_ssize_t nargs) {
  want(nargs, 13);
  const at::Tensor &x = *tensor(in[0], "x"), *inv = tensor(in[1], "inv_s_c", true), *packed = tensor(in[2], "packed");
  const at::Tensor *bias = tensor(in[7], "bias", true), *mul = tensor(in[9], "mul", true);
  const at::Tensor *residual = tensor(in[10], "residual", true), *ws = tensor(in[12], "ws", true);
  const int64_t n = integer(in[3]), k = integer(in[4]);
  const int32_t group = integer32(in[5], "group"), fmt = integer32(in[6], "fmt");
  if (x.dim() != 2 || x.size(1) != k) refuse(PyExc_ValueError, "%s must be [M, K]", "x");
  const Call call(x, "x");
  const int64_t m = x.size(0);
  const uint16_t* xp = call.vector<uint16_t>(&x, "x", at::kHalf, {m, k});
  const uint16_t* ip = call.vector<uint16_t>(inv, "inv_s_c", at::kHalf, {k});
  const uint8_t* pp = call.vector<uint8_t>(packed, "packed", at::kByte, {-1});
  const size_t need = awq_repacked_bytes(n, k, group, fmt);
  if (static_cast<size_t>(packed->size(0)) < need) refuse(PyExc_ValueError, "%s holds fewer bytes than the layer needs", "packed");
  awq_epilogue e{};
  e.bias = call.vector<uint16_t>(bias, "bias", at::kHalf, {n});
  e.mul = call.vector<uint16_t>(mul, "mul", at::kHalf, {m, n});
  e.residual = call.vector<uint16_t>(residual, "residual", at::kHalf, {m, n});
  e.act = integer32(in[8], "act");
  void* wp = call.vector<void>(ws, "ws", at::kByte, {-1});
  const size_t ws_bytes = ws == nullptr ? 0 : static_cast<size_t>(ws->size(0));
  at::Tensor y;
  if (in[11] == Py_None) {
    if (n < 0) refuse(PyExc_ValueError, "%s is out of range", "n");
    y = at::empty({m, n}, x.options());
  } else {
    y = *tensor(in[11], "y");
  }
  uint16_t* yp = call.vector<uint16_t>(&y, "y", at::kHalf, {m, n});
  const hipStream_t stream = call.stream();
  run("awq_gemm_fused",
      [&] { return awq_gemm_fused(xp, ip, pp, m, n, k, group, fmt, &e, yp, wp, ws_bytes, stream); });
  return THPVariable_Wrap(y);
}

// stream, workspace, error
PyObject* setup(PyObject* const* in, Py_ssize_t n) {
  want(n, 3);
  PyObject** to[3] = {&g_stream, &g_workspace, &g_error};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(in[i]);
    Py_XDECREF(*to[i]);
    *to[i] = in[i];
  }
  Py_RETURN_NONE;
}

// No C++ exception leaves a call: PyTorch's become its Python errors.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* in, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(in, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define AWQ_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {AWQ_METHOD(rope),       AWQ_METHOD(attn_prompt), AWQ_METHOD(attn_tree),
                         AWQ_METHOD(gemm_fused), AWQ_METHOD(setup),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block(void) { return PyModule_Create(&module); }
