// What the Python calls of the operators share (binding.cpp, binding_ffn.cpp): the checks of a
// call's tensors, PyTorch's current stream, workspaces and errors.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/awq_ffn.h"

namespace binding {

inline PyObject *g_stream = nullptr;     // device number -> the current stream's handle
inline PyObject *g_workspace = nullptr;  // (bytes, device number) -> tensor
inline PyObject *g_error = nullptr;      // AwqError(status, function)

struct Refused {};  // thrown with a Python error set

// A reference that ends with its scope
struct Owned {
  PyObject* object = nullptr;
  ~Owned() { Py_XDECREF(object); }
};

[[noreturn]] inline void refuse(PyObject* kind, const char* format, const char* name) {
  PyErr_Format(kind, format, name);
  throw Refused{};
}

// None is allowed and gives NULL where `optional`
inline const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
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

inline int32_t count(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(PyExc_ValueError, "%s has too large a dimension", name);
  return static_cast<int32_t>(n);
}
inline double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
inline int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
inline int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(v);
}
inline bool truth(PyObject* o) {
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
inline at::Tensor output(PyObject* o, const char* name, const at::Tensor& ref) {
  if (o == Py_None) return at::empty(ref.sizes(), ref.options());
  const at::Tensor& t = *tensor(o, name);
  if (t.sizes() != ref.sizes()) refuse(PyExc_ValueError, "%s has the wrong shape", name);
  return t;
}

inline void want(Py_ssize_t got, Py_ssize_t n) {
  if (got != n) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw Refused{};
  }
}

// the given workspace, or where the call needs one and none is given a scratch buffer that `made`
// holds until the launch (under capture nothing else holds it)
inline void workspace(const Call& call, const at::Tensor* ws, size_t need, Owned& made, void*& at, size_t& bytes) {
  if (ws == nullptr && need > 0) {
    made.object = PyObject_CallFunction(g_workspace, "nL", static_cast<Py_ssize_t>(need), static_cast<long long>(call.device));
    if (made.object == nullptr) throw Refused{};
    ws = &THPVariable_Unpack(made.object);
  }
  if (ws == nullptr) return;
  at = call.vector<void>(ws, "ws", at::kByte, {-1});
  bytes = static_cast<size_t>(ws->size(0));
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

extern PyMethodDef ffn_methods[];  // binding_ffn.cpp

}  // namespace binding
