// Python calls of the feed-forward operators (awq_ffn.h); int8.py and moe.py hold the signatures
// and the documentation.
#include <ATen/ops/empty.h>

#include "binding.hpp"

namespace binding {
namespace {

// rows [tokens, width] of a type, elements of a row contiguous; a single row's stride is not
// looked at
void* rows(const Call& call, const at::Tensor& t, const char* name, at::ScalarType type, int64_t tokens, int64_t width,
           int64_t& stride) {
  call.on_device(t, name);
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s has the wrong type", name);
  if (t.dim() != 2 || t.size(0) != tokens || t.size(1) != width) refuse(PyExc_ValueError, "%s has the wrong shape", name);
  if (width > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "the elements of a row of %s must be contiguous", name);
  stride = tokens > 1 ? t.stride(0) : width;
  return t.data_ptr();
}

// the given output, or a new contiguous one
at::Tensor made_or_given(PyObject* o, const char* name, at::IntArrayRef shape, const at::TensorOptions& options) {
  return o == Py_None ? at::empty(shape, options) : *tensor(o, name);
}

const at::Tensor& matrix(PyObject* o, const char* name) {
  const at::Tensor& t = *tensor(o, name);
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s must have two dimensions", name);
  return t;
}

// the tensors, None where there is none
PyObject* tuple_of(std::initializer_list<at::Tensor> list) {
  PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
  if (all == nullptr) throw Refused{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : list) {
    PyObject* o = Py_None;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
      if (o == nullptr) {
        Py_DECREF(all);
        throw Refused{};
      }
    } else {
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(all, i++, o);
  }
  return all;
}

// x, weight, eps, residual, want y, want i8, y, q, scale, h
PyObject* rms_norm(PyObject* const* in, Py_ssize_t n) {
  want(n, 10);
  const at::Tensor& x = matrix(in[0], "x");
  const at::Tensor *weight = tensor(in[1], "weight", true), *residual = tensor(in[3], "residual", true);
  const Call call(x, "x");
  awq_rms_norm_args a{};
  a.dtype = call.element_type("x");
  a.tokens = x.size(0);
  a.width = count(x.size(1), "x");
  a.eps = static_cast<float>(number(in[2]));
  a.x = rows(call, x, "x", call.dtype, a.tokens, a.width, a.x_stride);
  a.weight = call.vector<void>(weight, "weight", call.dtype, {a.width});
  const bool want_y = truth(in[4]) || in[6] != Py_None, want_q = truth(in[5]) || in[7] != Py_None || in[8] != Py_None;
  if (!want_y && !want_q) refuse(PyExc_ValueError, "%s or i8 must be asked for", "y16");
  at::Tensor y, q, scale, h;
  if (residual != nullptr) {
    a.residual = rows(call, *residual, "residual", call.dtype, a.tokens, a.width, a.residual_stride);
    h = made_or_given(in[9], "h", {a.tokens, a.width}, x.options());
    a.h_out = rows(call, h, "h", call.dtype, a.tokens, a.width, a.h_stride);
  } else if (in[9] != Py_None) {
    refuse(PyExc_ValueError, "h needs a %s", "residual");
  }
  if (want_y) {
    y = made_or_given(in[6], "y", {a.tokens, a.width}, x.options());
    a.y = rows(call, y, "y", call.dtype, a.tokens, a.width, a.y_stride);
  }
  if (want_q) {
    q = made_or_given(in[7], "q", {a.tokens, a.width}, x.options().dtype(at::kChar));
    a.q = static_cast<int8_t*>(rows(call, q, "q", at::kChar, a.tokens, a.width, a.q_stride));
    scale = made_or_given(in[8], "scale", {a.tokens}, x.options().dtype(at::kFloat));
    a.scale = call.vector<float>(&scale, "scale", at::kFloat, {a.tokens});
  }
  const hipStream_t stream = call.stream();
  run("awq_rms_norm", [&] { return awq_rms_norm(&a, stream); });
  return tuple_of({y, q, scale, h});
}

// x, inv_s_c, q, scale
PyObject* quant_i8(PyObject* const* in, Py_ssize_t n) {
  want(n, 4);
  const at::Tensor& x = matrix(in[0], "x");
  const Call call(x, "x");
  awq_quant_i8_args a{};
  a.dtype = call.element_type("x");
  a.tokens = x.size(0);
  a.width = count(x.size(1), "x");
  a.x = rows(call, x, "x", call.dtype, a.tokens, a.width, a.x_stride);
  a.inv_s_c = call.vector<void>(tensor(in[1], "inv_s_c", true), "inv_s_c", call.dtype, {a.width});
  at::Tensor q = made_or_given(in[2], "q", {a.tokens, a.width}, x.options().dtype(at::kChar));
  a.q = static_cast<int8_t*>(rows(call, q, "q", at::kChar, a.tokens, a.width, a.q_stride));
  at::Tensor scale = made_or_given(in[3], "scale", {a.tokens}, x.options().dtype(at::kFloat));
  a.scale = call.vector<float>(&scale, "scale", at::kFloat, {a.tokens});
  const hipStream_t stream = call.stream();
  run("awq_quant_i8", [&] { return awq_quant_i8(&a, stream); });
  return tuple_of({q, scale});
}

// w, s_c
PyObject* pack_i8(PyObject* const* in, Py_ssize_t n) {
  want(n, 2);
  const at::Tensor& w = matrix(in[0], "w");
  const Call call(w, "w");
  const int32_t dtype = call.element_type("w");
  const int64_t N = w.size(0), K = w.size(1);
  const void* wp = call.vector<void>(&w, "w", call.dtype, {N, K});
  const void* sp = call.vector<void>(tensor(in[1], "s_c", true), "s_c", call.dtype, {K});
  const size_t bytes = awq_packed_i8_bytes(N, K);
  at::Tensor packed = at::empty({static_cast<int64_t>(bytes)}, w.options().dtype(at::kByte));
  void* pp = packed.data_ptr();
  const hipStream_t stream = call.stream();
  run("awq_pack_i8", [&] { return awq_pack_i8(wp, sp, N, K, dtype, pp, bytes, stream); });
  return THPVariable_Wrap(packed);
}

// q, scale, packed, n, k, bias, act, mul, residual, dtype (0 float16, 1 bfloat16), y, ws
PyObject* gemm_i8(PyObject* const* in, Py_ssize_t nargs) {
  want(nargs, 12);
  const at::Tensor &q = matrix(in[0], "q"), *scale = tensor(in[1], "scale"), *packed = tensor(in[2], "packed");
  const at::Tensor *bias = tensor(in[5], "bias", true), *mul = tensor(in[7], "mul", true);
  const at::Tensor *residual = tensor(in[8], "residual", true), *ws = tensor(in[11], "ws", true);
  const Call call(q, "q");
  awq_gemm_i8_args a{};
  a.N = integer(in[3]);
  a.K = integer(in[4]);
  a.M = q.size(0);
  a.act = integer32(in[6], "act");
  a.dtype = integer32(in[9], "dtype");
  const at::ScalarType type = a.dtype == AWQ_DT_F16 ? at::kHalf : at::kBFloat16;
  a.q = static_cast<const int8_t*>(rows(call, q, "q", at::kChar, a.M, a.K, a.q_stride));
  a.scale = call.vector<float>(scale, "scale", at::kFloat, {a.M});
  a.packed = call.vector<void>(packed, "packed", at::kByte, {-1});
  if (static_cast<size_t>(packed->size(0)) < awq_packed_i8_bytes(a.N, a.K))
    refuse(PyExc_ValueError, "%s holds fewer bytes than the layer needs", "packed");
  a.bias = call.vector<void>(bias, "bias", type, {a.N});
  a.mul = call.vector<void>(mul, "mul", type, {a.M, a.N});
  a.residual = call.vector<void>(residual, "residual", type, {a.M, a.N});
  if (a.N < 0) refuse(PyExc_ValueError, "%s is out of range", "n");
  at::Tensor y = made_or_given(in[10], "y", {a.M, a.N}, q.options().dtype(type));
  a.y = call.vector<void>(&y, "y", type, {a.M, a.N});
  Owned made;
  workspace(call, ws, awq_gemm_i8_workspace_bytes(a.M, a.N, a.K), made, a.ws, a.ws_bytes);
  const hipStream_t stream = call.stream();
  run("awq_gemm_i8", [&] { return awq_gemm_i8(&a, stream); });
  return THPVariable_Wrap(y);
}

// x, w, k, bias, score, renormalize, scale, ids, weights, ws
PyObject* moe_route(PyObject* const* in, Py_ssize_t n) {
  want(n, 10);
  const at::Tensor &x = matrix(in[0], "x"), &w = matrix(in[1], "w");
  const at::Tensor* ws = tensor(in[9], "ws", true);
  const Call call(x, "x");
  awq_moe_route_args a{};
  a.dtype = call.element_type("x");
  a.tokens = x.size(0);
  a.hidden = count(x.size(1), "x");
  a.experts = count(w.size(0), "w");
  a.x = rows(call, x, "x", call.dtype, a.tokens, a.hidden, a.x_stride);
  a.w = call.vector<void>(&w, "w", call.dtype, {a.experts, a.hidden});
  a.k = integer32(in[2], "k");
  if (a.k < 0) refuse(PyExc_ValueError, "%s is out of range", "k");
  a.bias = call.vector<float>(tensor(in[3], "bias", true), "bias", at::kFloat, {a.experts});
  a.score = integer32(in[4], "score");
  a.renormalize = truth(in[5]);
  a.scale = static_cast<float>(number(in[6]));
  at::Tensor ids = made_or_given(in[7], "ids", {a.tokens, a.k}, x.options().dtype(at::kInt));
  a.ids = call.vector<int32_t>(&ids, "ids", at::kInt, {a.tokens, a.k});
  at::Tensor weights = made_or_given(in[8], "weights", {a.tokens, a.k}, x.options().dtype(at::kFloat));
  a.weights = call.vector<float>(&weights, "weights", at::kFloat, {a.tokens, a.k});
  Owned made;
  workspace(call, ws, awq_moe_route_workspace_bytes(a.tokens, a.hidden, a.experts), made, a.ws, a.ws_bytes);
  const hipStream_t stream = call.stream();
  run("awq_moe_route", [&] { return awq_moe_route(&a, stream); });
  return tuple_of({ids, weights});
}

// a factor for each channel of each expert [experts, width], or of all [width]
const uint16_t* factors(const Call& call, PyObject* o, const char* name, int64_t experts, int64_t width,
                        int64_t& stride) {
  const at::Tensor* t = tensor(o, name, true);
  stride = t != nullptr && t->dim() == 2 ? width : 0;
  if (stride != 0) return call.vector<uint16_t>(t, name, at::kHalf, {experts, width});
  return call.vector<uint16_t>(t, name, at::kHalf, {width});
}

// x, ids, weights, gate, up, down, ffn, group, fmt, act, inv_in, inv_down, residual, y, ws
PyObject* moe_layer(PyObject* const* in, Py_ssize_t n) {
  want(n, 15);
  const at::Tensor &x = matrix(in[0], "x"), &ids = matrix(in[1], "ids");
  const at::Tensor &weights = matrix(in[2], "weights"), &gate = matrix(in[3], "gate");
  const at::Tensor &up = matrix(in[4], "up"), &down = matrix(in[5], "down");
  const at::Tensor *residual = tensor(in[12], "residual", true), *ws = tensor(in[14], "ws", true);
  const Call call(x, "x");
  awq_moe_args a{};
  a.tokens = x.size(0);
  a.hidden = count(x.size(1), "x");
  a.ffn = integer32(in[6], "ffn");
  a.group = integer32(in[7], "group");
  a.fmt = integer32(in[8], "fmt");
  a.act = integer32(in[9], "act");
  a.experts = count(gate.size(0), "gate");
  a.k = count(ids.size(1), "ids");
  a.x = static_cast<const uint16_t*>(rows(call, x, "x", at::kHalf, a.tokens, a.hidden, a.x_stride));
  a.ids = call.vector<int32_t>(&ids, "ids", at::kInt, {a.tokens, a.k});
  a.weights = call.vector<float>(&weights, "weights", at::kFloat, {a.tokens, a.k});
  const int64_t wide = static_cast<int64_t>(awq_repacked_bytes(a.ffn, a.hidden, a.group, a.fmt));
  const int64_t tall = static_cast<int64_t>(awq_repacked_bytes(a.hidden, a.ffn, a.group, a.fmt));
  if (wide == 0 || tall == 0) refuse(PyExc_ValueError, "invalid shape of an expert's %s", "layers");
  a.gate = call.vector<void>(&gate, "gate", at::kByte, {a.experts, wide});
  a.up = call.vector<void>(&up, "up", at::kByte, {a.experts, wide});
  a.down = call.vector<void>(&down, "down", at::kByte, {a.experts, tall});
  a.inv_in = factors(call, in[10], "inv_in", a.experts, a.hidden, a.inv_in_stride);
  a.inv_down = factors(call, in[11], "inv_down", a.experts, a.ffn, a.inv_down_stride);
  if (residual != nullptr)
    a.residual = static_cast<const uint16_t*>(
        rows(call, *residual, "residual", at::kHalf, a.tokens, a.hidden, a.residual_stride));
  at::Tensor y = made_or_given(in[13], "y", {a.tokens, a.hidden}, x.options());
  a.y = static_cast<uint16_t*>(rows(call, y, "y", at::kHalf, a.tokens, a.hidden, a.y_stride));
  Owned made;
  workspace(call, ws, awq_moe_workspace_bytes(a.tokens, a.hidden, a.ffn, a.k), made, a.ws, a.ws_bytes);
  const hipStream_t stream = call.stream();
  run("awq_moe", [&] { return awq_moe(&a, stream); });
  return THPVariable_Wrap(y);
}

}  // namespace

PyMethodDef ffn_methods[] = {AWQ_METHOD(rms_norm), AWQ_METHOD(quant_i8),  AWQ_METHOD(pack_i8),          AWQ_METHOD(gemm_i8),
                             AWQ_METHOD(moe_route), AWQ_METHOD(moe_layer), {nullptr, nullptr, 0, nullptr}};

}  // namespace binding
