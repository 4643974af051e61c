// Compiled part of the Python binding: the operators in front of the expert layer, which cost a few
// microseconds each, so that their arguments are checked and marshalled in well under one.  It
// checks torch tensors against the problem, takes the stream and calls the C ABI (mega_moe.h); the
// status goes back to Python.  No arithmetic happens here.
//
// norm_quant(problem, x, weight, residual, residual_out, normed, q, q_sf, stream) -> status
// gate_logits(problem, x, weight, logits, stream) -> status
// gate_topk(problem, logits, topk_idx, topk_w, bias, num_valid, stream) -> status
//
// problem: a ctypes structure; stream: an int handle, or None for the current stream of the
// tensors' device, which is made the current device for the call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <sstream>
#include <stdexcept>

#include "mega_moe.h"

namespace {

// A refusal that becomes a Python ValueError; any other exception becomes a RuntimeError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor" + (optional ? " or None" : ""));
  return &THPVariable_Unpack(o);
}

void refuse(const char* name, const at::Tensor& t, at::Device dev, at::ScalarType type, at::IntArrayRef shape,
            const char* what) {
  std::ostringstream s;
  s << name << " is " << t.scalar_type() << " " << t.sizes() << " on " << t.device() << ", strides " << t.strides()
    << "; expected " << type << " " << shape << " on " << dev << ", " << what;
  throw Refused(s.str());
}

void check_buffer(const char* name, const at::Tensor* t, at::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  if (t && (t->scalar_type() != type || t->sizes() != shape || t->device() != dev || !t->is_contiguous()))
    refuse(name, *t, dev, type, shape, "contiguous");
}

// Rows `stride` elements apart (0: as wide as they are).  A single row has no stride.
void check_rows(const char* name, const at::Tensor* t, at::Device dev, at::ScalarType type, int64_t rows, int64_t cols,
                int64_t stride) {
  if (!t) return;
  const int64_t shape[] = {rows, cols};
  if (t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape) || t->device() != dev)
    refuse(name, *t, dev, type, shape, "as the problem says");
  if (rows && ((cols > 1 && t->stride(1) != 1) || (rows > 1 && t->stride(0) != (stride ? stride : cols))))
    refuse(name, *t, dev, type, shape, "contiguous rows as far apart as the problem says");
}

at::ScalarType type_of(int dtype) {
  if (dtype == MEGA_MOE_DTYPE_BF16) return at::kBFloat16;
  if (dtype == MEGA_MOE_DTYPE_F32) return at::kFloat;
  return at::ScalarType::Undefined;            // refused: no tensor has it
}

at::Device device_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) throw Refused(std::string(what) + " needs device tensors");
  return t.device();
}

void* ptr(const at::Tensor* t) { return t && t->numel() ? t->data_ptr() : nullptr; }

// The problem structure behind a ctypes instance, copied.
template <class P>
P problem_of(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) {
    PyErr_Clear();
    throw Refused("problem must be the operator's problem structure");
  }
  const bool fits = b.len == (Py_ssize_t)sizeof(P);
  P p{};
  if (fits) std::memcpy(&p, b.buf, sizeof(P));
  PyBuffer_Release(&b);
  if (!fits) throw Refused("problem must be the operator's problem structure");
  return p;
}

void* stream_of(PyObject* o, at::Device dev) {
  if (o != Py_None) {
    void* h = PyLong_AsVoidPtr(o);
    if (!h && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("stream must be a stream or its handle");
    }
    return h;
  }
  return c10::hip::getCurrentHIPStream(dev.index()).stream();
}

template <class F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error in the binding");
  }
  return nullptr;
}

PyObject* norm_quant(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("norm_quant", n, 9, [&] {
    const auto p = problem_of<mega_moe_norm_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x"), *weight = tensor(v[2], "weight"), *residual = tensor(v[3], "residual", true),
                     *residual_out = tensor(v[4], "residual_out", true), *normed = tensor(v[5], "normed", true),
                     *q = tensor(v[6], "q", true), *q_sf = tensor(v[7], "q_sf", true);
    const at::Device dev = device_of(*x, "mega_moe_norm_quant");
    const int64_t T = p.num_tokens, H = p.hidden, shape[] = {T, H};
    const at::ScalarType xt = type_of(p.x_dtype);
    check_rows("x", x, dev, xt, T, H, p.x_stride);
    check_buffer("weight", weight, dev, type_of(p.weight_dtype), {H});
    check_rows("residual", residual, dev, xt, T, H, p.residual_stride);
    check_rows("residual_out", residual_out, dev, xt, T, H, p.residual_stride);
    check_buffer("normed", normed, dev, at::kBFloat16, shape);
    check_buffer("q", q, dev, at::kByte, shape);
    if (p.recipe == MEGA_MOE_RECIPE_FP8_B128) check_buffer("q_sf", q_sf, dev, at::kFloat, {T, H / 128});
    else check_buffer("q_sf", q_sf, dev, at::kByte, {T, H / 32});
    void* s = stream_of(v[8], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_norm_quant(&p, ptr(x), ptr(residual), ptr(weight), ptr(residual_out), ptr(normed), ptr(q), ptr(q_sf), s);
  });
}

PyObject* gate_logits(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("gate_logits", n, 5, [&] {
    const auto p = problem_of<mega_moe_gate_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x"), *weight = tensor(v[2], "weight"), *logits = tensor(v[3], "logits");
    const at::Device dev = device_of(*x, "mega_moe_gate_logits");
    const int64_t T = p.num_tokens, H = p.hidden, E = p.num_experts;
    check_rows("x", x, dev, at::kBFloat16, T, H, p.x_stride);
    check_buffer("weight", weight, dev, type_of(p.weight_dtype), {E, H});
    check_buffer("logits", logits, dev, at::kFloat, {T, E});
    void* s = stream_of(v[4], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_gate_logits(&p, ptr(x), ptr(weight), static_cast<float*>(ptr(logits)), s);
  });
}

PyObject* gate_topk(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("gate_topk", n, 7, [&] {
    const auto p = problem_of<mega_moe_topk_problem>(v[0]);
    const at::Tensor *logits = tensor(v[1], "logits"), *idx = tensor(v[2], "topk_idx"), *w = tensor(v[3], "topk_w"),
                     *bias = tensor(v[4], "bias", true), *num_valid = tensor(v[5], "num_valid", true);
    const at::Device dev = device_of(*logits, "mega_moe_gate_topk");
    const int64_t T = p.num_tokens, E = p.num_experts, out[] = {T, (int64_t)p.topk + p.num_shared};
    check_rows("logits", logits, dev, type_of(p.logits_dtype), T, E, p.logits_stride);
    check_buffer("bias", bias, dev, at::kFloat, {E});
    check_buffer("num_valid", num_valid, dev, at::kInt, {1});
    check_buffer("topk_idx", idx, dev, at::kInt, out);
    check_buffer("topk_w", w, dev, at::kFloat, out);
    void* s = stream_of(v[6], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_gate_topk(&p, ptr(logits), static_cast<const float*>(ptr(bias)),
                              static_cast<const int32_t*>(ptr(num_valid)), static_cast<int32_t*>(ptr(idx)),
                              static_cast<float*>(ptr(w)), s);
  });
}

PyMethodDef methods[] = {
    {"norm_quant", (PyCFunction)(void (*)(void))norm_quant, METH_FASTCALL, nullptr},
    {"gate_logits", (PyCFunction)(void (*)(void))gate_logits, METH_FASTCALL, nullptr},
    {"gate_topk", (PyCFunction)(void (*)(void))gate_topk, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
