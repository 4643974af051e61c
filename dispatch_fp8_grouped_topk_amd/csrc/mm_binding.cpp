// Compiled part of the Python binding: the operators in front of the expert layer and the layer in parts, which cost
// a few microseconds each, so that their arguments are checked and marshalled in well under one.  It
// checks torch tensors against the problem, takes the stream and calls the C ABI (mega_moe.h); the
// status goes back to Python.  No arithmetic happens here.
//
// problem_classes(NormProblem, GateProblem, TopkProblem, SortProblem, UnsortProblem, ProductProblem, ActProblem): once, before
// the first call
// norm_quant(problem, x, weight, residual, residual_out, normed, q, q_sf, stream) -> status
// gate_logits(problem, x, weight, logits, stream) -> status
// gate_topk(problem, logits, topk_idx, topk_w, bias, num_valid, stream) -> status
// sort_tokens(problem, x, x_sf, topk_idx, rows, rows_sf, pool_src, pair_pos, expert_offset, workspace, stream) -> status
// unsort_tokens(problem, rows, pair_pos, topk_w, y, stream) -> status
// unsort_backward(problem, dy, rows, pair_pos, topk_w, d_rows, d_w, stream) -> status
// block_product(problem, x, x_sf, w, w_sf, group_offset, y, stream) -> status
// act_quant(problem, x, num_valid, q, q_sf, out, stream) -> status
// act_backward(problem, x, d_out, num_valid, d_x, stream) -> status
//
// problem: an instance of its operator's class; stream: an int handle, or None for the current stream of the
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

// The ctypes classes of the problem structures, as the package hands them over: structures of different operators have the
// same size, so only the class tells them apart.
template <class P>
PyObject* g_problem_class = nullptr;

// The problem structure behind an instance of its class, copied.
template <class P>
P problem_of(PyObject* o) {
  PyObject* const cls = g_problem_class<P>;
  const int is = cls ? PyObject_IsInstance(o, cls) : 0;
  Py_buffer b;
  if (is <= 0 || PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) {
    PyErr_Clear();
    throw Refused("problem must be the operator's problem structure");
  }
  const bool fits = b.len >= (Py_ssize_t)sizeof(P);      // a subclass may have fields of its own
  P p{};
  if (fits) std::memcpy(&p, b.buf, sizeof(P));
  PyBuffer_Release(&b);
  if (!fits) throw Refused("problem must be the operator's problem structure");
  return p;
}

template <class P>
void take_class(PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_problem_class<P>, cls);
}

PyObject* problem_classes(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "problem_classes takes 7 classes");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i)
    if (!PyType_Check(v[i])) {
      PyErr_SetString(PyExc_TypeError, "problem_classes takes classes");
      return nullptr;
    }
  take_class<mega_moe_norm_problem>(v[0]);
  take_class<mega_moe_gate_problem>(v[1]);
  take_class<mega_moe_topk_problem>(v[2]);
  take_class<mega_moe_sort_problem>(v[3]);
  take_class<mega_moe_unsort_problem>(v[4]);
  take_class<mega_moe_product_problem>(v[5]);
  take_class<mega_moe_act_problem>(v[6]);
  Py_RETURN_NONE;
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

// Scales that go with `rows` 8-bit rows of `cols` columns.
void check_scales(const char* name, const at::Tensor* t, at::Device dev, int recipe, int64_t rows, int64_t cols) {
  if (recipe == MEGA_MOE_RECIPE_FP8_B128) check_buffer(name, t, dev, at::kFloat, {rows, cols / 128});
  else check_buffer(name, t, dev, at::kByte, {rows, cols / 32});
}

PyObject* sort_tokens(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("sort_tokens", n, 11, [&] {
    const auto p = problem_of<mega_moe_sort_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x", true), *x_sf = tensor(v[2], "x_sf", true), *idx = tensor(v[3], "topk_idx"),
                     *rows = tensor(v[4], "rows", true), *rows_sf = tensor(v[5], "rows_sf", true),
                     *src = tensor(v[6], "pool_src"), *pos = tensor(v[7], "pair_pos"),
                     *offset = tensor(v[8], "expert_offset"), *ws = tensor(v[9], "workspace", true);
    const at::Device dev = device_of(*idx, "mega_moe_sort_tokens");
    const int64_t T = p.num_tokens, H = p.hidden, k = p.topk, pairs[] = {T, k};
    const at::ScalarType type = p.dtype == MEGA_MOE_DTYPE_E4M3 ? at::kByte : type_of(p.dtype);
    check_rows("x", x, dev, type, T, H, p.x_stride);
    check_buffer("topk_idx", idx, dev, at::kInt, pairs);
    check_buffer("rows", rows, dev, type, {T * k, H});
    check_scales("x_sf", x_sf, dev, p.recipe, T, H);
    check_scales("rows_sf", rows_sf, dev, p.recipe, T * k, H);
    check_buffer("pool_src", src, dev, at::kInt, {T * k});
    check_buffer("pair_pos", pos, dev, at::kInt, pairs);
    check_buffer("expert_offset", offset, dev, at::kInt, {(int64_t)p.num_experts + 1});
    if (ws && (ws->device() != dev || !ws->is_contiguous())) throw Refused("workspace must be a contiguous tensor on the same device");
    void* s = stream_of(v[10], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_sort_tokens(&p, ptr(x), ptr(x_sf), static_cast<const int32_t*>(ptr(idx)), ptr(rows), ptr(rows_sf),
                                static_cast<int32_t*>(ptr(src)), static_cast<int32_t*>(ptr(pos)),
                                static_cast<int32_t*>(ptr(offset)), ptr(ws), ws ? ws->nbytes() : 0, s);
  });
}

PyObject* unsort_tokens(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("unsort_tokens", n, 6, [&] {
    const auto p = problem_of<mega_moe_unsort_problem>(v[0]);
    const at::Tensor *rows = tensor(v[1], "rows"), *pos = tensor(v[2], "pair_pos"), *w = tensor(v[3], "topk_w", true),
                     *y = tensor(v[4], "y");
    const at::Device dev = device_of(*pos, "mega_moe_unsort_tokens");
    const int64_t T = p.num_tokens, H = p.hidden, k = p.topk, pairs[] = {T, k};
    check_buffer("rows", rows, dev, type_of(p.dtype), {p.num_rows ? p.num_rows : T * k, H});
    check_buffer("pair_pos", pos, dev, at::kInt, pairs);
    check_buffer("topk_w", w, dev, at::kFloat, pairs);
    check_rows("y", y, dev, type_of(p.dtype), T, H, p.stride);
    void* s = stream_of(v[5], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_unsort_tokens(&p, ptr(rows), static_cast<const int32_t*>(ptr(pos)),
                                  static_cast<const float*>(ptr(w)), ptr(y), s);
  });
}

PyObject* unsort_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("unsort_backward", n, 8, [&] {
    const auto p = problem_of<mega_moe_unsort_problem>(v[0]);
    const at::Tensor *dy = tensor(v[1], "dy"), *rows = tensor(v[2], "rows", true), *pos = tensor(v[3], "pair_pos"),
                     *w = tensor(v[4], "topk_w", true), *d_rows = tensor(v[5], "d_rows", true),
                     *d_w = tensor(v[6], "d_w", true);
    const at::Device dev = device_of(*pos, "mega_moe_unsort_backward");
    const int64_t T = p.num_tokens, H = p.hidden, k = p.topk, pairs[] = {T, k};
    const int64_t R = p.num_rows ? p.num_rows : T * k, all[] = {R, H};
    check_rows("dy", dy, dev, type_of(p.dtype), T, H, p.stride);
    check_buffer("rows", rows, dev, type_of(p.dtype), all);
    check_buffer("pair_pos", pos, dev, at::kInt, pairs);
    check_buffer("topk_w", w, dev, at::kFloat, pairs);
    check_buffer("d_rows", d_rows, dev, type_of(p.dtype), all);
    check_buffer("d_w", d_w, dev, at::kFloat, pairs);
    void* s = stream_of(v[7], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_unsort_backward(&p, ptr(dy), ptr(rows), static_cast<const int32_t*>(ptr(pos)),
                                    static_cast<const float*>(ptr(w)), ptr(d_rows), static_cast<float*>(ptr(d_w)), s);
  });
}

PyObject* block_product(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("block_product", n, 8, [&] {
    const auto p = problem_of<mega_moe_product_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x"), *x_sf = tensor(v[2], "x_sf"), *w = tensor(v[3], "w"),
                     *w_sf = tensor(v[4], "w_sf"), *offset = tensor(v[5], "group_offset", true), *y = tensor(v[6], "y");
    const at::Device dev = device_of(*x, "mega_moe_block_product");
    const int64_t M = p.num_rows, N = p.n, K = p.k, G = p.num_groups;
    check_rows("x", x, dev, at::kByte, M, K, p.x_stride);
    check_buffer("x_sf", x_sf, dev, at::kFloat, {M, K / 128});
    check_buffer("w", w, dev, at::kByte, {G, N, K});
    check_buffer("w_sf", w_sf, dev, at::kFloat, {G, (N + 127) / 128, K / 128});
    check_buffer("group_offset", offset, dev, at::kInt, {G + 1});
    check_rows("y", y, dev, at::kBFloat16, M, N, p.y_stride);
    void* s = stream_of(v[7], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_block_product(&p, ptr(x), static_cast<const float*>(ptr(x_sf)), ptr(w),
                                  static_cast<const float*>(ptr(w_sf)), static_cast<const int32_t*>(ptr(offset)), ptr(y), s);
  });
}

PyObject* act_quant(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("act_quant", n, 7, [&] {
    const auto p = problem_of<mega_moe_act_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x"), *num_valid = tensor(v[2], "num_valid", true), *q = tensor(v[3], "q", true),
                     *q_sf = tensor(v[4], "q_sf", true), *out = tensor(v[5], "out", true);
    const at::Device dev = device_of(*x, "mega_moe_act_quant");
    const int64_t M = p.num_rows, I = p.width, shape[] = {M, I};
    check_rows("x", x, dev, type_of(p.x_dtype), M, p.act == MEGA_MOE_ACT_SWIGLU ? 2 * I : I, p.x_stride);
    check_buffer("num_valid", num_valid, dev, at::kInt, {1});
    check_buffer("q", q, dev, at::kByte, shape);
    check_scales("q_sf", q_sf, dev, p.recipe, M, I);
    check_buffer("out", out, dev, at::kBFloat16, shape);
    void* s = stream_of(v[6], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_act_quant(&p, ptr(x), static_cast<const int32_t*>(ptr(num_valid)), ptr(q), ptr(q_sf), ptr(out), s);
  });
}

PyObject* act_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded("act_backward", n, 6, [&] {
    const auto p = problem_of<mega_moe_act_problem>(v[0]);
    const at::Tensor *x = tensor(v[1], "x"), *d_out = tensor(v[2], "d_out"), *num_valid = tensor(v[3], "num_valid", true),
                     *d_x = tensor(v[4], "d_x");
    const at::Device dev = device_of(*x, "mega_moe_act_backward");
    const int64_t M = p.num_rows, I = p.width;
    check_rows("x", x, dev, type_of(p.x_dtype), M, 2 * I, p.x_stride);
    check_buffer("d_out", d_out, dev, type_of(p.x_dtype), {M, I});
    check_buffer("num_valid", num_valid, dev, at::kInt, {1});
    check_rows("d_x", d_x, dev, type_of(p.x_dtype), M, 2 * I, p.x_stride);
    void* s = stream_of(v[5], dev);
    c10::DeviceGuard guard(dev);
    return mega_moe_act_backward(&p, ptr(x), ptr(d_out), static_cast<const int32_t*>(ptr(num_valid)), ptr(d_x), s);
  });
}

PyMethodDef methods[] = {
    {"problem_classes", (PyCFunction)(void (*)(void))problem_classes, METH_FASTCALL, nullptr},
    {"norm_quant", (PyCFunction)(void (*)(void))norm_quant, METH_FASTCALL, nullptr},
    {"gate_logits", (PyCFunction)(void (*)(void))gate_logits, METH_FASTCALL, nullptr},
    {"gate_topk", (PyCFunction)(void (*)(void))gate_topk, METH_FASTCALL, nullptr},
    {"sort_tokens", (PyCFunction)(void (*)(void))sort_tokens, METH_FASTCALL, nullptr},
    {"unsort_tokens", (PyCFunction)(void (*)(void))unsort_tokens, METH_FASTCALL, nullptr},
    {"unsort_backward", (PyCFunction)(void (*)(void))unsort_backward, METH_FASTCALL, nullptr},
    {"block_product", (PyCFunction)(void (*)(void))block_product, METH_FASTCALL, nullptr},
    {"act_quant", (PyCFunction)(void (*)(void))act_quant, METH_FASTCALL, nullptr},
    {"act_backward", (PyCFunction)(void (*)(void))act_backward, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
