// Python module _block: tensor checks and pointer marshalling of the block
// operators (add_rmsnorm, route_scored, linear) in front of the C ABI.  A whole
// call takes the host 2.3-2.7 us; the same checks in Python and ctypes took
// 11-14 us, several times the GPU time of the smallest calls.  block.py keeps
// the signatures, defaults and the allocation of outputs.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_w4a16.h"

namespace {

PyObject* g_error = nullptr;   // moe_w4a16.MoEError, set by block.py

// Fills *code with the library's element type; false for another type.
bool type_code(at::ScalarType t, int32_t* code) {
  switch (t) {
    case at::kHalf: *code = MOE_W4A16_F16; return true;
    case at::kBFloat16: *code = MOE_W4A16_BF16; return true;
    case at::kFloat: *code = MOE_W4A16_F32; return true;
    case at::kFloat8_e4m3fn: *code = MOE_W4A16_E4M3; return true;
    default: return false;
  }
}

bool bad(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s %s", name, what);
  return false;
}

const at::Tensor* tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor", name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// The first tensor of a call fixes the device.
bool input(const char* name, const at::Tensor& t, int* dev) {
  if (!t.is_cuda() || t.dim() != 2) return bad(name, "must be a 2-D CUDA tensor");
  *dev = t.get_device();
  return true;
}

// A [T, n] tensor whose rows are contiguous; None leaves *p NULL.
bool rows(const char* name, PyObject* o, int64_t T, int64_t n, at::ScalarType dt, int dev, void** p, int64_t* ld) {
  *p = nullptr;
  *ld = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(name, o);
  if (!t) return false;
  if (t->scalar_type() != dt) return bad(name, "has the wrong type");
  if (!t->is_cuda() || t->get_device() != dev) return bad(name, "is not on the device of the other arguments");
  if (t->dim() != 2 || t->size(0) != T || t->size(1) != n) {
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld)", name, (long long)T, (long long)n);
    return false;
  }
  const int64_t s = t->stride(0);
  if ((t->stride(1) != 1 && n > 1) || (s < n && T > 1)) return bad(name, "must have contiguous rows");
  *ld = s < n || T < 2 ? n : s;   // a single row needs no stride
  *p = t->data_ptr();
  return true;
}

bool vec(const char* name, PyObject* o, int64_t n, at::ScalarType dt, int dev, void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(name, o);
  if (!t) return false;
  if (t->scalar_type() != dt) return bad(name, "has the wrong type");
  if (!t->is_cuda() || t->get_device() != dev) return bad(name, "is not on the device of the other arguments");
  if (t->dim() != 1 || t->size(0) != n || (t->stride(0) != 1 && n > 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld", name, (long long)n);
    return false;
  }
  *p = t->data_ptr();
  return true;
}

bool int_arg(PyObject* o, int32_t* v) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x < INT32_MIN || x > INT32_MAX) return bad("an integer argument", "does not fit 32 bits");
  *v = (int32_t)x;
  return true;
}

bool float_arg(PyObject* o, float* v) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return false;
  *v = (float)x;
  return true;
}

// None: the device's current stream; else a torch stream.
bool stream_arg(PyObject* o, int dev, moe_w4a16_stream_t* st) {
  if (o == Py_None) {
    *st = reinterpret_cast<moe_w4a16_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    return true;
  }
  PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
  if (!a) return false;
  const unsigned long long v = PyLong_AsUnsignedLongLong(a);
  Py_DECREF(a);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) return false;
  *st = reinterpret_cast<moe_w4a16_stream_t>((uintptr_t)v);
  return true;
}

PyObject* finish(moe_w4a16_status st) {
  if (st == MOE_W4A16_OK) Py_RETURN_NONE;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", (int)st, moe_w4a16_last_error(nullptr)) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

bool nargs_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// C++ exceptions (of torch or of a full heap) end as Python errors here.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (x, residual, weight, eps, y, s, q, q_scale, stream)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!nargs_ok(n, 9)) return nullptr;
    const at::Tensor* x = tensor("x", a[0]);
    int dev;
    if (!x || !input("x", *x, &dev)) return nullptr;
    const int64_t T = x->size(0), H = x->size(1);
    const at::ScalarType dt = x->scalar_type();
    if (dt != at::kHalf && dt != at::kBFloat16) return bad("x", "must be fp16 or bf16"), nullptr;
    if (H > INT32_MAX) return bad("x", "has too long rows"), nullptr;
    moe_w4a16_rmsnorm_config c = {};
    type_code(dt, &c.dtype);
    c.hidden = (int32_t)H;
    void *px, *pr, *pw, *py, *ps, *pq, *pqs;
    moe_w4a16_stream_t st;
    if (!float_arg(a[3], &c.eps) || !rows("x", a[0], T, H, dt, dev, &px, &c.ld_x) ||
        !rows("residual", a[1], T, H, dt, dev, &pr, &c.ld_residual) || !vec("weight", a[2], H, dt, dev, &pw) ||
        !rows("out y", a[4], T, H, dt, dev, &py, &c.ld_y) ||
        !rows("out s", a[5], T, H, dt, dev, &ps, &c.ld_residual_out) ||
        !rows("out q", a[6], T, H, at::kFloat8_e4m3fn, dev, &pq, &c.ld_q) ||
        !vec("out q_scale", a[7], T, at::kFloat, dev, &pqs) || !stream_arg(a[8], dev, &st))
      return nullptr;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return finish(moe_w4a16_add_rmsnorm(&c, T, px, pr, pw, ps, py, pq, static_cast<float*>(pqs), st));
  });
}

// (logits, bias, ids, weights, top_k, score, groups, top_groups, group_rank, renormalize, scale, stream)
PyObject* route_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!nargs_ok(n, 12)) return nullptr;
    const at::Tensor* l = tensor("logits", a[0]);
    int dev;
    if (!l || !input("logits", *l, &dev)) return nullptr;
    const int64_t T = l->size(0), E = l->size(1);
    const at::ScalarType dt = l->scalar_type();
    moe_w4a16_route_config c = {};
    if (!type_code(dt, &c.dtype) || c.dtype == MOE_W4A16_E4M3) return bad("logits", "must be fp32, fp16 or bf16"), nullptr;
    if (E > INT32_MAX) return bad("logits", "has too long rows"), nullptr;
    c.num_experts = (int32_t)E;
    const int renorm = PyObject_IsTrue(a[9]);
    if (renorm < 0) return nullptr;
    c.renormalize = renorm;
    void *pl, *pb, *pi, *pw;
    int64_t li, lw;
    moe_w4a16_stream_t st;
    if (!int_arg(a[4], &c.top_k) || !int_arg(a[5], &c.score) || !int_arg(a[6], &c.num_groups) ||
        !int_arg(a[7], &c.top_groups) || !int_arg(a[8], &c.group_rank) || !float_arg(a[10], &c.scale) ||
        !rows("logits", a[0], T, E, dt, dev, &pl, &c.ld_logits) || !vec("bias", a[1], E, at::kFloat, dev, &pb) ||
        !rows("out ids", a[2], T, c.top_k, at::kInt, dev, &pi, &li) ||
        !rows("out weights", a[3], T, c.top_k, at::kFloat, dev, &pw, &lw) || !stream_arg(a[11], dev, &st))
      return nullptr;
    if (li != c.top_k || lw != c.top_k) return bad("out ids and weights", "must be contiguous"), nullptr;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return finish(moe_w4a16_route_scored(&c, T, pl, static_cast<float*>(pb), static_cast<int32_t*>(pi),
                                         static_cast<float*>(pw), st));
  });
}

// (x, w, x_scale, w_scale, bias, residual, out, act, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!nargs_ok(n, 9)) return nullptr;
    const at::Tensor *x = tensor("x", a[0]), *w = x ? tensor("w", a[1]) : nullptr, *o = w ? tensor("out", a[6]) : nullptr;
    int dev, wdev;
    if (!o || !input("x", *x, &dev) || !input("w", *w, &wdev)) return nullptr;
    const int64_t T = x->size(0), K = x->size(1), M = w->size(0);
    const at::ScalarType dt = x->scalar_type(), ot = o->scalar_type();
    moe_w4a16_linear_config c = {};
    if (!int_arg(a[7], &c.act)) return nullptr;
    const bool gated = c.act == MOE_W4A16_ACT_SWIGLU;
    if (gated && M % 2) return bad("w", "needs an even number of rows for swiglu"), nullptr;
    const int64_t N = gated ? M / 2 : M;
    if (!type_code(dt, &c.in_dtype) || c.in_dtype == MOE_W4A16_F32)
      return bad("x", "must be fp16, bf16 or float8_e4m3fn"), nullptr;
    if (!type_code(ot, &c.out_dtype) || c.out_dtype == MOE_W4A16_E4M3)
      return bad("the output", "must be fp16, bf16 or fp32"), nullptr;
    if (K > INT32_MAX || N > INT32_MAX) return bad("w", "is too large"), nullptr;
    c.n = (int32_t)N;
    c.k = (int32_t)K;
    void *px, *pw, *pxs, *pws, *pb, *pr, *po;
    moe_w4a16_stream_t st;
    if (!rows("x", a[0], T, K, dt, dev, &px, &c.ld_x) || !rows("w", a[1], M, K, dt, dev, &pw, &c.ld_w) ||
        !vec("x_scale", a[2], T, at::kFloat, dev, &pxs) || !vec("w_scale", a[3], M, at::kFloat, dev, &pws) ||
        !vec("bias", a[4], M, at::kFloat, dev, &pb) || !rows("residual", a[5], T, N, ot, dev, &pr, &c.ld_residual) ||
        !rows("out", a[6], T, N, ot, dev, &po, &c.ld_out) || !stream_arg(a[8], dev, &st))
      return nullptr;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return finish(moe_w4a16_linear(&c, T, px, pw, static_cast<float*>(pxs), static_cast<float*>(pws),
                                   static_cast<float*>(pb), pr, po, st));
  });
}

PyObject* set_error(PyObject*, PyObject* e) {
  Py_INCREF(e);
  Py_XSETREF(g_error, e);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"add_rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_rmsnorm)), METH_FASTCALL, nullptr},
    {"route_scored", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route_scored)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__block() { return PyModule_Create(&module); }
