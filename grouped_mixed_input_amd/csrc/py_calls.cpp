// py_calls.cpp -- argument marshalling of the block-scaled fp8
// mixture-of-experts calls for Python.
//
// A call on a few tokens takes the device 3 to 6 us; reading types, shapes,
// strides and addresses of up to nine tensors attribute by attribute and
// handing them over through ctypes took 3 to 4 us of host time besides the
// launch.  Here the same checks read the tensors directly.  The computation
// stays in libgmi.so, whose functions are handed over as addresses (bind).
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/gmi.h"

namespace {

decltype(&gmi_rmsnorm_quant) f_rmsnorm_quant;
decltype(&gmi_rmsnorm_bwd) f_rmsnorm_bwd;
decltype(&gmi_gemm_f8_block) f_gemm_f8_block;
decltype(&gmi_gemm_f8_block_grouped) f_gemm_f8_block_grouped;
decltype(&gmi_moe_route) f_moe_route;
decltype(&gmi_moe_route_bwd) f_moe_route_bwd;

// a refusal: becomes ValueError
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// the Python error is set already
struct PythonError {};

[[noreturn]] void refuse(const char* format, ...) {
  char text[256];
  va_list ap;
  va_start(ap, format);
  std::vsnprintf(text, sizeof text, format, ap);
  va_end(ap);
  throw Refused(text);
}

constexpr auto F8 = at::kFloat8_e4m3fn;
constexpr auto F32 = at::kFloat;
constexpr auto I32 = at::kInt;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// Device matrix with unit stride along its rows: address and leading dimension.
struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
// with at most one row the stride says nothing: any legal leading dimension does
int64_t leading(int64_t rows, int64_t cols, int64_t stride) { return rows > 1 ? stride : (cols + 15) / 16 * 16; }

Matrix matrix(PyObject* o, const char* name, int64_t rows, int64_t cols, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) {
    std::string shape;
    for (int64_t n : t.sizes()) shape += "[" + std::to_string(n) + "]";
    refuse("%s must be %s [%lld][%lld], got %s %s", name, at::toString(type), (long long)rows, (long long)cols,
           at::toString(t.scalar_type()), shape.c_str());
  }
  if (!t.is_cuda()) refuse("%s must be on the device", name);
  if (cols > 1 && t.stride(1) != 1) refuse("%s must have unit stride along its rows", name);
  return {t.data_ptr(), leading(rows, cols, t.stride(0))};
}
Matrix matrix_or_none(PyObject* o, const char* name, int64_t rows, int64_t cols, at::ScalarType type) {
  return o == Py_None ? Matrix{} : matrix(o, name, rows, cols, type);
}

void* vector(PyObject* o, const char* name, int64_t n, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous() || !t.is_cuda())
    refuse("%s must be a contiguous device tensor of %lld %s", name, (long long)n, at::toString(type));
  return t.data_ptr();
}

const uint8_t* mask(PyObject* o, int64_t tokens) {
  if (o == Py_None) return nullptr;
  const at::ScalarType type = tensor(o, "mask").scalar_type();
  if (type != at::kBool && type != at::kByte) refuse("mask must be bool or uint8");
  return (const uint8_t*)vector(o, "mask", tokens, type);
}

struct Scratch {
  void* p = nullptr;
  size_t bytes = 0;
};
Scratch scratch(PyObject* o) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || !t.is_contiguous()) refuse("workspace must be a contiguous device tensor");
  return {t.data_ptr(), (size_t)t.numel() * t.element_size()};
}

// the library's sizes are 32-bit
int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse("%s above 2^31 - 1", name);
  return (int32_t)n;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
// The caller's stream (None: the current one) as a handle, asked of Python only
// when everything else has been checked.
PyObject* stream_handle;
void* stream(PyObject* o) {
  PyObject* v = PyObject_CallFunctionObjArgs(stream_handle, o, nullptr);
  if (!v) throw PythonError{};
  void* p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!p && PyErr_Occurred()) throw PythonError{};
  return p;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return (float)v;
}
gmi_dtype half_type(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return GMI_F16;
  if (t == at::kBFloat16) return GMI_BF16;
  refuse("%s must be float16 or bfloat16", name);
}

// Runs `call` (which returns the library's status) and turns what it throws
// into a Python exception.
template <class F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, const void* bound, F call) {
  if (!bound) return PyErr_Format(PyExc_RuntimeError, "%s: no library bound", name);
  if (got != want) return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
  try {
    return PyLong_FromLong(call());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <class F>
gmi_status without_gil(F f) {
  gmi_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

// x, weight, residual, eps, h, y, q, scales, stream
PyObject* rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rmsnorm_quant", n, 9, (void*)f_rmsnorm_quant, [&] {
    const at::Tensor& x = tensor(a[0], "x");
    const at::ScalarType type = x.scalar_type();
    const gmi_dtype dt = half_type(type, "x");
    if (x.dim() != 2) refuse("x must be [rows][K]");
    const int64_t rows = x.size(0), K = x.size(1);
    const Matrix mx = matrix(a[0], "x", rows, K, type);
    const void* w = vector(a[1], "weight", K, type);
    const Matrix res = matrix_or_none(a[2], "residual", rows, K, type), h = matrix_or_none(a[4], "h", rows, K, type),
                 y = matrix_or_none(a[5], "y", rows, K, type), q = matrix_or_none(a[6], "q", rows, K, F8),
                 s = matrix_or_none(a[7], "scales", rows, blocks(K), F32);
    const float eps = real(a[3]);
    const int32_t r32 = size32(rows, "rows"), k32 = size32(K, "K");
    void* st = stream(a[8]);
    return without_gil([&] {
      return f_rmsnorm_quant(r32, k32, mx.p, mx.ld, res.p, res.ld, w, eps, dt, h.p, h.ld, y.p, y.ld, q.p, q.ld,
                             (float*)s.p, s.ld, st);
    });
  });
}

// dy, h, weight, dres, eps, dh, dweight, workspace, stream
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rmsnorm_bwd", n, 9, (void*)f_rmsnorm_bwd, [&] {
    const at::Tensor& h = tensor(a[1], "h");
    const at::ScalarType type = h.scalar_type();
    const gmi_dtype dt = half_type(type, "h");
    if (h.dim() != 2) refuse("h must be [rows][K]");
    const int64_t rows = h.size(0), K = h.size(1);
    const Matrix dy = matrix(a[0], "dy", rows, K, type), mh = matrix(a[1], "h", rows, K, type),
                 dres = matrix_or_none(a[3], "dres", rows, K, type), dh = matrix(a[5], "dh", rows, K, type);
    const void* w = vector(a[2], "weight", K, type);
    float* dw = a[6] == Py_None ? nullptr : (float*)vector(a[6], "dweight", K, F32);
    const Scratch ws = scratch(a[7]);
    const float eps = real(a[4]);
    const int32_t r32 = size32(rows, "rows"), k32 = size32(K, "K");
    void* st = stream(a[8]);
    return without_gil([&] {
      return f_rmsnorm_bwd(r32, k32, dy.p, dy.ld, mh.p, mh.ld, w, dres.p, dres.ld, eps, dt, dh.p, dh.ld, dw, ws.p,
                           ws.bytes, st);
    });
  });
}

// X, x_scales, W, w_scales, Y, workspace, stream
PyObject* gemm_f8_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gemm_f8_block", n, 7, (void*)f_gemm_f8_block, [&] {
    const at::Tensor &x = tensor(a[0], "X"), &w = tensor(a[2], "W");
    if (x.dim() != 2 || w.dim() != 2) refuse("X must be [M][K] and W [N][K]");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0), kb = blocks(K);
    const Matrix mx = matrix(a[0], "X", M, K, F8), xs = matrix(a[1], "x_scales", M, kb, F32),
                 mw = matrix(a[2], "W", N, K, F8), ws = matrix(a[3], "w_scales", blocks(N), kb, F32),
                 y = matrix(a[4], "Y", M, N, at::kBFloat16);
    const Scratch work = scratch(a[5]);
    const int32_t m32 = size32(M, "M"), n32 = size32(N, "N"), k32 = size32(K, "K");
    void* st = stream(a[6]);
    return without_gil([&] {
      return f_gemm_f8_block(m32, n32, k32, mx.p, mx.ld, (const float*)xs.p, xs.ld, mw.p, mw.ld, (const float*)ws.p,
                             ws.ld, y.p, y.ld, work.p, work.bytes, st);
    });
  });
}

// offsets, X, x_scales, W, w_scales, Y, workspace, stream
PyObject* gemm_f8_block_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gemm_f8_block_grouped", n, 8, (void*)f_gemm_f8_block_grouped, [&] {
    const at::Tensor &x = tensor(a[1], "X"), &w = tensor(a[3], "W"), &s = tensor(a[4], "w_scales");
    if (x.dim() != 2) refuse("X must be [rows][K]");
    const int64_t rows = x.size(0), K = x.size(1), kb = blocks(K);
    if (w.dim() != 3 || s.dim() != 3 || w.scalar_type() != F8 || s.scalar_type() != F32 || w.size(2) != K ||
        s.size(0) != w.size(0) || s.size(1) != blocks(w.size(1)) || s.size(2) != kb)
      refuse("W must be [groups][N][K] float8_e4m3fn and w_scales [groups][ceil(N / 128)][ceil(K / 128)] float32");
    const int64_t count = w.size(0), N = w.size(1);
    const void* off = vector(a[0], "offsets", count + 1, I32);
    const Matrix mx = matrix(a[1], "X", rows, K, F8), xs = matrix(a[2], "x_scales", rows, kb, F32),
                 y = matrix(a[5], "Y", rows, N, at::kBFloat16);
    if (!w.is_cuda() || !s.is_cuda()) refuse("W and w_scales must be on the device");
    if ((K > 1 && w.stride(2) != 1) || (kb > 1 && s.stride(2) != 1))
      refuse("W and w_scales must have unit stride along their rows");
    const Scratch work = scratch(a[6]);
    const int32_t c32 = size32(count, "groups"), r32 = size32(rows, "rows"), n32 = size32(N, "N"), k32 = size32(K, "K");
    const int64_t ldw = leading(N, K, w.stride(1)), lds = leading(blocks(N), kb, s.stride(1));
    const int64_t w_stride = w.stride(0), s_stride = s.stride(0);
    const void* wp = w.data_ptr();
    const float* sp = (const float*)s.data_ptr();
    void* st = stream(a[7]);
    return without_gil([&] {
      return f_gemm_f8_block_grouped(c32, (const int32_t*)off, r32, n32, k32, mx.p, mx.ld, (const float*)xs.p, xs.ld, wp,
                                     ldw, w_stride, sp, lds, s_stride, y.p, y.ld, work.p, work.bytes, st);
    });
  });
}

struct Logits {
  int64_t T, E;
  Matrix m;
  at::ScalarType type;
  gmi_dtype dt;
};
Logits logits_of(PyObject* o) {
  const at::Tensor& t = tensor(o, "logits");
  const at::ScalarType type = t.scalar_type();
  if (t.dim() != 2 || (type != at::kHalf && type != at::kBFloat16 && type != F32))
    refuse("logits must be [tokens][experts] in float16, bfloat16 or float32");
  const int64_t T = t.size(0), E = t.size(1);
  return {T, E, matrix(o, "logits", T, E, type), type,
          type == at::kHalf ? GMI_F16 : type == at::kBFloat16 ? GMI_BF16 : GMI_F32};
}

// logits, k, mask, renormalize, indices, weights, counts, offsets, slot_row, row_slot, loss, live, workspace, stream
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("moe_route", n, 14, (void*)f_moe_route, [&] {
    const Logits x = logits_of(a[0]);
    const int64_t k = integer(a[1]), slots = x.T * k;
    const uint8_t* m = mask(a[2], x.T);
    const int renorm = PyObject_IsTrue(a[3]);
    if (renorm < 0) throw PythonError{};
    int32_t* idx = (int32_t*)vector(a[4], "indices", slots, I32);
    float* w = (float*)vector(a[5], "weights", slots, F32);
    int32_t* counts = (int32_t*)vector(a[6], "counts", x.E, I32);
    int32_t* offsets = (int32_t*)vector(a[7], "offsets", x.E + 1, I32);
    int32_t* slot_row = (int32_t*)vector(a[8], "slot_row", slots, I32);
    int32_t* row_slot = (int32_t*)vector(a[9], "row_slot", slots, I32);
    float* loss = (float*)vector(a[10], "loss", 1, F32);
    int32_t* live = (int32_t*)vector(a[11], "live", 1, I32);
    const Scratch ws = scratch(a[12]);
    const int32_t t32 = size32(x.T, "tokens"), e32 = size32(x.E, "experts"), k32 = size32(k, "k");
    void* st = stream(a[13]);
    return without_gil([&] {
      return f_moe_route(t32, e32, k32, x.m.p, x.m.ld, x.dt, m, renorm, idx, w, counts, offsets, slot_row, row_slot, loss,
                         live, ws.p, ws.bytes, st);
    });
  });
}

// logits, indices, weights, offsets, live, dweights, dloss, mask, renormalize, dlogits, stream
PyObject* moe_route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("moe_route_bwd", n, 11, (void*)f_moe_route_bwd, [&] {
    const Logits x = logits_of(a[0]);
    const at::Tensor& it = tensor(a[1], "indices");
    if (it.dim() < 1) refuse("indices must be [tokens][k]");
    const int64_t k = it.size(-1), slots = x.T * k;
    const int32_t* idx = (const int32_t*)vector(a[1], "indices", slots, I32);
    const float* w = (const float*)vector(a[2], "weights", slots, F32);
    const int32_t* offsets = (const int32_t*)vector(a[3], "offsets", x.E + 1, I32);
    const int32_t* live = (const int32_t*)vector(a[4], "live", 1, I32);
    const float* dw = (const float*)vector(a[5], "dweights", slots, F32);
    const float* dl = (const float*)vector(a[6], "dloss", 1, F32);
    const uint8_t* m = mask(a[7], x.T);
    const int renorm = PyObject_IsTrue(a[8]);
    if (renorm < 0) throw PythonError{};
    const Matrix d = matrix(a[9], "dlogits", x.T, x.E, x.type);
    const int32_t t32 = size32(x.T, "tokens"), e32 = size32(x.E, "experts"), k32 = size32(k, "k");
    void* st = stream(a[10]);
    return without_gil([&] {
      return f_moe_route_bwd(t32, e32, k32, x.m.p, x.m.ld, x.dt, m, renorm, idx, w, offsets, live, dw, dl, d.p, d.ld, st);
    });
  });
}

// addresses of the library's functions, in the order of the declarations above,
// and the function that turns a stream argument into a handle
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return PyErr_Format(PyExc_TypeError, "bind takes 6 addresses and a function, got %zd arguments", n);
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a NULL address");
      return nullptr;
    }
  }
  Py_INCREF(a[6]);
  Py_XDECREF(stream_handle);
  stream_handle = a[6];
  f_rmsnorm_quant = (decltype(f_rmsnorm_quant))p[0];
  f_rmsnorm_bwd = (decltype(f_rmsnorm_bwd))p[1];
  f_gemm_f8_block = (decltype(f_gemm_f8_block))p[2];
  f_gemm_f8_block_grouped = (decltype(f_gemm_f8_block_grouped))p[3];
  f_moe_route = (decltype(f_moe_route))p[4];
  f_moe_route_bwd = (decltype(f_moe_route_bwd))p[5];
  Py_RETURN_NONE;
}

#define GMI_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GMI_METHOD(bind),          GMI_METHOD(rmsnorm_quant),         GMI_METHOD(rmsnorm_bwd),
                         GMI_METHOD(gemm_f8_block), GMI_METHOD(gemm_f8_block_grouped), GMI_METHOD(moe_route),
                         GMI_METHOD(moe_route_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Argument marshalling of libgmi.so's newer calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
