// Tensor forms of the layer operators, as a CPython module over libtilegemm.so: argument checks,
// result and workspace allocation on the current stream, the call.
//
// Native because these calls are short: a norm of one token runs 3.7 us on the GPU, and the same
// checks and four allocations took 15 us in Python, so the host set the pace of every small call.
// The library itself knows nothing of torch; this module is the only part that does.
//
// Positional arguments only: the documented functions with their defaults are in __init__.py.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "tilegemm.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;   // TileError(status, reason)

struct Refusal {
  int status;
  std::string why;
};

template <class... T>
[[noreturn]] void refuse(int status, const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refusal{status, s.str()};
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return TG_F16;
    case at::kBFloat16: return TG_BF16;
    case at::kFloat: return TG_F32;
    case at::kFloat8_e4m3fn: return TG_FP8_E4M3;
    case at::kFloat8_e5m2: return TG_FP8_E5M2;
    default: return 0;
  }
}
int dtype_code(const char* name, at::ScalarType t) {
  const int c = code_of(t);
  if (!c) refuse(TG_E_DTYPE, name, ": unsupported dtype ", t);
  return c;
}
bool is_float(at::ScalarType t) { return t == at::kHalf || t == at::kBFloat16 || t == at::kFloat; }

// A tensor argument; None gives nullptr where it is optional.
const Tensor* tensor(const char* name, PyObject* o, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor%s, got %s", name, optional ? " or None" : "",
                 Py_TYPE(o)->tp_name);
    throw python_error();
  }
  return &THPVariable_Unpack(o);
}

void on_gpu(const char* name, const Tensor& t) {
  if (!t.is_cuda()) refuse(TG_E_ARG, name, " is on ", t.device(), ", not on a GPU");
}

// Leading dimension of a matrix argument whose rows are contiguous; checks its shape and dtype.
int64_t matrix(const char* name, const Tensor& t, int64_t rows = -1, int64_t cols = -1,
               at::ScalarType dtype = at::ScalarType::Undefined) {
  if (t.dim() != 2) refuse(TG_E_SHAPE, name, " must be a matrix, got ", t.dim(), " dimensions");
  const int64_t r = t.size(0), c = t.size(1);
  if ((rows >= 0 && r != rows) || (cols >= 0 && c != cols))
    refuse(TG_E_SHAPE, name, " must be (", rows, ", ", cols, "), got (", r, ", ", c, ")");
  if (dtype != at::ScalarType::Undefined && t.scalar_type() != dtype)
    refuse(TG_E_DTYPE, name, " must be ", dtype, ", got ", t.scalar_type());
  on_gpu(name, t);
  const int64_t s0 = t.stride(0), s1 = t.stride(1);
  if (c > 1 && s1 != 1)
    refuse(TG_E_LAYOUT, name, ": elements of a row must be contiguous (strides (", s0, ", ", s1, "))");
  if (r <= 1) return 0;   // one row: the stride says nothing
  if (s0 < c) refuse(TG_E_LAYOUT, name, ": rows overlap (strides (", s0, ", ", s1, "))");
  return s0;
}

void vector(const char* name, const Tensor& t, int64_t n) {
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(TG_E_SHAPE, name, " must be a contiguous vector of ", n, ", got ", t.sizes());
  on_gpu(name, t);
}
void f32_vector(const char* name, const Tensor& t, int64_t n) {
  vector(name, t, n);
  if (t.scalar_type() != at::kFloat) refuse(TG_E_DTYPE, name, " must be float32, got ", t.scalar_type());
}

// The GPU of a call's tensors, which has to be the current one: the launch goes there.
at::Device one_gpu(std::initializer_list<const Tensor*> all) {
  const Tensor* first = nullptr;
  for (const Tensor* t : all) {
    if (!t) continue;
    if (!first) first = t;
    else if (t->device() != first->device())
      refuse(TG_E_ARG, "tensors on ", first->device(), " and ", t->device());
  }
  const auto current = c10::hip::current_device();
  if (first->device().index() != current)
    refuse(TG_E_ARG, "tensors on ", first->device(), ", the current GPU is ", (int)current);
  return first->device();
}

Tensor make(at::IntArrayRef size, at::ScalarType t, at::Device dev) {
  return at::detail::empty_cuda(size, t, dev, std::nullopt);
}
const void* address(const Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
void* address(Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// A tensor of the caller's that the call writes: autograd sees that saved tensors have changed.
void written(const Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
// The results carry no history (the backward calls give the gradients): said once where a gradient would
// be lost without a word.
void no_history(const char* call, std::initializer_list<const Tensor*> inputs) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : inputs)
    if (t && t->requires_grad()) {
      TORCH_WARN_ONCE(call, ": an input requires a gradient, but results of the layer operators carry no autograd "
                      "history; use gemm_ep_backward and rms_norm_backward (and torch.no_grad() around the calls)");
      return;
    }
}

void check(int status) {
  if (status != TG_OK) refuse(status, tile_last_error());
}
void* stream_of(at::Device dev) { return (void*)c10::hip::getCurrentHIPStream(dev.index()).stream(); }

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
at::ScalarType scalar_type(const char* name, PyObject* o) {
  if (!THPDtype_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a torch.dtype or None, got %s", name, Py_TYPE(o)->tp_name);
    throw python_error();
  }
  return ((THPDtype*)o)->scalar_type;
}

// M, N, K of a product's operands
struct Extents {
  int64_t M, N, K, lda, ldb;
};
Extents extents(const Tensor& A, const Tensor& B, bool ta, bool tb) {
  Extents e;
  e.lda = matrix("A", A);
  e.ldb = matrix("B", B);
  e.M = A.size(ta ? 1 : 0);
  e.K = A.size(ta ? 0 : 1);
  e.N = B.size(tb ? 0 : 1);
  const int64_t kb = B.size(tb ? 1 : 0);
  if (kb != e.K) refuse(TG_E_SHAPE, "A has K = ", e.K, ", B has K = ", kb);
  return e;
}

// A, B, bias, act, residual, row_scale, col_scale, trans_a, trans_b, out_dtype, keep_z, out
PyObject* gemm_ep(PyObject* const* a) {
  const Tensor &A = *tensor("A", a[0]), &B = *tensor("B", a[1]);
  const Tensor *bias = tensor("bias", a[2], true), *res = tensor("residual", a[4], true);
  const Tensor *rs = tensor("row_scale", a[5], true), *cs = tensor("col_scale", a[6], true);
  const Tensor* given = tensor("out", a[11], true);
  const bool ta = truth(a[7]), tb = truth(a[8]), keep_z = truth(a[10]);
  const Extents e = extents(A, B, ta, tb);
  const int at = dtype_code("A", A.scalar_type()), bt = dtype_code("B", B.scalar_type());
  const bool eight = at == TG_FP8_E4M3 || at == TG_FP8_E5M2;
  const at::ScalarType out_t = a[9] != Py_None ? scalar_type("out_dtype", a[9])
                               : given         ? given->scalar_type()
                               : eight         ? at::kBFloat16
                                               : A.scalar_type();
  const int dt = dtype_code("out_dtype", out_t);
  tg_epilogue ep{};
  ep.act = (int32_t)integer(a[3]);
  if (bias) {
    vector("bias", *bias, e.N);
    if (!is_float(bias->scalar_type())) refuse(TG_E_DTYPE, "bias: unsupported dtype ", bias->scalar_type());
    ep.bias = address(bias);
    ep.bias_dtype = code_of(bias->scalar_type());
  }
  if (res) {
    ep.ld_residual = matrix("residual", *res, e.M, e.N, out_t);
    ep.residual = address(res);
  }
  if (rs) {
    f32_vector("row_scale", *rs, e.M);
    ep.row_scale = (const float*)address(rs);
  }
  if (cs) {
    f32_vector("col_scale", *cs, e.N);
    ep.col_scale = (const float*)address(cs);
  }
  const int64_t ldd = given ? matrix("out", *given, e.M, e.N, out_t) : 0;
  const at::Device dev = one_gpu({&A, &B, bias, res, rs, cs, given});
  Tensor out = given ? *given : make({e.M, e.N}, out_t, dev), Z, ws;
  if (keep_z) Z = make({e.M, e.N}, out_t, dev);
  ep.Z = address(Z);
  const int64_t nb = tile_gemm_ep_workspace(e.M, e.N, e.K, ta, tb, at);
  if (nb) ws = make({nb}, at::kByte, dev);
  check(tile_gemm_ep(address(&A), address(&B), address(out), e.M, e.N, e.K, e.lda, e.ldb, ldd, ta, tb, at, bt, dt,
                     &ep, address(ws), nb, stream_of(dev)));
  written(given);
  no_history("gemm_ep", {&A, &B, bias, res, rs, cs});
  if (given && !keep_z) {
    Py_INCREF(a[11]);
    return a[11];
  }
  if (!keep_z) return wrap(out);
  return Py_BuildValue("(NN)", wrap(out), wrap(Z));
}

// dY, A, B, Z, act, trans_a, trans_b, need_dA, need_dB, need_dbias, row_scale, col_scale
PyObject* gemm_ep_backward(PyObject* const* a) {
  const Tensor &dY = *tensor("dY", a[0]), &A = *tensor("A", a[1]), &B = *tensor("B", a[2]);
  const Tensor *Z = tensor("Z", a[3], true), *rs = tensor("row_scale", a[10], true), *cs = tensor("col_scale", a[11], true);
  const int act = (int)integer(a[4]);
  const bool ta = truth(a[5]), tb = truth(a[6]);
  const Extents e = extents(A, B, ta, tb);
  if (B.scalar_type() != A.scalar_type()) refuse(TG_E_DTYPE, "B must be ", A.scalar_type(), ", got ", B.scalar_type());
  const at::ScalarType st = A.scalar_type();
  const int t = dtype_code("A", st);
  const int64_t ldy = matrix("dY", dY, e.M, e.N, st);
  int64_t ldz = 0;
  if (act == TG_ACT_NONE) Z = nullptr;
  else if (!Z) refuse(TG_E_NULL, "an activation's gradient needs Z");
  else ldz = matrix("Z", *Z, e.M, e.N, st);
  if (rs) f32_vector("row_scale", *rs, e.M);
  if (cs) f32_vector("col_scale", *cs, e.N);
  const at::Device dev = one_gpu({&dY, &A, &B, Z, rs, cs});
  Tensor dZ, dA, dB, dbias, ws;
  if (act != TG_ACT_NONE || rs || cs) dZ = make({e.M, e.N}, st, dev);
  if (truth(a[7])) dA = make(A.sizes(), st, dev);
  if (truth(a[8])) dB = make(B.sizes(), st, dev);
  if (truth(a[9])) dbias = make({e.N}, at::kFloat, dev);
  const int64_t nb = tile_gemm_ep_bwd_workspace(e.M, e.N, e.K, ta, tb, t);
  if (nb) ws = make({nb}, at::kByte, dev);
  check(tile_gemm_ep_bwd_scaled(address(&dY), address(Z), address(&A), address(&B), (const float*)address(rs),
                                (const float*)address(cs), address(dZ), address(dA), address(dB),
                                (float*)address(dbias), e.M, e.N, e.K, ldy, ldz, e.lda, e.ldb, ta, tb, t, act,
                                address(ws), nb, stream_of(dev)));
  PyObject* z;
  if (dZ.defined()) {
    z = wrap(dZ);
  } else {
    z = a[0];
    Py_INCREF(z);
  }
  return Py_BuildValue("(NNNN)", z, wrap(dA), wrap(dB), wrap(dbias));
}

// X, weight, eps, residual, out_dtype, scale kind, h_out -> (y, scale, rstd, h)
PyObject* rms_norm(PyObject* const* a) {
  const Tensor &X = *tensor("X", a[0]), &W = *tensor("weight", a[1]);
  const Tensor *res = tensor("residual", a[3], true), *given = tensor("h_out", a[6], true);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  const int kind = (int)integer(a[5]);
  const int64_t ldx = matrix("X", X), rows = X.size(0), cols = X.size(1);
  const at::ScalarType st = X.scalar_type();
  const at::ScalarType out_t = a[4] != Py_None          ? scalar_type("out_dtype", a[4])
                               : kind == TG_SCALE_NONE ? st
                                                       : at::kFloat8_e4m3fn;
  const int t = dtype_code("X", st), yt = dtype_code("out_dtype", out_t);
  vector("weight", W, cols);
  if (W.scalar_type() != st && W.scalar_type() != at::kFloat)
    refuse(TG_E_DTYPE, "weight must be ", st, " or float32, got ", W.scalar_type());
  int64_t ldr = 0, ldh = 0;
  if (res) ldr = matrix("residual", *res, rows, cols, st);
  else if (given) refuse(TG_E_ARG, "h_out is the sum X + residual: it needs a residual");
  if (given) ldh = matrix("h_out", *given, rows, cols, st);
  const at::Device dev = one_gpu({&X, &W, res, given});
  Tensor h, S;
  if (given) h = *given;
  else if (res) h = make({rows, cols}, st, dev);
  Tensor y = make({rows, cols}, out_t, dev), rstd = make({rows}, at::kFloat, dev);
  if (kind == TG_SCALE_ROW) S = make({rows}, at::kFloat, dev);
  else if (kind == TG_SCALE_BLOCK) S = make({rows, cols / 32}, at::kFloat8_e8m0fnu, dev);
  check(tile_rmsnorm(address(&X), address(res), address(&W), address(h), address(y), address(S),
                     (float*)address(rstd), rows, cols, ldx, ldr, ldh, 0, (float)eps, t, code_of(W.scalar_type()), yt,
                     kind, stream_of(dev)));
  written(given);
  no_history("rms_norm", {&X, &W, res});
  PyObject* ph;
  if (given || !res) {
    ph = given ? a[6] : a[0];
    Py_INCREF(ph);
  } else {
    ph = wrap(h);
  }
  return Py_BuildValue("(NNNN)", wrap(y), wrap(S), wrap(rstd), ph);
}

// dY, h, weight, rstd, dH, need_dw -> (dX, dweight)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Tensor &dY = *tensor("dY", a[0]), &H = *tensor("h", a[1]), &W = *tensor("weight", a[2]);
  const Tensor &rstd = *tensor("rstd", a[3]), *dH = tensor("dH", a[4], true);
  const int64_t ldh = matrix("h", H), rows = H.size(0), cols = H.size(1);
  const at::ScalarType st = H.scalar_type();
  const int t = dtype_code("h", st);
  const int64_t ldy = matrix("dY", dY, rows, cols, st);
  vector("weight", W, cols);
  if (W.scalar_type() != st && W.scalar_type() != at::kFloat)
    refuse(TG_E_DTYPE, "weight must be ", st, " or float32, got ", W.scalar_type());
  f32_vector("rstd", rstd, rows);
  const int64_t ldd = dH ? matrix("dH", *dH, rows, cols, st) : 0;
  const at::Device dev = one_gpu({&dY, &H, &W, &rstd, dH});
  Tensor dX = make({rows, cols}, st, dev), dw, ws;
  if (truth(a[5])) dw = make({cols}, at::kFloat, dev);
  const int64_t nb = tile_rmsnorm_bwd_workspace(rows, cols, t);
  if (nb) ws = make({nb}, at::kByte, dev);
  check(tile_rmsnorm_bwd(address(&dY), address(&H), address(&W), (const float*)address(&rstd), address(dH), address(dX),
                         (float*)address(dw), rows, cols, ldy, ldh, ldd, 0, t, code_of(W.scalar_type()), address(ws),
                         nb, stream_of(dev)));
  return Py_BuildValue("(NN)", wrap(dX), wrap(dw));
}

// Argument count, and C++ exceptions as Python ones.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    PyObject* v = Py_BuildValue("(is)", r.status, r.why.c_str());
    if (v) {
      PyErr_SetObject(g_error, v);
      Py_DECREF(v);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error_class(PyObject*, PyObject* c) {
  Py_INCREF(c);
  Py_XSETREF(g_error, c);
  Py_RETURN_NONE;
}

#define TG_METHOD(f, n) {#f, (PyCFunction)(void (*)(void))(entry<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TG_METHOD(gemm_ep, 12), TG_METHOD(gemm_ep_backward, 12), TG_METHOD(rms_norm, 7),
                         TG_METHOD(rms_norm_backward, 6),
                         {"set_error_class", set_error_class, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
