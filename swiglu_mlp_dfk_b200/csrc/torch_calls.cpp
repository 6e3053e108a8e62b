// torch_calls.cpp -- the block-scaled FP8 entry points called from Python: the
// operands' checks, the outputs' allocation and the C call in one step.
//
// On a small tensor such a call is bound by its host side.  Each function below
// takes the arguments of the Python function of the same name without its stream
// and either makes the whole call (on the operands' device, which must be the
// current one, and its current stream) or returns None without having done
// anything, and the Python function goes on: it names a refused argument,
// changes the device, reports an error.  A call takes 4.2 to 5.7 us here where the
// same steps in Python take 8.5 to 11.7 (the launch itself: 3).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>

#include "dfk.h"

namespace {

decltype(&dfk_quant_fp8_block) c_quant;
decltype(&dfk_add_rmsnorm_fp8_block) c_norm;
decltype(&dfk_gemm_fp8_block) c_gemm;
decltype(&dfk_swiglu_gate_up_fp8_block) c_gate_up;

constexpr at::ScalarType CODES = at::kFloat8_e4m3fn;

// A call's device and whether every operand so far is as it should be.
struct Call {
  int dev = -1;
  bool ok = true;

  // `o` as a tensor of this type on the call's device, contiguous (else a
  // tensor of the type alone, to go on with: `ok` is false then).
  const at::Tensor *operand(PyObject *o, at::ScalarType type, int dims) {
    static const at::Tensor none;
    ok = ok && THPVariable_CheckExact(o);
    if (!ok) return &none;
    const at::Tensor &t = THPVariable_Unpack(o);
    const at::ScalarType have = t.scalar_type();
    ok = t.is_cuda() && t.dim() == dims && t.is_contiguous() &&
         (have == type || (type == CODES && have == at::kByte));
    if (!ok) return &none;
    if (dev < 0) dev = t.get_device();
    ok = t.get_device() == dev;
    for (int d = 0; d < dims; ++d) ok = ok && t.size(d) <= INT_MAX;
    return &t;
  }
  void shape(const at::Tensor *t, int64_t rows, int64_t cols) {
    ok = ok && t->size(0) == rows && t->size(1) == cols;
  }
  bool ready() const { return ok && dev == c10::cuda::current_device(); }
};

// An output: the given tensor or, for None, a new one.
struct Out {
  PyObject *given;
  at::Tensor made;
  at::ScalarType type;
  int64_t rows, cols;

  Out(Call &c, PyObject *o, at::ScalarType t, int64_t r, int64_t n)
      : given(o == Py_None ? nullptr : o), type(t), rows(r), cols(n) {
    if (given) c.shape(c.operand(given, type, 2), rows, cols);
  }
  void *data(int dev) {
    if (given) return THPVariable_Unpack(given).data_ptr();
    made = at::empty({rows, cols}, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
    return made.data_ptr();
  }
  PyObject *object() {
    if (!given) return THPVariable_Wrap(std::move(made));
    Py_INCREF(given);
    return given;
  }
};

int64_t groups(int64_t k) { return (k + 127) >> 7; }

// The C call without the interpreter's lock.
template <typename F>
bool launched(int dev, F &&call) {
  void *stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = call(stream);
  Py_END_ALLOW_THREADS
  return status == DFK_OK;
}

PyObject *tuple_of(PyObject *a, PyObject *b, PyObject *c = nullptr) {
  PyObject *t = a && b ? PyTuple_New(c ? 3 : 2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  if (c) PyTuple_SET_ITEM(t, 2, c);
  return t;
}

// quant(x, q, s)
PyObject *quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 3 || !c_quant) Py_RETURN_NONE;
  const at::Tensor *x = c.operand(a[0], at::kBFloat16, 2);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t M = x->size(0), K = x->size(1);
  Out q(c, a[1], CODES, M, K), s(c, a[2], at::kFloat, groups(K), M);
  if (!c.ready()) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView below;
  void *pq = q.data(c.dev), *ps = s.data(c.dev);
  if (!launched(c.dev, [&](void *st) {
        return c_quant(x->data_ptr(), pq, static_cast<float *>(ps), static_cast<int>(M),
                       static_cast<int>(K), st);
      }))
    Py_RETURN_NONE;
  return tuple_of(q.object(), s.object());
  END_HANDLE_TH_ERRORS
}

// norm(x, residual, gamma, eps, residual_out, q, s)
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 7 || !c_norm) Py_RETURN_NONE;
  const bool has_res = a[1] != Py_None;
  const at::Tensor *x = c.operand(a[0], at::kBFloat16, 2);
  const at::Tensor *gamma = c.operand(a[2], at::kBFloat16, 1);
  if (!c.ok || !PyFloat_Check(a[3]) || (!has_res && a[4] != Py_None)) Py_RETURN_NONE;
  const int64_t M = x->size(0), D = x->size(1);
  c.ok = gamma->size(0) == D;
  const at::Tensor *res = has_res ? c.operand(a[1], at::kBFloat16, 2) : nullptr;
  if (!c.ok) Py_RETURN_NONE;
  if (has_res) c.shape(res, M, D);
  Out r(c, a[4], at::kBFloat16, M, D), q(c, a[5], CODES, M, D),
      s(c, a[6], at::kFloat, groups(D), M);
  if (!c.ready()) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView below;
  void *pr = has_res ? r.data(c.dev) : nullptr, *pq = q.data(c.dev), *ps = s.data(c.dev);
  const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[3]));
  if (!launched(c.dev, [&](void *st) {
        return c_norm(x->data_ptr(), has_res ? res->data_ptr() : nullptr, gamma->data_ptr(), eps,
                      pr, pq, static_cast<float *>(ps), static_cast<int>(M), static_cast<int>(D),
                      st);
      }))
    Py_RETURN_NONE;
  PyObject *last = Py_None;
  if (has_res) last = r.object();
  else Py_INCREF(last);
  return last ? tuple_of(q.object(), s.object(), last) : nullptr;
  END_HANDLE_TH_ERRORS
}

// A product's operands: activations and one weight matrix, with their scales.
struct Operands {
  const at::Tensor *qx, *sx, *qw, *sw;
  int64_t M = 0, K = 0, N = 0;

  Operands(Call &c, PyObject *const *a)
      : qx(c.operand(a[0], CODES, 2)), sx(c.operand(a[1], at::kFloat, 2)),
        qw(c.operand(a[2], CODES, 2)), sw(c.operand(a[3], at::kFloat, 2)) {
    if (!c.ok) return;
    M = qx->size(0);
    K = qx->size(1);
    N = qw->size(0);
    c.ok = qw->size(1) == K;
    c.shape(sx, groups(K), M);
    c.shape(sw, groups(N), groups(K));
  }
};

// gemm(q_x, s_x, q_w, s_w, y)
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 5 || !c_gemm) Py_RETURN_NONE;
  const Operands o(c, a);
  if (!c.ok) Py_RETURN_NONE;
  Out y(c, a[4], at::kBFloat16, o.M, o.N);
  if (!c.ready()) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView below;
  void *py = y.data(c.dev);
  if (!launched(c.dev, [&](void *st) {
        return c_gemm(o.qx->data_ptr(), static_cast<const float *>(o.sx->data_ptr()),
                      o.qw->data_ptr(), static_cast<const float *>(o.sw->data_ptr()), py,
                      static_cast<int>(o.M), static_cast<int>(o.K), static_cast<int>(o.N), st);
      }))
    Py_RETURN_NONE;
  return y.object();
  END_HANDLE_TH_ERRORS
}

// gate_up(q_x, s_x, q_gate, s_gate, q_up, s_up, fp8_out, h, q_h, s_h)
PyObject *gate_up(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 10 || !c_gate_up || !PyBool_Check(a[6])) Py_RETURN_NONE;
  const bool codes = a[6] == Py_True;
  if (codes ? a[7] != Py_None : a[8] != Py_None || a[9] != Py_None) Py_RETURN_NONE;
  const Operands o(c, a);
  const at::Tensor *qu = c.operand(a[4], CODES, 2), *su = c.operand(a[5], at::kFloat, 2);
  if (!c.ok) Py_RETURN_NONE;
  c.shape(qu, o.N, o.K);
  c.shape(su, groups(o.N), groups(o.K));
  Out h(c, a[7], at::kBFloat16, o.M, o.N), qh(c, a[8], CODES, o.M, o.N),
      sh(c, a[9], at::kFloat, groups(o.N), o.M);
  if (!c.ready()) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView below;
  void *ph = codes ? nullptr : h.data(c.dev), *pq = codes ? qh.data(c.dev) : nullptr,
       *ps = codes ? sh.data(c.dev) : nullptr;
  if (!launched(c.dev, [&](void *st) {
        return c_gate_up(o.qx->data_ptr(), static_cast<const float *>(o.sx->data_ptr()),
                         o.qw->data_ptr(), static_cast<const float *>(o.sw->data_ptr()),
                         qu->data_ptr(), static_cast<const float *>(su->data_ptr()), ph, pq,
                         static_cast<float *>(ps), static_cast<int>(o.M), static_cast<int>(o.K),
                         static_cast<int>(o.N), st);
      }))
    Py_RETURN_NONE;
  return codes ? tuple_of(qh.object(), sh.object()) : h.object();
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the four C entry points, in the order above)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[4];
  if (n != 4) return PyErr_Format(PyExc_TypeError, "four addresses");
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  c_quant = reinterpret_cast<decltype(c_quant)>(p[0]);
  c_norm = reinterpret_cast<decltype(c_norm)>(p[1]);
  c_gemm = reinterpret_cast<decltype(c_gemm)>(p[2]);
  c_gate_up = reinterpret_cast<decltype(c_gate_up)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"), method<quant>("quant"), method<norm>("norm"),
                         method<gemm>("gemm"), method<gate_up>("gate_up"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dfk_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dfk_torch() { return PyModule_Create(&module); }
