// marshal.cpp -- the quick way from Python tensors to the C ABI for the calls of dg_block.hip
// (module _marshal). A decoding step's kernels run for 3 to 5 us; reading ten tensors' types,
// shapes, strides and addresses through Python's attributes alone takes 4.
//
// Each function takes its Python wrapper's arguments in order, tests every tensor, makes the
// outputs that are None, and calls the library on torch's current stream. It returns the
// wrapper's result, or None where anything is not as the call wants it, or where the tensors'
// GPU is not the current one: the wrapper then goes its own way, which raises the specific
// error, or switches the device. None means that the library has not been called. Once it has
// been, its status is raised from here: a call may have run, in place too, whatever it reports,
// and is never made a second time.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cstdint>
#include <exception>

#include "../../include/dg.h"

namespace {

// Addresses of the library's calls, set once by bind(): the library that the binding has loaded.
decltype(&dg_layernorm_fp8_1x128) p_layernorm;
decltype(&dg_layernorm_backward) p_layernorm_backward;
decltype(&dg_fp8_gemm_nt_gated_fp8) p_gated;
decltype(&dg_gated_backward_fp8) p_gated_backward;
decltype(&dg_dropout_add) p_dropout_add;
decltype(&dg_dropout_backward_fp8) p_dropout_backward;
PyObject* p_check;  // raises a status as the binding's exception

struct NotPlain {};  // something is not as the call wants it; thrown before the library is called

constexpr int64_t kBlock = 128;

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotPlain{};
  return THPVariable_Unpack(o);
}

// The first tensor of a call: contiguous, on the current GPU.
const at::Tensor& first(PyObject* o, int64_t dims) {
  const at::Tensor& t = tensor(o);
  if (!t.is_cuda() || !t.is_contiguous() || (dims >= 0 && t.dim() != dims)) throw NotPlain{};
  if (t.get_device() != c10::hip::current_device()) throw NotPlain{};
  return t;
}

int32_t float_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return DG_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return DG_DTYPE_BF16;
  throw NotPlain{};
}

void* plain(const at::Tensor& t, at::ScalarType type, const at::Tensor& x) {
  if (t.scalar_type() != type || t.device() != x.device() || !t.is_contiguous()) throw NotPlain{};
  return t.data_ptr();
}

// The address of o, a tensor of this type and shape on x's GPU.
void* ptr(PyObject* o, at::ScalarType type, int64_t n, const at::Tensor& x) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 1 || t.size(0) != n) throw NotPlain{};
  return plain(t, type, x);
}
void* ptr(PyObject* o, at::ScalarType type, int64_t m, int64_t n, const at::Tensor& x) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 2 || t.size(0) != m || t.size(1) != n) throw NotPlain{};
  return plain(t, type, x);
}
// The same of a shape like x's, for tensors of any shape.
void* ptr_like(PyObject* o, const at::Tensor& x) {
  const at::Tensor& t = tensor(o);
  if (!t.sizes().equals(x.sizes())) throw NotPlain{};
  return plain(t, x.scalar_type(), x);
}
template <class... A>
void* optional(PyObject* o, A... a) {
  return o == Py_None ? nullptr : ptr(o, a...);
}

bool truth(PyObject* o) {
  if (o == Py_True) return true;
  if (o == Py_False) return false;
  throw NotPlain{};
}
double number(PyObject* o) {
  if (!PyFloat_CheckExact(o)) throw NotPlain{};
  return PyFloat_AS_DOUBLE(o);
}
int64_t whole(PyObject* o) {
  if (!PyLong_CheckExact(o)) throw NotPlain{};
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (overflow) throw NotPlain{};
  return v;
}

// An owned reference that becomes part of the result.
struct Out {
  PyObject* o = nullptr;
  void* p = nullptr;
  ~Out() { Py_XDECREF(o); }
  void given(PyObject* x, void* ptr) {
    Py_INCREF(x);
    o = x;
    p = ptr;
  }
  void made(at::Tensor t) {
    p = t.data_ptr();
    o = THPVariable_Wrap(std::move(t));
    if (!o) throw NotPlain{};
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& x) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(x.device()));
}

// A float32 [n]: the given one, a new one for None, or nothing where none is needed.
void sums(Out& out, PyObject* o, bool need, int64_t n, const at::Tensor& x) {
  if (o != Py_None)
    out.given(o, ptr(o, at::kFloat, n, x));
  else if (need)
    out.made(empty({n}, at::kFloat, x));
  else
    out.given(Py_None, nullptr);
}

// codes and sf of an FP8 output [m, n]; returns whether sf is packed.
bool fp8_out(Out& codes, Out& sf, PyObject* oc, PyObject* os, bool ue8m0, int64_t m, int64_t n,
             const at::Tensor& x) {
  if (oc != Py_None)
    codes.given(oc, ptr(oc, at::kFloat8_e4m3fn, m, n, x));
  else
    codes.made(empty({m, n}, at::kFloat8_e4m3fn, x));
  const int64_t kb = n / kBlock, words = (kb + 3) / 4;
  if (os == Py_None) {
    sf.made(ue8m0 ? empty({m, words}, at::kInt, x) : empty({m, kb}, at::kFloat, x));
    return ue8m0;
  }
  const bool packed = tensor(os).scalar_type() == at::kInt;
  sf.given(os, ptr(os, packed ? at::kInt : at::kFloat, m, packed ? words : kb, x));
  return packed;
}

void* stream_of(const at::Tensor& x) {
  return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)x.get_device()).stream();
}

// The library's call, without Python's lock: a launch may wait for room in its queue. An exception of
// it becomes a status: thrown on, it would read as a call that was not made.
template <class F, class... A>
dg_status run(F f, A... a) {
  PyThreadState* state = PyEval_SaveThread();
  dg_status s = DG_ERR_LAUNCH;
  try {
    s = f(a...);
  } catch (const std::exception&) {
  }
  PyEval_RestoreThread(state);
  return s;
}

// The outputs of a call that was made, or nullptr with a Python exception set.
template <class... O>
PyObject* result(dg_status s, O&... out) {
  if (s != DG_OK) {
    PyObject* r = PyObject_CallFunction(p_check, "i", (int)s);
    Py_XDECREF(r);
    if (r) PyErr_Format(PyExc_RuntimeError, "status %d", (int)s);
    return nullptr;
  }
  if constexpr (sizeof...(O) == 1) return (Py_INCREF(out.o), ...), (out.o, ...);
  else return PyTuple_Pack(sizeof...(O), out.o...);
}

// f(args): its result or the exception it set, and None for whatever it threw before the
// library's call.
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n == N) return F(args);
  } catch (const NotPlain&) {
  } catch (const std::exception&) {  // no memory for an output
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// x, weight, bias, eps, residual, h, mean, rstd, codes, sf, ue8m0, dropout_p, rng, subsequence
PyObject* layernorm(PyObject* const* a) {
  const at::Tensor& x = first(a[0], 2);
  const int64_t M = x.size(0), K = x.size(1);
  const at::Tensor& w = tensor(a[1]);
  const at::ScalarType t = x.scalar_type(), wt = w.scalar_type();
  const int32_t xc = float_code(x), wc = float_code(w);
  void* wp = ptr(a[1], wt, K, x);
  void* bias = optional(a[2], wt, K, x);
  const double eps = number(a[3]), p = number(a[11]);
  void* r = optional(a[4], t, M, K, x);
  void* h = optional(a[5], t, M, K, x);
  void* mean = optional(a[6], at::kFloat, M, x);
  void* rstd = optional(a[7], at::kFloat, M, x);
  void* rng = optional(a[12], at::kLong, 2, x);
  const int64_t sub = whole(a[13]);
  Out codes, sf;
  const bool packed = fp8_out(codes, sf, a[8], a[9], truth(a[10]), M, K, x);
  return result(run(p_layernorm, x.data_ptr(), r, xc, wp, bias, wc, (float)eps, p, (const int64_t*)rng, sub, h,
                            (float*)mean, (float*)rstd, codes.p, sf.p, packed, M, K, stream_of(x)),
                codes, sf);
}

// dy, h, weight, mean, rstd, dh, dx, dweight, dbias, need_dbias
PyObject* layernorm_backward(PyObject* const* a) {
  const at::Tensor& h = first(a[1], 2);
  const int64_t M = h.size(0), K = h.size(1);
  const at::Tensor& w = tensor(a[2]);
  const at::ScalarType t = h.scalar_type();
  const int32_t hc = float_code(h), wc = float_code(w);
  void* dy = ptr(a[0], t, M, K, h);
  void* wp = ptr(a[2], w.scalar_type(), K, h);
  void* mean = ptr(a[3], at::kFloat, M, h);
  void* rstd = ptr(a[4], at::kFloat, M, h);
  void* dh = optional(a[5], t, M, K, h);
  Out dx, dw, db;
  if (a[6] != Py_None) dx.given(a[6], ptr(a[6], t, M, K, h));
  else dx.made(at::empty_like(h));
  sums(dw, a[7], true, K, h);
  sums(db, a[8], truth(a[9]), K, h);
  return result(run(p_layernorm_backward, dy, dh, h.data_ptr(), hc, wp, wc, (const float*)mean, (const float*)rstd,
                                     dx.p, (float*)dw.p, (float*)db.p, M, K, stream_of(h)),
                dx, dw, db);
}

// a, b, a_sf, b_sf, bias, activation code, pre, codes, sf, ue8m0
PyObject* gated(PyObject* const* a) {
  const at::Tensor& x = first(a[0], 2);
  const int64_t M = x.size(0), K = x.size(1), KB = K / kBlock;
  const at::Tensor& b = tensor(a[1]);
  const auto fp8 = [](const at::Tensor& t) {
    return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte;
  };
  if (!fp8(x) || !fp8(b) || b.dim() != 2 || b.size(0) % 2) throw NotPlain{};
  const int64_t N = b.size(0), I = N / 2;
  void* bp = ptr(a[1], b.scalar_type(), N, K, x);
  const bool a_packed = tensor(a[2]).scalar_type() == at::kInt;
  void* asf = ptr(a[2], a_packed ? at::kInt : at::kFloat, M, a_packed ? (KB + 3) / 4 : KB, x);
  void* bsf = ptr(a[3], at::kFloat, (N + kBlock - 1) / kBlock, KB, x);
  const int32_t bias_code = a[4] == Py_None ? 0 : float_code(tensor(a[4]));
  void* bias = a[4] == Py_None ? nullptr : ptr(a[4], tensor(a[4]).scalar_type(), N, x);
  const int64_t act = whole(a[5]);
  void* pre = optional(a[6], at::kBFloat16, M, N, x);
  Out codes, sf;
  const bool packed = fp8_out(codes, sf, a[7], a[8], truth(a[9]), M, I, x);
  return result(run(p_gated, x.data_ptr(), bp, codes.p, sf.p, packed, asf, a_packed, (const float*)bsf, bias,
                        bias_code, (int32_t)act, pre, M, I, K, stream_of(x)),
                codes, sf);
}

// dh, pre, activation code, codes, sf, dbias, need_dbias, ue8m0
PyObject* gated_backward(PyObject* const* a) {
  const at::Tensor& dh = first(a[0], 2);
  if (dh.scalar_type() != at::kBFloat16) throw NotPlain{};
  const int64_t M = dh.size(0), I = dh.size(1);
  void* pre = ptr(a[1], at::kBFloat16, M, 2 * I, dh);
  const int64_t act = whole(a[2]);
  Out codes, sf, db;
  const bool packed = fp8_out(codes, sf, a[3], a[4], truth(a[7]), M, 2 * I, dh);
  sums(db, a[5], truth(a[6]), 2 * I, dh);
  return result(run(p_gated_backward, dh.data_ptr(), pre, (int32_t)act, codes.p, sf.p, packed, (float*)db.p, M, I,
                                 stream_of(dh)),
                codes, sf, db);
}

// x, p, rng, subsequence, residual, out
PyObject* dropout_add(PyObject* const* a) {
  const at::Tensor& x = first(a[0], -1);
  const int32_t xc = float_code(x);
  const double p = number(a[1]);
  void* rng = optional(a[2], at::kLong, 2, x);
  const int64_t sub = whole(a[3]);
  void* r = a[4] == Py_None ? nullptr : ptr_like(a[4], x);
  Out out;
  if (a[5] != Py_None) out.given(a[5], ptr_like(a[5], x));
  else out.made(at::empty_like(x));
  return result(run(p_dropout_add, x.data_ptr(), r, xc, p, (const int64_t*)rng, sub, out.p, x.numel(), stream_of(x)),
                out);
}

// dy, p, rng, subsequence, codes, sf, dbias, need_dbias, ue8m0
PyObject* dropout_backward(PyObject* const* a) {
  const at::Tensor& dy = first(a[0], 2);
  const int64_t M = dy.size(0), K = dy.size(1);
  const int32_t code = float_code(dy);
  const double p = number(a[1]);
  void* rng = optional(a[2], at::kLong, 2, dy);
  const int64_t sub = whole(a[3]);
  Out codes, sf, db;
  const bool packed = fp8_out(codes, sf, a[4], a[5], truth(a[8]), M, K, dy);
  sums(db, a[6], truth(a[7]), K, dy);
  return result(run(p_dropout_backward, dy.data_ptr(), code, p, (const int64_t*)rng, sub, codes.p, sf.p, packed,
                                   (float*)db.p, M, K, stream_of(dy)),
                codes, sf, db);
}

// bind(addresses of the six calls, in the order of their declaration above; check)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[6];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "KKKKKKO", f, f + 1, f + 2, f + 3, f + 4, f + 5, &check)) return nullptr;
  Py_INCREF(check);
  Py_XDECREF(p_check);
  p_check = check;
  p_layernorm = (decltype(p_layernorm))f[0];
  p_layernorm_backward = (decltype(p_layernorm_backward))f[1];
  p_gated = (decltype(p_gated))f[2];
  p_gated_backward = (decltype(p_gated_backward))f[3];
  p_dropout_add = (decltype(p_dropout_add))f[4];
  p_dropout_backward = (decltype(p_dropout_backward))f[5];
  Py_RETURN_NONE;
}

template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, (PyCFunction)(void (*)(void))(_PyCFunctionFast)call<N, F>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    method<14, layernorm>("layernorm"),
    method<10, layernorm_backward>("layernorm_backward"),
    method<10, gated>("gated"),
    method<8, gated_backward>("gated_backward"),
    method<6, dropout_add>("dropout_add"),
    method<9, dropout_backward>("dropout_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILD_ID", DG_BUILD_ID) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
