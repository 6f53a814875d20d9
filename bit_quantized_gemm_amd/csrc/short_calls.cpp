// Python extension module `_short`: the short way into libatom for calls whose tensors are all well-formed.
//
// A call from Python through ctypes spends most of a small operator's time on the host: each new tensor is 1.3 us (0.5 from
// torch's factory called here, 0.2 as `fresh` makes it), the checks 2 to 3 us, the launch itself 3.3.  Each function here checks what its
// namesake in the Python binding documents, allocates the outputs on the current stream and calls the C ABI.  Anything that is
// not well-formed, or that the C ABI refuses, returns None, and the binding's full checks name the problem.  Host time of a call
// (us), the same checks in Python and here: linear_mxfp4 of one token 7.2 and 4.6, atom_rmsnorm_w8a8 10.6 and 5.1, atom_kv4_extend 10.6 and
// 5.5, atom_kv4_release 8.3 and 5.0.
//
// The addresses of the C entry points come from the binding (`bind`), so this module loads without the library.  What it holds of
// tensors is inlined from torch's headers: `built_for` names the torch and the Python that it was built with, and the binding
// leaves a module of another one alone.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "atom_kv4_pages.h"
#include "atom_mxfp4.h"
#include "atom_norm.h"
#include "atom_w8a8.h"

namespace {

// ---- the C entry points, by name
#define ATOM_CALLS(X)                                                                                                     \
  X(atom_quantize_mxfp4) X(atom_dequantize_mxfp4) X(atom_linear_mxfp4_workspace_bytes) X(atom_linear_mxfp4)               \
  X(atom_gemm_mxfp4)                                                                                                      \
  X(atom_rmsnorm_w8a8) X(atom_rmsnorm_mxfp4) X(atom_dequantize_w8a8) X(atom_kv4_extend) X(atom_kv4_release)
struct {
#define X(name) decltype(&::name) name;
  ATOM_CALLS(X)
#undef X
} lib = {};

PyObject* raw_stream = nullptr;                         // torch's function from a device's number to its current hipStream_t

PyObject* bind(PyObject*, PyObject* args) {
  PyObject *addresses, *stream;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &addresses, &stream)) return nullptr;
  Py_INCREF(stream);
  Py_XDECREF(raw_stream);
  raw_stream = stream;
#define X(name)                                                                                              \
  {                                                                                                          \
    PyObject* a = PyDict_GetItemString(addresses, #name);                                                    \
    void* p = a ? PyLong_AsVoidPtr(a) : nullptr;                                                             \
    if (PyErr_Occurred()) return nullptr;                                                                    \
    lib.name = reinterpret_cast<decltype(lib.name)>(p);                                                      \
  }
  ATOM_CALLS(X)
#undef X
  Py_RETURN_NONE;
}

// ---- tensors
// A plain torch.Tensor's value, else null (subclasses take the full way).
const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Here {                                           // the current device
  c10::Device device = c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice();
  bool has(const at::Tensor& t) const { return t.is_cuda() && t.device() == device; }
};
// The current stream; false with a Python error set.
bool stream_of(const Here& h, void*& stream) {
  PyObject* d = PyLong_FromLong(h.device.index());
  PyObject* s = d ? PyObject_CallFunctionObjArgs(raw_stream, d, nullptr) : nullptr;
  Py_XDECREF(d);
  if (!s) return false;
  stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

bool is16(const at::Tensor& t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }
int32_t kind(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? ATOM_BF16 : ATOM_FP16; }

// A contiguous tensor of this type and shape on the current device.
bool dense(const Here& h, const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t && h.has(*t) && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}
// 16-bit rows [rows, K] that may lie apart; the distance of two of them.
bool rows2d(const Here& h, const at::Tensor* t, int64_t& ld) {
  if (!t || !h.has(*t) || t->dim() != 2 || !is16(*t)) return false;
  const int64_t rows = t->size(0), K = t->size(1);
  if (rows < 1 || rows > ATOM_MAX_ROWS || K < 1 || K > ATOM_MAX_K || (t->stride(1) != 1 && K != 1)) return false;
  ld = rows > 1 ? t->stride(0) : K;
  return ld >= K;
}
// A bias or weights [n] of this type, or None.
bool vector(const Here& h, PyObject* o, at::ScalarType type, int64_t n, const void*& p) {
  p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!dense(h, t, type, {n})) return false;
  p = t->data_ptr();
  return true;
}
// A new tensor on the current device, as torch's factory makes it when it has found its way there: from the allocator that the
// factory takes.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type) {
  static c10::Allocator* const allocator = at::empty({1}, at::TensorOptions().device(c10::DeviceType::CUDA)).storage().allocator();
  return at::Tensor(at::detail::empty_generic(shape, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}

// The status of call(stream), without the interpreter's lock: a launch may wait for its queue.
template <class F>
int on_stream(const Here& h, F&& call) {
  void* stream = nullptr;
  if (!stream_of(h, stream)) throw python_error();
  PyThreadState* s = PyEval_SaveThread();
  const int status = call(stream);
  PyEval_RestoreThread(s);
  return status;
}
PyObject* otherwise() { Py_RETURN_NONE; }

int64_t groups_of(int64_t K) { return (K + ATOM_MX_GROUP - 1) / ATOM_MX_GROUP; }
bool integer(PyObject* o, int64_t& v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}

// ---- MXFP4
PyObject* linear_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {   // X, Wq, sw, bias
  HANDLE_TH_ERRORS
  const at::Tensor *x = n == 4 ? tensor(a[0]) : nullptr, *w = x ? tensor(a[1]) : nullptr, *s = w ? tensor(a[2]) : nullptr;
  if (!s || !lib.atom_linear_mxfp4 || !x->is_cuda()) return otherwise();
  const Here h;
  int64_t ld;
  const void* bias;
  if (!rows2d(h, x, ld) || w->dim() != 2) return otherwise();
  const int64_t M = x->size(0), K = x->size(1), N = w->size(0), g = groups_of(K);
  if (N < 1 || N > ATOM_MAX_ROWS || !dense(h, w, at::kByte, {N, g * (ATOM_MX_GROUP / 2)}) || !dense(h, s, at::kByte, {g, N, 8}) ||
      !vector(h, a[3], x->scalar_type(), N, bias))
    return otherwise();
  const int64_t need = lib.atom_linear_mxfp4_workspace_bytes((int32_t)M, (int32_t)N, (int32_t)K);
  if (need < 0) return otherwise();
  at::Tensor y = fresh({M, N}, x->scalar_type()), work;
  if (need) work = fresh({need}, at::kByte);
  void* const p = need ? work.data_ptr() : nullptr;
  const int status = on_stream(h, [&](void* stream) {
    return lib.atom_linear_mxfp4(x->data_ptr(), ld, kind(*x), w->data_ptr(), s->data_ptr(), bias, (int32_t)M, (int32_t)N, (int32_t)K,
                                 y.data_ptr(), p, need, stream);
  });
  return status ? otherwise() : THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

PyObject* gemm_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {   // Xq, sx, Wq, sw, K, bias, bf16, workspace
  HANDLE_TH_ERRORS
  const at::Tensor *x = n == 8 ? tensor(a[0]) : nullptr, *s = x ? tensor(a[1]) : nullptr, *w = s ? tensor(a[2]) : nullptr,
                   *t = w ? tensor(a[3]) : nullptr, *scratch = nullptr;
  int64_t K;
  if (!t || !lib.atom_gemm_mxfp4 || !x->is_cuda() || x->dim() != 2 || w->dim() != 2 || !integer(a[4], K) || K < 1 || K > ATOM_MAX_K)
    return otherwise();
  const Here h;
  const int64_t M = x->size(0), N = w->size(0), g = groups_of(K), bytes = g * (ATOM_MX_GROUP / 2);
  const bool bf16 = PyObject_IsTrue(a[6]) == 1;
  const void* bias;
  if (M < 1 || M > ATOM_MAX_ROWS || N < 1 || N > ATOM_MAX_ROWS || !dense(h, x, at::kByte, {M, bytes}) || !dense(h, s, at::kByte, {g, M, 8}) ||
      !dense(h, w, at::kByte, {N, bytes}) || !dense(h, t, at::kByte, {g, N, 8}) || !vector(h, a[5], bf16 ? at::kBFloat16 : at::kHalf, N, bias))
    return otherwise();
  if (a[7] != Py_None) {
    scratch = tensor(a[7]);
    if (!scratch || scratch->dim() != 1 || !dense(h, scratch, at::kByte, {scratch->numel()})) return otherwise();
  }
  at::Tensor y = fresh({M, N}, bf16 ? at::kBFloat16 : at::kHalf);
  const int status = on_stream(h, [&](void* stream) {
    return lib.atom_gemm_mxfp4(x->data_ptr(), s->data_ptr(), w->data_ptr(), t->data_ptr(), bias, (int32_t)M, (int32_t)N, (int32_t)K, bf16,
                               y.data_ptr(), scratch ? scratch->data_ptr() : nullptr, scratch ? scratch->numel() : 0, stream);
  });
  return status ? otherwise() : THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

PyObject* quantize_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {   // X
  HANDLE_TH_ERRORS
  const at::Tensor* x = n == 1 ? tensor(a[0]) : nullptr;
  if (!x || !lib.atom_quantize_mxfp4 || !x->is_cuda()) return otherwise();
  const Here h;
  int64_t ld;
  if (!rows2d(h, x, ld)) return otherwise();
  const int64_t rows = x->size(0), K = x->size(1), g = groups_of(K);
  at::Tensor q = fresh({rows, g * (ATOM_MX_GROUP / 2)}, at::kByte), s = fresh({g, rows, 8}, at::kByte);
  const int status = on_stream(h, [&](void* stream) {
    return lib.atom_quantize_mxfp4(x->data_ptr(), ld, kind(*x), (int32_t)rows, (int32_t)K, q.data_ptr(), s.data_ptr(), stream);
  });
  return status ? otherwise() : Py_BuildValue("(NN)", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)));
  END_HANDLE_TH_ERRORS
}

// Xq, sx, K, bf16: what packed rows stand for.
PyObject* dequantize(PyObject* const* a, Py_ssize_t n, bool mx) {
  const at::Tensor *q = n == 4 ? tensor(a[0]) : nullptr, *s = q ? tensor(a[1]) : nullptr;
  int64_t K;
  if (!s || !q->is_cuda() || q->dim() != 2 || !integer(a[2], K) || K < 1 || K > ATOM_MAX_K) return otherwise();
  const Here h;
  const int64_t rows = q->size(0), g = groups_of(K);
  if (rows < 1 || rows > ATOM_MAX_ROWS) return otherwise();
  if (mx ? !lib.atom_dequantize_mxfp4 || !dense(h, q, at::kByte, {rows, g * (ATOM_MX_GROUP / 2)}) || !dense(h, s, at::kByte, {g, rows, 8})
         : !lib.atom_dequantize_w8a8 || !dense(h, q, at::kChar, {rows, (K + 127) / 128 * 128}) || !dense(h, s, at::kFloat, {rows}))
    return otherwise();
  const bool bf16 = PyObject_IsTrue(a[3]) == 1;
  at::Tensor x = fresh({rows, K}, bf16 ? at::kBFloat16 : at::kHalf);
  const int status = on_stream(h, [&](void* stream) {
    return mx ? lib.atom_dequantize_mxfp4(q->data_ptr(), s->data_ptr(), (int32_t)rows, (int32_t)K, bf16, x.data_ptr(), stream)
              : lib.atom_dequantize_w8a8(q->data_ptr(), static_cast<const float*>(s->data_ptr()), (int32_t)rows, (int32_t)K, bf16,
                                         x.data_ptr(), stream);
  });
  return status ? otherwise() : THPVariable_Wrap(std::move(x));
}
PyObject* dequantize_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return dequantize(a, n, true);
  END_HANDLE_TH_ERRORS
}
PyObject* dequantize_w8a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return dequantize(a, n, false);
  END_HANDLE_TH_ERRORS
}

// ---- norm: X, weight, eps, residual
PyObject* rmsnorm(PyObject* const* a, Py_ssize_t n, bool mx) {
  const at::Tensor *x = n == 4 ? tensor(a[0]) : nullptr, *r = nullptr;
  if (!x || !x->is_cuda() || !lib.atom_rmsnorm_w8a8 || !lib.atom_rmsnorm_mxfp4 || !PyFloat_CheckExact(a[2])) return otherwise();
  const Here h;
  int64_t ld, ldr = 0;
  const void* w;
  if (!rows2d(h, x, ld)) return otherwise();
  const int64_t rows = x->size(0), K = x->size(1), g = groups_of(K);
  if (!vector(h, a[1], x->scalar_type(), K, w) || !w) return otherwise();
  if (a[3] != Py_None) {
    r = tensor(a[3]);
    if (!rows2d(h, r, ldr) || r->scalar_type() != x->scalar_type() || r->sizes() != x->sizes()) return otherwise();
  }
  const double eps = PyFloat_AS_DOUBLE(a[2]);
  at::Tensor q = mx ? fresh({rows, g * (ATOM_MX_GROUP / 2)}, at::kByte) : fresh({rows, (K + 127) / 128 * 128}, at::kChar);
  at::Tensor s = mx ? fresh({g, rows, 8}, at::kByte) : fresh({rows}, at::kFloat), sum;
  if (r) sum = fresh({rows, K}, x->scalar_type());
  const void* const pr = r ? r->data_ptr() : nullptr;
  void* const ph = r ? sum.data_ptr() : nullptr;
  const int status = on_stream(h, [&](void* stream) {
    return mx ? lib.atom_rmsnorm_mxfp4(x->data_ptr(), ld, pr, ldr, w, eps, kind(*x), (int32_t)rows, (int32_t)K, ph, K, q.data_ptr(),
                                       s.data_ptr(), stream)
              : lib.atom_rmsnorm_w8a8(x->data_ptr(), ld, pr, ldr, w, eps, kind(*x), (int32_t)rows, (int32_t)K, ph, K, q.data_ptr(),
                                      static_cast<float*>(s.data_ptr()), stream);
  });
  if (status) return otherwise();
  PyObject* last = Py_None;
  if (r) last = THPVariable_Wrap(std::move(sum));
  else Py_INCREF(last);
  return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)), last);
}
PyObject* rmsnorm_w8a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rmsnorm(a, n, false);
  END_HANDLE_TH_ERRORS
}
PyObject* rmsnorm_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rmsnorm(a, n, true);
  END_HANDLE_TH_ERRORS
}

// ---- the KV cache's bookkeeping: a state's lens, table and pool
struct State {
  const at::Tensor *lens, *table, *free, *state;
  int32_t batch, width, capacity;
  bool of(const Here& h, PyObject* l, PyObject* t, PyObject* f, PyObject* s) {
    lens = tensor(l), table = tensor(t), free = tensor(f), state = tensor(s);
    if (!table || !free || table->dim() != 2 || free->dim() != 1) return false;
    const int64_t b = table->size(0), w = table->size(1), c = free->size(0);
    if (b < 1 || b > (1 << 20) || w < 1 || w > (1 << 30) || c < 1 || c > (1 << 27)) return false;
    batch = (int32_t)b, width = (int32_t)w, capacity = (int32_t)c;
    return dense(h, lens, at::kInt, {b}) && dense(h, table, at::kInt, {b, w}) && dense(h, free, at::kInt, {c}) && dense(h, state, at::kInt, {2});
  }
};
template <class T>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

PyObject* kv4_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {   // lens, new, table, free, state, page, total
  HANDLE_TH_ERRORS
  const at::Tensor* more = n == 7 ? tensor(a[1]) : nullptr;
  int64_t page, total;
  if (!more || !lib.atom_kv4_extend || !more->is_cuda() || !integer(a[5], page) || !integer(a[6], total) || page < 1 || page > 256 ||
      total < 1 || total > ATOM_MAX_ROWS)
    return otherwise();
  const Here h;
  State s;
  if (!s.of(h, a[0], a[2], a[3], a[4]) || !dense(h, more, at::kInt, {s.batch})) return otherwise();
  at::Tensor slots = fresh({total}, at::kLong), start = fresh({s.batch + 1}, at::kInt), lens = fresh({s.batch}, at::kInt),
             state = fresh({2}, at::kInt);
  const int status = on_stream(h, [&](void* stream) {
    return lib.atom_kv4_extend(ptr<int32_t>(*s.lens), ptr<int32_t>(*more), ptr<int32_t>(*s.table), s.batch, s.width, (int32_t)page,
                               ptr<int32_t>(*s.free), s.capacity, ptr<int32_t>(*s.state), ptr<int64_t>(slots), (int32_t)total,
                               ptr<int32_t>(start), ptr<int32_t>(lens), ptr<int32_t>(state), stream);
  });
  if (status) return otherwise();
  return Py_BuildValue("(NNNN)", THPVariable_Wrap(std::move(slots)), THPVariable_Wrap(std::move(start)), THPVariable_Wrap(std::move(lens)),
                       THPVariable_Wrap(std::move(state)));
  END_HANDLE_TH_ERRORS
}

PyObject* kv4_release(PyObject*, PyObject* const* a, Py_ssize_t n) {   // done, lens, table, free, state, page
  HANDLE_TH_ERRORS
  const at::Tensor* done = n == 6 ? tensor(a[0]) : nullptr;
  int64_t page;
  if (!done || !lib.atom_kv4_release || !done->is_cuda() || !integer(a[5], page) || page < 1 || page > 256) return otherwise();
  const Here h;
  State s;
  if (!s.of(h, a[1], a[2], a[3], a[4]) || !dense(h, done, at::kBool, {s.batch})) return otherwise();
  at::Tensor lens = fresh({s.batch}, at::kInt), state = fresh({2}, at::kInt);
  const int status = on_stream(h, [&](void* stream) {
    return lib.atom_kv4_release(ptr<uint8_t>(*done), ptr<int32_t>(*s.lens), ptr<int32_t>(*s.table), s.batch, s.width, (int32_t)page,
                                ptr<int32_t>(*s.free), s.capacity, ptr<int32_t>(*s.state), ptr<int32_t>(lens), ptr<int32_t>(state), stream);
  });
  if (status) return otherwise();
  return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(lens)), THPVariable_Wrap(std::move(state)));
  END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, "bind(addresses, stream): the C entry points by name, and the function that gives a device's current stream"},
                         FAST(linear_mxfp4), FAST(gemm_mxfp4), FAST(quantize_mxfp4), FAST(dequantize_mxfp4), FAST(dequantize_w8a8), FAST(rmsnorm_w8a8),
                         FAST(rmsnorm_mxfp4), FAST(kv4_extend), FAST(kv4_release), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_short", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__short(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", ATOM_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
