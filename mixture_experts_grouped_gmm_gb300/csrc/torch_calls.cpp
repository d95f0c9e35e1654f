// The host side of the operators whose calls take longer than their kernels at
// decode sizes: arguments read, outputs allocated and the C entry called without
// a Python frame per step.  One token's routing takes 4.9 us a call this way,
// against 15.9 through ctypes and torch.empty (its kernel 3.5).
//
// A function takes what its Python caller (moe.py, fp4.py) was given and
// returns the outputs; None where the arguments are not the plain case (another
// type or layout, a CPU tensor), which the caller then checks, mends or refuses;
// or an int, the C entry's negative return code.  Where the program has other
// Python threads, allocations and the C call run without the interpreter's lock:
// either may wait (for memory, for a place in a full launch queue), and the other
// threads go on meanwhile.  No step of a computation is here, and the library is reached through the addresses that bind() is given
// (those of the loaded libmgemm.so).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "../../include/mgemm.h"

namespace {

decltype(&mgemm_route) p_route = nullptr;
decltype(&mgemm_route_bwd) p_route_bwd = nullptr;
decltype(&mgemm_quant_fp4) p_quant = nullptr;
decltype(&mgemm_dequant_fp4) p_dequant = nullptr;
decltype(&mgemm_fp4_scale_bytes) p_scale_bytes = nullptr;
decltype(&mgemm_gmm_fp4_workspace_bytes) p_workspace_bytes = nullptr;
decltype(&mgemm_gmm_fp4) p_gmm = nullptr;

// The tensor of an argument; nullptr for anything else (None among it).
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
bool on_gpu(const at::Tensor *t, at::ScalarType type) { return t && t->is_cuda() && t->scalar_type() == type; }
// the same on the device of another tensor
bool beside(const at::Tensor *t, at::ScalarType type, const at::Tensor &other) {
  return on_gpu(t, type) && t->get_device() == other.get_device();
}

mgemm_stream_t stream_of(const at::Tensor &t) {
  return reinterpret_cast<mgemm_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}
PyObject *code(int rc) { return PyLong_FromLong(rc); }

// An int argument; sets `bad` for anything that is none.
int64_t integer(PyObject *o, bool &bad) {
  const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : (bad = true, 0);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad = true;
  }
  return v;
}
bool small(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }

// C++ exceptions (an allocation that fails) become Python's.
template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *type = PyObject_GetAttrString(PyImport_AddModule("torch"), "OutOfMemoryError");
    PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// Gives up the interpreter's lock while it lives, if there is another thread that could take it (giving it up and
// taking it back is 0.7 us of a call's 5).
struct Unlocked {
  PyThreadState *state = nullptr;
  Unlocked() {
    PyThreadState *first = PyInterpreterState_ThreadHead(PyInterpreterState_Get());
    if (first && PyThreadState_Next(first)) state = PyEval_SaveThread();
  }
  Unlocked(const Unlocked &) = delete;
  ~Unlocked() {
    if (state) PyEval_RestoreThread(state);
  }
};

PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// bind(addresses): a tuple of the entries' addresses, in the order below.
PyObject *bind(PyObject *, PyObject *arg) {
  void *p[7];
  if (!PyTuple_Check(arg) || PyTuple_GET_SIZE(arg) != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes a tuple of 7 addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(arg, i));
    if (PyErr_Occurred()) return nullptr;
  }
  p_route = reinterpret_cast<decltype(p_route)>(p[0]);
  p_route_bwd = reinterpret_cast<decltype(p_route_bwd)>(p[1]);
  p_quant = reinterpret_cast<decltype(p_quant)>(p[2]);
  p_dequant = reinterpret_cast<decltype(p_dequant)>(p[3]);
  p_scale_bytes = reinterpret_cast<decltype(p_scale_bytes)>(p[4]);
  p_workspace_bytes = reinterpret_cast<decltype(p_workspace_bytes)>(p[5]);
  p_gmm = reinterpret_cast<decltype(p_gmm)>(p[6]);
  Py_RETURN_NONE;
}

// Logits [T, E] with unit columns: 0 float32, 1 bf16, -1 another case.
int logits_type(const at::Tensor *l) {
  if (!l || !l->is_cuda() || l->dim() != 2 || l->stride(1) != 1 || l->stride(0) < l->size(1)) return -1;
  return l->scalar_type() == at::kFloat ? 0 : l->scalar_type() == at::kBFloat16 ? 1 : -1;
}

// route(logits, topk, scoring, bias, n_group, topk_group, group_top, renormalize, scale) -> (weights, ids)
PyObject *route(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 9 || !p_route) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *l = tensor(a[0]), *b = tensor(a[3]);
    const int type = logits_type(l);
    if (type >= 0 && l->requires_grad() && c10::GradMode::is_enabled()) Py_RETURN_NONE;  // (a differentiable call)
    if (type < 0 || (a[3] != Py_None && !(beside(b, at::kFloat, *l) && b->numel() == l->size(1) && b->is_contiguous())))
      Py_RETURN_NONE;
    bool bad = false;
    int64_t v[6];
    static const int at_[6] = {1, 2, 4, 5, 6, 7};
    for (int i = 0; i < 6; ++i) {
      v[i] = integer(a[at_[i]], bad);
      bad |= !small(v[i]);
    }
    const double scale = PyFloat_Check(a[8]) ? PyFloat_AS_DOUBLE(a[8]) : (bad = true, 0.0);
    const int64_t T = l->size(0), E = l->size(1);
    if (bad || !small(E) || v[0] < 1 || v[0] > MGEMM_ROUTE_MAX_TOPK) Py_RETURN_NONE;
    at::Tensor w, ids;
    int rc;
    {
      const Unlocked unlocked;
      w = empty({T, v[0]}, at::kFloat, l->device());
      ids = empty({T, v[0]}, at::kInt, l->device());
      rc = p_route(l->data_ptr(), type, l->stride(0), b ? b->data_ptr<float>() : nullptr, T, (int)E, (int)v[0], (int)v[1],
                   (int)v[2], (int)v[3], (int)v[4], v[5] != 0, (float)scale, w.data_ptr<float>(), ids.data_ptr<int32_t>(),
                   stream_of(*l));
    }
    return rc ? code(rc) : pair(std::move(w), std::move(ids));
  });
}

// route_bwd(grad_weights, logits, weights, ids, scoring, renormalize, scale) -> grad_logits
PyObject *route_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7 || !p_route_bwd) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *g = tensor(a[0]), *l = tensor(a[1]), *w = tensor(a[2]), *ids = tensor(a[3]);
    const int type = logits_type(l);
    if (type < 0 || !beside(g, at::kFloat, *l) || !beside(w, at::kFloat, *l) || !beside(ids, at::kInt, *l)) Py_RETURN_NONE;
    if (ids->dim() != 2 || ids->size(0) != l->size(0) || g->sizes() != ids->sizes() || w->sizes() != ids->sizes() ||
        !g->is_contiguous() || !w->is_contiguous() || !ids->is_contiguous())
      Py_RETURN_NONE;
    bool bad = false;
    const int64_t scoring = integer(a[4], bad), renorm = integer(a[5], bad);
    const double scale = PyFloat_Check(a[6]) ? PyFloat_AS_DOUBLE(a[6]) : (bad = true, 0.0);
    const int64_t T = l->size(0), E = l->size(1), k = ids->size(1);
    if (bad || !small(scoring) || !small(E) || !small(k)) Py_RETURN_NONE;
    at::Tensor out;
    int rc;
    {
      const Unlocked unlocked;
      out = empty({T, E}, l->scalar_type(), l->device());
      rc = p_route_bwd(g->data_ptr<float>(), l->data_ptr(), type, l->stride(0), w->data_ptr<float>(),
                       ids->data_ptr<int32_t>(), T, (int)E, (int)k, (int)scoring, renorm != 0, (float)scale, out.data_ptr(),
                       E, stream_of(*l));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

// quantize(x, format) -> (storage, codes address, scales address, row scales address or None, (E, N, K))
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 2 || !p_quant) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *x = tensor(a[0]);
    bool bad = false;
    const int64_t fmt = integer(a[1], bad);
    if (bad || !on_gpu(x, at::kBFloat16) || (x->dim() != 2 && x->dim() != 3)) Py_RETURN_NONE;
    const int d = (int)x->dim();
    const int64_t E = d == 3 ? x->size(0) : 1, N = x->size(d - 2), K = x->size(d - 1), ld = x->stride(d - 2);
    if (x->stride(d - 1) != 1 || ld < K || (E > 1 && x->stride(0) != N * ld) || !small(E) || !small(K) || ld % 8 ||
        reinterpret_cast<uintptr_t>(x->data_ptr()) % 16)
      Py_RETURN_NONE;
    const int64_t per = p_scale_bytes((int)fmt, N, (int)K);
    if (per < 0) Py_RETURN_NONE;
    const int64_t n_codes = (E * N * (K / 2) + 255) / 256 * 256, n_scales = E * per;
    const bool rows = fmt == MGEMM_NVFP4;
    at::Tensor s;
    uint8_t *p, *r;
    int rc;
    {
      const Unlocked unlocked;
      s = empty({n_codes + n_scales + (rows ? 4 * E * N : 0)}, at::kByte, x->device());
      p = s.data_ptr<uint8_t>();
      r = rows ? p + n_codes + n_scales : nullptr;
      rc = p_quant(x->data_ptr(), (int)E, N, (int)K, ld, (int)fmt, p, p + n_codes, reinterpret_cast<float *>(r),
                   stream_of(*x));
    }
    if (rc) return code(rc);
    PyObject *t = THPVariable_Wrap(std::move(s));
    if (!t) return nullptr;
    if (!rows)
      return Py_BuildValue("(N(LLO)(LLL))", t, (long long)(uintptr_t)p, (long long)(uintptr_t)(p + n_codes), Py_None,
                           (long long)E, (long long)N, (long long)K);
    return Py_BuildValue("(N(LLL)(LLL))", t, (long long)(uintptr_t)p, (long long)(uintptr_t)(p + n_codes),
                         (long long)(uintptr_t)r, (long long)E, (long long)N, (long long)K);
  });
}

// The three addresses of a 4-bit tensor (the last may be None).
bool addresses(PyObject *o, uintptr_t (&p)[3]) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) return false;
  bool bad = false;
  for (int i = 0; i < 3; ++i) {
    PyObject *v = PyTuple_GET_ITEM(o, i);
    p[i] = v == Py_None ? 0 : (uintptr_t)integer(v, bad);
  }
  return !bad;
}
bool shape3(PyObject *o, int64_t (&v)[3]) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) return false;
  bool bad = false;
  for (int i = 0; i < 3; ++i) v[i] = integer(PyTuple_GET_ITEM(o, i), bad);
  return !bad && small(v[0]) && small(v[1]) && small(v[2]);
}

// dequantize(addresses, shape, format, device index) -> bf16 [E, N, K]
PyObject *dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 4 || !p_dequant) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    uintptr_t p[3];
    int64_t s[3];
    bool bad = false;
    const int64_t fmt = integer(a[2], bad), dev = integer(a[3], bad);
    if (bad || !addresses(a[0], p) || !shape3(a[1], s) || dev < 0 || dev > 63) Py_RETURN_NONE;
    at::Tensor out;
    int rc;
    {
      const Unlocked unlocked;
      out = empty({s[0], s[1], s[2]}, at::kBFloat16, at::Device(at::kCUDA, (c10::DeviceIndex)dev));
      rc = p_dequant(reinterpret_cast<uint8_t *>(p[0]), reinterpret_cast<uint8_t *>(p[1]), reinterpret_cast<float *>(p[2]),
                     (int)s[0], s[1], (int)s[2], (int)fmt, out.data_ptr(), s[2], stream_of(out));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

// gmm(x, addresses, shape, format, their device, group_sizes, grad enabled) -> bf16 [M, N], with a workspace of its own
PyObject *gmm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7 || !p_gmm) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *x = tensor(a[0]), *g = tensor(a[5]);
    uintptr_t p[3];
    int64_t s[3];
    bool bad = false;
    const int64_t fmt = integer(a[3], bad);
    if (bad || !addresses(a[1], p) || !shape3(a[2], s) || !on_gpu(x, at::kBFloat16) ||
        !beside(g, at::kLong, *x) || !THPDevice_Check(a[4]) || reinterpret_cast<THPDevice *>(a[4])->device != x->device())
      Py_RETURN_NONE;
    const int64_t E = s[0], N = s[1], K = s[2], M = x->dim() == 2 ? x->size(0) : -1;
    if (M < 0 || x->size(1) != K || (x->requires_grad() && a[6] == Py_True) || g->numel() != E || !g->is_contiguous())
      Py_RETURN_NONE;
    const int64_t ld = x->stride(0);
    if (x->stride(1) != 1 || ld < K || ld % 8 || reinterpret_cast<uintptr_t>(x->data_ptr()) % 16) Py_RETURN_NONE;
    const int64_t nb = p_workspace_bytes((int)fmt, M, (int)K, (int)E);
    if (nb < 0) Py_RETURN_NONE;
    at::Tensor out, ws;
    int rc;
    {
      const Unlocked unlocked;
      out = empty({M, N}, at::kBFloat16, x->device());
      ws = empty({nb}, at::kByte, x->device());
      rc = p_gmm(g->data_ptr<int64_t>(), (int)E, (int)fmt, x->data_ptr(), ld, reinterpret_cast<uint8_t *>(p[0]),
                 reinterpret_cast<uint8_t *>(p[1]), reinterpret_cast<float *>(p[2]), out.data_ptr(), M, (int)K, (int)N,
                 ws.data_ptr(), nb, stream_of(*x));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

#define MGEMM_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr}, MGEMM_FAST(route),      MGEMM_FAST(route_bwd),
                         MGEMM_FAST(quantize),            MGEMM_FAST(dequantize), MGEMM_FAST(gmm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Host calls of the decode-size operators.", -1, methods,
                      nullptr,               nullptr,  nullptr,                                    nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
