// The host side of the operators whose calls take longer than their kernels at
// decode sizes: arguments read, outputs allocated and the C entry called without
// a Python frame per step.  One token's routing takes 4.9 us a call this way,
// against 15.9 through ctypes and torch.empty (its kernel 3.5).
//
// A function takes what its Python caller (moe.py, fp4.py, norm.py, int4.py) was given and
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
#include <c10/cuda/CUDAGuard.h>
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
decltype(&mgemm_rms_norm) p_norm = nullptr;
decltype(&mgemm_rms_norm_bwd_workspace_bytes) p_norm_workspace = nullptr;
decltype(&mgemm_rms_norm_bwd) p_norm_bwd = nullptr;
decltype(&mgemm_dequant_fp8) p_dequant8 = nullptr;
decltype(&mgemm_balance_workspace_bytes) p_balance_workspace = nullptr;
decltype(&mgemm_balance) p_balance = nullptr;
decltype(&mgemm_balance_bwd) p_balance_bwd = nullptr;
decltype(&mgemm_gmm_int4) p_gmm_int4 = nullptr;
constexpr int kAddresses = 15;

// The tensor of an argument; nullptr for anything else (None among it).
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
bool on_gpu(const at::Tensor *t, at::ScalarType type) { return t && t->is_cuda() && t->scalar_type() == type; }
// the same on the device of another tensor
bool beside(const at::Tensor *t, at::ScalarType type, const at::Tensor &other) {
  return on_gpu(t, type) && t->get_device() == other.get_device();
}

// Whether a call on the tensor is to be differentiated: it requires a gradient and gradients are on, or comes with a
// tangent (forward mode).  The caller records or refuses such a call.
bool differentiated(const at::Tensor *t, bool grads) {
  return t && ((grads && t->requires_grad()) || t->_fw_grad(0).defined());
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
  void *p[kAddresses];
  if (!PyTuple_Check(arg) || PyTuple_GET_SIZE(arg) != kAddresses) {
    PyErr_Format(PyExc_TypeError, "bind takes a tuple of %d addresses", kAddresses);
    return nullptr;
  }
  for (int i = 0; i < kAddresses; ++i) {
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
  p_norm = reinterpret_cast<decltype(p_norm)>(p[7]);
  p_norm_workspace = reinterpret_cast<decltype(p_norm_workspace)>(p[8]);
  p_norm_bwd = reinterpret_cast<decltype(p_norm_bwd)>(p[9]);
  p_dequant8 = reinterpret_cast<decltype(p_dequant8)>(p[10]);
  p_balance_workspace = reinterpret_cast<decltype(p_balance_workspace)>(p[11]);
  p_balance = reinterpret_cast<decltype(p_balance)>(p[12]);
  p_balance_bwd = reinterpret_cast<decltype(p_balance_bwd)>(p[13]);
  p_gmm_int4 = reinterpret_cast<decltype(p_gmm_int4)>(p[14]);
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
    if (type >= 0 && differentiated(l, c10::GradMode::is_enabled())) Py_RETURN_NONE;
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
    if (M < 0 || x->size(1) != K || differentiated(x, a[6] == Py_True) || g->numel() != E || !g->is_contiguous())
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

// The type code of a tensor on the GPU: bf16 or float32, else -1.
int real_type(const at::Tensor *t) {
  if (!t || !t->is_cuda()) return -1;
  return t->scalar_type() == at::kBFloat16 ? MGEMM_BF16 : t->scalar_type() == at::kFloat ? MGEMM_F32 : -1;
}
// Rows [T, C] with unit columns, each its own; `whole`: on 16-byte boundaries.
bool rows_of(const at::Tensor &t, int64_t T, int64_t C, bool whole) {
  return t.dim() == 2 && t.size(0) == T && t.size(1) == C && t.stride(1) == 1 && t.stride(0) >= C &&
         (!whole || (t.stride(0) * t.element_size() % 16 == 0 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0));
}
PyObject *wrap(at::Tensor t) {
  if (t.defined()) return THPVariable_Wrap(std::move(t));
  Py_RETURN_NONE;
}

// norm(x, weight, eps, residual or None, format, out wanted, grad enabled) -> (out, h, codes, scales), None for what is not wanted
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7 || !p_norm) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *r = tensor(a[3]);
    const int xt = real_type(x), wt = real_type(w), rt = real_type(r);
    bool bad = false;
    const int64_t fmt = integer(a[4], bad);
    const double eps = PyFloat_Check(a[2]) ? PyFloat_AS_DOUBLE(a[2]) : (bad = true, 0.0);
    const bool wanted = a[5] == Py_True, grads = a[6] == Py_True;
    if (bad || xt < 0 || wt < 0 || x->dim() != 2 || w->dim() != 1 || w->get_device() != x->get_device()) Py_RETURN_NONE;
    const int64_t T = x->size(0), C = x->size(1);
    const bool codes = fmt != MGEMM_BF16;
    if (!small(T) || !small(C) || !rows_of(*x, T, C, codes) || w->numel() != C || !w->is_contiguous()) Py_RETURN_NONE;
    if (codes && (C % 32 || reinterpret_cast<uintptr_t>(w->data_ptr()) % 16)) Py_RETURN_NONE;
    if (a[3] != Py_None && (rt < 0 || r->get_device() != x->get_device() || !rows_of(*r, T, C, codes))) Py_RETURN_NONE;
    if (differentiated(x, grads) || differentiated(w, grads) || differentiated(r, grads)) Py_RETURN_NONE;
    at::Tensor out, h, q, sc;
    int rc;
    {
      const Unlocked unlocked;
      const c10::cuda::CUDAGuard device(x->device());
      if (wanted) out = empty({T, C}, at::kBFloat16, x->device());
      if (r) h = empty({T, C}, r->scalar_type(), x->device());
      const int64_t ld_sf = fmt == MGEMM_MXFP8 ? (C / 32 + 15) / 16 * 16 : 0;
      if (codes) {
        q = empty({T, C}, at::kByte, x->device());
        sc = ld_sf ? empty({T, ld_sf}, at::kByte, x->device()) : empty({T}, at::kFloat, x->device());
      }
      rc = p_norm(x->data_ptr(), xt, x->stride(0), r ? r->data_ptr() : nullptr, r ? rt : 0, r ? r->stride(0) : C, w->data_ptr(),
                  wt, T, (int)C, (float)eps, r ? h.data_ptr() : nullptr, wanted ? out.data_ptr() : nullptr, (int)fmt,
                  codes ? q.data_ptr<uint8_t>() : nullptr, codes ? sc.data_ptr() : nullptr, ld_sf, stream_of(*x));
    }
    if (rc) return code(rc);
    return Py_BuildValue("(NNNN)", wrap(std::move(out)), wrap(std::move(h)), wrap(std::move(q)), wrap(std::move(sc)));
  });
}

// norm_bwd(grad_out, h, weight, eps, grad_h or None, grad_x wanted, grad_weight wanted) -> (grad_stream, grad_x, grad_weight)
PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7 || !p_norm_bwd) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *g = tensor(a[0]), *h = tensor(a[1]), *w = tensor(a[2]), *gh = tensor(a[4]);
    const int ht = real_type(h), wt = real_type(w);
    bool bad = false;
    const double eps = PyFloat_Check(a[3]) ? PyFloat_AS_DOUBLE(a[3]) : (bad = true, 0.0);
    if (bad || ht < 0 || wt < 0 || h->dim() != 2 || !beside(g, at::kBFloat16, *h) || w->get_device() != h->get_device())
      Py_RETURN_NONE;
    const int64_t T = h->size(0), C = h->size(1);
    if (!small(T) || !small(C) || !rows_of(*h, T, C, false) || !rows_of(*g, T, C, false) || w->dim() != 1 || w->numel() != C ||
        !w->is_contiguous())
      Py_RETURN_NONE;
    if (a[4] != Py_None && !(beside(gh, h->scalar_type(), *h) && rows_of(*gh, T, C, false))) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard device(h->device());  // (whose SMs the workspace goes by)
    const int64_t nb = p_norm_workspace(T, (int)C);
    if (nb < 0) Py_RETURN_NONE;
    at::Tensor gs, gx, gw, ws;
    int rc;
    {
      const Unlocked unlocked;
      gs = empty({T, C}, h->scalar_type(), h->device());
      if (a[5] == Py_True) gx = empty({T, C}, at::kBFloat16, h->device());
      if (a[6] == Py_True) {
        gw = empty({C}, w->scalar_type(), h->device());
        ws = empty({nb}, at::kByte, h->device());
      }
      rc = p_norm_bwd(g->data_ptr(), g->stride(0), h->data_ptr(), ht, h->stride(0), w->data_ptr(), wt,
                      gh ? gh->data_ptr() : nullptr, gh ? gh->stride(0) : C, T, (int)C, (float)eps, gs.data_ptr(),
                      gx.defined() ? gx.data_ptr() : nullptr, gw.defined() ? gw.data_ptr() : nullptr,
                      ws.defined() ? ws.data_ptr() : nullptr, nb, stream_of(*h));
    }
    if (rc) return code(rc);
    return Py_BuildValue("(NNN)", wrap(std::move(gs)), wrap(std::move(gx)), wrap(std::move(gw)));
  });
}

// dequantize8(codes, scales, format) -> bf16 [T, C]
PyObject *dequantize8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 3 || !p_dequant8) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *q = tensor(a[0]), *sc = tensor(a[1]);
    bool bad = false;
    const int64_t fmt = integer(a[2], bad);
    const bool mx = fmt == MGEMM_MXFP8;
    if (bad || !on_gpu(q, at::kByte) || !beside(sc, mx ? at::kByte : at::kFloat, *q)) Py_RETURN_NONE;
    if (q->dim() != 2 || !small(q->size(1)) || !q->is_contiguous() || sc->dim() < 1 || sc->size(0) != q->size(0) ||
        !sc->is_contiguous())
      Py_RETURN_NONE;
    at::Tensor out;
    int rc;
    {
      const Unlocked unlocked;
      const c10::cuda::CUDAGuard device(q->device());
      out = empty(q->sizes(), at::kBFloat16, q->device());
      rc = p_dequant8(q->data_ptr<uint8_t>(), sc->data_ptr(), (int)fmt, q->size(0), (int)q->size(1), mx ? sc->size(1) : 0,
                      out.data_ptr(), stream_of(*q));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

// The sequences' offsets (None: nullptr) and the rows' mask (None: nullptr) of T tokens beside the logits.
bool sequences(PyObject *oo, PyObject *om, const at::Tensor &l, const int64_t *&offsets, int64_t &S, const uint8_t *&mask) {
  const at::Tensor *o = tensor(oo), *m = tensor(om);
  offsets = nullptr, mask = nullptr, S = 1;
  if (oo != Py_None) {
    if (!beside(o, at::kLong, l) || o->dim() != 1 || o->numel() < 2 || !o->is_contiguous()) return false;
    offsets = o->data_ptr<int64_t>(), S = o->numel() - 1;
  }
  if (om != Py_None) {
    if (!(beside(m, at::kBool, l) || beside(m, at::kByte, l)) || m->dim() != 1 || m->numel() != l.size(0) || !m->is_contiguous())
      return false;
    mask = static_cast<const uint8_t *>(m->data_ptr());
  }
  return true;
}

// balance(logits, ids, scoring, scale, offsets or None, mask or None, slopes wanted, grad enabled) -> (loss, counts, slopes or None)
PyObject *balance(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 8 || !p_balance) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *l = tensor(a[0]), *ids = tensor(a[1]);
    const int type = logits_type(l);
    if (type < 0 || differentiated(l, a[7] == Py_True) || !beside(ids, at::kInt, *l) || ids->dim() != 2 ||
        ids->size(0) != l->size(0) || !ids->is_contiguous())
      Py_RETURN_NONE;
    bool bad = false;
    const int64_t scoring = integer(a[2], bad), T = l->size(0), E = l->size(1), k = ids->size(1);
    const double scale = PyFloat_Check(a[3]) ? PyFloat_AS_DOUBLE(a[3]) : (bad = true, 0.0);
    const int64_t *offsets;
    const uint8_t *mask;
    int64_t S;
    if (bad || !small(scoring) || !small(E) || !small(k) || !sequences(a[4], a[5], *l, offsets, S, mask)) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard device(l->device());  // (whose SMs the workspace goes by)
    const int64_t nb = p_balance_workspace(T, (int)E, S);
    if (nb < 0) Py_RETURN_NONE;
    at::Tensor loss, counts, slopes, ws;
    int rc;
    {
      const Unlocked unlocked;
      loss = empty({}, at::kFloat, l->device());
      counts = offsets ? empty({S, E}, at::kLong, l->device()) : empty({E}, at::kLong, l->device());
      if (a[6] == Py_True) slopes = empty({S * E + 1}, at::kFloat, l->device());
      ws = empty({nb}, at::kByte, l->device());
      rc = p_balance(l->data_ptr(), type, l->stride(0), ids->data_ptr<int32_t>(), (int)k, offsets, S, mask, T, (int)E,
                     (int)scoring, (float)scale, loss.data_ptr<float>(), counts.data_ptr<int64_t>(),
                     slopes.defined() ? slopes.data_ptr<float>() : nullptr, ws.data_ptr(), nb, stream_of(*l));
    }
    if (rc) return code(rc);
    return Py_BuildValue("(NNN)", wrap(std::move(loss)), wrap(std::move(counts)), wrap(std::move(slopes)));
  });
}

// balance_bwd(grad_loss, logits, slopes, scoring, offsets or None, mask or None) -> grad_logits
PyObject *balance_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 6 || !p_balance_bwd) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *g = tensor(a[0]), *l = tensor(a[1]), *sl = tensor(a[2]);
    const int type = logits_type(l);
    if (type < 0 || !beside(g, at::kFloat, *l) || g->numel() != 1 || !beside(sl, at::kFloat, *l) || !sl->is_contiguous())
      Py_RETURN_NONE;
    bool bad = false;
    const int64_t scoring = integer(a[3], bad), T = l->size(0), E = l->size(1);
    const int64_t *offsets;
    const uint8_t *mask;
    int64_t S;
    if (bad || !small(scoring) || !small(E) || !sequences(a[4], a[5], *l, offsets, S, mask) || sl->numel() != S * E + 1)
      Py_RETURN_NONE;
    at::Tensor out;
    int rc;
    {
      const Unlocked unlocked;
      const c10::cuda::CUDAGuard device(l->device());
      out = empty({T, E}, l->scalar_type(), l->device());
      rc = p_balance_bwd(g->data_ptr<float>(), l->data_ptr(), type, l->stride(0), sl->data_ptr<float>(), offsets, S, mask, T,
                         (int)E, (int)scoring, out.data_ptr(), E, stream_of(*l));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

// gmm_int4(x, codes, scales, zeros or None, group, group_sizes, grad enabled) -> bf16 [M, N]
PyObject *gmm_int4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7 || !p_gmm_int4) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *sc = tensor(a[2]), *z = tensor(a[3]), *g = tensor(a[5]);
    bool bad = false;
    const int64_t group = integer(a[4], bad);
    if (bad || !small(group) || group < 1 || !on_gpu(x, at::kBFloat16) || !beside(w, at::kByte, *x) ||
        !beside(sc, at::kBFloat16, *x) || !beside(g, at::kLong, *x) || (a[3] != Py_None && !beside(z, at::kByte, *x)))
      Py_RETURN_NONE;
    if (x->dim() != 2 || w->dim() != 3 || !small(w->size(0)) || !small(w->size(1)) || !small(2 * w->size(2))) Py_RETURN_NONE;
    const int64_t E = w->size(0), N = w->size(1), K = 2 * w->size(2), M = x->size(0), scales = E * N * (K / group);
    if (!w->is_contiguous() || sc->numel() != scales || !sc->is_contiguous() ||
        (z && (z->numel() != scales || !z->is_contiguous())))
      Py_RETURN_NONE;
    if (!rows_of(*x, M, K, true) || differentiated(x, a[6] == Py_True) || differentiated(sc, a[6] == Py_True) ||
        g->dim() != 1 || g->numel() != E || !g->is_contiguous())
      Py_RETURN_NONE;
    at::Tensor out;
    int rc;
    {
      const Unlocked unlocked;
      const c10::cuda::CUDAGuard device(x->device());
      out = empty({M, N}, at::kBFloat16, x->device());
      rc = p_gmm_int4(g->data_ptr<int64_t>(), (int)E, x->data_ptr(), x->stride(0), w->data_ptr<uint8_t>(), sc->data_ptr(),
                      z ? z->data_ptr<uint8_t>() : nullptr, (int)group, out.data_ptr(), M, (int)K, (int)N, nullptr,
                      stream_of(*x));
    }
    return rc ? code(rc) : THPVariable_Wrap(std::move(out));
  });
}

#define MGEMM_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr}, MGEMM_FAST(route),      MGEMM_FAST(route_bwd),
                         MGEMM_FAST(quantize),            MGEMM_FAST(dequantize), MGEMM_FAST(gmm),
                         MGEMM_FAST(norm),                MGEMM_FAST(norm_bwd),   MGEMM_FAST(dequantize8),
                         MGEMM_FAST(balance),             MGEMM_FAST(balance_bwd), MGEMM_FAST(gmm_int4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Host calls of the decode-size operators.", -1, methods,
                      nullptr,               nullptr,  nullptr,                                    nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
