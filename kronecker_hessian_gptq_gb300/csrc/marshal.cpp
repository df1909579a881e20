// marshal.cpp -- the calls of a projection in 8-bit floats from Python without
// Python's price: checks of a dozen tensors, three allocations and a call with
// twenty arguments take 18 us through ctypes, of which the GPU works 3 for one
// token's heads; here 4.5.  The same for the lists of AdamW: reading five
// attributes of 520 tensors takes 250 us from Python, 10 here.
//
// A call that is not handled (an argument that is not what it has to be, no
// tokens, a refusal by the library) returns None, and the checks and the call
// through ctypes, in _projection.py, follow and say what is wrong.  An error of
// the library that may have enqueued something is raised: made again, an AdamW
// step would be two.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <memory>
#include <optional>

#include "bakron.h"

namespace {

// The library's entry points, as the caller has loaded them.
struct Entries {
  decltype(&bakron_fp8_matmul) fp8;
  decltype(&bakron_fp8_matmul_workspace_size) fp8_size;
  decltype(&bakron_fp8_matmul_backward) fp8_back;
  decltype(&bakron_fp8_matmul_backward_workspace_size) fp8_back_size;
  decltype(&bakron_head_norm_rotary) heads;
  decltype(&bakron_head_norm_rotary_backward) heads_back;
  decltype(&bakron_head_norm_rotary_backward_workspace_size) heads_back_size;
  decltype(&bakron_adamw) adamw;
  decltype(&bakron_adamw_workspace_size) adamw_size;
  decltype(&bakron_status_string) text;
} lib;
bool bound = false;

template <class F>
bool find(void* handle, const char* name, F& f) {
  f = reinterpret_cast<F>(dlsym(handle, name));
  return f != nullptr;
}

constexpr int kE4M3 = BAKRON_E4M3;
// 0, 1, 2 for the float types, 4 for e4m3, -1 for others.
int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return BAKRON_F32;
    case at::kHalf: return BAKRON_F16;
    case at::kBFloat16: return BAKRON_BF16;
    case at::kFloat8_e4m3fn: return kE4M3;
    default: return -1;
  }
}
at::ScalarType type_of(int code) { return code == BAKRON_F32 ? at::kFloat : code == BAKRON_F16 ? at::kHalf : at::kBFloat16; }
bool is_float(int code) { return code >= 0 && code <= 2; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
// Dense on the device, of `n` values; -1 for any number.
const at::Tensor* dense(PyObject* o, int device, int64_t n) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->get_device() != device || !t->is_contiguous() || (n >= 0 && t->numel() != n)) return nullptr;
  return t;
}
// A matrix with contiguous rows; its row stride (that of a lone row is its length).
struct Matrix {
  const at::Tensor* t = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  void* p = nullptr;
};
bool matrix(PyObject* o, Matrix& m) {
  m.t = tensor(o);
  if (!m.t || !m.t->is_cuda() || m.t->dim() != 2) return false;
  m.rows = m.t->size(0), m.cols = m.t->size(1);
  if (m.rows < 1 || m.cols < 1 || (m.cols > 1 && m.t->stride(1) != 1)) return false;
  m.ld = m.rows > 1 ? m.t->stride(0) : m.cols;
  m.p = m.t->data_ptr();
  return m.ld >= m.cols;
}
// A dense vector or matrix of n values of a type, or None (null).
bool values(PyObject* o, at::ScalarType type, int64_t dim, int64_t first, int64_t n, int device, const void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = dense(o, device, n);
  if (!t || t->scalar_type() != type || t->dim() != dim || t->size(0) != first) return false;
  *p = t->data_ptr();
  return true;
}
int64_t blocks(int64_t n) { return (n + 127) / 128; }

at::Tensor room(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, device), std::nullopt);
}
void* stream_on(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }
bool ready(int device) { return bound && c10::cuda::current_device() == device; }
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// Whether the present call of this thread has enqueued work, or may have.
thread_local bool enqueued = false;
// A call of the library, with other threads free to run meanwhile: a launch may
// wait for room.  Whether it succeeded; if not, and it was no refusal, with the error set.
template <class F>
bool launched(const char* name, F call) {
  PyThreadState* state = PyEval_SaveThread();
  const int r = call();
  PyEval_RestoreThread(state);
  if (r == BAKRON_ERR_INVALID_ARG || r == BAKRON_ERR_WORKSPACE) return false;
  enqueued = true;
  if (r != BAKRON_OK) PyErr_Format(PyExc_RuntimeError, "%s failed: %s", name, lib.text(r));
  return r == BAKRON_OK;
}
// A tuple or a value of a dict; takes the references.
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}
bool put(PyObject* dict, const char* key, const at::Tensor& t) {
  PyObject* v = wrap(t);
  const bool ok = v && PyDict_SetItemString(dict, key, v) == 0;
  Py_XDECREF(v);
  return ok;
}

// Weights in e4m3 or bytes with a scale for each 128 x 128.
struct Weights {
  Matrix codes;
  const void* scales = nullptr;
  int copies = 0;
};
bool weights(PyObject* codes, PyObject* scales, int64_t K, int device, Weights& w) {
  if (!matrix(codes, w.codes) || w.codes.cols != K || w.codes.t->get_device() != device) return false;
  const at::ScalarType type = w.codes.t->scalar_type();
  if (type != at::kFloat8_e4m3fn && type != at::kChar && type != at::kByte) return false;
  if (scales == Py_None || !values(scales, at::kFloat, 2, blocks(w.codes.rows), blocks(w.codes.rows) * blocks(K), device, &w.scales))
    return false;
  w.copies = reinterpret_cast<uintptr_t>(w.codes.p) % 16 || w.codes.ld % 16;
  return true;
}

// (X, codes, scales, x_scales, bias, type of Y or -1)
PyObject* fp8_matmul(PyObject* const* a) {
  Matrix x;
  Weights w;
  const long want = PyLong_AsLong(a[5]);
  if (!matrix(a[0], x)) return nullptr;
  const int device = x.t->get_device(), kind = code_of(*x.t);
  if (kind < 0 || want > 2 || !ready(device) || !weights(a[1], a[2], x.cols, device, w)) return nullptr;
  const int64_t T = x.rows, K = x.cols, N = w.codes.rows;
  const void *xs, *bias;
  if ((kind == kE4M3) == (a[3] == Py_None) || !values(a[3], at::kFloat, 2, T, T * blocks(K), device, &xs) ||
      !values(a[4], at::kFloat, 1, N, N, device, &bias))
    return nullptr;
  const int out = want >= 0 ? (int)want : kind == kE4M3 ? BAKRON_F32 : kind;
  void* const stream = stream_on(device);
  const at::Tensor y = room({T, N}, type_of(out), device), status = room({1}, at::kInt, device);
  const size_t bytes = lib.fp8_size(T, K, N, kind, w.copies);
  if (!bytes) return nullptr;
  const at::Tensor ws = room({(int64_t)bytes}, at::kByte, device);
  if (!launched("bakron_fp8_matmul", [&] {
        return lib.fp8(x.p, kind, x.ld, static_cast<const float*>(xs), static_cast<const uint8_t*>(w.codes.p), w.codes.ld,
              static_cast<const float*>(w.scales), static_cast<const float*>(bias), T, K, N, y.data_ptr(), out, ws.data_ptr(), bytes,
              static_cast<int32_t*>(status.data_ptr()), stream);
      }))
    return nullptr;
  return pair(wrap(y), wrap(status));
}

// (dY, X, codes, scales, bias)
PyObject* fp8_matmul_backward(PyObject* const* a) {
  Matrix dy, x;
  Weights w;
  if (!matrix(a[0], dy)) return nullptr;
  const int device = dy.t->get_device(), kind = code_of(*dy.t);
  const at::Tensor* codes = tensor(a[2]);
  if (!is_float(kind) || !ready(device) || !codes || codes->dim() != 2) return nullptr;
  const int64_t T = dy.rows, N = dy.cols, K = codes->size(1);
  if (!weights(a[2], a[3], K, device, w) || w.codes.rows != N) return nullptr;
  const int wanted = PyObject_IsTrue(a[4]);
  if (wanted < 0) return nullptr;
  const bool has_x = a[1] != Py_None, has_bias = wanted;
  if (has_x && (!matrix(a[1], x) || x.rows != T || x.cols != K || x.t->get_device() != device || code_of(*x.t) != kind)) return nullptr;
  void* const stream = stream_on(device);
  const at::Tensor dx = room({T, K}, type_of(kind), device), status = room({1}, at::kInt, device);
  at::Tensor dw, dbias;
  if (has_x) dw = room({N, K}, type_of(kind), device);
  if (has_bias) dbias = room({N}, at::kFloat, device);
  const size_t bytes = lib.fp8_back_size(T, K, N, 1 + 2 * has_x + 4 * has_bias, w.copies);
  if (!bytes) return nullptr;
  const at::Tensor ws = room({(int64_t)bytes}, at::kByte, device);
  if (!launched("bakron_fp8_matmul_backward", [&] {
        return lib.fp8_back(dy.p, dy.ld, x.p, x.ld, kind, static_cast<const uint8_t*>(w.codes.p), w.codes.ld,
                   static_cast<const float*>(w.scales), T, K, N, dx.data_ptr(), has_x ? dw.data_ptr() : nullptr,
                   has_bias ? static_cast<float*>(dbias.data_ptr()) : nullptr, ws.data_ptr(), bytes,
                   static_cast<int32_t*>(status.data_ptr()), stream);
      }))
    return nullptr;
  PyObject* d = PyDict_New();
  if (!d || !put(d, "X", dx) || !put(d, "W", dw) || !put(d, "bias", dbias)) {
    Py_XDECREF(d);
    return nullptr;
  }
  return pair(d, wrap(status));
}

// T x heads x D with contiguous values; the strides of a lone token or head do not count.
struct Heads {
  void* p = nullptr;
  int64_t T = 0, heads = 0, D = 0, token = 0, head = 0;
};
bool heads_of(PyObject* o, at::ScalarType type, int device, Heads& h) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->dim() != 3 || t->scalar_type() != type || t->get_device() != device) return false;
  h = {t->data_ptr(), t->size(0), t->size(1), t->size(2), 0, 0};
  if (h.T < 1 || h.heads < 1 || h.D < 1 || (h.D > 1 && t->stride(2) != 1)) return false;
  h.token = h.T > 1 ? t->stride(0) : 0, h.head = h.heads > 1 ? t->stride(1) : 0;
  return true;
}
// What both directions take: (Q, K, positions, freqs, q_weight, k_weight, eps, pairs).
struct Norm {
  Heads q, k;
  const void *qw, *kw, *positions, *freqs;
  int64_t R = 0;
  float eps;
  int pairs, kind, device;
  at::ScalarType type;
};
bool norm_of(PyObject* const* a, Norm& n) {
  const at::Tensor* q = tensor(a[0]);
  if (!q || !q->is_cuda()) return false;
  n.kind = code_of(*q), n.device = q->get_device(), n.type = q->scalar_type();
  if (!is_float(n.kind) || !ready(n.device) || !heads_of(a[0], n.type, n.device, n.q)) return false;
  if (a[1] != Py_None && (!heads_of(a[1], n.type, n.device, n.k) || n.k.T != n.q.T || n.k.D != n.q.D)) return false;
  if (a[1] == Py_None && a[5] != Py_None) return false;
  if ((a[2] == Py_None) != (a[3] == Py_None)) return false;
  if (a[3] != Py_None) {
    const at::Tensor* f = tensor(a[3]);
    if (!f || f->dim() != 1) return false;
    n.R = 2 * f->size(0);
  }
  const int64_t D = n.q.D;
  const double eps = PyFloat_AsDouble(a[6]);
  n.eps = (float)eps, n.pairs = (int)PyLong_AsLong(a[7]);
  return n.R <= D && !PyErr_Occurred() && values(a[2], at::kLong, 1, n.q.T, n.q.T, n.device, &n.positions) &&
         values(a[3], at::kDouble, 1, n.R / 2, n.R / 2, n.device, &n.freqs) && values(a[4], at::kFloat, 1, D, D, n.device, &n.qw) &&
         values(a[5], at::kFloat, 1, D, D, n.device, &n.kw);
}
PyObject* head_norm_rotary(PyObject* const* a) {
  Norm n;
  if (!norm_of(a, n)) return nullptr;
  void* const stream = stream_on(n.device);
  const at::Tensor yq = room({n.q.T, n.q.heads, n.q.D}, n.type, n.device);
  at::Tensor yk;
  if (n.k.p) yk = room({n.k.T, n.k.heads, n.k.D}, n.type, n.device);
  if (!launched("bakron_head_norm_rotary", [&] {
        return lib.heads(n.q.p, n.q.token, n.q.head, n.q.heads, n.k.p, n.k.token, n.k.head, n.k.heads, static_cast<const float*>(n.qw),
                static_cast<const float*>(n.kw), static_cast<const int64_t*>(n.positions), static_cast<const double*>(n.freqs), n.R,
                n.pairs, n.eps, n.kind, n.q.T, n.q.D, yq.data_ptr(), n.k.p ? yk.data_ptr() : nullptr, stream);
      }))
    return nullptr;
  return pair(wrap(yq), wrap(yk));
}
// (dYQ, dYK, then as above)
PyObject* head_norm_rotary_backward(PyObject* const* a) {
  Norm n;
  Heads dq, dk;
  if (!norm_of(a + 2, n) || !heads_of(a[0], n.type, n.device, dq) || dq.T != n.q.T || dq.heads != n.q.heads || dq.D != n.q.D)
    return nullptr;
  if ((a[1] == Py_None) != (n.k.p == nullptr)) return nullptr;
  if (n.k.p && (!heads_of(a[1], n.type, n.device, dk) || dk.T != n.k.T || dk.heads != n.k.heads || dk.D != n.k.D)) return nullptr;
  void* const stream = stream_on(n.device);
  const at::Tensor gq = room({n.q.T, n.q.heads, n.q.D}, n.type, n.device);
  at::Tensor gk, gqw, gkw;
  if (n.k.p) gk = room({n.k.T, n.k.heads, n.k.D}, n.type, n.device);
  if (n.qw) gqw = room({n.q.D}, at::kFloat, n.device);
  if (n.kw) gkw = room({n.q.D}, at::kFloat, n.device);
  const size_t bytes = lib.heads_back_size(n.q.T, n.q.D);
  if (!bytes) return nullptr;
  const at::Tensor ws = room({(int64_t)bytes}, at::kByte, n.device);
  auto at = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  if (!launched("bakron_head_norm_rotary_backward", [&] {
        return lib.heads_back(dq.p, dq.token, dq.head, dk.p, dk.token, dk.head, n.q.p, n.q.token, n.q.head, n.q.heads, n.k.p, n.k.token,
                     n.k.head, n.k.heads, static_cast<const float*>(n.qw), static_cast<const float*>(n.kw),
                     static_cast<const int64_t*>(n.positions), static_cast<const double*>(n.freqs), n.R, n.pairs, n.eps, n.kind, n.q.T,
                     n.q.D, at(gq), at(gk), static_cast<float*>(at(gqw)), static_cast<float*>(at(gkw)), ws.data_ptr(), bytes,
                     stream_on(n.device));
      }))
    return nullptr;
  PyObject* d = PyDict_New();
  if (!d || !put(d, "Q", gq) || !put(d, "K", gk) || !put(d, "q_weight", gqw) || !put(d, "k_weight", gkw)) {
    Py_XDECREF(d);
    return nullptr;
  }
  return d;
}

// A number, or a tensor of one value of the type (then its address).
bool number(PyObject* o, at::ScalarType type, int device, double* value, const void** p) {
  *p = nullptr, *value = 1;
  if (const at::Tensor* t = tensor(o)) {
    if (!t->is_cuda() || t->get_device() != device || t->scalar_type() != type || t->numel() != 1) return false;
    *p = t->data_ptr();
    return true;
  }
  *value = PyFloat_AsDouble(o);
  return !PyErr_Occurred();
}

// Autograd has to know that a tensor changed: a graph that kept it from before would go
// backward with other values.
void changed(PyObject* o) {
  const at::Tensor* t = tensor(o);
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// (params, grads, m, v, m_scales, v_scales, copies, step, lr, beta1, beta2, eps, weight_decay, grad_scale, skip, seed);
// the last three lists and skip may be None.
PyObject* adamw(PyObject* const* a) {
  enum { kParams, kGrads, kM, kV, kMScales, kVScales, kCopies, kLists };
  if (!PyList_Check(a[kParams]) || PyList_GET_SIZE(a[kParams]) < 1) return nullptr;
  const Py_ssize_t count = PyList_GET_SIZE(a[kParams]);
  for (int l = 1; l < kLists; ++l)
    if (a[l] != Py_None && (!PyList_Check(a[l]) || PyList_GET_SIZE(a[l]) != count)) return nullptr;
  const at::Tensor* lead = tensor(PyList_GET_ITEM(a[kParams], 0));
  if (!lead || !lead->is_cuda()) return nullptr;
  const int device = lead->get_device();
  const bool eight = a[kMScales] != Py_None;
  if (!ready(device) || eight != (a[kVScales] != Py_None)) return nullptr;
  // The step as an integer: a double holds fewer.
  PyObject* const* n = a + kLists;
  double rate, scale, none;
  const void *step_dev, *rate_dev, *scale_dev, *skip = nullptr;
  long long step = 1;
  if (tensor(n[0])) {
    if (!number(n[0], at::kLong, device, &none, &step_dev)) return nullptr;
  } else {
    step_dev = nullptr, step = PyLong_AsLongLong(n[0]);
  }
  if (PyErr_Occurred() || step < 1 || !number(n[1], at::kFloat, device, &rate, &rate_dev) ||
      !number(n[6], at::kFloat, device, &scale, &scale_dev) ||
      (n[7] != Py_None && (!tensor(n[7]) || !number(n[7], at::kInt, device, &none, &skip))))
    return nullptr;
  const double b1 = PyFloat_AsDouble(n[2]), b2 = PyFloat_AsDouble(n[3]), eps = PyFloat_AsDouble(n[4]), decay = PyFloat_AsDouble(n[5]);
  const uint64_t seed = PyLong_AsUnsignedLongLongMask(n[8]);
  if (PyErr_Occurred()) return nullptr;
  std::unique_ptr<bakron_adamw_tensor[]> out(new bakron_adamw_tensor[count]);
  const at::ScalarType state = eight ? at::kFloat8_e4m3fn : at::kFloat;
  for (Py_ssize_t i = 0; i < count; ++i) {
    auto item = [&](int l) { return PyList_GET_ITEM(a[l], i); };
    bakron_adamw_tensor& e = out[i];
    e = {};
    const at::Tensor* p = dense(item(kParams), device, -1);
    if (!p) return nullptr;
    e.n = p->numel();
    const at::Tensor *g = dense(item(kGrads), device, e.n), *m = dense(item(kM), device, e.n), *v = dense(item(kV), device, e.n);
    if (!g || !m || !v || m->scalar_type() != state || v->scalar_type() != state) return nullptr;
    e.param_dtype = code_of(*p), e.grad_dtype = code_of(*g);
    if (!is_float(e.param_dtype) || !is_float(e.grad_dtype)) return nullptr;
    e.param = p->data_ptr(), e.grad = g->data_ptr(), e.m = m->data_ptr(), e.v = v->data_ptr();
    if (eight) {
      const int64_t groups = (e.n + 255) / 256;
      const at::Tensor *ms = dense(item(kMScales), device, groups), *vs = dense(item(kVScales), device, groups);
      if (!ms || !vs || ms->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat) return nullptr;
      e.m_scales = static_cast<float*>(ms->data_ptr()), e.v_scales = static_cast<float*>(vs->data_ptr());
    }
    if (a[kCopies] != Py_None && item(kCopies) != Py_None) {
      const at::Tensor* c = dense(item(kCopies), device, e.n);
      if (!c || code_of(*c) < 1 || code_of(*c) > 2) return nullptr;
      e.copy = c->data_ptr(), e.copy_dtype = code_of(*c);
    }
  }
  void* const stream = stream_on(device);
  const at::Tensor status = room({1}, at::kInt, device), ws = room({(int64_t)lib.adamw_size()}, at::kByte, device);
  const bool ok = launched("bakron_adamw", [&] {
        return lib.adamw(out.get(), count, eight ? 8 : 32, rate, static_cast<const float*>(rate_dev), step, static_cast<const int64_t*>(step_dev),
                b1, b2, eps, decay, scale, static_cast<const float*>(scale_dev), static_cast<const int32_t*>(skip), seed, ws.data_ptr(),
                ws.numel(), static_cast<int32_t*>(status.data_ptr()), stream);
      });
  // (Not the states, which no graph holds: they would take 4 us more of 130 tensors' 22.)
  if (enqueued)
    for (int l : {(int)kParams, (int)kCopies})
      for (Py_ssize_t i = 0; a[l] != Py_None && i < count; ++i) changed(PyList_GET_ITEM(a[l], i));
  return ok ? wrap(status) : nullptr;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject* r = nullptr;
  enqueued = false;
  try {
    if (n == kArgs) r = kCall(args);
  } catch (...) {
    r = nullptr;
  }
  if (r) return r;
  if (enqueued) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call was made, but its results cannot be handed out");
    return nullptr;
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// The path of the library that the entry points are taken from.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  bound = h && find(h, "bakron_fp8_matmul", lib.fp8) && find(h, "bakron_fp8_matmul_workspace_size", lib.fp8_size) &&
          find(h, "bakron_fp8_matmul_backward", lib.fp8_back) &&
          find(h, "bakron_fp8_matmul_backward_workspace_size", lib.fp8_back_size) && find(h, "bakron_head_norm_rotary", lib.heads) &&
          find(h, "bakron_head_norm_rotary_backward", lib.heads_back) &&
          find(h, "bakron_head_norm_rotary_backward_workspace_size", lib.heads_back_size) && find(h, "bakron_adamw", lib.adamw) &&
          find(h, "bakron_adamw_workspace_size", lib.adamw_size) && find(h, "bakron_status_string", lib.text);
  return PyBool_FromLong(bound);
}

#define CALL(name, args) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<name, args>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         CALL(fp8_matmul, 6),
                         CALL(fp8_matmul_backward, 5),
                         CALL(head_norm_rotary, 8),
                         CALL(head_norm_rotary_backward, 10),
                         CALL(adamw, 16),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__marshal(void) { return PyModule_Create(&module); }
