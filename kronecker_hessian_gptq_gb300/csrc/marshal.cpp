// marshal.cpp -- lists of torch tensors as the array of bakron_adamw_tensor that
// bakron_adamw takes.  A step over 130 small tensors takes the GPU about ten
// microseconds; reading five attributes of 520 tensors from Python takes 250.
//
// Called with the interpreter's lock held (ctypes.PyDLL).  Nothing is raised here:
// 0 when every tensor is what it has to be, else 1, and the caller's own
// checks, in Python, say what is wrong.
#include <torch/csrc/autograd/python_variable.h>

#include "bakron.h"

namespace {

// Dense on the device, of `n` values; -1 for any number.
const at::Tensor* dense(PyObject* o, int device, int64_t n) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous() || (n >= 0 && t.numel() != n)) return nullptr;
  return &t;
}
int float_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return BAKRON_F32;
    case at::kHalf: return BAKRON_F16;
    case at::kBFloat16: return BAKRON_BF16;
    default: return -1;
  }
}

int pack(PyObject* const* lists, Py_ssize_t count, int device, bakron_adamw_tensor* out) {
  enum { kParams, kGrads, kM, kV, kMScales, kVScales, kCopies, kLists };
  for (int l = 0; l < kLists; ++l) {
    if (lists[l] == Py_None) continue;
    if (!PyList_Check(lists[l]) || PyList_GET_SIZE(lists[l]) != count) return 1;
  }
  const bool eight = lists[kMScales] != Py_None;
  const at::ScalarType state = eight ? at::kFloat8_e4m3fn : at::kFloat;
  for (Py_ssize_t i = 0; i < count; ++i) {
    auto item = [&](int l) { return PyList_GET_ITEM(lists[l], i); };
    bakron_adamw_tensor& e = out[i];
    e = {};
    const at::Tensor* p = dense(item(kParams), device, -1);
    if (!p) return 1;
    e.n = p->numel();
    const at::Tensor *g = dense(item(kGrads), device, e.n), *m = dense(item(kM), device, e.n), *v = dense(item(kV), device, e.n);
    if (!g || !m || !v || m->scalar_type() != state || v->scalar_type() != state) return 1;
    e.param_dtype = float_code(*p), e.grad_dtype = float_code(*g);
    if (e.param_dtype < 0 || e.grad_dtype < 0) return 1;
    e.param = p->data_ptr(), e.grad = g->data_ptr(), e.m = m->data_ptr(), e.v = v->data_ptr();
    if (eight) {
      const int64_t groups = (e.n + 255) / 256;
      const at::Tensor *ms = dense(item(kMScales), device, groups), *vs = dense(item(kVScales), device, groups);
      if (!ms || !vs || ms->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat) return 1;
      e.m_scales = static_cast<float*>(ms->data_ptr()), e.v_scales = static_cast<float*>(vs->data_ptr());
    }
    if (lists[kCopies] != Py_None && item(kCopies) != Py_None) {
      const at::Tensor* c = dense(item(kCopies), device, e.n);
      if (!c || float_code(*c) <= BAKRON_F32) return 1;
      e.copy = c->data_ptr(), e.copy_dtype = float_code(*c);
    }
  }
  return 0;
}

}  // namespace

// lists: params, grads, m, v, m_scales, v_scales, copies; the last three may be None.
extern "C" int bakron_py_adamw_tensors(PyObject* params, PyObject* grads, PyObject* m, PyObject* v, PyObject* m_scales,
                                       PyObject* v_scales, PyObject* copies, int64_t count, int device, void* out) {
  PyObject* const lists[] = {params, grads, m, v, m_scales, v_scales, copies};
  try {
    return pack(lists, count, device, static_cast<bakron_adamw_tensor*>(out));
  } catch (...) {
    return 1;
  }
}
