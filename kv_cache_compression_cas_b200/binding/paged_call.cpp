// Argument marshalling of the serving calls for Python (vark_qk_norm_rope,
// vark_paged_append, vark_paged_attention): what __init__.py does for them,
// tensor by tensor, in one C++ call.  The smallest of these calls take 4 us on
// the device; checked in Python and passed through ctypes they took 12 to 16
// on the host.  A function returns the library's status, or None where an
// argument is not plainly right: __init__.py then looks at all of them and
// raises, or makes the call itself.  The library's functions come as addresses,
// so this module links against torch only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>

#include "vark.h"

namespace {

decltype(&vark_qk_norm_rope) norm_rope_fn = nullptr;
decltype(&vark_paged_append) append_fn = nullptr;
decltype(&vark_paged_attention) attention_fn = nullptr;

struct Unsure {};   // leave the call to __init__.py

// A tensor argument; null for None.
const at::Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Unsure{};
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(const at::Tensor* t) {
  if (t == nullptr || !t->defined()) throw Unsure{};
  return *t;
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unsure{};
  }
  return v;
}
int small(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) throw Unsure{};
  return int(v);
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Unsure{};
  }
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unsure{};
  }
  return float(v);
}

int dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return VARK_BF16;
  if (t.scalar_type() == at::kHalf) return VARK_FP16;
  throw Unsure{};
}

enum Layout { kContiguous, kReadRows, kWrittenRows };

// An output's rows must not overlap: from the smallest stride on, every axis
// steps over all that the ones before it span.
bool rows_distinct(const at::Tensor& t) {
  const int n = int(t.dim()) - 1;
  int order[8], m = 0;
  if (n > 8) return false;
  for (int i = 0; i < n; ++i) {
    if (t.size(i) <= 1) continue;
    int at = m++;
    for (; at > 0 && t.stride(order[at - 1]) > t.stride(i); --at) order[at] = order[at - 1];
    order[at] = i;
  }
  int64_t span = t.size(n);
  for (int k = 0; k < m; ++k) {
    const int64_t step = t.stride(order[k]);
    if (step < span) return false;
    span += step * (t.size(order[k]) - 1);
  }
  return true;
}

// Pointer of a tensor that has the type, shape, device and layout asked for
// (null for none).
template <typename T>
T* pointer(const at::Tensor* t, at::ScalarType type, int device, std::initializer_list<int64_t> shape,
           Layout layout = kContiguous) {
  if (t == nullptr) return nullptr;
  if (!t->defined() || !t->is_cuda() || t->scalar_type() != type || t->get_device() != device) throw Unsure{};
  if (t->sizes() != at::IntArrayRef(shape)) throw Unsure{};
  if (!t->is_contiguous()) {
    if (layout == kContiguous) throw Unsure{};
    const int n = int(t->dim());
    if (t->stride(n - 1) != 1) throw Unsure{};
    if (layout == kWrittenRows && !rows_distinct(*t)) throw Unsure{};
  }
  return static_cast<T*>(t->data_ptr());
}

int32_t* status_word(const at::Tensor* t, int device) {
  const at::Tensor& s = needed(t);
  if (!s.is_cuda() || s.scalar_type() != at::kInt || s.get_device() != device || s.numel() < 1 || !s.is_contiguous())
    throw Unsure{};
  return static_cast<int32_t*>(s.data_ptr());
}

struct Rope {
  const float* table = nullptr;
  int len = 0, dim = 0;
  const int32_t* positions = nullptr;
  Rope(const at::Tensor* rope, const at::Tensor* pos, int device, std::initializer_list<int64_t> tokens) {
    if ((rope == nullptr) != (pos == nullptr)) throw Unsure{};
    if (rope == nullptr) return;
    if (rope->dim() != 3 || rope->size(1) != 2) throw Unsure{};
    table = pointer<float>(rope, at::kFloat, device, {rope->size(0), 2, rope->size(2)});
    len = small(rope->size(0));
    dim = small(2 * rope->size(2));
    positions = pointer<int32_t>(pos, at::kInt, device, tokens);
  }
};

struct Pool {
  uint16_t *k, *v;
  const int32_t *table, *len, *cu;
  int64_t n_pages;
  int page_size, max_pages, head_pages, B;
  Pool(const at::Tensor& kp, const at::Tensor* vp, const at::Tensor& tab, const at::Tensor* lens,
       const at::Tensor& offsets, at::ScalarType type, int device, int64_t H, int64_t D) {
    head_pages = kp.dim() == 3;
    if (kp.dim() != 3 && kp.dim() != 4) throw Unsure{};
    n_pages = kp.size(0);
    page_size = small(kp.size(kp.dim() - 2));
    B = small(offsets.numel() - 1);
    if (B < 0 || tab.dim() != 2 + head_pages) throw Unsure{};
    max_pages = small(tab.size(tab.dim() - 1));
    cu = pointer<int32_t>(&offsets, at::kInt, device, {B + 1});
    needed(vp);
    needed(lens);
    if (head_pages) {
      k = pointer<uint16_t>(&kp, type, device, {n_pages, page_size, D});
      v = pointer<uint16_t>(vp, type, device, {n_pages, page_size, D});
      table = pointer<int32_t>(&tab, at::kInt, device, {B, H, max_pages});
      len = pointer<int32_t>(lens, at::kInt, device, {B, H});
    } else {
      k = pointer<uint16_t>(&kp, type, device, {n_pages, H, page_size, D});
      v = pointer<uint16_t>(vp, type, device, {n_pages, H, page_size, D});
      table = pointer<int32_t>(&tab, at::kInt, device, {B, max_pages});
      len = pointer<int32_t>(lens, at::kInt, device, {B});
    }
  }
};

// The tensors' device current, and the stream: None for the device's current
// one, or an int handle.
struct Place {
  std::optional<c10::cuda::CUDAGuard> guard;
  void* stream;
  Place(int device, PyObject* s) {
    if (c10::cuda::current_device() != device) guard.emplace(c10::DeviceIndex(device));
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream();
    } else {
      stream = PyLong_AsVoidPtr(s);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Unsure{};
      }
    }
  }
};

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const Unsure&) {
  } catch (const std::exception&) {      // whatever torch throws shows up again in the careful path
  }
  Py_RETURN_NONE;
}

// (q, k, q_out, k_out, norm, q_weight, k_weight, eps, rope, positions, dev_status, pairs, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    if (n != 13) throw Unsure{};
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *qo = tensor(a[2]), *ko = tensor(a[3]);
    const at::Tensor *qw = tensor(a[5]), *kw = tensor(a[6]);
    if ((q == nullptr) != (qo == nullptr) || (k == nullptr) != (ko == nullptr) || (!q && qw) || (!k && kw))
      throw Unsure{};
    const at::Tensor& x = needed(q ? q : k);
    if (!x.is_cuda() || x.dim() != 4 || (k && k->dim() != 4)) throw Unsure{};
    const int dt = dtype_of(x), dev = x.get_device();
    const auto type = x.scalar_type();
    const int64_t B = x.size(0), T = x.size(1), D = x.size(3);
    const int64_t Hq = q ? q->size(2) : 0, Hk = k ? k->size(2) : 0;
    const auto* pq = pointer<uint16_t>(q, type, dev, {B, T, Hq, D}, kReadRows);
    auto* pqo = pointer<uint16_t>(qo, type, dev, {B, T, Hq, D}, kWrittenRows);
    const auto* pk = pointer<uint16_t>(k, type, dev, {B, T, Hk, D}, kReadRows);
    auto* pko = pointer<uint16_t>(ko, type, dev, {B, T, Hk, D}, kWrittenRows);
    const auto* pqw = pointer<float>(qw, at::kFloat, dev, {D});
    const auto* pkw = pointer<float>(kw, at::kFloat, dev, {D});
    const Rope r(tensor(a[8]), tensor(a[9]), dev, {B, T});
    int32_t* st = status_word(tensor(a[10]), dev);
    const int norm = small(integer(a[4])), pairs = truth(a[11]);
    const float eps = real(a[7]);
    const Place at(dev, a[12]);
    return norm_rope_fn(dt, pq, q ? q->strides().data() : nullptr, pqo, q ? qo->strides().data() : nullptr, small(Hq),
                        pk, k ? k->strides().data() : nullptr, pko, k ? ko->strides().data() : nullptr, small(Hk),
                        small(B), small(T), small(D), norm, pqw, pkw, eps, r.table, r.len, r.dim, pairs, r.positions,
                        st, at.stream);
  });
}

// (k, v, cu_tokens, k_pages, v_pages, page_table, cache_len, norm, k_weight, eps, rope, positions, dev_status, pairs,
//  stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    if (n != 15) throw Unsure{};
    const at::Tensor& k = needed(tensor(a[0]));
    const at::Tensor* v = tensor(a[1]);
    needed(v);
    if (!k.is_cuda() || k.dim() != 3) throw Unsure{};
    const int dt = dtype_of(k), dev = k.get_device();
    const auto type = k.scalar_type();
    const int64_t N = k.size(0), H = k.size(1), D = k.size(2);
    const auto* pk = pointer<uint16_t>(&k, type, dev, {N, H, D}, kReadRows);
    const auto* pv = pointer<uint16_t>(v, type, dev, {N, H, D}, kReadRows);
    const Pool p(needed(tensor(a[3])), tensor(a[4]), needed(tensor(a[5])), tensor(a[6]), needed(tensor(a[2])), type,
                 dev, H, D);
    const auto* pw = pointer<float>(tensor(a[8]), at::kFloat, dev, {D});
    const Rope r(tensor(a[10]), tensor(a[11]), dev, {N});
    int32_t* st = status_word(tensor(a[12]), dev);
    const int norm = small(integer(a[7])), pairs = truth(a[13]);
    const float eps = real(a[9]);
    const Place at(dev, a[14]);
    return append_fn(dt, pk, k.strides().data(), pv, v->strides().data(), N, p.B, small(H), small(D), p.cu, p.k, p.v,
                     p.n_pages, p.page_size, p.table, p.max_pages, p.len, p.head_pages, norm, pw, eps, r.table, r.len,
                     r.dim, pairs, r.positions, st, at.stream);
  });
}

// (q, cu_tokens, k_pages, v_pages, page_table, cache_len, tau, causal, out, lse, workspace, dev_status, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    if (n != 13) throw Unsure{};
    const at::Tensor& q = needed(tensor(a[0]));
    const at::Tensor *out = tensor(a[8]), *ws = tensor(a[10]);
    needed(out);
    needed(ws);
    if (!q.is_cuda() || q.dim() != 3) throw Unsure{};
    const int dt = dtype_of(q), dev = q.get_device();
    const auto type = q.scalar_type();
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2);
    const at::Tensor &kp = needed(tensor(a[2])), &tab = needed(tensor(a[4]));
    if (kp.dim() < 3 || tab.dim() < 2) throw Unsure{};
    const int64_t H = kp.dim() == 3 ? tab.size(1) : kp.size(1);
    if (H < 1 || Hq % H != 0) throw Unsure{};
    const auto* pq = pointer<uint16_t>(&q, type, dev, {N, Hq, D}, kReadRows);
    auto* po = pointer<uint16_t>(out, type, dev, {N, Hq, D}, kWrittenRows);
    if (po == pq && po != nullptr) throw Unsure{};
    const Pool p(kp, tensor(a[3]), tab, tensor(a[5]), needed(tensor(a[1])), type, dev, H, D);
    const auto* pt = pointer<float>(tensor(a[6]), at::kFloat, dev, {Hq});
    auto* pl = pointer<float>(tensor(a[9]), at::kFloat, dev, {N, Hq});
    if (!ws->is_cuda() || ws->scalar_type() != at::kByte || ws->get_device() != dev || !ws->is_contiguous())
      throw Unsure{};
    int32_t* st = status_word(tensor(a[11]), dev);
    const int causal = truth(a[7]);
    const Place at(dev, a[12]);
    return attention_fn(dt, pq, q.strides().data(), N, p.B, small(Hq), small(H), small(D), p.cu, p.k, p.v, p.n_pages,
                        p.page_size, p.table, p.max_pages, p.len, p.head_pages, pt, causal, po, out->strides().data(),
                        pl, ws->data_ptr(), ws->numel(), st, at.stream);
  });
}

// (addresses of vark_qk_norm_rope, vark_paged_append, vark_paged_attention)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[3];
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "three addresses");
    return nullptr;
  }
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  norm_rope_fn = reinterpret_cast<decltype(norm_rope_fn)>(p[0]);
  append_fn = reinterpret_cast<decltype(append_fn)>(p[1]);
  attention_fn = reinterpret_cast<decltype(attention_fn)>(p[2]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call() { return PyModule_Create(&module); }
