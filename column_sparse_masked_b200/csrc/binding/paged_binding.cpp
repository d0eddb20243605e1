// Marshalling of the paged-cache calls from torch tensors to the C ABI
// (include/flashmask.h).  A decode step makes these calls once per layer with a
// few microseconds of work on the device each; through ctypes the checks and
// conversions took 30 to 40 us a call, here about 2 us (the launches come to it).
//
// Every function takes its arguments positionally in the order of the Python
// wrappers and returns the result, an int (the C ABI's error code), or
// NotImplemented for arguments that it does not accept: the wrapper then finds
// out why and raises.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../../include/flashmask.h"

namespace {

decltype(&flashmask_paged_append) f_append = nullptr;
decltype(&flashmask_paged_attention) f_attention = nullptr;
decltype(&flashmask_paged_attention_workspace_size) f_workspace = nullptr;
decltype(&flashmask_paged_gather) f_gather = nullptr;

using T = const at::Tensor*;

// The tensor behind an argument; none = nullptr for None.  False for anything else.
bool tensor(PyObject* o, T* t) {
  if (o == Py_None) {
    *t = nullptr;
    return true;
  }
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}

bool is(T t, at::ScalarType type, at::Device dev, std::initializer_list<int64_t> sizes) {
  return t && t->scalar_type() == type && t->device() == dev && t->is_contiguous() &&
         t->sizes() == at::IntArrayRef(sizes.begin(), sizes.size());
}
bool is_or_none(T t, at::ScalarType type, at::Device dev, std::initializer_list<int64_t> sizes) {
  return !t || is(t, type, dev, sizes);
}
void* ptr(T t) { return t ? t->data_ptr() : nullptr; }

// Rows [B, N, heads, d] bf16 of any strides that keep 16-byte loads aligned.
bool rows(T t, at::Device dev, int64_t B, int64_t N, int64_t d, int64_t* strides) {
  if (!t || t->dim() != 4 || t->scalar_type() != at::kBFloat16 || t->device() != dev) return false;
  const auto s = t->sizes(), st = t->strides();
  if (s[0] != B || s[1] != N || s[3] != d || st[3] != 1) return false;
  for (int i = 0; i < 3; ++i) {
    strides[i] = s[i] > 1 ? st[i] : 0;
    if (strides[i] & 7) return false;
  }
  return (reinterpret_cast<uintptr_t>(t->data_ptr()) & 15) == 0;
}

// Fits the C ABI's int32 sizes.
bool small(int64_t x) { return x >= 0 && x <= INT32_MAX; }

bool pages(T k, T v, T ks, T vs, T table, flashmask_pages* p) {
  if (!k || !v || !table || k->dim() != 4 || !k->is_cuda() || table->dim() != 2) return false;
  const auto s = k->sizes();
  const at::Device dev = k->device();
  const bool four = k->scalar_type() == at::kByte;
  if (!is(k, four ? at::kByte : at::kBFloat16, dev, {s[0], s[1], s[2], s[3]})) return false;
  if (!is(v, k->scalar_type(), dev, {s[0], s[1], s[2], s[3]})) return false;
  if (four ? !is(ks, at::kBFloat16, dev, {s[0], s[1], s[2], 2}) || !is(vs, at::kBFloat16, dev, {s[0], s[1], s[2], 2})
           : ks || vs)
    return false;
  if (table->scalar_type() != at::kInt || table->device() != dev || (table->size(1) > 1 && table->stride(1) != 1))
    return false;
  for (int64_t x : {s[0], s[1], s[2], 2 * s[3], table->size(0), table->size(1)})
    if (!small(x)) return false;
  if (s[1] == 0) return false;
  p->k = k->data_ptr();
  p->v = v->data_ptr();
  p->k_scales = ptr(ks);
  p->v_scales = ptr(vs);
  p->table = static_cast<const int32_t*>(table->data_ptr());
  p->table_stride = table->size(0) > 1 ? table->stride(0) : 0;
  p->B = (int32_t)table->size(0);
  p->table_width = (int32_t)table->size(1);
  p->num_pages = (int32_t)s[0];
  p->page_size = (int32_t)s[2];
  p->Hkv = (int32_t)s[1];
  p->d = (int32_t)(four ? 2 * s[3] : s[3]);
  p->bits = four ? 4 : 16;
  return true;
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

PyObject* refuse() { Py_RETURN_NOTIMPLEMENTED; }

// (a, b): the given tensors where the caller passed them, else the new ones.
PyObject* pair(const at::Tensor& a, PyObject* given_a, const at::Tensor& b, PyObject* given_b) {
  PyObject* x = a.defined() ? THPVariable_Wrap(a) : Py_NewRef(given_a);
  PyObject* y = b.defined() ? THPVariable_Wrap(b) : Py_NewRef(given_b);
  PyObject* t = PyTuple_New(2);
  if (!x || !y || !t) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(t);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}

// The C ABI launches on the current device: the tensors' one while a call runs.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  explicit On(at::Device dev) {
    if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
  }
};

// k, v, k_pages, v_pages, block_table, start, counts, q, cos, sin, positions, interleaved, k_scales, v_scales, q_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  T k, v, kp, vp, table, start, counts, q, cos, sin, positions, ks, vs, q_out;
  if (n != 15 || !tensor(a[0], &k) || !tensor(a[1], &v) || !tensor(a[2], &kp) || !tensor(a[3], &vp) ||
      !tensor(a[4], &table) || !tensor(a[5], &start) || !tensor(a[6], &counts) || !tensor(a[7], &q) ||
      !tensor(a[8], &cos) || !tensor(a[9], &sin) || !tensor(a[10], &positions) || !tensor(a[12], &ks) ||
      !tensor(a[13], &vs) || !tensor(a[14], &q_out))
    return refuse();
  flashmask_pages pg{};
  if (!pages(kp, vp, ks, vs, table, &pg)) return refuse();
  const at::Device dev = kp->device();
  const int64_t B = pg.B, d = pg.d;
  flashmask_append t{};
  if (!k || k->dim() != 4) return refuse();
  const int64_t N = k->size(1);
  if (!small(N) || !rows(k, dev, B, N, d, t.k_strides) || !rows(v, dev, B, N, d, t.v_strides)) return refuse();
  if (k->size(2) != pg.Hkv || v->size(2) != pg.Hkv) return refuse();
  if (!is(start, at::kInt, dev, {B}) || !is_or_none(counts, at::kInt, dev, {B})) return refuse();
  if ((cos == nullptr) != (sin == nullptr) || (!cos && positions)) return refuse();
  if (cos) {
    if (cos->dim() != 2 || !is(cos, at::kFloat, dev, {cos->size(0), cos->size(1)}) ||
        !is(sin, at::kFloat, dev, {cos->size(0), cos->size(1)}) || !small(cos->size(0)) || !small(2 * cos->size(1)))
      return refuse();
    t.table_len = (int32_t)cos->size(0);
    t.rot = (int32_t)(2 * cos->size(1));
  }
  if (!is_or_none(positions, at::kInt, dev, {B, N})) return refuse();
  at::Tensor out;
  if (q) {
    if (!rows(q, dev, B, N, d, t.q_strides) || !small(q->size(2))) return refuse();
    if (!is_or_none(q_out, at::kBFloat16, dev, {B, N, q->size(2), d})) return refuse();
    t.Hq = (int32_t)q->size(2);
  } else if (q_out) {
    return refuse();
  }
  const int inter = PyObject_IsTrue(a[11]);
  if (inter < 0) return nullptr;
  On on(dev);
  if (q) out = q_out ? *q_out : at::empty({B, N, q->size(2), d}, q->options());
  t.q = ptr(q);
  t.k = k->data_ptr();
  t.v = v->data_ptr();
  t.q_out = q ? out.data_ptr() : nullptr;
  t.start = static_cast<const int32_t*>(start->data_ptr());
  t.counts = static_cast<const int32_t*>(ptr(counts));
  t.positions = static_cast<const int32_t*>(ptr(positions));
  t.cos = static_cast<const float*>(ptr(cos));
  t.sin = static_cast<const float*>(ptr(sin));
  t.N = (int32_t)N;
  t.interleaved = inter;
  const int rc = f_append(&pg, &t, stream_of(dev));
  if (rc != 0) return PyLong_FromLong(rc);
  if (!q) Py_RETURN_NONE;
  if (q_out) return Py_NewRef(a[14]);
  return THPVariable_Wrap(out);
}

// q, k_pages, v_pages, block_table, lens, lts, lte, uts, ute, scale, start, causal, k_scales, v_scales, o, lse, workspace
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  T q, kp, vp, table, lens, m[4], start, ks, vs, o, lse, ws;
  if (n != 17 || !tensor(a[0], &q) || !tensor(a[1], &kp) || !tensor(a[2], &vp) || !tensor(a[3], &table) ||
      !tensor(a[4], &lens) || !tensor(a[5], &m[0]) || !tensor(a[6], &m[1]) || !tensor(a[7], &m[2]) ||
      !tensor(a[8], &m[3]) || !tensor(a[10], &start) || !tensor(a[12], &ks) || !tensor(a[13], &vs) ||
      !tensor(a[14], &o) || !tensor(a[15], &lse) || !tensor(a[16], &ws))
    return refuse();
  flashmask_pages pg{};
  if (!q || q->dim() != 4 || !pages(kp, vp, ks, vs, table, &pg)) return refuse();
  const at::Device dev = kp->device();
  const int64_t B = pg.B, Nq = q->size(1), Hq = q->size(2), d = pg.d;
  flashmask_paged_rows r{};
  if (!small(Nq) || !small(Hq) || !rows(q, dev, B, Nq, d, r.q_strides) || Hq % pg.Hkv != 0) return refuse();
  if (!is(lens, at::kInt, dev, {B}) || !is_or_none(start, at::kInt, dev, {B})) return refuse();
  T ref = nullptr;
  for (int i = 3; i >= 0; --i)
    if (m[i]) ref = m[i];
  r.Hm = 1;
  if (ref) {
    if (ref->dim() != 3 || (!m[0]) != (!m[1]) || (!m[2]) != (!m[3])) return refuse();
    const int64_t Hm = ref->size(1), Nm = ref->size(2);
    if ((Hm != 1 && Hm != Hq) || !small(Nm)) return refuse();
    for (T x : m)
      if (!is_or_none(x, at::kInt, dev, {B, Hm, Nm})) return refuse();
    r.Hm = (int32_t)Hm;
    r.Nm = (int32_t)Nm;
  }
  if ((o == nullptr) != (lse == nullptr) || !is_or_none(o, at::kBFloat16, dev, {B, Nq, Hq, d}) ||
      !is_or_none(lse, at::kFloat, dev, {B, Hq, Nq}))
    return refuse();
  if (ws && (ws->device() != dev || !ws->is_contiguous())) return refuse();
  r.scale = 0.f;
  if (a[9] != Py_None) {
    r.scale = (float)PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) return nullptr;
  }
  r.causal = PyObject_IsTrue(a[11]);
  if (r.causal < 0) return nullptr;
  On on(dev);
  at::Tensor new_o, new_lse, new_ws;
  if (!o) {
    new_o = at::empty({B, Nq, Hq, d}, q->options());
    new_lse = at::empty({B, Hq, Nq}, q->options().dtype(at::kFloat));
    o = &new_o;
    lse = &new_lse;
  }
  r.q = q->data_ptr();
  r.lens = static_cast<const int32_t*>(lens->data_ptr());
  r.start = static_cast<const int32_t*>(ptr(start));
  r.lts = static_cast<const int32_t*>(ptr(m[0]));
  r.lte = static_cast<const int32_t*>(ptr(m[1]));
  r.uts = static_cast<const int32_t*>(ptr(m[2]));
  r.ute = static_cast<const int32_t*>(ptr(m[3]));
  r.Nq = (int32_t)Nq;
  r.Hq = (int32_t)Hq;
  r.o = o->data_ptr();
  r.lse = static_cast<float*>(lse->data_ptr());
  if (!ws) {
    const int64_t need = (int64_t)f_workspace(&pg, &r);
    new_ws = at::empty({need > 256 ? need : 256}, q->options().dtype(at::kByte));
    ws = &new_ws;
  }
  const int rc = f_attention(&pg, &r, ws->data_ptr(), (size_t)(ws->numel() * ws->element_size()), stream_of(dev));
  if (rc != 0) return PyLong_FromLong(rc);
  return pair(new_o, a[14], new_lse, a[15]);
}

// k_pages, v_pages, block_table, lens, N, k_scales, v_scales, k, v
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  T kp, vp, table, lens, ks, vs, k, v;
  if (n != 9 || !tensor(a[0], &kp) || !tensor(a[1], &vp) || !tensor(a[2], &table) || !tensor(a[3], &lens) ||
      !tensor(a[5], &ks) || !tensor(a[6], &vs) || !tensor(a[7], &k) || !tensor(a[8], &v) || !PyLong_Check(a[4]))
    return refuse();
  flashmask_pages pg{};
  if (!pages(kp, vp, ks, vs, table, &pg)) return refuse();
  const at::Device dev = kp->device();
  const int64_t N = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  if (!small(N) || !is(lens, at::kInt, dev, {pg.B})) return refuse();
  if ((k == nullptr) != (v == nullptr) || !is_or_none(k, at::kBFloat16, dev, {pg.B, N, pg.Hkv, pg.d}) ||
      !is_or_none(v, at::kBFloat16, dev, {pg.B, N, pg.Hkv, pg.d}))
    return refuse();
  On on(dev);
  at::Tensor nk, nv;
  if (!k) {
    const auto opt = kp->options().dtype(at::kBFloat16);
    nk = at::empty({pg.B, N, pg.Hkv, pg.d}, opt);
    nv = at::empty({pg.B, N, pg.Hkv, pg.d}, opt);
    k = &nk;
    v = &nv;
  }
  const int rc = f_gather(&pg, static_cast<const int32_t*>(lens->data_ptr()), (int32_t)N, k->data_ptr(), v->data_ptr(),
                          stream_of(dev));
  if (rc != 0) return PyLong_FromLong(rc);
  return pair(nk, a[7], nv, a[8]);
}

// A C++ exception (an allocation that does not fit, say) becomes a Python one.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

// The library (path) whose entry points are called.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  f_append = reinterpret_cast<decltype(f_append)>(dlsym(h, "flashmask_paged_append"));
  f_attention = reinterpret_cast<decltype(f_attention)>(dlsym(h, "flashmask_paged_attention"));
  f_workspace = reinterpret_cast<decltype(f_workspace)>(dlsym(h, "flashmask_paged_attention_workspace_size"));
  f_gather = reinterpret_cast<decltype(f_gather)>(dlsym(h, "flashmask_paged_gather"));
  if (!f_append || !f_attention || !f_workspace || !f_gather) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks the paged-cache entry points");
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<append>)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<attention>)), METH_FASTCALL, nullptr},
    {"gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<gather>)), METH_FASTCALL, nullptr},
    {"bind", bind, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
const char key[] = PAGED_BINDING_KEY;
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", key, -1, methods};

}  // namespace

// Tensors are read through torch's C++ layout, which another version need not share; loading under one
// fails here, and the build finds the key in the file.
PyMODINIT_FUNC PyInit__paged_binding() {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  const char* text = version ? PyUnicode_AsUTF8(version) : nullptr;
  const bool same = text && std::strcmp(text, PAGED_BINDING_TORCH) == 0;
  if (text && !same) PyErr_Format(PyExc_ImportError, "%s, not for torch %s", key, text);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return same ? PyModule_Create(&module) : nullptr;
}
