// The Python binding's small calls without Python: the rotating append and the 4-bit
// cache, whose calls of one token per sequence take a few microseconds on the GPU.
//
// Each function gets the arguments that its namesake in bdattn.py got. It asks whether
// they are as they should be (types, shapes, places, the current device), allocates
// what was not given, and calls the C ABI on the current stream. Where something is not
// as it should be it does nothing and returns None, and bdattn.py goes on to say what:
// it holds the same checks in full, and the same call. Outputs are allocated and the
// kernels launched without the interpreter's lock, as both may wait for the GPU.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bdattn.h"

namespace {

PyTypeObject* g_paged_type = nullptr;  // bdattn.Paged

// What a call is about: the geometry and the device, which must be the current one.
struct Call {
  bd_paged g;
  c10::Device dev{c10::kCUDA, 0};
  bool ok = false;

  Call(PyObject* pg, PyObject* first) {
    if (g_paged_type == nullptr || Py_TYPE(pg) != g_paged_type || !THPVariable_Check(first)) return;
    Py_buffer view;
    if (PyObject_GetBuffer(pg, &view, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      return;
    }
    const bool whole = view.len == static_cast<Py_ssize_t>(sizeof(g));
    if (whole) memcpy(&g, view.buf, sizeof(g));
    PyBuffer_Release(&view);
    const c10::Device d = THPVariable_Unpack(first).device();
    if (!whole || !d.is_cuda() || d.index() != c10::cuda::current_device()) return;
    dev = d;
    ok = true;
  }
  bool is(PyObject* o, at::ScalarType type, at::IntArrayRef shape) const {
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.scalar_type() == type && t.device() == dev && t.sizes() == shape && t.is_contiguous();
  }
  // bf16 [T, heads, D] whose heads lie one after the other; the elements from token to token
  bool rows(PyObject* o, int64_t T, int64_t heads, int64_t* stride) const {
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kBFloat16 || t.device() != dev || t.dim() != 3) return false;
    if (t.size(0) != T || t.size(1) != heads || t.size(2) != g.D) return false;
    const int64_t dense = heads * g.D, s = T < 2 ? dense : t.stride(0);
    if (t.stride(2) != 1 || (t.stride(1) != g.D && heads > 1) || s < dense || s % 8 != 0) return false;
    *stride = s;
    return true;
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  }
  bd_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

void* data(PyObject* o) { return THPVariable_Unpack(o).data_ptr(); }
template <class T>
T* data_of(PyObject* o) {
  return static_cast<T*>(data(o));
}

bool cache_of(const Call& c, PyObject* o, bd_cache4* out) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) return false;
  const int64_t n = c.g.n_pages, h = c.g.Hkv, p = c.g.page_size, d = c.g.D;
  void* at[4];
  for (int i = 0; i < 4; ++i) {
    PyObject* t = PyTuple_GET_ITEM(o, i);
    if (!c.is(t, i < 2 ? at::kByte : at::kFloat8_e4m3fn, {n, h, p, i < 2 ? d / 2 : d / 16})) return false;
    at[i] = data(t);
  }
  PyObject *kg = PyTuple_GET_ITEM(o, 4), *vg = PyTuple_GET_ITEM(o, 5);
  if (!PyFloat_Check(kg) || !PyFloat_Check(vg)) return false;
  *out = bd_cache4{at[0], at[1], at[2], at[3], static_cast<float>(PyFloat_AS_DOUBLE(kg)),
                   static_cast<float>(PyFloat_AS_DOUBLE(vg))};
  return true;
}

bool places(const Call& c, PyObject* cu, PyObject* seq_lens, PyObject* table, PyObject* status) {
  const int64_t B = c.g.B, m = c.g.max_pages;
  return c.is(cu, at::kInt, {B + 1}) && c.is(seq_lens, at::kInt, {B}) && c.is(table, at::kInt, {B, m}) &&
         c.is(status, at::kInt, {1});
}

PyObject* failed(int rc, const char* what) {
  return PyErr_Format(PyExc_RuntimeError, "%s failed: %s (code %d)", what, bd_attn_strerror(rc), rc);
}

// None: outputs to be made; else one as it should be.
bool given(const Call& c, PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
  return o == Py_None || c.is(o, type, shape);
}
// An output: the one given, or one made here.
struct Out {
  PyObject* o;
  at::Tensor made;
  void* at = nullptr;

  explicit Out(PyObject* given) : o(given), at(given != Py_None ? data(given) : nullptr) {}
  // without the lock
  void make(const Call& c, at::ScalarType type, at::IntArrayRef shape) {
    if (o != Py_None) return;
    made = c.make(shape, type);
    at = made.data_ptr();
  }
  PyObject* give() const { return o != Py_None ? Py_NewRef(o) : THPVariable_Wrap(made); }
};

struct Unlocked {  // the interpreter's lock is free while one of these lives
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

struct Ref {  // a reference that ends here
  PyObject* o;
  explicit Ref(PyObject* x) : o(x) {}
  ~Ref() { Py_XDECREF(o); }
};

// (q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg, cache or (k_pages, v_pages), status, pairing,
//  q_out, k_out) -> q_out
PyObject* append(PyObject* const* a, bool four) {
  PyObject *q = a[0], *k = a[1], *v = a[2], *cs = a[3], *cu = a[4], *lens = a[5], *table = a[6], *kv = a[8],
           *status = a[9], *q_out = a[11], *k_out = a[12];
  const Call c(a[7], k);
  if (!c.ok || THPVariable_Unpack(k).dim() != 3) Py_RETURN_NONE;
  const int64_t T = THPVariable_Unpack(k).size(0), D = c.g.D, Hq = c.g.Hq, Hkv = c.g.Hkv;
  bd_cache4 cache;
  void *kp = nullptr, *vp = nullptr;
  if (four) {
    if (!cache_of(c, kv, &cache)) Py_RETURN_NONE;
  } else {
    if (!PyTuple_Check(kv) || PyTuple_GET_SIZE(kv) != 2) Py_RETURN_NONE;
    for (int i = 0; i < 2; ++i)
      if (!c.is(PyTuple_GET_ITEM(kv, i), at::kBFloat16, {c.g.n_pages, Hkv, c.g.page_size, D})) Py_RETURN_NONE;
    kp = data(PyTuple_GET_ITEM(kv, 0));
    vp = data(PyTuple_GET_ITEM(kv, 1));
  }
  bd_rope r{};
  if (!PyLong_CheckExact(a[10]) || T > 0x7fffffff) Py_RETURN_NONE;
  const long pairing = PyLong_AsLong(a[10]);
  if (pairing != BD_ROPE_HALVES && pairing != BD_ROPE_ADJACENT) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  r.pairing = static_cast<int>(pairing);
  if (!c.rows(k, T, Hkv, &r.k_stride) || !c.rows(v, T, Hkv, &r.v_stride)) Py_RETURN_NONE;
  if (!places(c, cu, lens, table, status) || !given(c, k_out, at::kBFloat16, {T, Hkv, D})) Py_RETURN_NONE;
  const float* angles = nullptr;
  if (cs != Py_None) {
    if (!THPVariable_CheckExact(cs)) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(cs);
    if (t.dim() != 2 || t.scalar_type() != at::kFloat || t.device() != c.dev || !t.is_contiguous() ||
        t.size(0) > 0x7fffffff || t.size(1) > D || t.size(1) % 16 != 0)
      Py_RETURN_NONE;
    r.n_pos = static_cast<int>(t.size(0));
    r.rot_dim = static_cast<int>(t.size(1));
    angles = data_of<const float>(cs);
  }
  const void* q_at = nullptr;
  if (q != Py_None) {
    if (!c.rows(q, T, Hq, &r.q_stride) || !given(c, q_out, at::kBFloat16, {T, Hq, D})) Py_RETURN_NONE;
    q_at = data(q);
  } else if (q_out != Py_None) {
    Py_RETURN_NONE;
  }
  Out to(q_out);
  const void *k_at = data(k), *v_at = data(v);
  void* k_to = k_out != Py_None ? data(k_out) : nullptr;
  const int n = static_cast<int>(T);
  const int32_t *cu_at = data_of<const int32_t>(cu), *lens_at = data_of<const int32_t>(lens),
                *table_at = data_of<const int32_t>(table);
  int32_t* status_at = data_of<int32_t>(status);
  int rc;
  {
    const Unlocked unlocked;
    if (q != Py_None) to.make(c, at::kBFloat16, {T, Hq, D});
    rc = four ? bd_attn_paged4_append(q_at, k_at, v_at, angles, &r, cu_at, lens_at, table_at, &c.g, n, to.at, k_to,
                                      &cache, status_at, c.stream())
              : bd_attn_paged_append_rope(q_at, k_at, v_at, angles, &r, cu_at, lens_at, table_at, &c.g, n, to.at, k_to,
                                          kp, vp, status_at, c.stream());
  }
  if (rc != BD_OK) return failed(rc, four ? "bd_attn_paged4_append" : "bd_attn_paged_append_rope");
  // a tuple, as None means that nothing was done
  const Ref result(q != Py_None ? to.give() : Py_NewRef(Py_None));
  return result.o != nullptr ? PyTuple_Pack(1, result.o) : nullptr;
}

PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) Py_RETURN_NONE;
  return append(a, false);
  END_HANDLE_TH_ERRORS
}

PyObject* append4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) Py_RETURN_NONE;
  return append(a, true);
  END_HANDLE_TH_ERRORS
}

PyObject* both(const Out& x, const Out& y) {
  const Ref a(x.give()), b(y.give());
  return a.o != nullptr && b.o != nullptr ? PyTuple_Pack(2, a.o, b.o) : nullptr;
}

// (cache, cu, seq_lens, page_table, pg, n_tokens, status, k_out, v_out) -> (k_out, v_out)
PyObject* read4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 6 || !PyLong_CheckExact(a[5])) Py_RETURN_NONE;
  const Call c(a[4], PyTuple_GET_ITEM(a[0], 0));
  bd_cache4 cache;
  if (!c.ok || !cache_of(c, a[0], &cache) || !places(c, a[1], a[2], a[3], a[6])) Py_RETURN_NONE;
  const long long T = PyLong_AsLongLong(a[5]);
  if (T < 0 || T > 0x7fffffff) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int64_t shape[3] = {T, c.g.Hkv, c.g.D};
  if (!given(c, a[7], at::kBFloat16, shape) || !given(c, a[8], at::kBFloat16, shape)) Py_RETURN_NONE;
  const int32_t *cu_at = data_of<const int32_t>(a[1]), *lens_at = data_of<const int32_t>(a[2]),
                *table_at = data_of<const int32_t>(a[3]);
  int32_t* status_at = data_of<int32_t>(a[6]);
  Out k(a[7]), v(a[8]);
  int rc;
  {
    const Unlocked unlocked;
    k.make(c, at::kBFloat16, shape);
    v.make(c, at::kBFloat16, shape);
    rc = bd_attn_paged4_read(&cache, cu_at, lens_at, table_at, &c.g, static_cast<int>(T), k.at, v.at, status_at,
                             c.stream());
  }
  if (rc != BD_OK) return failed(rc, "bd_attn_paged4_read");
  return both(k, v);
  END_HANDLE_TH_ERRORS
}

// (q, cache, page_table, seq_lens, pg, status, out, lse, workspace) -> (out, lse)
PyObject* decode4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  const Call c(a[4], a[0]);
  bd_cache4 cache;
  if (!c.ok || !cache_of(c, a[1], &cache)) Py_RETURN_NONE;
  const int64_t B = c.g.B, Hq = c.g.Hq, D = c.g.D, m = c.g.max_pages;
  if (!c.is(a[0], at::kBFloat16, {B, Hq, D}) || !c.is(a[2], at::kInt, {B, m}) || !c.is(a[3], at::kInt, {B}) ||
      !c.is(a[5], at::kInt, {1}) || !given(c, a[6], at::kBFloat16, {B, Hq, D}) || !given(c, a[7], at::kFloat, {B, Hq}))
    Py_RETURN_NONE;
  const int64_t bytes = static_cast<int64_t>(bd_attn_paged4_decode_workspace_bytes(&c.g));
  if (bytes == 0 || !given(c, a[8], at::kByte, {bytes})) Py_RETURN_NONE;
  const void* q_at = data(a[0]);
  const int32_t *table_at = data_of<const int32_t>(a[2]), *lens_at = data_of<const int32_t>(a[3]);
  int32_t* status_at = data_of<int32_t>(a[5]);
  Out out(a[6]), lse(a[7]), workspace(a[8]);
  int rc;
  {
    const Unlocked unlocked;
    out.make(c, at::kBFloat16, {B, Hq, D});
    lse.make(c, at::kFloat, {B, Hq});
    if (bytes > 16) workspace.make(c, at::kByte, {bytes});  // 16: the call needs none
    rc = bd_attn_paged4_decode(q_at, &cache, table_at, lens_at, &c.g, out.at, static_cast<float*>(lse.at),
                               workspace.at, status_at, c.stream());
  }
  if (rc != BD_OK) return failed(rc, "bd_attn_paged4_decode");
  return both(out, lse);
  END_HANDLE_TH_ERRORS
}

PyObject* setup(PyObject*, PyObject* paged) {
  if (!PyType_Check(paged)) return PyErr_Format(PyExc_TypeError, "a type expected");
  Py_INCREF(paged);
  g_paged_type = reinterpret_cast<PyTypeObject*>(paged);
  Py_RETURN_NONE;
}

template <PyObject* (*kF)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kF));
}
PyMethodDef g_methods[] = {{"setup", setup, METH_O, nullptr},
                           {"append_rope", fast<append_rope>(), METH_FASTCALL, nullptr},
                           {"append4", fast<append4>(), METH_FASTCALL, nullptr},
                           {"read4", fast<read4>(), METH_FASTCALL, nullptr},
                           {"decode4", fast<decode4>(), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
