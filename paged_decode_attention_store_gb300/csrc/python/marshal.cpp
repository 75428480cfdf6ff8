// Argument marshalling of the calls that a step makes once a layer (rotary stores, rows back, four-bit attention): binding.py's
// checks on plain arguments and the C call, without ctypes. A small call is bound by its host side: 10 us of which the checks in
// Python and ctypes' conversions were 7. Each function returns the call's status, or None where an argument is anything but
// what the call takes as it is: binding.py then goes its own way, which says what is wrong.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>

namespace {

// Reads arguments in order; ``ok`` turns false at the first that is not plain.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;
  bool ok = true;

  PyObject* next() {
    if (left <= 0) {
      ok = false;
      return Py_None;
    }
    --left;
    return *at++;
  }
  long long integer() {
    PyObject* o = next();
    if (!PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over) ok = false;
    return x;
  }
  int int32() {
    const long long x = integer();
    if (x < INT_MIN || x > INT_MAX) ok = false;
    return (int)x;
  }
  void* address() {
    PyObject* o = next();
    if (!PyLong_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    return reinterpret_cast<void*>((uintptr_t)PyLong_AsUnsignedLongLongMask(o));
  }
  double number() {
    PyObject* o = next();
    if (PyFloat_CheckExact(o)) return PyFloat_AS_DOUBLE(o);
    if (!PyLong_CheckExact(o)) ok = false;
    const double x = ok ? PyLong_AsDouble(o) : 0.0;
    if (PyErr_Occurred()) {  // past a double's range: Python's way says so
      PyErr_Clear();
      ok = false;
    }
    return x;
  }
  // None: the current stream
  void* stream() {
    PyObject* o = next();
    if (o == Py_None) return ok ? c10::cuda::getCurrentCUDAStream().stream() : nullptr;
    --at;
    ++left;
    return address();
  }
  const at::Tensor* tensor() {
    PyObject* o = next();
    if (!THPVariable_CheckExact(o)) {
      if (o != Py_None) ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
};

struct Where {
  int device;
  at::ScalarType type;
  bool holds(const at::Tensor* t) const {
    return t && t->layout() == at::kStrided && t->is_cuda() && t->get_device() == device && t->scalar_type() == type;
  }
  // contiguous int32
  bool indices(const at::Tensor* t) const {
    return t && t->layout() == at::kStrided && t->is_cuda() && t->get_device() == device && t->scalar_type() == at::kInt &&
           t->is_contiguous();
  }
};

Where where(Args& a) {
  Where w;
  w.type = a.int32() ? at::kBFloat16 : at::kFloat;
  w.device = a.int32();
  return w;
}

template <typename T = void>
T* pointer(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

struct Heads {
  void* p = nullptr;
  long long token = 0, head = 0, n = 0;
  int heads = 0;
};
bool heads_view(const at::Tensor* t, const Where& w, long long width, Heads* o) {
  if (!w.holds(t) || t->dim() != 3 || t->size(2) != width || t->size(1) > INT_MAX || (t->stride(2) != 1 && width > 1)) return false;
  o->p = pointer(t);
  o->n = t->size(0);
  o->heads = (int)t->size(1);
  o->head = o->heads <= 1 ? width : t->stride(1);
  o->token = o->n <= 1 ? std::max<long long>(t->stride(0), (o->heads - 1) * o->head + width) : t->stride(0);
  return true;
}

bool rows_view(const at::Tensor* t, const Where& w, long long n, long long heads, long long width, long long* stride) {
  if (!w.holds(t)) return false;
  bool good;
  if (t->dim() == 3)
    good = t->size(1) == heads && t->size(2) == width && (width == 1 || t->stride(2) == 1) && (heads == 1 || t->stride(1) == width);
  else
    good = t->dim() == 2 && heads == 1 && t->size(1) == width && (width == 1 || t->stride(1) == 1);
  *stride = n > 1 ? t->stride(0) : heads * width;
  return good && t->size(0) == n;
}

PyObject* none() { Py_RETURN_NONE; }

// What a function throws (a machine without CUDA, say) is left to Python's way.
template <typename F>
PyObject* guarded(const F& f) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    return none();
  }
}

template <typename F>
PyObject* called(const F& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

using Plain = int (*)(const void*, int, const void*, long long, long long, int, const void*, long long, const void*, long long,
                      const int32_t*, const int32_t*, int, const uint64_t*, int, int, float, void*, long long, long long, void*);
using OnAxes = int (*)(const void*, int, const void*, long long, long long, int, const void*, long long, const void*, long long,
                       const int32_t*, long long, const int32_t*, int, const uint64_t*, const uint8_t*, int, int, int, float,
                       void*, long long, long long, void*);

// (call, whether it takes axes, pool, dtype, device, layer, q, first, heads, width, second, heads, width, positions, out_loc,
//  frequencies, pair_axis, axes, rotary_dim, layout, factor, q_out, width, stream); rows as they are: no positions, no
//  frequencies
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    Args a{args, count};
    void* call = a.address();
    const bool takes_axes = a.int32();
    const void* pool = a.address();
    const Where w = where(a);
    const int layer = a.int32();
    const at::Tensor* q = a.tensor();
    const at::Tensor* k = a.tensor();
    const long long k_heads = a.integer(), k_width = a.integer();
    const at::Tensor* v = a.tensor();
    const long long v_heads = a.integer(), v_width = a.integer();
    const at::Tensor* positions = a.tensor();
    const at::Tensor* out_loc = a.tensor();
    const at::Tensor* freqs = a.tensor();
    const at::Tensor* pair_axis = a.tensor();
    const int axes = a.int32(), rot = a.int32(), layout = a.int32();
    const float factor = (float)a.number();
    const at::Tensor* q_out = a.tensor();
    const long long width = a.integer();
    void* stream = a.stream();
    if (!a.ok || a.left || (rot && !(freqs && freqs->is_cuda() && freqs->get_device() == w.device)) || rot > width) return none();
    if (!positions != !freqs || (!positions && q) || !k != !v || (!q && !k) || axes < 1 || (axes > 1 && !pair_axis)) return none();
    long long n, apart = 0;
    if (axes == 1) {  // positions, or, of rows as they are, slots
      if (!w.indices(positions ? positions : out_loc)) return none();
      n = (positions ? positions : out_loc)->numel();
    } else {
      if (positions->layout() != at::kStrided || !positions->is_cuda() || positions->get_device() != w.device ||
          positions->scalar_type() != at::kInt || positions->dim() != 2 || positions->size(0) != axes)
        return none();
      n = positions->size(1);
      if (n > 1 && positions->stride(1) != 1) return none();
      apart = n ? positions->stride(0) : 0;
      if (apart < n) return none();
    }
    if (n > INT_MAX) return none();
    Heads in, out;
    if (q && (!heads_view(q, w, width, &in) || !heads_view(q_out, w, width, &out) || in.heads != out.heads || in.n != n || out.n != n))
      return none();
    long long k_stride = 0, v_stride = 0;
    if (k && (!rows_view(k, w, n, k_heads, k_width, &k_stride) || !rows_view(v, w, n, v_heads, v_width, &v_stride) ||
              !w.indices(out_loc) || out_loc->numel() != n))
      return none();
    const int32_t* loc = k ? pointer<int32_t>(out_loc) : nullptr;
    const int32_t* pos = pointer<int32_t>(positions);
    const uint64_t* f = pointer<uint64_t>(freqs);
    if (takes_axes) {
      const uint8_t* of_pair = axes > 1 ? pointer<uint8_t>(pair_axis) : nullptr;
      return called([&] {
        return reinterpret_cast<OnAxes>(call)(pool, layer, in.p, in.token, in.head, in.heads, pointer(k), k_stride, pointer(v),
                                              v_stride, pos, apart, loc, (int)n, f, of_pair, axes, rot, layout, factor, out.p,
                                              out.token, out.head, stream);
      });
    }
    return called([&] {
      return reinterpret_cast<Plain>(call)(pool, layer, in.p, in.token, in.head, in.heads, pointer(k), k_stride, pointer(v),
                                           v_stride, pos, loc, (int)n, f, rot, layout, factor, out.p, out.token, out.head, stream);
    });
  });
}

using Load = int (*)(const void*, int, const int32_t*, int, void*, void*, void*);

// (call, pool, dtype, device, layer, slots, k_out, v_out, entries of a row, stream)
PyObject* load(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    Args a{args, count};
    void* call = a.address();
    const void* pool = a.address();
    const Where w = where(a);
    const int layer = a.int32();
    const at::Tensor* slots = a.tensor();
    const at::Tensor* k = a.tensor();
    const at::Tensor* v = a.tensor();
    const long long entries = a.integer();
    void* stream = a.stream();
    if (!a.ok || a.left || !w.indices(slots) || !w.holds(k) || !w.holds(v) || !k->is_contiguous() || !v->is_contiguous()) return none();
    const long long n = slots->numel();
    if (n > INT_MAX || k->numel() != n * entries || v->numel() != n * entries) return none();
    return called([&] {
      return reinterpret_cast<Load>(call)(pool, layer, pointer<int32_t>(slots), (int)n, pointer(k), pointer(v), stream);
    });
  });
}

using Attend = int (*)(const void*, int, const void*, int, int, int, const int32_t*, const int32_t*, int, int, int, const int32_t*,
                       const int32_t*, int, int, int, float, void*, void*, size_t, void*);

// (call, pool, dtype, device, head_dim, page_size, layer, q, q_lens, table, table_mode, table_rows, context_lens, max_context or
//  None, window, sinks, scale, out, workspace, stream)
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    Args a{args, count};
    void* call = a.address();
    const void* pool = a.address();
    const Where w = where(a);
    const long long head_dim = a.integer(), page_size = a.integer();
    const int layer = a.int32();
    const at::Tensor* q = a.tensor();
    const at::Tensor* q_lens = a.tensor();
    const at::Tensor* table = a.tensor();
    const int mode = a.int32();
    const at::Tensor* table_rows = a.tensor();
    const at::Tensor* context_lens = a.tensor();
    if (!a.ok || !w.holds(q) || q->dim() != 4 || !q->is_contiguous() || q->size(3) != head_dim || !w.indices(table) ||
        table->dim() != 2 || table->size(0) > INT_MAX || table->size(1) > INT_MAX)
      return none();
    long long longest = (mode == 1 ? 1 : page_size) * table->size(1);
    if (a.left && *a.at == Py_None) a.next();
    else longest = a.integer();
    longest = std::min<long long>(longest, INT_MAX);
    const int window = a.int32(), sinks = a.int32();
    const float scale = (float)a.number();
    const at::Tensor* out = a.tensor();
    const at::Tensor* workspace = a.tensor();
    void* stream = a.stream();
    if (!a.ok || a.left || longest < INT_MIN || !w.holds(out) || !out->is_contiguous() || !out->sizes().equals(q->sizes())) return none();
    if (!workspace || workspace->layout() != at::kStrided || !workspace->is_cuda() || workspace->get_device() != w.device ||
        !workspace->is_contiguous())
      return none();
    const long long B = q->size(0);
    for (int i = 0; i < 3; ++i)
      if (q->size(i) > INT_MAX) return none();
    if (!w.indices(context_lens) || context_lens->numel() != B) return none();
    for (const at::Tensor* t : {q_lens, table_rows})
      if (t && (!w.indices(t) || t->numel() != B)) return none();
    return called([&] {
      return reinterpret_cast<Attend>(call)(pool, layer, pointer(q), (int)B, (int)q->size(1), (int)q->size(2),
                                            pointer<int32_t>(q_lens), pointer<int32_t>(table), (int)table->size(0),
                                            (int)table->size(1), mode, pointer<int32_t>(table_rows),
                                            pointer<int32_t>(context_lens), (int)longest, window, sinks, scale, pointer(out),
                                            pointer(workspace), workspace->nbytes(), stream);
    });
  });
}

// Tensor ``i`` of a list or tuple.
const at::Tensor* item(PyObject* list, Py_ssize_t i) {
  PyObject* o = nullptr;
  if (PyList_CheckExact(list) && i < PyList_GET_SIZE(list)) o = PyList_GET_ITEM(list, i);
  else if (PyTuple_CheckExact(list) && i < PyTuple_GET_SIZE(list)) o = PyTuple_GET_ITEM(list, i);
  return o && THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// (dtype, device, layers, q, out, k, v, B, C, heads, K/V heads, head_dim): whether every layer's tensors are what a four-bit
// cache's step takes; None where one is not, or is nothing plain.
PyObject* step(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    Args a{args, count};
    const Where w = where(a);
    const long long layers = a.integer();
    PyObject *q = a.next(), *out = a.next(), *k = a.next(), *v = a.next();
    const long long B = a.integer(), C = a.integer(), H = a.integer(), hkv = a.integer(), D = a.integer();
    if (!a.ok || a.left) return none();
    for (long long l = 0; l < layers; ++l) {
      for (PyObject* list : {q, out}) {
        const at::Tensor* t = item(list, l);
        if (!w.holds(t) || t->dim() != 4 || t->size(0) != B || t->size(1) != C || t->size(2) != H || t->size(3) != D ||
            !t->is_contiguous() || (reinterpret_cast<uintptr_t>(t->data_ptr()) & 15))
          return none();
      }
      for (PyObject* list : {k, v}) {
        const at::Tensor* t = item(list, l);
        long long stride;
        if (!w.holds(t) || !rows_view(t, w, B * C, hkv, D, &stride)) return none();
      }
    }
    Py_RETURN_TRUE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef methods[] = {{"rotary", entry<rotary>(), METH_FASTCALL, nullptr},
                         {"load", entry<load>(), METH_FASTCALL, nullptr},
                         {"attend", entry<attend>(), METH_FASTCALL, nullptr},
                         {"step", entry<step>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", KVP_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
