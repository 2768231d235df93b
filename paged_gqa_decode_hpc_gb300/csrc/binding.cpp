// The Python binding's calls whose host time is most of a small step, as an
// extension module: torch tensors become hpc_tensor descriptors here (0.2 us each
// instead of 0.6 by struct packing) and the C entry is called through the address
// that the package's ctypes binding has loaded. Arguments that are not as expected
// make a call return None before anything has run; the package then takes its
// ctypes path, which raises the error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <cstring>

#include "hpc_decode.h"

namespace {

PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride;  // attribute names
PyObject* dtypes;                                     // {torch dtype: hpc_dtype}
decltype(&hpc_block_table_append) append_entry;
decltype(&hpc_block_table_truncate) truncate_entry;
decltype(&hpc_rope_kv_write) rope_entry;
decltype(&hpc_decode_prefix_attn) prefix_entry;

bool longs(PyObject* t, int64_t* out, int* n) {
  if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return false;
  const int count = (int)PyTuple_GET_SIZE(t);
  if (*n >= 0 && *n != count) return false;
  *n = count;
  for (int i = 0; i < count; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

bool address(PyObject* t, void** out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return false;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

// A descriptor, or null for None.
struct Tensor {
  hpc_tensor d;
  hpc_tensor* p = nullptr;
  bool set(PyObject* t, double scale = 1.0) {
    if (t == Py_None) return true;
    std::memset(&d, 0, sizeof d);
    if (!address(t, &d.data)) return false;
    PyObject* type = PyObject_GetAttr(t, s_dtype);
    if (!type) return false;
    PyObject* code = PyDict_GetItemWithError(dtypes, type);
    Py_DECREF(type);
    if (!code) return false;
    d.dtype = (int32_t)PyLong_AsLong(code);
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    int n = -1;
    bool ok = longs(shape, d.shape, &n);
    Py_XDECREF(shape);
    if (!ok) return false;
    PyObject* stride = PyObject_CallMethodNoArgs(t, s_stride);
    ok = longs(stride, d.stride, &n);
    Py_XDECREF(stride);
    if (!ok) return false;
    d.ndim = n;
    d.scale = (float)scale;
    p = &d;
    return true;
  }
};

bool number(PyObject* o, double* out) {
  *out = PyFloat_AsDouble(o);
  return !(*out == -1.0 && PyErr_Occurred());
}
bool int32(PyObject* o, int32_t* out) {
  const long v = PyLong_AsLong(o);
  if ((v == -1 && PyErr_Occurred()) || v < INT_MIN || v > INT_MAX) return false;
  *out = (int32_t)v;
  return true;
}
bool error_word(PyObject* t, int32_t** out) {
  void* p = nullptr;
  if (t != Py_None && !address(t, &p)) return false;
  *out = (int32_t*)p;
  return true;
}
bool handle(PyObject* o, void** out) {
  *out = o == Py_None ? nullptr : PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}

PyObject* not_called() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <typename F>
PyObject* called(F call) {
  hpc_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)st);
}

// (seq_lens, new_lens, free_blocks, free_count, num_blocks, block_table, seq_lens_out,
//  cu_q_lens, positions, slots, free_count_out, device_error, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor t[10];
  int32_t blocks, *err;
  void* stream;
  if (n != 13 || !int32(a[4], &blocks) || !error_word(a[11], &err) || !handle(a[12], &stream))
    return not_called();
  for (int i = 0; i < 10; ++i)
    if (!t[i].set(a[i < 4 ? i : i + 1])) return not_called();
  return called([&] {
    return append_entry(t[0].p, t[1].p, t[2].p, t[3].p, blocks, t[4].p, t[5].p, t[6].p, t[7].p,
                        t[8].p, t[9].p, err, stream);
  });
}

// (seq_lens, to_lens, block_table, num_blocks, free_blocks, free_count, seq_lens_out,
//  free_count_out, device_error, stream)
PyObject* truncate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor t[7];
  int32_t blocks, *err;
  void* stream;
  if (n != 10 || !int32(a[3], &blocks) || !error_word(a[8], &err) || !handle(a[9], &stream))
    return not_called();
  for (int i = 0; i < 7; ++i)
    if (!t[i].set(a[i < 3 ? i : i + 1])) return not_called();
  return called([&] {
    return truncate_entry(t[0].p, t[1].p, t[2].p, blocks, t[3].p, t[4].p, t[5].p, t[6].p, err,
                          stream);
  });
}

// (q_in, k_in, v_in, positions, slots, rope, q_norm_weight, k_norm_weight, eps, q_out,
//  q_out_fp8, q_fp8_scale, k_cache, k_scale, v_cache, v_scale, device_error, stream)
PyObject* rope_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, v, pos, slots, wq, wk, out, out8, kc, vc;
  double eps, qs, ks, vs;
  int32_t* err;
  void* stream;
  if (n != 18 || !number(a[8], &eps) || !number(a[11], &qs) || !number(a[13], &ks) ||
      !number(a[15], &vs) || !error_word(a[16], &err) || !handle(a[17], &stream) || !q.set(a[0]) ||
      !k.set(a[1]) || !v.set(a[2]) || !pos.set(a[3]) || !slots.set(a[4]) || !wq.set(a[6]) ||
      !wk.set(a[7]) || !out.set(a[9]) || !out8.set(a[10], qs) || !kc.set(a[12], ks) ||
      !vc.set(a[14], vs))
    return not_called();
  Py_buffer b;
  if (PyObject_GetBuffer(a[5], &b, PyBUF_SIMPLE) != 0) return not_called();
  hpc_rope table;
  const bool ok = b.len == (Py_ssize_t)sizeof table;
  if (ok) std::memcpy(&table, b.buf, sizeof table);
  PyBuffer_Release(&b);
  if (!ok) return not_called();
  return called([&] {
    return rope_entry(q.p, k.p, v.p, pos.p, slots.p, &table, wq.p, wk.p, (float)eps, out.p, out8.p,
                      kc.p, vc.p, err, stream);
  });
}

// (q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu_groups, prefix_lens,
//  plan, out, lse, softmax_scale, stream)
PyObject* prefix_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, v, bt, lens, cu, prefixes, out, lse;
  double ks, vs, scale;
  void *plan, *stream;
  if (n != 14 || !number(a[2], &ks) || !number(a[4], &vs) || !number(a[12], &scale) ||
      !handle(a[9], &plan) || !handle(a[13], &stream) || !q.set(a[0]) || !k.set(a[1], ks) ||
      !v.set(a[3], vs) || !bt.set(a[5]) || !lens.set(a[6]) || !cu.set(a[7]) ||
      !prefixes.set(a[8]) || !out.set(a[10]) || !lse.set(a[11]))
    return not_called();
  return called([&] {
    return prefix_entry(q.p, k.p, v.p, bt.p, lens.p, cu.p, prefixes.p, (hpc_plan_t)plan, out.p,
                        lse.p, (float)scale, stream);
  });
}

// bind(dtypes, append, truncate, rope_kv_write, prefix_attn): the entries' addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[4];
  if (n != 5 || !PyDict_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "bind(dtypes, four addresses)");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XSETREF(dtypes, a[0]);
  append_entry = (decltype(append_entry))f[0];
  truncate_entry = (decltype(truncate_entry))f[1];
  rope_entry = (decltype(rope_entry))f[2];
  prefix_entry = (decltype(prefix_entry))f[3];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(append), FAST(truncate), FAST(rope_kv_write),
                         FAST(prefix_attn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "hpc_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_hpc_binding(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  if (!s_data_ptr || !s_dtype || !s_shape || !s_stride) return nullptr;
  return PyModule_Create(&module);
}
