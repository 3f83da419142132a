// marshal.cpp -- what the Python binding reads off torch tensors, in one native call each: a decode step's kernels
// run for a few microseconds, and a tensor's shape, strides, dtype and pointer cost one microsecond of
// Python attribute reads (0.1 here).  The decoding calls are made whole from here: an append 6.5 us -> 3.7 on a Grace core,
// a gradient 8.6 -> 4.6, a verification 6.9 -> 3.3, an attention 8.4 -> 5.4.  Built where torch's headers are found; the
// binding falls back to Python reads without it, with the same checks and the same errors.
// Everything here answers None where a read fails, or throws (a sparse tensor's strides): the binding's Python reads
// then name what is wrong.
#include <ATen/Context.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <Python.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/qnre.h"

namespace {

// qnre_dtype_t, then 3 = int32, 4 = int64; -1 for the rest.
int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return QNRE_DTYPE_BF16;
    case at::kHalf: return QNRE_DTYPE_FP16;
    case at::kFloat: return QNRE_DTYPE_FP32;
    case at::kInt: return 3;
    case at::kLong: return 4;
    default: return -1;
  }
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    Py_RETURN_NONE;
  }
}

bool read_view4(PyObject* obj, qnre_tensor4_t* v) {
  if (!THPVariable_Check(obj)) return false;
  const at::Tensor& t = THPVariable_Unpack(obj);
  const int code = code_of(t);
  if (t.dim() != 4 || code < 0 || code > QNRE_DTYPE_FP32) return false;
  std::memset(v, 0, sizeof(*v));
  v->data = t.data_ptr();
  for (int i = 0; i < 4; ++i) {
    v->shape[i] = t.size(i);
    v->stride[i] = t.stride(i);
  }
  v->dtype = code;
  return true;
}

// The address of a contiguous tensor of that type and shape.
template <typename T>
bool read_pointer(PyObject* obj, int code, std::initializer_list<int64_t> shape, T** out) {
  if (!THPVariable_Check(obj)) return false;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (code_of(t) != code || !t.is_contiguous() || !t.sizes().equals(at::IntArrayRef(shape))) return false;
  *out = static_cast<T*>(t.data_ptr());
  return true;
}

// Every tensor given (None passes) lies on one device, and that is the current CUDA device, where the kernels run.  (Where
// there is no CUDA at all tensors of the CPU pass: the entry points check them and launch nothing.)
bool on_device(std::initializer_list<PyObject*> objs) {
  const at::Tensor* first = nullptr;
  for (PyObject* o : objs) {
    if (o == Py_None) continue;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (first == nullptr) first = &t;
    if (t.device() != first->device()) return false;
  }
  if (first == nullptr) return false;
  if (!first->is_cuda()) return first->is_cpu() && !at::hasCUDA();
  return first->device() == c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice();
}

// view4(tensor) -> the bytes of its qnre_tensor4_t, or None where it is no rank-4 tensor of a known float type.
PyObject* view4(PyObject*, PyObject* obj) {
  return guarded([&]() -> PyObject* {
    qnre_tensor4_t v;
    if (!read_view4(obj, &v)) Py_RETURN_NONE;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&v), sizeof(v));
  });
}

// pointer(tensor, code, *shape) -> its address, or None unless it is contiguous, of that type and (where given) shape.
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n < 2 || !THPVariable_Check(args[0])) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    if (code_of(t) != PyLong_AsLong(args[1]) || !t.is_contiguous()) Py_RETURN_NONE;
    if (n > 2) {
      if (t.dim() != n - 2) Py_RETURN_NONE;
      for (Py_ssize_t i = 0; i < n - 2; ++i)
        if (t.size(i) != PyLong_AsLongLong(args[2 + i])) Py_RETURN_NONE;
    }
    return PyLong_FromVoidPtr(t.data_ptr());
  });
}

// sizes(tensor) -> its shape as a plain tuple.
PyObject* sizes(PyObject*, PyObject* obj) {
  return guarded([&]() -> PyObject* {
    if (!THPVariable_Check(obj)) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(obj);
    PyObject* r = PyTuple_New(t.dim());
    if (r == nullptr) return nullptr;
    for (int64_t i = 0; i < t.dim(); ++i) PyTuple_SET_ITEM(r, i, PyLong_FromLongLong(t.size(i)));
    return r;
  });
}

// type_code(tensor) -> as code_of.
PyObject* type_code(PyObject*, PyObject* obj) {
  return PyLong_FromLong(THPVariable_Check(obj) ? code_of(THPVariable_Unpack(obj)) : -1);
}

// ------------------------------------------------------------------ whole calls
// name(entry point's address, its arguments in the binding's order.., style code, stream reader, stream) -> status, or
// None where an argument does not read.  The stream is asked for last, as the binding does.

bool read_int(PyObject* obj, int* out) {
  const long x = PyLong_Check(obj) ? PyLong_AsLong(obj) : LONG_MAX;
  if (PyErr_Occurred()) PyErr_Clear();
  if (x > INT_MAX || x < INT_MIN) return false;
  *out = static_cast<int>(x);
  return true;
}

// What the three calls share: q, k, the norm weights, the table and the positions, six arguments.
struct Head {
  qnre_tensor4_t q, k;
  void *wq, *wk;
  float* cos_sin;
  int64_t n_pos;
  int rot;
  int32_t* positions;
};

bool read_head(PyObject* const* args, PyObject* positions, Head* h) {
  if (!read_view4(args[0], &h->q) || !read_view4(args[1], &h->k)) return false;
  const int64_t dim = h->q.shape[3];
  if (!read_pointer(args[2], h->q.dtype, {dim}, &h->wq) || !read_pointer(args[3], h->k.dtype, {dim}, &h->wk)) return false;
  if (!THPVariable_Check(args[4])) return false;
  const at::Tensor& table = THPVariable_Unpack(args[4]);
  if (table.dim() != 2 || table.size(1) > INT_MAX) return false;
  h->n_pos = table.size(0);
  h->rot = static_cast<int>(table.size(1));
  if (!read_pointer(args[4], QNRE_DTYPE_FP32, {table.size(0), table.size(1)}, &h->cos_sin)) return false;
  h->positions = nullptr;
  return positions == Py_None || read_pointer(positions, 3, {h->q.shape[0], h->q.shape[1]}, &h->positions);
}

bool read_entry(PyObject* obj, void** fn) {
  *fn = PyLong_AsVoidPtr(obj);
  if (PyErr_Occurred()) PyErr_Clear();
  return *fn != nullptr;
}

// stream(reader, stream) -> false with a Python error set.
bool read_stream(PyObject* reader, PyObject* stream, qnre_stream_t* out) {
  PyObject* r = PyObject_CallOneArg(reader, stream);
  if (r == nullptr) return false;
  *out = r == Py_None ? nullptr : reinterpret_cast<qnre_stream_t>(PyLong_AsVoidPtr(r));
  Py_DECREF(r);
  return PyErr_Occurred() == nullptr;
}

// norm(fn, q, k, wq, wk, cos_sin, positions, q_out, k_out, style, reader, stream)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    Head h;
    qnre_tensor4_t qo, ko;
    int style;
    qnre_stream_t stream;
    if (n != 12 || !read_entry(args[0], &fn) || !read_head(args + 1, args[6], &h) || !read_view4(args[7], &qo) ||
        !read_view4(args[8], &ko) || !read_int(args[9], &style) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6], args[7], args[8]}))
      Py_RETURN_NONE;
    if (!read_stream(args[10], args[11], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_qk_norm_rope)>(fn)(&h.q, &h.k, h.wq, h.wk, h.cos_sin, h.n_pos, h.rot, style,
                                                            h.positions, &qo, &ko, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// norm_backward(fn, gq, gk, q, k, wq, wk, cos_sin, positions, dq, dk, dwq, dwk, workspace, style, reader, stream)
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    Head h;
    qnre_tensor4_t gq, gk, dq, dk;
    float *dwq, *dwk;
    int style;
    qnre_stream_t stream;
    if (n != 17 || !read_entry(args[0], &fn) || !read_view4(args[1], &gq) || !read_view4(args[2], &gk) ||
        !read_head(args + 3, args[8], &h) || !read_view4(args[9], &dq) || !read_view4(args[10], &dk) ||
        !read_pointer(args[11], QNRE_DTYPE_FP32, {h.q.shape[3]}, &dwq) ||
        !read_pointer(args[12], QNRE_DTYPE_FP32, {h.q.shape[3]}, &dwk) || !THPVariable_Check(args[13]) ||
        !read_int(args[14], &style) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6], args[7], args[8], args[9], args[10], args[11],
                    args[12], args[13]}))
      Py_RETURN_NONE;
    const at::Tensor& ws = THPVariable_Unpack(args[13]);
    if (!ws.is_contiguous()) Py_RETURN_NONE;
    void* ws_data = ws.data_ptr();
    const uint64_t ws_bytes = ws.nbytes();
    if (!read_stream(args[15], args[16], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_qk_norm_rope_backward)>(fn)(&gq, &gk, &h.q, &h.k, h.wq, h.wk, h.cos_sin, h.n_pos,
                                                                     h.rot, style, h.positions, &dq, &dk, dwq, dwk,
                                                                     ws_data, ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// append(fn, q, k, v, wq, wk, cos_sin, positions, q_out, cache address, its k, layer, rows, counts, style, reader, stream)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache;
    Head h;
    qnre_tensor4_t v, qo;
    int32_t *rows, *counts = nullptr;
    int layer, style;
    qnre_stream_t stream;
    if (n != 17) Py_RETURN_NONE;
    PyObject* const head[] = {args[1], args[2], args[4], args[5], args[6]};
    if (!read_entry(args[0], &fn) || !read_head(head, args[7], &h) || !read_view4(args[3], &v) ||
        !read_view4(args[8], &qo) || !read_entry(args[9], &cache) || !read_int(args[11], &layer) ||
        !read_pointer(args[12], 3, {h.q.shape[0]}, &rows) ||
        (args[13] != Py_None && !read_pointer(args[13], 3, {h.q.shape[0]}, &counts)) || !read_int(args[14], &style) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6], args[7], args[8], args[10], args[12], args[13]}))
      Py_RETURN_NONE;
    if (!read_stream(args[15], args[16], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_qkv_norm_rope_append)>(fn)(
        &h.q, &h.k, &v, h.wq, h.wk, h.cos_sin, h.n_pos, h.rot, style, h.positions, &qo,
        static_cast<const qnre_cache_t*>(cache), layer, rows, counts, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// attention(fn, q, cache address, its k, layer, rows, mask, out, lse, counts, scale, workspace, reader, stream)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache, *out;
    qnre_tensor4_t q;
    int layer;
    int32_t *rows, *counts = nullptr;
    uint64_t* mask = nullptr;
    float* lse = nullptr;
    qnre_stream_t stream;
    if (n != 14 || !read_entry(args[0], &fn) || !read_view4(args[1], &q) || !read_entry(args[2], &cache) ||
        !read_int(args[4], &layer) || !read_pointer(args[5], 3, {q.shape[0]}, &rows) ||
        (args[6] != Py_None && !read_pointer(args[6], 4, {q.shape[0], q.shape[1]}, &mask)) ||
        !read_pointer(args[7], q.dtype, {q.shape[0], q.shape[1], q.shape[2], q.shape[3]}, &out) ||
        (args[8] != Py_None &&
         !read_pointer(args[8], QNRE_DTYPE_FP32, {q.shape[0], q.shape[1], q.shape[2]}, &lse)) ||
        (args[9] != Py_None && !read_pointer(args[9], 3, {q.shape[0]}, &counts)) ||
        (args[10] != Py_None && !PyFloat_Check(args[10])) || !THPVariable_Check(args[11]) ||
        !on_device({args[1], args[3], args[5], args[6], args[7], args[8], args[9], args[11]}))
      Py_RETURN_NONE;
    const double scale =
        args[10] == Py_None ? std::pow(static_cast<double>(q.shape[3]), -0.5) : PyFloat_AS_DOUBLE(args[10]);
    const at::Tensor& ws = THPVariable_Unpack(args[11]);
    if (!ws.is_contiguous()) Py_RETURN_NONE;
    void* ws_data = ws.data_ptr();
    const uint64_t ws_bytes = ws.nbytes();
    if (!read_stream(args[12], args[13], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_tree_attention)>(fn)(&q, static_cast<const qnre_cache_t*>(cache), layer, rows, mask,
                                                              counts, static_cast<float>(scale), out, lse, ws_data,
                                                              ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// Rows of probabilities [n, nodes, vocab], each contiguous, or None.
struct Rows {
  const float* data = nullptr;
  int64_t stride0 = 0, stride1 = 0;
};

bool read_rows(PyObject* obj, at::IntArrayRef shape, Rows* r) {
  if (!THPVariable_Check(obj)) return false;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (t.scalar_type() != at::kFloat || !t.sizes().equals(shape)) return false;
  const bool whole = t.is_contiguous();
  if (!whole && t.stride(2) != 1 && shape[2] > 1) return false;
  r->data = static_cast<const float*>(t.data_ptr());
  r->stride0 = whole ? shape[1] * shape[2] : t.stride(0);
  r->stride1 = whole ? shape[2] : t.stride(1);
  return true;
}

// verify(fn, target, draft, tokens, parents, accept_u, sample_u, path, counts, next, node_counts, reader, stream)
PyObject* verify(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void* fn;
    Rows target, draft;
    int32_t *tokens, *parents, *path, *counts, *next, *node_counts = nullptr;
    float *accept, *sample;
    qnre_stream_t stream;
    if (argc != 13 || !read_entry(args[0], &fn) || !THPVariable_Check(args[1])) Py_RETURN_NONE;
    const at::IntArrayRef shape = THPVariable_Unpack(args[1]).sizes();
    if (shape.size() != 3 || shape[0] > INT_MAX || shape[1] > INT_MAX) Py_RETURN_NONE;
    const int64_t n = shape[0], nodes = shape[1];
    if (!read_rows(args[1], shape, &target) || (args[2] != Py_None && !read_rows(args[2], shape, &draft)) ||
        !read_pointer(args[3], 3, {n, nodes}, &tokens) || !read_pointer(args[4], 3, {n, nodes}, &parents) ||
        !read_pointer(args[5], QNRE_DTYPE_FP32, {n, nodes}, &accept) ||
        !read_pointer(args[6], QNRE_DTYPE_FP32, {n}, &sample) || !read_pointer(args[7], 3, {n, nodes}, &path) ||
        !read_pointer(args[8], 3, {n}, &counts) || !read_pointer(args[9], 3, {n}, &next) ||
        (args[10] != Py_None && !read_pointer(args[10], 3, {n}, &node_counts)) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6], args[7], args[8], args[9], args[10]}))
      Py_RETURN_NONE;
    if (!read_stream(args[11], args[12], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_verify_tree)>(fn)(
        target.data, target.stride0, target.stride1, draft.data, draft.stride0, draft.stride1, static_cast<int>(n),
        static_cast<int>(nodes), shape[2], tokens, parents, node_counts, accept, sample, path, counts, next, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// cache_rows(fn, cache address, its k, first, second, reader, stream): truncate, fork, reserve, copy_pages
PyObject* cache_rows(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache;
    int32_t *first, *second;
    qnre_stream_t stream;
    if (argc != 7 || !read_entry(args[0], &fn) || !read_entry(args[1], &cache) || !THPVariable_Check(args[3]))
      Py_RETURN_NONE;
    const int64_t n = THPVariable_Unpack(args[3]).numel();
    if (n > INT_MAX || !read_pointer(args[3], 3, {n}, &first) || !read_pointer(args[4], 3, {n}, &second) ||
        !on_device({args[2], args[3], args[4]}))
      Py_RETURN_NONE;
    if (!read_stream(args[5], args[6], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_cache_truncate)>(fn)(static_cast<const qnre_cache_t*>(cache), first, second,
                                                              static_cast<int>(n), stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// compact(fn, cache address, its k, rows, path, counts, reader, stream)
PyObject* compact(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache;
    int32_t *rows, *path, *counts;
    qnre_stream_t stream;
    if (argc != 8 || !read_entry(args[0], &fn) || !read_entry(args[1], &cache) || !THPVariable_Check(args[3]) ||
        !THPVariable_Check(args[4]))
      Py_RETURN_NONE;
    const int64_t n = THPVariable_Unpack(args[3]).numel();
    const at::IntArrayRef shape = THPVariable_Unpack(args[4]).sizes();
    if (n > INT_MAX || shape.size() != 2 || shape[1] > INT_MAX || !read_pointer(args[3], 3, {n}, &rows) ||
        !read_pointer(args[4], 3, {n, shape[1]}, &path) || !read_pointer(args[5], 3, {n}, &counts) ||
        !on_device({args[2], args[3], args[4], args[5]}))
      Py_RETURN_NONE;
    if (!read_stream(args[6], args[7], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_cache_compact)>(fn)(static_cast<const qnre_cache_t*>(cache), rows, path, counts,
                                                             static_cast<int>(n), static_cast<int>(shape[1]), stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// A list of group starts and one entry a group, or None for both.
bool read_groups(PyObject* starts, PyObject* entries, int32_t** groups, int* n_groups, int32_t** shared) {
  *groups = *shared = nullptr;
  *n_groups = 0;
  if (starts == Py_None && entries == Py_None) return true;
  if (!THPVariable_Check(entries)) return false;
  const int64_t count = THPVariable_Unpack(entries).numel();
  if (count >= INT_MAX || !read_pointer(starts, 3, {count + 1}, groups) || !read_pointer(entries, 3, {count}, shared))
    return false;
  *n_groups = static_cast<int>(count);
  return true;
}

// shared_prefix(fn, cache address, its k, rows, groups, shared, reader, stream)
PyObject* shared_prefix(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache;
    int32_t *rows, *groups, *shared;
    int n_groups;
    qnre_stream_t stream;
    if (argc != 8 || !read_entry(args[0], &fn) || !read_entry(args[1], &cache) || !THPVariable_Check(args[3]))
      Py_RETURN_NONE;
    const int64_t n = THPVariable_Unpack(args[3]).numel();
    if (n > INT_MAX || !read_pointer(args[3], 3, {n}, &rows) || args[4] == Py_None ||
        !read_groups(args[4], args[5], &groups, &n_groups, &shared) || !on_device({args[2], args[3], args[4], args[5]}))
      Py_RETURN_NONE;
    if (!read_stream(args[6], args[7], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_cache_shared_prefix)>(fn)(static_cast<const qnre_cache_t*>(cache), rows,
                                                                   static_cast<int>(n), groups, n_groups, shared, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// prefix_attention(fn, q, cache address, its k, layer, rows, groups, shared, mask, out, lse, counts, depths, scale, softcap,
// slopes, workspace, reader, stream)
PyObject* prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void *fn, *cache, *out;
    qnre_tensor4_t q;
    int layer, n_groups;
    int32_t *rows, *groups, *shared, *counts = nullptr, *depths = nullptr;
    uint64_t* mask = nullptr;
    float *lse = nullptr, *slopes = nullptr;
    qnre_stream_t stream;
    if (argc != 19 || !read_entry(args[0], &fn) || !read_view4(args[1], &q) || !read_entry(args[2], &cache) ||
        !read_int(args[4], &layer) || !read_pointer(args[5], 3, {q.shape[0]}, &rows) ||
        !read_groups(args[6], args[7], &groups, &n_groups, &shared) ||
        (args[8] != Py_None && !read_pointer(args[8], 4, {q.shape[0], q.shape[1]}, &mask)) ||
        !read_pointer(args[9], q.dtype, {q.shape[0], q.shape[1], q.shape[2], q.shape[3]}, &out) ||
        (args[10] != Py_None &&
         !read_pointer(args[10], QNRE_DTYPE_FP32, {q.shape[0], q.shape[1], q.shape[2]}, &lse)) ||
        (args[11] != Py_None && !read_pointer(args[11], 3, {q.shape[0]}, &counts)) ||
        (args[12] != Py_None && !read_pointer(args[12], 3, {q.shape[0], q.shape[1]}, &depths)) ||
        (args[13] != Py_None && !PyFloat_Check(args[13])) || !PyFloat_Check(args[14]) ||
        (args[15] != Py_None && !read_pointer(args[15], QNRE_DTYPE_FP32, {q.shape[2]}, &slopes)) ||
        !THPVariable_Check(args[16]) ||
        !on_device({args[1], args[3], args[5], args[6], args[7], args[8], args[9], args[10], args[11], args[12], args[15],
                    args[16]}))
      Py_RETURN_NONE;
    const double scale =
        args[13] == Py_None ? std::pow(static_cast<double>(q.shape[3]), -0.5) : PyFloat_AS_DOUBLE(args[13]);
    const at::Tensor& ws = THPVariable_Unpack(args[16]);
    if (!ws.is_contiguous()) Py_RETURN_NONE;
    void* ws_data = ws.data_ptr();
    const uint64_t ws_bytes = ws.nbytes();
    const float softcap = static_cast<float>(PyFloat_AS_DOUBLE(args[14]));
    if (!read_stream(args[17], args[18], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_prefix_attention)>(fn)(
        &q, static_cast<const qnre_cache_t*>(cache), layer, rows, groups, n_groups, shared, mask, depths, counts,
        static_cast<float>(scale), softcap, slopes, out, lse, ws_data, ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

bool read_double(PyObject* obj, double* out) {
  if (PyFloat_Check(obj)) {
    *out = PyFloat_AS_DOUBLE(obj);
    return true;
  }
  if (!PyLong_Check(obj)) return false;
  *out = PyLong_AsDouble(obj);
  const bool read = PyErr_Occurred() == nullptr;
  if (!read) PyErr_Clear();
  return read;
}

// rope_table(fn, cos_sin, theta, first, kind, factor, original, low, high, magnitude, reader, stream)
PyObject* rope_table(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void* fn;
    float* out;
    double theta;
    int first;
    qnre_rope_scaling_t s;
    qnre_stream_t stream;
    if (argc != 12 || !read_entry(args[0], &fn) || !THPVariable_Check(args[1])) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(args[1]);
    if (t.dim() != 2 || t.size(1) > INT_MAX || !read_pointer(args[1], QNRE_DTYPE_FP32, {t.size(0), t.size(1)}, &out) ||
        !read_double(args[2], &theta) || !read_int(args[3], &first) || !read_int(args[4], &s.kind) ||
        !read_double(args[5], &s.factor) || !read_double(args[6], &s.original) || !read_double(args[7], &s.low) ||
        !read_double(args[8], &s.high) || !read_double(args[9], &s.magnitude) || !on_device({args[1]}))
      Py_RETURN_NONE;
    const int64_t n_pos = t.size(0);
    const int rot = static_cast<int>(t.size(1));
    if (!read_stream(args[10], args[11], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_rope_table)>(fn)(out, n_pos, rot, first, theta, &s, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// Logits with `rank` axes, each row contiguous, and the settings of its requests: five arguments.
struct Logits {
  const void* data;
  int64_t shape[3], stride[3];
  int dtype;
  float *temperature = nullptr, *top_p = nullptr, *min_p = nullptr;
  int32_t* top_k = nullptr;
};

bool read_logits(PyObject* obj, PyObject* const* settings, int rank, Logits* g) {
  if (!THPVariable_Check(obj)) return false;
  const at::Tensor& t = THPVariable_Unpack(obj);
  g->dtype = code_of(t);
  if (t.dim() != rank || g->dtype < 0 || g->dtype > QNRE_DTYPE_FP32) return false;
  for (int i = 0; i < rank; ++i) {
    g->shape[i] = t.size(i);
    g->stride[i] = t.stride(i);
  }
  if (g->stride[rank - 1] != 1 && g->shape[rank - 1] > 1) return false;
  g->data = t.data_ptr();
  const int64_t n = g->shape[0];
  return n <= INT_MAX && (settings[0] == Py_None || read_pointer(settings[0], QNRE_DTYPE_FP32, {n}, &g->temperature)) &&
         (settings[1] == Py_None || read_pointer(settings[1], 3, {n}, &g->top_k)) &&
         (settings[2] == Py_None || read_pointer(settings[2], QNRE_DTYPE_FP32, {n}, &g->top_p)) &&
         (settings[3] == Py_None || read_pointer(settings[3], QNRE_DTYPE_FP32, {n}, &g->min_p));
}

// sample(fn, logits, u, tokens, temperature, top_k, top_p, min_p, reader, stream)
PyObject* sample(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void* fn;
    Logits g;
    float* u;
    int32_t* tokens;
    qnre_stream_t stream;
    if (argc != 10 || !read_entry(args[0], &fn) || !read_logits(args[1], args + 4, 2, &g) ||
        !read_pointer(args[2], QNRE_DTYPE_FP32, {g.shape[0]}, &u) || !read_pointer(args[3], 3, {g.shape[0]}, &tokens) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6], args[7]}))
      Py_RETURN_NONE;
    if (!read_stream(args[8], args[9], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_sample)>(fn)(g.data, g.stride[0], g.dtype, static_cast<int>(g.shape[0]), g.shape[1],
                                                      g.temperature, g.top_k, g.top_p, g.min_p, u, tokens, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// filter(fn, logits, probs, temperature, top_k, top_p, min_p, reader, stream)
PyObject* filter(PyObject*, PyObject* const* args, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    void* fn;
    Logits g;
    float* probs;
    qnre_stream_t stream;
    if (argc != 9 || !read_entry(args[0], &fn) || !read_logits(args[1], args + 3, 3, &g) || g.shape[1] > INT_MAX ||
        !read_pointer(args[2], QNRE_DTYPE_FP32, {g.shape[0], g.shape[1], g.shape[2]}, &probs) ||
        !on_device({args[1], args[2], args[3], args[4], args[5], args[6]}))
      Py_RETURN_NONE;
    if (!read_stream(args[7], args[8], &stream)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = reinterpret_cast<decltype(&qnre_filter_probs)>(fn)(g.data, g.stride[0], g.stride[1], g.dtype,
                                                            static_cast<int>(g.shape[0]), static_cast<int>(g.shape[1]),
                                                            g.shape[2], g.temperature, g.top_k, g.top_p, g.min_p, probs,
                                                            stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"view4", view4, METH_O, nullptr},
                         {"pointer", fast(pointer), METH_FASTCALL, nullptr},
                         {"norm", fast(norm), METH_FASTCALL, nullptr},
                         {"norm_backward", fast(norm_backward), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"attention", fast(attention), METH_FASTCALL, nullptr},
                         {"verify", fast(verify), METH_FASTCALL, nullptr},
                         {"cache_rows", fast(cache_rows), METH_FASTCALL, nullptr},
                         {"compact", fast(compact), METH_FASTCALL, nullptr},
                         {"shared_prefix", fast(shared_prefix), METH_FASTCALL, nullptr},
                         {"prefix_attention", fast(prefix_attention), METH_FASTCALL, nullptr},
                         {"rope_table", fast(rope_table), METH_FASTCALL, nullptr},
                         {"sample", fast(sample), METH_FASTCALL, nullptr},
                         {"filter", fast(filter), METH_FASTCALL, nullptr},
                         {"sizes", sizes, METH_O, nullptr},
                         {"type_code", type_code, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
