// tensors.cpp -- the calls a decode loop makes every few microseconds, as a
// CPython extension: a dozen tensors' type, device, shape and layout are looked
// at and the library is called within a microsecond or two, where Python and
// ctypes take six.  Each function returns the library's status, or None when a
// tensor is not as the call wants it; the caller then finds out which and
// raises.  What torch throws here (for a tensor without storage, as a transform
// hands out, or of a layout without strides) becomes a Python exception.  On one
// GB300's host a call of rope_kv_append for one verify block takes the calling
// thread 3.6 us, most of it the launch (8.8 us when the checks returned
// addresses to Python and ctypes made the call).
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "specverify.h"

namespace {

decltype(&kv_pages_step) pages_fn = nullptr;
decltype(&rope_kv_append) append_fn = nullptr;
decltype(&paged_attention) attend_fn = nullptr;
decltype(&gdn_inputs) inputs_fn = nullptr;
decltype(&gdn_advance) advance_fn = nullptr;
decltype(&moe_smallm) experts_fn = nullptr;

// What a call's arguments are read with.  `fits` turns false at the first
// tensor that is not as wanted; later reads of that call then give null.
struct Reader {
  PyObject *const *args;
  long index;        // the device that all tensors are on
  bool fits = true;

  const at::Tensor *tensor(int i) {
    if (!fits) return nullptr;
    if (THPVariable_Check(args[i])) {
      const at::Tensor &x = THPVariable_Unpack(args[i]);
      if (x.is_cuda() && x.get_device() == index) return &x;
    }
    fits = false;
    return nullptr;
  }
  const at::Tensor *dense(int i, at::ScalarType type) {
    const at::Tensor *x = tensor(i);
    if (x && (x->scalar_type() != type || !x->is_contiguous())) fits = false;
    return fits ? x : nullptr;
  }
  // The address of a contiguous tensor of this type and shape.
  template <class T>
  T *at(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor *x = dense(i, type);
    if (x && x->sizes() != at::IntArrayRef(shape)) fits = false;
    return fits ? static_cast<T *>(const_cast<void *>(x->const_data_ptr())) : nullptr;
  }
  // The same, of any shape: its values are counted.
  template <class T>
  T *any(int i, at::ScalarType type, int64_t *count) {
    const at::Tensor *x = dense(i, type);
    if (!fits) return nullptr;
    *count = x->numel();
    return static_cast<T *>(const_cast<void *>(x->const_data_ptr()));
  }
  // Packed rows [rows, heads, dim] with contiguous heads: address, row stride.
  template <class T>
  T *rows(int i, at::ScalarType type, int64_t n, int64_t heads, int64_t dim, long long *stride) {
    const at::Tensor *x = tensor(i);
    if (!x || x->scalar_type() != type || x->dim() != 3 || x->size(0) != n ||
        x->size(1) != heads || x->size(2) != dim || x->stride(2) != 1 ||
        (heads > 1 && x->stride(1) != dim)) {
      fits = false;
      return nullptr;
    }
    *stride = n > 1 ? x->stride(0) : heads * dim;
    return static_cast<T *>(const_cast<void *>(x->const_data_ptr()));
  }
  // Rows of numbers [rows, width]: address, row stride.
  const void *rows(int i, at::ScalarType type, int64_t n, int64_t width, long long *stride) {
    const at::Tensor *x = tensor(i);
    if (!x || x->scalar_type() != type || x->dim() != 2 || x->size(0) != n ||
        x->size(1) != width || (width > 1 && x->stride(1) != 1)) {
      fits = false;
      return nullptr;
    }
    *stride = n > 1 ? x->stride(0) : width;
    return x->const_data_ptr();
  }
  bool given(int i) const { return args[i] != Py_None; }
};

// Whole numbers go to the library as int; one that does not fit is refused, not
// cut off.
bool to_int(int64_t v, int *out) {
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "a size or number does not fit 31 bits");
    return false;
  }
  *out = (int)v;
  return true;
}
bool to_int(PyObject *o, int *out) {
  const long long v = PyLong_AsLongLong(o);
  return !(v == -1 && PyErr_Occurred()) && to_int((int64_t)v, out);
}
bool begin(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, Reader *r, sv_stream_t *stream) {
  if (n != want || !pages_fn) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or no library");
    return false;
  }
  const unsigned long long s = PyLong_AsUnsignedLongLong(args[1]);
  *stream = reinterpret_cast<sv_stream_t>((uintptr_t)s);
  *r = Reader{args, PyLong_AsLong(args[0])};
  return !PyErr_Occurred();
}
// The library is called without the interpreter's lock, held again on any way out.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
PyObject *call(F library) {
  sv_status st;
  {
    const Unlocked unlocked;
    st = library();
  }
  return PyLong_FromLong(st);
}

// bind(kv_pages_step, rope_kv_append, paged_attention, gdn_inputs, gdn_advance, moe_smallm):
// the library's addresses
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  constexpr int kCalls = 6;
  void *at[kCalls] = {};
  for (int i = 0; i < kCalls && n == kCalls; ++i) at[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  pages_fn = reinterpret_cast<decltype(pages_fn)>(at[0]);
  append_fn = reinterpret_cast<decltype(append_fn)>(at[1]);
  attend_fn = reinterpret_cast<decltype(attend_fn)>(at[2]);
  inputs_fn = reinterpret_cast<decltype(inputs_fn)>(at[3]);
  advance_fn = reinterpret_cast<decltype(advance_fn)>(at[4]);
  experts_fn = reinterpret_cast<decltype(experts_fn)>(at[5]);
  Py_RETURN_NONE;
}

// kv_pages_step(device, stream, length, held, cursor, ring, block_table, n_new, n_commit or
// None, n_commit_bias, page_size, rows, length_out, held_out, cursor_out, q_start, kv_len,
// slots, positions, err_flags)
PyObject *pages(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 20, &r, &stream)) return nullptr;
  int bias, page_size, rows, B, max_pages, ring_n, commits_n;
  if (!to_int(args[9], &bias) || !to_int(args[10], &page_size) || !to_int(args[11], &rows))
    return nullptr;
  const auto i32 = at::kInt;
  const at::Tensor *table = r.dense(6, i32);
  if (!table || table->dim() != 2) Py_RETURN_NONE;
  const int64_t b = table->size(0), each = rows > 0 ? rows : 0;
  int64_t in_ring = 0, commits = 0, entries;
  using I = int32_t;
  I *length = r.at<I>(2, i32, {b}), *held = r.at<I>(3, i32, {b}), *cursor = r.at<I>(4, i32, {2}),
    *ring = r.any<I>(5, i32, &in_ring), *pages = r.any<I>(6, i32, &entries),
    *n_new = r.at<I>(7, i32, {b});
  I *n_commit = r.given(8) ? r.any<I>(8, i32, &commits) : nullptr;
  I *length_out = r.at<I>(12, i32, {b}), *held_out = r.at<I>(13, i32, {b}),
    *cursor_out = r.at<I>(14, i32, {2}), *q_start = r.at<I>(15, i32, {b + 1}),
    *kv_len = r.at<I>(16, i32, {b}), *slots = r.at<I>(17, i32, {each}),
    *positions = r.at<I>(18, i32, {each}), *flags = r.at<I>(19, i32, {b});
  if (!r.fits) Py_RETURN_NONE;
  if (!to_int(b, &B) || !to_int(table->size(1), &max_pages) || !to_int(in_ring, &ring_n) ||
      !to_int(commits, &commits_n))
    return nullptr;
  return call([&] {
    return pages_fn(length, held, cursor, n_new, n_commit, commits_n, bias, B, page_size,
                    max_pages, ring_n, rows, pages, ring, length_out, held_out, cursor_out,
                    q_start, kv_len, slots, positions, flags, stream);
  });
  END_HANDLE_TH_ERRORS
}

// rope_kv_append(device, stream, q, k, v, positions, slots, freqs or None, k_cache, v_cache,
// axis, q_weight, k_weight (each or None), eps, interleaved, q_out)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 16, &r, &stream)) return nullptr;
  const double eps = PyFloat_AsDouble(args[13]);
  const int interleaved = PyObject_IsTrue(args[14]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *q = r.tensor(2), *cache = r.tensor(8), *positions = r.tensor(5);
  if (!r.fits || q->dim() != 3 || cache->dim() != 4 || positions->dim() < 1 ||
      positions->dim() > 2)
    Py_RETURN_NONE;
  const auto type = q->scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
  const int64_t rows = q->size(0), hq = q->size(1), d = q->size(2);
  const int64_t pages = cache->size(0), hkv = cache->size(1), page = cache->size(2);
  const int64_t axes = positions->dim() == 1 ? 1 : positions->size(1);
  long long qs = 0, ks = 0, vs = 0;
  const void *q_at = r.rows<void>(2, type, rows, hq, d, &qs);
  const void *k_at = r.rows<void>(3, type, rows, hkv, d, &ks);
  const void *v_at = r.rows<void>(4, type, rows, hkv, d, &vs);
  const int32_t *pos_at = positions->dim() == 1 ? r.at<int32_t>(5, at::kInt, {rows})
                                                : r.at<int32_t>(5, at::kInt, {rows, axes});
  const int32_t *slots = r.at<int32_t>(6, at::kInt, {rows});
  int64_t half = 0;
  const uint64_t *freqs = nullptr;
  if (r.given(7)) {
    const at::Tensor *f = r.tensor(7);
    if (!f || f->dim() != 1) Py_RETURN_NONE;
    freqs = r.any<uint64_t>(7, at::kLong, &half);
  }
  auto *kc = r.at<uint16_t>(8, at::kBFloat16, {pages, hkv, page, d});
  auto *vc = r.at<uint16_t>(9, at::kBFloat16, {pages, hkv, page, d});
  const auto *axis = r.given(10) ? r.at<uint8_t>(10, at::kByte, {half}) : nullptr;
  const auto *qw = r.given(11) ? r.at<float>(11, at::kFloat, {d}) : nullptr;
  const auto *kw = r.given(12) ? r.at<float>(12, at::kFloat, {d}) : nullptr;
  auto *q_out = r.at<uint16_t>(15, at::kBFloat16, {rows, hq, d});
  if (!r.fits) Py_RETURN_NONE;
  int v[8];
  const int64_t sizes[8] = {axes, rows, hq, hkv, d, 2 * half, page, pages};
  for (int i = 0; i < 8; ++i)
    if (!to_int(sizes[i], &v[i])) return nullptr;
  return call([&] {
    return append_fn(q_at, k_at, v_at, type == at::kBFloat16 ? SV_BF16 : SV_F32, qs, ks, vs,
                     pos_at, v[0], slots, freqs, axis, qw, kw, (float)eps, v[1], v[2], v[3],
                     v[4], v[5], interleaved, v[6], v[7], q_out, kc, vc, stream);
  });
  END_HANDLE_TH_ERRORS
}

// paged_attention(device, stream, q, k_cache, v_cache, block_table, q_start, kv_len, max_new,
// scale or None for 1 / sqrt(D), window, out, lse or None, workspace)
PyObject *attend(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 14, &r, &stream)) return nullptr;
  int max_new, window;
  if (!to_int(args[8], &max_new) || !to_int(args[10], &window)) return nullptr;
  double scale = r.given(9) ? PyFloat_AsDouble(args[9]) : 0.0;
  if (PyErr_Occurred()) return nullptr;
  const auto bf16 = at::kBFloat16;
  const at::Tensor *q = r.tensor(2), *cache = r.tensor(3), *table = r.tensor(5);
  if (!r.fits || q->dim() != 3 || cache->dim() != 4 || table->dim() != 2) Py_RETURN_NONE;
  const int64_t rows = q->size(0), hq = q->size(1), d = q->size(2), b = table->size(0);
  const int64_t pages = cache->size(0), hkv = cache->size(1), page = cache->size(2);
  if (!r.given(9)) scale = 1.0 / std::sqrt((double)d);
  long long qs = 0, outs = 0;
  int64_t entries, bytes = 0;
  const auto *q_at = r.rows<uint16_t>(2, bf16, rows, hq, d, &qs);
  const auto *kc = r.at<uint16_t>(3, bf16, {pages, hkv, page, d});
  const auto *vc = r.at<uint16_t>(4, bf16, {pages, hkv, page, d});
  const auto *table_at = r.any<int32_t>(5, at::kInt, &entries);
  const auto *q_start = r.at<int32_t>(6, at::kInt, {b + 1});
  const auto *kv_len = r.at<int32_t>(7, at::kInt, {b});
  auto *out = r.rows<uint16_t>(11, bf16, rows, hq, d, &outs);
  auto *lse = r.given(12) ? r.at<float>(12, at::kFloat, {rows, hq}) : nullptr;
  auto *workspace = r.any<uint8_t>(13, at::kByte, &bytes);
  if (!r.fits) Py_RETURN_NONE;
  int v[8];
  const int64_t sizes[8] = {b, rows, hq, hkv, d, page, pages, table->size(1)};
  for (int i = 0; i < 8; ++i)
    if (!to_int(sizes[i], &v[i])) return nullptr;
  return call([&] {
    return attend_fn(q_at, qs, kc, vc, table_at, q_start, kv_len, v[0], v[1], max_new, v[2],
                     v[3], v[4], v[5], v[6], v[7], (float)scale, window, out, outs, lse,
                     workspace, (size_t)bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

// gdn_inputs(device, stream, x, a, b, weight, window, a_log, dt_bias, q_start, window_index or
// None, max_new, update_window, q_scale, eps, q, k, v, alpha, beta)
PyObject *inputs(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 20, &r, &stream)) return nullptr;
  int max_new;
  if (!to_int(args[11], &max_new)) return nullptr;
  const int update = PyObject_IsTrue(args[12]);
  const double scale = PyFloat_AsDouble(args[13]), eps = PyFloat_AsDouble(args[14]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *x = r.tensor(2), *a = r.tensor(3), *weight = r.tensor(5), *window = r.tensor(6),
                   *start = r.tensor(9), *q = r.tensor(15), *v = r.tensor(17);
  if (!r.fits || x->dim() != 2 || a->dim() != 2 || weight->dim() != 2 || window->dim() != 3 ||
      start->dim() != 1 || q->dim() != 3 || v->dim() != 3)
    Py_RETURN_NONE;
  const auto type = x->scalar_type(), to = q->scalar_type(), f32 = at::kFloat;
  if ((type != f32 && type != at::kBFloat16) || (to != f32 && to != at::kBFloat16)) Py_RETURN_NONE;
  const int64_t rows = x->size(0), c = x->size(1), hv = a->size(1), w = weight->size(0),
                slots = window->size(0), b = start->size(0) - 1, hk = q->size(1), dk = q->size(2),
                dv = v->size(2);
  if (b < 0 || c != 2 * hk * dk + hv * dv) Py_RETURN_NONE;
  long long xs = 0, as = 0, bs = 0;
  const void *x_at = r.rows(2, type, rows, c, &xs), *a_at = r.rows(3, type, rows, hv, &as),
             *b_at = r.rows(4, type, rows, hv, &bs);
  const auto *w_at = r.at<float>(5, f32, {w, c});
  auto *win = r.at<float>(6, f32, {slots, w - 1, c});
  const auto *a_log = r.at<float>(7, f32, {hv}), *dt = r.at<float>(8, f32, {hv});
  const auto *q_start = r.at<int32_t>(9, at::kInt, {b + 1});
  const auto *index = r.given(10) ? r.at<int32_t>(10, at::kInt, {b}) : nullptr;
  void *q_at = r.at<void>(15, to, {rows, hk, dk}), *k_at = r.at<void>(16, to, {rows, hk, dk}),
       *v_at = r.at<void>(17, to, {rows, hv, dv});
  auto *al = r.at<float>(18, f32, {rows, hv}), *be = r.at<float>(19, f32, {rows, hv});
  if (!r.fits) Py_RETURN_NONE;
  int s[8];
  const int64_t sizes[8] = {b, rows, slots, w, hk, hv, dk, dv};
  for (int i = 0; i < 8; ++i)
    if (!to_int(sizes[i], &s[i])) return nullptr;
  return call([&] {
    return inputs_fn(x_at, a_at, b_at, type == f32 ? SV_F32 : SV_BF16, xs, as, bs, w_at, win,
                     a_log, dt, q_start, index, s[0], s[1], max_new, s[2], s[3], s[4], s[5], s[6],
                     s[7], update, (float)scale, (float)eps, to == f32 ? SV_F32 : SV_BF16, q_at,
                     k_at, v_at, al, be, stream);
  });
  END_HANDLE_TH_ERRORS
}

// gdn_advance(device, stream, q, k, v, alpha, beta, state, q_start, state_index or None, max_new,
// out, workspace or None)
PyObject *advance(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 13, &r, &stream)) return nullptr;
  int max_new;
  if (!to_int(args[10], &max_new)) return nullptr;
  const at::Tensor *q = r.tensor(2), *state = r.tensor(7), *start = r.tensor(8);
  if (!r.fits || q->dim() != 3 || state->dim() != 4 || start->dim() != 1) Py_RETURN_NONE;
  const auto type = q->scalar_type(), f32 = at::kFloat;
  if (type != f32 && type != at::kBFloat16) Py_RETURN_NONE;
  const int64_t rows = q->size(0), hk = q->size(1), dk = q->size(2), b = start->size(0) - 1,
                slots = state->size(0), hv = state->size(1), dv = state->size(2);
  if (b < 0) Py_RETURN_NONE;
  long long qs = 0, ks = 0, vs = 0, os = 0;
  const void *q_at = r.rows<void>(2, type, rows, hk, dk, &qs);
  const void *k_at = r.rows<void>(3, type, rows, hk, dk, &ks);
  const void *v_at = r.rows<void>(4, type, rows, hv, dv, &vs);
  const auto *al = r.at<float>(5, f32, {rows, hv}), *be = r.at<float>(6, f32, {rows, hv});
  auto *state_at = r.at<float>(7, f32, {slots, hv, dv, dk});
  const auto *q_start = r.at<int32_t>(8, at::kInt, {b + 1});
  const auto *index = r.given(9) ? r.at<int32_t>(9, at::kInt, {b}) : nullptr;
  void *out = r.rows<void>(11, type, rows, hv, dv, &os);
  int64_t bytes = 0;
  void *workspace = r.given(12) ? r.any<void>(12, at::kByte, &bytes) : nullptr;
  if (!r.fits) Py_RETURN_NONE;
  int s[7];
  const int64_t sizes[7] = {b, rows, slots, hk, hv, dk, dv};
  for (int i = 0; i < 7; ++i)
    if (!to_int(sizes[i], &s[i])) return nullptr;
  return call([&] {
    return advance_fn(q_at, k_at, v_at, type == f32 ? SV_F32 : SV_BF16, qs, ks, vs, al, be,
                      state_at, q_start, index, s[0], s[1], max_new, s[2], s[3], s[4], s[5], s[6],
                      out, os, workspace, (size_t)bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

// moe_smallm(device, stream, x, router, gate w, s, b, up w, s, b, down w, s, b, top_k,
// renormalize, out, ids or None, weights or None, workspace)
PyObject *experts(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Reader r;
  sv_stream_t stream;
  if (!begin(args, n, 19, &r, &stream)) return nullptr;
  int top;
  if (!to_int(args[13], &top)) return nullptr;
  const int renormalize = PyObject_IsTrue(args[14]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *x = r.tensor(2), *gate = r.tensor(4);
  if (!r.fits || x->dim() != 2 || gate->dim() != 3) Py_RETURN_NONE;
  const auto bf16 = at::kBFloat16;
  const int64_t rows = x->size(0), hidden = x->size(1), e = gate->size(0), inter = gate->size(1);
  const auto *x_at = r.at<uint16_t>(2, bf16, {rows, hidden});
  const auto *router = r.at<uint16_t>(3, bf16, {e, hidden});
  const uint32_t *w[3];
  const uint16_t *s[3], *b[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t out = i < 2 ? inter : hidden, in = i < 2 ? hidden : inter;
    w[i] = r.at<uint32_t>(4 + 3 * i, at::kInt, {e, out, in / 8});
    s[i] = r.at<uint16_t>(5 + 3 * i, bf16, {e, out, in / 64});
    b[i] = r.at<uint16_t>(6 + 3 * i, bf16, {e, out, in / 64});
  }
  auto *y = r.at<uint16_t>(15, bf16, {rows, hidden});
  auto *ids = r.given(16) ? r.at<int32_t>(16, at::kInt, {rows, top}) : nullptr;
  auto *weights = r.given(17) ? r.at<float>(17, at::kFloat, {rows, top}) : nullptr;
  int64_t bytes = 0;
  void *workspace = r.any<void>(18, at::kByte, &bytes);
  if (!r.fits) Py_RETURN_NONE;
  int v[4];
  const int64_t sizes[4] = {rows, hidden, inter, e};
  for (int i = 0; i < 4; ++i)
    if (!to_int(sizes[i], &v[i])) return nullptr;
  return call([&] {
    return experts_fn(x_at, router, w[0], s[0], b[0], w[1], s[1], b[1], w[2], s[2], b[2], v[0],
                      v[1], v[2], v[3], top, renormalize, y, ids, weights, workspace,
                      (size_t)bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

#define METHOD(name, function) \
  {name, (PyCFunction)(void *)function, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("bind", bind), METHOD("kv_pages_step", pages),
                         METHOD("rope_kv_append", append), METHOD("paged_attention", attend),
                         METHOD("gdn_inputs", inputs), METHOD("gdn_advance", advance),
                         METHOD("moe_smallm", experts),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
