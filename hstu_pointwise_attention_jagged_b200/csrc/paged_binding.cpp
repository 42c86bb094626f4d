// paged_binding.cpp — Python binding of include/hstu_paged.h: the module _paged_native.
//
// Argument marshalling only: every function checks the torch tensors it is given, passes pointers,
// sizes, strides and the current CUDA stream to the C entry point of the same name, and raises
// HstuError on a non-zero status.  It does in C++ what binding.py does in Python, because a call for a few
// rows takes the GPU about three microseconds and the same checks in Python took 13 to 16.  The entry
// points' addresses come from paged.load_library(), which loads libhstu_attn.so; this module does not link it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstring>
#include <optional>
#include <utility>

#include "hstu_paged.h"

namespace {

decltype(&hstu_rotary) g_rotary = nullptr;
decltype(&hstu_paged_append) g_append = nullptr;
decltype(&hstu_paged_attn_fwd) g_attn = nullptr;
decltype(&hstu_paged_selfcheck_fwd_timeout) g_selfcheck = nullptr;
PyObject* g_error = nullptr;  // HstuError

// A Python exception is set; unwinds to the function's entry.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised();
}

// ---------------------------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------------------------
// Places positional and keyword arguments by name; absent ones are null.  The first `required` must be there.
template <size_t kCount>
void place(const char* fn, const char* const (&names)[kCount], size_t required, PyObject* const* args, Py_ssize_t nargs,
           PyObject* kwnames, PyObject* (&out)[kCount]) {
  if (nargs > static_cast<Py_ssize_t>(kCount)) raise(PyExc_TypeError, "%s takes at most %d arguments", fn, (int)kCount);
  for (size_t i = 0; i < kCount; ++i) out[i] = i < static_cast<size_t>(nargs) ? args[i] : nullptr;
  const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < nkw; ++k) {
    PyObject* name = PyTuple_GET_ITEM(kwnames, k);
    size_t i = 0;
    while (i < kCount && PyUnicode_CompareWithASCIIString(name, names[i]) != 0) ++i;
    if (i == kCount) raise(PyExc_TypeError, "%s got an unexpected keyword argument '%U'", fn, name);
    if (out[i]) raise(PyExc_TypeError, "%s got multiple values for argument '%s'", fn, names[i]);
    out[i] = args[nargs + k];
  }
  for (size_t i = 0; i < required; ++i)
    if (!out[i]) raise(PyExc_TypeError, "%s missing required argument: '%s'", fn, names[i]);
}

bool given(PyObject* o) { return o && o != Py_None; }

bool flag(PyObject* o) {
  if (!o) return false;
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

int32_t int32_of(const char* name, PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised();
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &overflow);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (overflow || v > INT32_MAX || v < INT32_MIN) raise(PyExc_ValueError, "%s does not fit 32 bits", name);
  return static_cast<int32_t>(v);
}

float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

const at::Tensor& tensor_of(const char* name, PyObject* o, const char* want) {
  if (!o || !THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be %s", name, want);
  return THPVariable_Unpack(o);
}

bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

const void* address(const at::Tensor& t) { return t.const_data_ptr(); }

// A token tensor: bf16 [rows, H, d], heads packed.
struct Rows {
  const void* p = nullptr;
  int64_t ld = 0;
  int64_t rows = 0, H = 0, d = 0;
  int device = -1;
};

Rows rows_of(const char* name, PyObject* o, const Rows* like = nullptr) {
  const char* want = "a bf16 CUDA tensor [rows, H, d]";
  const at::Tensor& t = tensor_of(name, o, want);
  if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.layout() != at::kStrided)
    raise(PyExc_TypeError, "%s must be %s", name, want);
  Rows r;
  r.rows = t.size(0);
  r.H = t.size(1);
  r.d = t.size(2);
  r.device = t.get_device();
  if (like) {
    if (r.rows != like->rows || r.H != like->H || r.d != like->d)
      raise(PyExc_ValueError, "%s has shape (%lld, %lld, %lld), expected (%lld, %lld, %lld)", name, (long long)r.rows,
            (long long)r.H, (long long)r.d, (long long)like->rows, (long long)like->H, (long long)like->d);
    if (r.device != like->device) raise(PyExc_ValueError, "%s must be on cuda:%d", name, like->device);
  }
  if (r.rows > INT32_MAX || r.H > INT32_MAX || r.d > INT32_MAX) raise(PyExc_ValueError, "%s is too large", name);
  if (r.rows && ((r.d > 1 && t.stride(2) != 1) || (r.H > 1 && t.stride(1) != r.d)))
    raise(PyExc_TypeError, "%s must have its heads packed (only the row stride is free)", name);
  r.p = address(t);
  r.ld = r.rows > 1 ? t.stride(0) : r.H * r.d;  // the stride of a single row is never used
  return r;
}

const int32_t* index_of(const char* name, PyObject* o, int64_t n, int device) {
  const at::Tensor& t = tensor_of(name, o, "an int32 tensor");
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !on(t, device) || !t.is_contiguous())
    raise(PyExc_TypeError, "%s must be a contiguous int32 tensor of %lld elements on cuda:%d", name, (long long)n, device);
  return static_cast<const int32_t*>(address(t));
}

int32_t users_of(PyObject* q_offsets) {
  const at::Tensor& t = tensor_of("q_offsets", q_offsets, "an int32 vector");
  if (t.dim() != 1 || t.size(0) < 1 || t.size(0) > INT32_MAX)
    raise(PyExc_TypeError, "q_offsets must be an int32 vector of one element more than there are users");
  return static_cast<int32_t>(t.size(0) - 1);
}

hstu_rotation_t rotation_of(PyObject* freqs, PyObject* sections, PyObject* positions, PyObject* interleaved, int64_t rows,
                            int device, bool need_positions) {
  hstu_rotation_t r;
  std::memset(&r, 0, sizeof(r));
  const at::Tensor& f = tensor_of("freqs", freqs, "a float64 vector");
  if (f.scalar_type() != at::kDouble || f.dim() != 1 || !on(f, device) || !f.is_contiguous() || f.size(0) > INT32_MAX)
    raise(PyExc_TypeError, "freqs must be a contiguous float64 vector on cuda:%d", device);
  r.freqs = static_cast<const double*>(address(f));
  r.pairs = static_cast<int32_t>(f.size(0));
  r.axes = 1;
  r.sections[0] = r.pairs;
  if (given(sections)) {
    PyObject* seq = PySequence_Fast(sections, "sections must be a sequence of whole numbers");
    if (!seq) throw Raised();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    try {
      if (n < 1 || n > HSTU_MAX_AXES) raise(PyExc_ValueError, "1 to %d sections, got %zd", HSTU_MAX_AXES, n);
      r.axes = static_cast<int32_t>(n);
      for (Py_ssize_t i = 0; i < n; ++i) r.sections[i] = int32_of("sections", PySequence_Fast_GET_ITEM(seq, i));
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
    Py_DECREF(seq);
  }
  r.interleaved = flag(interleaved);
  if (!given(positions)) {
    if (need_positions) raise(PyExc_TypeError, "positions are required");
    return r;
  }
  const at::Tensor& p = tensor_of("positions", positions, "an int32 tensor");
  if (p.scalar_type() != at::kInt || !on(p, device))
    raise(PyExc_TypeError, "positions must be an int32 tensor on cuda:%d", device);
  if (!(p.dim() == 2 && p.size(0) == r.axes && p.size(1) == rows) && !(p.dim() == 1 && r.axes == 1 && p.size(0) == rows))
    raise(PyExc_ValueError, "positions must be [%d, %lld], one row for each axis", r.axes, (long long)rows);
  if (rows > 1 && p.stride(-1) != 1) raise(PyExc_TypeError, "positions of one axis must be contiguous");
  r.positions = static_cast<const int32_t*>(address(p));
  r.positions_ld = r.axes > 1 ? p.stride(0) : rows;
  return r;
}

hstu_paged_cache_t cache_of(PyObject* k_cache, PyObject* v_cache, PyObject* page_table, int32_t B, const Rows& rows) {
  const char* want = "a bf16 tensor [pages, page_size, H, d]";
  const at::Tensor &k = tensor_of("k_cache", k_cache, want), &v = tensor_of("v_cache", v_cache, want);
  if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 || k.dim() != 4 || v.dim() != 4 ||
      !on(k, rows.device) || !on(v, rows.device))
    raise(PyExc_TypeError, "k_cache and v_cache must be bf16 tensors [pages, page_size, H, d] on cuda:%d", rows.device);
  if (k.sizes() != v.sizes()) raise(PyExc_ValueError, "k_cache and v_cache must have the same shape");
  if (k.size(2) != rows.H || k.size(3) != rows.d)
    raise(PyExc_ValueError, "the cache holds [%lld, %lld] rows, the new rows are [%lld, %lld]", (long long)k.size(2),
          (long long)k.size(3), (long long)rows.H, (long long)rows.d);
  if (k.numel() == 0) raise(PyExc_ValueError, "the cache has no rows");
  if (k.size(0) > INT32_MAX || k.size(1) > INT32_MAX) raise(PyExc_ValueError, "the cache is too large");
  // The stride of a dimension of one entry is never used.
  int64_t strides[3];
  for (int i = 0; i < 4; ++i) {
    if (k.size(i) > 1 && k.stride(i) != v.stride(i))
      raise(PyExc_ValueError, "k_cache and v_cache must have the same strides");
    if (i < 3) strides[i] = k.size(i) > 1 ? k.stride(i) : rows.d;
    else if (k.size(i) > 1 && k.stride(i) != 1) raise(PyExc_TypeError, "the last dimension of the cache must be contiguous");
  }
  const at::Tensor& table = tensor_of("page_table", page_table, "an int32 tensor [users, pages of a user]");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || !on(table, rows.device) ||
      table.size(1) > INT32_MAX)
    raise(PyExc_TypeError, "page_table must be an int32 tensor [%d, pages of a user] on cuda:%d", B, rows.device);
  if (table.size(1) > 1 && table.stride(1) != 1)
    raise(PyExc_TypeError, "a user's entries of page_table must be contiguous");
  hstu_paged_cache_t c;
  c.k = const_cast<void*>(address(k));
  c.v = const_cast<void*>(address(v));
  c.page_stride = strides[0];
  c.row_stride = strides[1];
  c.head_stride = strides[2];
  c.num_pages = static_cast<int32_t>(k.size(0));
  c.page_size = static_cast<int32_t>(k.size(1));
  c.page_table = static_cast<const int32_t*>(address(table));
  c.table_width = static_cast<int32_t>(table.size(1));
  c.table_ld = B > 1 && c.table_width > 0 ? table.stride(0) : c.table_width;
  return c;
}

// ---------------------------------------------------------------------------------------------
// Calls
// ---------------------------------------------------------------------------------------------
// Runs `f`, which touches no Python object, without the interpreter's lock: an allocation or a launch may have
// to wait for the driver, and other threads go on meanwhile.
template <typename F>
auto unlocked(F&& f) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
}

// The call's device is current, and `stream` is the one given or the device's current one.
struct Place {
  std::optional<c10::cuda::CUDAGuard> guard;
  c10::cuda::CUDAStream stream;
  bool own_stream;  // one was given

  Place(int device, PyObject* given_stream) : stream(c10::cuda::getCurrentCUDAStream(device)), own_stream(false) {
    if (c10::cuda::current_device() != device) guard.emplace(static_cast<c10::DeviceIndex>(device));
    if (!given(given_stream)) return;
    PyObject* raw = PyObject_GetAttrString(given_stream, "cuda_stream");
    if (!raw) throw Raised();
    void* handle = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (!handle && PyErr_Occurred()) throw Raised();
    stream = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), static_cast<c10::DeviceIndex>(device));
    own_stream = true;
  }
};

// The output given as `o`, or a new packed one like `in`.  A new one belongs to the stream that the call
// runs on: memory of another stream might still be in use there.  Returns a new reference in `object`.
Rows output_of(const char* name, PyObject* o, const Rows& in, const Place& place, PyObject*& object) {
  if (given(o)) {
    const Rows r = rows_of(name, o, &in);
    Py_INCREF(o);
    object = o;
    return r;
  }
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  if (place.own_stream) guard.emplace(place.stream);
  at::Tensor t = unlocked([&]() -> at::Tensor {
    return at::detail::empty_cuda({in.rows, in.H, in.d}, at::kBFloat16,
                                  c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(in.device)), std::nullopt);
  });
  Rows r = in;
  r.p = address(t);
  r.ld = in.H * in.d;
  object = THPVariable_Wrap(std::move(t));
  if (!object) throw Raised();
  return r;
}

void check(hstu_status_t status, const char* where) {
  if (status == HSTU_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(status), where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

void need_library() {
  if (g_attn) return;
  PyObject* m = PyImport_ImportModule("hstu_pointwise_attention_jagged_b200.paged");
  PyObject* r = m ? PyObject_CallMethod(m, "load_library", nullptr) : nullptr;
  Py_XDECREF(m);
  Py_XDECREF(r);
  if (!r) throw Raised();
}

// Runs `body`, which returns a new reference, and turns C++ exceptions into Python's.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// A reference that an exception drops.
struct Held {
  PyObject* o = nullptr;
  ~Held() { Py_XDECREF(o); }
  PyObject* release() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q",           "k",       "positions", "freqs", "sections",
                                        "interleaved", "inverse", "q_out",     "k_out", "stream"};
    PyObject* a[10];
    place("hstu_rotary", names, 4, args, nargs, kwnames, a);
    need_library();
    const Rows q = rows_of("q", a[0]);
    Rows k, ko;
    if (given(a[1])) k = rows_of("k", a[1], &q);
    else if (given(a[8])) raise(PyExc_ValueError, "k_out without k");
    const hstu_rotation_t rot = rotation_of(a[3], a[4], a[2], a[5], q.rows, q.device, true);
    const bool inverse = flag(a[6]);
    const Place at(q.device, a[9]);
    Held out_q, out_k;
    const Rows qo = output_of("q_out", a[7], q, at, out_q.o);
    if (k.p || given(a[1])) ko = output_of("k_out", a[8], q, at, out_k.o);
    check(unlocked([&] {
            return g_rotary(q.p, q.ld, k.p, k.ld, &rot, inverse, static_cast<int32_t>(q.H), static_cast<int32_t>(q.d),
                            static_cast<int32_t>(q.rows), const_cast<void*>(qo.p), qo.ld, const_cast<void*>(ko.p), ko.ld,
                            at.stream.stream());
          }),
          "hstu_rotary");
    PyObject* kr = out_k.o ? out_k.o : Py_None;
    return PyTuple_Pack(2, out_q.o, kr);
  });
}

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"k", "v",         "k_cache", "v_cache",  "page_table",  "q_offsets", "kv_len",
                                        "q", "positions", "freqs",   "sections", "interleaved", "q_out",     "stream"};
    PyObject* a[14];
    place("hstu_paged_append", names, 7, args, nargs, kwnames, a);
    need_library();
    const Rows k = rows_of("k", a[0]), v = rows_of("v", a[1], &k);
    const int32_t B = users_of(a[5]);
    const int32_t* offsets = index_of("q_offsets", a[5], static_cast<int64_t>(B) + 1, k.device);
    const int32_t* lens = index_of("kv_len", a[6], B, k.device);
    const hstu_paged_cache_t cache = cache_of(a[2], a[3], a[4], B, k);
    hstu_rotation_t rot;
    const bool turn = given(a[9]);
    if (turn) rot = rotation_of(a[9], a[10], a[8], a[11], k.rows, k.device, false);
    else if (given(a[7]) || given(a[8]) || given(a[10])) raise(PyExc_ValueError, "q, positions and sections need freqs");
    if (given(a[12]) && !given(a[7])) raise(PyExc_ValueError, "q_out without q");
    const Place at(k.device, a[13]);
    Rows q, qo;
    Held out;
    if (given(a[7])) {
      q = rows_of("q", a[7], &k);
      qo = output_of("q_out", a[12], k, at, out.o);
    }
    check(unlocked([&] {
            return g_append(q.p, q.ld, k.p, k.ld, v.p, v.ld, turn ? &rot : nullptr, &cache, offsets, lens, B,
                            static_cast<int32_t>(k.H), static_cast<int32_t>(k.d), static_cast<int32_t>(k.rows),
                            const_cast<void*>(qo.p), qo.ld, at.stream.stream());
          }),
          "hstu_paged_append");
    if (out.o) return out.release();
    Py_RETURN_NONE;
  });
}

// hstu_paged_attn_fwd's arguments, then out and stream; with `limit`, limit_ns before those two.
PyObject* attn(PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, bool limit) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q",     "k_cache", "v_cache", "page_table", "q_offsets", "kv_len", "num_targets",
                                        "alpha", "N",       "max_new", "max_kv",     "out",       "stream"};
    static const char* const limited[] = {"q", "k_cache", "v_cache", "page_table", "q_offsets", "kv_len", "num_targets",
                                          "alpha", "N", "max_new", "max_kv", "limit_ns", "out", "stream"};
    const char* const fn = limit ? "hstu_paged_selfcheck_fwd_timeout" : "hstu_paged_attn_fwd";
    PyObject *a[13], *b[14];
    if (limit) {
      place(fn, limited, 12, args, nargs, kwnames, b);
      std::memcpy(a, b, 11 * sizeof(a[0]));
      a[11] = b[12];
      a[12] = b[13];
    } else {
      place(fn, names, 11, args, nargs, kwnames, a);
    }
    need_library();
    const Rows q = rows_of("q", a[0]);
    const int32_t B = users_of(a[4]);
    const int32_t* offsets = index_of("q_offsets", a[4], static_cast<int64_t>(B) + 1, q.device);
    const int32_t* lens = index_of("kv_len", a[5], B, q.device);
    const int32_t* targets = given(a[6]) ? index_of("num_targets", a[6], B, q.device) : nullptr;
    const hstu_paged_cache_t cache = cache_of(a[1], a[2], a[3], B, q);
    const float alpha = float_of(a[7]), N = float_of(a[8]);
    const int32_t max_new = int32_of("max_new", a[9]), max_kv = int32_of("max_kv", a[10]);
    const int32_t limit_ns = limit ? int32_of("limit_ns", b[11]) : 0;
    const Place at(q.device, a[12]);
    Held out;
    const Rows o = output_of("out", a[11], q, at, out.o);
    const int32_t H = static_cast<int32_t>(q.H), d = static_cast<int32_t>(q.d), rows = static_cast<int32_t>(q.rows);
    check(unlocked([&] {
            if (!limit)
              return g_attn(q.p, q.ld, &cache, offsets, lens, targets, B, H, d, rows, max_new, max_kv, alpha, N,
                            const_cast<void*>(o.p), o.ld, at.stream.stream());
            return g_selfcheck(q.p, q.ld, &cache, offsets, lens, targets, B, H, d, rows, max_new, max_kv, alpha, N,
                               const_cast<void*>(o.p), o.ld, limit_ns < 0 ? 0u : static_cast<uint64_t>(limit_ns),
                               at.stream.stream());
          }),
          fn);
    return out.release();
  });
}

PyObject* attn_fwd(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return attn(args, nargs, kwnames, false);
}

PyObject* selfcheck(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return attn(args, nargs, kwnames, true);
}

// bind(HstuError, rotary, append, attn_fwd, selfcheck): the error class and the entry points' addresses.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long p[4];
  if (!PyArg_ParseTuple(args, "OKKKK", &error, &p[0], &p[1], &p[2], &p[3])) return nullptr;
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  g_rotary = reinterpret_cast<decltype(g_rotary)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_attn = reinterpret_cast<decltype(g_attn)>(p[2]);
  g_selfcheck = reinterpret_cast<decltype(g_selfcheck)>(p[3]);
  Py_RETURN_NONE;
}

PyDoc_STRVAR(kRotaryDoc,
             "hstu_rotary(q, k, positions, freqs, sections=None, interleaved=False, inverse=False, q_out=None, k_out=None, "
             "stream=None)\n--\n\n"
             "Rotates q and (unless None) k, bf16 [rows, H, d], by their positions; returns (q_out, k_out).\n"
             "``positions``: int32 [rows] or [axes, rows]; ``freqs``: float64 [pairs]; ``sections``: pairs of each axis.\n"
             "``inverse`` turns back, which is the gradient.  ``q_out`` may be q (in place).  See include/hstu_paged.h.");
PyDoc_STRVAR(kAppendDoc,
             "hstu_paged_append(k, v, k_cache, v_cache, page_table, q_offsets, kv_len, q=None, positions=None, freqs=None, "
             "sections=None, interleaved=False, q_out=None, stream=None)\n--\n\n"
             "Writes the new rows k, v (bf16 [total_new, H, d], users packed by q_offsets) to the last places of each\n"
             "user's kv_len rows in the paged cache, bf16 [pages, page_size, H, d].  With ``freqs`` K is rotated on the\n"
             "way, and q too if given; ``positions`` default to the place in the cache.  Returns the rotated q (or None).\n"
             "See include/hstu_paged.h.");
PyDoc_STRVAR(kAttnDoc,
             "hstu_paged_attn_fwd(q, k_cache, v_cache, page_table, q_offsets, kv_len, num_targets, alpha, N, max_new, "
             "max_kv, out=None, stream=None)\n--\n\n"
             "Attention of each user's new rows q (bf16 [total_new, H, d], packed by q_offsets) over its kv_len rows in\n"
             "the paged cache, the new ones included; the last num_targets of them are candidates.  Returns ``out``.\n"
             "See include/hstu_paged.h.");

PyDoc_STRVAR(kSelfcheckDoc,
             "hstu_paged_selfcheck_fwd_timeout(q, k_cache, v_cache, page_table, q_offsets, kv_len, num_targets, alpha, N, "
             "max_new, max_kv, limit_ns, out=None, stream=None)\n--\n\n"
             "hstu_paged_attn_fwd on the kernel for many rows with every wait limited to limit_ns (test hook of the abort\n"
             "path); returns ``out``, partly written.");

PyMethodDef kMethods[] = {
    {"hstu_rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rotary)), METH_FASTCALL | METH_KEYWORDS,
     kRotaryDoc},
    {"hstu_paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL | METH_KEYWORDS,
     kAppendDoc},
    {"hstu_paged_attn_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn_fwd)),
     METH_FASTCALL | METH_KEYWORDS, kAttnDoc},
    {"hstu_paged_selfcheck_fwd_timeout", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(selfcheck)),
     METH_FASTCALL | METH_KEYWORDS, kSelfcheckDoc},
    {"bind", bind, METH_VARARGS, "bind(error, rotary, append, attn_fwd, selfcheck): the error class and the C entry points."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged_native", "Marshalling of the paged calls; see paged.py.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native() { return PyModule_Create(&kModule); }
