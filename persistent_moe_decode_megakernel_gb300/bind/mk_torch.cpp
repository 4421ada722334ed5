// mk_torch.cpp -- the chunk operators' argument marshalling for torch tensors, as a CPython module
// (_mk_torch) beside libmk.so.  It checks what the C calls cannot see (types, shapes, devices), makes new
// outputs, takes the current stream of the cache's device and calls the C ABI; nothing else.
//
// These calls are short next to what Python spends on marshalling: for a few tokens the device needs
// 3 to 8 us, and the same checks written in Python with ctypes took about 10 us more a call (attention of a
// prompt of 65 tokens 17.9 us, now 8.4; 8 tokens appended 22.2, now 9.9).

#define PY_SSIZE_T_CLEAN
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>

#include "mk_chunk.h"
#include "mk_span_call.h"

namespace {

PyObject* g_error = nullptr;   // the package's MkError(code, text)

// The C calls, of the libmk.so that the package has loaded.
struct {
  decltype(&mk_append_chunk) append;
  decltype(&mk_chunk_attention_workspace) workspace;
  decltype(&mk_chunk_attention) attention;
  decltype(&mk_read_cache) read;
  decltype(&mk_last_error) last_error;
  decltype(&mk_window_attention_in) window;
  decltype(&mk_prefix_attention_in) prefix;
} g_mk = {};

// Other Python threads run while a call launches or allocates: a launch waits when the device's queue is
// full, an allocation for the allocator's lock, whose holder may want the interpreter's.
struct Unlocked {
  PyThreadState* s = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(s); }
};

// Raises MkError and leaves the call: caught by `guarded`, which returns NULL to Python.
struct Raised {};
[[noreturn]] void raise(int code, const char* text) {
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", code, text) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, text);
  }
  throw Raised();
}
void need(bool ok, const char* text) {
  if (!ok) raise(MK_ERR_INVALID_ARG, text);
}
template <class F>
void run(F&& call) {
  int rc;
  {
    Unlocked u;
    rc = call();
  }
  if (rc != MK_OK) raise(rc, g_mk.last_error());
}
template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// A ctypes structure's bytes.
template <class T>
T structure(PyObject* o, const char* what) {
  Py_buffer v;
  if (PyObject_GetBuffer(o, &v, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    raise(MK_ERR_INVALID_ARG, what);
  }
  T out;
  const bool ok = v.len == static_cast<Py_ssize_t>(sizeof out);
  if (ok) std::memcpy(&out, v.buf, sizeof out);
  PyBuffer_Release(&v);
  need(ok, what);
  return out;
}

constexpr int kMaxSeqs = 64;
struct Lengths {
  int64_t n = 0, sum = 0;
  int32_t v[kMaxSeqs + 1] = {};    // (one too many is refused by the C call)
  void add(int64_t x) {
    need(x >= INT32_MIN && x <= INT32_MAX, "a length does not fit 32 bits");
    if (n <= kMaxSeqs) v[n] = static_cast<int32_t>(x);
    ++n;
    sum += x;
  }
};
// Whole numbers: a buffer of 32- or 64-bit ones (numpy), or a sequence.
Lengths lengths(PyObject* o, const char* what = "chunk_lens and seq_lens: one whole number per sequence each",
                const char* where = "chunk_lens and seq_lens: in host memory") {
  Lengths out;
  need(!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda(), where);
  Py_buffer b;
  if (PyObject_CheckBuffer(o) && PyObject_GetBuffer(o, &b, PyBUF_FORMAT | PyBUF_ND) == 0) {
    struct Release {                  // (a length that `add` refuses leaves by an exception)
      Py_buffer* b;
      ~Release() { PyBuffer_Release(b); }
    } release{&b};
    const char f = b.format && b.format[0] && !b.format[1] ? b.format[0] : 0;
    const bool w4 = f == 'i' && b.itemsize == 4, w8 = (f == 'l' || f == 'q') && b.itemsize == 8;
    const bool ok = b.ndim == 1 && (w4 || w8);
    if (ok)
      for (Py_ssize_t i = 0; i < b.shape[0] && i <= kMaxSeqs; ++i)
        out.add(w4 ? static_cast<const int32_t*>(b.buf)[i] : static_cast<const int64_t*>(b.buf)[i]);
    if (ok) return out;
    out = Lengths();
  }
  PyErr_Clear();
  PyObject* s = PySequence_Fast(o, what);
  if (!s) {
    PyErr_Clear();
    raise(MK_ERR_INVALID_ARG, what);
  }
  bool ok = true;
  for (Py_ssize_t i = 0; ok && i < PySequence_Fast_GET_SIZE(s); ++i) {
    PyObject* x = PyNumber_Index(PySequence_Fast_GET_ITEM(s, i));
    const long long v = x ? PyLong_AsLongLong(x) : -1;
    Py_XDECREF(x);
    ok = !PyErr_Occurred() && v >= INT32_MIN && v <= INT32_MAX;
    if (ok) out.add(v);
  }
  Py_DECREF(s);
  if (!ok) {
    PyErr_Clear();
    raise(MK_ERR_INVALID_ARG, what);
  }
  return out;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  need(THPVariable_Check(o), what);
  return THPVariable_Unpack(o);
}

// What every call has: the shape, the sequences, the block tables and the cache.
struct Call {
  mk_cache_shape shape;
  Lengths chunk, len;
  int64_t rows;
  int dev;
  const at::Tensor &bt, &kv;
  Call(PyObject* const* a)   // shape, (the rows), chunk_lens, seq_lens, block_tables, kv_layer
      : shape(structure<mk_cache_shape>(a[0], "shape: a CacheShape")),
        chunk(lengths(a[2])),
        len(lengths(a[3])),
        bt(tensor(a[4], "block_tables: a tensor")),
        kv(tensor(a[5], "kv_layer: a tensor")) {
    need(chunk.n == len.n, "chunk_lens and seq_lens: one length per sequence each");
    rows = chunk.sum;
    need(rows >= 0 && rows < (int64_t(1) << 24), "chunk_lens: fewer than 2^24 rows");
    need(kv.is_cuda() && bt.is_cuda() && bt.get_device() == kv.get_device() && bt.scalar_type() == at::kInt &&
             bt.dim() == 2 && bt.size(0) >= chunk.n && bt.size(1) == shape.max_pages_per_seq && bt.is_contiguous(),
         "block_tables: contiguous int32 [num_seqs, max_pages_per_seq] on the cache's CUDA device");
    dev = kv.get_device();
    const bool q8 = shape.flags & MK_FLAG_KV_Q8;
    // (products of a shape that the C call refuses may wrap: as unsigned, and it is refused there)
    const uint64_t n = uint64_t(2) * uint32_t(shape.num_pages) * uint32_t(shape.num_kv_heads) * uint32_t(shape.page_size) *
                       uint32_t(shape.head_dim);
    need(kv.scalar_type() == (q8 ? at::kByte : at::kBFloat16) && uint64_t(kv.numel()) == (q8 ? n + n / 16 : n) &&
             kv.is_contiguous(),
         "kv_layer: one layer of the shape's cache, contiguous CUDA tensor, bf16 (q8_0: uint8 codes, then f16 scales)");
  }
  bool bf16(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == dev && t.scalar_type() == at::kBFloat16; }
  // The row stride of t, bf16 rows of heads * D contiguous values, as [rows, heads * D] or [rows, heads, D].
  int64_t rows_of(const at::Tensor& t, int64_t heads, const char* what) const {
    const int64_t D = shape.head_dim;
    need(bf16(t) && t.dim() >= 2 && t.size(0) >= rows &&
             ((t.dim() == 2 && t.size(1) == heads * D && t.stride(1) == 1) ||
              (t.dim() == 3 && t.size(1) == heads && t.size(2) == D && t.stride(2) == 1 && (t.stride(1) == D || heads == 1))),
         what);
    return t.size(0) > 1 ? t.stride(0) : heads * D;
  }
  at::Tensor make(at::IntArrayRef size, at::ScalarType type) const {
    Unlocked u;
    return at::empty(size, kv.options().dtype(type));
  }
  at::Tensor out(PyObject* o, int64_t heads, const char* what) const {
    const int64_t D = shape.head_dim;
    if (o == Py_None) {
      need(heads > 0 && D > 0 && heads <= (int64_t(1) << 20) && D <= 4096, "shape: heads or head_dim out of range");
      return make({rows, heads, D}, at::kBFloat16);
    }
    const at::Tensor& t = tensor(o, what);
    need(bf16(t) && t.is_contiguous() && t.dim() == 3 && t.size(0) >= rows && t.size(1) == heads && t.size(2) == D, what);
    return t;
  }
  int32_t* status(PyObject* o) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "status: a tensor or None");
    need(t.is_cuda() && t.get_device() == dev && t.scalar_type() == at::kInt && t.numel() == 1,
         "status: int32 tensor of one value on the cache's device");
    return t.data_ptr<int32_t>();
  }
  mk_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  int n() const { return static_cast<int>(std::min<int64_t>(chunk.n, kMaxSeqs + 1)); }
  const int32_t* tables() const { return bt.data_ptr<int32_t>(); }
};

PyObject* keep(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}
bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// append_chunk(shape, qkv, chunk_lens, seq_lens, block_tables, kv_layer, rope, q_norm, k_norm, eps, q_out, status)
PyObject* append_chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a);
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
    const at::Tensor& qkv = tensor(a[1], "qkv: a tensor");
    const int64_t stride = c.rows_of(qkv, int64_t(c.shape.num_q_heads) + 2 * int64_t(c.shape.num_kv_heads),
                                     "qkv: bf16 rows of num_q_heads + 2*num_kv_heads heads of head_dim contiguous values on the "
                                     "cache's device, one for each new token at least");
    mk_rope rope;
    if (a[6] != Py_None) rope = structure<mk_rope>(a[6], "rope: a Rope or None");
    const void* gain[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (a[7 + i] == Py_None) continue;
      const at::Tensor& t = tensor(a[7 + i], "q_norm / k_norm: a tensor or None");
      need(c.bf16(t) && t.is_contiguous() && t.numel() == c.shape.head_dim,
           "q_norm / k_norm: contiguous bf16 [head_dim] on the cache's device");
      gain[i] = t.data_ptr();
    }
    const double eps = PyFloat_AsDouble(a[9]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    int32_t* status = c.status(a[11]);
    const at::Tensor out = c.out(a[10], c.shape.num_q_heads, "q_out: contiguous bf16 [rows, num_q_heads, head_dim] on the cache's device");
    const mk_stream_t on = c.stream();
    run([&] {
      return g_mk.append(&c.shape, c.n(), c.chunk.v, c.len.v, c.tables(), qkv.data_ptr(), stride,
                         a[6] == Py_None ? nullptr : &rope, gain[0], gain[1], static_cast<float>(eps), out.data_ptr(),
                         c.kv.data_ptr(), status, on);
    });
    return keep(a[10], out);
  });
}

// What the attention calls share: (shape, q, chunk_lens, seq_lens, block_tables, kv_layer, out, workspace, status, ..)
// with what is their own behind that.
struct Rows {
  const at::Tensor& q;
  const int64_t stride;
  int32_t* const status;
  const at::Tensor out;
  at::Tensor ws;               // as given
  Rows(PyObject* const* a, const Call& c)
      : q(tensor(a[1], "q: a tensor")),
        stride(c.rows_of(q, c.shape.num_q_heads,
                         "q: bf16 rows of num_q_heads heads of head_dim contiguous values on the cache's device, one for each "
                         "new token at least")),
        status(c.status(a[8])),
        out(c.out(a[6], c.shape.num_q_heads, "out: contiguous bf16 [rows, num_q_heads, head_dim] on the cache's device")) {
    if (a[7] == Py_None) return;
    ws = tensor(a[7], "workspace: a tensor or None");
    need(ws.is_cuda() && ws.get_device() == c.dev && ws.is_contiguous(), "workspace: contiguous tensor on the cache's device");
  }
  void* ws_ptr() const { return ws.defined() ? ws.data_ptr() : nullptr; }
  size_t ws_bytes() const { return ws.defined() ? ws.nbytes() : 0; }
};

// chunk_attention(.., status)
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a);
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
    Rows r(a, c);
    if (!r.ws.defined()) {
      size_t bytes = 0;
      run([&] { return g_mk.workspace(&c.shape, c.n(), c.chunk.v, c.len.v, &bytes); });
      if (bytes) r.ws = c.make({static_cast<int64_t>(bytes)}, at::kByte);
    }
    const mk_stream_t on = c.stream();
    run([&] {
      return g_mk.attention(&c.shape, c.n(), c.chunk.v, c.len.v, c.tables(), r.q.data_ptr(), r.stride, c.kv.data_ptr(),
                            r.out.data_ptr(), r.ws_ptr(), r.ws_bytes(), r.status, on);
    });
    return keep(a[6], r.out);
  });
}

// A workspace that the call asks for (inside `run`, so without the interpreter's lock).
struct Taken {
  const Call& c;
  at::Tensor ws;
  std::exception_ptr failed;
  static void* take(void* self, size_t bytes) noexcept {
    Taken& t = *static_cast<Taken*>(self);
    try {
      t.ws = at::empty({static_cast<int64_t>(bytes)}, t.c.kv.options().dtype(at::kByte));
      return t.ws.data_ptr();
    } catch (...) {
      t.failed = std::current_exception();
      return nullptr;
    }
  }
};
template <class Attend>
PyObject* span_attention(PyObject* const* a, const Call& c, Attend&& attend) {
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
  const Rows r(a, c);
  Taken taken{c, {}, {}};
  const mk_span_workspace ws = {r.ws_ptr(), r.ws_bytes(), r.ws.defined() ? nullptr : Taken::take, &taken};
  const mk_stream_t on = c.stream();
  int rc;
  {
    Unlocked u;
    rc = attend(r, &ws, on);
  }
  if (taken.failed) std::rethrow_exception(taken.failed);
  if (rc != MK_OK) raise(rc, g_mk.last_error());
  return keep(a[6], r.out);
}

int32_t number(PyObject* o, const char* what) {
  PyObject* x = PyNumber_Index(o);
  const long long v = x ? PyLong_AsLongLong(x) : -1;
  Py_XDECREF(x);
  if (PyErr_Occurred() || v < INT32_MIN || v > INT32_MAX) {
    PyErr_Clear();
    raise(MK_ERR_INVALID_ARG, what);
  }
  return static_cast<int32_t>(v);
}

// window_attention(.., status, window, sinks)
PyObject* window_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a);
    const int32_t window = number(a[9], "window: a whole number of 32 bits"), sinks = number(a[10], "sinks: a whole number of 32 bits");
    return span_attention(a, c, [&](const Rows& r, const mk_span_workspace* ws, mk_stream_t on) {
      return g_mk.window(&c.shape, c.n(), c.chunk.v, c.len.v, window, sinks, c.tables(), r.q.data_ptr(), r.stride,
                         c.kv.data_ptr(), r.out.data_ptr(), ws, r.status, on);
    });
  });
}

// prefix_attention(.., status, group_seqs, prefix_lens)
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a);
    const char *what = "group_seqs and prefix_lens: one whole number per group each", *where = "group_seqs and prefix_lens: in host memory";
    const Lengths seqs = lengths(a[9], what, where), shared = lengths(a[10], what, where);
    need(seqs.n == shared.n, "group_seqs and prefix_lens: one number per group each");
    const int groups = static_cast<int>(std::min<int64_t>(seqs.n, kMaxSeqs + 1));
    return span_attention(a, c, [&](const Rows& r, const mk_span_workspace* ws, mk_stream_t on) {
      return g_mk.prefix(&c.shape, c.n(), c.chunk.v, c.len.v, groups, seqs.v, shared.v, c.tables(), r.q.data_ptr(), r.stride,
                         c.kv.data_ptr(), r.out.data_ptr(), ws, r.status, on);
    });
  });
}

// read_cache(shape, None, counts, seq_lens, block_tables, kv_layer, k_out, v_out, status)
PyObject* read_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a);
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
    int32_t* status = c.status(a[8]);
    const char* what = "k_out / v_out: contiguous bf16 [rows, num_kv_heads, head_dim] on the cache's device";
    const at::Tensor k = c.out(a[6], c.shape.num_kv_heads, what), v = c.out(a[7], c.shape.num_kv_heads, what);
    const mk_stream_t on = c.stream();
    run([&] {
      return g_mk.read(&c.shape, c.n(), c.chunk.v, c.len.v, c.tables(), c.kv.data_ptr(), k.data_ptr(), v.data_ptr(), status, on);
    });
    PyObject *pk = keep(a[6], k), *pv = keep(a[7], v);
    PyObject* r = pk && pv ? PyTuple_Pack(2, pk, pv) : nullptr;
    Py_XDECREF(pk);
    Py_XDECREF(pv);
    return r;
  });
}

// init(the exception class, called with (code, text); the addresses of the seven calls in the order of g_mk)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 8)) return nullptr;
  void* f[7];
  for (int i = 0; i < 7; ++i) f[i] = PyLong_AsVoidPtr(a[1 + i]);
  if (PyErr_Occurred()) return nullptr;
  static_assert(sizeof f == sizeof g_mk, "seven calls");
  std::memcpy(&g_mk, f, sizeof f);
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}
PyMethodDef methods[] = {
    {"append_chunk", fast<append_chunk>(), METH_FASTCALL, "mk_append_chunk on torch tensors"},
    {"chunk_attention", fast<chunk_attention>(), METH_FASTCALL, "mk_chunk_attention on torch tensors"},
    {"window_attention", fast<window_attention>(), METH_FASTCALL, "mk_window_attention on torch tensors"},
    {"prefix_attention", fast<prefix_attention>(), METH_FASTCALL, "mk_prefix_attention on torch tensors"},
    {"read_cache", fast<read_cache>(), METH_FASTCALL, "mk_read_cache on torch tensors"},
    {"init", fast<init>(), METH_FASTCALL, "the exception class and the C calls' addresses"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mk_torch", "argument marshalling of the chunk operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mk_torch() { return PyModule_Create(&module); }
