// calls.cpp -- the Python calls of the windowed attention and the paged cache,
// as a CPython module (_calls).
//
// Their smallest kernels run for a few microseconds, less than the host needs
// to check and pass five to ten tensors from Python (0.5 us a tensor; on one
// host 12.2 us of host time for window_attn at T=2048, 9.9 us for paged_tables
// and 8.7 us for paged_append, of which 4 to 6 us in the library).  Here a tensor's
// type, device, shape and strides are read from the tensor itself.
//
// Each function takes the Python call's arguments in order, the stream (or
// None) last, checks the tensors, makes their device current and calls the C
// ABI at the address that bind() got.  It returns the INFLLMV2_* code; what
// is not a tensor, an integer or the right parameter struct raises TypeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "infllmv2.h"

namespace {

decltype(&infllmv2_window_attn) f_window_attn;
decltype(&infllmv2_window_attn_backward) f_window_attn_backward;
decltype(&infllmv2_paged_tables) f_paged_tables;
decltype(&infllmv2_paged_append) f_paged_append;
decltype(&infllmv2_paged_attn) f_paged_attn;

// A Python error is set; unwinds to guarded().
struct PythonError {};
// A tensor that does not fit.
struct BadTensor {};

template <typename P>
P params(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PythonError{};
  const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(P));
  P p{};
  if (fits) p = *static_cast<const P*>(b.buf);
  PyBuffer_Release(&b);
  if (!fits) {
    PyErr_SetString(PyExc_TypeError, "not this call's parameter struct");
    throw PythonError{};
  }
  return p;
}

int32_t int32(PyObject* o) {
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (overflow || v != static_cast<int32_t>(v)) {
    PyErr_SetString(PyExc_OverflowError, "not a 32-bit integer");
    throw PythonError{};
  }
  return static_cast<int32_t>(v);
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    throw PythonError{};
  }
  return THPVariable_Unpack(o);
}

// The device that all of a call's tensors have to be on.
struct Device {
  int index;
  explicit Device(PyObject* o) {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda()) throw BadTensor{};
    index = t.get_device();
  }
  const at::Tensor& here(PyObject* o, at::ScalarType type) const {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type) throw BadTensor{};
    return t;
  }
  // Address of a densely packed tensor of this type and shape.
  void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = here(o, type);
    if (t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) throw BadTensor{};
    return t.data_ptr();
  }
  void* bf16(PyObject* o, std::initializer_list<int64_t> shape) const {
    return dense(o, at::kBFloat16, shape);
  }
  float* f32(PyObject* o, std::initializer_list<int64_t> shape) const {
    return static_cast<float*>(dense(o, at::kFloat, shape));
  }
  int32_t* i32(PyObject* o, std::initializer_list<int64_t> shape) const {
    return static_cast<int32_t*>(dense(o, at::kInt, shape));
  }
  // [n, heads, d] bf16 rows, packed within a row; their stride in elements.
  void* rows(PyObject* o, int64_t n, int64_t heads, int64_t d, int64_t* stride) const {
    const at::Tensor& t = here(o, at::kBFloat16);
    if (t.sizes() != at::IntArrayRef({n, heads, d})) throw BadTensor{};
    const auto s = t.strides();
    if (n > 0 && (s[2] != 1 || (heads > 1 && s[1] != d))) throw BadTensor{};
    *stride = n > 1 ? s[0] : heads * d;
    return t.data_ptr();
  }
  // A workspace of any type, dense.
  void* workspace(PyObject* o, size_t* bytes) const {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != index || !t.is_contiguous()) throw BadTensor{};
    *bytes = t.nbytes();
    return t.data_ptr();
  }
  // The tensors' device made current, without the interpreter's lock; on its
  // current stream, or on `stream`.
  template <typename F>
  int run(PyObject* stream, F&& f) const {
    void* st;
    if (stream == Py_None) {
      st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    } else {
      PyObject* handle = PyObject_GetAttrString(stream, "cuda_stream");
      if (!handle) throw PythonError{};
      st = PyLong_AsVoidPtr(handle);
      Py_DECREF(handle);
      if (PyErr_Occurred()) throw PythonError{};
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = f(st);
    Py_END_ALLOW_THREADS
    return code;
  }
};

int window_attn(PyObject* const* a) {
  const auto p = params<infllmv2_params>(a[0]);
  const int32_t window = int32(a[1]), n_sink = int32(a[2]);
  const Device dev(a[3]);
  const void *Q = dev.bf16(a[3], {p.B, p.T, p.Hq, p.head_dim}),
             *K = dev.bf16(a[4], {p.B, p.T, p.Hkv, p.head_dim}),
             *V = dev.bf16(a[5], {p.B, p.T, p.Hkv, p.head_dim});
  void* O = dev.bf16(a[6], {p.B, p.T, p.Hq, p.head_dim});
  float* lse = dev.f32(a[7], {p.B, p.Hq, p.T});
  return dev.run(a[8],
                 [&](void* st) { return f_window_attn(&p, window, n_sink, Q, K, V, O, lse, st); });
}

int window_attn_backward(PyObject* const* a) {
  const auto p = params<infllmv2_params>(a[0]);
  const int32_t window = int32(a[1]), n_sink = int32(a[2]);
  const Device dev(a[3]);
  auto q = [&](PyObject* o) { return dev.bf16(o, {p.B, p.T, p.Hq, p.head_dim}); };
  auto kv = [&](PyObject* o) { return dev.bf16(o, {p.B, p.T, p.Hkv, p.head_dim}); };
  const void *Q = q(a[3]), *K = kv(a[4]), *V = kv(a[5]), *O = q(a[6]);
  const float* lse = dev.f32(a[7], {p.B, p.Hq, p.T});
  const void* dO = q(a[8]);
  void *dQ = q(a[9]), *dK = kv(a[10]), *dV = kv(a[11]);
  size_t bytes;
  void* ws = dev.workspace(a[12], &bytes);
  return dev.run(a[13], [&](void* st) {
    return f_window_attn_backward(&p, window, n_sink, Q, K, V, O, lse, dO, dQ, dK, dV, ws, bytes,
                                  st);
  });
}

int paged_tables(PyObject* const* a) {
  const auto p = params<infllmv2_paged_params>(a[0]);
  const int64_t n = p.n_seqs, rows = p.n_tokens;
  const Device dev(a[6]);
  const int64_t n_free = tensor(a[3]).numel();
  const int32_t *kv_lens = dev.i32(a[1], {n}), *q_lens = dev.i32(a[2], {n}),
                *free_pages = dev.i32(a[3], {n_free}), *free_count = dev.i32(a[4], {1});
  // an empty tensor has no address; a list of no pages is not read
  if (n_free == 0) free_pages = free_count;
  int32_t *table = dev.i32(a[5], {n, p.max_pages}), *cu_q = dev.i32(a[6], {n + 1}),
          *seqlens = dev.i32(a[7], {n}), *slots = dev.i32(a[8], {rows}),
          *positions = dev.i32(a[9], {rows}), *free_left = dev.i32(a[10], {1});
  return dev.run(a[11], [&](void* st) {
    return f_paged_tables(&p, kv_lens, q_lens, free_pages, free_count, table, cu_q, seqlens, slots,
                          positions, free_left, st);
  });
}

int paged_append(PyObject* const* a) {
  const auto p = params<infllmv2_paged_params>(a[0]);
  const Device dev(a[4]);
  const int32_t* slots = dev.i32(a[1], {p.n_tokens});
  int64_t ks, vs;
  const void *k = dev.rows(a[2], p.n_tokens, p.Hkv, p.head_dim, &ks),
             *v = dev.rows(a[3], p.n_tokens, p.Hkv, p.head_dim, &vs);
  void *K = dev.bf16(a[4], {p.n_pages, p.page_size, p.Hkv, p.head_dim}),
       *V = dev.bf16(a[5], {p.n_pages, p.page_size, p.Hkv, p.head_dim});
  return dev.run(a[6],
                 [&](void* st) { return f_paged_append(&p, slots, k, ks, v, vs, K, V, st); });
}

int paged_attn(PyObject* const* a) {
  const auto p = params<infllmv2_paged_params>(a[0]);
  const Device dev(a[2]);
  int64_t qs;
  const void *Q = dev.rows(a[1], p.n_tokens, p.Hq, p.head_dim, &qs),
             *K = dev.bf16(a[2], {p.n_pages, p.page_size, p.Hkv, p.head_dim}),
             *V = dev.bf16(a[3], {p.n_pages, p.page_size, p.Hkv, p.head_dim});
  const int32_t *table = dev.i32(a[4], {p.n_seqs, p.max_pages}),
                *cu_q = dev.i32(a[5], {static_cast<int64_t>(p.n_seqs) + 1}),
                *seqlens = dev.i32(a[6], {p.n_seqs});
  void* O = dev.bf16(a[7], {p.n_tokens, p.Hq, p.head_dim});
  float* lse = dev.f32(a[8], {p.n_tokens, p.Hq});
  size_t bytes;
  void* ws = dev.workspace(a[9], &bytes);
  return dev.run(a[10], [&](void* st) {
    return f_paged_attn(&p, Q, qs, K, V, table, cu_q, seqlens, O, lse, ws, bytes, st);
  });
}

// Runs a call of N arguments; no C++ exception leaves it.
template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const BadTensor&) {
    return PyLong_FromLong(INFLLMV2_ERR_INVALID_ARG);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(addresses): the library's functions, in the order below.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void** f[] = {reinterpret_cast<void**>(&f_window_attn),
                reinterpret_cast<void**>(&f_window_attn_backward),
                reinterpret_cast<void**>(&f_paged_tables),
                reinterpret_cast<void**>(&f_paged_append),
                reinterpret_cast<void**>(&f_paged_attn)};
  constexpr Py_ssize_t kN = sizeof(f) / sizeof(f[0]);
  if (n != kN) {
    PyErr_Format(PyExc_TypeError, "expected %zd addresses, got %zd", kN, n);
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kN; ++i) {
    void* address = PyLong_AsVoidPtr(args[i]);
    if (!address) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
    *f[i] = address;
  }
  Py_RETURN_NONE;
}

#define CALL(name, n) \
  {#name, reinterpret_cast<PyCFunction>(&guarded<name, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(&bind), METH_FASTCALL, nullptr},
    CALL(window_attn, 9), CALL(window_attn_backward, 14), CALL(paged_tables, 12),
    CALL(paged_append, 7), CALL(paged_attn, 11), {nullptr, nullptr, 0, nullptr}};
#undef CALL
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was compiled with; its tensors'
// layout is that version's alone.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", INFLLMV2_TORCH) != 0) Py_CLEAR(m);
  return m;
}
