// binding.cpp -- marshals torch tensors into attn_tensor structs and calls the C
// ABI: a CPython extension for the calls whose kernels are shorter than a
// marshalling in Python takes.  Reading one tensor's address, sizes and strides
// through Python attributes costs about 0.75 us, and the serving calls have nine
// tensors each; here a call costs about 1 us before its launch.
//
// Each function takes (stream, arguments in the C order) with stream None for the
// device's current stream or a cudaStream_t as an int, checks that every tensor is
// on one CUDA device, makes that device current for the call, and returns the
// attn_status code.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/attnsink.h"

namespace {

// One tensor argument; false (with a Python error set) if it cannot be passed.
// `device` is -1 before the first one.
bool describe(PyObject *o, attn_tensor *d, int *device) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
    return false;
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided || (*device >= 0 && t.get_device() != *device)) {
    PyErr_SetString(PyExc_ValueError, "tensors must be on one CUDA device");
    return false;
  }
  *device = static_cast<int>(t.get_device());
  switch (t.scalar_type()) {
    case at::kBFloat16: d->dtype = ATTN_DTYPE_BF16; break;
    case at::kFloat: d->dtype = ATTN_DTYPE_F32; break;
    case at::kInt: d->dtype = ATTN_DTYPE_I32; break;
    case at::kFloat8_e4m3fn: d->dtype = ATTN_DTYPE_E4M3; break;
    case at::kFloat8_e8m0fnu: d->dtype = ATTN_DTYPE_E8M0; break;
    default:
      PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
      return false;
  }
  if (t.dim() > 4) {
    PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
    return false;
  }
  d->ndim = static_cast<int32_t>(t.dim());
  const c10::IntArrayRef size = t.sizes(), stride = t.strides();
  for (int i = 0; i < d->ndim; ++i) {
    d->shape[i] = size[i];
    d->stride[i] = stride[i];
  }
  d->data = t.numel() > 0 ? const_cast<void *>(t.const_data_ptr()) : nullptr;
  return true;
}

constexpr int kMaxTensors = 9;

// The arguments of one call: tensors in order, integers and floats by position.
struct Call {
  attn_tensor t[kMaxTensors];
  attn_tensor *p[kMaxTensors];
  int device = -1;
  cudaStream_t stream = nullptr;
};

// Reads `n` tensors at the positions in `at`; None is a null pointer where the
// bit of `optional` allows it.
bool tensors(PyObject *const *args, const int *at, int n, unsigned optional, Call *c) {
  for (int i = 0; i < n; ++i) {
    PyObject *o = args[at[i]];
    if (o == Py_None && (optional >> i & 1u)) {
      c->p[i] = nullptr;
      continue;
    }
    if (!describe(o, &c->t[i], &c->device)) return false;
    c->p[i] = &c->t[i];
  }
  if (args[0] == Py_None) {
    c->stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c->device)).stream();
  } else {
    c->stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(args[0]));
    if (PyErr_Occurred()) return false;
  }
  return true;
}

bool as_int32(PyObject *o, int32_t *v) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x < INT32_MIN || x > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return false;
  }
  *v = static_cast<int32_t>(x);
  return true;
}

bool as_float(PyObject *o, float *v) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return false;
  *v = static_cast<float>(x);
  return true;
}

// Runs `f` on the tensors' device without the interpreter lock; its code as a
// Python int.
template <typename F>
PyObject *run(const Call &c, F f) {
  int rc;
  {
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
  }
  return PyLong_FromLong(rc);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// No C++ exception crosses into the interpreter.
template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

constexpr int kNine[9] = {1, 2, 3, 4, 5, 6, 7, 8, 9};

PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c;
    if (!count(n, 10) || !tensors(a, kNine, 9, 0, &c)) return nullptr;
    return run(c, [&] {
      return attn_sink_cache_append_fp8(c.p[0], c.p[1], c.p[2], c.p[3], c.p[4], c.p[5], c.p[6], c.p[7], c.p[8], c.stream);
    });
  });
}

PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Call c;
    if (!count(n, 10) || !tensors(a, kNine, 9, 0, &c)) return nullptr;
    return run(c, [&] {
      return attn_sink_cache_read_fp8(c.p[0], c.p[1], c.p[2], c.p[3], c.p[4], c.p[5], c.p[6], c.p[7], c.p[8], c.stream);
    });
  });
}

// (stream, q, kpages, vpages, kscales, vscales, block_table, seqlens, sinks, window, scale, out)
PyObject *decode_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    static constexpr int at[9] = {1, 2, 3, 4, 5, 6, 7, 8, 11};
    Call c;
    int32_t window;
    float scale;
    if (!count(n, 12) || !tensors(a, at, 9, 0, &c) || !as_int32(a[9], &window) || !as_float(a[10], &scale))
      return nullptr;
    return run(c, [&] {
      return attn_sink_decode_paged_fp8(c.p[0], c.p[1], c.p[2], c.p[3], c.p[4], c.p[5], c.p[6], c.p[7], window, scale,
                                        c.p[8], c.stream);
    });
  });
}

// (stream, q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, sinks, window, scale, out, lse or None)
PyObject *fwd_extend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    static constexpr int at[8] = {1, 2, 3, 4, 5, 7, 10, 11};
    Call c;
    int32_t max_q, window;
    float scale;
    if (!count(n, 12) || !tensors(a, at, 8, 1u << 7, &c) || !as_int32(a[6], &max_q) || !as_int32(a[8], &window) ||
        !as_float(a[9], &scale))
      return nullptr;
    return run(c, [&] {
      return attn_sink_fwd_extend(c.p[0], c.p[1], c.p[2], c.p[3], c.p[4], max_q, c.p[5], window, scale, c.p[6], c.p[7],
                                  c.stream);
    });
  });
}

// (stream, q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, sinks, window, scale, terms, out, lse or None)
PyObject *fwd_extend_terms(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    static constexpr int at[8] = {1, 2, 3, 4, 5, 7, 11, 12};
    Call c;
    int32_t max_q, window, terms;
    float scale;
    if (!count(n, 13) || !tensors(a, at, 8, 1u << 7, &c) || !as_int32(a[6], &max_q) || !as_int32(a[8], &window) ||
        !as_float(a[9], &scale) || !as_int32(a[10], &terms))
      return nullptr;
    return run(c, [&] {
      return attn_sink_fwd_extend_terms(c.p[0], c.p[1], c.p[2], c.p[3], c.p[4], max_q, c.p[5], window, scale, terms,
                                        c.p[6], c.p[7], c.stream);
    });
  });
}

// (METH_FASTCALL functions have a signature of their own)
PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"cache_append", fast(cache_append), METH_FASTCALL, nullptr},
    {"cache_read", fast(cache_read), METH_FASTCALL, nullptr},
    {"decode_paged", fast(decode_paged), METH_FASTCALL, nullptr},
    {"fwd_extend", fast(fwd_extend), METH_FASTCALL, nullptr},
    {"fwd_extend_terms", fast(fwd_extend_terms), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (built_for: the versions that the caller compares before it calls anything)
PyMODINIT_FUNC PyInit__binding(void) {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", ATTN_SINK_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
