// What the Python functions of the module _mktorch share: the arguments of a call, the checks of its tensors against
// what the kernels read and write, its stream and workspace, and its errors.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <exception>
#include <optional>
#include <string>
#include <utility>

#include "../../include/mk.h"

namespace mkt {

struct Bad {            // a ValueError
  std::string what;
};
struct Raised {};       // a Python exception that is already set
struct Failed {         // an MKError
  int code;
  const char *what;
};

inline void need(bool ok, const char *what) {
  if (!ok) throw Bad{what};
}

// ---- arguments ---------------------------------------------------------------

constexpr int kMaxArgs = 24;

struct Signature {
  const char *function;
  int required, positional, count;
  const char *names[kMaxArgs];
  PyObject *interned[kMaxArgs];

  void intern() {
    for (int i = 0; i < count; ++i) interned[i] = PyUnicode_InternFromString(names[i]);
  }
  int find(PyObject *name) const {
    for (int i = 0; i < count; ++i)
      if (interned[i] == name) return i;
    for (int i = 0; i < count; ++i)
      if (PyUnicode_Compare(interned[i], name) == 0) return i;
    return -1;
  }
  void parse(PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames, PyObject **out) const {
    for (int i = 0; i < count; ++i) out[i] = nullptr;
    if (nargs > positional) {
      PyErr_Format(PyExc_TypeError, "%s() takes %d positional arguments but %zd were given", function, positional, nargs);
      throw Raised{};
    }
    for (Py_ssize_t i = 0; i < nargs; ++i) out[i] = args[i];
    const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t i = 0; i < nkw; ++i) {
      PyObject *name = PyTuple_GET_ITEM(kwnames, i);
      const int at = find(name);
      if (at < 0 || out[at]) {
        PyErr_Format(PyExc_TypeError, at < 0 ? "%s() got an unexpected keyword argument '%U'" : "%s() got multiple values for argument '%U'",
                     function, name);
        throw Raised{};
      }
      out[at] = args[nargs + i];
    }
    for (int i = 0; i < count; ++i) {
      if (out[i] == nullptr && i < required) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", function, names[i]);
        throw Raised{};
      }
      if (out[i] == Py_None) out[i] = nullptr;             // None stands for what is not given
    }
  }
};

// a tensor that autograd does not follow: none of the operators has a backward, and none may be left out unnoticed
inline const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!o || !THPVariable_Check(o)) throw Bad{std::string(name) + " must be a tensor"};
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    throw Bad{std::string(name) + " requires grad, and this operator has no gradient: call it under torch.no_grad()"};
  if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    throw Bad{std::string(name) + " has a tangent (forward-mode differentiation), and this operator has none: unpack_dual it first"};
  return t;
}

// what a call has written counts as changed for autograd graphs that saved it
inline void changed(PyObject *o) {
  if (!o) return;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

inline double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

inline long integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

inline int type_of(c10::ScalarType t) { return t == at::kFloat ? MK_F32 : MK_BF16; }

inline int32_t small(int64_t n, const char *name) {
  if (n > INT32_MAX) throw Bad{std::string(name) + " is too large"};
  return static_cast<int32_t>(n);
}

// the address of an optional contiguous [n] tensor
inline void *vector(PyObject *o, const char *name, c10::ScalarType type, int64_t n, const c10::Device &dev) {
  if (!o) return nullptr;
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || t.device() != dev || !t.is_contiguous())
    throw Bad{std::string(name) + " must be a contiguous tensor [" + std::to_string(n) + "] of dtype " + c10::toString(type) + " on " + dev.str()};
  return t.data_ptr();
}

// ---- memory that is written --------------------------------------------------------

// A tensor's bytes: pieces of `inner` bytes at multiples of up to three strides (zero strides and dimensions of one
// element add none).
struct Region {
  uintptr_t at;
  int64_t inner, extent;       // of a piece, and from the first byte to the last
  int64_t size[3], stride[3];
  int dims = 0;

  Region(const at::Tensor &t, int64_t inner_elements) {
    const int64_t es = static_cast<int64_t>(t.element_size());
    at = reinterpret_cast<uintptr_t>(t.data_ptr());
    inner = extent = inner_elements * es;
    if (t.numel() == 0) inner = extent = 0;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) {
      if (t.size(i) <= 1 || t.stride(i) == 0) continue;
      size[dims] = t.size(i), stride[dims] = t.stride(i) * es;
      extent += (size[dims] - 1) * stride[dims];
      ++dims;
    }
  }
  // from the first byte to the last of what lies between multiples of strides of `cut` and more
  int64_t below(int64_t cut) const {
    int64_t e = inner;
    for (int i = 0; i < dims; ++i)
      if (stride[i] < cut) e += (size[i] - 1) * stride[i];
    return e;
  }
  bool operator==(const Region &o) const {
    if (at != o.at || inner != o.inner || dims != o.dims) return false;
    for (int i = 0; i < dims; ++i)
      if (size[i] != o.size[i] || stride[i] != o.stride[i]) return false;
    return true;
  }
};

inline int64_t common(int64_t a, int64_t b) {
  while (b) std::swap(a %= b, b);
  return a;
}

// Whether two tensors certainly share no byte: one lies behind the other, or, modulo what the strides of `cut` and more
// have in common, what lies between them does (rows of one buffer, heads of one row, slots of one page).
inline bool disjoint(const Region &a, const Region &b) {
  if (a.extent == 0 || b.extent == 0 || a.at + a.extent <= b.at || b.at + b.extent <= a.at) return true;
  for (const Region *r : {&a, &b})
    for (int i = 0; i < r->dims; ++i) {
      const int64_t cut = r->stride[i];
      int64_t g = 0;
      for (const Region *o : {&a, &b})
        for (int j = 0; j < o->dims; ++j)
          if (o->stride[j] >= cut) g = common(o->stride[j], g);
      const int64_t from = b.at >= a.at ? static_cast<int64_t>((b.at - a.at) % g) : (g - static_cast<int64_t>((a.at - b.at) % g)) % g;
      if (a.below(cut) <= from && from + b.below(cut) <= g) return true;
    }
  return false;
}

// a tensor that is written: no two of its elements may be the same memory
inline Region written(const at::Tensor &t, const char *name, int64_t inner) {
  for (int64_t i = 0; i + 1 < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) throw Bad{std::string(name) + " must not be expanded: it is written"};
  const Region r(t, inner);
  int64_t done = 0;                                        // every stride beyond what the smaller ones reach
  for (int k = 0; k < r.dims; ++k) {
    int64_t next = INT64_MAX;
    int equal = 0;
    for (int i = 0; i < r.dims; ++i) {
      if (r.stride[i] > done && r.stride[i] < next) next = r.stride[i], equal = 1;
      else if (r.stride[i] == next) ++equal;
    }
    if (next == INT64_MAX) break;
    if (equal > 1 || next < r.below(next)) throw Bad{std::string(name) + " must not overlap itself: it is written"};
    done = next;
  }
  return r;
}

// a stride that is used: 0 of a dimension of one element, whose stride torch leaves as it came
inline int64_t step(const at::Tensor &t, int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// row and head strides of [n][heads][d]: the last dimension contiguous, every row on 16 bytes
inline void heads(const at::Tensor &t, const char *name, int64_t n, int64_t d, int64_t h, c10::ScalarType type, const c10::Device &dev,
           int64_t *row, int64_t *head) {
  if (t.dim() != 3 || t.scalar_type() != type || t.device() != dev)
    throw Bad{std::string(name) + " must be [rows][heads][head_dim] of dtype " + c10::toString(type) + " on " + dev.str()};
  const auto s = t.sizes();
  if (s[0] != n || s[2] != d || (h > 0 && s[1] != h))
    throw Bad{std::string(name) + " must have " + std::to_string(n) + " rows of " + (h > 0 ? std::to_string(h) + " " : "") +
              "heads of " + std::to_string(d) + " elements"};
  const int64_t unit = type == at::kFloat ? 4 : 8;
  *row = step(t, 0);
  *head = step(t, 1);
  if (n && (t.stride(2) != 1 || *row % unit || *head % unit || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16))
    throw Bad{std::string(name) + ": the last dimension must be contiguous and every row start on 16 bytes"};
}

inline bool on16(const at::Tensor &t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }

inline mk_paged_kv cache(PyObject *ko, PyObject *vo, PyObject *to, PyObject *kso, PyObject *vso, bool on_device, c10::Device *device) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache"), &table = tensor(to, "table");
  const auto type = k.scalar_type();
  const c10::Device dev = k.device();
  need(k.dim() == 4 && (type == at::kBFloat16 || type == at::kFloat8_e4m3fn),
       "k_cache must be [n_pages][n_kv_heads][page_size][head_dim] of bf16 or float8_e4m3fn");
  need(v.sizes() == k.sizes() && v.scalar_type() == type && v.device() == dev && v.stride(3) == k.stride(3) && step(v, 0) == step(k, 0) &&
           step(v, 1) == step(k, 1) && step(v, 2) == step(k, 2),
       "v_cache must have k_cache's shape, strides, dtype and device");
  need(!on_device || dev.is_cuda(), "the cache must be on a CUDA device");
  const auto s = k.sizes();
  const int64_t page = step(k, 0), head = step(k, 1), slot = step(k, 2);
  need(s[3] == 64 || s[3] == 128, "head_dim must be 64 or 128");
  const int64_t unit = type == at::kBFloat16 ? 8 : 16;
  need(s[0] > 0 && s[1] > 0 && s[2] > 0 && k.stride(3) == 1 && page % unit == 0 && head % unit == 0 && slot % unit == 0 && on16(k) && on16(v),
       "the cache's last dimension must be contiguous and every slot start on 16 bytes");
  need(table.dim() == 2 && table.scalar_type() == at::kInt && table.device() == dev && (table.stride(1) == 1 || table.size(1) <= 1),
       "table must be int32 [rows][pages] on the cache's device, its rows contiguous");
  need(!kso == !vso, "k_scale and v_scale go together");
  need(!kso || type == at::kFloat8_e4m3fn, "scales are for a float8_e4m3fn cache");
  mk_paged_kv c = {};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.dtype = type == at::kBFloat16 ? MK_BF16 : MK_E4M3;
  c.n_pages = small(s[0], "k_cache"), c.n_kv_heads = small(s[1], "k_cache"), c.page_size = small(s[2], "k_cache"), c.head_dim = static_cast<int32_t>(s[3]);
  c.page_stride = page, c.head_stride = head, c.slot_stride = s[2] > 1 ? slot : s[3];   // (slots one behind the other, if there is one)
  c.k_scale = static_cast<const float *>(vector(kso, "k_scale", at::kFloat, s[1], dev));
  c.v_scale = static_cast<const float *>(vector(vso, "v_scale", at::kFloat, s[1], dev));
  c.table = static_cast<const int32_t *>(table.data_ptr());
  c.table_rows = small(table.size(0), "table"), c.table_cols = small(table.size(1), "table");
  c.table_stride = table.stride(0);
  *device = dev;
  return c;
}

// ---- a call's stream ------------------------------------------------------------

// The device made current, and the stream of the call: the device's current one, or `stream` (a torch stream of that
// device), which is made current so that memory allocated for the call is its own.
struct Launch {
  c10::cuda::OptionalCUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  cudaStream_t stream = nullptr;

  Launch(const c10::Device &dev, PyObject *o) {
    if (o) {
      const c10::cuda::CUDAStream s = unpack(o);
      need(s.device() == dev, "stream must be one of the tensors' device");
      guard.emplace(s.unwrap());
      stream = s.stream();
    } else {
      device.set_device(dev);
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
  }
  static long field(PyObject *o, const char *name) {
    PyObject *v = PyObject_GetAttrString(o, name);
    if (!v) throw Raised{};
    const long n = PyLong_AsLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw Raised{};
    return n;
  }
  static c10::cuda::CUDAStream unpack(PyObject *o) {
    return c10::cuda::CUDAStream::unpack3(field(o, "stream_id"), static_cast<c10::DeviceIndex>(field(o, "device_index")),
                                          static_cast<c10::DeviceType>(field(o, "device_type")));
  }
};

template <class F>
inline void enqueue(const char *what, F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call();
  Py_END_ALLOW_THREADS;
  if (rc != MK_OK) throw Failed{rc, what};
}

template <class S>
inline PyObject *bytes_of(const S &s) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&s), sizeof(S));
}

inline PyObject *given(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// a workspace from torch's allocator, of the current device and stream; what it throws does not pass the C entry point
struct Memory {
  c10::DataPtr held;
  std::exception_ptr error;

  static void *ask(void *context, int64_t bytes) {
    Memory &m = *static_cast<Memory *>(context);
    try {
      m.held = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
    } catch (...) {
      m.error = std::current_exception();
    }
    return m.held.get();
  }
};

// A new tensor on the current device: at::empty's where something else has a part in that (deterministic mode may fill it,
// dispatch modes and profilers see it), else as it makes it without the way through the dispatcher (half a microsecond less
// a call).
inline at::Tensor fresh(c10::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
  if (at::globalContext().deterministicAlgorithms() || c10::impl::dispatch_mode_enabled() || at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION)) {
    at::Tensor t = at::empty(sizes, like.options().dtype(type));
    // (what a mode makes in its place may have no memory)
    need(t.device() == like.device() && (t.numel() == 0 || (t.has_storage() && t.storage().data())), "a dispatch mode made a result without memory on the tensors' device");
    return t;
  }
  return at::Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}

// ---- functions of the module ----------------------------------------------------------

static PyObject *mk_error = nullptr;   // _binding.MKError

template <Signature *SIG, PyObject *(*F)(PyObject *const *)>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames) {
  try {
    PyObject *o[kMaxArgs];
    SIG->parse(args, nargs, kwnames, o);
    return F(o);
  } catch (const Raised &) {
  } catch (const Bad &e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Failed &e) {
    if (PyObject *err = PyObject_CallFunction(mk_error, "is", e.code, e.what)) {
      PyErr_SetObject(mk_error, err);
      Py_DECREF(err);
    }
  } catch (...) {                                          // torch's own: out of memory among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

template <Signature *SIG, PyObject *(*F)(PyObject *const *)>
PyMethodDef method(const char *name, const char *doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&call<SIG, F>)), METH_FASTCALL | METH_KEYWORDS, doc};
}

}  // namespace mkt
