// The Python functions of the batched serving operators (module _mktorch):
// paged_append, paged_attention and matvec_q4 on torch tensors.
//
// A decode step calls these once a layer and more, on kernels of a few
// microseconds, so the checks of a call's tensors and the filling of its C
// struct are done here and not in Python: with ctypes they took 13 us
// (paged_append) and 8 us (matvec_q4) of a call on the host, several times the
// kernels.  Nothing is kept between calls.  Everything that runs on the GPU is
// behind the C ABI of include/mk.h.
//
// Each check_* function makes the checks of its operator alone and returns the
// bytes of the C struct it would pass; the tensors may then be anywhere.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <exception>
#include <optional>
#include <string>
#include <utility>

#include "../../include/mk.h"

namespace {

struct Bad {            // a ValueError
  std::string what;
};
struct Raised {};       // a Python exception that is already set
struct Failed {         // an MKError
  int code;
  const char *what;
};

void need(bool ok, const char *what) {
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
const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!o || !THPVariable_Check(o)) throw Bad{std::string(name) + " must be a tensor"};
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    throw Bad{std::string(name) + " requires grad, and this operator has no gradient: call it under torch.no_grad()"};
  return t;
}

// what a call has written counts as changed for autograd graphs that saved it
void changed(PyObject *o) {
  if (!o) return;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

long integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int type_of(c10::ScalarType t) { return t == at::kFloat ? MK_F32 : MK_BF16; }

int32_t small(int64_t n, const char *name) {
  if (n > INT32_MAX) throw Bad{std::string(name) + " is too large"};
  return static_cast<int32_t>(n);
}

// the address of an optional contiguous [n] tensor
void *vector(PyObject *o, const char *name, c10::ScalarType type, int64_t n, const c10::Device &dev) {
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

int64_t common(int64_t a, int64_t b) {
  while (b) std::swap(a %= b, b);
  return a;
}

// Whether two tensors certainly share no byte: one lies behind the other, or, modulo what the strides of `cut` and more
// have in common, what lies between them does (rows of one buffer, heads of one row, slots of one page).
bool disjoint(const Region &a, const Region &b) {
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
Region written(const at::Tensor &t, const char *name, int64_t inner) {
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
int64_t step(const at::Tensor &t, int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// row and head strides of [n][heads][d]: the last dimension contiguous, every row on 16 bytes
void heads(const at::Tensor &t, const char *name, int64_t n, int64_t d, int64_t h, c10::ScalarType type, const c10::Device &dev,
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

bool on16(const at::Tensor &t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }

mk_paged_kv cache(PyObject *ko, PyObject *vo, PyObject *to, PyObject *kso, PyObject *vso, bool on_device, c10::Device *device) {
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
void enqueue(const char *what, F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call();
  Py_END_ALLOW_THREADS;
  if (rc != MK_OK) throw Failed{rc, what};
}

template <class S>
PyObject *bytes_of(const S &s) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&s), sizeof(S));
}

PyObject *given(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// ---- paged_append -----------------------------------------------------------------

enum { A_K, A_V, A_KC, A_VC, A_TABLE, A_SLOTS, A_SEQS, A_Q, A_QOUT, A_ROPE, A_POS, A_SECTIONS, A_INTER, A_QN, A_KN, A_EPS, A_KS, A_VS,
       A_STATUS, A_STREAM };
Signature append_sig = {"paged_append", 6, 6, 20,
                        {"k", "v", "k_cache", "v_cache", "table", "slots", "seqs", "q", "q_out", "rope", "positions", "mrope_sections",
                         "mrope_interleaved", "q_norm", "k_norm", "eps", "k_scale", "v_scale", "status", "stream"}, {}};

mk_append_args append_args(PyObject *const *o, const mk_paged_kv &kv, const c10::Device &dev) {
  const at::Tensor &k_cache = THPVariable_Unpack(o[A_KC]), &v_cache = THPVariable_Unpack(o[A_VC]);
  const Region kc = written(k_cache, "k_cache", kv.head_dim), vc = written(v_cache, "v_cache", kv.head_dim);
  need(disjoint(kc, vc), "k_cache and v_cache must not overlap: they are written");
  const at::Tensor &k = tensor(o[A_K], "k"), &v = tensor(o[A_V], "v");
  const auto type = k.scalar_type();
  need(type == at::kFloat || type == at::kBFloat16, "k must be fp32 or bf16");
  need(k.device() == dev, "k and the cache must be on the same device");
  need(k.dim() == 3, "k must be [rows][heads][head_dim]");
  const int64_t n = k.size(0), d = kv.head_dim;
  mk_append_args a = {};
  a.n = small(n, "k");
  a.dtype = type_of(type);
  heads(k, "k", n, d, kv.n_kv_heads, type, dev, &a.k_row, &a.k_head);
  heads(v, "v", n, d, kv.n_kv_heads, type, dev, &a.v_row, &a.v_head);
  a.k = k.data_ptr();
  a.v = v.data_ptr();
  if (o[A_Q]) {
    const at::Tensor &q = tensor(o[A_Q], "q");
    heads(q, "q", n, d, 0, type, dev, &a.q_row, &a.q_head);
    a.n_q_heads = small(q.size(1), "q");
    a.q = q.data_ptr();
    if (o[A_QOUT]) {
      const at::Tensor &out = tensor(o[A_QOUT], "q_out");
      heads(out, "q_out", n, d, a.n_q_heads ? a.n_q_heads : -1, type, dev, &a.out_row, &a.out_head);
      need(out.size(1) == q.size(1), "q_out must have q's heads");
      const Region r = written(out, "q_out", d), of_q(q, d);
      need(r == of_q || disjoint(r, of_q), "q_out must be q itself or not overlap it");
      need(disjoint(r, Region(k, d)) && disjoint(r, Region(v, d)) && disjoint(r, kc) && disjoint(r, vc),
           "q_out must not overlap k, v or the cache");
      a.q_out = out.data_ptr();
    }
  } else {
    need(!o[A_QOUT], "q_out needs q");
  }
  need(o[A_SLOTS], "slots are needed");
  a.slots = static_cast<const int32_t *>(vector(o[A_SLOTS], "slots", at::kInt, n, dev));
  need(o[A_SEQS] || n <= kv.table_rows, "without seqs, row i is sequence i: the table needs a row for each");
  a.seqs = static_cast<const int32_t *>(vector(o[A_SEQS], "seqs", at::kInt, n, dev));
  if (o[A_ROPE]) {
    const at::Tensor &r = tensor(o[A_ROPE], "rope");
    need(r.dim() == 3 && r.size(1) == d / 2 && r.size(2) == 2 && r.scalar_type() == at::kFloat && r.is_contiguous() && r.device() == dev && on16(r),
         "rope must be the contiguous fp32 [rows][head_dim / 2][2] of rope_table");
    need(r.size(0) > 0, "rope has no rows");                 // (its address would be that of no table: no rotation)
    a.rope = static_cast<const float *>(r.data_ptr());
    a.rope_rows = small(r.size(0), "rope");
    if (o[A_SECTIONS]) {
      PyObject *seq = PySequence_Fast(o[A_SECTIONS], "mrope_sections must be three counts");
      if (!seq) throw Raised{};
      const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
      long v[3] = {-1, -1, -1};
      for (Py_ssize_t i = 0; i < len && i < 3; ++i) v[i] = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
      Py_DECREF(seq);
      if (PyErr_Occurred()) throw Raised{};
      need(len == 3 && v[0] >= 0 && v[1] >= 0 && v[2] >= 0 && v[0] <= d && v[1] <= d && v[2] <= d && v[0] + v[1] + v[2] == d / 2,
           "mrope_sections must be three counts that sum to head_dim / 2");
      need(o[A_POS], "mrope_sections need positions");
      const at::Tensor &p = tensor(o[A_POS], "positions");
      need(p.dim() == 2 && p.size(0) == 3 && p.size(1) == n && p.scalar_type() == at::kInt && p.device() == dev && p.is_contiguous(),
           "positions must be contiguous int32 [3][n] with mrope_sections");
      int inter = 0;
      if (o[A_INTER]) inter = PyObject_IsTrue(o[A_INTER]);
      if (inter < 0) throw Raised{};
      a.rope_mode = inter ? 2 : 1;
      for (int i = 0; i < 3; ++i) a.mrope_sections[i] = static_cast<int32_t>(v[i]);
      a.positions = static_cast<const int32_t *>(p.data_ptr());
    } else {
      a.positions = static_cast<const int32_t *>(vector(o[A_POS], "positions", at::kInt, n, dev));
    }
  } else {
    need(!o[A_POS] && !o[A_SECTIONS], "positions need a rope table");
  }
  a.q_norm = vector(o[A_QN], "q_norm", at::kBFloat16, d, dev);
  a.k_norm = vector(o[A_KN], "k_norm", at::kBFloat16, d, dev);
  need(reinterpret_cast<uintptr_t>(a.q_norm) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k_norm) % 16 == 0, "q_norm and k_norm must start on 16 bytes");
  a.rms_eps = o[A_EPS] ? static_cast<float>(number(o[A_EPS])) : 1e-6f;
  need(a.rms_eps >= 0.f, "eps must not be negative");
  a.status = static_cast<int32_t *>(vector(o[A_STATUS], "status", at::kInt, 1, dev));
  return a;
}

PyObject *paged_append(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[A_KC], o[A_VC], o[A_TABLE], o[A_KS], o[A_VS], true, &dev);
  mk_append_args a = append_args(o, kv, dev);
  const Launch on(dev, o[A_STREAM]);
  at::Tensor made;
  if (o[A_Q] && !o[A_QOUT]) {
    const at::Tensor &q = THPVariable_Unpack(o[A_Q]);
    made = at::empty(q.sizes(), q.options());
    a.q_out = made.data_ptr();
    a.out_row = made.stride(0);
    a.out_head = made.stride(1);
  }
  if (a.n) {
    enqueue("mk_paged_append", [&] { return mk_paged_append(&kv, &a, on.stream); });
    for (int i : {A_KC, A_VC, A_QOUT, A_STATUS}) changed(o[i]);
  }
  if (!o[A_Q]) Py_RETURN_NONE;
  return o[A_QOUT] ? given(o[A_QOUT]) : THPVariable_Wrap(made);
}

PyObject *check_append(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[A_KC], o[A_VC], o[A_TABLE], o[A_KS], o[A_VS], false, &dev);
  return bytes_of(append_args(o, kv, dev));
}

// ---- paged_attention ----------------------------------------------------------------

enum { T_Q, T_KC, T_VC, T_TABLE, T_LENGTHS, T_SCALE, T_WINDOW, T_KS, T_VS, T_OUT, T_LSE, T_STATUS, T_STREAM };
Signature attention_sig = {"paged_attention", 5, 5, 13,
                           {"q", "k_cache", "v_cache", "table", "lengths", "scale", "window", "k_scale", "v_scale", "out", "lse", "status", "stream"}, {}};

mk_attention_args attention_args(PyObject *const *o, const mk_paged_kv &kv, const c10::Device &dev) {
  const at::Tensor &q = tensor(o[T_Q], "q");
  const auto type = q.scalar_type();
  need(type == at::kFloat || type == at::kBFloat16, "q must be fp32 or bf16");
  need(q.device() == dev, "q and the cache must be on the same device");
  need(q.dim() == 3, "q must be [rows][heads][head_dim]");
  const int64_t n = q.size(0), hq = q.size(1), d = kv.head_dim;
  mk_attention_args a = {};
  a.n = small(n, "q");
  a.dtype = type_of(type);
  heads(q, "q", n, d, 0, type, dev, &a.q_row, &a.q_head);
  if (hq < 1 || hq % kv.n_kv_heads) throw Bad{"q must have a multiple of the cache's " + std::to_string(kv.n_kv_heads) + " heads"};
  need(n <= kv.table_rows, "the table needs a row for each row of q");
  a.n_q_heads = small(hq, "q");
  a.q = q.data_ptr();
  if (o[T_OUT]) {
    const at::Tensor &out = tensor(o[T_OUT], "out");
    heads(out, "out", n, d, hq, type, dev, &a.out_row, &a.out_head);
    const Region r = written(out, "out", d), of_q(q, d);
    need(r == of_q || disjoint(r, of_q), "out must be q itself or not overlap it");
    need(disjoint(r, Region(THPVariable_Unpack(o[T_KC]), d)) && disjoint(r, Region(THPVariable_Unpack(o[T_VC]), d)), "out must not overlap the cache");
    a.out = out.data_ptr();
  }
  if (o[T_LSE]) {
    const at::Tensor &lse = tensor(o[T_LSE], "lse");
    need(lse.dim() == 2 && lse.size(0) == n && lse.size(1) == hq && lse.scalar_type() == at::kFloat && lse.device() == dev && lse.is_contiguous(),
         "lse must be a contiguous fp32 [rows][heads] on q's device");
    const Region r(lse, hq);
    need(disjoint(r, Region(q, d)) && (!o[T_OUT] || disjoint(r, Region(THPVariable_Unpack(o[T_OUT]), d))), "lse must not overlap q or out");
    a.lse = static_cast<float *>(lse.data_ptr());
  }
  need(o[T_LENGTHS], "lengths are needed");
  a.lengths = static_cast<const int32_t *>(vector(o[T_LENGTHS], "lengths", at::kInt, n, dev));
  const long window = o[T_WINDOW] ? integer(o[T_WINDOW]) : 0;
  need(window >= 0, "window must be 0 (all) or the number of last tokens");
  a.window = window > INT32_MAX ? INT32_MAX : static_cast<int32_t>(window);
  a.scale = o[T_SCALE] ? static_cast<float>(number(o[T_SCALE])) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  need(std::isfinite(a.scale), "scale must be finite");
  a.status = static_cast<int32_t *>(vector(o[T_STATUS], "status", at::kInt, 1, dev));
  return a;
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

PyObject *paged_attention(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[T_KC], o[T_VC], o[T_TABLE], o[T_KS], o[T_VS], true, &dev);
  mk_attention_args a = attention_args(o, kv, dev);
  const Launch on(dev, o[T_STREAM]);
  at::Tensor made;
  if (!o[T_OUT]) {
    const at::Tensor &q = THPVariable_Unpack(o[T_Q]);
    made = at::empty(q.sizes(), q.options());
    a.out = made.data_ptr();
    a.out_row = made.stride(0);
    a.out_head = made.stride(1);
  }
  if (a.n) {
    Memory workspace;
    try {
      enqueue("mk_paged_attention", [&] { return mk_paged_attention_ask(&kv, &a, &Memory::ask, &workspace, on.stream); });
    } catch (const Failed &) {
      if (workspace.error) std::rethrow_exception(workspace.error);
      throw;
    }
    for (int i : {T_OUT, T_LSE, T_STATUS}) changed(o[i]);
  }
  return o[T_OUT] ? given(o[T_OUT]) : THPVariable_Wrap(made);
}

PyObject *check_attention(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[T_KC], o[T_VC], o[T_TABLE], o[T_KS], o[T_VS], false, &dev);
  return bytes_of(attention_args(o, kv, dev));
}

// ---- matvec_q4 ------------------------------------------------------------------------

enum { M_X, M_CODES, M_SCALES, M_ZEROS, M_RESIDUAL, M_OUT, M_STREAM };
Signature matvec_sig = {"matvec_q4", 3, 3, 7, {"x", "codes", "scales", "zeros", "residual", "out", "stream"}, {}};

mk_matvec_q4_args matvec_args(PyObject *const *o, bool on_device, c10::Device *device) {
  const at::Tensor &x = tensor(o[M_X], "x"), &codes = tensor(o[M_CODES], "codes"), &scales = tensor(o[M_SCALES], "scales");
  const auto type = x.scalar_type();
  const c10::Device dev = x.device();
  need(x.dim() == 2 && (type == at::kFloat || type == at::kBFloat16), "x must be [rows][k] of fp32 or bf16");
  need(!on_device || dev.is_cuda(), "x must be on a CUDA device");
  const int64_t m = x.size(0), k = x.size(1);
  need(codes.dim() == 2 && codes.size(1) * 2 == k && k > 0 && codes.scalar_type() == at::kByte && codes.is_contiguous() && codes.device() == dev && on16(codes),
       "codes must be contiguous uint8 [n][k / 2] on x's device, from 16 bytes on");
  const int64_t n = codes.size(0);
  need(scales.dim() == 2 && scales.size(0) == n && scales.scalar_type() == at::kBFloat16 && scales.is_contiguous() && scales.device() == dev &&
           scales.size(1) > 0 && k % scales.size(1) == 0,
       "scales must be contiguous bf16 [n][k / group] on x's device");
  const int64_t group = k / scales.size(1);
  need(group == 32 || group == 64 || group % 128 == 0, "the group must be 32, 64 or a multiple of 128");
  mk_matvec_q4_args a = {};
  a.m = small(m, "x"), a.n = small(n, "codes"), a.k = small(k, "x"), a.group = small(group, "group");
  a.dtype = type_of(type);
  need(!m || (x.stride(1) == 1 && step(x, 0) % (type == at::kFloat ? 4 : 8) == 0 && on16(x)),
       "x's last dimension must be contiguous and every row start on 16 bytes");
  a.x = x.data_ptr();
  a.x_row = step(x, 0);
  a.codes = codes.data_ptr();
  a.scales = scales.data_ptr();
  if (o[M_ZEROS]) {
    const at::Tensor &z = tensor(o[M_ZEROS], "zeros");
    need(z.sizes() == scales.sizes() && z.scalar_type() == at::kByte && z.is_contiguous() && z.device() == dev, "zeros must be contiguous uint8 of scales' shape");
    a.zeros = static_cast<const uint8_t *>(z.data_ptr());
  }
  for (int i : {M_RESIDUAL, M_OUT}) {
    if (!o[i]) continue;
    const at::Tensor &t = tensor(o[i], i == M_OUT ? "out" : "residual");
    if (t.dim() != 2 || t.size(0) != m || t.size(1) != n || t.scalar_type() != type || t.device() != dev || (t.stride(1) != 1 && n > 1))
      throw Bad{std::string(i == M_OUT ? "out" : "residual") + " must be [" + std::to_string(m) + "][" + std::to_string(n) + "] of x's dtype on its device, rows contiguous"};
    if (i == M_OUT) {
      const Region r = written(t, "out", n);
      need(disjoint(r, Region(x, k)), "out must not be x or overlap it: x is read until the last of out is written");
      if (o[M_RESIDUAL]) {
        const Region of(THPVariable_Unpack(o[M_RESIDUAL]), n);
        need(r == of || disjoint(r, of), "out must be residual itself or not overlap it");
      }
      a.y = t.data_ptr(), a.y_row = step(t, 0);
    } else a.residual = t.data_ptr(), a.residual_row = step(t, 0);
  }
  *device = dev;
  return a;
}

PyObject *matvec_q4(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  mk_matvec_q4_args a = matvec_args(o, true, &dev);
  const Launch on(dev, o[M_STREAM]);
  at::Tensor made;
  if (!o[M_OUT]) {
    made = at::empty({a.m, a.n}, THPVariable_Unpack(o[M_X]).options());
    a.y = made.data_ptr();
    a.y_row = a.n;
  }
  if (a.m && a.n) {
    enqueue("mk_matvec_q4", [&] { return mk_matvec_q4(&a, on.stream); });
    changed(o[M_OUT]);
  }
  return o[M_OUT] ? given(o[M_OUT]) : THPVariable_Wrap(made);
}

PyObject *check_matvec(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(matvec_args(o, false, &dev));
}

// ---- a cache's struct (Decoder.export_kv) -------------------------------------------------

Signature cache_sig = {"paged_kv", 3, 3, 6, {"k_cache", "v_cache", "table", "k_scale", "v_scale", "on_device"}, {}};

PyObject *paged_kv(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(cache(o[0], o[1], o[2], o[3], o[4], !o[5] || PyObject_IsTrue(o[5]), &dev));
}

// ---- the module ---------------------------------------------------------------------------

PyObject *mk_error = nullptr;      // _binding.MKError

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

PyMethodDef methods[] = {
    method<&append_sig, &paged_append>("paged_append", R"(paged_append(k, v, k_cache, v_cache, table, slots, *, seqs=None, q=None, q_out=None, rope=None, positions=None, mrope_sections=None, mrope_interleaved=False, q_norm=None, k_norm=None, eps=1e-06, k_scale=None, v_scale=None, status=None, stream=None)
--

``mk_paged_append``: write ``k`` and ``v`` [n][kv heads][d] (fp32 or bf16, any
row and head strides on 16 bytes) to their slots of the paged cache, with
RMSNorm by the gains ``q_norm`` / ``k_norm`` (bf16 [d]) and the rotation by
``rope`` (``rope_table``) on the way, and return the queries ``q`` treated alike
(into ``q_out``, which may be ``q`` but overlap no other tensor of the call; a new
tensor by default; None without ``q``).

``k_cache`` and ``v_cache`` are [n_pages][kv heads][page_size][d] of bf16 or
float8_e4m3fn (equal strides, the first three dimensions in any order in
memory); ``k_scale`` and ``v_scale``, fp32 [kv heads], are what the values of a
float8_e4m3fn cache stand in units of.  ``table`` is int32 [sequences][pages].
``slots`` int32 [n] are token indices in each row's sequence: row i of
``table``, or row ``seqs[i]``.  A negative slot marks a padding row: nothing
of it is written, in ``q_out`` neither.  ``positions`` int32 [n] rotate by
something else than the slot; with ``mrope_sections`` they are three streams
[3][n] (``mrope_interleaved`` as ``rope_mode`` 2).  No two rows of a call may
name the same slot of the cache.  What the device finds wrong goes to
``status`` (int32 [1], zeroed by the caller; ``check_status``).)"),
    method<&attention_sig, &paged_attention>("paged_attention", R"(paged_attention(q, k_cache, v_cache, table, lengths, *, scale=None, window=0, k_scale=None, v_scale=None, out=None, lse=None, status=None, stream=None)
--

``mk_paged_attention``: attention of one new token per row, ``q`` [n][heads][d]
(fp32 or bf16), over the first ``lengths[i]`` (the last ``window`` of them,
if not 0) tokens of row i of ``table``; the cache as for ``paged_append``.
Returns ``out`` like ``q`` (it may be ``q``, but not overlap it otherwise);
``lse`` fp32 [n][heads] receives the log of each softmax's sum.  ``scale`` is 1 / sqrt(d) by default.  A row of
length 0 gives zeros and -inf, one of negative length is left as it was.)"),
    method<&matvec_sig, &matvec_q4>("matvec_q4", R"(matvec_q4(x, codes, scales, *, zeros=None, residual=None, out=None, stream=None)
--

``mk_matvec_q4``: ``x`` [rows][k] (fp32 or bf16) times the transpose of the
4-bit weights of ``quantize_q4``, plus ``residual`` [rows][n] (which may be
``out``; ``out`` must not overlap ``x``).  ``codes`` uint8 [n][k / 2], ``scales`` bf16 and ``zeros`` uint8 (8
everywhere if None) [n][k / group].)"),
    method<&append_sig, &check_append>("check_append", "The checks of paged_append; the bytes of its mk_append_args."),
    method<&attention_sig, &check_attention>("check_attention", "The checks of paged_attention; the bytes of its mk_attention_args."),
    method<&matvec_sig, &check_matvec>("check_matvec", "The checks of matvec_q4; the bytes of its mk_matvec_q4_args."),
    method<&cache_sig, &paged_kv>("paged_kv", "The checks of a paged cache; the bytes of its mk_paged_kv."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mktorch", "The batched serving operators on torch tensors.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mktorch() {
  for (Signature *s : {&append_sig, &attention_sig, &matvec_sig, &cache_sig}) s->intern();
  PyObject *binding = PyImport_ImportModule("persistent_transformer_megakernel_gb300._binding");
  if (!binding) return nullptr;
  mk_error = PyObject_GetAttrString(binding, "MKError");
  Py_DECREF(binding);
  return mk_error ? PyModule_Create(&module) : nullptr;
}
