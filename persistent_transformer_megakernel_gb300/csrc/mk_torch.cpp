// The Python functions of the batched serving operators (module _mktorch) on torch
// tensors: paged_append, paged_attention and matvec_q4 here, the operators of prompts
// and of a step's two ends in mk_torch_prompts.h, what both share in mk_torch.h.
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
#include "mk_torch.h"
#include "mk_torch_prompts.h"

namespace mkt {

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
    made = fresh(q.sizes(), q.scalar_type(), q);
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

enum { T_Q, T_KC, T_VC, T_TABLE, T_LENGTHS, T_SCALE, T_WINDOW, T_SINKS, T_KS, T_VS, T_OUT, T_LSE, T_STATUS, T_STREAM };
Signature attention_sig = {"paged_attention", 5, 5, 14,
                           {"q", "k_cache", "v_cache", "table", "lengths", "scale", "window", "sinks", "k_scale", "v_scale", "out", "lse", "status", "stream"}, {}};

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
  const long sinks = o[T_SINKS] ? integer(o[T_SINKS]) : 0;
  need(sinks >= 0, "sinks must not be negative");
  a.sinks = sinks > INT32_MAX ? INT32_MAX : static_cast<int32_t>(sinks);
  a.scale = o[T_SCALE] ? static_cast<float>(number(o[T_SCALE])) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  need(std::isfinite(a.scale), "scale must be finite");
  a.status = static_cast<int32_t *>(vector(o[T_STATUS], "status", at::kInt, 1, dev));
  return a;
}

PyObject *paged_attention(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[T_KC], o[T_VC], o[T_TABLE], o[T_KS], o[T_VS], true, &dev);
  mk_attention_args a = attention_args(o, kv, dev);
  const Launch on(dev, o[T_STREAM]);
  at::Tensor made;
  if (!o[T_OUT]) {
    const at::Tensor &q = THPVariable_Unpack(o[T_Q]);
    made = fresh(q.sizes(), q.scalar_type(), q);
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
    const at::Tensor &x = THPVariable_Unpack(o[M_X]);
    made = fresh({a.m, a.n}, x.scalar_type(), x);
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
    method<&attention_sig, &paged_attention>("paged_attention", R"(paged_attention(q, k_cache, v_cache, table, lengths, *, scale=None, window=0, sinks=0, k_scale=None, v_scale=None, out=None, lse=None, status=None, stream=None)
--

``mk_paged_attention``: attention of one new token per row, ``q`` [n][heads][d]
(fp32 or bf16), over the first ``lengths[i]`` tokens of row i of ``table`` (with
a ``window``, not 0, the last ``window`` of them and the first ``sinks``); the
cache as for ``paged_append``.
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

}  // namespace mkt

PyMODINIT_FUNC PyInit__mktorch() {
  using namespace mkt;
  for (Signature *s : {&append_sig, &attention_sig, &matvec_sig, &cache_sig}) s->intern();
  prompts::intern();
  PyObject *binding = PyImport_ImportModule("persistent_transformer_megakernel_gb300._binding");
  if (!binding) return nullptr;
  mk_error = PyObject_GetAttrString(binding, "MKError");
  Py_DECREF(binding);
  if (!mk_error) return nullptr;
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddFunctions(m, prompts::methods) < 0) Py_CLEAR(m);
  return m;
}
