// The Python functions of the module _mktorch for what surrounds a batched step: paged_plan before it, prompts' attention
// and 8-bit products in it, adjust_logits behind it.  As in mk_torch.cpp, each check_* function makes an operator's checks
// alone and returns the bytes of its C struct.
#pragma once
#include "mk_torch.h"

namespace mkt {
namespace prompts {

// New results of a call that belong together, one behind the other in one allocation, each on 16 bytes: five tensors of an
// allocation each cost the host 1.3 us more (paged_plan 4.4 us a call, 5.7).
class Results {
 public:
  // room for a result, before the allocation
  void want(int64_t bytes) { bytes_ += (bytes + 15) / 16 * 16, any_ = true; }
  void allocate(const at::Tensor &like) {
    if (any_) memory_ = fresh({bytes_}, at::kByte, like);
  }
  // the next result, in the order of the wants
  at::Tensor take(c10::IntArrayRef sizes, at::ScalarType type) {
    const int64_t element = static_cast<int64_t>(c10::elementSize(type));
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(memory_.storage()), memory_.key_set(), c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl *impl = t.unsafeGetTensorImpl();
    impl->set_storage_offset(used_ / element);
    impl->set_sizes_contiguous(sizes);
    used_ += (t.numel() * element + 15) / 16 * 16;
    TORCH_INTERNAL_ASSERT(used_ <= bytes_);                // (nothing has been launched yet)
    return t;
  }

 private:
  at::Tensor memory_;
  int64_t bytes_ = 0, used_ = 0;
  bool any_ = false;
};
PyObject *of(PyObject *o, const at::Tensor &made) { return o ? given(o) : THPVariable_Wrap(made); }

// the address and row stride of an optional [n][columns] tensor whose rows are contiguous; columns < 0: any
const void *rows_of(PyObject *o, const char *name, c10::ScalarType type, int64_t n, int64_t columns, const c10::Device &dev, int64_t *stride, int64_t *found) {
  if (!o) return nullptr;
  const at::Tensor &t = tensor(o, name);
  if (t.dim() != 2 || t.scalar_type() != type || t.size(0) != n || (columns >= 0 && t.size(1) != columns) || t.device() != dev || (t.size(1) > 1 && t.stride(1) != 1))
    throw Bad{std::string(name) + " must be [" + std::to_string(n) + "][" + (columns >= 0 ? std::to_string(columns) : "any") + "] of dtype " +
              c10::toString(type) + " on " + dev.str() + ", its rows contiguous"};
  *stride = step(t, 0);
  if (found) *found = t.size(1);
  return t.data_ptr();
}

// ---- paged_plan ----------------------------------------------------------------------

enum { P_LENGTHS, P_TABLE, P_FREE, P_USED, P_PAGE, P_COUNTS, P_ROWS, P_SEQS, P_SLOTS, P_STARTS, P_TOTALS, P_USED_OUT, P_STATUS, P_STREAM };
Signature plan_sig = {"paged_plan", 5, 5, 14,
                      {"lengths", "table", "free", "used", "page_size", "counts", "rows", "seqs", "slots", "starts", "totals", "used_out", "status",
                       "stream"}, {}};

constexpr int kPlanOutputs[] = {P_SEQS, P_SLOTS, P_STARTS, P_TOTALS, P_USED_OUT};

mk_plan_args plan_args(PyObject *const *o, bool on_device, c10::Device *device) {
  const at::Tensor &lengths = tensor(o[P_LENGTHS], "lengths"), &table = tensor(o[P_TABLE], "table"), &free = tensor(o[P_FREE], "free");
  const c10::Device dev = lengths.device();
  need(!on_device || dev.is_cuda(), "lengths must be on a CUDA device");
  need(lengths.dim() == 1, "lengths must be int32 [sequences]");
  const int64_t n = lengths.size(0);
  need(free.dim() == 1, "free must be int32 [pages]");
  mk_plan_args a = {};
  a.n = small(n, "lengths");
  a.lengths = static_cast<const int32_t *>(vector(o[P_LENGTHS], "lengths", at::kInt, n, dev));
  need(table.dim() == 2 && table.scalar_type() == at::kInt && table.device() == dev && table.size(0) >= n && (table.stride(1) == 1 || table.size(1) <= 1),
       "table must be int32 [sequences or more][pages] on lengths' device, its rows contiguous");
  const Region of_table = written(table, "table", table.size(1));
  a.table = static_cast<int32_t *>(table.data_ptr());
  a.table_cols = small(table.size(1), "table");
  a.table_stride = step(table, 0);
  a.free_count = small(free.size(0), "free");
  a.free = static_cast<const int32_t *>(vector(o[P_FREE], "free", at::kInt, free.size(0), dev));
  need(o[P_USED], "used is needed");
  a.used = static_cast<const int32_t *>(vector(o[P_USED], "used", at::kInt, 1, dev));
  need(o[P_PAGE], "page_size is needed");
  const long page = integer(o[P_PAGE]);
  need(page >= 1 && page <= INT32_MAX, "page_size must be positive");
  a.page_size = static_cast<int32_t>(page);
  a.counts = static_cast<const int32_t *>(vector(o[P_COUNTS], "counts", at::kInt, n, dev));
  const long rows = o[P_ROWS] ? integer(o[P_ROWS]) : n;
  need(rows >= 0 && rows <= INT32_MAX, "rows must not be negative");
  need(o[P_COUNTS] || rows == n, "without counts there is a row for each sequence");
  a.rows = static_cast<int32_t>(rows);
  const int64_t sizes[] = {rows, rows, n + 1, n, 1};
  for (int i = 0; i < 5; ++i) {
    PyObject *mine = o[kPlanOutputs[i]];
    if (!mine) continue;
    const char *name = plan_sig.names[kPlanOutputs[i]];
    int32_t *at = static_cast<int32_t *>(vector(mine, name, at::kInt, sizes[i], dev));
    (i == 0 ? a.seqs : i == 1 ? a.slots : i == 2 ? a.starts : i == 3 ? a.totals : a.used_out) = at;
    const Region r(THPVariable_Unpack(mine), sizes[i]);
    auto apart = [&](PyObject *other, const char *other_name, bool may_be_same) {
      if (!other || (may_be_same && THPVariable_Unpack(other).data_ptr() == at)) return;
      if (!disjoint(r, Region(THPVariable_Unpack(other), THPVariable_Unpack(other).numel())))
        throw Bad{std::string(name) + " must not overlap " + other_name + ": it is written"};
    };
    apart(o[P_LENGTHS], "lengths", kPlanOutputs[i] == P_TOTALS);
    apart(o[P_USED], "used", kPlanOutputs[i] == P_USED_OUT);
    apart(o[P_COUNTS], "counts", false);
    apart(o[P_FREE], "free", false);
    for (int j = 0; j < i; ++j) apart(o[kPlanOutputs[j]], plan_sig.names[kPlanOutputs[j]], false);
    if (!disjoint(r, of_table)) throw Bad{std::string(name) + " must not overlap table: both are written"};
  }
  for (int i : {P_LENGTHS, P_USED, P_COUNTS, P_FREE})
    if (o[i] && !disjoint(of_table, Region(THPVariable_Unpack(o[i]), THPVariable_Unpack(o[i]).numel()))) throw Bad{std::string("table must not overlap ") + plan_sig.names[i] + ": it is written"};
  a.status = static_cast<int32_t *>(vector(o[P_STATUS], "status", at::kInt, 1, dev));
  *device = dev;
  return a;
}

PyObject *paged_plan(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  mk_plan_args a = plan_args(o, true, &dev);
  const at::Tensor &lengths = THPVariable_Unpack(o[P_LENGTHS]);
  const Launch on(dev, o[P_STREAM]);
  const int64_t sizes[] = {a.rows, a.rows, a.n + int64_t{1}, a.n, 1};
  int32_t **const to[] = {&a.seqs, &a.slots, &a.starts, &a.totals, &a.used_out};
  at::Tensor made[5];
  Results results;
  for (int i = 0; i < 5; ++i)
    if (!o[kPlanOutputs[i]]) results.want(4 * sizes[i]);
  results.allocate(lengths);
  for (int i = 0; i < 5; ++i) {
    if (o[kPlanOutputs[i]]) continue;
    made[i] = results.take({sizes[i]}, at::kInt);
    *to[i] = static_cast<int32_t *>(made[i].data_ptr());
  }
  enqueue("mk_paged_plan", [&] { return mk_paged_plan(&a, on.stream); });
  changed(o[P_TABLE]);
  changed(o[P_STATUS]);
  PyObject *out = PyTuple_New(5);
  if (!out) throw Raised{};
  for (int i = 0; i < 5; ++i) {
    changed(o[kPlanOutputs[i]]);
    PyTuple_SET_ITEM(out, i, of(o[kPlanOutputs[i]], made[i]));
  }
  return out;
}

PyObject *check_plan(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(plan_args(o, false, &dev));
}

// ---- paged_prompt_attention --------------------------------------------------------------

enum { T_Q, T_KC, T_VC, T_TABLE, T_STARTS, T_LENGTHS, T_SCALE, T_WINDOW, T_SINKS, T_KS, T_VS, T_OUT, T_LSE, T_STATUS, T_STREAM };
Signature prompt_sig = {"paged_prompt_attention", 6, 6, 15,
                        {"q", "k_cache", "v_cache", "table", "starts", "lengths", "scale", "window", "sinks", "k_scale", "v_scale", "out", "lse", "status",
                         "stream"}, {}};

mk_prompt_args prompt_args(PyObject *const *o, const mk_paged_kv &kv, const c10::Device &dev) {
  const at::Tensor &q = tensor(o[T_Q], "q");
  need(q.scalar_type() == at::kBFloat16, "q must be bf16 (paged_attention takes fp32 queries, a row for each token)");
  need(q.device() == dev, "q and the cache must be on the same device");
  need(q.dim() == 3, "q must be [rows][heads][head_dim]");
  const int64_t rows = q.size(0), hq = q.size(1), d = kv.head_dim;
  mk_prompt_args a = {};
  a.rows = small(rows, "q");
  a.dtype = MK_BF16;
  heads(q, "q", rows, d, 0, at::kBFloat16, dev, &a.q_row, &a.q_head);
  if (hq < 1 || hq % kv.n_kv_heads) throw Bad{"q must have a multiple of the cache's " + std::to_string(kv.n_kv_heads) + " heads"};
  a.n_q_heads = small(hq, "q");
  a.q = q.data_ptr();
  need(o[T_LENGTHS] && o[T_STARTS], "starts and lengths are needed");
  const at::Tensor &lengths = tensor(o[T_LENGTHS], "lengths");
  need(lengths.dim() == 1, "lengths must be int32 [sequences]");
  const int64_t n = lengths.size(0);
  a.n = small(n, "lengths");
  need(n <= kv.table_rows, "the table needs a row for each sequence");
  a.lengths = static_cast<const int32_t *>(vector(o[T_LENGTHS], "lengths", at::kInt, n, dev));
  a.starts = static_cast<const int32_t *>(vector(o[T_STARTS], "starts", at::kInt, n + 1, dev));
  if (o[T_OUT]) {
    const at::Tensor &out = tensor(o[T_OUT], "out");
    heads(out, "out", rows, d, hq, at::kBFloat16, dev, &a.out_row, &a.out_head);
    const Region r = written(out, "out", d), of_q(q, d);
    need(r == of_q || disjoint(r, of_q), "out must be q itself or not overlap it");
    need(disjoint(r, Region(THPVariable_Unpack(o[T_KC]), d)) && disjoint(r, Region(THPVariable_Unpack(o[T_VC]), d)), "out must not overlap the cache");
    a.out = out.data_ptr();
  }
  if (o[T_LSE]) {
    const at::Tensor &lse = tensor(o[T_LSE], "lse");
    need(lse.dim() == 2 && lse.size(0) == rows && lse.size(1) == hq && lse.scalar_type() == at::kFloat && lse.device() == dev && lse.is_contiguous(),
         "lse must be a contiguous fp32 [rows][heads] on q's device");
    const Region r(lse, hq);
    need(disjoint(r, Region(q, d)) && (!o[T_OUT] || disjoint(r, Region(THPVariable_Unpack(o[T_OUT]), d))), "lse must not overlap q or out");
    a.lse = static_cast<float *>(lse.data_ptr());
  }
  for (int i : {T_WINDOW, T_SINKS}) {
    const long v = o[i] ? integer(o[i]) : 0;
    need(v >= 0, i == T_WINDOW ? "window must be 0 (all) or the number of last tokens" : "sinks must not be negative");
    (i == T_WINDOW ? a.window : a.sinks) = v > INT32_MAX ? INT32_MAX : static_cast<int32_t>(v);
  }
  a.scale = o[T_SCALE] ? static_cast<float>(number(o[T_SCALE])) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  need(std::isfinite(a.scale), "scale must be finite");
  a.status = static_cast<int32_t *>(vector(o[T_STATUS], "status", at::kInt, 1, dev));
  return a;
}

PyObject *paged_prompt_attention(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[T_KC], o[T_VC], o[T_TABLE], o[T_KS], o[T_VS], true, &dev);
  mk_prompt_args a = prompt_args(o, kv, dev);
  const Launch on(dev, o[T_STREAM]);
  at::Tensor made;
  if (!o[T_OUT]) {
    const at::Tensor &q = THPVariable_Unpack(o[T_Q]);
    made = fresh(q.sizes(), q.scalar_type(), q);
    a.out = made.data_ptr();
    a.out_row = made.stride(0);
    a.out_head = made.stride(1);
  }
  if (a.rows && a.n) {
    Memory workspace;
    try {
      enqueue("mk_paged_prompt_attention", [&] { return mk_paged_prompt_attention_ask(&kv, &a, &Memory::ask, &workspace, on.stream); });
    } catch (const Failed &) {
      if (workspace.error) std::rethrow_exception(workspace.error);
      throw;
    }
    for (int i : {T_OUT, T_LSE, T_STATUS}) changed(o[i]);
  }
  return of(o[T_OUT], made);
}

PyObject *check_prompt(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  const mk_paged_kv kv = cache(o[T_KC], o[T_VC], o[T_TABLE], o[T_KS], o[T_VS], false, &dev);
  return bytes_of(prompt_args(o, kv, dev));
}

// ---- quantize_fp8 ------------------------------------------------------------------------

enum { Q_X, Q_CODES, Q_SCALES, Q_STREAM };
Signature quantize_sig = {"quantize_fp8", 1, 1, 4, {"x", "codes", "scales", "stream"}, {}};

mk_quantize_fp8_args quantize_args(PyObject *const *o, bool on_device, c10::Device *device) {
  const at::Tensor &x = tensor(o[Q_X], "x");
  const auto type = x.scalar_type();
  const c10::Device dev = x.device();
  need(x.dim() == 2 && (type == at::kFloat || type == at::kBFloat16), "x must be [rows][k] of fp32 or bf16");
  need(!on_device || dev.is_cuda(), "x must be on a CUDA device");
  const int64_t m = x.size(0), k = x.size(1), kb = (k + 127) / 128;
  need(k > 0 && k % 16 == 0, "k must be a multiple of 16");
  mk_quantize_fp8_args a = {};
  a.m = small(m, "x"), a.k = small(k, "x");
  a.dtype = type_of(type);
  need(!m || (x.stride(1) == 1 && step(x, 0) % (type == at::kFloat ? 4 : 8) == 0 && on16(x)),
       "x's last dimension must be contiguous and every row start on 16 bytes");
  a.x = x.data_ptr();
  a.x_row = step(x, 0);
  a.codes_row = k, a.scales_row = kb;
  const Region of_x(x, k);
  if (o[Q_CODES]) {
    const at::Tensor &c = tensor(o[Q_CODES], "codes");
    need(c.dim() == 2 && c.size(0) == m && c.size(1) == k && c.scalar_type() == at::kFloat8_e4m3fn && c.device() == dev && (!m || c.stride(1) == 1) &&
             step(c, 0) % 16 == 0 && on16(c),
         "codes must be float8_e4m3fn of x's shape on its device, every row contiguous from 16 bytes on");
    need(disjoint(written(c, "codes", k), of_x), "codes must not overlap x");
    a.codes = c.data_ptr();
    if (c.size(0) > 1) a.codes_row = c.stride(0);
  }
  if (o[Q_SCALES]) {
    const at::Tensor &s = tensor(o[Q_SCALES], "scales");
    need(s.dim() == 2 && s.size(0) == m && s.size(1) == kb && s.scalar_type() == at::kFloat && s.device() == dev && (s.stride(1) == 1 || kb == 1),
         "scales must be fp32 [rows][k / 128, rounded up] on x's device, rows contiguous");
    const Region r = written(s, "scales", kb);
    need(disjoint(r, of_x) && (!o[Q_CODES] || disjoint(r, Region(THPVariable_Unpack(o[Q_CODES]), k))), "scales must not overlap x or codes");
    a.scales = static_cast<float *>(s.data_ptr());
    if (s.size(0) > 1) a.scales_row = s.stride(0);
  }
  *device = dev;
  return a;
}

PyObject *quantize_fp8(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  mk_quantize_fp8_args a = quantize_args(o, true, &dev);
  const Launch on(dev, o[Q_STREAM]);
  const at::Tensor &x = THPVariable_Unpack(o[Q_X]);
  // (an allocation each, as codes are kept, saved and resized without their scales: 0.15 us a call more than one for both)
  at::Tensor codes, scales;
  if (!o[Q_CODES]) {
    codes = fresh({a.m, a.k}, at::kFloat8_e4m3fn, x);
    a.codes = codes.data_ptr();
  }
  if (!o[Q_SCALES]) {
    scales = fresh({a.m, (a.k + int64_t{127}) / 128}, at::kFloat, x);
    a.scales = static_cast<float *>(scales.data_ptr());
  }
  if (a.m) {
    enqueue("mk_quantize_fp8", [&] { return mk_quantize_fp8(&a, on.stream); });
    changed(o[Q_CODES]);
    changed(o[Q_SCALES]);
  }
  PyObject *out = PyTuple_New(2);
  if (!out) throw Raised{};
  PyTuple_SET_ITEM(out, 0, of(o[Q_CODES], codes));
  PyTuple_SET_ITEM(out, 1, of(o[Q_SCALES], scales));
  return out;
}

PyObject *check_quantize(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(quantize_args(o, false, &dev));
}

// ---- matmul_fp8 ---------------------------------------------------------------------------

enum { M_X, M_XS, M_W, M_WS, M_RESIDUAL, M_OUT, M_DTYPE, M_STATUS, M_STREAM };
Signature matmul_sig = {"matmul_fp8", 4, 4, 9, {"x", "x_scale", "w", "w_scale", "residual", "out", "dtype", "status", "stream"}, {}};

mk_matmul_fp8_args matmul_args(PyObject *const *o, bool on_device, c10::Device *device) {
  const at::Tensor &x = tensor(o[M_X], "x"), &xs = tensor(o[M_XS], "x_scale"), &w = tensor(o[M_W], "w"), &ws = tensor(o[M_WS], "w_scale");
  const c10::Device dev = x.device();
  need(x.dim() == 2 && x.scalar_type() == at::kFloat8_e4m3fn, "x must be [rows][k] of float8_e4m3fn (quantize_fp8)");
  need(!on_device || dev.is_cuda(), "x must be on a CUDA device");
  const int64_t m = x.size(0), k = x.size(1), kb = (k + 127) / 128;
  need(k > 0 && k % 16 == 0, "k must be a multiple of 16");
  need(w.dim() == 2 && w.size(1) == k && w.scalar_type() == at::kFloat8_e4m3fn && w.device() == dev, "w must be [n][k] of float8_e4m3fn on x's device");
  const int64_t n = w.size(0);
  mk_matmul_fp8_args a = {};
  a.m = small(m, "x"), a.n = small(n, "w"), a.k = small(k, "x");
  // rows one behind another or further apart, from 16 bytes on
  a.x_row = m > 1 ? x.stride(0) : k, a.w_row = n > 1 ? w.stride(0) : k;
  need(!m || (x.stride(1) == 1 && a.x_row % 16 == 0 && a.x_row >= k && on16(x)), "x's rows must be contiguous, not overlap and start on 16 bytes");
  need(!n || (w.stride(1) == 1 && a.w_row % 16 == 0 && a.w_row >= k && on16(w)), "w's rows must be contiguous, not overlap and start on 16 bytes");
  a.x = x.data_ptr(), a.w = w.data_ptr();
  need(xs.dim() == 2 && xs.size(0) == m && xs.size(1) == kb && xs.scalar_type() == at::kFloat && xs.device() == dev && (xs.stride(1) == 1 || kb == 1),
       "x_scale must be fp32 [rows][k / 128, rounded up] on x's device, rows contiguous");
  need(ws.dim() == 2 && ws.size(0) == (n + 127) / 128 && ws.size(1) == kb && ws.scalar_type() == at::kFloat && ws.device() == dev && ws.is_contiguous(),
       "w_scale must be a contiguous fp32 [n / 128][k / 128] (rounded up) on x's device");
  a.x_scale = static_cast<const float *>(xs.data_ptr());
  a.x_scale_row = step(xs, 0);
  a.w_scale = static_cast<const float *>(ws.data_ptr());
  auto type = at::kBFloat16;
  if (o[M_DTYPE]) {
    need(THPDtype_Check(o[M_DTYPE]), "dtype must be a torch dtype");
    type = reinterpret_cast<THPDtype *>(o[M_DTYPE])->scalar_type;
  } else if (o[M_OUT]) {
    type = tensor(o[M_OUT], "out").scalar_type();
  } else if (o[M_RESIDUAL]) {
    type = tensor(o[M_RESIDUAL], "residual").scalar_type();
  }
  need(type == at::kFloat || type == at::kBFloat16, "the result must be fp32 or bf16");
  a.dtype = type_of(type);
  for (int i : {M_RESIDUAL, M_OUT}) {
    if (!o[i]) continue;
    const char *name = i == M_OUT ? "out" : "residual";
    const at::Tensor &t = tensor(o[i], name);
    if (t.dim() != 2 || t.size(0) != m || t.size(1) != n || t.scalar_type() != type || t.device() != dev || (t.stride(1) != 1 && n > 1))
      throw Bad{std::string(name) + " must be [" + std::to_string(m) + "][" + std::to_string(n) + "] of " + c10::toString(type) + " on x's device, rows contiguous"};
    if (i == M_OUT) {
      const Region r = written(t, "out", n);
      need(disjoint(r, Region(x, k)) && disjoint(r, Region(w, k)) && disjoint(r, Region(xs, kb)) && disjoint(r, Region(ws, kb)),
           "out must not overlap x, w or their scales: they are read until the last of out is written");
      if (o[M_RESIDUAL]) {
        const Region of_residual(THPVariable_Unpack(o[M_RESIDUAL]), n);
        need(r == of_residual || disjoint(r, of_residual), "out must be residual itself or not overlap it");
      }
      a.y = t.data_ptr(), a.y_row = step(t, 0);
    } else {
      a.residual = t.data_ptr(), a.residual_row = step(t, 0);
    }
  }
  a.status = static_cast<int32_t *>(vector(o[M_STATUS], "status", at::kInt, 1, dev));
  *device = dev;
  return a;
}

PyObject *matmul_fp8(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  mk_matmul_fp8_args a = matmul_args(o, true, &dev);
  const Launch on(dev, o[M_STREAM]);
  at::Tensor made;
  if (!o[M_OUT]) {
    made = fresh({a.m, a.n}, a.dtype == MK_F32 ? at::kFloat : at::kBFloat16, THPVariable_Unpack(o[M_X]));
    a.y = made.data_ptr();
    a.y_row = a.n;
  }
  if (a.m && a.n) {
    enqueue("mk_matmul_fp8", [&] { return mk_matmul_fp8(&a, on.stream); });
    changed(o[M_OUT]);
    changed(o[M_STATUS]);
  }
  return of(o[M_OUT], made);
}

PyObject *check_matmul(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(matmul_args(o, false, &dev));
}

// ---- adjust_logits -------------------------------------------------------------------------

enum { L_X, L_TOKENS, L_LENGTHS, L_PROMPTS, L_REPETITION, L_PRESENCE, L_FREQUENCY, L_BIAS_IDS, L_BIAS, L_MASK, L_OUT, L_STREAM };
Signature logits_sig = {"adjust_logits", 1, 1, 12,
                        {"logits", "tokens", "lengths", "prompts", "repetition", "presence", "frequency", "bias_ids", "bias", "mask", "out", "stream"}, {}};

mk_logits_args logits_args(PyObject *const *o, bool on_device, c10::Device *device) {
  const at::Tensor &x = tensor(o[L_X], "logits");
  const auto type = x.scalar_type();
  const c10::Device dev = x.device();
  need(x.dim() == 2 && (type == at::kFloat || type == at::kBFloat16) && (x.size(1) <= 1 || x.stride(1) == 1),
       "logits must be [rows][vocabulary] of fp32 or bf16, rows contiguous");
  need(!on_device || dev.is_cuda(), "logits must be on a CUDA device");
  const int64_t n = x.size(0), v = x.size(1);
  mk_logits_args a = {};
  a.n = small(n, "logits"), a.vocab = small(v, "logits");
  a.dtype = type_of(type);
  a.x = x.data_ptr();
  a.x_row = step(x, 0);
  int64_t found = 0;
  a.tokens = static_cast<const int32_t *>(rows_of(o[L_TOKENS], "tokens", at::kInt, n, -1, dev, &a.tokens_row, &found));
  a.columns = small(found, "tokens");
  need(o[L_TOKENS] || !o[L_PROMPTS], "prompts need tokens");
  need(o[L_TOKENS] || !(o[L_REPETITION] || o[L_PRESENCE] || o[L_FREQUENCY]), "penalties need tokens");
  a.lengths = static_cast<const int32_t *>(vector(o[L_LENGTHS], "lengths", at::kInt, n, dev));
  a.prompts = static_cast<const int32_t *>(vector(o[L_PROMPTS], "prompts", at::kInt, n, dev));
  a.repetition = static_cast<const float *>(vector(o[L_REPETITION], "repetition", at::kFloat, n, dev));
  a.presence = static_cast<const float *>(vector(o[L_PRESENCE], "presence", at::kFloat, n, dev));
  a.frequency = static_cast<const float *>(vector(o[L_FREQUENCY], "frequency", at::kFloat, n, dev));
  need(!o[L_BIAS_IDS] == !o[L_BIAS], "bias_ids and bias go together");
  a.bias_ids = static_cast<const int32_t *>(rows_of(o[L_BIAS_IDS], "bias_ids", at::kInt, n, -1, dev, &a.ids_row, &found));
  if (o[L_BIAS_IDS]) a.biases = small(found, "bias_ids");
  a.bias = static_cast<const float *>(rows_of(o[L_BIAS], "bias", at::kFloat, n, found, dev, &a.bias_row, nullptr));
  a.mask = static_cast<const int32_t *>(rows_of(o[L_MASK], "mask", at::kInt, n, (v + 31) / 32, dev, &a.mask_row, nullptr));
  if (o[L_OUT]) {
    const at::Tensor &out = tensor(o[L_OUT], "out");
    need(out.dim() == 2 && out.size(0) == n && out.size(1) == v && out.scalar_type() == type && out.device() == dev && (v <= 1 || out.stride(1) == 1),
         "out must be like logits, rows contiguous");
    const Region r = written(out, "out", v), of_x(x, v);
    need(r == of_x || disjoint(r, of_x), "out must be logits itself or not overlap it");
    for (int i : {L_TOKENS, L_LENGTHS, L_PROMPTS, L_REPETITION, L_PRESENCE, L_FREQUENCY, L_BIAS_IDS, L_BIAS, L_MASK}) {
      if (!o[i]) continue;
      const at::Tensor &t = THPVariable_Unpack(o[i]);
      if (!disjoint(r, Region(t, t.size(t.dim() - 1)))) throw Bad{std::string("out must not overlap ") + logits_sig.names[i]};
    }
    a.out = out.data_ptr();
    a.out_row = step(out, 0);
  }
  *device = dev;
  return a;
}

PyObject *adjust_logits(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  mk_logits_args a = logits_args(o, true, &dev);
  const Launch on(dev, o[L_STREAM]);
  at::Tensor made;
  if (!o[L_OUT]) {
    const at::Tensor &x = THPVariable_Unpack(o[L_X]);
    made = fresh({a.n, a.vocab}, x.scalar_type(), x);
    a.out = made.data_ptr();
    a.out_row = a.vocab;
  }
  if (a.n && a.vocab) {
    enqueue("mk_adjust_logits", [&] { return mk_adjust_logits(&a, on.stream); });
    changed(o[L_OUT]);
  }
  return of(o[L_OUT], made);
}

PyObject *check_logits(PyObject *const *o) {
  c10::Device dev(c10::kCPU);
  return bytes_of(logits_args(o, false, &dev));
}

inline void intern() {
  for (Signature *s : {&plan_sig, &prompt_sig, &quantize_sig, &matmul_sig, &logits_sig}) s->intern();
}

PyMethodDef methods[] = {
    method<&plan_sig, &paged_plan>("paged_plan", R"(paged_plan(lengths, table, free, used, page_size, *, counts=None, rows=None, seqs=None, slots=None, starts=None, totals=None, used_out=None, status=None, stream=None)
--

``mk_paged_plan``: rows, slots and pages of a step's new tokens.  Returns
``(seqs, slots, starts, totals, used_out)``, int32 tensors, and extends
``table`` in place.  Those that are not given are new, and parts of one
allocation: one that is kept keeps the others' memory, and ``resize_`` or
``torch.save`` of one reaches all of it.

``lengths`` int32 [n] are the tokens that each sequence has (negative: a
padding row), ``counts`` int32 [n] those that it gets; new pages come from
``free`` int32 [pages] behind the first ``used`` (int32 [1]) of them.
``seqs`` and ``slots`` [rows] are what ``paged_append`` takes (-1 behind
the last token), ``starts`` [n + 1] and ``totals`` [n] what
``paged_prompt_attention`` takes.  Without ``counts`` every sequence gets one
token and row i is sequence i: ``slots`` and ``totals`` are then what
``paged_append`` and ``paged_attention`` take.  ``totals`` may be
``lengths`` and ``used_out`` ``used``.  A step that does not fit is not made:
no tokens for anyone, and ``check_status(status)`` raises.)"),
    method<&prompt_sig, &paged_prompt_attention>("paged_prompt_attention", R"(paged_prompt_attention(q, k_cache, v_cache, table, starts, lengths, *, scale=None, window=0, sinks=0, k_scale=None, v_scale=None, out=None, lse=None, status=None, stream=None)
--

``mk_paged_prompt_attention``: causal attention of the last tokens of each
sequence (a whole prompt, or a chunk behind what is cached) over the paged cache
that holds their keys and values already.  ``q`` bf16 [rows][heads][d]; sequence
i, row i of ``table``, has ``lengths[i]`` tokens in all, the last
``starts[i + 1] - starts[i]`` of which are rows ``starts[i]`` .. of ``q``.
A token sees itself and the tokens before it, with a ``window`` the last
``window`` of them and the first ``sinks``.  Returns ``out`` like ``q`` (it
may be ``q``, but not overlap it otherwise); ``lse`` fp32 [rows][heads] receives
the log of each softmax's sum.  Rows of no sequence, and those of a negative
length, are left as they were (in a new result: whatever its memory holds).  fp32 queries: ``paged_attention`` with a table
row for each token.)"),
    method<&quantize_sig, &quantize_fp8>("quantize_fp8", R"(quantize_fp8(x, *, codes=None, scales=None, stream=None)
--

``mk_quantize_fp8``: ``(codes, scales)`` of ``x`` [rows][k] (fp32 or bf16,
k a multiple of 16): float8_e4m3fn [rows][k] and fp32 [rows][k / 128, rounded
up], so that x is nearly code times scale; a block's scale is its largest
element / 448.)"),
    method<&matmul_sig, &matmul_fp8>("matmul_fp8", R"(matmul_fp8(x, x_scale, w, w_scale, *, residual=None, out=None, dtype=None, status=None, stream=None)
--

``mk_matmul_fp8``: ``x`` [rows][k] (``quantize_fp8``) times the transpose of
``w`` [n][k] (``quantize_fp8_weight``), plus ``residual`` [rows][n] (which may
be ``out``).  The result is of ``dtype``, fp32 or bf16 (else ``out``'s, or
``residual``'s, or bf16).)"),
    method<&logits_sig, &adjust_logits>("adjust_logits", R"(adjust_logits(logits, *, tokens=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, mask=None, out=None, stream=None)
--

``mk_adjust_logits``: ``logits`` [n][vocabulary] (fp32 or bf16) with penalties
for the tokens of each row's history, biases of single tokens and a mask; into
``out`` (which may be ``logits``; a new tensor by default).

``tokens`` int32 [n][columns] are the histories, the first ``lengths[i]`` of
each row (all by default; a negative length marks a padding row, which is left as
it was, in a new result whatever its memory holds) and the first ``prompts[i]`` of those the prompt.  A token of the history
is divided by ``repetition[i]`` if positive and multiplied by it if not; one
that came c > 0 times behind the prompt loses ``frequency[i]`` * c + ``presence[i]``
(all fp32 [n]).  ``bias`` fp32 [n][b] is added to the tokens ``bias_ids`` int32
[n][b] (an id outside the vocabulary: unused; of one token more than once: all of
them).  ``mask`` int32 [n][vocabulary / 32, rounded up]: a token whose bit is 0
becomes -inf.)"),
    method<&plan_sig, &check_plan>("check_plan", "The checks of paged_plan; the bytes of its mk_plan_args."),
    method<&prompt_sig, &check_prompt>("check_prompt", "The checks of paged_prompt_attention; the bytes of its mk_prompt_args."),
    method<&quantize_sig, &check_quantize>("check_quantize", "The checks of quantize_fp8; the bytes of its mk_quantize_fp8_args."),
    method<&matmul_sig, &check_matmul>("check_matmul", "The checks of matmul_fp8; the bytes of its mk_matmul_fp8_args."),
    method<&logits_sig, &check_logits>("check_logits", "The checks of adjust_logits; the bytes of its mk_logits_args."),
    {nullptr, nullptr, 0, nullptr}};

}  // namespace prompts
}  // namespace mkt
