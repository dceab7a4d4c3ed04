// Attention of whole prompts over a paged KV cache (mk_paged_prompt_attention): checks, launches, bf16 caches.
#include "mk_prompt.cuh"

namespace mkprompt {

// mk_prompt_fp8.cu
extern template int launch<true, 64>(PromptParams &, int, cudaStream_t);
extern template int launch<true, 128>(PromptParams &, int, cudaStream_t);

// pairs of tiles of a call: a sequence has one that is not full
int64_t most_items(int64_t n, int64_t rows, int item) { return std::min(rows, rows / item + n); }

int64_t parts_bytes(int sms, int d) { return 2 * static_cast<int64_t>(sms) * 2 * kRows * (d + 4) * 4; }
// header, records (an item that is cut has more than a share of the work: fewer of them than SMs), tasks (one for each item
// and for every share of the work one more), partial results (at most two for every share)
int64_t workspace_bytes(int sms, int d, int64_t ctas) {
  return 16 + static_cast<int64_t>(sms) * 16 + ctas * static_cast<int64_t>(sizeof(Task)) + parts_bytes(sms, d);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stride_ok(int64_t s, int elem) { return s >= 0 && s <= (int64_t{1} << 48) && s * elem % 16 == 0; }

}  // namespace mkprompt

using namespace mkprompt;

namespace {

// tokens of a tile, virtual heads, and CTAs of a call; < 0: an error
struct Shape {
  int heads, blocks, tokens, vh;
  bool few;                    // an SM for each pair of tiles
  int64_t ctas;
  Shape(int64_t n, int64_t rows, int hq, int hkv, int sms) {
    const int group = hq / hkv;
    blocks = (group + kRows - 1) / kRows;
    heads = (group + blocks - 1) / blocks;
    tokens = kRows / heads;
    vh = hkv * blocks;
    few = most_items(n, rows, 2 * tokens) * vh <= sms;
    ctas = most_items(n, rows, few ? tokens : 2 * tokens) * vh + sms;
  }
};

}  // namespace

extern "C" int64_t mk_paged_prompt_attention_workspace(int32_t n, int32_t rows, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n < 0 || rows < 0 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads) return MK_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MK_ERR_UNSUPPORTED;
  const int sms = mkv::sm_count(nullptr);
  return sms < 0 ? MK_ERR_CUDA : workspace_bytes(sms, head_dim, Shape(n, rows, n_q_heads, n_kv_heads, sms).ctas);
}

namespace {

int prompt_attention(const mk_paged_kv *kv, const mk_prompt_args *a, mk_stream stream, mk_workspace_fn ask, void *context) {
  const int rc = mkv::check_cache(kv);
  if (rc != MK_OK) return rc;
  if (!a || a->n < 0 || a->rows < 0 || a->n > kv->table_rows || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->window < 0 || a->sinks < 0 ||
      !std::isfinite(a->scale) || a->n_q_heads < 1 || a->n_q_heads % kv->n_kv_heads)
    return MK_ERR_INVALID_ARG;
  if (a->dtype != MK_BF16) return MK_ERR_UNSUPPORTED;
  if (a->n == 0 || a->rows == 0) return MK_OK;
  if (!a->q || !a->out || !a->starts || !a->lengths || !aligned16(a->q) || !aligned16(a->out) || !stride_ok(a->q_row, 2) || !stride_ok(a->q_head, 2) ||
      !stride_ok(a->out_row, 2) || !stride_ok(a->out_head, 2))
    return MK_ERR_INVALID_ARG;
  const int64_t slots = static_cast<int64_t>(kv->table_cols) * kv->page_size;
  if (a->n > kMaxSequences || slots > INT32_MAX - 1024 || a->rows > INT32_MAX / 2 - 1024 || a->n_q_heads > (1 << 20)) return MK_ERR_UNSUPPORTED;
  int dev = 0;
  const int sms = mkv::sm_count(&dev);
  if (sms < 0) return MK_ERR_CUDA;
  PromptParams p = {};
  p.q = a->q, p.k = kv->k, p.v = kv->v, p.out = a->out, p.lse = a->lse;
  p.q_row = a->q_row, p.q_head = a->q_head, p.out_row = a->out_row, p.out_head = a->out_head;
  p.page_stride = kv->page_stride, p.head_stride = kv->head_stride, p.slot_stride = kv->slot_stride;
  p.table = kv->table, p.table_stride = kv->table_stride;
  p.starts = a->starts, p.lengths = a->lengths;
  p.k_scale = kv->k_scale, p.v_scale = kv->v_scale;
  p.status = a->status;
  p.page_size.set(kv->page_size);
  p.n = a->n, p.rows = a->rows, p.hq = a->n_q_heads, p.hkv = kv->n_kv_heads;
  p.group = p.hq / p.hkv;
  const Shape shape(a->n, a->rows, p.hq, p.hkv, sms);
  p.blocks = shape.blocks;
  p.heads.set(shape.heads);
  p.vh = shape.vh;
  p.tokens = shape.tokens;
  p.n_pages = kv->n_pages;
  p.capacity = static_cast<int>(slots);
  p.window = a->window;
  p.sinks = a->window > 0 ? std::min(a->sinks, p.capacity) : 0;
  p.sms = sms;
  p.scale = a->scale;
  if (shape.ctas > INT32_MAX / 2) return MK_ERR_UNSUPPORTED;   // (task numbers and sums of them are 32 bits)
  p.item = 2 * p.tokens;
  // blocks of an item: of all its row's tokens, or of the window, its own rows and the first tokens
  const int64_t span = p.window > 0 ? static_cast<int64_t>(p.window) + p.item + p.sinks + 3 * kBlock : slots + kBlock;
  p.joins = std::min<int64_t>(span, slots + kBlock) / kBlock > kLeastBlocks;
  // one tile a CTA where that leaves no SM with more to do (1000 tokens 16.0 us, two 18.9); not where items are cut, as two
  // tiles share their blocks (200 tokens behind 8000: 54 us, two 29)
  if (shape.few && !p.joins) p.item = p.tokens;
  const int items = static_cast<int>(most_items(p.n, p.rows, p.item) * p.vh);
  p.ctas = items + (p.joins ? sms : 0);
  // No list for few items of few sequences: a CTA that finds its own task takes longer, and a kernel before it more (77 tokens
  // 7.8 us, with a list 12.6; 2000 tokens 34 and 40; from two items an SM on the list is quicker: 8192 tokens 195, without 200).
  p.how = p.n > 32 ? kListed : !p.joins ? kWhole : items <= 2 * sms ? kCut : kListed;
  const int64_t bytes = workspace_bytes(sms, kv->head_dim, shape.ctas);
  if (!ask && (!a->workspace || a->workspace_bytes < bytes)) return MK_ERR_INVALID_ARG;
  if (p.how != kWhole) {
    // (what cannot be cut needs no room for partial results)
    p.header = static_cast<int4 *>(ask ? ask(context, p.joins ? bytes : bytes - parts_bytes(sms, kv->head_dim)) : a->workspace);
    if (!p.header) return MK_ERR_NO_MEMORY;
    if (!aligned16(p.header)) return MK_ERR_INVALID_ARG;
    p.records = p.header + 1;
    p.tasks = reinterpret_cast<Task *>(p.records + sms);
    p.parts = reinterpret_cast<float *>(p.tasks + shape.ctas);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (kv->dtype == MK_BF16)
    return kv->head_dim == 64 ? launch<false, 64>(p, dev, s) : launch<false, 128>(p, dev, s);
  return kv->head_dim == 64 ? launch<true, 64>(p, dev, s) : launch<true, 128>(p, dev, s);
}

}  // namespace

extern "C" int mk_paged_prompt_attention(const mk_paged_kv *kv, const mk_prompt_args *a, mk_stream stream) {
  return prompt_attention(kv, a, stream, nullptr, nullptr);
}

extern "C" int mk_paged_prompt_attention_ask(const mk_paged_kv *kv, const mk_prompt_args *a, mk_workspace_fn workspace, void *context, mk_stream stream) {
  return workspace ? prompt_attention(kv, a, stream, workspace, context) : MK_ERR_INVALID_ARG;
}
