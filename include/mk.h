/*
 * mk.h -- C ABI of the GB300 persistent decode megakernel library (libmk.so).
 *
 * Batch-1 autoregressive decode of a Qwen3-style decoder run as ONE
 * cooperatively launched kernel that loops over layers and decode steps
 * without exiting (page A, section "The idea: one kernel that never exits":
 * a single resident kernel that takes the whole GPU and runs the decode loop
 * itself instead of a chain of per-op launches).
 * Around that loop: a batched prompt prefill on tensor cores (mk_prefill), a
 * streaming mailbox the kernel fills with each greedy id while it runs
 * (mk_decode_start / mk_mailbox_read), and the per-op ablation of the same
 * math, plain or replayed from a CUDA graph (MK_DECODE_PER_OP*).
 *
 * Sources cited below:
 *   page A = "Porting a 1,200-line persistent CUDA megakernel to Qwen3-TTS:
 *            ~25 ms to first audio chunk" (dev.to)
 *   page B = "I made a single CUDA kernel speak: streaming Qwen3-TTS at 50ms
 *            latency on an RTX 5090" (theaicatchup.com)
 *
 * Conventions for every entry point:
 *   - Return value: MK_OK (0) or a negative MK_ERR_* code.  Nothing aborts the
 *     process.  mk_error_string() names a code.
 *   - "device" pointers are CUDA global-memory addresses on the handle's device
 *     (the device current at mk_create); "host" pointers are ordinary host memory.
 *   - Streams are passed as `mk_stream` (a cudaStream_t); NULL is the legacy
 *     default stream.
 *   - A handle is not thread-safe: one caller at a time.
 */
#ifndef MK_H
#define MK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MK_OK               0
#define MK_ERR_INVALID_ARG (-1)  /* bad pointer, size or option, checked on the host */
#define MK_ERR_UNSUPPORTED (-2)  /* shape or launch geometry this build does not handle */
#define MK_ERR_KV_FULL     (-3)  /* position + forwards would pass max_seq (host check); a step that
                                    mk_paged_plan has no room for (found on the device) */
#define MK_ERR_BAD_TOKEN   (-4)  /* id >= vocab_in, or a sentinel row outside the buffer
                                    (found on the device; later forwards are skipped) */
#define MK_ERR_TIMEOUT     (-5)  /* a device wait (grid barrier, ring, merge) ran past
                                    its time budget; the kernel returned early */
#define MK_ERR_NUMERIC     (-6)  /* a logit was NaN or infinite */
#define MK_ERR_CUDA        (-7)  /* a CUDA runtime call failed */
#define MK_ERR_NO_MEMORY   (-8)  /* a device allocation failed */
#define MK_ERR_BAD_POSITION (-9) /* a rotary position (an MRoPE position-stream value) outside the
                                     rotary table */
#define MK_ERR_BAD_PAGE   (-10)  /* a sequence index, slot, length or page id outside the page table
                                    or the cache (found on the device by the paged operators) */

typedef struct mk_handle mk_handle;
typedef void *mk_stream; /* cudaStream_t */

/* ---- model description ---------------------------------------------------
 * Qwen3-style decoder (page B, "Why Does a Single Kernel Even Matter for
 * TTS?": the TTS talker has the dimensions, layer count and heads of
 * Qwen3-0.6B; vocab, RoPE frequencies and the untied head differ).  The page's
 * kernel bakes these into compile-time constants (page A, "Porting it to
 * Qwen3-TTS-1.7B"); here they are runtime fields checked at mk_create, with
 * head_dim a template parameter of the kernel.
 *
 * Limits checked by mk_create (MK_ERR_UNSUPPORTED otherwise):
 *   head_dim in {64, 128}; n_q_heads % n_kv_heads == 0 with group size
 *   n_q_heads / n_kv_heads in {1, 2, 4, 8} and group * head_dim <= 512;
 *   every GEMV input width (hidden, n_q_heads * head_dim, intermediate) is
 *   K = KPT * T with KPT in {8, 12, 16, 24} and T in {32, 64, 128, 256};
 *   rope_modes 1 and 2 need mrope_sections summing to head_dim / 2.       */
typedef struct {
  int32_t n_layers;
  int32_t hidden;          /* H */
  int32_t n_q_heads;       /* Hq */
  int32_t n_kv_heads;      /* Hkv */
  int32_t head_dim;        /* d */
  int32_t intermediate;    /* I, SiLU-gated MLP width */
  int32_t vocab;           /* V, rows of the LM head */
  int32_t vocab_in;        /* rows of the input embedding table */
  float rms_eps;           /* RMSNorm epsilon inside the root (Qwen3: 1e-6) */
  float rope_theta;        /* rotary base (Qwen3: 1e6) */
  int32_t rope_mode;       /* 0 = RoPE, 1 = sectioned MRoPE (page A, "Porting it to
                              Qwen3-TTS-1.7B": the talker's rotary positions come in
                              sections, one position stream each): contiguous runs of
                              pairs per stream; 2 = interleaved MRoPE:
                              pair i with i % 3 = s in {1, 2} follows stream s while
                              i < 3 * mrope_sections[s], every other pair stream 0 */
  int32_t mrope_sections[3]; /* rotary pairs driven by position streams 0, 1, 2 */
  int32_t max_seq;         /* KV-cache capacity in positions */
  int32_t rope_positions;  /* rows of the host-built cos/sin table; 0 = 2*max_seq + 8
                              (page B, "So, What's the Catch with These Megakernels?":
                              the rotary frequencies come from tables the host
                              builds, not from the kernel) */
  uint32_t flags;          /* reserved, must be 0 */
} mk_config;

/* Per-layer weights: device pointers to bf16, row-major [out][in] (the
 * torch.nn.Linear layout), each 16-byte aligned.  Norm gains are [H] or [d].
 *   wq [Hq*d][H], wk/wv [Hkv*d][H], wo [H][Hq*d],
 *   w_gate/w_up [I][H], w_down [H][I].
 * BORROWED: the caller keeps them alive and unchanged until mk_destroy. */
typedef struct {
  const void *attn_norm, *wq, *wk, *wv, *q_norm, *k_norm, *wo;
  const void *mlp_norm, *w_gate, *w_up, *w_down;
} mk_layer_weights;

typedef struct {
  const void *embed;      /* [vocab_in][H] bf16, device, borrowed */
  const void *lm_head;    /* [vocab][H] bf16, or NULL = tied to embed (requires
                             vocab == vocab_in); page A, "Porting it to Qwen3-TTS-1.7B":
                             the text model ties them, the talker does not */
  const void *final_norm; /* [H] bf16 */
  const mk_layer_weights *layers; /* HOST array of n_layers entries, read at mk_create */
} mk_weights;

/* ---- per-call options (all optional; pass NULL for defaults) ------------ */
#define MK_DECODE_PER_OP 1u  /* run the same math as one ordinary kernel launch per
                                phase: this kernel relaunched once per phase (the
                                launch-overhead ablation; page A, "The idea: one kernel
                                that never exits": a conventional decode step is a long
                                chain of separate kernel launches) */
#define MK_DECODE_STREAM 4u    /* publish each forward's greedy id to the handle's
                                host-mapped mailbox the moment it is chosen, so the
                                host can consume ids while the launch still runs
                                (page A, "Porting a 1,200-line persistent CUDA
                                megakernel...": the talker streams audio tokens out
                                chunk by chunk); see mk_decode_start */
#define MK_DECODE_PER_OP_GRAPH 2u /* the same per-phase launches, captured once per
                                handle as a CUDA graph of one forward and replayed
                                once per forward (the ablation without host launch
                                cost); the first such call captures and instantiates */

typedef struct {
  uint32_t flags;             /* MK_DECODE_* bits */
  const float *embeds;        /* device [n_embed_rows][H] fp32 precomputed input rows;
                                 id -(r+1) selects row r (page B, "Why Does a Single
                                 Kernel Even Matter for TTS?": a non-negative id is
                                 looked up, any other input comes precomputed from a
                                 buffer) */
  int32_t n_embed_rows;
  const int32_t *pos3;        /* device [3][n_in + n_steps] position streams for MRoPE;
                                 NULL = the slot index in every stream */
  float *logits;              /* device [n_in + n_steps][vocab] fp32 out, or NULL */
  float *hidden;              /* device [n_in + n_steps][n_layers + 1][H] fp32 out, or NULL:
                                 the input row then the residual stream after each layer */
  uint64_t *trace;            /* device [n_fwd][5*n_layers + 1][grid][4] %globaltimer stamps
                                 of each CTA's thread 0 per phase: start, input in
                                 registers, tiles and epilogue done, phase left (the LM
                                 phase: after the grid barrier that closes the forward);
                                 or NULL */
  int32_t attn_chunks;        /* split-KV chunks per kv head; 0 = the library's policy
                                 (at least 4, one per 48 cached positions up to 8, then
                                 one per 256 positions up to grid / n_kv_heads; up to 8
                                 chunks merge by polling, more by the last CTA) */
  int64_t spin_ns;            /* budget of every device wait; 0 = 1 s */
  int32_t fault_skip_barrier; /* test hook: N > 0 makes CTA 0 skip its arrival at the
                                 grid barrier that closes forward N - 1 (persistent path
                                 only), so the other CTAs time out; 0 = off (a zeroed
                                 struct runs normally) */
  /* Talker inputs summed inside the kernel.  When codes != NULL a negative id
     -(r+1) selects code row r: the forward's input is
       sum_{j<n_books} books[j][codes[r][j]] + text[text_ids[r]]
     accumulated in fp32 in table order (codebook 0 .. n_books-1, then text) --
     the same sum mk_embed_sum writes, so the result is bitwise that of the
     embeds path fed by mk_embed_sum (page B, "Why Does a Single Kernel Even
     Matter for TTS?": each talker input is the 17-way codebook + text sum).
     codes and embeds are exclusive.  A code or text id out of range
     gives MK_ERR_BAD_TOKEN. */
  const void *books;          /* device bf16 [n_books][book_rows][H] */
  int32_t n_books;            /* 0 .. 64 */
  int32_t book_rows;
  const void *text;           /* device bf16 [text_rows][H] */
  int32_t text_rows;
  const int32_t *codes;       /* device int32 [n_code_rows][n_books] */
  const int32_t *text_ids;    /* device int32 [n_code_rows] */
  int32_t n_code_rows;
} mk_decode_opts;

typedef struct {
  int32_t grid;          /* CTAs = SMs of the device, one per SM */
  int32_t threads;       /* per CTA: consumer warps + 1 producer warp */
  int32_t stages;        /* shared-memory ring stages */
  int32_t stage_bytes;
  int32_t smem_bytes;    /* dynamic shared memory per CTA */
  int32_t position;      /* next KV slot */
  int32_t max_chunks;    /* split-KV chunk capacity per kv head */
  int64_t weight_bytes;  /* bf16 bytes streamed per forward (layers + head) */
  int64_t kv_bytes;      /* KV-cache allocation */
  int32_t plan;          /* decode kernel: 0 the general one (layouts chosen at run time,
                            phases out of line), 1 compiled for hidden 1024 / MLP 3072 /
                            16:8 heads of 128, 2 for hidden 2048 / MLP 6144 / 16:8 heads of 128 */
} mk_info;

/* Validate cfg, allocate the KV cache [L][Hkv][max_seq][d] bf16 (keys and
 * values), scratch, barrier/error words and the cos/sin table (built on the
 * host in double precision), and check that one CTA per SM fits.  *out gets
 * the handle.  The pages fix no interface beyond the model constants and the
 * token-id-or-buffer input (page A, "Porting it to Qwen3-TTS-1.7B"; page B,
 * "Why Does a Single Kernel Even Matter for TTS?"); the handle holds what the
 * persistent kernel keeps between calls (page A, "The idea: one kernel that
 * never exits": the KV cache and the step loop's state).  Errors:
 * MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED, MK_ERR_NO_MEMORY, MK_ERR_CUDA
 * (nothing is leaked on failure). */
int mk_create(const mk_config *cfg, const mk_weights *w, mk_handle **out);

/* Forget the cached context: the cursor returns to slot 0 and the last id to 0
 * (a new sequence; the KV cache of page A, "The idea: one kernel that never
 * exits", starts empty).  Enqueued on `stream`; returns after the stream
 * completes.  Errors: MK_ERR_INVALID_ARG (NULL, or a started decode not yet
 * waited for), MK_ERR_CUDA. */
int mk_reset_kv(mk_handle *h, mk_stream stream);

/* Run n_in + n_steps forwards from the handle's cursor in ONE cooperative launch.
 * Forward i < n_in consumes d_in_ids[i] (device int32; a negative id picks a
 * row of opts->embeds); forward i >= n_in consumes the greedy id of forward
 * i-1 (for i == 0, the last id of the previous call).  d_out_ids[i] (device
 * int32, n_in + n_steps entries) receives the greedy argmax of forward i,
 * lowest index on ties.  Blocks until `stream` completes and returns the
 * device status.  After an error the cached context is undefined: call
 * mk_reset_kv.  Errors: all codes above. */
int mk_decode(mk_handle *h, const int32_t *d_in_ids, int32_t n_in, int32_t n_steps,
              int32_t *d_out_ids, const mk_decode_opts *opts, mk_stream stream);

/* Batched prompt prefill: the n forwards of mk_decode(h, d_in_ids, n, 0, ...)
 * computed all at once per layer instead of one token per forward -- the
 * projections as the library's own tcgen05 tensor-core GEMMs with fp32
 * accumulation in tensor memory (each fp32 activation enters as three bf16
 * terms, hi + mid + lo: all 24 bits, each in its own accumulator), then
 * QK-norm, RoPE / MRoPE,
 * the bf16 KV append and causal attention over the cache in the library's own
 * kernels.  It fills the same KV cache and advances the same cursor, so a
 * following mk_decode(h, NULL, 0, n_steps, ...) continues from the prompt's
 * greedy id (page A, "Porting a 1,200-line persistent CUDA megakernel to
 * Qwen3-TTS": the time to the first chunk is what the listener waits for).
 *   d_in_ids: device int32 [n] (negative ids pick rows of opts->embeds).
 *   d_out_ids: device int32 [n] greedy ids after every prompt token, or NULL
 *   (then only the last token's logits are computed).  opts: embeds, pos3,
 *   logits ([n][vocab]) and hidden ([n][L+1][H]) as for mk_decode; flags,
 *   trace and code rows must be unset.  Not bitwise equal to mk_decode (other
 *   summation orders); both follow the oracle within the parity tolerance.
 * The first call of a handle creates its scratch for 256-token chunks (tens
 * of MB at the 0.6B shape, plus V x 256 fp32 logits when every id is wanted)
 * and the TMA descriptors of every weight matrix; the launch sequence of each
 * prompt length is captured as a CUDA graph on its first use and replayed
 * afterwards (the call's ids, cursor and output pointers are read from device
 * memory, so a replay serves any call of that length; at most 8 lengths are
 * kept per handle, the least recently used replaced).
 * Blocks until `stream` completes.  Errors: MK_ERR_INVALID_ARG, MK_ERR_KV_FULL,
 * MK_ERR_BAD_TOKEN, MK_ERR_BAD_POSITION, MK_ERR_NUMERIC, MK_ERR_NO_MEMORY,
 * MK_ERR_UNSUPPORTED, MK_ERR_CUDA. */
int mk_prefill(mk_handle *h, const int32_t *d_in_ids, int32_t n, int32_t *d_out_ids,
               const mk_decode_opts *opts, mk_stream stream);

/* mk_decode without the wait: enqueue the launch on `stream` and return.  Same
 * arguments and argument errors as mk_decode; the device status comes from
 * mk_decode_wait, which must be called exactly once before the handle's next
 * call (another mk_decode / mk_decode_start / mk_reset_kv first gives
 * MK_ERR_INVALID_ARG).  With MK_DECODE_STREAM in opts->flags the mailbox is
 * reset to zero ids before the launch and every forward's id appears in it as
 * soon as the kernel has chosen it (mk_mailbox_read). */
int mk_decode_start(mk_handle *h, const int32_t *d_in_ids, int32_t n_in, int32_t n_steps,
                    int32_t *d_out_ids, const mk_decode_opts *opts, mk_stream stream);

/* Wait for the launch mk_decode_start enqueued; returns its status exactly as
 * mk_decode would and advances the cursor on success.  MK_ERR_INVALID_ARG when
 * nothing is pending. */
int mk_decode_wait(mk_handle *h);

/* Non-blocking read of the streaming mailbox: *n_out = ids the current (or last)
 * MK_DECODE_STREAM launch has published so far -- ids 0 .. *n_out-1 of that call,
 * each final -- and the first min(*n_out, cap) of them are copied to dst (host
 * memory).  The mailbox is host-mapped pinned memory the handle owns (max_seq
 * ids); the kernel writes an id, fences at system scope, then raises the count,
 * and this read takes the count with acquire ordering before the ids. */
int mk_mailbox_read(mk_handle *h, int32_t *dst, int32_t cap, int32_t *n_out);

/* mk_decode with HOST id buffers: copies h_in_ids to the device, decodes and
 * copies the ids back to h_out_ids (n_in + n_steps entries) -- the token-id
 * input of page B, "Why Does a Single Kernel Even Matter for TTS?", from host
 * memory.  The copies use handle-owned staging; at most max_seq ids per call.
 * Errors: as mk_decode. */
int mk_decode_host(mk_handle *h, const int32_t *h_in_ids, int32_t n_in, int32_t n_steps,
                   int32_t *h_out_ids, const mk_decode_opts *opts, mk_stream stream);

/* Launch geometry, cursor and byte counts of a handle (the bytes one forward
 * streams: the quantity page B, "Why Does a Single Kernel Even Matter for
 * TTS?", measures the kernel's bandwidth use by).  MK_ERR_INVALID_ARG on NULL. */
int mk_get_info(const mk_handle *h, mk_info *info);

/* The decode kernel mk_create would pick for this shape on a device with n_sm
 * multiprocessors (one CTA each), as mk_info.plan: 0 the general kernel, 1 the
 * one compiled for hidden 1024 / MLP 3072 / 16:8 heads of 128, 2 the one for
 * hidden 2048 / MLP 6144 / 16:8 heads of 128.  Runs the same shape checks and
 * layout choice as mk_create, needs no device and allocates nothing (the
 * compiled instantiations are an implementation choice; the pages have no
 * counterpart of this call).  Errors: MK_ERR_INVALID_ARG (NULL pointers,
 * n_sm < 1, a config mk_create rejects as invalid), MK_ERR_UNSUPPORTED. */
int mk_plan_for(const mk_config *cfg, int32_t n_sm, int32_t *plan);

/* Talker input rows: out[r] = sum_{j<n_books} books[j][codes[r][j]] + text[text_ids[r]],
 * accumulated in fp32 in table order (page B, "Why Does a Single Kernel Even
 * Matter for TTS?": each talker input is the sum of the 16 codebook embeddings
 * and the text embedding).
 * books: device bf16 [n_books][book_rows][H]; text: device bf16 [text_rows][H];
 * codes: device int32 [n][n_books]; text_ids: device int32 [n]; out: device fp32
 * [n][H].  Ids out of range give MK_ERR_BAD_TOKEN.  Blocks until `stream` completes. */
int mk_embed_sum(const void *books, int32_t n_books, int32_t book_rows, const void *text,
                 int32_t text_rows, int32_t hidden, const int32_t *codes,
                 const int32_t *text_ids, int32_t n, float *out, mk_stream stream);

/* mk_embed_sum for callers that cannot allocate device memory -- for example a
 * host that runs inside another allocator's fixed memory pool, or a streaming
 * thread that must not call cudaMalloc because it can block and synchronise the
 * device mid-stream.  The pages have no counterpart of this entry point.
 * Same arguments, result and errors as mk_embed_sum, and it allocates nothing:
 * its scratch (one status word per output row) is a 16 KB static device array
 * that every GPU loading the library holds until the process exits.
 *   - n may be at most 4096; larger n gives MK_ERR_INVALID_ARG.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that first call before any stream capture.
 *   - All calls share the array, which keeps the last call's contents; each
 *     call clears the words it uses.  Calls from several host threads are
 *     serialised; calls that overlap on the GPU (e.g. issued on different
 *     streams by other means) would race on the array. */
int mk_embed_sum_noalloc(const void *books, int32_t n_books, int32_t book_rows, const void *text,
                         int32_t text_rows, int32_t hidden, const int32_t *codes,
                         const int32_t *text_ids, int32_t n, float *out, mk_stream stream);

/* ---- paged KV cache: several sequences ------------------------------------
 * A decode step of many sequences at once, for callers that hold the layer loop
 * themselves: the operators below are one layer's attention block
 * (mk_matvec_q4 or mk_matmul_fp8 for the projections, mk_paged_append,
 * mk_paged_attention or, for prompts, mk_paged_prompt_attention) and what is
 * before and behind a step (mk_paged_plan, mk_adjust_logits), and
 * mk_export_kv hands them a context that mk_prefill or mk_decode has built.  The
 * pages cover one sequence per kernel only; these entry points have no
 * counterpart there.
 *
 * They differ from the handle's calls in one way: they enqueue on `stream` and
 * return, allocate nothing, keep nothing between calls and can be captured into
 * a CUDA graph (mk_export_kv is a call of the handle: it allocates a word, waits
 * and makes the handle's device current).  Argument errors are returned before
 * anything is enqueued.
 * What only the device sees (a page id outside the cache, a position outside
 * the table) is written to *status if it is not NULL -- the first error's code;
 * the caller zeroes it -- and no address outside the caller's buffers is formed.
 * All pointers are on the device that is current at the call; the stream is that
 * device's.  Tensors named in elements below have a contiguous last dimension,
 * and their base pointers and all other strides are multiples of 16 bytes.   */

#define MK_F32  0  /* element types of the operators below */
#define MK_BF16 1
#define MK_E4M3 2  /* 8-bit float, 4 exponent and 3 mantissa bits, largest value 448 */

/* One layer's cache: n_pages pages of page_size slots each for n_kv_heads heads
 * of head_dim (64 or 128) elements, in any order of pages, heads and slots given
 * by the strides (elements; the same for keys and values; not negative).  Token p
 * of sequence s is slot p % page_size of page table[s][p / page_size]; pages
 * may be shared by sequences that read them. */
typedef struct {
  void *k, *v;                 /* device, dtype MK_BF16 or MK_E4M3 */
  int32_t dtype;
  int32_t n_pages, n_kv_heads, page_size, head_dim;
  int64_t page_stride, head_stride, slot_stride;
  const float *k_scale, *v_scale; /* MK_E4M3: device [n_kv_heads], what a stored value is multiplied
                                     by (not subnormal); both or neither (NULL = 1).  MK_BF16: NULL */
  const int32_t *table;        /* device [table_rows][table_cols] page ids */
  int32_t table_rows, table_cols;
  int64_t table_stride;        /* elements from row to row; 0 = every row the same pages */
} mk_paged_kv;

typedef struct {
  int32_t n;                   /* token rows; 0 is a no-op */
  int32_t dtype;               /* of q, k, v and q_out: MK_F32 or MK_BF16 */
  int32_t n_q_heads;           /* heads of q; 0 = no q */
  const void *q, *k, *v;       /* device [n][heads][head_dim] */
  void *q_out;                 /* device [n][n_q_heads][head_dim]; may be q itself (same strides), else
                                  no part of q, k, v or the cache */
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head; /* strides, elements */
  const int32_t *seqs;         /* device [n] table row of each token row; NULL = row i is sequence i */
  const int32_t *slots;        /* device [n] token index p in its sequence; negative = a padding row,
                                  nothing of which is written */
  const float *rope;           /* device [rope_rows][head_dim / 2][2] cos, sin; NULL = no rotation */
  int32_t rope_rows;
  int32_t rope_mode;           /* as mk_config.rope_mode; 1 and 2 need positions and sections */
  int32_t mrope_sections[3];
  const int32_t *positions;    /* device [n] (rope_mode 0; NULL = the slots) or [3][n] */
  const void *q_norm, *k_norm; /* device bf16 [head_dim] RMSNorm gains before the rotation; NULL = none */
  float rms_eps;
  int32_t *status;             /* device, or NULL */
} mk_append_args;

/* Append n tokens' keys and values to their slots, QK-norm and rotation on the
 * way, and write the normalised and rotated queries: for every row
 *   q_out = rope(norm(q)), cache_k = round(rope(norm(k)) / k_scale), cache_v = round(v / v_scale)
 * with norm(x) = x / sqrt(mean(x^2) + eps) * gain per head, rope turning the
 * pairs (i, i + head_dim / 2), all in fp32 and rounded once (to nearest even,
 * MK_E4M3 saturating at +-448).  One row (a decode step's token) or many
 * (prompts: seqs and slots say where each row goes).  The keys' and the values'
 * memory is not the same, and no input is in a slot that the call writes.  A slot may be written by
 * at most one row of a call; with two, each element is one of theirs.  A row
 * whose sequence, slot or page is outside the table or the cache
 * (MK_ERR_BAD_PAGE) or whose position is outside the rotary table
 * (MK_ERR_BAD_POSITION) is skipped: nothing of it is written.  Errors:
 * MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED (head_dim), MK_ERR_CUDA. */
int mk_paged_append(const mk_paged_kv *kv, const mk_append_args *a, mk_stream stream);

typedef struct {
  int32_t n;                   /* query rows, one per table row: 0 <= n <= table_rows */
  int32_t dtype;               /* of q and out: MK_F32 or MK_BF16 */
  int32_t n_q_heads;           /* a multiple of n_kv_heads; head j reads kv head j / (n_q_heads / n_kv_heads) */
  int32_t sinks;               /* with a window: the first `sinks` tokens stay visible beside it; else unused.  (Where there
                                  was padding: a host built without it, which clears the struct, calls as before.) */
  const void *q;               /* device [n][n_q_heads][head_dim] */
  void *out;                   /* device, the same shape; may be q itself (same strides), else no part
                                  of it or the cache */
  int64_t q_row, q_head, out_row, out_head; /* strides, elements */
  float *lse;                  /* device [n][n_q_heads] log of the softmax's sum, or NULL; no part of q
                                  or out */
  const int32_t *lengths;      /* device [n] tokens a row reads, its own included; 0 = none, negative =
                                  a padding row, whose outputs are left as they were */
  int32_t window;              /* > 0: only the last `window` of them; 0 = all */
  float scale;                 /* of q.k; usually 1 / sqrt(head_dim) */
  void *workspace;             /* device, 16-byte aligned; the call's own until the stream has passed it */
  int64_t workspace_bytes;     /* at least mk_paged_attention_workspace */
  int32_t *status;             /* device, or NULL */
} mk_attention_args;

/* Attention of one new token per row over the paged cache:
 *   out = sum_p softmax_p(scale * q.k[p]) v[p],  lse = log sum_p exp(scale * q.k[p])
 * over p in [max(0, length - window), length) and, with a window, p in
 * [0, min(sinks, length)).  The work of several rows is cut
 * into equal shares over the SMs whatever the lengths (read on the device, so
 * that a captured call follows them); rows of up to about a thousand slots are
 * not cut, and a single row has at most 16 SMs a kv head.  The shares of a row are
 * joined in a fixed order: the same inputs give the same bits.  Scores are fp32
 * numbers (a q.k beyond their range is an infinity); over an MK_E4M3 cache, query
 * elements are rounded to 2^-38 of their head's largest and fp32 ones to 22 bits.  A row with no tokens gives
 * zeros and lse -inf.  Slots at and past a row's length are never read into a
 * result, whatever they hold.  A row with a page id outside the cache, or a
 * length past table_cols * page_size, gives NaN and MK_ERR_BAD_PAGE.  Several
 * new tokens of one sequence (drafted tokens) are rows with the same pages and
 * growing lengths.  Errors: MK_ERR_INVALID_ARG (a workspace too small among
 * them), MK_ERR_UNSUPPORTED (head_dim, more than 2^31 tiles of work), MK_ERR_CUDA. */
int mk_paged_attention(const mk_paged_kv *kv, const mk_attention_args *a, mk_stream stream);

/* mk_paged_attention for callers with an allocator of their own: `workspace` is
 * called, at most once and before anything is enqueued, with `context` and the
 * bytes of a workspace if the call needs one (rows of up to about a thousand
 * slots, and one row of not too many heads, need none); the arguments' workspace
 * and workspace_bytes are not looked at.  Its result is device memory on a 16-byte boundary that is the
 * call's own until the stream has passed it, or NULL (MK_ERR_NO_MEMORY).  It must
 * return: an exception must not pass through this call. */
typedef void *(*mk_workspace_fn)(void *context, int64_t bytes);
int mk_paged_attention_ask(const mk_paged_kv *kv, const mk_attention_args *a, mk_workspace_fn workspace,
                           void *context, mk_stream stream);

/* Bytes of workspace any mk_paged_attention call with these heads needs on the
 * current device (it does not depend on rows or lengths).  MK_ERR_INVALID_ARG,
 * MK_ERR_UNSUPPORTED or MK_ERR_CUDA as a negative result. */
int64_t mk_paged_attention_workspace(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim);

typedef struct {
  int32_t n;                   /* sequences, one per table row: 0 <= n <= table_rows; at most 16384 */
  int32_t rows;                /* of q and out */
  int32_t dtype;               /* of q and out: MK_BF16 (MK_F32: MK_ERR_UNSUPPORTED; mk_paged_attention takes it, a row
                                  for each token) */
  int32_t n_q_heads;           /* a multiple of n_kv_heads */
  const void *q;               /* device [rows][n_q_heads][head_dim] */
  void *out;                   /* device, the same shape; may be q itself (same strides), else no part of it or the cache */
  int64_t q_row, q_head, out_row, out_head; /* strides, elements */
  float *lse;                  /* device [rows][n_q_heads], or NULL; no part of q or out */
  const int32_t *starts;       /* device [n + 1], not decreasing: sequence i has rows [starts[i], starts[i + 1]); other rows
                                  are left as they were */
  const int32_t *lengths;      /* device [n] tokens of each sequence, those of its rows included; negative = its rows are
                                  padding, left as they were */
  int32_t window, sinks;       /* as for mk_paged_attention, at each row's own place */
  float scale;
  void *workspace;             /* device, 16-byte aligned; the call's own until the stream has passed it */
  int64_t workspace_bytes;     /* at least mk_paged_prompt_attention_workspace */
  int32_t *status;             /* device, or NULL */
} mk_prompt_args;

/* Causal attention of the last tokens of each sequence over the paged cache, their
 * own keys and values (appended before) included: row r of sequence i is its token
 *   t = lengths[i] - (starts[i + 1] - starts[i]) + r - starts[i]
 * and sees tokens p <= t, with a window those of (t - window, t] and [0, sinks).
 * Whole prompts (lengths = rows), chunks behind what is cached, drafted tokens.
 * Scores and sums are fp32; the weights multiply the values rounded to bf16,
 * over an MK_E4M3 cache to fp16, and query elements there to 2^-38 of their head's
 * largest.  (mk_paged_attention holds the weights over an MK_BF16 cache to 16 bits
 * and more: a token's result here may be off from that by 2^-8 of the sum of its
 * weighted |values|, beside the rounding of both.)  The same inputs give the same bits.  A row that sees nothing (t < 0)
 * gives zeros and lse -inf; tokens that a row does not see are never read into
 * its result, whatever they hold.  A row that sees a page id outside the cache, or
 * whose sequence is longer than table_cols * page_size, gives NaN and MK_ERR_BAD_PAGE;
 * a sequence whose starts are outside rows or decrease is skipped (MK_ERR_BAD_PAGE),
 * and all are where the others then overlap to more than 2^30 tiles.
 * Rows whose results are infinite or NaN take a slow path, a position at a time up
 * to the first score that is NaN (a prompt of 8192 tokens of 16 heads, all of which
 * see a NaN among the values: 80 ms instead of 0.2).  Errors:
 * MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED (dtype, head_dim, sizes), MK_ERR_CUDA; in
 * *status also MK_ERR_TIMEOUT if a wait inside the kernel ran out. */
int mk_paged_prompt_attention(const mk_paged_kv *kv, const mk_prompt_args *a, mk_stream stream);

/* The same as mk_paged_attention_ask is to mk_paged_attention. */
int mk_paged_prompt_attention_ask(const mk_paged_kv *kv, const mk_prompt_args *a, mk_workspace_fn workspace,
                                  void *context, mk_stream stream);

/* Bytes of workspace a mk_paged_prompt_attention call of these sizes needs on the
 * current device at most, or a negative error. */
int64_t mk_paged_prompt_attention_workspace(int32_t n, int32_t rows, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim);

typedef struct {
  int32_t n;                   /* sequences; at most 16384 */
  int32_t rows;                /* token rows of seqs and slots; n without counts */
  int32_t page_size;
  const int32_t *lengths;      /* device [n] tokens that each sequence has; negative = a padding row, which gets none */
  const int32_t *counts;       /* device [n] tokens that it gets (negative = 0), or NULL = one each */
  int32_t *table;              /* device [n][table_cols] page ids, extended in place */
  int32_t table_cols;
  int64_t table_stride;
  const int32_t *free;         /* device [free_count] pages that may be taken */
  int32_t free_count;
  const int32_t *used;         /* device [1] how many of them are taken already */
  int32_t *seqs, *slots;       /* device [rows] each token row's sequence and slot; rows without a token: -1 */
  int32_t *starts;             /* device [n + 1] first row of each sequence, and the end */
  int32_t *totals;             /* device [n] lengths + counts; may be lengths */
  int32_t *used_out;           /* device [1]; may be used */
  int32_t *status;             /* device, or NULL */
} mk_plan_args;

/* Plan a step: give each sequence's new tokens their rows, slots and, where its
 * last page is full, pages: token p of sequence i is in page table[i][p / page_size],
 * which is the next of `free` (counted through the sequences in order) if the
 * sequence had no such page.  With counts the rows are the sequences' tokens one
 * behind the other (for mk_paged_append with seqs and mk_paged_prompt_attention);
 * without, row i is sequence i (mk_paged_attention: totals are its lengths), and
 * starts are 0, 1, .. n.  A step that does not fit (rows, free pages or table_cols)
 * is not made: MK_ERR_KV_FULL in *status, no tokens for anyone, table, totals and
 * used_out as before.  Apart from the pairs named, outputs overlap nothing else
 * of the call.  Errors: MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED (n, rows near 2^31),
 * MK_ERR_CUDA. */
int mk_paged_plan(const mk_plan_args *a, mk_stream stream);

/* Copy cached tokens [first, first + count) of layer `layer` from the handle's
 * own cache to slots [slot, slot + count) of sequence `seq` of a paged cache of
 * the same heads (rotated keys as they are; rounded to MK_E4M3 with the cache's
 * scales if it is one): a prompt prefilled by mk_prefill continues in a batch.
 * Blocks until `stream` completes.  Errors: MK_ERR_INVALID_ARG (a range the
 * handle has not filled, a decode not yet waited for), MK_ERR_UNSUPPORTED (other
 * heads than the handle's), MK_ERR_BAD_PAGE (tokens whose page is bad are
 * skipped, the others copied), MK_ERR_NO_MEMORY, MK_ERR_CUDA. */
int mk_export_kv(mk_handle *h, int32_t layer, int32_t first, int32_t count, const mk_paged_kv *kv,
                 int32_t seq, int32_t slot, mk_stream stream);

/* ---- 4-bit weights ---------------------------------------------------------
 * w[n][k] = scales[n][k / group] * (code[n][k] - zero[n][k / group]), codes and
 * zeros 0 .. 15; byte k / 2 of a row holds code k in its low four bits when k is
 * even, in its high four when k is odd. */
typedef struct {
  int32_t m, n, k;             /* y [m][n] = x [m][k] w[n][k]^T; m or n 0 is a no-op; k <= 32768 */
  int32_t group;               /* 32, 64 or a multiple of 128 that divides k */
  int32_t dtype;               /* of x, residual and y: MK_F32 or MK_BF16 */
  const void *x;               /* device [m][k] */
  int64_t x_row;               /* row strides, elements */
  const void *codes;           /* device uint8 [n][k / 2], contiguous */
  const void *scales;          /* device bf16 [n][k / group], contiguous */
  const uint8_t *zeros;        /* device [n][k / group], contiguous; NULL = 8 everywhere */
  const void *residual;        /* device [m][n] added to the products, or NULL; may be y itself (same
                                  stride) */
  int64_t residual_row;
  void *y;                     /* device [m][n]; no part of x, and of the residual all or none */
  int64_t y_row;               /* residual_row and y_row need no alignment */
} mk_matvec_q4_args;

/* y = x w^T (+ residual) for a few rows x, accumulated in fp32 and rounded once.
 * x and the codes enter the products as they are (of x elements below 2^-141 of
 * their row's largest, bits below 2^-165 of it may be lost; scales of 2^80 and
 * more may overflow in a sum whose result would not).  Made for decode (m
 * of 1 to some tens); further rows read the weights again.  A zero above 15
 * counts modulo 16.  Errors: MK_ERR_INVALID_ARG,
 * MK_ERR_UNSUPPORTED (group, k), MK_ERR_CUDA. */
int mk_matvec_q4(const mk_matvec_q4_args *a, mk_stream stream);

/* ---- 8-bit floating-point products with block scales ------------------------
 * For the projections of many rows (prompts, large batches).  Both operands are
 * MK_E4M3 codes that stand for code * scale: of a row of x each 128 elements have a
 * scale, of w each 128 x 128 block (the last block of a row or column may be
 * shorter). */
typedef struct {
  int32_t m, k;                /* rows; 0 is a no-op.  k: a multiple of 16 */
  int32_t dtype;               /* of x: MK_F32 or MK_BF16 */
  const void *x;               /* device [m][k]; rows on 16 bytes */
  int64_t x_row;               /* row strides, elements */
  void *codes;                 /* device MK_E4M3 [m][k]; rows on 16 bytes; no part of x or scales */
  int64_t codes_row;
  float *scales;               /* device [m][(k + 127) / 128]; no part of x */
  int64_t scales_row;
} mk_quantize_fp8_args;

/* scale = largest |x| of the 128 / 448 as fp32 (1 for a block of zeros), code = x
 * / scale as fp32, rounded to nearest even and saturating.  NaN stays NaN and does
 * not count for the scale.  Errors: MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED (2^31
 * blocks and more), MK_ERR_CUDA. */
int mk_quantize_fp8(const mk_quantize_fp8_args *a, mk_stream stream);

typedef struct {
  int32_t m, n, k;             /* y [m][n] = x [m][k] w [n][k]^T; m or n 0 is a no-op; k a multiple of 16 */
  int32_t dtype;               /* of residual and y: MK_F32 or MK_BF16 */
  const void *x;               /* device MK_E4M3 [m][k]; rows on 16 bytes, not overlapping */
  int64_t x_row;               /* row strides, elements */
  const float *x_scale;        /* device [m][(k + 127) / 128] */
  int64_t x_scale_row;
  const void *w;               /* device MK_E4M3 [n][k]; rows on 16 bytes, not overlapping */
  int64_t w_row;
  const float *w_scale;        /* device [(n + 127) / 128][(k + 127) / 128], contiguous */
  const void *residual;        /* device [m][n] added to the products, or NULL; may be y itself (same stride) */
  int64_t residual_row;
  void *y;                     /* device [m][n]; no part of x, w or the scales, of the residual all or none */
  int64_t y_row;
  int32_t *status;             /* device, or NULL: MK_ERR_TIMEOUT if a wait inside the kernel ran out */
} mk_matmul_fp8_args;

/* y[t][j] = sum_b x_scale[t][b] w_scale[j / 128][b] sum_{k in block b} x[t][k] w[j][k]
 * (+ residual): a block's products are summed by the tensor cores and multiplied by
 * the product of the two scales, the blocks are added in fp32, rounded once.  (Blocks whose
 * scales' product leaves fp32's normal numbers, 2^-126 to 2^128, lose bits or are
 * infinite or NaN.)  The same inputs give the same bits.  Errors:
 * MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED (sizes near 2^31), MK_ERR_CUDA. */
int mk_matmul_fp8(const mk_matmul_fp8_args *a, mk_stream stream);

/* ---- logits ------------------------------------------------------------------ */
typedef struct {
  int32_t n, vocab;            /* rows, tokens; 0 is a no-op */
  int32_t dtype;               /* of x and out: MK_F32 or MK_BF16 */
  const void *x;               /* device [n][vocab] logits */
  void *out;                   /* device [n][vocab]; may be x itself (same stride), else no part of it */
  int64_t x_row, out_row;      /* row strides, elements (any) */
  const int32_t *tokens;       /* device [n][columns] each row's history; ids outside the vocabulary do not count */
  int64_t tokens_row;
  int32_t columns;
  const int32_t *lengths;      /* device [n] tokens of the history (at most columns count), or NULL = columns;
                                  negative = a padding row, whose logits in out are left as they were */
  const int32_t *prompts;      /* device [n] how many of them are the prompt, or NULL = none */
  const float *repetition, *presence, *frequency; /* device [n], or NULL = 1, 0, 0 */
  const int32_t *bias_ids;     /* device [n][biases] tokens; ids outside the vocabulary do not count */
  const float *bias;           /* device [n][biases] */
  int64_t ids_row, bias_row;
  int32_t biases;
  const int32_t *mask;         /* device [n][(vocab + 31) / 32], bit t % 32 of word t / 32 set = allowed; or NULL */
  int64_t mask_row;            /* 0 = the same mask for every row */
} mk_logits_args;

/* Adjust logits before a token is chosen, in this order:
 *   in the history:                    x = x > 0 ? x / repetition : x * repetition
 *   c > 0 times in it behind the prompt: x = x - frequency c - presence
 *   x = x + the biases of the token (in their order), x = -inf if it is not allowed
 * in fp32, rounded once; a token that none of them touches is copied.  A row whose
 * mask allows nothing is -inf throughout.  A token with several biases takes a look
 * at all of its row's: tens of thousands of tokens may have one, few several.  Errors: MK_ERR_INVALID_ARG,
 * MK_ERR_UNSUPPORTED (sizes near 2^31), MK_ERR_CUDA. */
int mk_adjust_logits(const mk_logits_args *a, mk_stream stream);

/* Free everything the handle owns (not the borrowed weights): the end of the
 * handle lifecycle that mk_create starts.  NULL is a no-op; always MK_OK. */
int mk_destroy(mk_handle *h);

/* Static string naming a status code (the error words the kernel sets instead
 * of trapping, so that a failed step never takes the GPU down; the pages
 * define no error model).  Unknown codes give "unknown error". */
const char *mk_error_string(int code);

#ifdef __cplusplus
}
#endif
#endif /* MK_H */
