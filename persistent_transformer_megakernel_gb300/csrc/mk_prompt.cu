// Attention of whole prompts over a paged KV cache (mk_paged_prompt_attention).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_mma.cuh"
#include "mk_paged.h"
#include "mk_tc.cuh"

namespace mkprompt {

using namespace mktc;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kCopyWarps = 4, kWarps = kSoftWarps + 1 + kCopyWarps, kThreads = 32 * kWarps;
constexpr int kRows = 128;            // of a query tile (the MMA's M); a CTA has two
constexpr int kBlock = 128;           // cached positions of a step
constexpr int kSlots = 4;             // key and value tiles in shared memory, in turn
constexpr int kMaxSequences = 16384;
constexpr int kLeastBlocks = 8;       // an item of at most so many blocks is not split
constexpr long long kWaitNs = 2000000000LL;

struct PromptParams {
  const void *q, *k, *v;
  void *out;
  float *lse;
  int64_t q_row, q_head, out_row, out_head, page_stride, head_stride, slot_stride, table_stride;
  const int32_t *table, *starts, *lengths;
  const float *k_scale, *v_scale;
  int32_t *status;
  int4 *records;               // [0].x: partial results in all; then of each {first row, tokens, virtual head, parts or 0}
  float *parts;                // [partial result][2 kRows][D + 4]: O, maximum, sum
  mkw::Divisor page_size, heads;   // heads: query heads of a tile's token
  int n, rows, hq, hkv, group, n_pages, capacity, window, sinks;
  int blocks, vh;              // head blocks of a kv head, virtual heads hkv * blocks
  int tokens;                  // of a tile: kRows / heads
  int sms;
  float scale;
};

template <int D>
struct Layout {
  static constexpr int ATOMS = D / 64;
  static constexpr uint32_t TILE = ATOMS * 128 * 128;      // 128 rows of D 16-bit elements
  static constexpr uint32_t CONTROL = 1024, Q = CONTROL, KV = Q + 2 * TILE;
  static constexpr int SMEM = static_cast<int>(1024 + KV + kSlots * TILE);
  static constexpr uint32_t S_COLS = kBlock, O_COL = 2 * S_COLS, TMEM_COLS = 512;
};

__device__ __forceinline__ void report(int32_t *status, int code) {
  if (status) atomicCAS(status, 0, code);
}
// byte offset of 16-byte piece c of row r of a tile
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * (128 * 128) + static_cast<uint32_t>(r) * 128 + ((static_cast<uint32_t>(c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void fence_to_tensor_cores() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- which part of which rows a CTA has ---------------------------------------------

// a pair of tiles: rows of one sequence and virtual head
struct Pair {
  int row, count, pos;         // first row, tokens, and the first one's position
  int lo, head, skip, blocks;  // blocks of keys: number(0) .. number(blocks - 1)
  __device__ __forceinline__ int number(int j) const { return j < head ? j : j + skip; }
};
__device__ __forceinline__ Pair pair_of(const PromptParams &p, int start, int count, int length, int t) {
  Pair x;
  const int first = t * 2 * p.tokens;
  x.row = start + first;
  x.count = min(2 * p.tokens, count - first);
  x.pos = length - count + first;
  const int hi = x.pos + x.count;
  x.lo = p.window > 0 && x.pos + 1 > p.window ? x.pos + 1 - p.window : 0;
  const int low = x.lo / kBlock;
  x.head = min((p.sinks + kBlock - 1) / kBlock, low);
  x.skip = low - x.head;
  x.blocks = hi > 0 && length <= p.capacity ? (hi + kBlock - 1) / kBlock - x.skip : 0;
  return x;
}

struct Task {
  int seq, pair, vh, part, parts, slot;
};

// exclusive sum over the block's threads, and the total
__device__ __forceinline__ long long block_sum(long long x, long long *warps, long long &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) warps[w] = s;
  __syncthreads();
  total = 0;
  long long before = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += warps[i];
    total += warps[i];
  }
  return before + s - x;
}

__device__ __forceinline__ int count_of(const PromptParams &p, int i, bool *bad) {
  const int a = p.starts[i], b = p.starts[i + 1];
  if (a < 0 || b < a || b > p.rows) {
    *bad = true;
    return 0;
  }
  return p.lengths[i] < 0 ? 0 : b - a;
}

// Task `index` in the order of sequences, their last rows (which see most) first; false if there are fewer.  Every item
// (pair of tiles and virtual head) of more blocks than an equal share of all the work is cut into parts.
__device__ bool find_task(const PromptParams &p, int index, int *before, Task *s_task, int *results) {
  __shared__ long long s_warps[kWarps];
  const int tid = threadIdx.x, n = p.n, step = 2 * p.tokens;
  bool bad = false;
  for (int i = tid; i < n; i += kThreads) before[i] = (count_of(p, i, &bad) + step - 1) / step;
  if (bad) report(p.status, MK_ERR_BAD_PAGE);
  __syncthreads();
  const int per = (n + kThreads - 1) / kThreads, a = min(n, tid * per), b = min(n, a + per);
  int mine = 0;
  for (int i = a; i < b; ++i) mine += before[i];
  long long total;
  int at = static_cast<int>(block_sum(mine, s_warps, total));
  for (int i = a; i < b; ++i) {
    const int c = before[i];
    before[i] = at;
    at += c;
  }
  const int pairs = static_cast<int>(total);
  if (tid == 0) before[n] = pairs;
  __syncthreads();
  const int share = (pairs + kThreads - 1) / kThreads, p0 = min(pairs, tid * share), p1 = min(pairs, p0 + share);
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= p0) lo = mid;
    else hi = mid;
  }
  const int i0 = lo;
  long long cost = 0;
  for (int pass = 0;; ++pass) {
    // pass 0: all blocks; pass 1: tasks and partial results before this thread's; pass 2: the task
    const long long limit = pass == 0 ? 0 : max(static_cast<long long>(kLeastBlocks), (total * p.vh + p.sms - 1) / p.sms);
    long long sum = 0;
    const long long from = pass == 2 ? cost : 0;
    int i = i0, start = 0, count = 0, length = 0, of = -1;
    for (int x = p0; x < p1; ++x) {
      while (x >= before[i + 1]) ++i;
      if (of != i) {
        of = i;
        start = p.starts[i];
        count = p.starts[i + 1] - start;
        length = p.lengths[i];
      }
      const int t = before[i + 1] - 1 - x;
      const int blocks = pair_of(p, start, count, length, t).blocks;
      if (pass == 0) {
        sum += blocks;
        continue;
      }
      const int parts = blocks > limit ? static_cast<int>((blocks + limit - 1) / limit) : 1, tasks = parts * p.vh;
      if (pass == 2) {
        const int first = static_cast<int>((from + sum) >> 32), slots = static_cast<int>(from + sum);
        if (index >= first && index < first + tasks) {
          const int k = index - first;
          *s_task = Task{i, t, k / parts, k % parts, parts, parts > 1 ? slots + k : -1};
        }
      }
      sum += (static_cast<long long>(tasks) << 32) | (parts > 1 ? tasks : 0);
    }
    if (pass == 0) {
      block_sum(sum, s_warps, total);
    } else if (pass == 1) {
      long long all;
      cost = block_sum(sum, s_warps, all);
      *results = static_cast<int>(all);
      if (index >= static_cast<int>(all >> 32)) return false;
    } else {
      break;
    }
  }
  __syncthreads();
  return true;
}

// ---- the kernel ------------------------------------------------------------------------

// the 8 16-bit operands of a 16-byte piece of a bf16 query row: as they are, or times a power of two as fp16
template <bool FP8>
__device__ __forceinline__ uint4 query_piece(uint4 w, float f, uint32_t flip) {
  w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
  if constexpr (!FP8) return w;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (&w.x)[i];
    const __half2 h = __floats2half2_rn(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f);
    r[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack_weights(float a, float b) {
  if constexpr (FP8) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// where a token of a sequence is: element offset of its slot of kv head 0, or -1
__device__ __forceinline__ int64_t slot_of(const PromptParams &p, int seq, int pos) {
  const int col = p.page_size.quotient(pos);
  const int page = p.table[seq * p.table_stride + col];
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) return -1;
  return page * p.page_stride + (pos - col * static_cast<int>(p.page_size.value)) * p.slot_stride;
}

template <bool FP8, int N>
__device__ __forceinline__ void cached(const void *base, int64_t at, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (FP8) x[i] = static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(base)[at + i]);
    else x[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at + i]);
  }
}

// A row by fp32 products, one warp, position by position: for rows whose tensor-core result is not finite.  There a
// value outside the row's mask (infinity or NaN times a weight of 0) or a sum of large values can have done it, so that
// the answer may be finite all the same.  Leaves the row's maximum (log2 units), sum and O (lane's elements) where the sum
// counts weights times `shrink`.
template <bool FP8, int D>
__device__ void row_alone(const PromptParams &p, const Task &task, const Pair &x, int b0, int b1, int row, int head, int pos, int lane, float &m, float &l,
                          float (&o)[D / 32], float &shrink) {
  constexpr int E = D / 32;
  float q[E];
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + row * p.q_row + head * p.q_head + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = __bfloat162float(src[i]), o[i] = 0.f;
  const int kvh = task.vh / p.blocks;
  const float c = p.scale * 1.4426950408889634f * (FP8 && p.k_scale ? p.k_scale[kvh] : 1.f);
  shrink = 1.f;
  for (int i = 1; i < pos + 1 && i > 0; i <<= 1) shrink *= 0.5f;
  m = -INFINITY;
  l = 0.f;
  for (int b = b0; b < b1; ++b) {
    const int first = x.number(b) * kBlock;
    for (int at = first; at < first + kBlock && at <= pos; ++at) {
      if (p.window > 0 && at <= pos - p.window && at >= p.sinks) continue;
      const int64_t slot = slot_of(p, task.seq, at);
      if (slot < 0) {
        m = l = NAN;
        return;
      }
      float k[E], v[E];
      cached<FP8>(p.k, slot + kvh * p.head_stride + lane * E, k);
      cached<FP8>(p.v, slot + kvh * p.head_stride + lane * E, v);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) s += q[i] * k[i];
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
      s *= c;
      const float mx = fmaxf(m, s), base = mx == -INFINITY ? 0.f : mx;
      const float f = mkw::exp2_fast(m - base), w = mkw::exp2_fast(s - base) * shrink;
      m = mx;
      l = l * f + w;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        // an infinity stays one, however small its weight (fp32's may be 0; a score of -infinity makes it 0 in truth)
        const float old = fabsf(o[i]) < INFINITY ? o[i] * f : o[i];
        o[i] = old + (fabsf(v[i]) < INFINITY ? w * v[i] : s == -INFINITY ? NAN : v[i]);
      }
    }
  }
}

template <bool FP8, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using LY = Layout<D>;
  // over an 8-bit cache weights are fp16 numbers up to 2^15: the running maximum may lag by 1 (log2) behind 2^14; bf16
  // ones may lag by 8
  constexpr float kShift = FP8 ? 14.f : 0.f, kLag = FP8 ? 1.f : 8.f;
  constexpr uint32_t kIdS = FP8 ? idesc_f32(kRows, kBlock) : idesc_bf16_f32(kRows, kBlock);
  constexpr uint32_t kIdO = (FP8 ? idesc_f32(kRows, D) : idesc_bf16_f32(kRows, D)) | kBMajorN;
  extern __shared__ unsigned char smraw[];
  __shared__ Task s_task;
  mkw::follow_previous_kernel();
  unsigned char *sm = smraw + ((1024u - (smem_addr(smraw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  int results = 0;
  const bool any = find_task(p, blockIdx.x, reinterpret_cast<int *>(sm + LY::Q), &s_task, &results);
  if (blockIdx.x == 0 && tid == 0 && p.records) p.records[0] = make_int4(results, 0, 0, 0);
  if (!any) return;
  const Task task = s_task;
  const int start = p.starts[task.seq], length = p.lengths[task.seq];
  const Pair x = pair_of(p, start, p.starts[task.seq + 1] - start, length, task.pair);
  const int b0 = static_cast<int>(static_cast<int64_t>(x.blocks) * task.part / task.parts), b1 = static_cast<int>(static_cast<int64_t>(x.blocks) * (task.part + 1) / task.parts);
  const int kvh = task.vh / p.blocks, head0 = kvh * p.group + (task.vh - kvh * p.blocks) * static_cast<int>(p.heads.value);
  const int heads = min(static_cast<int>(p.heads.value), (kvh + 1) * p.group - head0);
  // the positions of a tile's first and last row, and whether any of its rows sees any of block b
  auto first_of = [&](int tile) { return x.pos + tile * p.tokens; };
  auto last_of = [&](int tile) { return x.pos + min(x.count, (tile + 1) * p.tokens) - 1; };
  auto sees = [&](int tile, int b) {
    const int from = b * kBlock;
    return x.count > tile * p.tokens && from <= last_of(tile) && (p.window == 0 || from + kBlock - 1 > first_of(tile) - p.window || from < p.sinks);
  };

  uint64_t *full = reinterpret_cast<uint64_t *>(sm), *empty = full + kSlots, *sfull = empty + kSlots, *pfull = sfull + 2, *ofull = pfull + 2;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(ofull + 2);
  unsigned char *Qs = sm + LY::Q, *KVs = sm + LY::KV;
  __syncthreads();                                         // (the sums of find_task were where Q goes)
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], kCopyWarps), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sfull[i], 1), mbar_init(&pfull[i], 4), mbar_init(&ofull[i], 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tslot, LY::TMEM_COLS);

  // ---- softmax warps: a thread a row; its query to shared memory --------------------------
  const int tile = warp >> 2, r = (warp & 3) * 32 + lane;
  const int token = p.heads.quotient(r), head = r - token * static_cast<int>(p.heads.value), index = tile * p.tokens + token;
  const bool live = warp < kSoftWarps && token < p.tokens && head < heads && index < x.count;
  float to_log2 = p.scale * 1.4426950408889634f * (FP8 && p.k_scale ? p.k_scale[kvh] : 1.f);
  const uint32_t flip = to_log2 < 0.f ? 0x80008000u : 0u;   // a negative factor's sign goes to the query
  to_log2 = fabsf(to_log2);
  if (warp < kSoftWarps) {
    uint4 w[D / 8];
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + (x.row + index) * p.q_row + (head0 + head) * p.q_head;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) w[c] = live ? *reinterpret_cast<const uint4 *>(src + c * 8) : make_uint4(0, 0, 0, 0);
    float f = 1.f;
    if constexpr (FP8) {
      // the row's largest element to [2^13, 2^14): fp16 holds what is at least 2^-38 of it
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = (&w[c].x)[i];
          a = fmaxf(a, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
        }
      const int e = a > 0.f && a < INFINITY ? max(-126, min(126, 13 - ilogbf(a))) : 0;
      f = ldexpf(1.f, e);
      to_log2 *= ldexpf(1.f, -e);
    }
#pragma unroll
    for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4 *>(Qs + tile * LY::TILE + piece_at(r, c)) = query_piece<FP8>(w[c], f, flip);
    fence_to_tensor_cores();
  }
  // (a factor of 0 would make the -infinity of a hidden score NaN; the smallest normal one does what 0 does)
  to_log2 = fmaxf(to_log2, 1.2e-38f);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);

  if (warp > kMmaWarp) {
    // ---- copies: a warp has 32 positions of a block, a lane looks one of them up ------------
    constexpr int ES = FP8 ? 1 : 2, PIECES = D * ES / 16, ROWS = 32 / PIECES;   // 16-byte pieces of a row, rows a copy
    const int cw = warp - kMmaWarp - 1;
    int n_tiles = 0, told = 0;                             // tiles asked for, tiles told of
    bool ok = true;
    auto tell = [&](int upto) {
      fence_to_tensor_cores();
      __syncwarp();
      for (; told < upto; ++told)
        if (lane == 0) mbar_arrive(&full[told % kSlots]);
    };
    auto look_up = [&](int b) -> int64_t {                 // byte offset of this lane's slot; -1 not read, -2 bad
      const int pos = x.number(b) * kBlock + cw * 32 + lane;
      if (pos > last_of(1) || (pos < x.lo && pos >= p.sinks)) return -1;
      const int64_t at = slot_of(p, task.seq, pos);
      return at < 0 ? -2 : (at + kvh * p.head_stride) * ES;
    };
    int64_t next = b0 < b1 ? look_up(b0) : -1;
    for (int b = b0; b < b1 && ok; ++b) {
      const int64_t at = next;
      const bool bad = at == -2;
      if (bad) report(p.status, MK_ERR_BAD_PAGE);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++n_tiles) {
        const int slot = n_tiles % kSlots;
        if (n_tiles >= kSlots) {
          const uint32_t parity = (n_tiles / kSlots - 1) & 1;
          if (!__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], parity))) {
            if constexpr (!FP8) mkw::cp_async_wait<0>();
            tell(n_tiles);
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], parity, kWaitNs))) {
              if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
              ok = false;
              break;
            }
          }
        }
        const unsigned char *base = static_cast<const unsigned char *>(kv ? p.v : p.k);
        unsigned char *to = KVs + slot * LY::TILE;
        if constexpr (!FP8) {
          const uint32_t to_at = smem_addr(to);
#pragma unroll
          for (int i = 0; i < 32 / ROWS; ++i) {
            const int rr = i * ROWS + lane / PIECES, c = lane % PIECES;
            const int64_t o = __shfl_sync(0xffffffffu, at, rr);
            mkw::cp_async16(to_at + piece_at(cw * 32 + rr, c), base + (o < 0 ? 0 : o + c * 16), o >= 0);
          }
          mkw::cp_async_commit();
        } else {
#pragma unroll
          for (int i0 = 0; i0 < 32 / ROWS; i0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = (i0 + i) * ROWS + lane / PIECES, c = lane % PIECES;
              const int64_t o = __shfl_sync(0xffffffffu, at, rr);
              w[i] = o < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(base + o + c * 16);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = (i0 + i) * ROWS + lane / PIECES, c = lane % PIECES;
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) mkw::e4m3x4_to_half2((&w[i].x)[e], h[2 * e], h[2 * e + 1]);
              *reinterpret_cast<uint4 *>(to + piece_at(cw * 32 + rr, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4 *>(to + piece_at(cw * 32 + rr, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
        }
        if (kv == 0) {
          if (__any_sync(0xffffffffu, bad)) {
            // a key that is not there is NaN: so are the scores of rows that see it
            if constexpr (!FP8) mkw::cp_async_wait<0>();
            __syncwarp();
            if (bad)
              for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4 *>(to + piece_at(cw * 32 + lane, c)) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
          }
          if (b + 1 < b1) next = look_up(b + 1);
        }
        if constexpr (FP8) {
          tell(n_tiles + 1);
        } else if (n_tiles >= 2) {
          mkw::cp_async_wait<2>();
          tell(n_tiles - 1);
        }
      }
    }
    if constexpr (!FP8) mkw::cp_async_wait<0>();
    if (ok) tell(n_tiles);
  } else if (warp == kMmaWarp) {
    // ---- products: S = Q K^T of a tile, then O += P V with P where S was, so that the next S of the tile comes behind it
    if (b0 < b1) {
      // descriptors: the low words move with the tile, the high ones are constants
      const uint64_t kd = desc_sw128(smem_addr(KVs)), vd = desc_mn_sw128_at(smem_addr(KVs), kBlock * 128, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(desc_sw128(smem_addr(Qs))), k_lo = static_cast<uint32_t>(kd), v_lo = static_cast<uint32_t>(vd);
      const uint32_t k_hi = static_cast<uint32_t>(kd >> 32), v_hi = static_cast<uint32_t>(vd >> 32);
      bool ok = true;
      uint32_t pph[2] = {0, 0};
      bool first[2] = {true, true};
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_test(bar, parity)) && !__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs))) {
          if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
          ok = false;
        }
        tc_fence_after();
        return ok;
      };
      auto scores = [&](int t, int n_tile) {
        if (elect_one()) {
          const uint32_t k_at = k_lo + (n_tile % kSlots) * (LY::TILE >> 4), q_at = q_lo + t * (LY::TILE >> 4);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = ((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4;
            mma_bf16(tmem + t * LY::S_COLS, desc_of(q_at + off, k_hi), desc_of(k_at + off, k_hi), kIdS, s != 0);
          }
          mma_commit(&sfull[t]);
        }
        __syncwarp();
      };
      auto release = [&](int n_tile) {
        if (elect_one()) mma_commit(&empty[n_tile % kSlots]);
        __syncwarp();
      };
      if (wait(&full[0], 0)) {
        for (int t = 0; t < 2; ++t)
          if (sees(t, x.number(b0))) scores(t, 0);
        release(0);
      }
      for (int b = b0; b < b1 && ok; ++b) {
        const int j = b - b0, vt = 2 * j + 1, kt = 2 * j + 2;
        if (!wait(&full[vt % kSlots], (vt / kSlots) & 1)) break;
        const bool more = b + 1 < b1;
        for (int t = 0; t < 2 && ok; ++t) {
          if (sees(t, x.number(b))) {
            if (!wait(&pfull[t], pph[t])) break;
            pph[t] ^= 1;
            if (elect_one()) {
              const uint32_t v_at = v_lo + (vt % kSlots) * (LY::TILE >> 4);
#pragma unroll
              for (int s = 0; s < kBlock / 16; ++s)
                mma_f16_ta(tmem + LY::O_COL + t * D, tmem + t * LY::S_COLS + s * 8, desc_of(v_at + s * (2048 >> 4), v_hi), kIdO, !(first[t] && s == 0));
            }
            __syncwarp();
            first[t] = false;
          }
          if (more && sees(t, x.number(b + 1)) && wait(&full[kt % kSlots], (kt / kSlots) & 1)) scores(t, kt);
        }
        if (more && !wait(&full[kt % kSlots], (kt / kSlots) & 1)) break;
        release(vt);
        if (more) release(kt);
      }
      if (elect_one()) mma_commit(&ofull[0]);              // all of it is done (also where a wait ran out)
      __syncwarp();
      mbar_wait(&ofull[0], 0, kWaitNs);
      if (lane == 0) mbar_arrive(&ofull[1]);
    }
  } else {
    // ---- softmax ---------------------------------------------------------------------------
    const int pos = first_of(tile) + token;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + tile * LY::S_COLS, o_at = tmem + lanes + LY::O_COL + tile * D;
    // the warp's rows see all of a block whose positions are in [row_lo, row_hi] (or first tokens up to it)
    const int hidden_below = p.window > 0 ? pos - p.window : -1;   // hidden: at <= hidden_below and not a first token
    float m = -INFINITY, l = 0.f;                          // m: of scores before to_log2
    uint32_t phase = 0;
    bool started = false, ok = true;
    for (int b = b0; b < b1 && ok; ++b) {
      const int blk = x.number(b);
      if (!sees(tile, blk)) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(&sfull[tile], phase, kWaitNs))) {
        if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
        ok = false;
        break;
      }
      phase ^= 1;
      tc_fence_after();
      const int from = blk * kBlock;
      const bool edge = __any_sync(0xffffffffu, from + kBlock - 1 > pos || (from <= hidden_below && from + kBlock > p.sinks));
      auto load = [&](int c, float (&v)[32]) {
        uint32_t u[32];
        tmem_ld32(s_at + c, u);
        tmem_ld_wait(u);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
        if (edge) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int at = from + c + i;
            if (at > pos || (at <= hidden_below && at >= p.sinks)) v[i] = -INFINITY;
          }
        }
      };
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < kBlock; c += 32) {
        float v[32];
        load(c, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, v[i]);
      }
      const bool grows = (mx - m) * to_log2 > kLag;        // (also from -infinity; not if both are)
      if (__any_sync(0xffffffffu, grows)) {
        const float alpha = grows ? mkw::exp2_fast((m - mx) * to_log2) : 1.f;
        if (grows) m = mx;
        l *= alpha;
        if (started) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t u[32];
            tmem_ld32(o_at + c, u);
            tmem_ld_wait(u);
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
            tmem_st32(o_at + c, u);
          }
        }
      }
      started = true;
      const float base = m == -INFINITY ? 0.f : fmaf(-m, to_log2, kShift);
#pragma unroll 1
      for (int c = 0; c < kBlock; c += 32) {
        float v[32];
        load(c, v);
        uint32_t w[16];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = mkw::exp2_fast(fmaf(v[2 * i], to_log2, base)), z = mkw::exp2_fast(fmaf(v[2 * i + 1], to_log2, base));
          sum[0] += a;
          sum[1] += z;
          w[i] = pack_weights<FP8>(a, z);
        }
        l += sum[0] + sum[1];
        tmem_st16(s_at + c / 2, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[tile]);
    }
    // ---- results ------------------------------------------------------------------------------
    if (b0 < b1 && !__all_sync(0xffffffffu, mbar_wait(&ofull[1], 0, kWaitNs))) {
      if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
      ok = false;
    }
    tc_fence_after();
    const bool whole = task.parts == 1;
    const float vs = FP8 && p.v_scale ? p.v_scale[kvh] : 1.f;
    const bool outside = length > p.capacity;              // a sequence longer than its row of the table
    if (outside && lane == 0) report(p.status, MK_ERR_BAD_PAGE);
    float *part = whole ? nullptr : p.parts + (static_cast<int64_t>(task.slot) * 2 * kRows + tile * kRows + r) * (D + 4);
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (x.row + index) * p.out_row + (head0 + head) * p.out_head;
    const float inv = outside || !ok ? NAN : !whole ? 1.f : l == 0.f ? 0.f : __frcp_rn(l) * vs;
    bool strange = false;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t u[32];
      float y[32];
      if (started && ok) {
        tmem_ld32(o_at + c, u);
        tmem_ld_wait(u);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        y[i] = (started && ok && l != 0.f ? __uint_as_float(u[i]) : 0.f) * inv;
        strange |= !(fabsf(y[i]) < INFINITY);
      }
      if (live) {
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(dst + c + 8 * i) =
                make_uint4(pack_weights<false>(y[8 * i], y[8 * i + 1]), pack_weights<false>(y[8 * i + 2], y[8 * i + 3]),
                           pack_weights<false>(y[8 * i + 4], y[8 * i + 5]), pack_weights<false>(y[8 * i + 6], y[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4 *>(part + c + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
      }
    }
    m = m == -INFINITY ? m : m * to_log2 - kShift;         // log2 units, as the sum is scaled
    if (outside || !ok) m = l = NAN;
    if (live) {
      if (!whole) part[D] = m, part[D + 1] = l;
      else if (p.lse) p.lse[static_cast<int64_t>(x.row + index) * p.hq + head0 + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
    strange |= !(fabsf(l) < INFINITY);
    for (unsigned rest = __ballot_sync(0xffffffffu, strange && live && ok && !outside); rest; rest &= rest - 1u) {
      const int from = __ffs(rest) - 1;
      const int row = x.row + __shfl_sync(0xffffffffu, index, from), hd = head0 + __shfl_sync(0xffffffffu, head, from);
      float rm, rl, o[D / 32], shrink;
      row_alone<FP8, D>(p, task, x, b0, b1, row, hd, __shfl_sync(0xffffffffu, pos, from), lane, rm, rl, o, shrink);
      // (the sum is of weights times shrink: as many log2 units less for the maximum)
      const float grow = 1.f / shrink;
      if (whole) {
        const float f = rl == 0.f ? 0.f : rl != rl ? NAN : __frcp_rn(rl);
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) + row * p.out_row + hd * p.out_head + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) to[i] = __float2bfloat16_rn(o[i] * f * vs);
        if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(row) * p.hq + hd] = rl == 0.f ? -INFINITY : (rm + log2f(rl * grow)) * 0.69314718055994531f;
      } else {
        float *to = p.parts + (static_cast<int64_t>(task.slot) * 2 * kRows + tile * kRows + (warp & 3) * 32 + from) * (D + 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) to[lane * (D / 32) + i] = o[i];
        if (lane == 0) to[D] = rm + log2f(grow), to[D + 1] = rl;
      }
    }
    if (!whole && tid == 0) p.records[1 + task.slot] = make_int4(x.row, x.count, task.vh, task.part == 0 ? task.parts : 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, LY::TMEM_COLS);
}

// Joins the parts of an item, a row a warp: CTA (c, y) takes rows y 8 .. of the item whose first part is partial result c.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PromptParams p) {
  constexpr int E = D / 32;
  mkw::follow_previous_kernel();
  if (static_cast<int>(blockIdx.x) >= p.records[0].x) return;
  const int4 rec = p.records[1 + blockIdx.x];
  if (rec.w == 0) return;
  const int lane = threadIdx.x & 31;
  const int kvh = rec.z / p.blocks, head0 = kvh * p.group + (rec.z - kvh * p.blocks) * static_cast<int>(p.heads.value);
  const int heads = min(static_cast<int>(p.heads.value), (kvh + 1) * p.group - head0);
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
  for (int i = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); i < 2 * kRows; i += gridDim.y * kJoinWarps) {
    const int r = i % kRows, token = p.heads.quotient(r), head = r - token * static_cast<int>(p.heads.value), index = i / kRows * p.tokens + token;
    if (token >= p.tokens || head >= heads || index >= rec.y) continue;
    const float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 * kRows + i) * (D + 4);
    float m = -INFINITY, l = 0.f, o[E] = {};
#pragma unroll 2
    for (int j = 0; j < rec.w; ++j, part += 2 * kRows * (D + 4)) {
      const float mj = part[D], lj = part[D + 1];
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = part[lane * E + e];
      const float mx = fmaxf(m, mj), base = mx == -INFINITY ? 0.f : mx, f = mkw::exp2_fast(m - base), fj = mkw::exp2_fast(mj - base);
      m = mx;
      l = l * f + lj * fj;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + x[e] * fj;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l * vs;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (rec.x + index) * p.out_row + (head0 + head) * p.out_head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(rec.x + index) * p.hq + head0 + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <bool FP8, int D>
int launch(PromptParams &p, bool joins, int ctas, int dev, cudaStream_t s) {
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &prompt_kernel<FP8, D>;
  static_assert((kMaxSequences + 1) * 4 <= 2 * Layout<64>::TILE + kSlots * Layout<64>::TILE, "find_task's sums");
  if (!ready[dev].get(reinterpret_cast<const void *>(fn), kThreads, Layout<D>::SMEM)) return MK_ERR_CUDA;
  const int rc = mkw::launch_after(fn, dim3(ctas), kThreads, Layout<D>::SMEM, s, p);
  if (rc != MK_OK || !joins) return rc;
  return mkw::launch_after(&join_kernel<D>, dim3(2 * p.sms, 2 * kRows / kJoinWarps / 4), 32 * kJoinWarps, 0, s, p);
}

int64_t workspace_bytes(int sms, int d) { return (1 + 2 * static_cast<int64_t>(sms)) * 16 + 2 * static_cast<int64_t>(sms) * 2 * kRows * (d + 4) * 4; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stride_ok(int64_t s, int elem) { return s >= 0 && s <= (int64_t{1} << 48) && s * elem % 16 == 0; }

}  // namespace mkprompt

using namespace mkprompt;

extern "C" int64_t mk_paged_prompt_attention_workspace(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return MK_ERR_UNSUPPORTED;
  const int sms = mkv::sm_count(nullptr);
  return sms < 0 ? MK_ERR_CUDA : workspace_bytes(sms, head_dim);
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
  p.blocks = (p.group + kRows - 1) / kRows;
  const int heads = (p.group + p.blocks - 1) / p.blocks;
  p.heads.set(heads);
  p.vh = p.hkv * p.blocks;
  p.tokens = kRows / heads;
  p.n_pages = kv->n_pages;
  p.capacity = static_cast<int>(slots);
  p.window = a->window;
  p.sinks = a->window > 0 ? std::min(a->sinks, p.capacity) : 0;
  p.sms = sms;
  p.scale = a->scale;
  // pairs of tiles: a sequence has one that is not full; a task more for every share of the work
  const int64_t pairs = std::min<int64_t>(a->rows, a->rows / (2 * p.tokens) + a->n), ctas = pairs * p.vh + sms;
  if (ctas > INT32_MAX) return MK_ERR_UNSUPPORTED;
  // blocks of an item: of all its row's tokens, or of the window, its own rows and the first tokens
  const int64_t span = p.window > 0 ? static_cast<int64_t>(p.window) + 2 * p.tokens + p.sinks + 3 * kBlock : slots + kBlock;
  const bool joins = std::min<int64_t>(span, slots + kBlock) / kBlock > kLeastBlocks;
  if (joins) {
    const int64_t bytes = workspace_bytes(sms, kv->head_dim);
    if (!ask && (!a->workspace || a->workspace_bytes < bytes)) return MK_ERR_INVALID_ARG;
    p.records = static_cast<int4 *>(ask ? ask(context, bytes) : a->workspace);
    if (!p.records) return MK_ERR_NO_MEMORY;
    if (!aligned16(p.records)) return MK_ERR_INVALID_ARG;
    p.parts = reinterpret_cast<float *>(p.records + 1 + 2 * sms);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (kv->dtype == MK_BF16)
    return kv->head_dim == 64 ? launch<false, 64>(p, joins, static_cast<int>(ctas), dev, s) : launch<false, 128>(p, joins, static_cast<int>(ctas), dev, s);
  return kv->head_dim == 64 ? launch<true, 64>(p, joins, static_cast<int>(ctas), dev, s) : launch<true, 128>(p, joins, static_cast<int>(ctas), dev, s);
}

}  // namespace

extern "C" int mk_paged_prompt_attention(const mk_paged_kv *kv, const mk_prompt_args *a, mk_stream stream) {
  return prompt_attention(kv, a, stream, nullptr, nullptr);
}

extern "C" int mk_paged_prompt_attention_ask(const mk_paged_kv *kv, const mk_prompt_args *a, mk_workspace_fn workspace, void *context, mk_stream stream) {
  return workspace ? prompt_attention(kv, a, stream, workspace, context) : MK_ERR_INVALID_ARG;
}
