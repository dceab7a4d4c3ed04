// Attention of whole prompts over a paged KV cache (mk_paged_prompt_attention): kernels, one translation unit per type of cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_mma.cuh"
#include "mk_paged.h"
#include "mk_tc.cuh"

namespace mkprompt {

using namespace mktc;

// ---------------------------------------------------------------------------
// For each new token t (position p_t of its sequence) and query head: out = sum_p w_p v_p / sum_p w_p, w_p = e^(scale q k_p), over
// p <= p_t with p > p_t - window or p < sinks; lse = log sum_p w_p.
//
// A tile is 128 rows: as many tokens as fit with all the query heads of one kv head, so that a key is read once for all of
// them.  A CTA has two tiles (one, where a call is small) of consecutive tokens and walks the blocks of 128 positions that any of their rows sees: S = Q K^T by
// tcgen05 into tensor memory, a thread a row takes 64 scores out, P = 2^(S - maximum) goes back over them as 16-bit numbers,
// and O += P V takes P from there.  O stays in tensor memory and is rescaled only when a row's maximum has grown by more than
// kLag.  Four warps bring keys and values (16 bytes a copy: a page may start anywhere), two issue products, eight have the
// rows.  Items with many blocks are cut where that ends earlier, and their parts joined in order (the same bits each time).
// P is rounded to bf16, whose steps are those of the values that it multiplies; over an 8-bit cache keys, values, queries and
// P are fp16 numbers, which hold e4m3 exactly.  Maximum, sum and O are fp32.
//
// Bound by the softmax, not by the products: one prompt of 8192 tokens, 16 heads of 128 on 8, takes 195 us (1410 TFLOP/s; its
// products alone 137 at the rate of a long matrix product, and their pipe is 52 % busy), over an e4m3 cache 204 us, with
// heads of 64 193; 32768 tokens take 2.5 ms (1760 TFLOP/s), 2000 34 us.  Per 64 scores a row waits for the products, for the exponential's
// pipe and for tensor memory in turn, and tensor memory (512 columns: 2 x 128 of scores, 2 x 128 of O) has no room for a third
// place of scores.  Few rows are bound by latency: 77 tokens 7.8 us.
// ---------------------------------------------------------------------------

constexpr int kSoftWarps = 8, kMmaWarps = 2, kCopyWarps = 4, kWarps = kSoftWarps + kMmaWarps + kCopyWarps, kThreads = 32 * kWarps;
constexpr int kRows = 128;            // of a query tile (the MMA's M); a CTA has two
constexpr int kBlock = 128;           // cached positions of a key or value tile
constexpr int kHalf = 64;             // of a softmax step: a thread holds their scores in registers
constexpr int kMaxSequences = 16384, kTaskThreads = 256;
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
  int4 *header;                // .x: tasks, .y: items that are cut
  int4 *records;               // of each such item {first row, tokens, virtual head, first partial result and above its 16 bits the parts}
  struct Task *tasks;
  float *parts;                // [partial result][tile][kRows][D + 4]: O, maximum, sum
  mkw::Divisor page_size, heads;   // heads: query heads of a tile's token
  int n, rows, hq, hkv, group, n_pages, capacity, window, sinks;
  int blocks, vh;              // head blocks of a kv head, virtual heads hkv * blocks
  int tokens, item;            // of a tile: kRows / heads; of an item: one tile or two
  int sms, ctas;               // ctas: of the attention kernel, at least as many as there are tasks
  int joins;                   // whether any item can be cut
  int how;                     // how a CTA comes by its task
  float scale;
};

template <int D>
struct Layout {
  static constexpr int ATOMS = D / 64;
  static constexpr uint32_t TILE = ATOMS * 128 * 128;      // 128 rows of D 16-bit elements
  static constexpr int SLOTS = D == 128 ? 5 : 4;           // key and value tiles in shared memory, in turn
  static constexpr uint32_t CONTROL = 1024, Q = CONTROL, KV = Q + 2 * TILE;
  static constexpr int SMEM = static_cast<int>(1024 + KV + SLOTS * TILE);
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
  const int first = t * p.item;
  x.row = start + first;
  x.count = min(p.item, count - first);
  x.pos = length - count + first;
  const int hi = x.pos + x.count;
  x.lo = p.window > 0 && x.pos + 1 > p.window ? x.pos + 1 - p.window : 0;
  const int low = x.lo / kBlock;
  x.head = min((p.sinks + kBlock - 1) / kBlock, low);
  x.skip = low - x.head;
  x.blocks = hi > 0 && length <= p.capacity ? (hi + kBlock - 1) / kBlock - x.skip : 0;
  return x;
}

// A CTA's part of the work, 48 bytes: of a pair of tiles and a virtual head the blocks b0 .. b1 - 1.
struct __align__(16) Task {
  int row, count, pos, seq;    // as in Pair
  int lo, head, skip, vh;
  int b0, b1, slot, outside;   // slot: of the partial result, < 0: none, the task is whole; outside: longer than its row of the table
};
static_assert(sizeof(Task) == 48, "read as three 16-byte words");

// parts of an item: part i has blocks begin(i) .. begin(i + 1) - 1
struct Parts {
  int count, each, more;
  __device__ __forceinline__ Parts(int blocks, int limit) {
    count = blocks > limit ? (blocks - 1) / limit + 1 : 1;
    each = blocks / count;
    more = blocks - each * count;
  }
  __device__ __forceinline__ int begin(int i) const { return i * each + min(i, more); }
};

// pairs of tiles of sequence i
__device__ __forceinline__ int items_of(const PromptParams &p, int i, bool &bad) {
  const int a = p.starts[i], b = p.starts[i + 1], length = p.lengths[i];
  const bool fine = a >= 0 && b >= a && b <= p.rows;
  bad |= !fine;
  return fine && length >= 0 ? (b - a + p.item - 1) / p.item : 0;
}

// The most blocks of a task: an equal share of all of them, twice that, or no limit, whichever promises the earliest end.  In
// blocks: a task has kBegin of them to set up and store, a join takes kJoining.  Tasks that run all at once end with the
// longest; else the SMs' equal shares, and half a task for what is uneven (long ones begin first).  4 tokens behind 30000:
// cut 35 us, whole 274; 2000 tokens: whole 34, cut to shares 46.  (fp32 numbers, the same everywhere: 64-bit divisions took
// each CTA a microsecond.)
__device__ __forceinline__ int share_of(const PromptParams &p, float blocks) {
  return max(kLeastBlocks, static_cast<int>(fminf(blocks / p.sms * 1.0001f, 1e9f)) + 1);   // (no less than the share)
}
template <class Tasks>
__device__ __forceinline__ int limit_of(const PromptParams &p, float blocks, int most, float items, Tasks tasks) {
  constexpr float kBegin = 4.f, kJoining = 3.f;
  const int share = share_of(p, blocks);
  auto ends = [&](int limit, float count) {
    const int parts = (most - 1) / limit + 1;              // of the longest
    const float longest = static_cast<float>((most - 1) / parts + 1) + kBegin, all = blocks + kBegin * count;
    return (count <= p.sms ? longest : all / p.sms + all / count / 2) + (limit < most ? kJoining : 0.f);
  };
  const float one = ends(share, tasks(share)), twice = ends(2 * share, tasks(2 * share)), none = ends(INT32_MAX, items);
  return none <= one && none <= twice ? INT32_MAX : one <= twice ? share : 2 * share;
}

// The tasks of a call, in the order of sequences, their last rows (which see most) first; CTA i of the attention kernel takes
// task i.  An item (one or two tiles and a virtual head) of more blocks than `limit` is cut into parts.
// One CTA, as a call's lengths are on the device.  For few items of at most 32 sequences every CTA finds its own task instead.
static __global__ void __launch_bounds__(kTaskThreads) task_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ int before[];                          // pairs before a sequence: [n + 1]
  __shared__ long long s_warps[kTaskThreads / 32];
  __shared__ int s_tasks, s_items, s_most;
  mkw::follow_previous_kernel();
  const int tid = threadIdx.x, lane = tid & 31, n = p.n;
  bool bad = false;
  if (tid == 0) s_most = 0;
  for (int i = tid; i < n; i += kTaskThreads) before[i] = items_of(p, i, bad);
  if (bad) report(p.status, MK_ERR_BAD_PAGE);
  const int per = (n + kTaskThreads - 1) / kTaskThreads, a = min(n, tid * per), b = min(n, a + per);
  int p0 = 0, p1 = 0, i0 = 0, limit = INT32_MAX, share = INT32_MAX;
  long long at = 0;
  float blocks = 0.f;
  __syncthreads();
  // Passes: 0 the pairs before this thread's sequences; then over its share of the pairs 1 their blocks, 2 their tasks with
  // either limit, 3 its tasks (in the upper half), partial results and items that are cut, 4 the same written down.  One copy
  // of the loop and of the sum over threads: code that runs once takes as long as it is.
#pragma unroll 1
  for (int pass = 0; pass < 5; ++pass) {
    if ((pass == 1 || pass == 2) && !p.joins) continue;
    long long mine = 0;
    if (pass == 0) {
      for (int i = a; i < b; ++i) mine += before[i];
    } else {
      int i = i0, start = 0, count = 0, length = 0, of = -1;
#pragma unroll 1
      for (int x = p0; __any_sync(0xffffffffu, x < p1); ++x) {
        Pair pair{};
        Parts parts(0, 1);
        int tasks = 0;
        if (x < p1) {
          while (x >= before[i + 1]) ++i;
          if (of != i) {
            of = i;
            start = p.starts[i];
            count = p.starts[i + 1] - start;
            length = p.lengths[i];
          }
          pair = pair_of(p, start, count, length, before[i + 1] - 1 - x);
          parts = Parts(pair.blocks, limit);
          tasks = parts.count * p.vh;
        }
        // (the pass is the same for all lanes, whether they have a pair or not)
        if (pass == 1) {
          mine += pair.blocks;
          if (pair.blocks > s_most) atomicMax(&s_most, pair.blocks);
          continue;
        }
        if (pass == 2) {
          if (tasks) mine += (static_cast<long long>(Parts(pair.blocks, share).count) << 32) | Parts(pair.blocks, 2 * share).count;
          continue;
        }
        const int first = static_cast<int>((at + mine) >> 32), slots = static_cast<int>(at + mine) >> 16, items = static_cast<int>(at + mine) & 0xffff;
        mine += static_cast<long long>(tasks) << 32;
        if (parts.count > 1) mine += (tasks << 16) + p.vh;
        if (pass == 3) continue;
        if (first + tasks > p.ctas) {                      // (starts that overlap: what is past the end is not done)
          atomicMin(&s_tasks, first);
          atomicMin(&s_items, items);
          tasks = 0;
        }
        // the tasks of a lane's pair, by all of its warp
#pragma unroll 1
        for (unsigned rest = __ballot_sync(0xffffffffu, tasks > 0); rest; rest &= rest - 1u) {
          auto of_lane = [&](int v) { return __shfl_sync(0xffffffffu, v, __ffs(rest) - 1); };
          Task t{of_lane(pair.row), of_lane(pair.count), of_lane(pair.pos), of_lane(i), of_lane(pair.lo), of_lane(pair.head), of_lane(pair.skip), 0, 0, 0, 0,
                 of_lane(length > p.capacity)};
          Parts q = parts;
          q.count = of_lane(parts.count), q.each = of_lane(parts.each), q.more = of_lane(parts.more);
          const int to = of_lane(first), slot0 = of_lane(slots), item0 = of_lane(items), all = of_lane(tasks);
          for (int k = lane; k < all; k += 32) {
            t.vh = k / q.count;
            const int part = k - t.vh * q.count;
            t.b0 = q.begin(part), t.b1 = q.begin(part + 1);
            t.slot = q.count > 1 ? slot0 + k : -1;
            p.tasks[to + k] = t;
            if (q.count > 1 && part == 0) p.records[item0 + t.vh] = make_int4(t.row, t.count, t.vh, q.count << 16 | t.slot);
          }
        }
      }
      if (pass == 4) break;
    }
    long long s = mine;                                    // before this thread's, and all
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) s_warps[tid >> 5] = s;
    __syncthreads();
    long long total = 0;
    at = s - mine;
#pragma unroll 1
    for (int i = 0; i < kTaskThreads / 32; ++i) {
      if (i < tid >> 5) at += s_warps[i];
      total += s_warps[i];
    }
    if (pass == 0) {
      // Starts that overlap can promise more tasks than a number of 32 bits holds; no others pass p.ctas, which is at most half
      // of that.  (The same for all threads.)
      if (total > INT32_MAX / 2 / p.vh) {
        if (tid == 0) report(p.status, MK_ERR_BAD_PAGE);
        for (int i = a; i < b; ++i) before[i] = 0;
        at = total = 0;
      }
      int pairs = static_cast<int>(at);
      for (int i = a; i < b; ++i) {
        const int c = before[i];
        before[i] = pairs;
        pairs += c;
      }
      pairs = static_cast<int>(total);
      if (tid == 0) before[n] = pairs;
      __syncthreads();
      const int each = (pairs + kTaskThreads - 1) / kTaskThreads;
      p0 = min(pairs, tid * each), p1 = min(pairs, p0 + each);
      for (int hi = n; hi - i0 > 1;) {                     // the sequence of the first of them
        const int mid = (i0 + hi) >> 1;
        if (before[mid] <= p0) i0 = mid;
        else hi = mid;
      }
    } else if (pass == 1) {
      blocks = static_cast<float>(total * p.vh);
      share = share_of(p, blocks);
    } else if (pass == 2) {
      limit = limit_of(p, blocks, max(s_most, 1), static_cast<float>(static_cast<long long>(before[n]) * p.vh),
                       [&](int at_most) { return static_cast<float>((at_most == share ? total >> 32 : total & 0xffffffff) * p.vh); });
    } else if (tid == 0) {
      s_tasks = static_cast<int>(total >> 32), s_items = static_cast<int>(total) & 0xffff;
    }
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) *p.header = make_int4(s_tasks, s_items, 0, 0);
}

// How a CTA comes by its task: from the list; by itself, where nothing can be cut; by itself, where items may be.
enum { kListed, kWhole, kCut };

// Task `index` of a call whose sequences a warp holds, a lane each; count 0: there is none.  The same order and the same
// choice of a limit, from bounds of the blocks instead of their sums.  The thread that may `write` leaves what the join needs.
template <bool CUT>
__device__ __forceinline__ Task find_task(const PromptParams &p, int index, int lane, bool write) {
  bool bad = false;
  int start = 0, count = 0, length = 0;
  const int items = lane < p.n ? items_of(p, lane, bad) : 0;
  if (lane < p.n) start = p.starts[lane], count = p.starts[lane + 1] - start, length = p.lengths[lane];
  if (__any_sync(0xffffffffu, bad) && index == 0) report(p.status, MK_ERR_BAD_PAGE);
  int upto = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int all = __shfl_sync(0xffffffffu, upto, 31);
  int limit = INT32_MAX;
  if constexpr (CUT) {
    // an item's blocks: (its last position + 1) / 128 rounded up, a window's at most
    const bool some = items > 0 && length <= p.capacity;
    const float h0 = static_cast<float>(max(length - count + min(p.item, count), 0)), of = static_cast<float>(items);
    const int wide = p.window > 0 ? min(p.window, p.capacity) / kBlock + p.sinks / kBlock + p.item / kBlock + 6 : INT32_MAX / kBlock;
    float blocks = some ? fminf(of * (2 * h0 + (of - 1) * static_cast<float>(p.item)) * (0.5f / kBlock) + of, of * static_cast<float>(wide)) : 0.f;
    int most = some ? min((length + kBlock - 1) / kBlock, wide) : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    const float vh = static_cast<float>(p.vh);
    limit = limit_of(p, blocks * vh, max(most, 1), all * vh, [&](int at_most) { return (all + blocks / at_most) * vh; });
  }
  int i = 0, item = 0, part = 0, slot = -1, record = 0;
  Parts parts(0, 1);
  if (limit == INT32_MAX) {
    if (CUT && write && index == p.ctas) *p.header = make_int4(0, 0, 0, 0);
    item = index / p.vh;
    const unsigned behind = __ballot_sync(0xffffffffu, upto > item);
    if (!behind || index >= p.ctas) return Task{};
    i = __ffs(behind) - 1;
    index -= item * p.vh;
  } else if constexpr (CUT) {
    int to = 0, slots = 0, cut = 0, found = -1;
    bool past = false;                                     // (starts that overlap: what is past the end is not done)
#pragma unroll 1
    for (int x0 = 0; x0 < all && found < 0 && !past; x0 += 32) {
      const int x = x0 + lane;
      int of = 0;                                          // sequences whose items end before x
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (__shfl_sync(0xffffffffu, upto, of + o - 1) <= x) of += o;
      const int s0 = __shfl_sync(0xffffffffu, start, of), c0 = __shfl_sync(0xffffffffu, count, of), l0 = __shfl_sync(0xffffffffu, length, of);
      const int last = __shfl_sync(0xffffffffu, upto, of) - 1;
      const Parts mine(x < all ? pair_of(p, s0, c0, l0, last - x).blocks : 0, limit);
      const int tasks = x < all ? mine.count * p.vh : 0;
      const long long own = (static_cast<long long>(tasks) << 32) + (tasks && mine.count > 1 ? (tasks << 16) + p.vh : 0);
      long long sum = own;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const long long before = sum - own;
      const int first = to + static_cast<int>(before >> 32);
      const unsigned over = __ballot_sync(0xffffffffu, first + tasks > p.ctas), here = __ballot_sync(0xffffffffu, index >= first && index < first + tasks && first + tasks <= p.ctas);
      past = over != 0;
      const int from = here ? __ffs(here) - 1 : over ? __ffs(over) - 1 : 31;
      const long long upto_here = __shfl_sync(0xffffffffu, here || over ? before : sum, from);
      const int first_here = __shfl_sync(0xffffffffu, first, from);
      slots += static_cast<int>(upto_here & 0xffffffff) >> 16;
      cut += static_cast<int>(upto_here) & 0xffff;
      to += static_cast<int>(upto_here >> 32);
      if (here) {
        found = x0 + from;
        parts.count = __shfl_sync(0xffffffffu, mine.count, from), parts.each = __shfl_sync(0xffffffffu, mine.each, from), parts.more = __shfl_sync(0xffffffffu, mine.more, from);
        i = __shfl_sync(0xffffffffu, of, from);
        const int k = index - first_here;
        index = k / parts.count, part = k - index * parts.count;
        if (parts.count > 1) slot = slots + k;
      }
    }
    if (found < 0) {
      if (write && index == p.ctas) *p.header = make_int4(0, cut, 0, 0);
      return Task{};
    }
    item = found;
    record = cut + index;
  }
  const int t = __shfl_sync(0xffffffffu, upto, i) - 1 - item;
  start = __shfl_sync(0xffffffffu, start, i), count = __shfl_sync(0xffffffffu, count, i), length = __shfl_sync(0xffffffffu, length, i);
  const Pair pair = pair_of(p, start, count, length, t);
  if (parts.count == 1) parts.each = pair.blocks, parts.more = 0;
  else if (write && part == 0) p.records[record] = make_int4(pair.row, pair.count, index, parts.count << 16 | slot);
  return Task{pair.row, pair.count, pair.pos, i, pair.lo, pair.head, pair.skip, index, parts.begin(part), parts.begin(part + 1), slot, length > p.capacity};
}

// ---- the kernel ------------------------------------------------------------------------

// two fp32 numbers that one instruction works on
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 numbers_of(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the 8 16-bit operands of a 16-byte piece of a bf16 query row: as they are, or times a power of two as fp16
template <bool FP8>
__device__ __forceinline__ uint4 query_piece(uint4 w, float f, uint32_t flip) {
  w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = (&w.x)[i];
      const __half2 h = __floats2half2_rn(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f);
      (&w.x)[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return w;
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

// N elements of the cache, as they are and as numbers
template <bool FP8, int N>
struct Raw;
template <>
struct Raw<false, 4> {
  using type = uint2;
  static __device__ __forceinline__ uint32_t word(const type &w, int i) { return i ? w.y : w.x; }
};
template <>
struct Raw<false, 2> {
  using type = uint32_t;
  static __device__ __forceinline__ uint32_t word(type w, int) { return w; }
};
template <>
struct Raw<true, 4> {
  using type = uint32_t;
};
template <>
struct Raw<true, 2> {
  using type = uint16_t;
};
template <bool FP8, int N>
__device__ __forceinline__ void numbers_of(const typename Raw<FP8, N>::type &w, float (&x)[N]) {
  if constexpr (FP8) {
    uint32_t h[2];
    mkw::e4m3x4_to_half2(w, h[0], h[1]);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i / 2]));
      x[i] = f.x, x[i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t u = Raw<false, N>::word(w, i / 2);
      x[i] = __uint_as_float(u << 16), x[i + 1] = __uint_as_float(u & 0xffff0000u);
    }
  }
}

// A row by fp32 products, one warp, eight positions at a time: for rows whose tensor-core result is not finite.  There a
// value outside the row's mask (infinity or NaN times a weight of 0) or a sum of large values can have done it, so that
// the answer may be finite all the same.  Leaves the row's maximum (log2 units), sum and O (lane's elements) where the sum
// counts weights times `shrink`.  Each row reads keys and values for itself: 8192 tokens that all see a NaN among the values
// take 82 ms (one position at a time 216); a score that is NaN ends its row.
template <bool FP8, int D>
__device__ void row_alone(const PromptParams &p, const Task &task, const Pair &pair, int b0, int b1, int row, int head, int pos, int lane, float &m, float &l,
                          float (&o)[D / 32], float &shrink) {
  constexpr int E = D / 32, ES = FP8 ? 1 : 2;
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
  constexpr int U = 8;                                     // positions whose keys and values are on their way together
#pragma unroll 1
  for (int i = 4 * b0; i < 4 * b1; ++i) {                  // 32 positions, a lane looks up one
    const int at = pair.number(i >> 2) * kBlock + (i & 3) * 32 + lane;
    const bool want = at <= pos && (p.window == 0 || at > pos - p.window || at < p.sinks);
    const int64_t slot = want ? slot_of(p, task.seq, at) : 0;
    if (__any_sync(0xffffffffu, slot < 0)) {
      m = l = NAN;
      return;
    }
    const unsigned wanted = __ballot_sync(0xffffffffu, want);
#pragma unroll 1
    for (int j = 0; j < 32; j += U) {
      if (!(wanted >> j & ((1u << U) - 1u))) continue;
      typename Raw<FP8, E>::type k[U], v[U];
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t from = __shfl_sync(0xffffffffu, slot, j + u) + kvh * p.head_stride + lane * E;
        k[u] = v[u] = {};
        if (wanted >> (j + u) & 1) {
          k[u] = *reinterpret_cast<const typename Raw<FP8, E>::type *>(static_cast<const unsigned char *>(p.k) + from * ES);
          v[u] = *reinterpret_cast<const typename Raw<FP8, E>::type *>(static_cast<const unsigned char *>(p.v) + from * ES);
        }
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
        float x[E];
        numbers_of<FP8, E>(k[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) s[u] += q[e] * x[e];
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o2);
        s[u] = wanted >> (j + u) & 1 ? s[u] * c : -INFINITY;
        mx = fmaxf(mx, s[u]);
      }
      const float base = mx == -INFINITY ? 0.f : mx, f = mkw::exp2_fast(m - base);
      m = mx;
      l *= f;
      // an infinity stays one, however small its weight (fp32's may be 0; a score of -infinity makes it 0 in truth)
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fabsf(o[e]) < INFINITY ? o[e] * f : o[e];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = mkw::exp2_fast(s[u] - base) * shrink;
        l += w;
        float x[E];
        numbers_of<FP8, E>(v[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += fabsf(x[e]) < INFINITY ? w * x[e] : s[u] == -INFINITY ? NAN : x[e];
      }
      if (l != l) return;                                  // (a score that is no number: so is all of the row, whatever follows)
    }
  }
}

template <bool FP8, int D, int HOW>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using LY = Layout<D>;
  constexpr int kSlots = LY::SLOTS;
  // The running maximum may lag behind by kLag (log2), so that O is rarely rescaled.  Over an 8-bit cache weights are fp16
  // numbers, scaled to 2^11 and up to 2^15 with the lag (what is below 2^-25 of the largest loses bits: 2^-36 of it at most).
  constexpr float kShift = FP8 ? 11.f : 0.f, kLag = FP8 ? 4.f : 8.f;
  constexpr uint32_t kIdS = FP8 ? idesc_f32(kRows, kHalf) : idesc_bf16_f32(kRows, kHalf);
  constexpr uint32_t kIdO = (FP8 ? idesc_f32(kRows, D) : idesc_bf16_f32(kRows, D)) | kBMajorN;
  extern __shared__ unsigned char smraw[];
  mkw::let_next_kernel_start();
  unsigned char *sm = smraw + ((1024u - (smem_addr(smraw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm), *empty = full + kSlots, *sfull = empty + kSlots, *pfull = sfull + 4, *odone = pfull + 4, *ofull = odone + 4;   // [tile][half]
  uint32_t *tslot = reinterpret_cast<uint32_t *>(ofull + 1);
  unsigned char *Qs = sm + LY::Q, *KVs = sm + LY::KV;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], FP8 ? kCopyWarps / 2 : kCopyWarps), mbar_init(&empty[i], kMmaWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&sfull[i], 1), mbar_init(&pfull[i], 4), mbar_init(&odone[i], 1);
    mbar_init(ofull, kMmaWarps);
    fence_mbar_init();
  }
  __syncthreads();
  mkw::wait_for_previous_kernel();
  Task task;
  if constexpr (HOW != kListed) {
    task = find_task<HOW == kCut>(p, blockIdx.x, lane, tid == 0);
  } else {
    const int4 *words = reinterpret_cast<const int4 *>(p.tasks + blockIdx.x);
    const int4 w0 = words[0], w1 = words[1], w2 = words[2];  // (no more than what the workspace has; not a task's perhaps)
    task = Task{w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w, w2.x, w2.y, w2.z, w2.w};
    if (static_cast<int>(blockIdx.x) >= p.header->x) task.count = 0;
  }
  if (task.count == 0) return;
  const Pair x{task.row, task.count, task.pos, task.lo, task.head, task.skip, 0};
  const int b0 = task.b0, b1 = task.b1;
  const bool whole = task.slot < 0;
  const int kvh = task.vh / p.blocks, head0 = kvh * p.group + (task.vh - kvh * p.blocks) * static_cast<int>(p.heads.value);
  const int heads = min(static_cast<int>(p.heads.value), (kvh + 1) * p.group - head0);
  // the positions of a tile's first and last row, and whether any of its rows sees any of block b
  auto first_of = [&](int tile) { return x.pos + tile * p.tokens; };
  auto last_of = [&](int tile) { return x.pos + min(x.count, (tile + 1) * p.tokens) - 1; };
  auto sees = [&](int tile, int b) {
    const int from = b * kBlock;
    // (rows before the sequence's first token see nothing, and their positions less a window may pass 32 bits)
    return x.count > tile * p.tokens && from <= last_of(tile) && (p.window == 0 || from + kBlock - 1 > max(first_of(tile), 0) - p.window || from < p.sinks);
  };
  if (warp == kSoftWarps) tmem_alloc(tslot, LY::TMEM_COLS);

  // ---- softmax warps: a thread a row; its query to shared memory --------------------------
  const int tile = warp >> 2, r = (warp & 3) * 32 + lane;
  const int token = p.heads.quotient(r), head = r - token * static_cast<int>(p.heads.value), index = tile * p.tokens + token;
  const bool live = warp < kSoftWarps && token < p.tokens && head < heads && index < x.count;
  float to_log2 = p.scale * 1.4426950408889634f * (FP8 && p.k_scale ? p.k_scale[kvh] : 1.f);
  const uint32_t flip = to_log2 < 0.f ? 0x80008000u : 0u;   // a negative factor's sign goes to the query
  to_log2 = fabsf(to_log2);
  if (warp < kSoftWarps) {
    // a row's bytes together, as they are; where its numbers are to change, each thread then changes its own row's
    constexpr int PIECES = D / 8, ROWS = 32 / PIECES;
    unsigned char *mine = Qs + tile * LY::TILE;
    const uint64_t src = reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16 *>(p.q) + (live ? (x.row + index) * p.q_row + (head0 + head) * p.q_head : 0));
    const unsigned alive = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int i = 0; i < 32; i += ROWS) {
      const int rr = i + lane / PIECES, c = lane % PIECES;
      const uint64_t from = __shfl_sync(0xffffffffu, src, rr);
      mkw::cp_async16(smem_addr(mine + piece_at((warp & 3) * 32 + rr, c)), reinterpret_cast<const void *>(from + c * 16), alive >> rr & 1);
    }
    mkw::cp_async_commit();
    mkw::cp_async_wait<0>();
    __syncwarp();
    float f = 1.f;
    if constexpr (FP8) {
      // the row's largest element to [2^13, 2^14): fp16 holds what is at least 2^-38 of it
      float a = 0.f;
#pragma unroll 4
      for (int c = 0; c < PIECES; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(mine + piece_at(r, c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = (&w.x)[i];
          a = fmaxf(a, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
        }
      }
      const int e = a > 0.f && a < INFINITY ? max(-126, min(126, 13 - ilogbf(a))) : 0;
      f = ldexpf(1.f, e);
      to_log2 *= ldexpf(1.f, -e);
    }
    if (FP8 || flip) {
#pragma unroll 4
      for (int c = 0; c < PIECES; ++c) {
        uint4 *w = reinterpret_cast<uint4 *>(mine + piece_at(r, c));
        *w = query_piece<FP8>(*w, f, flip);
      }
    }
    fence_to_tensor_cores();
  }
  // (a factor of 0 would make the -infinity of a hidden score NaN; the smallest normal one does what 0 does.  NaN stays NaN.)
  if (to_log2 < 1.2e-38f) to_log2 = 1.2e-38f;
  uint32_t tmem = 0;
  if (warp < kSoftWarps + kMmaWarps) {                     // (the copies begin meanwhile)
    tc_fence_before();
    asm volatile("barrier.sync 1, %0;" ::"n"(32 * (kSoftWarps + kMmaWarps)) : "memory");
    tc_fence_after();
    tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  }

  if (warp >= kSoftWarps + kMmaWarps) {
    // ---- copies: a lane looks up a position of a block ---------------------------------------
    constexpr int ES = FP8 ? 1 : 2, PIECES = D * ES / 16, ROWS = 32 / PIECES;   // 16-byte pieces of a row, rows a copy
    const int cw = warp - kSoftWarps - kMmaWarps;
    auto look_up = [&](int b, int i) -> int64_t {          // byte offset of position i of the block; -1 not read, -2 bad
      const int pos = x.number(b) * kBlock + i;
      if (pos > last_of(1) || (pos < x.lo && pos >= p.sinks)) return -1;
      const int64_t at = slot_of(p, task.seq, pos);
      return at < 0 ? -2 : (at + kvh * p.head_stride) * ES;
    };
    // a key that is not there is NaN: so are the scores of rows that see it
    auto no_key = [&](unsigned char *to, int row) {
      report(p.status, MK_ERR_BAD_PAGE);
      for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4 *>(to + piece_at(row, c)) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    };
    bool ok = true;
    if constexpr (!FP8) {
      // 32 positions a warp, keys and values in turn, one tile on its way while the one before is told of
      int n_tiles = 0, told = 0;                           // tiles asked for, tiles told of
      auto tell = [&](int upto) {
        fence_to_tensor_cores();
        __syncwarp();
        for (; told < upto; ++told)
          if (lane == 0) mbar_arrive(&full[told % kSlots]);
      };
      const int64_t slot_bytes = p.slot_stride * ES, row_step = ROWS * slot_bytes, lane_off = lane / PIECES * slot_bytes + lane % PIECES * 16;
      int64_t next = b0 < b1 ? look_up(b0, cw * 32 + lane) : -1;
      for (int b = b0; b < b1 && ok; ++b) {
        const int64_t at = next;
        const bool bad = at == -2;
        // Whether 16 positions each lie one behind the other, as in a page of as many slots: then a copy's address is the one
        // before and a step (one prompt of 8192 tokens 195 us; each address from its position's own offset 207).  (An 8-bit
        // cache, whose rows are half as long, gains nothing by it.)
        const int64_t leading = __shfl_sync(0xffffffffu, at, lane & 16);
        const bool runs = __all_sync(0xffffffffu, at >= 0 && at == leading + (lane & 15) * slot_bytes);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++n_tiles) {
          const int slot = n_tiles % kSlots;
          if (n_tiles >= kSlots) {
            const uint32_t parity = (n_tiles / kSlots - 1) & 1;
            if (!__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], parity))) {
              mkw::cp_async_wait<0>();
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
          const uint32_t to_at = smem_addr(to);
          if (runs) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const unsigned char *from = base + __shfl_sync(0xffffffffu, at, 16 * half) + lane_off;
#pragma unroll
              for (int i = 0; i < 16 / ROWS; ++i, from += row_step)
                mkw::cp_async16(to_at + piece_at(cw * 32 + 16 * half + i * ROWS + lane / PIECES, lane % PIECES), from);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32 / ROWS; ++i) {
              const int rr = i * ROWS + lane / PIECES, c = lane % PIECES;
              const int64_t o = __shfl_sync(0xffffffffu, at, rr);
              mkw::cp_async16(to_at + piece_at(cw * 32 + rr, c), base + (o < 0 ? 0 : o + c * 16), o >= 0);
            }
          }
          mkw::cp_async_commit();
          if (kv == 0) {
            if (__any_sync(0xffffffffu, bad)) {
              mkw::cp_async_wait<0>();
              __syncwarp();
              if (bad) no_key(to, cw * 32 + lane);
            }
            if (b + 1 < b1) next = look_up(b + 1, cw * 32 + lane);
          }
          if (n_tiles >= 1) {
            mkw::cp_async_wait<1>();
            tell(n_tiles);
          }
        }
      }
      mkw::cp_async_wait<0>();
      if (ok) tell(n_tiles);
    } else {
      // Through registers, to fp16.  Two warps have the keys and two the values, 64 positions each: what tells of a tile (the
      // fence) waits for a warp's loads too, so that these are hidden by the other warps only.
      constexpr int COPIES = 64 / ROWS;
      const int kv = cw >> 1, row0 = (cw & 1) * 64;
      const unsigned char *base = static_cast<const unsigned char *>(kv ? p.v : p.k);
      int64_t next[2] = {-1, -1};
      if (b0 < b1) next[0] = look_up(b0, row0 + lane), next[1] = look_up(b0, row0 + 32 + lane);
      for (int b = b0; b < b1; ++b) {
        const int64_t at[2] = {next[0], next[1]};
        uint4 w[COPIES];
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int rr = i * ROWS + lane / PIECES;
          const int64_t o = __shfl_sync(0xffffffffu, at[i * ROWS / 32], rr & 31);
          w[i] = o < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(base + o + lane % PIECES * 16);
        }
        if (b + 1 < b1) next[0] = look_up(b + 1, row0 + lane), next[1] = look_up(b + 1, row0 + 32 + lane);
        const int n_tile = 2 * (b - b0) + kv, slot = n_tile % kSlots;
        if (n_tile >= kSlots && !__all_sync(0xffffffffu, mbar_wait(&empty[slot], (n_tile / kSlots - 1) & 1, kWaitNs))) {
          if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
          break;
        }
        unsigned char *to = KVs + slot * LY::TILE;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int rr = row0 + i * ROWS + lane / PIECES, c = lane % PIECES;
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) mkw::e4m3x4_to_half2((&w[i].x)[e], h[2 * e], h[2 * e + 1]);
          *reinterpret_cast<uint4 *>(to + piece_at(rr, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(to + piece_at(rr, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        if (kv == 0) {
          __syncwarp();
          if (at[0] == -2) no_key(to, row0 + lane);
          if (at[1] == -2) no_key(to, row0 + 32 + lane);
        }
        fence_to_tensor_cores();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
      }
    }
  } else if (warp >= kSoftWarps) {
    // ---- products: S = Q K^T for half a block of a tile, then O += P V with P where S was, so that the next S there comes
    // behind it.  A tile has two such places: one is in its softmax while the other is multiplied.
    if (b0 < b1) {
      // descriptors: the low words move with the tile, the high ones are constants
      const uint64_t kd = desc_sw128(smem_addr(KVs)), vd = desc_mn_sw128_at(smem_addr(KVs), kBlock * 128, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(desc_sw128(smem_addr(Qs))), k_lo = static_cast<uint32_t>(kd), v_lo = static_cast<uint32_t>(vd);
      const uint32_t k_hi = static_cast<uint32_t>(kd >> 32), v_hi = static_cast<uint32_t>(vd >> 32);
      const int t = warp - kSoftWarps;
      bool ok = true, begun = false;                       // begun: O has been written
      uint32_t phase = 0;
      int slot = 0;                                        // of the next key or value tile, and the parity of its round
      uint32_t round = 0;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && !__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs))) {
          if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
          ok = false;
        }
        return ok;
      };
      auto next = [&]() {
        if (++slot == kSlots) slot = 0, round ^= 1u;
      };
      auto scores = [&](int h, int k_slot) {
        const uint32_t k_at = k_lo + ((k_slot * LY::TILE + h * (kHalf * 128)) >> 4), q_at = q_lo + t * (LY::TILE >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = ((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4;
          mma_bf16(tmem + t * LY::S_COLS + h * kHalf, desc_of(q_at + off, k_hi), desc_of(k_at + off, k_hi), kIdS, s != 0);
        }
        mma_commit(&sfull[2 * t + h]);
      };
      bool seen = sees(t, x.number(b0));
      if (wait(&full[0], 0)) {
        tc_fence_after();
        if (elect_one()) {
          if (seen) scores(0, 0), scores(1, 0);
          mma_commit(&empty[0]);
        }
        __syncwarp();
        next();
      }
      for (int b = b0; b < b1 && ok; ++b) {
        const bool more = b + 1 < b1, then = more && sees(t, x.number(b + 1));
        const int v_slot = slot;
        if (!wait(&full[v_slot], round)) break;
        next();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (seen && !wait(&pfull[2 * t + h], phase)) break;
          if (more && h == 0 && !wait(&full[slot], round)) break;
          tc_fence_after();
          if (elect_one()) {
            if (seen) {
              const uint32_t v_at = v_lo + ((v_slot * LY::TILE + h * (kHalf * 128)) >> 4);
#pragma unroll
              for (int s = 0; s < kHalf / 16; ++s)
                mma_f16_ta(tmem + LY::O_COL + t * D, tmem + t * LY::S_COLS + h * kHalf + s * 8, desc_of(v_at + s * (2048 >> 4), v_hi), kIdO, begun || s != 0);
              mma_commit(&odone[2 * t + h]);
            }
            if (h == 1) mma_commit(&empty[v_slot]);
            if (then) scores(h, slot);
            if (more && h == 1) mma_commit(&empty[slot]);
          }
          __syncwarp();
          begun |= seen;
        }
        if (seen) phase ^= 1u;
        if (more) next();
        seen = then;
      }
      if (elect_one()) mma_commit(ofull);                  // all of it is done (also where a wait ran out)
      __syncwarp();
      mbar_wait(ofull, 0, kWaitNs);
    }
  } else {
    // ---- softmax ---------------------------------------------------------------------------
    const int pos = first_of(tile) + token;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + tile * LY::S_COLS, o_at = tmem + lanes + LY::O_COL + tile * D;
    const int hidden_below = p.window > 0 ? max(pos, 0) - p.window : -1;   // hidden: at <= hidden_below and not a first token
    float m = -INFINITY, l = 0.f;                          // m: of scores before to_log2
    uint32_t phase = 0;                                    // parity of the blocks that the tile has seen
    bool started = false, ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && !__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs))) {
        if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
        ok = false;
      }
      tc_fence_after();
      return ok;
    };
    for (int b = b0; b < b1 && ok; ++b) {
      const int blk = x.number(b);
      if (!sees(tile, blk)) continue;
#pragma unroll 1
      for (int h = 0; h < 2 && ok; ++h) {
        if (!wait(&sfull[2 * tile + h], phase)) break;
        uint32_t u[2][32];
        tmem_ld32(s_at + h * kHalf, u[0]);
        tmem_ld32(s_at + h * kHalf + 32, u[1]);
        const int from = blk * kBlock + h * kHalf;
        const bool edge = __any_sync(0xffffffffu, from + kHalf - 1 > pos || (from <= hidden_below && from + kHalf > p.sinks));
        tmem_ld_wait(u[0]);
        tmem_ld_wait(u[1]);
        if (edge) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            const int at = from + i;
            if (at > pos || (at <= hidden_below && at >= p.sinks)) u[i / 32][i % 32] = 0xff800000u;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kHalf; i += 2) top[i / 2 & 3] = max3(top[i / 2 & 3], __uint_as_float(u[i / 32][i % 32]), __uint_as_float(u[i / 32][i % 32 + 1]));
        const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
        const bool grows = (mx - m) * to_log2 > kLag;      // (also from -infinity; not if both are)
        if (__any_sync(0xffffffffu, grows)) {
          const float alpha = grows ? mkw::exp2_fast((m - mx) * to_log2) : 1.f;
          if (grows) m = mx;
          l *= alpha;
          if (started) {
            if (!wait(&odone[2 * tile + 1 - h], h ? phase : phase ^ 1u)) break;   // (the product of the half before may be on its way)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_at + c, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_at + c, o);
            }
          }
        }
        started = true;
        // P = 2^(S to_log2 + base).  (Some of the exponentials as polynomials on the multipliers, as these have time left in
        // their own pipe: 12 to 50 % of them took 5 to 28 % longer, for the instructions.)
        const float base = m == -INFINITY ? 0.f : fmaf(-m, to_log2, kShift);
        const Two factor = two(to_log2, to_log2), shift = two(base, base);
        Two sum = two(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 f = numbers_of(fma2(two(__uint_as_float(u[c][2 * i]), __uint_as_float(u[c][2 * i + 1])), factor, shift));
            f.x = mkw::exp2_fast(f.x), f.y = mkw::exp2_fast(f.y);
            sum = add2(sum, two(f.x, f.y));
            w[i] = pack_weights<FP8>(f.x, f.y);
          }
          tmem_st16(s_at + h * kHalf + c * 16, w);         // (where the scores were)
        }
        const float2 both = numbers_of(sum);
        l += both.x + both.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * tile + h]);
      }
      phase ^= 1;
    }
    // ---- results ------------------------------------------------------------------------------
    if (b0 < b1 && !__all_sync(0xffffffffu, mbar_wait(ofull, 0, kWaitNs))) {
      if (lane == 0) report(p.status, MK_ERR_TIMEOUT);
      ok = false;
    }
    tc_fence_after();
    const float vs = FP8 && p.v_scale ? p.v_scale[kvh] : 1.f;
    if (task.outside && lane == 0) report(p.status, MK_ERR_BAD_PAGE);
    float *part = whole ? nullptr : p.parts + ((static_cast<int64_t>(task.slot) * 2 + tile) * kRows + r) * (D + 4);
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (x.row + index) * p.out_row + (head0 + head) * p.out_head;
    const float inv = task.outside || !ok ? NAN : !whole ? 1.f : l == 0.f ? 0.f : __frcp_rn(l) * vs;
    // whether the row is to be worked on alone: a sum or an element of O that is not finite
    bool strange = !(fabsf(l) < INFINITY);
    // to where the warp's queries were, and from there a row's bytes together: rounded results, or half of fp32 ones at a time
    constexpr int PIECES = D / 8, ROWS = 32 / PIECES;
    const unsigned alive = __ballot_sync(0xffffffffu, live);
    unsigned char *mine = Qs + tile * LY::TILE;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t u[32];
      if (started && ok) {
        tmem_ld32(o_at + c, u);
        tmem_ld_wait(u);
      }
      float y[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        y[i] = (started && ok && l != 0.f ? __uint_as_float(u[i]) : 0.f) * inv;
        strange |= !(fabsf(y[i]) < INFINITY);
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4 *>(mine + piece_at(r, c / 8 + i)) =
              make_uint4(pack_weights<false>(y[8 * i], y[8 * i + 1]), pack_weights<false>(y[8 * i + 2], y[8 * i + 3]),
                         pack_weights<false>(y[8 * i + 4], y[8 * i + 5]), pack_weights<false>(y[8 * i + 6], y[8 * i + 7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4 *>(mine + piece_at(r, c % (D / 2) / 4 + i)) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      }
      const bool full_rows = whole ? c + 32 == D : (c + 32) % (D / 2) == 0;
      if (full_rows) {
        __syncwarp();
        // (an output may be its query, which row_alone reads again)
        const unsigned put = alive & ~__ballot_sync(0xffffffffu, strange && whole && ok && !task.outside);
        const uint64_t to = whole ? reinterpret_cast<uint64_t>(dst) : reinterpret_cast<uint64_t>(part + (c + 32 - D / 2));
#pragma unroll 4
        for (int i = 0; i < 32; i += ROWS) {
          const int rr = i + lane / PIECES, piece = lane % PIECES;
          const uint64_t row_at = __shfl_sync(0xffffffffu, to, rr);
          const uint4 w = *reinterpret_cast<const uint4 *>(mine + piece_at((warp & 3) * 32 + rr, piece));
          if (put >> rr & 1) *reinterpret_cast<uint4 *>(row_at + piece * 16) = w;
        }
        __syncwarp();
      }
    }
    m = m == -INFINITY ? m : m * to_log2 - kShift;         // log2 units, as the sum is scaled
    if (task.outside || !ok) m = l = NAN;
    if (live) {
      if (!whole) part[D] = m, part[D + 1] = l;
      else if (p.lse) p.lse[static_cast<int64_t>(x.row + index) * p.hq + head0 + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
    __syncwarp();                                          // (what was put by a row's own lane, the warp puts again)
    for (unsigned rest = __ballot_sync(0xffffffffu, strange && live && ok && !task.outside); rest; rest &= rest - 1u) {
      const int of = __ffs(rest) - 1;
      const int row = x.row + __shfl_sync(0xffffffffu, index, of), hd = head0 + __shfl_sync(0xffffffffu, head, of);
      float rm, rl, o[D / 32], shrink;
      row_alone<FP8, D>(p, task, x, b0, b1, row, hd, __shfl_sync(0xffffffffu, pos, of), lane, rm, rl, o, shrink);
      // (the sum is of weights times shrink: as many log2 units less for the maximum)
      const float grow = 1.f / shrink;
      if (whole) {
        const float f = rl == 0.f ? 0.f : rl != rl ? NAN : __frcp_rn(rl);
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) + row * p.out_row + hd * p.out_head + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) to[i] = __float2bfloat16_rn(o[i] * f * vs);
        if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(row) * p.hq + hd] = rl == 0.f ? -INFINITY : (rm + log2f(rl * grow)) * 0.69314718055994531f;
      } else {
        float *to = p.parts + ((static_cast<int64_t>(task.slot) * 2 + tile) * kRows + (warp & 3) * 32 + of) * (D + 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) to[lane * (D / 32) + i] = o[i];
        if (lane == 0) to[D] = rm + log2f(grow), to[D + 1] = rl;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps) tmem_dealloc(tmem, LY::TMEM_COLS);
}

// Joins the parts of items, in order, a row a warp, in units of 16 rows that the CTAs (two an SM: one that finds nothing costs
// a microsecond in all) take in turn.  Up to 32 parts' maxima and sums are read at once, a lane each.
constexpr int kJoinWarps = 16, kUnits = 2 * kRows / kJoinWarps;
__device__ __forceinline__ void load_part(const float *p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_part(const float *p, float (&x)[2]) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  x[0] = v.x, x[1] = v.y;
}
// (an infinity stays one, however small its weight: fp32's may be 0)
__device__ __forceinline__ float weighted(float x, float w) { return fabsf(x) < INFINITY ? x * w : x; }
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PromptParams p) {
  constexpr int E = D / 32;
  mkw::follow_previous_kernel();
  const int lane = threadIdx.x & 31, units = p.header->y * kUnits;
#pragma unroll 1
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int4 rec = p.records[unit / kUnits];
    const int parts = rec.w >> 16, slot = rec.w & 0xffff, i = unit % kUnits * kJoinWarps + (threadIdx.x >> 5);
    const int kvh = rec.z / p.blocks, head0 = kvh * p.group + (rec.z - kvh * p.blocks) * static_cast<int>(p.heads.value);
    const int heads = min(static_cast<int>(p.heads.value), (kvh + 1) * p.group - head0);
    const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
    const int r = i % kRows, token = p.heads.quotient(r), head = r - token * static_cast<int>(p.heads.value), index = i / kRows * p.tokens + token;
    if (token >= p.tokens || head >= heads || index >= rec.y) continue;
    constexpr int64_t kPart = 2 * kRows * (D + 4);
    const float *part = p.parts + static_cast<int64_t>(slot) * kPart + i * (D + 4);
    // The parts' sums are finite, what they add up to may not be before it is divided: weights are scaled down by the number
    // of parts, rounded up to a power of two.
    const int spare = 32 - __clz(parts - 1);
    const float shrink = __int_as_float((127 - spare) << 23), grow = __int_as_float((127 + spare) << 23);
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int j0 = 0; j0 < parts; j0 += 32) {
      const bool mine = j0 + lane < parts;
      const float mj = mine ? part[(j0 + lane) * kPart + D] : -INFINITY, lj = mine ? part[(j0 + lane) * kPart + D + 1] : 0.f;
      float top = fmaxf(m, mj);
#pragma unroll
      for (int o2 = 16; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
      const float base = top == -INFINITY ? 0.f : top, f = mkw::exp2_fast(m - base), fj = mkw::exp2_fast(mj - base) * shrink;
      m = top;
      l = l * f + lj * fj;                                 // (a lane's own; added up at the end)
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = weighted(o[e], f);
      const int count = min(32, parts - j0);
#pragma unroll 1
      for (int j = 0; j < count; j += 8) {                 // eight parts' elements on their way together
        float x[8][E];
#pragma unroll
        for (int k = 0; k < 8; ++k) load_part(part + (j0 + min(j + k, count - 1)) * kPart + lane * E, x[k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w = __shfl_sync(0xffffffffu, fj, j + k & 31);   // (0 for a lane without a part)
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += j + k < count ? weighted(x[k][e], w) : 0.f;
        }
      }
    }
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
    const float inv = l == 0.f ? 0.f : 1.f / l * vs;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (rec.x + index) * p.out_row + (head0 + head) * p.out_head + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = pack_weights<false>(o[e] * inv, o[e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(rec.x + index) * p.hq + head0 + head] = l == 0.f ? -INFINITY : (m + log2f(l * grow)) * 0.69314718055994531f;
  }
}

template <bool FP8, int D, int HOW>
int launch_kernel(PromptParams &p, int dev, cudaStream_t s) {
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &prompt_kernel<FP8, D, HOW>;
  if (!ready[dev].get(reinterpret_cast<const void *>(fn), kThreads, Layout<D>::SMEM)) return MK_ERR_CUDA;
  // (where items may be cut and there is no list, a CTA more tells the join how much there is)
  const int rc = mkw::launch_after(fn, dim3(p.ctas + (HOW == kCut ? 1 : 0)), kThreads, Layout<D>::SMEM, s, p);
  if (rc != MK_OK || !p.joins) return rc;
  return mkw::launch_after(&join_kernel<D>, dim3(2 * p.sms), 32 * kJoinWarps, 0, s, p);
}

template <bool FP8, int D>
int launch(PromptParams &p, int dev, cudaStream_t s) {
  if (p.how == kWhole) return launch_kernel<FP8, D, kWhole>(p, dev, s);
  if (p.how == kCut) return launch_kernel<FP8, D, kCut>(p, dev, s);
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto tasks = &task_kernel;
  if (!ready[dev].get(reinterpret_cast<const void *>(tasks), kTaskThreads, (kMaxSequences + 1) * 4)) return MK_ERR_CUDA;
  const int rc = mkw::launch_after(tasks, dim3(1), kTaskThreads, (p.n + 1) * 4, s, p);
  return rc != MK_OK ? rc : launch_kernel<FP8, D, kListed>(p, dev, s);
}

}  // namespace mkprompt
