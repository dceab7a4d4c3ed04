// Page tables and slot maps of a step of several sequences, from their lengths (mk_paged_plan).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_paged.h"
#include "mk_mma.cuh"

namespace mkplan {

// ---------------------------------------------------------------------------
// Sequence i has lengths[i] tokens in ceil(lengths[i] / page_size) pages and gets c_i more.  Exclusive sums of c_i give
// each sequence its rows, those of the pages that it lacks its part of the free list; a row finds its sequence by
// bisection of the first sums, a new page of the second.
//
// Bound by latency: a megabyte at most, behind one chain of length -> sums -> place -> store.  One launch of CTAs each of
// which forms all the sums in its own shared memory (reading n lengths again is shorter than passing sums around) and then
// writes its share of rows and pages.  Where totals are lengths or used_out is used, all reading has to end before the
// first write: then the CTAs are one cluster, which meets once.  A step of one token each of 64 sequences 2.7 us; 512
// prompts in 131072 rows 4.5 us (a cluster of 16 CTAs, two rounds of rows and more each, 7.9); 16384 sequences 13.3 (58
// with a thread's sequences next to each other, 32 to a bank).
// ---------------------------------------------------------------------------

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxSequences = 16384;
constexpr int kRowsACta = 4 * kThreads;
// of a step, which takes no more pages: a step of all threads beyond them stays within 32 bits
constexpr int kMostRows = INT32_MAX - (1 << 20);
constexpr int smem_of(int n) { return (3 * n + 2) * 4; }

struct PlanParams {
  const int32_t *lengths, *counts, *free, *used;
  int32_t *table, *seqs, *slots, *starts, *totals, *used_out, *status;
  int64_t table_stride;
  mkw::Divisor page_size;
  int n, rows, free_count, table_cols;
  int meet;                    // outputs in the place of inputs: the CTAs are one cluster
  int step;                    // no counts: a token each, row i is sequence i
  int wide;                    // seqs and slots on 16 bytes
};

__device__ __forceinline__ int pages_of(const PlanParams &p, int tokens) { return tokens > 0 ? p.page_size.quotient(tokens - 1) + 1 : 0; }

// the last i with before[i] <= x, where before[0] <= x < before[n]
__device__ __forceinline__ int place_of(const int *before, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int smem[];
  __shared__ int64_t s_rows[kWarps], s_pages[kWarps];
  mkw::follow_previous_kernel();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, n = p.n;
  int *rows_before = smem, *pages_before = smem + n + 1, *len = pages_before + n + 1;
  // a warp's consecutive sequences, 32 at a time
  const int per = (n + kThreads - 1) / kThreads * 32, first = min(n, w * per), last = min(n, first + per);
  bool bad = false;
  int64_t rows = 0, pages = 0;
  for (int i = first + lane; i < last; i += 32) {
    const int l = p.lengths[i], c = l < 0 ? 0 : p.step ? 1 : max(p.counts[i], 0);
    const int64_t total = static_cast<int64_t>(max(l, 0)) + c;
    const int have = pages_of(p, l), need = total > INT32_MAX ? have : pages_of(p, static_cast<int>(total));
    if (c > 0 && (total > INT32_MAX || need > p.table_cols)) bad = true;
    rows_before[i] = c;
    pages_before[i] = c > 0 ? need - have : 0;
    len[i] = l;
    rows += c, pages += c > 0 ? need - have : 0;
  }
  const int used = p.used[0];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    rows += __shfl_xor_sync(0xffffffffu, rows, o);
    pages += __shfl_xor_sync(0xffffffffu, pages, o);
  }
  if (lane == 0) s_rows[w] = rows, s_pages[w] = pages;
  bad = __syncthreads_or(bad);

  // exclusive sums: the warps before, 32 sequences before, the lanes before
  int64_t r64 = 0, g64 = 0;
  rows = pages = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == w) r64 = rows, g64 = pages;
    rows += s_rows[i], pages += s_pages[i];
  }
  const bool fits = !bad && rows <= p.rows && (pages == 0 || (used >= 0 && used + pages <= p.free_count));
  int r = static_cast<int>(r64), g = static_cast<int>(g64);   // within 32 bits where the step fits
  for (int i = first; i < last; i += 32) {
    const bool there = i + lane < last;
    const int c = there && fits ? rows_before[i + lane] : 0, q = there && fits ? pages_before[i + lane] : 0;
    int cs = c, qs = q;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, cs, o), b = __shfl_up_sync(0xffffffffu, qs, o);
      if (lane >= o) cs += a, qs += b;
    }
    if (there) rows_before[i + lane] = fits ? r + cs - c : 0, pages_before[i + lane] = fits ? g + qs - q : 0;
    r += __shfl_sync(0xffffffffu, cs, 31), g += __shfl_sync(0xffffffffu, qs, 31);
  }
  if (!fits) rows = pages = 0;
  if (tid == 0) rows_before[n] = static_cast<int>(rows), pages_before[n] = static_cast<int>(pages);
  if (p.meet) {
    mkw::cluster_arrive();
    mkw::cluster_wait();
  }
  __syncthreads();

  const int at = blockIdx.x * kThreads + tid, all = gridDim.x * kThreads;
  if (at == 0) {
    p.used_out[0] = used + static_cast<int>(pages);
    if (!fits && p.status) atomicCAS(p.status, 0, MK_ERR_KV_FULL);
  }
  for (int i = at; i <= n; i += all) {
    p.starts[i] = p.step ? i : rows_before[i];
    if (i < n) p.totals[i] = len[i] + rows_before[i + 1] - rows_before[i];
  }
  for (int j = at; j < static_cast<int>(pages); j += all) {
    const int i = place_of(pages_before, n, j);
    p.table[i * p.table_stride + pages_of(p, len[i]) + j - pages_before[i]] = p.free[used + j];
  }
  if (p.step) {
    for (int i = at; i < p.rows; i += all) {
      const bool there = rows_before[i + 1] > rows_before[i];
      p.seqs[i] = there ? i : -1;
      p.slots[i] = there ? len[i] : -1;
    }
    return;
  }
  const int end = static_cast<int>(rows);
  for (int q = at; q < (p.rows + 3) / 4; q += all) {
    int s[4], t[4], i = 4 * q < end ? place_of(rows_before, n, 4 * q) : n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 4 * q + e;
      while (i < n && row >= rows_before[i + 1]) ++i;
      s[e] = i < n ? i : -1;
      t[e] = i < n ? len[i] + row - rows_before[i] : -1;
    }
    if (p.wide && 4 * q + 3 < p.rows) {
      reinterpret_cast<int4 *>(p.seqs)[q] = make_int4(s[0], s[1], s[2], s[3]);
      reinterpret_cast<int4 *>(p.slots)[q] = make_int4(t[0], t[1], t[2], t[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * q + e < p.rows) p.seqs[4 * q + e] = s[e], p.slots[4 * q + e] = t[e];
    }
  }
}

}  // namespace mkplan

using namespace mkplan;

extern "C" int mk_paged_plan(const mk_plan_args *a, mk_stream stream) {
  if (!a || a->n < 0 || a->rows < 0 || a->free_count < 0 || a->table_cols < 0 || a->page_size < 1 || a->table_stride < 0) return MK_ERR_INVALID_ARG;
  if (!a->used || !a->used_out || !a->starts || (a->n > 0 && (!a->lengths || !a->totals)) || (a->rows > 0 && (!a->seqs || !a->slots)) ||
      (a->free_count > 0 && !a->free) || (a->n > 0 && a->table_cols > 0 && !a->table) || (!a->counts && a->n > 0 && a->rows != a->n))
    return MK_ERR_INVALID_ARG;
  if (a->n > kMaxSequences || a->rows > kMostRows) return MK_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= mkw::kMaxDevices) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  static mkw::Ready ready[mkw::kMaxDevices];
  mkw::Ready &r = ready[dev];
  if (!r.get(reinterpret_cast<const void *>(&plan_kernel), kThreads, smem_of(kMaxSequences))) return MK_ERR_CUDA;
  PlanParams p = {};
  p.lengths = a->lengths, p.counts = a->counts, p.free = a->free, p.used = a->used;
  p.table = a->table, p.seqs = a->seqs, p.slots = a->slots, p.starts = a->starts, p.totals = a->totals, p.used_out = a->used_out;
  p.status = a->status;
  p.table_stride = a->table_stride;
  p.page_size.set(a->page_size);
  p.n = a->n, p.rows = a->rows, p.free_count = a->free_count, p.table_cols = a->table_cols;
  p.step = !a->counts && a->n > 0;
  p.wide = ((reinterpret_cast<uintptr_t>(a->seqs) | reinterpret_cast<uintptr_t>(a->slots)) & 15u) == 0;
  // A CTA for every kRowsACta rows, a round of four rows a thread, and no more than run at once (131072 rows 4.5 us; two
  // rounds 5.3, half a round 5.0); in place one for every 4096, as far as a cluster reaches
  p.meet = a->totals == a->lengths || a->used_out == a->used;
  int ctas = p.meet ? 1 : std::max(1, std::min({(a->rows - 1) / kRowsACta + 1, mkv::sm_count(&dev), (1 << 20) / kThreads}));
  for (int i = 0; p.meet && i < 4 && r.clusters[i] > 0 && a->rows > 4096 * ctas; ++i) ctas = 2 << i;
  return mkw::launch_after(&plan_kernel, dim3(ctas), kThreads, smem_of(a->n), reinterpret_cast<cudaStream_t>(stream), p, p.meet ? ctas : 1);
}
