// Operators over a paged KV cache that several sequences share (mk_paged_append,
// mk_paged_attention, and the copy behind mk_export_kv).
#include "mk_paged.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "mk_launch_after.h"
#include "mk_mma.cuh"

namespace mkv {

__device__ __forceinline__ void report(int32_t *status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// ---------------------------------------------------------------------------
// Append: q, k and v heads of n tokens, normalised, rotated and stored.
//
// Bound by bytes: every element is read once and written once; the arithmetic
// is a sum of squares and one rotation, on two fp32 numbers an instruction.
// D / 2 / N threads hold a head, each N consecutive elements of the first half
// and the N elements half a head further, the pairs of the rotation, so that
// every load and store is 16 bytes of an input row and a pair meets in one
// thread; the squares are summed over the head's threads by shuffles.  A token
// that would need a page outside the cache or a rotary row outside the table is
// not written.
// Two kernels: for few tokens a thread for every part of every head (in graphs, one
// token 2.7 us, 256 of 32 heads 3.5), for many persistent warps that copy ahead (20011
// tokens of 32 heads of 128, bf16 to e4m3, 291 MB: 50 us, 5.8 TB/s).  They meet
// where the threads of the first are no longer resident at once (about 450
// tokens: 384 take 3.7 and 4.4 us, 512 4.7 both ways); the first kernel with 4
// heads a thread took 62 us for the 20011, its threads waiting for slot, page and
// elements one after the other.
// ---------------------------------------------------------------------------

struct AppendParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  int64_t page_stride, head_stride, slot_stride, table_stride;
  const int32_t *table, *seqs, *slots, *positions;
  const float2 *rope;
  const uint16_t *q_norm, *k_norm;
  const float *k_scale, *v_scale;
  int32_t *status;
  mkw::Divisor page_size;
  int n, hq, hkv, n_pages, table_rows, table_cols, rope_rows, rope_mode, sec0, sec1, sec2;
  int seq0, slot0;             // slots == NULL: row i is slot slot0 + i of sequence seq0
  mkw::Divisor groups;         // few tokens: heads of a CTA
  int rows;                    // and its token rows
  mkw::Divisor parts;          // many: warps of a token
  int streams;                 // tokens at once
  int q_groups, kv_groups;     // groups of heads (a thread's) of q, of k and of v
  float eps;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

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
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 16 bytes of a row: N values, as they are in memory and as pairs of numbers
template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void numbers(const uint4 &w, Two *x) {
    x[0] = two(__uint_as_float(w.x), __uint_as_float(w.y)), x[1] = two(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ uint4 bits(const Two *x) {
    const float2 a = numbers_of(x[0]), b = numbers_of(x[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
__device__ __forceinline__ uint32_t pack_bf16(Two x) {
  const float2 f = numbers_of(x);
  return pack_bf16(f.x, f.y);
}
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void numbers(const uint4 &w, Two *x) {
    x[0] = two(bf16_lo(w.x), bf16_hi(w.x)), x[1] = two(bf16_lo(w.y), bf16_hi(w.y));
    x[2] = two(bf16_lo(w.z), bf16_hi(w.z)), x[3] = two(bf16_lo(w.w), bf16_hi(w.w));
  }
  static __device__ __forceinline__ uint4 bits(const Two *x) {
    return make_uint4(pack_bf16(x[0]), pack_bf16(x[1]), pack_bf16(x[2]), pack_bf16(x[3]));
  }
};

// N values to the cache: bf16, or e4m3
template <int N>
__device__ __forceinline__ void store_cache(__nv_bfloat16 *p, const Two *x) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4 *>(p) = Vec<__nv_bfloat16>::bits(x);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x[0]), pack_bf16(x[1]));
}
template <int N>
__device__ __forceinline__ void store_cache(__nv_fp8_e4m3 *p, const Two *x) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(numbers_of(x[2 * i]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(numbers_of(x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i] = a | (b << 16);
  }
  if constexpr (N == 8)
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(p) = w[0];
}

constexpr int kAppendThreads = 128, kAppendCtas = 6;

template <int N>
__device__ __forceinline__ void load_gains(const uint16_t *p, Two *x) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) x[i] = two(1.f, 1.f);
  } else if constexpr (N == 8) {
    Vec<__nv_bfloat16>::numbers(*reinterpret_cast<const uint4 *>(p), x);
  } else {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    x[0] = two(bf16_lo(w.x), bf16_hi(w.x)), x[1] = two(bf16_lo(w.y), bf16_hi(w.y));
  }
}

// a token's slot, sequence and rows of the rotary table
struct Token {
  int slot, seq, at[3];
};
__device__ __forceinline__ Token token_of(const AppendParams &p, int row) {
  Token t;
  t.slot = p.slots ? p.slots[row] : p.slot0 + row;
  t.seq = p.seqs ? p.seqs[row] : p.slots ? row : p.seq0;
  t.at[0] = t.at[1] = t.at[2] = t.slot;
  if (p.positions) {
    t.at[0] = t.at[1] = t.at[2] = p.positions[row];
    if (p.rope_mode) {
      t.at[1] = p.positions[static_cast<int64_t>(p.n) + row];
      t.at[2] = p.positions[2 * static_cast<int64_t>(p.n) + row];
    }
  }
  return t;
}
// its element offset in the cache (of head 0), < 0 for a token that is not stored: refused for every head alike, so that
// it is stored whole or not at all
__device__ __forceinline__ int64_t place_of(const AppendParams &p, const Token &t) {
  if (t.slot < 0) return -1;
  const int col = p.page_size.quotient(t.slot);
  int page = -1;
  if (t.seq >= 0 && t.seq < p.table_rows && col < p.table_cols) page = p.table[t.seq * p.table_stride + col];
  if (p.rope && (t.at[0] < 0 || t.at[0] >= p.rope_rows || t.at[1] < 0 || t.at[1] >= p.rope_rows || t.at[2] < 0 || t.at[2] >= p.rope_rows)) {
    report(p.status, MK_ERR_BAD_POSITION);
    return -1;
  }
  if (page < 0 || page >= p.n_pages) {
    report(p.status, MK_ERR_BAD_PAGE);
    return -1;
  }
  return page * p.page_stride + (t.slot - col * static_cast<int>(p.page_size.value)) * p.slot_stride;
}
// the position stream that rotates pair j
__device__ __forceinline__ int stream_of(const AppendParams &p, int j) {
  const int m = j % 3;
  return p.rope_mode == 1 ? (j >= p.sec0) + (j >= p.sec0 + p.sec1) : (m == 1 && j < 3 * p.sec1) ? 1 : (m == 2 && j < 3 * p.sec2) ? 2 : 0;
}

// a thread's head or heads: i of q, of k or of v; byte addresses of its part of the first one, without the row's
struct AppendHeads {
  bool is_q, is_v;
  int i, count;                // the first head, and how many there are of its kind
  const unsigned char *src;
  unsigned char *out;
  int64_t src_row, src_head, out_row, out_head;
  const uint16_t *gain;
  const float *scales;
};
template <class T, class C>
__device__ __forceinline__ AppendHeads append_heads(const AppendParams &p, int i, int q, int kv, int i0) {
  AppendHeads h;
  h.is_q = i < q;
  h.is_v = i >= q + kv;
  h.i = i - (h.is_q ? 0 : h.is_v ? q + kv : q);
  h.count = h.is_q ? p.hq : p.hkv;
  h.src_row = (h.is_q ? p.q_row : h.is_v ? p.v_row : p.k_row) * static_cast<int64_t>(sizeof(T));
  h.src_head = (h.is_q ? p.q_head : h.is_v ? p.v_head : p.k_head) * static_cast<int64_t>(sizeof(T));
  h.src = static_cast<const unsigned char *>(h.is_q ? p.q : h.is_v ? p.v : p.k) + h.i * h.src_head + i0 * sizeof(T);
  h.out_row = h.is_q ? p.out_row * static_cast<int64_t>(sizeof(T)) : 0;
  h.out_head = h.is_q ? p.out_head * static_cast<int64_t>(sizeof(T)) : p.head_stride * static_cast<int64_t>(sizeof(C));
  h.out = static_cast<unsigned char *>(h.is_q ? p.q_out : h.is_v ? p.v_cache : p.k_cache) + h.i * h.out_head + i0 * (h.is_q ? sizeof(T) : sizeof(C));
  h.gain = h.is_q ? p.q_norm : h.is_v ? nullptr : p.k_norm;
  h.scales = h.is_q ? nullptr : h.is_v ? p.v_scale : p.k_scale;
  return h;
}

// Gains, and times cos and sin: with them a pair of elements x, y becomes r (x xa + y ya), r (y yb + x xb).
template <int N>
struct Turn {
  Two xa[N / 2], ya[N / 2], xb[N / 2], yb[N / 2];
  __device__ __forceinline__ void set(int i, Two ga, Two gb, float4 f) {   // cos and sin of pairs 2 i and 2 i + 1
    const Two c = two(f.x, f.z);
    xa[i] = mul2(ga, c);
    ya[i] = mul2(gb, two(-f.y, -f.w));
    xb[i] = mul2(ga, two(f.y, f.w));
    yb[i] = mul2(gb, c);
  }
};

// 1 / rms of a head, by all its threads
template <int D, int N>
__device__ __forceinline__ float norm_factor(const Two *x, const Two *y, float eps) {
  Two sq = two(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) sq = fma2(y[i], y[i], fma2(x[i], x[i], sq));
  const float2 f = numbers_of(sq);
  float ss = f.x + f.y;
#pragma unroll
  for (int o = D / 4 / N; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(ss * (1.0f / D) + eps);
}

template <class T, class C, int D>
__device__ __forceinline__ void store_head(const AppendHeads &h, unsigned char *out, Two *x, Two *y, float r, const Turn<Vec<T>::N> &t, bool rotated) {
  constexpr int N = Vec<T>::N;
  const Two r2 = two(r, r);
  if (rotated) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const Two a = fma2(y[i], t.ya[i], mul2(x[i], t.xa[i])), b = fma2(x[i], t.xb[i], mul2(y[i], t.yb[i]));
      x[i] = mul2(a, r2), y[i] = mul2(b, r2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) x[i] = mul2(mul2(x[i], t.xa[i]), r2), y[i] = mul2(mul2(y[i], t.yb[i]), r2);
  }
  if (h.is_q) {
    *reinterpret_cast<uint4 *>(out) = Vec<T>::bits(x);
    *reinterpret_cast<uint4 *>(out + D / 2 * sizeof(T)) = Vec<T>::bits(y);
  } else {
    store_cache<N>(reinterpret_cast<C *>(out), x);
    store_cache<N>(reinterpret_cast<C *>(out) + D / 2, y);
  }
}

// Few tokens: one head a thread.
template <class T, class C, int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = Vec<T>::N, TPH = D / 2 / N;           // threads of one head
  mkw::follow_previous_kernel();
  const int item = threadIdx.x / TPH, i0 = (threadIdx.x % TPH) * N, heads = p.hq + 2 * p.hkv;
  const int row_in = p.groups.quotient(item);
  const int head = blockIdx.y * static_cast<int>(p.groups.value) + item - row_in * static_cast<int>(p.groups.value);
  const int64_t row64 = static_cast<int64_t>(blockIdx.x) * p.rows + row_in;
  // every thread of a warp stays to the shuffles below; one with nothing to do works on zeros
  const bool live = row_in < p.rows && row64 < p.n && head < heads;
  const int64_t row = live ? row64 : 0;
  Token token;
  if (live) token = token_of(p, static_cast<int>(row));
  const AppendHeads h = append_heads<T, C>(p, live ? head : 0, p.hq, p.hkv, i0);
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (live) {
    lo = __ldcs(reinterpret_cast<const uint4 *>(h.src + row * h.src_row));
    hi = __ldcs(reinterpret_cast<const uint4 *>(h.src + row * h.src_row + D / 2 * sizeof(T)));
  }
  Two ga[N / 2], gb[N / 2];
  load_gains<N>(h.gain ? h.gain + i0 : nullptr, ga);
  load_gains<N>(h.gain ? h.gain + i0 + D / 2 : nullptr, gb);
  const int64_t dst = live ? place_of(p, token) : -1;
  const bool rotated = p.rope && !h.is_v;
  float4 cs[N / 2] = {};
  if (rotated && dst >= 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (p.rope_mode == 0) {
        cs[i] = *reinterpret_cast<const float4 *>(p.rope + static_cast<int64_t>(token.at[0]) * (D / 2) + i0 + 2 * i);
      } else {
        const float2 a = p.rope[static_cast<int64_t>(token.at[stream_of(p, i0 + 2 * i)]) * (D / 2) + i0 + 2 * i];
        const float2 b = p.rope[static_cast<int64_t>(token.at[stream_of(p, i0 + 2 * i + 1)]) * (D / 2) + i0 + 2 * i + 1];
        cs[i] = make_float4(a.x, a.y, b.x, b.y);
      }
    }
  }
  Two x[N / 2], y[N / 2];
  Vec<T>::numbers(lo, x);
  Vec<T>::numbers(hi, y);
  float r = 1.f;
  if (p.q_norm || p.k_norm) {                              // (the same for the whole grid)
    const float f = norm_factor<D, N>(x, y, p.eps);
    if (h.gain) r = f;
  }
  if (dst < 0) return;
  // e4m3 holds value / scale, here times the scale's reciprocal: a last place of fp32 away
  if (h.scales) r *= __frcp_rn(h.scales[h.i]);
  Turn<N> t;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (rotated) t.set(i, ga[i], gb[i], cs[i]);
    else t.xa[i] = ga[i], t.yb[i] = gb[i];
  }
  store_head<T, C, D>(h, h.out + row * h.out_row + (h.is_q ? 0 : dst * static_cast<int64_t>(sizeof(C))), x, y, r, t, rotated);
}

// Many tokens: a warp has 32 / TPH groups of up to 4 heads, the same ones of every `streams`th token, so that what
// depends on the heads stays in registers; a token's elements, cos and sin are on their way to shared memory while
// those of the one before are worked on.  A thread copies the elements it needs itself; cos and sin are the warp's (read
// by each head's threads they were a third of the reads: 58 us).  12 warps an SM: 16 had 54 us, 8 56.
constexpr int kStreamWarps = 12, kStreamHeads = 4;
constexpr int kStreamPieces = 2 * kStreamHeads + 1;       // 16 bytes each, of a thread, a token
// where the 16 bytes i (of N / 2) of cos and sin of a head's tth thread are, so that 8 threads meet 8 different banks
template <int N>
__device__ __forceinline__ int turn_at(int t, int i) {
  constexpr int CH = N / 2;
  return (CH * t + (i ^ (t / (8 / CH) % CH))) * 16;
}
template <class T, class C, int D>
__global__ void __launch_bounds__(32 * kStreamWarps, 1) append_many_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = Vec<T>::N, TPH = D / 2 / N, STAGE = kStreamPieces * 512;
  extern __shared__ __align__(128) unsigned char smem[];
  mkw::follow_previous_kernel();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i0 = lane % TPH * N;
  const int warp = blockIdx.x * kStreamWarps + w, first = p.parts.quotient(warp), part = warp - first * static_cast<int>(p.parts.value);
  if (first >= p.streams || first >= p.n) return;
  int group = part * (32 / TPH) + lane / TPH;
  const int groups = p.q_groups + 2 * p.kv_groups;
  const bool live = group < groups;
  AppendHeads h = append_heads<T, C>(p, live ? group : 0, p.q_groups, p.kv_groups, i0);
  if (!live) h.count = 0;
  const int step = h.is_q ? p.q_groups : p.kv_groups;     // heads i, i + step, ...
  const bool rotated = p.rope && !h.is_v;
  Two ga[N / 2], gb[N / 2];
  load_gains<N>(h.gain ? h.gain + i0 : nullptr, ga);
  load_gains<N>(h.gain ? h.gain + i0 + D / 2 : nullptr, gb);

  float inv[kStreamHeads];                                 // (e4m3 holds value / scale, here times the scale's reciprocal)
#pragma unroll
  for (int j = 0; j < kStreamHeads; ++j) inv[j] = h.scales && h.i + j * step < h.count ? __frcp_rn(h.scales[h.i + j * step]) : 1.f;

  const int count = (p.n - 1 - first) / p.streams + 1;
  unsigned char *ring = smem + w * 2 * STAGE + lane * 16;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const bool turned = __any_sync(0xffffffffu, rotated && h.count);
  const uint32_t turn = ring_at - lane * 16 + 2 * kStreamHeads * 512 + turn_at<N>(lane / (N / 2), lane % (N / 2));   // this lane copies
  Token batch;                                             // token 32 b + lane of the warp's
  int64_t batch_dst = -1;
  int64_t next_dst = -1;
  auto produce = [&](int k) {
    const int64_t row = first + static_cast<int64_t>(k) * p.streams;
    if ((k & 31) == 0) {
      batch_dst = -1;
      if (k + lane < count) {
        batch = token_of(p, static_cast<int>(row + static_cast<int64_t>(lane) * p.streams));
        batch_dst = place_of(p, batch);
      }
    }
    next_dst = __shfl_sync(0xffffffffu, batch_dst, k & 31);
    int at[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) at[j] = __shfl_sync(0xffffffffu, batch.at[j], k & 31);
    if (next_dst < 0) return;
    const uint32_t stage = ring_at + (k & 1) * STAGE;
    const unsigned char *src = h.src + row * h.src_row;
#pragma unroll
    for (int j = 0; j < kStreamHeads; ++j) {
      if (h.i + j * step < h.count) {
        mkw::cp_async16(stage + 2 * j * 512, src);
        mkw::cp_async16(stage + (2 * j + 1) * 512, src + D / 2 * sizeof(T));
      }
      src += step * h.src_head;
    }
    if (!turned || lane >= D / 4) return;
    const uint32_t to = turn + (k & 1) * STAGE;
    const int j = 2 * lane;                                // pairs j and j + 1
    if (p.rope_mode == 0) {
      mkw::cp_async16(to, p.rope + static_cast<int64_t>(at[0]) * (D / 2) + j);
    } else {
      const int s0 = stream_of(p, j), s1 = stream_of(p, j + 1);
      mkw::cp_async8(to, p.rope + static_cast<int64_t>(s0 == 0 ? at[0] : s0 == 1 ? at[1] : at[2]) * (D / 2) + j);
      mkw::cp_async8(to + 8, p.rope + static_cast<int64_t>(s1 == 0 ? at[0] : s1 == 1 ? at[1] : at[2]) * (D / 2) + j + 1);
    }
  };
  produce(0);
  mkw::cp_async_commit();
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int64_t dst = next_dst;
    __syncwarp();                                          // all have read what the next token's cos and sin replace
    if (k + 1 < count) produce(k + 1);
    mkw::cp_async_commit();
    mkw::cp_async_wait<1>();
    __syncwarp();
    if (dst < 0) continue;
    const unsigned char *stage = ring + (k & 1) * STAGE;
    Turn<N> t;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (rotated) t.set(i, ga[i], gb[i], *reinterpret_cast<const float4 *>(stage - lane * 16 + 2 * kStreamHeads * 512 + turn_at<N>(lane % TPH, i)));
      else t.xa[i] = ga[i], t.yb[i] = gb[i];
    }
    unsigned char *out = h.out + (h.is_q ? (first + static_cast<int64_t>(k) * p.streams) * h.out_row : dst * static_cast<int64_t>(sizeof(C)));
#pragma unroll
    for (int j = 0; j < kStreamHeads; ++j) {
      Two x[N / 2], y[N / 2];
      Vec<T>::numbers(*reinterpret_cast<const uint4 *>(stage + 2 * j * 512), x);
      Vec<T>::numbers(*reinterpret_cast<const uint4 *>(stage + (2 * j + 1) * 512), y);
      float r = inv[j];
      if (p.q_norm || p.k_norm) {
        const float f = norm_factor<D, N>(x, y, p.eps);   // (of whatever the memory holds where there is no head)
        if (h.gain) r *= f;
      }
      if (h.i + j * step < h.count) {
        store_head<T, C, D>(h, out, x, y, r, t, rotated);
      }
      out += step * h.out_head;
    }
  }
}

template <class T, class C, int D>
int launch_append(AppendParams p, cudaStream_t s) {
  if (p.hq > (1 << 20) || p.hkv > (1 << 20)) return MK_ERR_UNSUPPORTED;
  constexpr int TPH = D / 2 / Vec<T>::N, items = kAppendThreads / TPH;
  int dev = 0;
  const int sms = sm_count(&dev), heads = p.hq + 2 * p.hkv;
  if (sms < 0) return MK_ERR_CUDA;
  p.q_groups = (p.hq + kStreamHeads - 1) / kStreamHeads;
  p.kv_groups = (p.hkv + kStreamHeads - 1) / kStreamHeads;
  const int parts = (p.q_groups + 2 * p.kv_groups + 32 / TPH - 1) / (32 / TPH);   // warps of a token
  if (static_cast<int64_t>(p.n) * heads * TPH > static_cast<int64_t>(sms) * kAppendCtas * kAppendThreads && parts <= sms * kStreamWarps) {
    static mkw::Ready ready[mkw::kMaxDevices];
    constexpr int smem = kStreamWarps * 2 * kStreamPieces * 512;
    const auto fn = &append_many_kernel<T, C, D>;
    if (!ready[dev].get(reinterpret_cast<const void *>(fn), 32 * kStreamWarps, smem)) return MK_ERR_CUDA;
    p.parts.set(parts);
    p.streams = sms * kStreamWarps / parts;
    return mkw::launch_after(fn, dim3(sms), 32 * kStreamWarps, smem, s, p);
  }
  const int groups = std::min(heads, items);
  p.groups.set(groups);
  p.rows = items / groups;
  const int ctas = (p.n - 1) / p.rows + 1, per_row = (heads + groups - 1) / groups;
  if (per_row > 65535) return MK_ERR_UNSUPPORTED;
  return mkw::launch_after(&append_kernel<T, C, D>, dim3(ctas, per_row), kAppendThreads, 0, s, p);
}

int run_append(const AppendParams &p, int dtype, int cache, int d, cudaStream_t s) {
  using B = __nv_bfloat16;
  using E = __nv_fp8_e4m3;
  if (dtype == MK_F32) {
    if (cache == MK_BF16) return d == 64 ? launch_append<float, B, 64>(p, s) : launch_append<float, B, 128>(p, s);
    return d == 64 ? launch_append<float, E, 64>(p, s) : launch_append<float, E, 128>(p, s);
  }
  if (cache == MK_BF16) return d == 64 ? launch_append<B, B, 64>(p, s) : launch_append<B, B, 128>(p, s);
  return d == 64 ? launch_append<B, E, 64>(p, s) : launch_append<B, E, 128>(p, s);
}

// ---------------------------------------------------------------------------
// Attention of one token per row.
//
// Per row and kv head the scores s_p = scale q.k_p and the weighted sum of the
// values are taken in one pass over the cache with a running maximum m and sum
// l (kept in log2 units): o = sum 2^(s_p - m) v_p, rescaled when m grows.  Bound
// by the cache's bytes.
//
// The cache is read once for all query heads of a kv head (up to 16 a pass): the
// keys of 16 slots are the rows of a 16x8x16 matrix product and 8 query heads its
// columns, and the values, transposed on the way out of shared memory, the rows
// of a second one whose columns are the heads' probabilities.  Heads as columns
// waste nothing on a group of up to 8 (twice the columns for 16), half of what
// heads as rows would multiply.
// bf16 keys and values multiply bf16 terms: a bf16 query is one term, an fp32
// query three, and the probabilities two terms (three for fp32 outputs), which
// keeps the result as exact as fp32 products would.  e4m3 keys and values become
// fp16, exactly; the query row is scaled by a power of two into fp16's range (one
// term, two for fp32; what that rounds, 2^-38 of the row's largest element at
// most, is far below what the keys' own rounding does to that element's product)
// and the probabilities by 2^14, one term for bf16 results, whose rounding of 2^-9
// hides its 2^-12 (16 rows of 32768: 1.679e-3 of the definition's norm away, 1.677e-3
// with a second term, which takes 1 to 5 % longer), two for fp32 results.
// Over a bf16 cache they are multiplied by a power of two of at most 1 / the tokens
// a row may have: values near bf16's largest would else overflow in the sum that the
// weights' sum has yet to divide.  Each tile's value sums start from zero and are
// added to the running ones by an fp32 multiply-add: matrix products truncate what
// they add to an accumulator, which over thousands of tiles would show.
//
// Work: a warp has a range of tiles (POS slots of one row and kv head), streams
// it through its own ring of shared memory with asynchronous 16-byte copies and
// never waits for another warp until the end.  The ranges depend on the lengths,
// which only the device knows, in one of three ways that the host chooses:
//   - one row: a cluster of CTAs for each kv head, joined through their shared
//     memory.
//   - short rows (by the table's width): the tiles of all rows, in order, cut
//     into ranges of equal cost for the CTAs, moved to where a row and head
//     begins, and these for their warps; joined in shared memory.
//   - else the same with the CTAs' ranges as they fall: what a CTA has of a row
//     at its range's ends goes through the workspace to join_kernel.
// Parts are joined in order: the same lengths give the same bits.
// Measured (graph replays; where a call is shorter than its launch a loop of plain calls takes longer, 8 to 9 us for one
// row of 257 tokens): 16 query heads on 8 of 128, 64 rows of 0 to 8192 tokens in bf16 (306 MB) 53 us, 5.7 TB/s; 16 rows of
// 30 to 32 k in e4m3 (1034 MB) 158 us, 6.5 TB/s; one row of 257 tokens 6.8 us, of 5119 12.6 (fp32 queries); 256 rows of up
// to 300 tokens, 8 heads on 2 of 64, 9.6 us.
// ---------------------------------------------------------------------------

constexpr int kWarps = 8, kAttnThreads = 32 * kWarps;
constexpr int kMinUnitsPerCta = 16;
// What the start and end of a row and head cost (its queries' loads, its results' stores), in tiles: more the more query
// heads there are.  64 rows of up to 8192 tokens took 86 us with 2 for 128 query heads on 8, 66 with 8 (and 58.9 and 56.8 for 64
// on 8, with 2 and 4); 256 short rows of 4 heads on 1 take 9.6 with 2, 10.3 with 3.
constexpr int row_cost(int heads) { return heads / 2 > 2 ? heads / 2 : 2; }
constexpr int kMaxRowCost = row_cost(16);
// rows of up to so many tiles are not cut over CTAs
constexpr int kShortTiles = 64;
// Tiles of a warp's ring: one being read, one on its way, 64 KB an SM.  A third only crowds the memory (a warp's copies
// wait longer and the last warps end later): 64 rows of up to 8192 tokens took 55.5 us with it, 53.4 without; 16 rows of
// 32768 in e4m3 168 and 158.
constexpr int kStages = 2;
constexpr int kMaxSmem = 212992;       // dynamic, of 16 query heads and their inbox; the static part is below 2 KB

enum { kByCluster, kWhole, kJoined };  // how rows are dealt out: the three ways above

struct AttnParams {
  const void *q, *k, *v;
  void *out;
  float *lse;
  int64_t q_row, q_head, out_row, out_head, page_stride, head_stride, slot_stride, table_stride;
  const int32_t *table, *lengths;
  const float *k_scale, *v_scale;
  int32_t *status;
  int4 *records;       // [grid] {row, virtual head, last CTA, 1} of a row that goes on in the next CTA
  float *parts;        // [grid][2][gr][D + 4]: a row's middle or end (0) and its beginning (1)
  mkw::Divisor page_size;
  int n, hq, hkv, group, n_pages, capacity, window;   // capacity: slots of a table row
  mkw::Divisor chunks;       // of 16 query heads
  mkw::Divisor blocks, vh;   // head blocks of 16 query heads a kv head, virtual heads hkv * blocks
  int gr;              // query heads of a block: min(group, 16)
  int row_cost;
  int way, cluster;
  int dense;           // a page's slots of a head lie one behind the other
  float scale;
  float shrink, grow;  // what a probability is multiplied by on the way into the sums, and its inverse: powers of two
};

template <int D, bool FP8>
struct Tile {
  static constexpr int ES = FP8 ? 1 : 2, ROWB = D * ES, CPR = ROWB / 16;
  static constexpr int POS = (D == 128 && !FP8) ? 16 : 32;
  static constexpr int KBYTES = POS * ROWB, STAGE = 2 * KBYTES;
  // 16-byte chunk c of row r is in place c ^ turn(r), so that the same chunk of 8 rows meets 8 different banks
  static __host__ __device__ constexpr int turn(int r) { return ROWB >= 128 ? r & 7 : (r >> 1) & 3; }
  static __device__ __forceinline__ int at(int r, int c) { return r * ROWB + ((c ^ turn(r)) << 4); }
  // copies of a tile: lane l fills place l % CPR of row i ROWS + l / CPR, i < COPIES; turn() of these rows, apart from
  // the lane's part, takes TURNS values
  static constexpr int ROWS = 32 / CPR, COPIES = POS / ROWS, TURNS = ROWB == 256 ? 4 : ROWB == 128 ? 2 : 1;
};

// two elements as they are in memory, and their values
template <class T>
struct Pair;
template <>
struct Pair<float> {
  using type = float2;
  static __device__ __forceinline__ type load(const float *p) { return *reinterpret_cast<const float2 *>(p); }
  static __device__ __forceinline__ type none() { return make_float2(0.f, 0.f); }
  static __device__ __forceinline__ float2 values(type x) { return x; }
};
template <>
struct Pair<__nv_bfloat16> {
  using type = uint32_t;
  static __device__ __forceinline__ type load(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint32_t *>(p); }
  static __device__ __forceinline__ type none() { return 0u; }
  static __device__ __forceinline__ float2 values(type w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
};

// tiles of a row: those that hold any of its slots [lo, hi), and their cost, the row's start included
struct Span {
  int lo, hi, first, count, cost;
};
template <int POS>
__device__ __forceinline__ Span span_of(const AttnParams &p, int len) {
  Span s;
  s.hi = len > 0 && len <= p.capacity ? len : 0;
  s.lo = p.window > 0 && s.hi > p.window ? s.hi - p.window : 0;
  s.first = s.lo / POS;
  s.count = s.hi > 0 ? (s.hi + POS - 1) / POS - s.first : 0;
  s.cost = s.count ? s.count + p.row_cost : 0;
  return s;
}

// `total` in equal shares, as equal as whole numbers are: where the ith begins, and which one has unit u
struct Shares {
  int each, more;   // units of a share, and how many of the first have one more
  __device__ __forceinline__ Shares(int total, int parts) : each(total / parts), more(total - each * parts) {}
  __device__ __forceinline__ int begin(int i) const { return i * each + min(i, more); }
  __device__ __forceinline__ int of(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// what the ring's reader needs to know of a tile
struct TileInfo {
  int pos, lo, hi, flags, row, vh;
};
// the row's first tile, its last, a page outside the cache, the last tile of the warp
constexpr int kFirst = 1, kLast = 2, kBad = 4, kEnd = 8;

struct PartInfo {
  int row, vh, begins, ends;   // row < 0: no part
};

template <int D>
constexpr int kPartStride = D + 4;      // o[D], m, l

// the join of parts (m_j, l_j, o_j): m = max m_j, weights 2^(m_j - m)
__device__ __forceinline__ float join_base(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ void write_lse(const AttnParams &p, int row, int head, float m, float l) {
  if (p.lse) p.lse[static_cast<int64_t>(row) * p.hq + head] = l == 0.f ? -INFINITY : (m + log2f(l * p.grow)) * 0.69314718055994531f;
}

// a virtual head's kv head, first query head and number of query heads
struct Heads {
  int kvh, first, count;
};
__device__ __forceinline__ Heads heads_of(const AttnParams &p, int vh) {
  Heads h;
  h.kvh = p.blocks.quotient(vh);
  const int blk = vh - h.kvh * static_cast<int>(p.blocks.value);
  h.first = h.kvh * p.group + blk * 16;
  h.count = min(16, p.group - blk * 16);
  return h;
}

// a lane's part of a row of D fp32 elements, on a boundary of its size
__device__ __forceinline__ void load_part(const float *p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_part(const float *p, float (&x)[2]) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  x[0] = v.x, x[1] = v.y;
}

// Join parts of a query head in shared memory, in order, by a warp: lane l gets elements l D / 32 ..; lane j of `there`
// knows the byte `mine_at` where its part's o[D], m, l are.  (Small on purpose: code that runs once a launch takes as
// long as it is.)
template <int D>
__device__ __forceinline__ void join_shared(int lane, unsigned there, const unsigned char *smem, int mine_at, float &m, float &l, float (&x)[D / 32]) {
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) x[k] = 0.f;
#pragma unroll 1
  for (; there; there &= there - 1u) {
    const float *part = reinterpret_cast<const float *>(smem + __shfl_sync(0xffffffffu, mine_at, __ffs(there) - 1));
    float xj[D / 32];
    load_part(part + lane * (D / 32), xj);
    const float mj = part[D], lj = part[D + 1], mx = fmaxf(m, mj), base = join_base(mx);
    const float f = mkw::exp2_fast(m - base), fj = mkw::exp2_fast(mj - base);
    m = mx;
    l = l * f + lj * fj;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) x[k] = x[k] * f + xj[k] * fj;
  }
}

// The same in global memory: lane l gets elements l D / 32 ..; lane j of `there` knows where its
// part's o[D], m, l are, in bytes from `base`.
template <int D>
__device__ __forceinline__ void join_parts(int lane, unsigned there, const void *base, int mine_at, float &m, float &l, float (&x)[D / 32]) {
  auto at = [&](int bytes) { return reinterpret_cast<const float *>(static_cast<const unsigned char *>(base) + bytes); };
  const bool mine = there >> lane & 1;
  const float mj = mine ? at(mine_at)[D] : -INFINITY, lj = mine ? at(mine_at)[D + 1] : 0.f;
  m = mj;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float f = mkw::exp2_fast(mj - join_base(m));
  l = mine ? f * lj : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) x[k] = 0.f;
#pragma unroll 8
  for (unsigned rest = there; rest; rest &= rest - 1u) {
    const int j = __ffs(rest) - 1;
    const float fj = __shfl_sync(0xffffffffu, f, j);
    const float *part = at(__shfl_sync(0xffffffffu, mine_at, j)) + lane * (D / 32);
    float xj[D / 32];
    load_part(part, xj);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) x[k] += fj * xj[k];
  }
}

__device__ __forceinline__ void store_row(float *p, const float (&x)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store_row(float *p, const float (&x)[2]) { *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]); }
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&x)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&x)[2]) { *reinterpret_cast<uint32_t *>(p) = pack_bf16(x[0], x[1]); }

// a joined query head: o / l and the log-sum-exp
template <class T, int D>
__device__ __forceinline__ void write_head(const AttnParams &p, int lane, int row, int head, float m, float l, float (&x)[D / 32], float vs) {
  const float r = (l == 0.f ? 0.f : __frcp_rn(l)) * vs;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) x[k] *= r;
  store_row(static_cast<T *>(p.out) + row * p.out_row + head * p.out_head + lane * (D / 32), x);
  if (lane == 0) write_lse(p, row, head, m, l);
}

// over the 8 rows of a column of a product: lanes with the same t
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// HB: blocks of 8 query heads
template <class T, bool FP8, int D, int HB>
__global__ void __launch_bounds__(kAttnThreads, 1) attend_kernel(const __grid_constant__ AttnParams p) {
  using TL = Tile<D, FP8>;
  using Op = std::conditional_t<FP8, mkw::FP16Op, mkw::BF16Op>;
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int TQ = F32 ? (FP8 ? 2 : 3) : 1, TP = F32 ? (FP8 ? 2 : 3) : (FP8 ? 1 : 2);
  constexpr int POS = TL::POS, KS = D / 16, DB = D / 16, PN = POS / 16, PST = kPartStride<D>;
  constexpr float kShift = FP8 ? 14.f : 0.f;             // probabilities are scaled by 2^kShift
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TileInfo s_tile[kWarps][kStages];
  __shared__ PartInfo s_part[2 * kWarps];
  __shared__ int s_scan[kAttnThreads], s_warp[kWarps], s_range[2];

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;
  mkw::follow_previous_kernel();
  if (tid < 2 * kWarps) s_part[tid].row = -1;

  // ---- the warp's range: where it starts, and how much it covers -------------------
  int row = 0, vh = 0, tile = 0, left = 0;                   // left: units from the tile the producer stands at to the range's end
  Span sp{0, 0, 0, 0, 0};
  int per = 0, units = 0, ctas = 0;
  if (p.way == kByCluster) {
    mkw::cluster_arrive();                                   // (to be waited for before the others' memory is written)
    vh = cta / p.cluster;                                    // the cluster's kv head (and head block)
    sp = span_of<POS>(p, p.lengths[0]);
    const int i = cta % p.cluster * kWarps + w;
    const Shares shares(sp.count, p.cluster * kWarps);
    tile = shares.begin(i);
    left = shares.begin(i + 1) - tile;
    __syncthreads();
  } else {
    // Units: a row and head of cost c covers c of them, tile j the (row_cost + j)th.  A warp has the tiles whose unit
    // is in its range.  First the cost of the rows before every group of rows.
    per = (p.n + kAttnThreads - 1) / kAttnThreads;           // rows a thread counts
    int mine = 0;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < p.n) mine += span_of<POS>(p, p.lengths[r]).cost;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[w] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < w) before += s_warp[i];
      total += s_warp[i];
    }
    s_scan[tid] = before + incl - mine;                      // cost of the rows before this thread's
    __syncthreads();
    units = total * static_cast<int>(p.vh.value);
    ctas = max(1, min(static_cast<int>(gridDim.x), (units - 1) / kMinUnitsPerCta + 1));

    // The row and head that has a unit, and where in it that is: for where the CTA's range begins and ends, if these are
    // moved to where a row and head begins, then for the warp's beginning.
    int c_begin = 0, c_end = 0, begin = 0;
    if (cta < ctas) {
      const Shares shares(units, ctas);
      c_begin = shares.begin(cta);
      c_end = shares.begin(cta + 1);
    }
#pragma unroll 1
    for (int step = p.way == kWhole ? 0 : 1; step < 2; ++step) {
      int u = w == 0 ? c_begin : c_end;                      // step 0: by the first two warps
      if (step == 0) {
        if (w < 2 && lane == 0) s_range[w] = u;
      } else {
        if (p.way == kWhole) {
          __syncthreads();
          c_begin = s_range[0], c_end = s_range[1];
        }
        const int range = c_end - c_begin;
        u = begin = c_begin + range * w / kWarps;
        left = c_begin + range * (w + 1) / kWarps - begin;
        if (left <= 0) break;
      }
      if (u >= units || (step == 0 && w >= 2)) continue;
      const int x = p.vh.quotient(u);                        // in [before(row), before(row) + cost(row))
      // the last of the 256 sums that is not above x: of every eighth, then of eight
      int a = __popc(__ballot_sync(0xffffffffu, s_scan[8 * lane] <= x)) * 8 - 8;
      a += __popc(__ballot_sync(0xffffffffu, lane < 8 && s_scan[a + (lane & 7)] <= x)) - 1;
      int at = s_scan[a];
      row = a * per;
      sp = span_of<POS>(p, p.lengths[row]);
#pragma unroll 1
      while (at + sp.cost <= x) {
        at += sp.cost;
        sp = span_of<POS>(p, p.lengths[++row]);
      }
      const int rest = u - at * static_cast<int>(p.vh.value), cost = sp.cost;
      vh = rest / cost;
      const int in = rest - vh * cost;
      if (step == 0) {
        if (in > 0 && lane == 0) s_range[w] = u + cost - in;
      } else {
        tile = in - p.row_cost;
        if (tile < 0) left += tile, tile = 0;                // from the row's start on: its cost comes first
      }
    }
  }

  const uint32_t smem_at = static_cast<uint32_t>(__cvta_generic_to_shared(smem)), ring = smem_at + w * kStages * TL::STAGE;
  const unsigned char *k_base = static_cast<const unsigned char *>(p.k);
  const int64_t to_v = static_cast<const unsigned char *>(p.v) - k_base;

  // the producer's place besides row, vh, tile: its kv head and block, this lane's slot in its page and that page
  int kvh = p.blocks.quotient(vh), blk = vh - kvh * static_cast<int>(p.blocks.value), slot = 0, page = -1;
  auto look_up = [&]() {
    const int pos = (sp.first + tile) * POS + lane, col = p.page_size.quotient(pos);
    slot = pos - col * static_cast<int>(p.page_size.value);
    page = -1;
    if (lane < POS && pos >= sp.lo && pos < sp.hi) page = p.table[row * p.table_stride + col];
  };
  if (left > 0) look_up();
  int in_stage = 0;                                          // the producer's stage
  const int r0 = lane / TL::CPR, place = lane % TL::CPR;     // this lane's first slot of a tile and its place in every row
  auto produce = [&]() {
    const int pos0 = (sp.first + tile) * POS, pos = pos0 + lane;
    const bool want = lane < POS && pos >= sp.lo && pos < sp.hi;
    const bool fine = static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
    const unsigned have = __ballot_sync(0xffffffffu, want && fine);
    const bool bad = __any_sync(0xffffffffu, want && !fine);
    int64_t off = 0;
    if (want && fine) off = (page * p.page_stride + kvh * p.head_stride + slot * p.slot_stride) * TL::ES;
    const uint32_t ks = ring + in_stage * TL::STAGE + r0 * TL::ROWB + place * 16;
    if (p.dense && have == (POS == 32 ? 0xffffffffu : 0xffffu) &&
        __shfl_sync(0xffffffffu, slot, 0) + POS <= static_cast<int>(p.page_size.value)) {
      // a whole tile inside a page: its bytes follow one another
      const unsigned char *from = k_base + __shfl_sync(0xffffffffu, off, 0) + r0 * TL::ROWB;
#pragma unroll
      for (int v = 0; v < TL::TURNS; ++v) {
        const unsigned char *ka = from + ((place ^ TL::turn(r0) ^ TL::turn(v * TL::ROWS)) << 4), *va = ka + to_v;
#pragma unroll
        for (int i = v; i < TL::COPIES; i += TL::TURNS) {
          mkw::cp_async16(ks + i * TL::ROWS * TL::ROWB, ka + i * TL::ROWS * TL::ROWB);
          mkw::cp_async16(ks + TL::KBYTES + i * TL::ROWS * TL::ROWB, va + i * TL::ROWS * TL::ROWB);
        }
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < TL::COPIES; ++i) {
        const int r = i * TL::ROWS + r0;
        const int64_t o = __shfl_sync(0xffffffffu, off, r) + ((place ^ TL::turn(r)) << 4);
        const bool ok = (have >> r) & 1;
        const unsigned char *ka = k_base + (ok ? o : 0);
        mkw::cp_async16(ks + i * TL::ROWS * TL::ROWB, ka, ok);
        mkw::cp_async16(ks + TL::KBYTES + i * TL::ROWS * TL::ROWB, ka + to_v, ok);
      }
    }
    TileInfo ti{pos0, sp.lo, sp.hi, (tile == 0 ? kFirst : 0) | (bad ? kBad : 0), row, vh};
    --left;
    if (++tile == sp.count) {
      ti.flags |= kLast;
      left -= p.row_cost;
      tile = 0;
      ++vh;
      if (++blk == static_cast<int>(p.blocks.value)) blk = 0, ++kvh;
      if (vh == static_cast<int>(p.vh.value)) {
        vh = kvh = 0;
        if (left > 0) {
          do sp = span_of<POS>(p, p.lengths[++row]);
          while (sp.count == 0);
        }
      }
    }
    if (left > 0) look_up();
    else ti.flags |= kEnd;
    if (lane == 0) {
      s_tile[w][in_stage] = ti;
      if (bad) report(p.status, MK_ERR_BAD_PAGE);
    }
    in_stage ^= 1;
  };
  // ---- a row's query heads as they are in memory: asked for before the tiles, else their answer waits behind those ----
  // columns: heads 8 hb + g in the query's fragments, 8 hb + 2t and 2t + 1 in scores, states and outputs
  typename Pair<T>::type raw[KS][HB][2];
  auto load_query = [&](int q_row, int q_vh) {
    const Heads h = heads_of(p, q_vh);
    const T *q = static_cast<const T *>(p.q) + q_row * p.q_row + (h.first + g) * p.q_head;
#pragma unroll
    for (int hb = 0; hb < HB; ++hb)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // bf16: k = 2t, 2t+1, 2t+8, 2t+9 of the step; e4m3: 4t .. 4t+3, as the key's 16-bit pairs hold them
        const int d0 = 16 * s + (FP8 ? 4 * t : 2 * t), d1 = d0 + (FP8 ? 2 : 8);
        const bool there = 8 * hb + g < h.count;
        raw[s][hb][0] = there ? Pair<T>::load(q + 8 * hb * p.q_head + d0) : Pair<T>::none();
        raw[s][hb][1] = there ? Pair<T>::load(q + 8 * hb * p.q_head + d1) : Pair<T>::none();
      }
  };
  // (16 heads of 128 fp32 elements have no registers to wait in)
  constexpr bool EARLY = !(F32 && HB == 2 && D == 128);
  const bool any = left > 0;
  if (EARLY && any) load_query(row, vh);

  // ---- rows without tiles, 16 query heads a warp --------------------------------
#pragma unroll 1
  for (int i = cta * kWarps + w; i < p.n * static_cast<int>(p.chunks.value); i += gridDim.x * kWarps) {
    const int r = p.chunks.quotient(i), h0 = 16 * (i - r * static_cast<int>(p.chunks.value)), len = p.lengths[r];
    if (len < 0 || span_of<POS>(p, len).count > 0) continue;
    const float l = len == 0 ? 0.f : NAN;
    if (len > 0 && lane == 0) report(p.status, MK_ERR_BAD_PAGE);
#pragma unroll 1
    for (int h = h0; h < min(p.hq, h0 + 16); ++h) {
      float x[D / 32] = {};
      write_head<T, D>(p, lane, r, h, 0.f, l, x, 1.f);
    }
  }

  // ---- the warp's tiles ---------------------------------------------------------
  uint32_t qf[TQ][KS][HB][2];
  float o[DB][HB][4], m[HB][2], l[HB][2], mult[HB][2];
  int rows = 0, head0 = 0, begins = 0;
  int stage = 0, ahead = 1 - kStages;                        // the first round only produces
  bool start = true;
#pragma unroll 1
  for (bool more = any; more; ++ahead) {
    if (left > 0) produce();
    mkw::cp_async_commit();
    if (ahead < 0) continue;
    mkw::cp_async_wait<kStages - 1>();
    __syncwarp();
    const TileInfo ti = s_tile[w][stage];
    const uint32_t kt = ring + stage * TL::STAGE, vt = kt + TL::KBYTES;
    stage ^= 1;
    more = !(ti.flags & kEnd);

    if (start) {                                             // a row's query heads
      start = false;
      if (!EARLY) load_query(ti.row, ti.vh);
      const Heads h = heads_of(p, ti.vh);
      head0 = h.first;
      rows = h.count;
      begins = ti.flags & kFirst;
      const float to_log2 = p.scale * 1.4426950408889634f * (FP8 && p.k_scale ? p.k_scale[h.kvh] : 1.f);
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        float2 x[KS][2];
#pragma unroll
        for (int s = 0; s < KS; ++s) x[s][0] = Pair<T>::values(raw[s][hb][0]), x[s][1] = Pair<T>::values(raw[s][hb][1]);
        mult[hb][0] = mult[hb][1] = to_log2;
        if constexpr (FP8) {
          float a = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s)
            a = fmaxf(a, fmaxf(fmaxf(fabsf(x[s][0].x), fabsf(x[s][0].y)), fmaxf(fabsf(x[s][1].x), fabsf(x[s][1].y))));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
          // largest element to [2^13, 2^14); the exponent of 2^e stays within fp32's
          const int e = a > 0.f && a < INFINITY ? max(-126, min(126, 13 - ilogbf(a))) : 0;
          const float f = ldexpf(1.f, e), back = ldexpf(1.f, -e);
#pragma unroll
          for (int s = 0; s < KS; ++s) x[s][0].x *= f, x[s][0].y *= f, x[s][1].x *= f, x[s][1].y *= f;
          mult[hb][0] *= __shfl_sync(0xffffffffu, back, 8 * t);
          mult[hb][1] *= __shfl_sync(0xffffffffu, back, 8 * t + 4);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int u = 0; u < TQ; ++u)
              qf[u][s][hb][j] = u + 1 < TQ ? mkw::take_query_term(Op{}, x[s][j].x, x[s][j].y) : mkw::take_input_term(Op{}, x[s][j].x, x[s][j].y);
#pragma unroll
        for (int c = 0; c < DB; ++c) o[c][hb][0] = o[c][hb][1] = o[c][hb][2] = o[c][hb][3] = 0.f;
        m[hb][0] = m[hb][1] = -INFINITY;
        l[hb][0] = l[hb][1] = 0.f;
      }
    }

    // ---- scores: slots 16 nb + g, + 8 by heads 2t, 2t + 1 -----------------------
    // two sums a block (even and odd steps; the first term and the others), for shorter chains
    float sc[PN][HB][4], sl[PN][HB][4];
#pragma unroll
    for (int s = 0; s < KS; s += 2) {
#pragma unroll
      for (int nb = 0; nb < PN; ++nb) {
        uint32_t a[2][4];
        const int r = nb * 16 + (lane & 15);
        if constexpr (!FP8) {
          mkw::ldmatrix4(a[0], kt + TL::at(r, 2 * s + (lane >> 4)));
          mkw::ldmatrix4(a[1], kt + TL::at(r, 2 * s + 2 + (lane >> 4)));
        } else {
          uint32_t f[4];
          mkw::ldmatrix4(f, kt + TL::at(r, s + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mkw::e4m3x4_to_half2(f[2 * j], a[j][0], a[j][2]);
            mkw::e4m3x4_to_half2(f[2 * j + 1], a[j][1], a[j][3]);
          }
        }
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          float *c = sc[nb][hb], *e = sl[nb][hb];
          if constexpr (TQ == 1) {
            if (s == 0) {
              mkw::mma_zero(Op{}, c, a[0], qf[0][s][hb][0], qf[0][s][hb][1]);
              mkw::mma_zero(Op{}, e, a[1], qf[0][s + 1][hb][0], qf[0][s + 1][hb][1]);
            } else {
              mkw::mma(Op{}, c, a[0], qf[0][s][hb][0], qf[0][s][hb][1]);
              mkw::mma(Op{}, e, a[1], qf[0][s + 1][hb][0], qf[0][s + 1][hb][1]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (s + j == 0) mkw::mma_zero(Op{}, c, a[j], qf[0][s + j][hb][0], qf[0][s + j][hb][1]);
              else mkw::mma(Op{}, c, a[j], qf[0][s + j][hb][0], qf[0][s + j][hb][1]);
#pragma unroll
              for (int u = TQ - 1; u > 0; --u) {
                if (s + j == 0 && u == TQ - 1) mkw::mma_zero(Op{}, e, a[j], qf[u][s + j][hb][0], qf[u][s + j][hb][1]);
                else mkw::mma(Op{}, e, a[j], qf[u][s + j][hb][0], qf[u][s + j][hb][1]);
              }
            }
          }
        }
      }
    }
    const bool edge = ti.pos < ti.lo || ti.pos + POS > ti.hi;
    float alpha[HB][2];
    uint32_t pf[TP][PN][HB][2];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nb = 0; nb < PN; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float s = (sc[nb][hb][c] + sl[nb][hb][c]) * mult[hb][c & 1];
          if (edge) {
            const int pos = ti.pos + 16 * nb + g + (c >> 1) * 8;
            if (pos < ti.lo || pos >= ti.hi) s = -INFINITY;
          }
          sc[nb][hb][c] = s;
          x[c & 1] = fmaxf(x[c & 1], s);
        }
      float base[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float n = fmaxf(m[hb][j], column_max(x[j]) - kShift);
        base[j] = join_base(n);
        alpha[hb][j] = mkw::exp2_fast(m[hb][j] - base[j]);
        m[hb][j] = n;
        l[hb][j] *= alpha[hb][j];
      }
#pragma unroll
      for (int nb = 0; nb < PN; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float a = mkw::exp2_fast(sc[nb][hb][2 * j] - base[0]), b = mkw::exp2_fast(sc[nb][hb][2 * j + 1] - base[1]);
          if constexpr (!FP8) a *= p.shrink, b *= p.shrink;
          l[hb][0] += a;
          l[hb][1] += b;
#pragma unroll
          for (int u = 0; u < TP - 1; ++u) pf[u][nb][hb][j] = mkw::transpose8(mkw::take_weight_term(Op{}, a, b));
          pf[TP - 1][nb][hb][j] = mkw::transpose8(mkw::take_term(Op{}, a, b));
        }
    }

    // ---- values: block c of 16 elements by heads 2t, 2t + 1; rows g and g + 8 of a block are its elements of that
    // number (bf16) or elements 2g and 2g + 1 (e4m3, whose 16-bit pairs the transposition keeps together) ----------
    constexpr int CB = FP8 ? 2 : 1;                          // blocks a matrix load brings
#pragma unroll
    for (int c = 0; c < DB; c += CB) {
      float e[CB][HB][4];
#pragma unroll
      for (int nb = 0; nb < PN; ++nb) {
        uint32_t a[CB][4];
        if constexpr (!FP8) {
          mkw::ldmatrix4_trans(a[0], vt + TL::at(nb * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * c + ((lane >> 3) & 1)));
        } else {
          uint32_t f[4];
          mkw::ldmatrix4_trans(f, vt + TL::at(nb * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j)                        // bytes (slot, element) 00 01 10 11 to 00 10 01 11
            mkw::e4m3x4_to_half2(__byte_perm(f[j], 0, 0x3120), a[j >> 1][2 * (j & 1)], a[j >> 1][2 * (j & 1) + 1]);
        }
#pragma unroll
        for (int k = 0; k < CB; ++k)
#pragma unroll
          for (int hb = 0; hb < HB; ++hb)
#pragma unroll
            for (int u = TP - 1; u >= 0; --u) {
              if (nb == 0 && u == TP - 1) mkw::mma_zero(Op{}, e[k][hb], a[k], pf[u][nb][hb][0], pf[u][nb][hb][1]);
              else mkw::mma(Op{}, e[k][hb], a[k], pf[u][nb][hb][0], pf[u][nb][hb][1]);
            }
      }
#pragma unroll
      for (int k = 0; k < CB; ++k)
#pragma unroll
        for (int hb = 0; hb < HB; ++hb)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[c + k][hb][j] = o[c + k][hb][j] * alpha[hb][j & 1] + e[k][hb][j];
    }
    if (ti.flags & kBad) {
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) l[hb][0] = l[hb][1] = NAN;
    }
    __syncwarp();                                            // every lane has read the stage (and, at the end, the ring)

    const bool ends = ti.flags & kLast;
    if (ends || !more) {
      start = true;
      // A whole row of the warp is stored from the stage just read, 8 query heads at a time; a part stays where the join
      // finds it (a cluster's parts are all joined at the end).
      const bool whole = begins && ends && p.way != kByCluster;
      float *part = reinterpret_cast<float *>(smem + w * kStages * TL::STAGE);
      if (ends) part = reinterpret_cast<float *>(whole ? smem + (kt - smem_at) : smem + kWarps * kStages * TL::STAGE + w * p.gr * PST * 4);
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int h = 8 * hb + 2 * t + k;
          const float sum = column_sum(l[hb][k]);
          if (h < rows) {
            float *to = part + (whole ? h - 8 * hb : h) * PST;
            if (g == 0) to[D] = m[hb][k], to[D + 1] = sum;
            to += FP8 ? 2 * g : g;
#pragma unroll
            for (int c = 0; c < DB; ++c) {
              to[16 * c] = o[c][hb][k];
              to[16 * c + (FP8 ? 1 : 8)] = o[c][hb][2 + k];
            }
          }
        }
        __syncwarp();
        if (whole) {
          const float vsc = FP8 && p.v_scale ? p.v_scale[heads_of(p, ti.vh).kvh] : 1.f;
#pragma unroll 1
          for (int h = 0; h < min(8, rows - 8 * hb); ++h) {
            const float *from = part + h * PST;
            float x[D / 32];
            load_part(from + lane * (D / 32), x);
            write_head<T, D>(p, lane, ti.row, head0 + 8 * hb + h, from[D], from[D + 1], x, vsc);
          }
          __syncwarp();
        }
      }
      if (!whole && lane == 0) s_part[2 * w + (ends ? 0 : 1)] = PartInfo{ti.row, ti.vh, begins, ends};
      if (EARLY && more) load_query(s_tile[w][stage].row, s_tile[w][stage].vh);   // (the next tile has been asked for, and written down)
    }
  }
  mkw::cp_async_wait<0>();
  if (p.way == kJoined && tid == 0) p.records[cta] = make_int4(0, 0, 0, 0);
  __syncthreads();

  // ---- join the warps' parts, in order, a query head of a row a warp -----------------------------------------
  // lane j knows the jth part, and where it is: the ring of its warp (a part that does not end its row), or the space
  // beside the rings
  const PartInfo mine = lane < 2 * kWarps ? s_part[lane] : PartInfo{-1, 0, 0, 0};
  const unsigned valid = __ballot_sync(0xffffffffu, mine.row >= 0);
  const int beside = kWarps * kStages * TL::STAGE;
  int mine_at = (lane & 1) ? (lane >> 1) * kStages * TL::STAGE : beside + (lane >> 1) * p.gr * PST * 4;
  // a group: consecutive parts of the same row and head; lane j says whether part j begins one
  const unsigned below = valid & ((1u << lane) - 1u);
  const int prev = below ? 31 - __clz(below) : lane;
  const int prev_row = __shfl_sync(0xffffffffu, mine.row, prev), prev_vh = __shfl_sync(0xffffffffu, mine.vh, prev);
  const unsigned starts = __ballot_sync(0xffffffffu, mine.row >= 0 && (!below || prev_row != mine.row || prev_vh != mine.vh));
  int items = __popc(starts) * p.gr;
  // A cluster's parts are all of one row and head.  Query head r goes to the inbox of CTA r % cluster, which in a second
  // round joins what all have of it.
  const int owned = p.way == kByCluster ? (p.gr + p.cluster - 1) / p.cluster : 0, inbox = beside + kWarps * p.gr * PST * 4;   // [CTA][owned][PST]
  const int rank = p.way == kByCluster ? cta % p.cluster : 0;
  if (p.way == kByCluster) {
    items = p.gr;
    mkw::cluster_wait();
  }
#pragma unroll 1
  for (int round = 0;; ++round) {
#pragma unroll 1
    for (int i = w; i < items; i += kWarps) {
      int group = i / p.gr, r = i - group * p.gr, a = 0, b = 0, row_of = 0, vh_of = cta / p.cluster, first = 1, ends = 1;
      unsigned in_group = valid;
      if (p.way == kByCluster) {
        if (round == 1) in_group = (1u << p.cluster) - 1u;
      } else {
        unsigned rest = starts;
        for (int k = 0; k < group; ++k) rest &= rest - 1u;
        a = __ffs(rest) - 1;                                 // the group's first part
        const unsigned later = rest & (rest - 1u);
        in_group = valid & ~((1u << a) - 1u) & (later ? (later & -later) - 1u : ~0u);
        b = 31 - __clz(in_group);                            // and its last
        row_of = __shfl_sync(0xffffffffu, mine.row, a), vh_of = __shfl_sync(0xffffffffu, mine.vh, a);
        first = __shfl_sync(0xffffffffu, mine.begins, a), ends = __shfl_sync(0xffffffffu, mine.ends, b);
      }
      const Heads h = heads_of(p, vh_of);
      float mx, sum, x[D / 32];
      join_shared<D>(lane, in_group, smem, mine_at + r * PST * 4, mx, sum, x);
      if (round == 1) r = i * p.cluster + rank;
      if (r >= h.count) continue;
      if (p.way == kByCluster && round == 0) {
        const uint32_t to = mkw::remote(smem + inbox + (rank * owned + r / p.cluster) * PST * 4, r % p.cluster);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) mkw::store_remote(to + (lane * (D / 32) + k) * 4, x[k]);
        if (lane == 0) {
          mkw::store_remote(to + D * 4, mx);
          mkw::store_remote(to + D * 4 + 4, sum);
        }
      } else if (first && ends) {
        if (sp.count || p.way != kByCluster)                 // (a row without tokens is written above)
          write_head<T, D>(p, lane, row_of, h.first + r, mx, sum, x, FP8 && p.v_scale ? p.v_scale[h.kvh] : 1.f);
      } else {
        float *to = p.parts + ((static_cast<int64_t>(cta) * 2 + (first ? 1 : 0)) * p.gr + r) * PST;
        store_row(to + lane * (D / 32), x);
        if (lane == 0) {
          to[D] = mx;
          to[D + 1] = sum;
          if (first && r == 0) {
            // the last CTA with tiles of this row: the one whose range holds the row's last unit
            int before_row = s_scan[row_of / per];
#pragma unroll 1
            for (int k = row_of / per * per; k < row_of; ++k) before_row += span_of<POS>(p, p.lengths[k]).cost;
            const int cost = span_of<POS>(p, p.lengths[row_of]).cost;
            p.records[cta] = make_int4(row_of, vh_of, Shares(units, ctas).of(before_row * static_cast<int>(p.vh.value) + (vh_of + 1) * cost - 1), 1);
          }
        }
      }
    }
    if (p.way != kByCluster || round == 1) return;
    mkw::cluster_arrive();
    mkw::cluster_wait();
    items = owned;
    mine_at = inbox + lane * owned * PST * 4;
  }
}

// Joins the rows that more than one CTA had a share of: CTA c takes the row that
// begins in attend_kernel's CTA c and goes on in the next ones, a query head a warp.
template <class T, int D>
__global__ void __launch_bounds__(kAttnThreads) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int PST = kPartStride<D>;
  const int cta = blockIdx.x, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  mkw::follow_previous_kernel();
  const int4 rec = p.records[cta];
  if (!rec.w) return;
  const Heads h = heads_of(p, rec.y);
  const float vsc = p.v_scale ? p.v_scale[h.kvh] : 1.f;
  const int n = rec.z - cta + 1;
  if (const int r = blockIdx.y * kWarps + w; r < h.count) {
    float m = -INFINITY, l = 0.f, x[D / 32] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
      float mj, lj, xj[D / 32];
      const unsigned there = n - j0 >= 32 ? ~0u : (1u << (n - j0)) - 1u;
      join_parts<D>(lane, there, p.parts + (static_cast<int64_t>(cta + j0) * 2 * p.gr + r) * PST,
                    (lane * 2 + (j0 + lane == 0 ? 1 : 0)) * p.gr * PST * 4, mj, lj, xj);
      const float mx = fmaxf(m, mj), base = join_base(mx), f = mkw::exp2_fast(m - base), fj = mkw::exp2_fast(mj - base);
      m = mx;
      l = l * f + lj * fj;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) x[k] = x[k] * f + xj[k] * fj;
    }
    write_head<T, D>(p, lane, rec.x, h.first + r, m, l, x, vsc);
  }
}

int sm_count(int *device) {
  static std::atomic<int> known[mkw::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (device) *device = dev;
  if (dev < 0 || dev >= mkw::kMaxDevices) return -1;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return -1;
    }
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// where a call's workspace comes from: the caller's, or his function, asked only if the call needs one
struct Workspace {
  void *given;
  mk_workspace_fn ask;
  void *context;
  int64_t bytes;
};

template <class T, bool FP8, int D, int HB>
int launch_heads(AttnParams &p, const Workspace &ws, int grid, int dev, cudaStream_t s) {
  using TL = Tile<D, FP8>;
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &attend_kernel<T, FP8, D, HB>;
  mkw::Ready &r = ready[dev];
  if (!r.get(reinterpret_cast<const void *>(fn), kAttnThreads, kMaxSmem)) return MK_ERR_CUDA;
  const int64_t tiles = (p.window > 0 ? std::min(p.window, p.capacity) : p.capacity) / TL::POS + 2;   // of a row at most
  p.way = tiles <= kShortTiles ? kWhole : kJoined;
  p.cluster = 1;
  if (p.n == 1) {
    // the largest clusters of which there is one for each head at once, as long as their warps have a tile each
    for (int i = 0; i < 4 && static_cast<int>(p.vh.value) <= r.clusters[i] && (i == 0 || tiles > p.cluster * kWarps); ++i) p.cluster = 2 << i;
    if (p.cluster > 1) p.way = kByCluster;
  }
  const int inbox = p.way == kByCluster ? p.cluster * ((p.gr + p.cluster - 1) / p.cluster) : 0;
  static_assert(kWarps * kStages * TL::STAGE + (kWarps * 16 + 16) * kPartStride<D> * 4 <= kMaxSmem, "16 heads, 16 CTAs");
  const int parts = (kWarps * p.gr + inbox) * kPartStride<D> * 4;
  const int ctas = p.way == kByCluster ? static_cast<int>(p.vh.value) * p.cluster : grid, smem = kWarps * kStages * TL::STAGE + parts;
  if (p.way == kJoined) {
    p.records = static_cast<int4 *>(ws.ask ? ws.ask(ws.context, ws.bytes) : ws.given);
    if (!p.records) return MK_ERR_NO_MEMORY;
    if (reinterpret_cast<uintptr_t>(p.records) & 15u) return MK_ERR_INVALID_ARG;
    p.parts = reinterpret_cast<float *>(p.records + grid);
  }
  const int rc = mkw::launch_after(fn, dim3(ctas), kAttnThreads, smem, s, p, p.cluster);
  if (rc != MK_OK || p.way != kJoined) return rc;
  return mkw::launch_after(&join_kernel<T, D>, dim3(grid, (p.gr + kWarps - 1) / kWarps), kAttnThreads, 0, s, p);
}

template <class T, bool FP8, int D>
int launch_attend(AttnParams &p, const Workspace &ws, int grid, int dev, cudaStream_t s) {
  return p.gr <= 8 ? launch_heads<T, FP8, D, 1>(p, ws, grid, dev, s) : launch_heads<T, FP8, D, 2>(p, ws, grid, dev, s);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// an element stride (>= 0) that is a multiple of 16 bytes
bool stride_ok(int64_t s, int elem) { return s >= 0 && s <= (int64_t{1} << 48) && s * elem % 16 == 0; }

int check_cache(const mk_paged_kv *kv) {
  if (!kv || !kv->k || !kv->v || (kv->dtype != MK_BF16 && kv->dtype != MK_E4M3)) return MK_ERR_INVALID_ARG;
  if (kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->page_size < 1 || kv->table_rows < 0 || kv->table_cols < 0 ||
      kv->table_stride < 0 || (!kv->table && kv->table_rows > 0 && kv->table_cols > 0))
    return MK_ERR_INVALID_ARG;
  const int es = kv->dtype == MK_E4M3 ? 1 : 2;
  if (!aligned16(kv->k) || !aligned16(kv->v) || !stride_ok(kv->page_stride, es) || !stride_ok(kv->head_stride, es) ||
      !stride_ok(kv->slot_stride, es))
    return MK_ERR_INVALID_ARG;
  if ((kv->k_scale == nullptr) != (kv->v_scale == nullptr) || (kv->k_scale && kv->dtype != MK_E4M3)) return MK_ERR_INVALID_ARG;
  if (kv->head_dim != 64 && kv->head_dim != 128) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

void fill_cache(AppendParams &p, const mk_paged_kv *kv) {
  p.k_cache = kv->k;
  p.v_cache = kv->v;
  p.page_stride = kv->page_stride, p.head_stride = kv->head_stride, p.slot_stride = kv->slot_stride;
  p.table = kv->table;
  p.table_stride = kv->table_stride;
  p.table_rows = kv->table_rows, p.table_cols = kv->table_cols;
  p.n_pages = kv->n_pages;
  p.page_size.set(kv->page_size);
  p.hkv = kv->n_kv_heads;
  p.k_scale = kv->k_scale, p.v_scale = kv->v_scale;
}

int append_range(const mk_paged_kv *kv, const void *k, const void *v, int64_t row, int64_t head, int32_t count,
                 int32_t seq, int32_t slot0, int32_t *status, cudaStream_t stream) {
  AppendParams p = {};
  fill_cache(p, kv);
  p.k = k, p.v = v;
  p.k_row = p.v_row = row, p.k_head = p.v_head = head;
  p.n = count;
  p.seq0 = seq, p.slot0 = slot0;
  p.status = status;
  return run_append(p, MK_BF16, kv->dtype, kv->head_dim, stream);
}

}  // namespace mkv

using namespace mkv;

extern "C" int mk_paged_append(const mk_paged_kv *kv, const mk_append_args *a, mk_stream stream) {
  const int rc = check_cache(kv);
  if (rc != MK_OK) return rc;
  if (!a || a->n < 0 || a->n_q_heads < 0 || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->rope_mode < 0 ||
      a->rope_mode > 2 || a->rope_rows < 0)
    return MK_ERR_INVALID_ARG;
  if (a->n == 0) return MK_OK;
  const int es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->k || !a->v || !a->slots || !aligned16(a->k) || !aligned16(a->v) || !stride_ok(a->k_row, es) ||
      !stride_ok(a->k_head, es) || !stride_ok(a->v_row, es) || !stride_ok(a->v_head, es))
    return MK_ERR_INVALID_ARG;
  if (a->n_q_heads > 0 && (!a->q || !a->q_out || !aligned16(a->q) || !aligned16(a->q_out) || !stride_ok(a->q_row, es) ||
                           !stride_ok(a->q_head, es) || !stride_ok(a->out_row, es) || !stride_ok(a->out_head, es)))
    return MK_ERR_INVALID_ARG;
  if ((a->q_norm || a->k_norm) && (!(a->rms_eps >= 0.f) || !aligned16(a->q_norm) || !aligned16(a->k_norm))) return MK_ERR_INVALID_ARG;
  if (a->rope) {
    if (!aligned16(a->rope)) return MK_ERR_INVALID_ARG;
    if (a->rope_mode != 0 &&
        (!a->positions || a->mrope_sections[0] < 0 || a->mrope_sections[1] < 0 || a->mrope_sections[2] < 0 ||
         static_cast<int64_t>(a->mrope_sections[0]) + a->mrope_sections[1] + a->mrope_sections[2] != kv->head_dim / 2))
      return MK_ERR_INVALID_ARG;
  }
  AppendParams p = {};
  fill_cache(p, kv);
  p.q = a->q, p.k = a->k, p.v = a->v, p.q_out = a->q_out;
  p.q_row = a->q_row, p.q_head = a->q_head, p.k_row = a->k_row, p.k_head = a->k_head;
  p.v_row = a->v_row, p.v_head = a->v_head, p.out_row = a->out_row, p.out_head = a->out_head;
  p.seqs = a->seqs, p.slots = a->slots, p.positions = a->positions;
  p.rope = reinterpret_cast<const float2 *>(a->rope);
  p.rope_rows = a->rope_rows, p.rope_mode = a->rope_mode;
  p.sec0 = a->mrope_sections[0], p.sec1 = a->mrope_sections[1], p.sec2 = a->mrope_sections[2];
  p.q_norm = static_cast<const uint16_t *>(a->q_norm), p.k_norm = static_cast<const uint16_t *>(a->k_norm);
  p.eps = a->rms_eps;
  p.n = a->n, p.hq = a->n_q_heads;
  p.status = a->status;
  return run_append(p, a->dtype, kv->dtype, kv->head_dim, reinterpret_cast<cudaStream_t>(stream));
}

namespace {

int64_t workspace_bytes(int grid, int group, int d) {
  return static_cast<int64_t>(grid) * (16 + 2 * std::min(group, 16) * (d + 4) * 4);
}

int check_heads(int32_t hq, int32_t hkv, int32_t d) {
  if (hkv < 1 || hq < 1 || hq % hkv) return MK_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? MK_OK : MK_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" int64_t mk_paged_attention_workspace(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  const int rc = check_heads(n_q_heads, n_kv_heads, head_dim);
  if (rc != MK_OK) return rc;
  const int grid = sm_count(nullptr);
  return grid < 0 ? MK_ERR_CUDA : workspace_bytes(grid, n_q_heads / n_kv_heads, head_dim);
}

namespace {

int attention(const mk_paged_kv *kv, const mk_attention_args *a, mk_stream stream, mk_workspace_fn ask, void *context) {
  int rc = check_cache(kv);
  if (rc != MK_OK) return rc;
  if (!a || a->n < 0 || a->n > kv->table_rows || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->window < 0 ||
      !std::isfinite(a->scale))
    return MK_ERR_INVALID_ARG;
  rc = check_heads(a->n_q_heads, kv->n_kv_heads, kv->head_dim);
  if (rc != MK_OK) return rc;
  if (a->n == 0) return MK_OK;
  const int es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->q || !a->out || !a->lengths || (!ask && !a->workspace) || !aligned16(a->q) || !aligned16(a->out) ||
      (!ask && !aligned16(a->workspace)) || !stride_ok(a->q_row, es) || !stride_ok(a->q_head, es) || !stride_ok(a->out_row, es) ||
      !stride_ok(a->out_head, es))
    return MK_ERR_INVALID_ARG;
  // slots and the cost of all rows and heads are counted in 32 bits
  const int64_t slots = static_cast<int64_t>(kv->table_cols) * kv->page_size;
  if (slots > INT32_MAX - 64 || a->n_q_heads > (1 << 20) ||
      (slots / 16 + 2 + kMaxRowCost) * a->n > INT32_MAX / (kv->n_kv_heads * ((a->n_q_heads / kv->n_kv_heads + 15) / 16)))
    return MK_ERR_UNSUPPORTED;
  int dev = 0;
  const int grid = sm_count(&dev);
  if (grid < 0) return MK_ERR_CUDA;
  AttnParams p = {};
  p.group = a->n_q_heads / kv->n_kv_heads;
  const Workspace ws = {a->workspace, ask, context, workspace_bytes(grid, p.group, kv->head_dim)};
  if (!ask && a->workspace_bytes < ws.bytes) return MK_ERR_INVALID_ARG;
  p.q = a->q, p.k = kv->k, p.v = kv->v, p.out = a->out, p.lse = a->lse;
  p.q_row = a->q_row, p.q_head = a->q_head, p.out_row = a->out_row, p.out_head = a->out_head;
  p.page_stride = kv->page_stride, p.head_stride = kv->head_stride, p.slot_stride = kv->slot_stride;
  p.table = kv->table, p.table_stride = kv->table_stride;
  p.capacity = static_cast<int>(slots);
  p.dense = kv->slot_stride == kv->head_dim;
  p.lengths = a->lengths;
  p.k_scale = kv->k_scale, p.v_scale = kv->v_scale;
  p.status = a->status;
  p.n = a->n, p.hq = a->n_q_heads, p.hkv = kv->n_kv_heads;
  p.n_pages = kv->n_pages;
  p.page_size.set(kv->page_size);
  p.window = a->window;
  p.chunks.set((p.hq + 15) / 16);
  p.blocks.set((p.group + 15) / 16);
  p.vh.set(p.hkv * ((p.group + 15) / 16));
  p.gr = std::min(p.group, 16);
  p.row_cost = row_cost(p.gr);
  p.scale = a->scale;
  int spare = 0;                                             // 2^spare: as many tokens as a row may have, or more
  for (const int tokens = p.window > 0 ? std::min(p.window, p.capacity) : p.capacity; (int64_t{1} << spare) < tokens;) ++spare;
  if (kv->dtype != MK_BF16) spare = 0;                       // (e4m3 values are far from fp32's largest)
  p.shrink = std::ldexp(1.f, -spare), p.grow = std::ldexp(1.f, spare);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (a->dtype == MK_F32) {
    if (kv->dtype == MK_BF16)
      return kv->head_dim == 64 ? launch_attend<float, false, 64>(p, ws, grid, dev, s) : launch_attend<float, false, 128>(p, ws, grid, dev, s);
    return kv->head_dim == 64 ? launch_attend<float, true, 64>(p, ws, grid, dev, s) : launch_attend<float, true, 128>(p, ws, grid, dev, s);
  }
  if (kv->dtype == MK_BF16)
    return kv->head_dim == 64 ? launch_attend<B, false, 64>(p, ws, grid, dev, s) : launch_attend<B, false, 128>(p, ws, grid, dev, s);
  return kv->head_dim == 64 ? launch_attend<B, true, 64>(p, ws, grid, dev, s) : launch_attend<B, true, 128>(p, ws, grid, dev, s);
}

}  // namespace

extern "C" int mk_paged_attention(const mk_paged_kv *kv, const mk_attention_args *a, mk_stream stream) {
  return attention(kv, a, stream, nullptr, nullptr);
}

extern "C" int mk_paged_attention_ask(const mk_paged_kv *kv, const mk_attention_args *a, mk_workspace_fn workspace, void *context,
                                      mk_stream stream) {
  return workspace ? attention(kv, a, stream, workspace, context) : MK_ERR_INVALID_ARG;
}
