// Adjustment of logits before a token is chosen (mk_adjust_logits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_paged.h"
#include "mk_mma.cuh"

namespace mklogits {

// ---------------------------------------------------------------------------
// y = penalties(x, how often the row's history holds the token) + bias, -inf where the mask's bit is 0.
//
// Bound by the logits' bytes for a batch, by latency for one row.  A CTA has a slice of a row's vocabulary and a word of
// shared memory for each of its tokens.  It asks for its logits first (one or two 16-byte loads a thread, all in flight),
// walks the row's whole history and counts the tokens of its slice by integer atomics (any order gives the same counts)
// while those loads are on their way, stores the logits with the mask, and then goes over the tokens that it has counted:
// those are few, and a warp that looked at each of its tokens on the way took longer (64 rows of 151936 28 us for 16).  The one
// who counts a token first writes it down; which order that gives does not matter, as each is adjusted on its own.  Biases
// set a bit of the word: a token's only entry adjusts it, and of a token with several, which has a bit in a set of its own, who
// has the token adds them up in their order (20000 biases for each of 64 rows
// 73 us, 7330 where each token looked for all of its own).
// ---------------------------------------------------------------------------

constexpr int kThreads = 1024;
constexpr int kMost = 2;       // 16-byte pieces a thread

struct LogitsParams {
  const void *x;
  void *out;
  const int32_t *tokens, *lengths, *prompts, *bias_ids;
  const float *repetition, *presence, *frequency, *bias;
  const uint32_t *mask;
  int64_t x_row, out_row, tokens_row, ids_row, bias_row, mask_row;
  int n, vocab, columns, biases;
  int per, slices;             // pieces a thread, CTAs a row
};

template <class T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float value(const uint4 &w, int e) { return __uint_as_float((&w.x)[e]); }
  static __device__ __forceinline__ void put(uint4 &w, int e, float x) { (&w.x)[e] = __float_as_uint(x); }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float value(const uint4 &w, int e) {
    const uint32_t u = (&w.x)[e >> 1];
    return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
  }
  static __device__ __forceinline__ void put(uint4 &w, int e, __nv_bfloat16 x) {
    const uint32_t u = __bfloat16_as_ushort(x);
    uint32_t &to = (&w.x)[e >> 1];
    to = e & 1 ? (to & 0xffffu) | u << 16 : (to & 0xffff0000u) | u;
  }
};

// W: a token's word, 16 bits where the history is short enough for its count
template <class W>
struct Word {
  static constexpr uint32_t kPrompt = sizeof(W) == 2 ? 0x8000u : 0x80000000u, kBias = kPrompt >> 1, kCount = kBias - 1;
  // count, or mark, token t: its word before
  static __device__ __forceinline__ uint32_t add(uint32_t *words, int t, uint32_t by) {
    if (sizeof(W) == 2) return atomicAdd(&words[t >> 1], by << (16 * (t & 1))) >> (16 * (t & 1)) & 0xffffu;
    return atomicAdd(&words[t], by);
  }
  static __device__ __forceinline__ uint32_t mark(uint32_t *words, int t, uint32_t bit) {
    if (sizeof(W) == 2) return atomicOr(&words[t >> 1], bit << (16 * (t & 1))) >> (16 * (t & 1)) & 0xffffu;
    return atomicOr(&words[t], bit);
  }
  static __device__ __forceinline__ uint32_t of(const uint32_t *words, int t) { return reinterpret_cast<const W *>(words)[t]; }
};

template <class T, class W>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int N = Piece<T>::N;
  using Wd = Word<W>;
  extern __shared__ __align__(16) uint32_t words[];
  mkw::follow_previous_kernel();
  const int tid = threadIdx.x, row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
  int length = p.columns;
  if (p.lengths) {
    length = p.lengths[row];
    if (length < 0) return;                                // a padding row
    length = min(length, p.columns);
  }
  const T *x = static_cast<const T *>(p.x) + row * p.x_row;
  T *out = static_cast<T *>(p.out) + row * p.out_row;
  // Pieces are counted from the 16-byte boundary at or below the row: piece c has elements c N - head ..
  const int head = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const bool together = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int size = p.per * kThreads * N, first = slice * size - head;   // the slice's tokens: [first, first + size)
  uint4 raw[kMost];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k >= p.per) break;
    const int e0 = first + (k * kThreads + tid) * N;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (e0 >= 0 && e0 + N <= p.vocab) {
      raw[k] = __ldcs(reinterpret_cast<const uint4 *>(x + e0));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e0 + e >= 0 && e0 + e < p.vocab) Piece<T>::put(raw[k], e, x[e0 + e]);
    }
  }
  float repetition = 1.f, presence = 0.f, frequency = 0.f;
  if (p.repetition) repetition = p.repetition[row];
  if (p.presence) presence = p.presence[row];
  if (p.frequency) frequency = p.frequency[row];
  const bool counted = length > 0 && (repetition != 1.f || presence != 0.f || frequency != 0.f), marked = counted || p.biases > 0;
  __shared__ int s_found;
  uint16_t *found = reinterpret_cast<uint16_t *>(words + size * static_cast<int>(sizeof(W)) / 4);   // the slice's tokens that have a word
  // a bit for four tokens: whether any of them has more than one bias (with a bit each the shared memory of two CTAs passes
  // 132 KB, and 256 rows take 70.3 us for 69.2)
  uint32_t *several = reinterpret_cast<uint32_t *>(found + size);
  if (marked) {
    for (int i = tid; i < size * static_cast<int>(sizeof(W)) / 16; i += kThreads) reinterpret_cast<uint4 *>(words)[i] = make_uint4(0, 0, 0, 0);
    if (p.biases > 0)
      for (int i = tid; i < size / 128; i += kThreads) several[i] = 0;
    if (tid == 0) s_found = 0;
    __syncthreads();
    if (counted) {
      const int32_t *history = p.tokens + row * p.tokens_row;
      const int prompt = p.prompts ? p.prompts[row] : 0;
#pragma unroll 4
      for (int j = tid; j < length; j += kThreads) {
        const int id = history[j], t = id - first;          // (first is not below -7; ids past the vocabulary do not count, whatever t is)
        if (id < 0 || id >= p.vocab || t < 0 || t >= size) continue;
        if ((j < prompt ? Wd::mark(words, t, Wd::kPrompt) : Wd::add(words, t, 1)) == 0) found[atomicAdd(&s_found, 1)] = static_cast<uint16_t>(t);
      }
    }
    for (int j = tid; j < p.biases; j += kThreads) {
      const int id = p.bias_ids[row * p.ids_row + j], t = id - first;
      if (id < 0 || id >= p.vocab || t < 0 || t >= size) continue;
      const uint32_t before = Wd::mark(words, t, Wd::kBias);
      if (before == 0) found[atomicAdd(&s_found, 1)] = static_cast<uint16_t>(t);
      if (before & Wd::kBias) atomicOr(&several[t >> 7], 1u << (t >> 2 & 31));
    }
  }
  const uint32_t *mask = p.mask ? p.mask + row * p.mask_row : nullptr;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k >= p.per) break;
    const int e0 = first + (k * kThreads + tid) * N;
    if (e0 >= p.vocab || e0 + N <= 0) continue;
    if (mask) {
      const int a = max(e0, 0), z = min(e0 + N, p.vocab) - 1;
      const uint32_t allowed = __funnelshift_r(mask[a >> 5], mask[z >> 5], a & 31) << (a - e0);   // bits of the piece's elements
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (!(allowed >> e & 1)) Piece<T>::put(raw[k], e, static_cast<T>(-INFINITY));
    }
    if (together && e0 >= 0 && e0 + N <= p.vocab) {
      *reinterpret_cast<uint4 *>(out + e0) = raw[k];
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e0 + e >= 0 && e0 + e < p.vocab) out[e0 + e] = static_cast<T>(Piece<T>::value(raw[k], e));
    }
  }
  if (!marked) return;
  __syncthreads();                                         // (in place, x is out: what is not masked has been put back as it was)
  // the tokens that have been written down, and the biases that are the only ones of theirs
  const int32_t *ids = p.bias_ids + row * p.ids_row;
  const float *bias = p.bias + row * p.bias_row;
  auto alone = [&](int t) { return !(several[t >> 7] >> (t >> 2 & 31) & 1); };
  const int tokens = s_found;
  for (int i = tid; i < tokens + p.biases; i += kThreads) {
    const int j = i - tokens, id = j < 0 ? first + found[i] : ids[j], t = id - first;
    if (j >= 0 && (id < 0 || id >= p.vocab || t < 0 || t >= size || !alone(t))) continue;
    if (mask && !(mask[id >> 5] >> (id & 31) & 1)) continue;
    const uint32_t word = Wd::of(words, t);
    const bool biased = word & Wd::kBias;
    if (j < 0 && biased && alone(t)) continue;
    const int count = word & Wd::kCount;
    float y = static_cast<float>(x[id]);
    if (count || (word & Wd::kPrompt)) y = y > 0.f ? __fdiv_rn(y, repetition) : y * repetition;
    if (count) y = __fsub_rn(__fsub_rn(y, __fmul_rn(frequency, static_cast<float>(count))), presence);
    if (j >= 0) {
      y += bias[j];
    } else if (biased) {
      float sum = 0.f;
      int k0 = 0;
#pragma unroll 1
      for (; k0 + 8 <= p.biases; k0 += 8) {                // (eight on their way together)
        int at[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) at[k] = ids[k0 + k];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (at[k] == id) sum += bias[k0 + k];
      }
#pragma unroll 1
      for (; k0 < p.biases; ++k0)
        if (ids[k0] == id) sum += bias[k0];
      y += sum;
    }
    out[id] = static_cast<T>(y);
  }
}

template <class T, class W>
int launch(LogitsParams &p, int sms, int dev, cudaStream_t s) {
  constexpr int N = Piece<T>::N;
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &adjust_kernel<T, W>;
  // a word and a place in the list a token, a bit for four
  auto room = [](int per) { return per * kThreads * N * static_cast<int>(sizeof(W) + 2) + per * kThreads * N / 32; };
  if (!ready[dev].get(reinterpret_cast<const void *>(fn), kThreads, room(kMost))) return MK_ERR_CUDA;
  // the largest slices that give every SM two CTAs: a slice walks the whole history
  const int64_t elements = static_cast<int64_t>(p.vocab) + N - 1;
  auto slices = [&](int per) { return (elements - 1) / (per * kThreads * N) + 1; };
  p.per = kMost;
  while (p.per > 1 && slices(p.per) * p.n < 2 * sms) p.per /= 2;
  const int64_t ctas = slices(p.per) * p.n;
  if (ctas > INT32_MAX) return MK_ERR_UNSUPPORTED;
  p.slices = static_cast<int>(slices(p.per));
  return mkw::launch_after(fn, dim3(static_cast<unsigned>(ctas)), kThreads, room(p.per), s, p);
}

}  // namespace mklogits

using namespace mklogits;

extern "C" int mk_adjust_logits(const mk_logits_args *a, mk_stream stream) {
  if (!a || a->n < 0 || a->vocab < 0 || a->columns < 0 || a->biases < 0 || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->x_row < 0 ||
      a->out_row < 0 || a->tokens_row < 0 || a->ids_row < 0 || a->bias_row < 0 || a->mask_row < 0)
    return MK_ERR_INVALID_ARG;
  if (a->n == 0 || a->vocab == 0) return MK_OK;
  const uintptr_t es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->x || !a->out || reinterpret_cast<uintptr_t>(a->x) % es || reinterpret_cast<uintptr_t>(a->out) % es || (a->columns > 0 && !a->tokens) ||
      (a->biases > 0 && (!a->bias_ids || !a->bias)))
    return MK_ERR_INVALID_ARG;
  constexpr int kMostOf = INT32_MAX - 65536;               // (a CTA's steps over them, and its tokens beside them, stay within 32 bits)
  if (a->vocab > kMostOf || a->columns > kMostOf || a->biases > kMostOf) return MK_ERR_UNSUPPORTED;
  int dev = 0;
  const int sms = mkv::sm_count(&dev);
  if (sms < 0) return MK_ERR_CUDA;
  LogitsParams p = {};
  p.x = a->x, p.out = a->out;
  p.tokens = a->tokens, p.lengths = a->lengths, p.prompts = a->prompts, p.bias_ids = a->bias_ids;
  p.repetition = a->repetition, p.presence = a->presence, p.frequency = a->frequency, p.bias = a->bias;
  p.mask = reinterpret_cast<const uint32_t *>(a->mask);
  p.x_row = a->x_row, p.out_row = a->out_row, p.tokens_row = a->tokens_row, p.ids_row = a->ids_row, p.bias_row = a->bias_row;
  p.mask_row = a->mask_row;
  p.n = a->n, p.vocab = a->vocab, p.columns = a->columns, p.biases = a->biases;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool narrow = p.columns <= static_cast<int>(Word<uint16_t>::kCount);
  if (a->dtype == MK_F32) return narrow ? launch<float, uint16_t>(p, sms, dev, s) : launch<float, uint32_t>(p, sms, dev, s);
  return narrow ? launch<__nv_bfloat16, uint16_t>(p, sms, dev, s) : launch<__nv_bfloat16, uint32_t>(p, sms, dev, s);
}
