// Matrix-vector products with 4-bit weights (mk_matvec_q4): the kernel and its launch for one type of x.
//
// y[m][n] = sum_k x[m][k] scale[n][k / group] (code[n][k] - zero[n][k / group])
//
// Bound by the weights' bytes: N K / 2 plus the scales.  A warp takes 16 weight
// rows (32 where there are enough rows for every warp) as the rows of 16x8x16 matrix
// products and the x rows as their columns, 8 a tile.  A code minus its
// zero is a small whole number, exact in bf16.  A bf16 value of x is one term of a
// product, an fp32 value three of 8 bits, all of it; so what an element is worth does
// not depend on its neighbours.  (fp16 terms after a power of two a row took fewer
// instructions, but what is below 2^-31 of its row's largest lost bits and below 2^-40
// all, whatever the largest one's weight.)  An x row is still multiplied by the power of two
// that brings its largest finite value to 2^32 .. 2^33 (undone at the end), so that
// fp32's largest values stay finite in the sums; only an element below 2^-141 of its row's
// largest loses bits by it.  Products are summed in fp32 over a block's part of one
// group, multiplied by the group's scale and added to the row's sum in fp32.
//
// A warp's block is 128 elements of k of its rows, 64 bytes a row, which it copies
// ahead through its own ring of shared memory; registers as the
// place of what is on its way made the loop a copy per slot, and fetching its
// instructions took as long as the loop.  Where an element of k sits in a matrix
// product is free as long as both operands agree: lane t of a quad takes, of each
// row, four 32-bit words of 8 codes, 16 bytes in a row where one group covers the
// block, 8 bytes of each of two groups of 64, 4 of each of four groups of 32, so
// that a product never mixes two groups.  The x columns are staged in shared memory
// with each 8 elements in the order 0 4 1 5 2 6 3 7: codes j and j + 4 of a word are
// taken out together, as the low four mantissa bits of the bf16 number 128, less
// 128 + zero (a published way to make floats of small integers: the mantissa's last
// places of a number whose unit is 1).
//
// One persistent CTA of 16 warps an SM, so that x is staged once an SM (for 8 rows
// that is a third of the work of a 1.7B-shaped gate and up projection).  The rows'
// tiles are dealt out to its warps; 2 to 16 of them share a tile's k where that
// deals the blocks out more evenly, their sums added in order.  Where x is large
// beside the weights, reading and staging all of it in every SM is most of the
// time: there clusters of four CTAs take a quarter of k each, and add the sums of
// their tiles in order through their shared memory.
//
// Measured (graph replays, weights that stay in the L2 but for the first): 1 x 151936 x 1024, groups of 128 (80 MB) 18.8 us,
// 4.3 TB/s: instructions beside bytes (17.4 with fp16 terms); 8 x 12288 x 2048, groups of 32 with zeros, bf16 x, 11.0 us
// (10.7) and 3 x 2048 x 6144, groups of 64, 7.9 us (7.5): instructions and the staging of x; 1 x 4096 x 1024 4.1 us: latency.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_mma.cuh"
#include "mk_q4.h"

namespace mkq {

constexpr int kWarps = 16, kThreads = 32 * kWarps, kBlock = 128;
constexpr int kRing = 4096;            // bytes of codes a warp has room for: 4 blocks of 16 rows (twice as many measured slower)
constexpr int kMaxSmem = 225 * 1024;   // dynamic shared memory of a CTA
constexpr int kMaxInbox = 32768;       // of a cluster's CTA, for the tiles that it joins
constexpr int red_bytes(int parts) { return kWarps * parts * 512; }   // sums of the warps

// G: 32, 64, or 128 for every multiple of it
template <int G>
struct Layout {
  static constexpr int groups = kBlock / G;             // of a block
  // Pitch of the staged columns beyond a multiple of 128 bytes: with it the 8 lanes of a shared-memory phase (two
  // columns, the four lanes of a quad) meet 8 different 16-byte banks.
  static constexpr int pad = G == 128 ? 32 : G == 64 ? 16 : 64;
  // the 8 elements of k, within a block, of word w of lane t, and where a column has them
  static __device__ __forceinline__ int eighth(int t, int w) {
    return G == 128 ? 4 * t + w : G == 64 ? 8 * (w >> 1) + 2 * t + (w & 1) : 4 * w + t;
  }
  static __device__ __forceinline__ int staged(int b) { return G == 128 ? b ^ ((b >> 3) & 1) : b; }
};

// where chunk c (16 bytes, 32 codes) of row r of a block is in the ring: so that words of any of the three kinds of the
// rows of a phase meet different banks
__device__ __forceinline__ int chunk_at(int r, int c) { return r * 64 + ((c ^ ((r & 2) | ((r >> 2) & 1))) << 4); }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }


// eight elements of x as they are in memory, their values, and the largest magnitude's bits as a float's
template <class T>
struct Eight;
template <>
struct Eight<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float *p) { a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1]; }
  __device__ __forceinline__ void values(float *x) const {
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
  }
  __device__ __forceinline__ uint32_t largest() const {
    constexpr uint32_t M = 0x7fffffffu;
    return max(max(max(a.x & M, a.y & M), max(a.z & M, a.w & M)), max(max(b.x & M, b.y & M), max(b.z & M, b.w & M)));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void values(float *x) const {
    const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t largest() const {
    constexpr uint32_t M = 0x7fff7fffu;
    const uint32_t x = __vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M));
    return max(x << 16, x & 0xffff0000u);
  }
};

template <class T>
constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// the low four bits of each half of x as the last mantissa bits of 128 in bf16: one operation
__device__ __forceinline__ uint32_t take_codes(uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(0x000f000fu), "r"(0x43004300u));
  return r;
}

// Which x row and term column `col` of tile c is, and which x rows' sums a lane has in the end.
// One term: column by column.  Three: the terms of an x row are in columns of one lane (of columns 2t and 2t + 1 of every
// tile), which adds them up: two x rows a lane for every three tiles; one for two; with a single tile two lanes share one.
template <class T, int NT>
struct Columns {
  static constexpr int rows = 8 * NT, parts = NT;         // x rows; 16-byte parts of a lane's sums
  static __device__ __forceinline__ int row(int c, int col) { return 8 * c + col; }
  static __device__ __forceinline__ int term(int, int) { return 0; }
  static __device__ __forceinline__ int row_of_part(int t, int o, int j) { return 8 * o + 2 * t + j; }   // -1: none
  static __device__ __forceinline__ float4 part(const float (&s)[NT][4], int o) { return make_float4(s[o][0], s[o][1], s[o][2], s[o][3]); }
};
template <int NT>
struct Columns<float, NT> {
  static_assert(NT == 1 || NT == 2 || NT % 3 == 0);
  static constexpr int rows = NT == 1 ? 2 : NT == 2 ? 4 : NT / 3 * 8, parts = NT < 3 ? 1 : NT / 3;
  static __device__ __forceinline__ int row(int c, int col) { return NT == 1 ? col / 4 : (2 * c + (col & 1)) / 3 * 4 + col / 2; }
  static __device__ __forceinline__ int term(int c, int col) { return NT == 1 ? col % 4 : (2 * c + (col & 1)) % 3; }   // 3: none
  static __device__ __forceinline__ int row_of_part(int t, int o, int j) {
    return NT == 1 ? (j || t % 2 ? -1 : t / 2) : NT == 2 ? (j ? -1 : t) : (2 * o + j) * 4 + t;
  }
  // the least term first
  static __device__ __forceinline__ float4 part(const float (&s)[NT][4], int o) {
    if constexpr (NT == 1) {
      const float a = __shfl_xor_sync(0xffffffffu, s[0][0], 1), b = __shfl_xor_sync(0xffffffffu, s[0][2], 1);
      return make_float4(a + s[0][1] + s[0][0], 0.f, b + s[0][3] + s[0][2], 0.f);
    } else {
      auto sum = [&](int j, int h) {
        const int f = 3 * (2 * o + j);                    // terms f, f + 1, f + 2 of the lane's columns
        return s[(f + 2) / 2][2 * h + f % 2] + s[(f + 1) / 2][2 * h + (f + 1) % 2] + s[f / 2][2 * h + f % 2];
      };
      return NT == 2 ? make_float4(sum(0, 0), 0.f, sum(0, 1), 0.f) : make_float4(sum(0, 0), sum(1, 0), sum(0, 1), sum(1, 1));
    }
  }
};

// C: CTAs of a cluster, which have a slice of k each
template <class T, int NT, int RT, int G, bool ZEROS, int C>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(const __grid_constant__ Q4Params p) {
  using L = Layout<G>;
  using X = Columns<T, NT>;
  constexpr int TERMS = kTerms<T>, GB = L::groups, PARTS = RT * X::parts;
  constexpr int ROWS = 16 * RT, STAGE = ROWS * 64, STAGES = kRing / STAGE;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t s_max[X::rows];
  __shared__ float s_to[X::rows], s_back[X::rows];               // the powers of two that x rows are multiplied by, and their inverses
  mkw::follow_previous_kernel();
  if (C > 1) mkw::cluster_arrive();                        // (waited for before the others' memory is written)
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % C, cluster = blockIdx.x / C, clusters = gridDim.x / C;
  const int wn = w / p.wk, wk = w % p.wk, per_cta = kWarps / p.wk;
  const int m0 = blockIdx.y * p.pass_rows, mr = min(p.pass_rows, p.m - m0);
  unsigned char *ring = smem + w * kRing, *xs = smem + kWarps * kRing;
  float *red = reinterpret_cast<float *>(xs + p.pass_rows * TERMS * p.pitch) + wn * p.wk * PARTS * 128;   // sums of the warps of this tile

  // the CTA's blocks of k, this warp's slice of them, its tiles
  const int c0 = p.blocks * rank / C, cb = p.blocks * (rank + 1) / C - c0;
  const int b0 = cb * wk / p.wk, nb = cb * (wk + 1) / p.wk - b0;
  const int tile0 = cluster * per_cta + wn, step = clusters * per_cta;
  const int rounds = tile0 < p.tiles ? (p.tiles - tile0 + step - 1) / step : 0;
  const int items = rounds * nb;

  // ---- x, and the largest value of every row.  The weights are asked for when x is there: before, its answer waits
  // behind theirs ------------------------------------------------------------------------------------------------
  const T *x = static_cast<const T *>(p.x) + m0 * p.x_row + c0 * kBlock;
  const int eighths = p.eighths.value, last = C == 1 ? p.k / 8 : min(p.k / 8 - c0 * (kBlock / 8), cb * (kBlock / 8)), all = mr * eighths;
  auto read = [&](int i, Eight<T> &e) {                    // eighth i % eighths of row i / eighths, if it is there
    const int r = p.eighths.quotient(i), b = i - r * eighths;
    if (b < last) e.load(x + r * p.x_row + b * 8);
    return b < last ? r : -1;
  };
  if (tid < X::rows) s_max[tid] = 0;
  __syncthreads();
  constexpr int AT_ONCE = 4;
#pragma unroll 1
  for (int i0 = tid; i0 - tid < all; i0 += AT_ONCE * kThreads) {
    Eight<T> e[AT_ONCE];
    int row[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) row[j] = i0 + j * kThreads < all ? read(i0 + j * kThreads, e[j]) : -1;
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (i0 - tid + j * kThreads >= all) break;
      const uint32_t mx = row[j] >= 0 ? e[j].largest() : 0u;
      if (__all_sync(0xffffffffu, row[j] == __shfl_sync(0xffffffffu, row[j], 0))) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0 && row[j] >= 0) atomicMax(&s_max[row[j]], top);
      } else if (row[j] >= 0) {                            // eighths of several rows
        atomicMax(&s_max[row[j]], mx);
      }
    }
  }

  // ---- codes: this lane copies chunk t of rows g, g + 8, ... of every block ----------------------------------
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  int c_tile = tile0, c_blk = 0, c_left = items, c_stage = 0;    // the copies' place
  const unsigned char *code_at[2 * RT];
  auto copy = [&]() {
    if (c_left > 0) {
      --c_left;
      if (c_blk == 0) {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          const int64_t row = min(c_tile * ROWS + 8 * r + g, p.n - 1);             // rows past the last are read as it and not stored
          code_at[r] = p.codes + row * (p.k / 2) + (c0 + b0) * (kBlock / 2) + t * 16;
        }
      }
      const bool there = G == 128 || (c0 + b0 + c_blk) * kBlock + t * 32 < p.k;
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        const uint32_t to = ring_at + c_stage * STAGE + chunk_at(8 * r + g, t);
        if (G == 128) mkw::cp_async16(to, code_at[r]);
        else mkw::cp_async16(to, there ? code_at[r] : p.codes, there);
        code_at[r] += kBlock / 2;
      }
      if (++c_blk == nb) c_blk = 0, c_tile += step;
      if (++c_stage == STAGES) c_stage = 0;
    }
    mkw::cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) copy();

  // ---- scales and zeros of a block, two blocks ahead: lane l has those of row l % ROWS, at once where they lie on a
  // boundary of their size ------------------------------------------------------------------------------------------
  struct Scales {
    uint32_t pair[G == 32 ? 2 : 1], zeros;               // bf16 of two groups, a byte a group
  };
  int s_tile = tile0, s_blk = 0, s_left = items;
  int64_t group_at = 0;
  auto look_up = [&]() {
    Scales s;
    if (s_left > 0) {
      --s_left;
      if (s_blk == 0) group_at = static_cast<int64_t>(min(s_tile * ROWS + lane % ROWS, p.n - 1)) * p.groups;
      const int blk = c0 + b0 + s_blk;
      const int64_t at = group_at + (G == 128 ? p.blocks_a_group.quotient(blk) : blk * GB);
      const uint16_t *sc = p.scales + at;
      const uint8_t *z = p.zeros + at;
      if (G == 128) {
        s.pair[0] = *sc;
        if (ZEROS) s.zeros = *z;
      } else if (p.vec && (blk + 1) * GB <= p.groups) {
        if constexpr (G == 64) {
          s.pair[0] = *reinterpret_cast<const uint32_t *>(sc);
          if (ZEROS) s.zeros = *reinterpret_cast<const uint16_t *>(z);
        } else if constexpr (G == 32) {
          const uint2 v = *reinterpret_cast<const uint2 *>(sc);
          s.pair[0] = v.x, s.pair[1] = v.y;
          if (ZEROS) s.zeros = *reinterpret_cast<const uint32_t *>(z);
        }
      } else {
        s.zeros = 0;
#pragma unroll
        for (int i = 0; i < GB; ++i) {
          const bool there = blk * GB + i < p.groups;    // a scale of 0 past the end
          const uint32_t v = there ? sc[i] : 0u;
          s.pair[i / 2] = i % 2 ? s.pair[i / 2] | (v << 16) : v;
          if (ZEROS && there) s.zeros |= static_cast<uint32_t>(z[i]) << (8 * i);
        }
      }
      if (++s_blk == nb) s_blk = 0, s_tile += step;
    }
    return s;
  };
  Scales next = look_up(), after = look_up();

  // ---- the x rows as columns of bf16 terms, zeros past k ----------------------------------------------------
  __syncthreads();
  for (int r = w; r < mr; r += kWarps) {
    uint32_t mx = s_max[r];
    if (mx >= 0x7f800000u) {                               // infinities (or NaN) in the row: its largest finite value
      mx = 0;
      for (int b = lane; b < last; b += 32) {
        Eight<T> e;
        float v[8];
        e.load(x + r * p.x_row + b * 8);
        e.values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
          if (a < 0x7f800000u) mx = max(mx, a);
        }
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
    }
    const int e = mx ? min(126, 32 - ilogbf(__uint_as_float(mx))) : 0;
    if (lane == 0) s_to[r] = ldexpf(1.f, e), s_back[r] = ldexpf(1.f, -e);
  }
  __syncthreads();
  // (read again, from the L1, in a loop that is not unrolled: held in registers the code is four times as long, and
  // fetching it takes longer)
#pragma unroll 1
  for (int i = tid; i < all; i += kThreads) {
    const int r = p.eighths.quotient(i), b = i - r * eighths;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (b < last) {
      Eight<T> e;
      e.load(x + r * p.x_row + b * 8);
      e.values(v);
    }
    const float f = s_to[r];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    unsigned char *to = xs + r * TERMS * p.pitch + L::staged(b) * 16;
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
      uint4 o;
      o.x = mkw::take_input_term(mkw::BF16Op{}, v[0], v[4]);
      o.y = mkw::take_input_term(mkw::BF16Op{}, v[1], v[5]);
      o.z = mkw::take_input_term(mkw::BF16Op{}, v[2], v[6]);
      o.w = mkw::take_input_term(mkw::BF16Op{}, v[3], v[7]);
      *reinterpret_cast<uint4 *>(to + u * p.pitch) = o;
    }
  }
  __syncthreads();

  float sum[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) sum[r][c][0] = sum[r][c][1] = sum[r][c][2] = sum[r][c][3] = 0.f;
  int tile = tile0, blk = 0, at_stage = 0;
  const unsigned char *column[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int m = X::row(c, g), u = X::term(c, g);
    column[c] = xs + (m < mr && u < TERMS ? m * TERMS + u : 0) * p.pitch;   // a column that is none computes what nobody stores
  }

  auto compute = [&](const Scales &sc) {
    const unsigned char *codes = ring + at_stage * STAGE;
    uint32_t v[RT][2][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * r + 8 * h + g;
        if constexpr (G == 128) {
          const uint4 a = *reinterpret_cast<const uint4 *>(codes + chunk_at(row, t));
          v[r][h][0] = a.x, v[r][h][1] = a.y, v[r][h][2] = a.z, v[r][h][3] = a.w;
        } else if constexpr (G == 64) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 a = *reinterpret_cast<const uint2 *>(codes + chunk_at(row, 2 * j + (t >> 1)) + (t & 1) * 8);
            v[r][h][2 * j] = a.x, v[r][h][2 * j + 1] = a.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[r][h][j] = *reinterpret_cast<const uint32_t *>(codes + chunk_at(row, j) + t * 4);
        }
      }
    const int e0 = (b0 + blk) * (kBlock / 8);
    float acc[RT][NT][4];
    uint32_t pair[RT][2], zeros[RT][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // words; a group ends with every (4 / GB)th
      uint4 b[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) b[c] = *reinterpret_cast<const uint4 *>(column[c] + e0 * 16 + L::staged(L::eighth(t, i)) * 16);
      const int grp = i * GB / 4;
      const bool fresh = i % (4 / GB) == 0, done = (i + 1) % (4 / GB) == 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i == 0 && ZEROS) zeros[r][h] = __shfl_sync(0xffffffffu, sc.zeros, 16 * r + 8 * h + g) & 0x0f0f0f0fu;
          if (done && grp % 2 == 0) pair[r][h] = __shfl_sync(0xffffffffu, sc.pair[grp / 2], 16 * r + 8 * h + g);
          // -(128 + zero), twice
          const uint32_t less = ZEROS ? __byte_perm(zeros[r][h], 0, 0x4040 | grp * 0x0101) | 0xc300c300u : 0xc308c308u;
          const uint32_t w0 = v[r][h][i];
          a[0][h] = add_bf16x2(take_codes(w0), less);
          a[0][2 + h] = add_bf16x2(take_codes(w0 >> 4), less);
          a[1][h] = add_bf16x2(take_codes(w0 >> 8), less);
          a[1][2 + h] = add_bf16x2(take_codes(w0 >> 12), less);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (fresh) mkw::mma_zero(mkw::BF16Op{}, acc[r][c], a[0], b[c].x, b[c].y);
          else mkw::mma(mkw::BF16Op{}, acc[r][c], a[0], b[c].x, b[c].y);
          mkw::mma(mkw::BF16Op{}, acc[r][c], a[1], b[c].z, b[c].w);
        }
        if (done) {
          float s[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) s[h] = __uint_as_float(grp % 2 ? pair[r][h] & 0xffff0000u : pair[r][h] << 16);
#pragma unroll
          for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[r][c][j] += s[j / 2] * acc[r][c][j];
        }
      }
    }
  };
  auto store = [&](int row, int m, float y) {
    if (row >= p.n || m >= mr) return;
    if (p.residual) y += to_float(static_cast<const T *>(p.residual)[(m0 + m) * p.residual_row + row]);
    put(static_cast<T *>(p.y) + (m0 + m) * p.y_row + row, y);
  };
  // a part of a tile's sums: a lane has rows g and g + 8 of one or two x rows
  auto store_part = [&](int row, int o, float4 y) {
    const int ma = X::row_of_part(t, o, 0), mb = X::row_of_part(t, o, 1);
    if (ma >= 0) {
      store(row, ma, y.x);
      store(row + 8, ma, y.z);
    }
    if (mb >= 0) {
      store(row, mb, y.y);
      store(row + 8, mb, y.w);
    }
  };
  // A cluster's CTAs have a slice of k each of the same tiles: what each has of the jth of a CTA's tiles goes to the inbox of
  // CTA j % C, in place j / C.
  float4 *inbox = reinterpret_cast<float4 *>(smem + p.inbox);   // [place][CTA][PARTS][32 lanes]
  int round = 0;
  auto finish = [&]() {
    float4 y[PARTS];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int o = 0; o < X::parts; ++o) y[r * X::parts + o] = X::part(sum[r], o);
#pragma unroll
      for (int c = 0; c < NT; ++c) sum[r][c][0] = sum[r][c][1] = sum[r][c][2] = sum[r][c][3] = 0.f;
    }
    if (p.wk > 1) {
      // over the warps that share the tile, each adding up its part of the lanes' values
      float4 *mine = reinterpret_cast<float4 *>(red) + lane;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) mine[(i * p.wk + wk) * 32] = y[i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + wn), "r"(32 * p.wk) : "memory");
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
        if (i % p.wk == wk) {
          y[i] = mine[i * p.wk * 32];
          for (int j = 1; j < p.wk; ++j) {
            const float4 z = mine[(i * p.wk + j) * 32];
            y[i].x += z.x, y[i].y += z.y, y[i].z += z.z, y[i].w += z.w;
          }
        }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + wn), "r"(32 * p.wk) : "memory");
    }
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      if (p.wk == 1 || i % p.wk == wk) {
        // undo the powers of two of the x rows
        const int o = i % X::parts, ma = X::row_of_part(t, o, 0), mb = X::row_of_part(t, o, 1);
        const float fa = ma >= 0 && ma < mr ? s_back[ma] : 0.f, fb = mb >= 0 && mb < mr ? s_back[mb] : 0.f;
        y[i].x *= fa, y[i].y *= fb, y[i].z *= fa, y[i].w *= fb;
        if constexpr (C == 1) {
          store_part(tile * ROWS + i / X::parts * 16 + g, o, y[i]);
        } else {
          const int j = round * per_cta + wn;
          const uint32_t to = mkw::remote(inbox + ((j / C * C + rank) * PARTS + i) * 32 + lane, j % C);
          mkw::store_remote(to, y[i].x), mkw::store_remote(to + 4, y[i].y), mkw::store_remote(to + 8, y[i].z), mkw::store_remote(to + 12, y[i].w);
        }
      }
    tile += step;
    ++round;
  };

  if (C > 1) mkw::cluster_wait();
  if (nb == 0)                                             // fewer blocks than warps: this one only joins in
    for (int i = 0; i < rounds; ++i) finish();
#pragma unroll 1
  for (int i = 0; i < items; ++i) {
    copy();
    const Scales now = next;
    next = after;
    after = look_up();
    mkw::cp_async_wait<STAGES - 1>();
    __syncwarp();
    compute(now);
    __syncwarp();                                          // every lane has read the stage
    if (++at_stage == STAGES) at_stage = 0;
    if (++blk == nb) {
      blk = 0;
      finish();
    }
  }
  mkw::cp_async_wait<0>();
  if constexpr (C == 1) return;
  mkw::cluster_arrive();
  mkw::cluster_wait();
  // the slices' sums, in order, by a warp each 16 rows and 8 columns
#pragma unroll 1
  for (int i = w;; i += kWarps) {
    const int part = i % PARTS, place = i / PARTS, j = place * C + rank, at = cluster * per_cta + j % per_cta + j / per_cta * step;
    if (j / per_cta * step + cluster * per_cta >= p.tiles) break;
    if (at >= p.tiles) continue;
    float4 y = inbox[(place * C * PARTS + part) * 32 + lane];
#pragma unroll 1
    for (int c = 1; c < C; ++c) {
      const float4 z = inbox[((place * C + c) * PARTS + part) * 32 + lane];
      y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
    }
    store_part(at * ROWS + part / X::parts * 16 + g, part % X::parts, y);
  }
}

// bytes from staged column to column, of a CTA's blocks of k
template <int G>
int pitch_of(int blocks) { return blocks * kBlock * 2 + Layout<G>::pad; }

// a launch that cannot be: clusters that do not fit, more tiles than an inbox holds, no room for one x row
constexpr int kRefused = 1;

// How a launch's CTAs (or clusters of c, `units` of them at once) share the tiles, and what shared memory leaves room for.
struct Plan {
  int wk, want, red, inbox;    // warps a tile, CTAs or clusters, bytes of the warps' sums and of the inbox
  int rows;                    // x rows of a pass: as many as the columns hold and there is room for; 0: none, or no inbox
};
template <class T, int NT, int RT>
Plan plan_of(const Q4Params &p, int tiles, int blocks, int pitch, int c, int units) {
  constexpr int PARTS = RT * Columns<T, NT>::parts;
  Plan r = {};
  // the sharing of k that leaves the busiest warp the fewest blocks, fewer warps a tile where that is equal
  int64_t best = 0;
  for (int wk = 1; wk <= kWarps; wk *= 2) {
    const int64_t per_round = static_cast<int64_t>(units) * (kWarps / wk), rounds = (tiles + per_round - 1) / per_round;
    const int64_t cost = rounds * ((blocks + wk - 1) / wk);
    if (wk == 1 || cost < best) best = cost, r.wk = wk;
  }
  const int per_cta = kWarps / r.wk;
  r.want = std::min((tiles + per_cta - 1) / per_cta, units);
  r.red = r.wk > 1 ? red_bytes(PARTS) : 0;
  const int64_t rounds = (tiles + static_cast<int64_t>(r.want) * per_cta - 1) / (static_cast<int64_t>(r.want) * per_cta);
  const int64_t inbox = c > 1 ? (rounds * per_cta + c - 1) / c * c * PARTS * 512 : 0;
  if (inbox > kMaxInbox) return r;
  r.inbox = static_cast<int>(inbox);
  r.rows = std::min({p.m, Columns<T, NT>::rows, (kMaxSmem - kWarps * kRing - r.red - r.inbox) / pitch / kTerms<T>});
  return r;
}

template <class T, int NT, int RT, int G, bool ZEROS, int C>
int launch_as(Q4Params p, int sms, int dev, cudaStream_t s) {
  static_assert(C == 1 || C == 4);
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &matvec_kernel<T, NT, RT, G, ZEROS, C>;
  mkw::Ready &r = ready[dev];
  if (!r.get(reinterpret_cast<const void *>(fn), kThreads, kMaxSmem)) return MK_ERR_CUDA;
  p.tiles = (p.n + 16 * RT - 1) / (16 * RT);
  constexpr int per = kBlock / G;
  p.vec = p.groups % per == 0 && reinterpret_cast<uintptr_t>(p.scales) % (2 * per) == 0 &&
          reinterpret_cast<uintptr_t>(p.zeros) % per == 0;
  const int clusters = C == 1 ? sms : r.clusters[1];
  if (clusters < 1) return kRefused;
  const int blocks = (p.blocks + C - 1) / C;   // of a CTA
  p.pitch = pitch_of<G>(blocks);
  p.eighths.set(blocks * (kBlock / 8));
  const Plan plan = plan_of<T, NT, RT>(p, p.tiles, blocks, p.pitch, C, clusters);
  if (plan.rows < 1) return kRefused;
  p.wk = plan.wk, p.pass_rows = plan.rows;
  p.inbox = kWarps * kRing + plan.red + p.pass_rows * kTerms<T> * p.pitch;
  const int passes = (p.m - 1) / p.pass_rows + 1;
  if (passes > 65535) return MK_ERR_UNSUPPORTED;
  return mkw::launch_after(fn, dim3(plan.want * C, passes), kThreads, p.inbox + plan.inbox, s, p, C);
}

template <class T, int NT, int RT, int G, bool ZEROS>
int launch(const Q4Params &p, int sms, int dev, cudaStream_t s) {
  if constexpr (RT == 1) {
    if (p.cluster > 1) return launch_as<T, NT, RT, G, ZEROS, 4>(p, sms, dev, s);
  }
  return launch_as<T, NT, RT, G, ZEROS, 1>(p, sms, dev, s);
}

template <class T, int NT, int RT, bool ZEROS>
int by_group(Q4Params &p, int group, int sms, int dev, cudaStream_t s) {
  if (group == 32) return launch<T, NT, RT, 32, ZEROS>(p, sms, dev, s);
  if (group == 64) return launch<T, NT, RT, 64, ZEROS>(p, sms, dev, s);
  p.blocks_a_group.set(group / kBlock);
  return launch<T, NT, RT, 128, ZEROS>(p, sms, dev, s);
}

// passes over the weights with NT column tiles, 16 RT rows a tile and clusters of c CTAs (if all SMs can be in one); 0: not
// one x row fits
template <class T, int NT, int RT = 1>
int passes_of(const Q4Params &p, int c, int sms) {
  const int blocks = (p.blocks + c - 1) / c;
  const int rows = plan_of<T, NT, RT>(p, (p.n + 16 * RT - 1) / (16 * RT), blocks, pitch_of<32>(blocks), c, std::max(1, sms / c)).rows;
  return rows < 1 ? 0 : (p.m - 1) / rows + 1;
}

template <class T, bool ZEROS>
int by_columns(Q4Params &p, int group, int sms, int dev, cudaStream_t s) {
  // the fewest passes, and of these the fewest columns
  constexpr int A = std::is_same<T, float>::value ? 3 : 4, B = std::is_same<T, float>::value ? 6 : 4;
  const int one = passes_of<T, 1>(p, p.cluster, sms);
  if (one == 1) {
    // 32 rows a tile, whose matrix products share what is read of x, where every warp has one of them
    if (p.cluster == 1 && p.n / 32 >= sms * kWarps && passes_of<T, 1, 2>(p, 1, sms) == 1) return by_group<T, 1, 2, ZEROS>(p, group, sms, dev, s);
    return by_group<T, 1, 1, ZEROS>(p, group, sms, dev, s);
  }
  const int two = passes_of<T, 2>(p, p.cluster, sms), some = passes_of<T, A>(p, p.cluster, sms), most = passes_of<T, B>(p, p.cluster, sms);
  const int fewest = std::min({one ? one : INT32_MAX, two ? two : INT32_MAX, some ? some : INT32_MAX, most ? most : INT32_MAX});
  if (fewest == INT32_MAX) return kRefused;
  if (one == fewest) return by_group<T, 1, 1, ZEROS>(p, group, sms, dev, s);
  if (two == fewest) return by_group<T, 2, 1, ZEROS>(p, group, sms, dev, s);
  if (some == fewest) return by_group<T, A, 1, ZEROS>(p, group, sms, dev, s);
  return by_group<T, B, 1, ZEROS>(p, group, sms, dev, s);
}

template <class T, bool ZEROS>
int by_rows(Q4Params &p, int group, int sms, int dev, cudaStream_t s) {
  p.blocks = (p.k + kBlock - 1) / kBlock;
  // Clusters of 4 CTAs with a quarter of k each, where what is staged of x is 48 KB and as much as a CTA's codes.  (In clusters
  // and with all of x in every CTA: 8 x 2048 x 6144 in bf16 8.2 and 11.9 us, 16 x 4096 x 4096 10.8 and 15.5, 8 x 4096 x 6144,
  // 1.2 times the codes, 10.4 and 13.8, 2 x 1024 x 16384 in fp32 8.6 and 11.7, 3 x 4096 x 6144, 1.3 times, 10.4 and 11.8, 12 x
  // 12288 x 2048 18.7 and 21.6; but 2 x 4096 x 6144, 0.9 times, 9.4 and 9.2, 1 x 2048 x 8192, 0.9 times, 7.7 both ways, 16 x
  // 12288 x 2048 in bf16, 0.8 times, 14.4 and 12.8, 8 x 12288 x 2048, 32 KB, 12.3 and 11.0: a cluster's launch alone costs
  // 1 us.  Clusters of 2 or 8 were slower where clusters paid.)
  const int64_t staged = static_cast<int64_t>(p.m) * p.k * kTerms<T> * 2, codes = static_cast<int64_t>(p.n) * p.k / 2 / sms;
  const bool fits = (kMaxSmem - kWarps * kRing - red_bytes(Columns<T, 1>::parts)) / pitch_of<32>(p.blocks) >= kTerms<T>;   // an x row in a CTA
  p.cluster = !fits || (staged >= 49152 && staged >= codes) ? 4 : 1;
  if (fits) {
    int rc = by_columns<T, ZEROS>(p, group, sms, dev, s);
    if (rc == kRefused && p.cluster > 1) {
      p.cluster = 1;
      rc = by_columns<T, ZEROS>(p, group, sms, dev, s);
    }
    return rc == kRefused ? MK_ERR_UNSUPPORTED : rc;
  }
  // x rows of which not one fits in a CTA (fp32, k above 25 thousand): always in clusters, the weights' rows in launches
  // of as many as their inboxes hold
  constexpr int kRows = 16384;
  for (int64_t n0 = 0; n0 < p.n; n0 += kRows) {
    Q4Params q = p;
    q.n = static_cast<int>(std::min<int64_t>(kRows, p.n - n0));
    q.codes += n0 * (p.k / 2);
    q.scales += n0 * p.groups;
    if (q.zeros) q.zeros += n0 * p.groups;
    q.y = static_cast<T *>(q.y) + n0;
    if (q.residual) q.residual = static_cast<const T *>(q.residual) + n0;
    const int rc = by_columns<T, ZEROS>(q, group, sms, dev, s);
    if (rc != MK_OK) return rc == kRefused ? MK_ERR_UNSUPPORTED : rc;
  }
  return MK_OK;
}

template <class T>
int run(Q4Params &p, int group, int sms, int dev, cudaStream_t s) {
  return p.zeros ? by_rows<T, true>(p, group, sms, dev, s) : by_rows<T, false>(p, group, sms, dev, s);
}

}  // namespace mkq
