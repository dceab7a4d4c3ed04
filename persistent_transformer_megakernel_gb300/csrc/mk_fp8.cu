// Products in 8-bit floating point with block scales (mk_quantize_fp8, mk_matmul_fp8).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_mma.cuh"
#include "mk_paged.h"
#include "mk_tc.cuh"
#include "mk_tmap.h"

namespace mkf8 {

using namespace mktc;

constexpr int kBlock = 128;

// ---------------------------------------------------------------------------
// Quantisation of rows: for each 128 of a row scale = largest / 448, code = x / scale rounded to e4m3.
//
// Bound by bytes: x read once, a byte an element and 4 a block written.  16 lanes have a block, 8 elements each, or (bf16)
// four blocks at a time, all asked for before the first is worked on.  The quotient is fp32's (a bf16 element over its scale is
// often half way between two codes, so that a last place decides): the product with the reciprocal, corrected by its
// remainder, which is the correctly rounded quotient if the reciprocal is (P. Markstein, Computation of elementary functions
// on the IBM RISC System/6000 processor, 1990), away from the ends of the exponents' range.
// ---------------------------------------------------------------------------

struct QuantParams {
  const void *x;
  uint8_t *codes;
  float *scales;
  int64_t x_row, codes_row, scales_row;
  int k;
  mkw::Divisor blocks;         // of a row
  int items;                   // blocks in all
};

constexpr int kQuantThreads = 256;

__device__ __forceinline__ void numbers8(const float4 (&w)[2], float (&x)[8]) {
  x[0] = w[0].x, x[1] = w[0].y, x[2] = w[0].z, x[3] = w[0].w, x[4] = w[1].x, x[5] = w[1].y, x[6] = w[1].z, x[7] = w[1].w;
}
__device__ __forceinline__ void numbers8(const uint4 (&w)[1], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float((&w[0].x)[i] << 16);
    x[2 * i + 1] = __uint_as_float((&w[0].x)[i] & 0xffff0000u);
  }
}

// U: blocks that 16 lanes have at a time
template <class T, int U>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const __grid_constant__ QuantParams p) {
  using Word = std::conditional_t<sizeof(T) == 4, float4, uint4>;
  constexpr int WORDS = sizeof(T) / 2;
  mkw::follow_previous_kernel();
  const int lane = threadIdx.x & 15, first = (static_cast<int>(blockIdx.x) * (kQuantThreads / 16) + (threadIdx.x >> 4)) * U;
  int row[U], b[U];
  bool there[U];
  Word w[U][WORDS];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    row[i] = p.blocks.quotient(first + i);
    b[i] = first + i - row[i] * static_cast<int>(p.blocks.value);
    there[i] = first + i < p.items && b[i] * kBlock + lane * 8 < p.k;      // (k is a multiple of 16: 8 elements are there or not)
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
      w[i][j] = Word{};
      if (there[i]) w[i][j] = __ldcs(reinterpret_cast<const Word *>(static_cast<const T *>(p.x) + row[i] * p.x_row + b[i] * kBlock + lane * 8) + j);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float x[8], top = 0.f;
    numbers8(w[i], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float scale = __fdiv_rn(top, 448.f);
    if (!(scale > 0.f)) scale = 1.f;
    float y[8];
    if (scale > 0x1p-60f && scale < 0x1p60f) {
      const float r = __frcp_rn(scale);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = x[e] * r;
        y[e] = fmaf(fmaf(-q, scale, x[e]), r, q);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], scale);
    }
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * e], y[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
    if (there[i]) *reinterpret_cast<uint2 *>(p.codes + row[i] * p.codes_row + b[i] * kBlock + lane * 8) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (first + i < p.items && lane == 0) p.scales[row[i] * p.scales_row + b[i]] = scale;
  }
}

// ---------------------------------------------------------------------------
// y[t][j] = sum_b xs[t][b] ws[j / 128][b] sum_{k in b} x[t][k] w[j][k]  (+ residual)
//
// A CTA has 128 rows of x and 128 rows of w.  The inner sums of a block of 128 are four tensor instructions into one of the
// accumulators in tensor memory (a row of x a lane, a row of w a column); eight warps take it out, multiply it by xs ws --
// one number for all of a thread's columns -- and add it to fp32 sums in registers while the next block is multiplied into
// others.  Warp 0 asks for x and w by TMA, warps 1 and 2 multiply, warp 3 brings the scales, warps 4-11 add up.
// Bound by no part alone (8192 x 12288 x 2048: 169 us, 2440 TFLOP/s, 500 clocks a block; with four stages 176): the tensor
// pipe is busy for 256 of those, reading its operands from shared memory takes as many (32 KB at 128 bytes a clock), as many
// bytes arrive there, and sums leave tensor memory and are added beside it.  Timed with parts left out: without the copies
// 163 us, without the additions 153, without both 129; what is left there are the hand-overs between warps.  So two blocks
// are handed over at a time, and two warps multiply in turn, one waiting while the other's instructions run (one warp, with
// four stages: 186 us).  Tiles of 256 columns hold fewer accumulators and spill (230 us and more).
// Pairs of CTAs that ask for shared tiles once (multicast) took as long (178 us for 177, with four stages): not kept.
// splits > 1 (few tiles): K is shared by the CTAs of a cluster, whose sums are added in order through their shared memory.
// ---------------------------------------------------------------------------

constexpr int kRows = 128;     // of x (the MMA's M)
constexpr int kColumns = 128;  // rows of w (its N)
constexpr int kHelpers = 4, kAddWarps = 8, kWarps = kHelpers + kAddWarps, kThreads = 32 * kWarps;
constexpr int kMmaWarps = 2;   // each a block in turn: the waits and commits of one pass while the other's products run
constexpr int kGroup = 4, kGroups = 4;   // scales travel in groups of four blocks, four of them at most on their way
constexpr uint32_t kXTile = kRows * 128;
constexpr long long kWaitNs = 2000000000LL;

struct MatmulParams {
  const float *x_scale, *w_scale;
  const void *residual;
  void *y;
  int32_t *status;
  int64_t x_scale_row, residual_row, y_row;
  int64_t residual_map_row, y_map_row;   // as a tensor map has them
  int m, n, kb;                // kb: blocks of K
  int tiles_m, tiles;          // tiles along m, in all
  int splits;                  // CTAs of a cluster that share a tile's K
  int x_rows;                  // rows that a copy of x brings: no more than there are (what else is in a tile is no row's)
  int wide_scales;             // rows of x's scales on 16 bytes
};

// numbers of a row of sums that a cluster's CTAs leave each other (16 bytes of eight rows are in different banks)
constexpr int kSplitRow = kColumns + 4;
constexpr uint32_t kStage = kXTile + kColumns * 128;
constexpr int kStages = 5;
constexpr int kTensorColumns = 512, kSums = kTensorColumns / (2 * kColumns);   // pairs of accumulators
constexpr int kCols = kColumns / 2;                        // of an adding warp
constexpr int kBoxRow = 128;                               // results leave (and the residual comes) in boxes of 32 rows and 128 bytes
constexpr uint32_t kResults = kStages * kStage;            // behind the stages: a box an adding warp
constexpr uint32_t kScales = kResults + kAddWarps * 32 * kBoxRow;              // [group][row][4] of x, [group][4] of w
constexpr uint32_t kControl = kScales + kGroups * (kRows + 1) * 16;
constexpr int kSmem = static_cast<int>(1024 + kControl + 512);
static_assert(kSmem <= 232448 && kRows * kSplitRow * 4 <= kResults, "shared memory");
static_assert(kColumns == kBlock, "a tile has one row of w's scales");

__device__ __forceinline__ void fail(int32_t *status) {
  if (status) atomicCAS(status, 0, MK_ERR_TIMEOUT);
}
__device__ __forceinline__ float4 load_remote4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
  return x;
}
// places 0 .. N - 1 in turn, and the parity of the round
template <int N>
struct Turn {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) i = 0, parity ^= 1u;
  }
};
// two fp32 sums and one factor: c += a f
__device__ __forceinline__ void add_scaled(unsigned long long &c, uint32_t a0, uint32_t a1, unsigned long long f) {
  unsigned long long a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "r"(a0), "r"(a1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(f));
}

// 16 bytes of a row of results: N numbers
template <class T>
struct Out;
template <>
struct Out<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void add(const uint4 &r, float *y) {
    y[0] += __uint_as_float(r.x), y[1] += __uint_as_float(r.y), y[2] += __uint_as_float(r.z), y[3] += __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 bits(const float *y) {
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
  }
};
template <>
struct Out<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void add(const uint4 &r, float *y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] += __uint_as_float((&r.x)[i] << 16);
      y[2 * i + 1] += __uint_as_float((&r.x)[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 bits(const float *y) {
    uint4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      (&w.x)[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return w;
  }
};

// TMA: rows of y and of the residual start and end on 16 bytes.  (Both ways in one kernel cost 8192 x 12288 x 2048 six microseconds.)
template <class T, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ty,
                  const __grid_constant__ CUtensorMap tr, const __grid_constant__ MatmulParams p) {
  constexpr int N = Out<T>::N, PIECE = kBoxRow / static_cast<int>(sizeof(T));   // numbers in 16 bytes and in a row of a box
  constexpr uint32_t kId = idesc_f32(kRows, kColumns);
  extern __shared__ unsigned char smraw[];
  mkw::follow_previous_kernel();
  unsigned char *sm = smraw + ((1024u - (smem_addr(smraw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + kControl), *empty = full + kStages, *tfull = empty + kStages, *tempty = tfull + kSums,
           *sfull = tempty + kSums, *sempty = sfull + kGroups, *rfull = sempty + kGroups;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(rfull + kAddWarps);
  float4 *scales = reinterpret_cast<float4 *>(sm + kScales);               // a group: kRows of x, one of w
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kSums; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], kAddWarps);
    for (int i = 0; i < kGroups; ++i) mbar_init(&sfull[i], 1), mbar_init(&sempty[i], kAddWarps);
    for (int i = 0; i < kAddWarps; ++i) mbar_init(&rfull[i], 1);
    fence_mbar_init();
    prefetch_tmap(&tw);
    prefetch_tmap(&tx);
  }
  if (warp == 1) tmem_alloc(tslot, kTensorColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);

  const int split = static_cast<int>(blockIdx.x) % p.splits, step = static_cast<int>(gridDim.x) / p.splits, first = static_cast<int>(blockIdx.x) / p.splits;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * split / p.splits), kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (split + 1) / p.splits);
  auto row_of = [&](int tile) { return tile % p.tiles_m * kRows; };
  auto column_of = [&](int tile) { return tile / p.tiles_m * kColumns; };

  if (warp < kHelpers) {
    if (warp == 0) {
      Turn<kStages> at;
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int t0 = row_of(tile), j0 = column_of(tile);
        for (int kb = kb0; kb < kb1; ++kb, ++it, at.next()) {
          const int s = at.i;
          if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait(&empty[s], at.parity ^ 1u, kWaitNs))) {
            if (lane == 0) fail(p.status);
            ok = false;
            break;
          }
          unsigned char *to = sm + s * kStage;
          if (elect_one()) {
            mbar_expect_tx(&full[s], p.x_rows * 128 + kColumns * 128);
            tma_load_2d(to, &tx, kb * kBlock, t0, &full[s]);
            tma_load_2d(to + kXTile, &tw, kb * kBlock, j0, &full[s]);
          }
          __syncwarp();
        }
      }
      // no copy may be on its way when the CTA ends
      for (int i = it - kStages < 0 ? 0 : it - kStages; i < it; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1, kWaitNs);
    } else if (warp <= kMmaWarps) {
      // descriptors: the low words move with the stage, the high ones are constants
      const uint32_t base = smem_addr(sm);
      const uint32_t lo = static_cast<uint32_t>(desc_sw128(base)), hi = static_cast<uint32_t>(desc_sw128(base) >> 32);
      Turn<kStages> at;
      Turn<kSums> sums;
      int pair = 0;
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && !__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs))) {
          if (lane == 0) fail(p.status);
          ok = false;
        }
        return ok;
      };
      for (int tile = first; tile < p.tiles && ok; tile += step)
        for (int kb = kb0; kb < kb1 && ok; kb += 2, ++pair, sums.next()) {
          const bool two = kb + 1 < kb1;
          if (pair % kMmaWarps != warp - 1) {
            at.next();
            if (two) at.next();
            continue;
          }
          // (tempty's phase before its first is over as it begins)
          if (!wait(&tempty[sums.i], sums.parity ^ 1u)) break;
          for (int i = 0; i < 1 + two; ++i, at.next()) {
            if (!wait(&full[at.i], at.parity)) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t x = lo + at.i * (kStage >> 4), w = x + (kXTile >> 4), d = tmem + (sums.i * 2 + i) * kColumns;
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_e4m3(d, desc_of(x + 2 * k, hi), desc_of(w + 2 * k, hi), kId, k != 0);
              mma_commit(&empty[at.i]);
              if (i == two) mma_commit(&tfull[sums.i]);
            }
            __syncwarp();
          }
        }
      // every product is finished before tensor memory goes
      for (int i = pair - kSums < 0 ? 0 : pair - kSums; i < pair && ok; ++i) mbar_wait(&tfull[i % kSums], (i / kSums) & 1, kWaitNs);
    } else {
      // scales: a lane has four rows of x; copies of two groups are on their way while a third is told of
      constexpr int kAhead = 2;
      Turn<kGroups> at, ready;
      int g = 0, told = 0;
      bool ok = true;
      auto tell = [&](int upto) {
        __syncwarp();
        for (; told < upto; ++told, ready.next())
          if (lane == 0) mbar_arrive(&sfull[ready.i]);
      };
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int t0 = row_of(tile) + lane, jb = column_of(tile) / kBlock;
        for (int kb = kb0; kb < kb1; kb += kGroup, ++g, at.next()) {
          if (g >= kGroups && !__all_sync(0xffffffffu, mbar_wait(&sempty[at.i], at.parity ^ 1u, kWaitNs))) {
            if (lane == 0) fail(p.status);
            ok = false;
            break;
          }
          const uint32_t to = smem_addr(scales + at.i * (kRows + 1));
          auto copy = [&](int place, const float *row, bool there, bool wide) {
            if (wide && kb + 4 <= p.kb) {
              mkw::cp_async16(to + place * 16, row + (there ? kb : 0), there);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool some = there && kb + e < kb1;
                mkw::cp_async4(to + place * 16 + e * 4, row + (some ? kb + e : 0), some);
              }
            }
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool there = t0 + 32 * i < p.m;
            copy(lane + 32 * i, p.x_scale + (there ? (t0 + 32 * i) * p.x_scale_row : 0), there, p.wide_scales && kb0 % 4 == 0);
          }
          if (lane == 0) copy(kRows, p.w_scale + static_cast<int64_t>(jb) * p.kb, true, false);
          mkw::cp_async_commit();
          mkw::cp_async_wait<kAhead>();
          if (g >= kAhead) tell(g - kAhead + 1);
        }
      }
      mkw::cp_async_wait<0>();
      if (ok) tell(g);
    }
  } else {
    const int q = warp & 3, part = (warp - kHelpers) >> 2; // lanes of tensor memory, half of the columns
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + part * kCols;
    Turn<kSums> sums;
    Turn<kGroups> groups;
    unsigned char *mine = sm + kResults + (warp - kHelpers) * 32 * kBoxRow;
    uint64_t *loaded = rfull + (warp - kHelpers);
    uint32_t load_parity = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && !__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs))) {
        if (lane == 0) fail(p.status);
        ok = false;
      }
      return ok;
    };
    for (int tile = first; tile < p.tiles; tile += step) {
      const int t = row_of(tile) + 32 * q + lane, j0 = column_of(tile) + part * kCols;
      const bool idle = __all_sync(0xffffffffu, t >= p.m || j0 >= p.n);   // a warp without a result only takes part
      unsigned long long acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
      // the residual comes to where the results will be, once what was there has been stored
      const bool by_tma = TMA && p.splits == 1 && !idle;
      auto ask_residual = [&](int c) {
        if (lane == 0) {
          bulk_wait_read();
          mbar_expect_tx(loaded, 32 * kBoxRow);
          tma_load_2d(mine, &tr, j0 + c, t - lane, loaded);
        }
      };
      for (int kbg = kb0; kbg < kb1 && ok; kbg += kGroup, groups.next()) {
        if (by_tma && p.residual && kbg + kGroup >= kb1) ask_residual(0);
        const float4 *sc = scales + groups.i * (kRows + 1);
        if (!wait(&sfull[groups.i], groups.parity)) break;
        const float4 fx = sc[32 * q + lane], fw = sc[kRows];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[groups.i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kbg + 2 * h >= kb1) break;
          const bool two = kbg + 2 * h + 1 < kb1;
          if (!wait(&tfull[sums.i], sums.parity)) break;
          tc_fence_after();
          if (!idle) {
            const uint32_t from = at + sums.i * 2 * kColumns;
            uint32_t v[2][32];
            tmem_ld32(from, v[0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i == 1 && !two) break;
              const float f = (&fx.x)[2 * h + i] * (&fw.x)[2 * h + i];
              unsigned long long ff;
              asm("mov.b64 %0, {%1, %1};" : "=l"(ff) : "f"(f));
#pragma unroll
              for (int c = 0; c < kCols; c += 32) {
                uint32_t(&now)[32] = v[c / 32 & 1];
                tmem_ld_wait(now);
                if (c + 32 < kCols) tmem_ld32(from + i * kColumns + c + 32, v[(c / 32 + 1) & 1]);
                else if (i == 0 && two) tmem_ld32(from + kColumns, v[(c / 32 + 1) & 1]);
#pragma unroll
                for (int e = 0; e < 16; ++e) add_scaled(acc[c / 2 + e], now[2 * e], now[2 * e + 1], ff);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[sums.i]);
          sums.next();
        }
      }
      if (!ok) break;
      auto sum = [&](int i) { return __uint_as_float(static_cast<uint32_t>(i & 1 ? acc[i / 2] >> 32 : acc[i / 2])); };
      if (p.splits > 1) {
        // (one tile a cluster; its stages have been read)
        float4 *to = reinterpret_cast<float4 *>(reinterpret_cast<float *>(sm) + (32 * q + lane) * kSplitRow + part * kCols);
        if (!idle) {
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) to[i] = make_float4(sum(4 * i), sum(4 * i + 1), sum(4 * i + 2), sum(4 * i + 3));
        }
      } else if (by_tma) {
        // a box of 32 rows at a time: the residual is there, the results go out
#pragma unroll
        for (int c = 0; c < kCols; c += PIECE) {
          if (!p.residual) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
          } else {
            if (c > 0) ask_residual(c);
            __syncwarp();
            if (!wait(loaded, load_parity)) break;
            load_parity ^= 1u;
          }
#pragma unroll
          for (int i = 0; i < PIECE / N; ++i) {
            uint4 *at = reinterpret_cast<uint4 *>(mine + lane * kBoxRow + ((i ^ (lane & 7)) << 4));
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = sum(c + i * N + e);
            if (p.residual) Out<T>::add(*at, v);
            *at = Out<T>::bits(v);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (j0 + c < p.n) tma_store_2d(&ty, mine, j0 + c, t - lane);
            bulk_commit();
          }
        }
        if (!ok) break;
      } else if (!TMA && !idle) {
        // rows that are not on 16 bytes: 32 columns of 32 rows at a time through shared memory, then a row's numbers together,
        // 16 rows of the residual on their way at once (1101 x 83799 x 880 with a residual 292 us; 16 columns and four rows 865)
        auto at = [&](int row, int col) { return reinterpret_cast<float *>(mine) + row * 32 + (col ^ ((row & 7) << 2)); };
        const int rows = min(32, p.m - (t - lane));
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4 *>(at(lane, i)) = make_float4(sum(c + i), sum(c + i + 1), sum(c + i + 2), sum(c + i + 3));
          __syncwarp();
          const int col = j0 + c + lane;
          if (col < p.n) {
            T *y = static_cast<T *>(p.y) + (t - lane) * p.y_row + col;
            const T *res = p.residual ? static_cast<const T *>(p.residual) + (t - lane) * p.residual_row + col : nullptr;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += 16) {
              T r[16];
              if (res) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  if (r0 + k < rows) r[k] = res[(r0 + k) * p.residual_row];
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (r0 + k >= rows) break;
                const float v = *at(r0 + k, lane);
                y[(r0 + k) * p.y_row] = static_cast<T>(res ? v + static_cast<float>(r[k]) : v);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  if (p.splits > 1) {
    mkw::cluster_arrive();
    mkw::cluster_wait();
    // kColumns / splits columns each, four a thread: the CTAs' sums in order
    const int t0 = first % p.tiles_m * kRows, j0 = first / p.tiles_m * kColumns, rows = min(kRows, p.m - t0), columns = kColumns / p.splits, fours = columns / 4;
    for (int i = threadIdx.x; i < fours * rows; i += kThreads) {
      const int t = i / fours, c = split * columns + i % fours * 4, col = j0 + c;
      if (col >= p.n) continue;
      const float *own = reinterpret_cast<const float *>(sm) + t * kSplitRow + c;
      float4 part[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.splits) part[r] = load_remote4(mkw::remote(own, r));
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.splits) v[0] += part[r].x, v[1] += part[r].y, v[2] += part[r].z, v[3] += part[r].w;
      T *y = static_cast<T *>(p.y) + (t0 + t) * p.y_row + col;
      const T *res = p.residual ? static_cast<const T *>(p.residual) + (t0 + t) * p.residual_row + col : nullptr;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) y[e] = static_cast<T>(res ? v[e] + static_cast<float>(res[e]) : v[e]);
    }
    mkw::cluster_arrive();                                 // nobody leaves while its sums are read
    mkw::cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kTensorColumns);
}

// ---- host side ---------------------------------------------------------------------------

// rows of T, `row` apart, in boxes of 32 rows, 128 bytes of each
template <class T>
bool result_map(CUtensorMap *map, const void *base, int64_t columns, int64_t rows, int64_t row) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(row) * sizeof(T)};
  const cuuint32_t box[2] = {kBoxRow / sizeof(T), 32}, es[2] = {1, 1};
  return enc(map, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of `inner` bytes, `row` apart, in boxes of 128 bytes by box_rows
bool byte_map(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t row, int box_rows) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(row)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, bool TMA>
int launch(const mk_matmul_fp8_args *a, MatmulParams &p, int sms, int dev, cudaStream_t s) {
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &matmul_kernel<T, TMA>;
  mkw::Ready &r = ready[dev];
  if (!r.get(reinterpret_cast<const void *>(fn), kThreads, kSmem)) return MK_ERR_CUDA;
  p.x_rows = std::min(kRows, (a->m + 7) / 8 * 8);
  CUtensorMap tw, tx, ty = {}, tr = {};
  if (TMA && (!result_map<T>(&ty, a->y, a->n, a->m, p.y_map_row) || (a->residual && !result_map<T>(&tr, a->residual, a->n, a->m, p.residual_map_row))))
    return MK_ERR_CUDA;
  if (!byte_map(&tx, a->x, a->k, a->m, a->x_row, p.x_rows) || !byte_map(&tw, a->w, a->k, a->n, a->w_row, kColumns)) return MK_ERR_CUDA;
  p.tiles_m = (a->m - 1) / kRows + 1;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * ((a->n - 1) / kColumns + 1);
  if (tiles > INT32_MAX - 65536) return MK_ERR_UNSUPPORTED;
  p.tiles = static_cast<int>(tiles);
  p.splits = 1;
  for (int i = 0; i < 3 && tiles * (2 << i) <= sms && p.kb >= 2 * (2 << i) && tiles <= r.clusters[i]; ++i) p.splits = 2 << i;
  const int clusters = p.splits > 1 ? p.tiles : std::min(p.tiles, sms);
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * p.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fn, tx, tw, ty, tr, p) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace mkf8

using namespace mkf8;

extern "C" int mk_quantize_fp8(const mk_quantize_fp8_args *a, mk_stream stream) {
  if (!a || a->m < 0 || a->k < 1 || a->k % 16 || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->x_row < 0 || a->codes_row < 0 || a->scales_row < 0)
    return MK_ERR_INVALID_ARG;
  if (a->m == 0) return MK_OK;
  const int es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->x || !a->codes || !a->scales || !aligned16(a->x) || !aligned16(a->codes) || a->x_row * es % 16 || a->codes_row % 16) return MK_ERR_INVALID_ARG;
  const int sms = mkv::sm_count(nullptr);
  if (sms < 0) return MK_ERR_CUDA;
  QuantParams p = {};
  p.x = a->x, p.codes = static_cast<uint8_t *>(a->codes), p.scales = a->scales;
  p.x_row = a->x_row, p.codes_row = a->codes_row, p.scales_row = a->scales_row;
  p.k = a->k;
  p.blocks.set((a->k - 1) / kBlock + 1);
  const int64_t items = static_cast<int64_t>(a->m) * p.blocks.value;
  if (items > INT32_MAX - 65536) return MK_ERR_UNSUPPORTED;
  p.items = static_cast<int>(items);
  // bf16: four blocks at a time where there are enough to fill the SMs several times over (32768 x 2048: 40.5 us, one at a time
  // 46; 8192 x 2048, which is about as quick either way, 11.0 and 10.5; 1024 x 2048 3.2 and 2.5).  fp32, with twice the bytes
  // on their way, always one (32768 x 2048: 49.0 us, four at a time 49.1; 8192 x 2048 10.3 and 10.9).
  const bool many = a->dtype == MK_BF16 && items >= int64_t{4} * 16 * 16 * sms;
  const int each = kQuantThreads / 16 * (many ? 4 : 1);
  const dim3 grid(static_cast<unsigned>((items - 1) / each + 1));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (a->dtype == MK_F32) return mkw::launch_after(&quantize_kernel<float, 1>, grid, kQuantThreads, 0, s, p);
  return many ? mkw::launch_after(&quantize_kernel<B, 4>, grid, kQuantThreads, 0, s, p) : mkw::launch_after(&quantize_kernel<B, 1>, grid, kQuantThreads, 0, s, p);
}

extern "C" int mk_matmul_fp8(const mk_matmul_fp8_args *a, mk_stream stream) {
  if (!a || a->m < 0 || a->n < 0 || a->k < 1 || a->k % 16 || (a->dtype != MK_F32 && a->dtype != MK_BF16) || a->x_row < 0 || a->w_row < 0 ||
      a->x_scale_row < 0 || a->y_row < 0 || a->residual_row < 0)
    return MK_ERR_INVALID_ARG;
  if (a->m == 0 || a->n == 0) return MK_OK;
  const uintptr_t es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->x || !a->w || !a->x_scale || !a->w_scale || !a->y || !aligned16(a->x) || !aligned16(a->w) || a->x_row % 16 || a->w_row % 16 || a->x_row < a->k ||
      a->w_row < a->k || reinterpret_cast<uintptr_t>(a->y) % es || reinterpret_cast<uintptr_t>(a->residual) % es)
    return MK_ERR_INVALID_ARG;
  if (a->x_row >= (int64_t{1} << 40) || a->w_row >= (int64_t{1} << 40) || a->m > INT32_MAX - 512 || a->n > INT32_MAX - 512 || a->k > INT32_MAX - 512)
    return MK_ERR_UNSUPPORTED;
  int dev = 0;
  const int sms = mkv::sm_count(&dev);
  if (sms < 0) return MK_ERR_CUDA;
  MatmulParams p = {};
  p.x_scale = a->x_scale, p.w_scale = a->w_scale, p.residual = a->residual, p.y = a->y, p.status = a->status;
  p.x_scale_row = a->x_scale_row, p.residual_row = a->residual_row, p.y_row = a->y_row;
  p.m = a->m, p.n = a->n, p.kb = (a->k - 1) / kBlock + 1;
  // (an expanded residual has no stride that a tensor map takes; a single row may have any)
  p.y_map_row = a->m == 1 ? a->n : a->y_row, p.residual_map_row = a->m == 1 ? a->n : a->residual_row;
  auto mapped = [&](const void *t, int64_t row) { return aligned16(t) && row * es % 16 == 0 && row >= a->n && row < (int64_t{1} << 36); };
  // A copy to memory writes whole pieces of 16 bytes: a row that ends inside one would lose what is behind it.
  const bool tma = a->n * es % 16 == 0 && mapped(a->y, p.y_map_row) && (!a->residual || mapped(a->residual, p.residual_map_row));
  p.wide_scales = aligned16(a->x_scale) && a->x_scale_row % 4 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (tma) return a->dtype == MK_F32 ? launch<float, true>(a, p, sms, dev, s) : launch<B, true>(a, p, sms, dev, s);
  return a->dtype == MK_F32 ? launch<float, false>(a, p, sms, dev, s) : launch<B, false>(a, p, sms, dev, s);
}
