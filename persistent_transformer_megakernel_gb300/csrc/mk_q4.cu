// Matrix-vector products with 4-bit weights (mk_matvec_q4).
//
// y[m][n] = sum_k x[m][k] scale[n][k / group] (code[n][k] - zero[n][k / group])
//
// Bound by the weights' bytes: N K / 2 plus the scales.  A warp takes 16 weight
// rows (32 where several column tiles share them) as the rows of 16x8x16 matrix
// products and the x rows as their columns, up to 8 a tile: a code minus its
// zero is a small whole number, exact in bf16, and so is its product with a bf16
// x; an fp32 x is three bf16 terms in three columns, which together hold all its
// bits.  Products are summed in fp32 over a lane's block of one group, then
// multiplied by the group's scale and added to the row's sum in fp32.
//
// Where an element of k sits in a matrix product is free as long as both operands
// agree.  A warp's block is 128 elements of k of its rows; lane t of a quad holds,
// of each row, four 32-bit words of 8 codes: 16 bytes in a row where one group
// covers the block, 8 bytes of each of two groups of 64, 4 of each of four groups
// of 32, so that a product never mixes two groups.  The x columns are staged in
// shared memory, each 8 elements in the order 0 4 1 5 2 6 3 7: codes j and j + 4 of
// a word are taken out together, (w >> 4j) & 0x000f000f in the low mantissa bits of
// the bf16 number 2^-5, whose last place is 2^-12, less 2^-5 and the zero in the
// same place.  The products are thus 2^-12 of their value until the end, which
// keeps those of the largest finite x finite.
//
// The rows' tiles are dealt out to persistent CTAs; 2, 4 or 8 warps share a tile's
// k where that deals them out more evenly, and 2 or 4 CTAs (a cluster) where there
// are too few tiles for the SMs, which also divides the staging of x.  Their sums
// are added in a fixed order.  Every warp keeps U blocks of weights on their way in
// registers, across tiles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/mk.h"
#include "mk_mma.cuh"
#include "mk_paged.h"

namespace mkq {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kBlock = 128;
constexpr int kMaxSmem = 225 * 1024;   // dynamic shared memory of a CTA
constexpr int kMaxK = 24576;           // an fp32 row's three columns of this length, and one of zeros, still fit

struct Q4Params {
  const void *x, *residual;
  void *y;
  const unsigned char *codes;
  const uint16_t *scales;
  const uint8_t *zeros;
  int64_t x_row, residual_row, y_row;
  int m, n, k, group, groups;
  int blocks;           // of k, the last one maybe short
  int pass_rows;        // x rows of one pass (blockIdx.y)
  int wk;               // warps that share a tile's k: 1, 2, 4 or 8
  int cluster;          // CTAs that share a tile's k (then wk is 8)
  int tiles;            // tiles of 16 RT rows
  int pitch;            // bytes from staged column to column
  int vec;              // a block's scales (and zeros) of a row can be loaded at once
};

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

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ void load8(const float *p, float *x) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <class T>
constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// the 8 elements of an eighth as the bf16 terms of its columns, in staging order
__device__ __forceinline__ void stage8(const float *x, unsigned char *to, int pitch) {
  float v[8];
  load8(x, v);
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    uint4 o;
    o.x = mkw::take_input_term(mkw::BF16Op{}, v[0], v[4]);
    o.y = mkw::take_input_term(mkw::BF16Op{}, v[1], v[5]);
    o.z = mkw::take_input_term(mkw::BF16Op{}, v[2], v[6]);
    o.w = mkw::take_input_term(mkw::BF16Op{}, v[3], v[7]);
    *reinterpret_cast<uint4 *>(to + u * pitch) = o;
  }
}
__device__ __forceinline__ void stage8(const __nv_bfloat16 *x, unsigned char *to, int) {
  const uint4 w = *reinterpret_cast<const uint4 *>(x);
  *reinterpret_cast<uint4 *>(to) = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                                              __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
}

template <class T, int NT, int RT, int G, int U>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 2 : 1) matvec_kernel(const Q4Params p) {
  using L = Layout<G>;
  constexpr int TERMS = kTerms<T>, GB = L::groups;
  constexpr int ROWS = 16 * RT, COLS = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int wn = w / p.wk, wk = w % p.wk, per_cta = kWarps / p.wk;
  const int rank = p.cluster > 1 ? blockIdx.x % p.cluster : 0, unit = blockIdx.x / p.cluster, units = gridDim.x / p.cluster;
  const int m0 = blockIdx.y * p.pass_rows, mr = min(p.pass_rows, p.m - m0), cols = mr * TERMS;
  float *red = reinterpret_cast<float *>(smem) + wn * p.wk * ROWS * COLS;         // sums of the warps of this tile
  unsigned char *xs = smem + kWarps * ROWS * COLS * 4;

  // this CTA's blocks of k, this warp's slice of them, its tiles
  const int c0 = p.blocks * rank / p.cluster, cn = p.blocks * (rank + 1) / p.cluster - c0;
  const int b0 = c0 + cn * wk / p.wk, nb = c0 + cn * (wk + 1) / p.wk - b0;
  const int tile0 = unit * per_cta + wn, step = units * per_cta;
  const int rounds = tile0 < p.tiles ? (p.tiles - tile0 + step - 1) / step : 0;

  struct Slot {
    uint32_t code[RT][2][4];
    uint32_t scale[RT][2][G == 32 ? 2 : 1];              // bf16 pairs
    uint32_t zero[RT][2];                                // a byte each
  } slot[U];
  int l_tile = tile0, l_blk = 0, l_left = rounds * nb;   // the loads' place
  const unsigned char *code_at[RT][2];
  int64_t group_at[RT][2];
  auto rows_of = [&]() {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = min(l_tile * ROWS + r * 16 + h * 8 + g, p.n - 1);   // rows past the last are read as it and not stored
        code_at[r][h] = p.codes + row * (p.k / 2) + b0 * (kBlock / 2) + t * (16 / GB);
        group_at[r][h] = row * p.groups;
      }
  };
  if (l_left > 0) rows_of();
  auto load = [&](Slot &s) {
    if (l_left <= 0) return;
    --l_left;
    const int blk = b0 + l_blk;
    const bool full = G == 128 || (blk + 1) * kBlock <= p.k;
    int grp = blk * GB;
    if (G == 128 && p.group > kBlock) grp = blk / (p.group / kBlock);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned char *c = code_at[r][h];
        const uint16_t *sc = p.scales + group_at[r][h] + grp;
        if (full) {
          if constexpr (G == 128) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(c));
            s.code[r][h][0] = v.x, s.code[r][h][1] = v.y, s.code[r][h][2] = v.z, s.code[r][h][3] = v.w;
          } else if constexpr (G == 64) {
            const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(c)), b = __ldcs(reinterpret_cast<const uint2 *>(c + 32));
            s.code[r][h][0] = a.x, s.code[r][h][1] = a.y, s.code[r][h][2] = b.x, s.code[r][h][3] = b.y;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s.code[r][h][i] = __ldcs(reinterpret_cast<const uint32_t *>(c + 16 * i));
          }
        } else {
          // the short last block: no codes and scales of 0 past the end
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = G == 64 ? 32 * (i >> 1) + 4 * (i & 1) : 16 * i;
            s.code[r][h][i] = blk * kBlock + (G == 64 ? 64 * (i >> 1) : 32 * i) < p.k ? *reinterpret_cast<const uint32_t *>(c + at) : 0u;
          }
        }
        if (GB == 1) {
          s.scale[r][h][0] = *sc;
          s.zero[r][h] = p.zeros ? p.zeros[group_at[r][h] + grp] : 8u;
        } else if (full && p.vec) {
          if constexpr (GB == 2) {
            s.scale[r][h][0] = *reinterpret_cast<const uint32_t *>(sc);
            s.zero[r][h] = p.zeros ? *reinterpret_cast<const uint16_t *>(p.zeros + group_at[r][h] + grp) : 0x0808u;
          } else if constexpr (GB == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(sc);
            s.scale[r][h][0] = v.x, s.scale[r][h][1] = v.y;
            s.zero[r][h] = p.zeros ? *reinterpret_cast<const uint32_t *>(p.zeros + group_at[r][h] + grp) : 0x08080808u;
          }
        } else {
          s.zero[r][h] = 0;
#pragma unroll
          for (int i = 0; i < GB; ++i) {
            const bool there = full || blk * kBlock + i * G < p.k;
            const uint32_t v = there ? sc[i] : 0u;
            s.scale[r][h][i >> 1] = (i & 1) ? s.scale[r][h][i >> 1] | (v << 16) : v;
            s.zero[r][h] |= (there && p.zeros ? p.zeros[group_at[r][h] + grp + i] : 8u) << (8 * i);
          }
        }
        code_at[r][h] = c + kBlock / 2;
      }
    if (++l_blk == nb) {
      l_blk = 0;
      l_tile += step;
      if (l_left > 0) rows_of();
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(slot[u]);

  // ---- the x rows as columns of bf16 terms, zeros past k and in one more column for those of the tiles that are none ----------------
  const T *x = static_cast<const T *>(p.x) + m0 * p.x_row;
  const int eighths = cn * (kBlock / 8), last = p.k / 8 - c0 * (kBlock / 8);
  for (int r = 0; r < mr; ++r)
    for (int b = tid; b < eighths; b += kThreads) {
      unsigned char *to = xs + r * TERMS * p.pitch + L::staged(b) * 16;
      if (b < last) {
        stage8(x + r * p.x_row + (c0 * (kBlock / 8) + b) * 8, to, p.pitch);
      } else {
#pragma unroll
        for (int u = 0; u < TERMS; ++u) *reinterpret_cast<uint4 *>(to + u * p.pitch) = make_uint4(0, 0, 0, 0);
      }
    }
  if (cols < COLS)
    for (int b = tid; b < eighths; b += kThreads) *reinterpret_cast<uint4 *>(xs + cols * p.pitch + b * 16) = make_uint4(0, 0, 0, 0);
  __syncthreads();

  float sum[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) sum[r][c][0] = sum[r][c][1] = sum[r][c][2] = sum[r][c][3] = 0.f;
  int tile = tile0, blk = 0;
  const unsigned char *column[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) column[c] = xs + min(c * 8 + g, cols) * p.pitch;

  auto compute = [&](const Slot &s) {
    const int e0 = (b0 - c0 + blk) * (kBlock / 8);
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // words; a group ends with every (4 / GB)th
      uint4 b[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) b[c] = *reinterpret_cast<const uint4 *>(column[c] + L::staged(e0 + L::eighth(t, i)) * 16);
      const int grp = i * GB / 4;
      const bool fresh = i % (4 / GB) == 0, done = (i + 1) % (4 / GB) == 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = s.code[r][h][i];
          const uint32_t z = (0x3d00u | ((s.zero[r][h] >> (8 * grp)) & 15u)) * 0x10001u;      // 2^-5 + 2^-12 zero, twice
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j >> 1][(j & 1) * 2 + h] = minus(((v >> (4 * j)) & 0x000f000fu) | 0x3d003d00u, z);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (fresh) mkw::mma_zero(mkw::BF16Op{}, acc[r][c], a[0], b[c].x, b[c].y);
          else mkw::mma(mkw::BF16Op{}, acc[r][c], a[0], b[c].x, b[c].y);
          mkw::mma(mkw::BF16Op{}, acc[r][c], a[1], b[c].z, b[c].w);
        }
        if (done) {
          const float s0 = bf16_float((s.scale[r][0][grp >> 1] >> (16 * (grp & 1))) & 0xffffu);
          const float s1 = bf16_float((s.scale[r][1][grp >> 1] >> (16 * (grp & 1))) & 0xffffu);
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            sum[r][c][0] += s0 * acc[r][c][0];
            sum[r][c][1] += s0 * acc[r][c][1];
            sum[r][c][2] += s1 * acc[r][c][2];
            sum[r][c][3] += s1 * acc[r][c][3];
          }
        }
      }
    }
  };
  auto meet = [&]() {                                      // the warps of a tile
    if (p.wk == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + wn), "r"(32 * p.wk) : "memory");
  };
  auto finish = [&]() {
    float *mine = red + wk * ROWS * COLS;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        *reinterpret_cast<float2 *>(mine + (r * 16 + g) * COLS + c * 8 + 2 * t) = make_float2(sum[r][c][0], sum[r][c][1]);
        *reinterpret_cast<float2 *>(mine + (r * 16 + 8 + g) * COLS + c * 8 + 2 * t) = make_float2(sum[r][c][2], sum[r][c][3]);
        sum[r][c][0] = sum[r][c][1] = sum[r][c][2] = sum[r][c][3] = 0.f;
      }
    meet();
    if (p.cluster > 1) {                                   // (then this tile has the whole CTA)
      // each CTA's sum over its warps, in the place of the first warp's; CTA 0 adds them
      for (int i = tid; i < ROWS * COLS; i += kThreads) {
        float y = red[i];
        for (int j = 1; j < kWarps; ++j) y += red[j * ROWS * COLS + i];
        red[i] = y;
      }
      mkw::cluster_meet();
    }
    if (rank == 0) {
      for (int i = wk * 32 + lane; i < ROWS * mr; i += 32 * p.wk) {
        const int r = i % ROWS, m = i / ROWS, row = tile * ROWS + r;
        float y = 0.f;
#pragma unroll
        for (int u = TERMS - 1; u >= 0; --u) {
          const float *at = red + r * COLS + m * TERMS + u;
          if (p.cluster > 1) {
            for (int j = 0; j < p.cluster; ++j) y += mkw::load_remote(at, j);
          } else {
            for (int j = 0; j < p.wk; ++j) y += at[j * ROWS * COLS];
          }
        }
        y *= 4096.f;
        if (row < p.n) {
          if (p.residual) y += to_float(static_cast<const T *>(p.residual)[(m0 + m) * p.residual_row + row]);
          put(static_cast<T *>(p.y) + (m0 + m) * p.y_row + row, y);
        }
      }
    }
    if (p.cluster > 1) mkw::cluster_meet();
    else meet();
    tile += step;
  };

  if (nb == 0) {                                           // fewer blocks than warps: this one only joins in
    for (int i = 0; i < rounds; ++i) finish();
    return;
  }
  const int items = rounds * nb;
  for (int i = 0; i < items; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < items) {
        compute(slot[u]);
        load(slot[u]);
        if (++blk == nb) {
          blk = 0;
          finish();
        }
      }
    }
  }
}

template <class T, int NT, int RT, int G, int U>
int launch(Q4Params p, int sms, int dev, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const auto fn = &matvec_kernel<T, NT, RT, G, U>;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  constexpr int per = kBlock / G;
  p.vec = p.groups % per == 0 && reinterpret_cast<uintptr_t>(p.scales) % (2 * per) == 0 &&
          (!p.zeros || reinterpret_cast<uintptr_t>(p.zeros) % per == 0);
  p.blocks = (p.k + kBlock - 1) / kBlock;
  p.tiles = (p.n + 16 * RT - 1) / (16 * RT);
  const int red = kWarps * 16 * RT * 8 * NT * 4;
  // a cluster while the tiles leave SMs idle and every warp still has two blocks of k
  p.cluster = 1;
  while (p.cluster < 4 && p.tiles * p.cluster * 2 <= 2 * sms && p.blocks >= 2 * kWarps * 2 * p.cluster) p.cluster *= 2;
  const int staged_blocks = (p.blocks + p.cluster - 1) / p.cluster;
  p.pitch = staged_blocks * kBlock * 2 + Layout<G>::pad;
  // x rows of a pass: as many as its columns hold and shared memory has room for, a column of zeros beside them
  p.pass_rows = std::min({p.m, 8 * NT / kTerms<T>, ((kMaxSmem - red) / p.pitch - 1) / kTerms<T>});
  const int smem = red + (p.pass_rows * kTerms<T> + 1) * p.pitch;
  const int passes = (p.m + p.pass_rows - 1) / p.pass_rows;
  if (passes > 65535) return MK_ERR_UNSUPPORTED;
  const int ctas = sms * (RT == 1 && smem <= kMaxSmem / 2 ? 2 : 1);
  if (p.cluster > 1) {
    p.wk = kWarps;
  } else {
    // the sharing of k that leaves the busiest warp the least: rounds / wk, fewer warps a tile where that is equal
    int64_t best = 0;
    for (int wk = 1; wk <= kWarps; wk *= 2) {
      const int64_t per_round = static_cast<int64_t>(ctas) * (kWarps / wk), rounds = (p.tiles + per_round - 1) / per_round;
      const int64_t cost = rounds * (kWarps / wk);
      if (wk == 1 || cost < best) best = cost, p.wk = wk;
    }
  }
  const int per_cta = kWarps / p.wk, want = (p.tiles + per_cta - 1) / per_cta;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(std::min(want, std::max(1, ctas / p.cluster)) * p.cluster, passes);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, static_cast<const Q4Params>(p)) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

template <class T, int NT, int RT>
int by_group(const Q4Params &p, int sms, int dev, cudaStream_t s) {
  constexpr int U = RT == 1 ? 4 : 2;     // blocks on their way: 64 bytes of codes a lane and row
  if (p.group == 32) return launch<T, NT, RT, 32, U>(p, sms, dev, s);
  if (p.group == 64) return launch<T, NT, RT, 64, U>(p, sms, dev, s);
  return launch<T, NT, RT, 128, U>(p, sms, dev, s);
}

template <class T>
int by_rows(const Q4Params &p, int sms, int dev, cudaStream_t s) {
  const int cols = p.m > 32 ? 32 : p.m * kTerms<T>;
  if (cols <= 8) return by_group<T, 1, 1>(p, sms, dev, s);
  if (cols <= 16) return by_group<T, 2, 1>(p, sms, dev, s);
  return by_group<T, 4, 2>(p, sms, dev, s);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace mkq

extern "C" int mk_matvec_q4(const mk_matvec_q4_args *a, mk_stream stream) {
  using namespace mkq;
  if (!a || a->m < 0 || a->n < 0 || a->k < 1 || a->group < 1 || (a->dtype != MK_F32 && a->dtype != MK_BF16)) return MK_ERR_INVALID_ARG;
  if (a->k % a->group) return MK_ERR_INVALID_ARG;
  if ((a->group != 32 && a->group != 64 && a->group % 128) || a->k > kMaxK) return MK_ERR_UNSUPPORTED;
  if (a->m == 0 || a->n == 0) return MK_OK;
  const int es = a->dtype == MK_F32 ? 4 : 2;
  if (!a->x || !a->codes || !a->scales || !a->y || !aligned16(a->x) || !aligned16(a->codes) || a->x_row < 0 ||
      a->x_row * es % 16 || a->y_row < 0 || (a->residual && a->residual_row < 0))
    return MK_ERR_INVALID_ARG;
  if (a->n > INT32_MAX - 64) return MK_ERR_UNSUPPORTED;
  int dev = 0;
  const int sms = mkv::sm_count(&dev);
  if (sms < 0) return MK_ERR_CUDA;
  Q4Params p = {};
  p.x = a->x, p.residual = a->residual, p.y = a->y;
  p.codes = static_cast<const unsigned char *>(a->codes);
  p.scales = static_cast<const uint16_t *>(a->scales);
  p.zeros = a->zeros;
  p.x_row = a->x_row, p.residual_row = a->residual_row, p.y_row = a->y_row;
  p.m = a->m, p.n = a->n, p.k = a->k, p.group = a->group, p.groups = a->k / a->group;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == MK_F32 ? by_rows<float>(p, sms, dev, s) : by_rows<__nv_bfloat16>(p, sms, dev, s);
}
