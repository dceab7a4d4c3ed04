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
// agree: lane t of a quad takes 4 (group 32), 8 (group 64) or 16 bytes (groups of
// 128 and multiples) of its rows at once, so that a product never mixes two
// groups, and the x columns are staged in shared memory in that order.  Codes j
// and j + 4 of a 32-bit word are taken out together: (w >> 4j) & 0x000f000f in the
// low mantissa bits of the bf16 number 2^-5, whose last place is 2^-12, less 2^-5
// and the zero in the same place.  The products are thus 2^-12 of their value
// until the end, which keeps those of the largest finite x finite.
//
// The rows' tiles are dealt out to persistent CTAs; up to 8 warps share a tile's
// k when there are too few tiles to fill the SMs.  Every warp keeps U blocks of
// weights on their way in registers, across tiles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/mk.h"
#include "mk_mma.cuh"
#include "mk_paged.h"

namespace mkq {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxSmem = 225 * 1024;   // dynamic shared memory of a CTA
constexpr int kMaxK = 32768;           // an fp32 row's three columns of this length still fit

struct Q4Params {
  const void *x, *residual;
  void *y;
  const unsigned char *codes;
  const uint16_t *scales;
  const uint8_t *zeros;
  int64_t x_row, residual_row, y_row;
  int m, n, k, group, groups;
  int pass_rows;        // x rows of one pass (blockIdx.y)
  int wk;               // warps that share a tile's k: 1, 2, 4 or 8
  int tiles;            // tiles of 16 RT rows
  int pitch;            // bytes from staged column to column
};

template <int BYTES>
struct Load;
template <>
struct Load<16> {
  using type = uint4;
  static constexpr int pad = 32;
};
template <>
struct Load<8> {
  using type = uint2;
  static constexpr int pad = 16;
};
template <>
struct Load<4> {
  using type = uint32_t;
  static constexpr int pad = 64;
};
// where 8-element block b of a column is staged: with the column pitch's `pad`, the 8 lanes of a shared-memory
// phase (two columns, four lanes of a quad) meet 8 different 16-byte banks
template <int BYTES>
__device__ __forceinline__ int staged(int b) {
  return BYTES == 16 ? b ^ ((b >> 3) & 1) : b;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ void load8(const float *p, float *x) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <class T>
constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;

template <class T, int NT, int RT, int BYTES, int U>
__global__ void __launch_bounds__(kThreads) matvec_kernel(const Q4Params p) {
  using W = typename Load<BYTES>::type;
  constexpr int TERMS = kTerms<T>;
  constexpr int WORDS = BYTES / 4, KB = 8 * BYTES;         // 32-bit words of a lane's load; elements a quad covers
  constexpr int ROWS = 16 * RT, COLS = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int wn = w / p.wk, wk = w % p.wk, per_cta = kWarps / p.wk;
  const int m0 = blockIdx.y * p.pass_rows, mr = min(p.pass_rows, p.m - m0), cols = mr * TERMS;
  float *red = reinterpret_cast<float *>(smem) + wn * p.wk * ROWS * COLS;         // sums of the warps of this tile
  unsigned char *xs = smem + kWarps * ROWS * COLS * 4;

  // this warp's items: its slice of k's blocks in each of its tiles
  const int blocks = p.k / KB, b0 = blocks * wk / p.wk, nb = blocks * (wk + 1) / p.wk - b0;
  const int tile0 = blockIdx.x * per_cta + wn, step = gridDim.x * per_cta;
  const int rounds = tile0 < p.tiles ? (p.tiles - tile0 + step - 1) / step : 0;
  const int items = rounds * nb;

  struct Slot {
    W code[RT][2];
    uint16_t scale[RT][2];
    uint8_t zero[RT][2];
  } slot[U];
  int l_tile = tile0, l_blk = 0, l_left = items;           // the loads' place
  auto load = [&](Slot &s) {
    if (l_left <= 0) return;
    --l_left;
    const int kblk = b0 + l_blk, grp = kblk * KB / p.group;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = min(l_tile * ROWS + r * 16 + h * 8 + g, p.n - 1);   // rows past the last are read as it and not stored
        s.code[r][h] = __ldcs(reinterpret_cast<const W *>(p.codes + row * (p.k / 2) + kblk * (KB / 2) + t * BYTES));
        s.scale[r][h] = p.scales[row * p.groups + grp];
        s.zero[r][h] = p.zeros ? p.zeros[row * p.groups + grp] : 8;
      }
    if (++l_blk == nb) {
      l_blk = 0;
      l_tile += step;
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(slot[u]);

  // ---- the x rows as columns of bf16 terms ----------------------------------
  const T *x = static_cast<const T *>(p.x) + m0 * p.x_row;
  const int k8 = p.k / 8;
  for (int i = tid; i < mr * k8; i += kThreads) {
    const int r = i / k8, b = i % k8;
    float v[8];
    load8(x + r * p.x_row + 8 * b, v);
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
      uint4 o;
      o.x = mkw::take_input_term(mkw::BF16Op{}, v[0], v[4]);
      o.y = mkw::take_input_term(mkw::BF16Op{}, v[1], v[5]);
      o.z = mkw::take_input_term(mkw::BF16Op{}, v[2], v[6]);
      o.w = mkw::take_input_term(mkw::BF16Op{}, v[3], v[7]);
      *reinterpret_cast<uint4 *>(xs + (r * TERMS + u) * p.pitch + staged<BYTES>(b) * 16) = o;
    }
  }
  __syncthreads();

  float sum[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < NT; ++c) sum[r][c][0] = sum[r][c][1] = sum[r][c][2] = sum[r][c][3] = 0.f;
  int tile = tile0, blk = 0;

  auto compute = [&](const Slot &s) {
    float acc[RT][NT][4];
    uint32_t z[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[r][c][0] = acc[r][c][1] = acc[r][c][2] = acc[r][c][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) z[r][h] = (0x3d00u | (s.zero[r][h] & 15u)) * 0x10001u;      // 2^-5 + 2^-12 zero, twice
    }
    const int e0 = (b0 + blk) * (KB / 8) + t * WORDS;      // first 8-element block of this lane
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      uint4 b[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        b[c] = make_uint4(0, 0, 0, 0);
        if (c * 8 + g < cols) b[c] = *reinterpret_cast<const uint4 *>(xs + (c * 8 + g) * p.pitch + staged<BYTES>(e0 + i) * 16);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = reinterpret_cast<const uint32_t *>(&s.code[r][h])[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j >> 1][(j & 1) * 2 + h] = minus(((v >> (4 * j)) & 0x000f000fu) | 0x3d003d00u, z[r][h]);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          mkw::mma(mkw::BF16Op{}, acc[r][c], a[0], b[c].x, b[c].y);
          mkw::mma(mkw::BF16Op{}, acc[r][c], a[1], b[c].z, b[c].w);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float s0 = __uint_as_float(static_cast<uint32_t>(s.scale[r][0]) << 16), s1 = __uint_as_float(static_cast<uint32_t>(s.scale[r][1]) << 16);
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        sum[r][c][0] += s0 * acc[r][c][0];
        sum[r][c][1] += s0 * acc[r][c][1];
        sum[r][c][2] += s1 * acc[r][c][2];
        sum[r][c][3] += s1 * acc[r][c][3];
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
    for (int i = wk * 32 + lane; i < ROWS * mr; i += 32 * p.wk) {
      const int r = i % ROWS, m = i / ROWS, row = tile * ROWS + r;
      float y = 0.f;
#pragma unroll
      for (int u = TERMS - 1; u >= 0; --u)
        for (int j = 0; j < p.wk; ++j) y += red[(j * ROWS + r) * COLS + m * TERMS + u];
      y *= 4096.f;
      if (row < p.n) {
        if (p.residual) y += to_float(static_cast<const T *>(p.residual)[(m0 + m) * p.residual_row + row]);
        put(static_cast<T *>(p.y) + (m0 + m) * p.y_row + row, y);
      }
    }
    meet();
    tile += step;
  };

  if (nb == 0) {                                           // fewer blocks than warps: this one only joins in
    for (int i = 0; i < rounds; ++i) finish();
    return;
  }
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

template <class T, int NT, int RT, int BYTES, int U>
int launch(Q4Params p, int sms, int dev, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const void *fn = reinterpret_cast<const void *>(&matvec_kernel<T, NT, RT, BYTES, U>);
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  const int red = kWarps * 16 * RT * 8 * NT * 4;
  p.tiles = (p.n + 16 * RT - 1) / (16 * RT);
  p.pitch = (p.k * 2 + 127) / 128 * 128 + Load<BYTES>::pad;
  p.pass_rows = std::min({p.m, 8 * NT / kTerms<T>, (kMaxSmem - red) / (kTerms<T> * p.pitch)});
  const int smem = red + p.pass_rows * kTerms<T> * p.pitch;
  const int passes = (p.m + p.pass_rows - 1) / p.pass_rows;
  // CTAs of an SM: two where their staged x leaves room
  const int ctas = sms * (smem <= kMaxSmem / 2 ? 2 : 1);
  // the fewest warps a tile that still give every SM its warps
  p.wk = 1;
  while (p.wk < kWarps && static_cast<int64_t>(p.tiles) * p.wk < static_cast<int64_t>(ctas) * kWarps) p.wk *= 2;
  const int per_cta = kWarps / p.wk, want = (p.tiles + per_cta - 1) / per_cta;
  if (passes > 65535) return MK_ERR_UNSUPPORTED;
  matvec_kernel<T, NT, RT, BYTES, U><<<dim3(std::min(want, ctas), passes), kThreads, smem, s>>>(p);
  if (cudaPeekAtLastError() != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

template <class T, int NT, int RT>
int by_group(const Q4Params &p, int sms, int dev, cudaStream_t s) {
  // 32 codes a lane and block in flight for every group size
  if (p.group == 32) return launch<T, NT, RT, 4, RT == 1 ? 8 : 4>(p, sms, dev, s);
  if (p.group == 64) return launch<T, NT, RT, 8, RT == 1 ? 4 : 2>(p, sms, dev, s);
  return launch<T, NT, RT, 16, RT == 1 ? 4 : 2>(p, sms, dev, s);
}

template <class T>
int by_rows(const Q4Params &p, int sms, int dev, cudaStream_t s) {
  const int cols = p.m > 32 ? 32 : p.m * kTerms<T>;
  if (cols <= 8) return by_group<T, 1, 1>(p, sms, dev, s);
  if (cols <= 16) return by_group<T, 2, 2>(p, sms, dev, s);
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
