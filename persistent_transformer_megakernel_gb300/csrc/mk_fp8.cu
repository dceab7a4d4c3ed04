// Products in 8-bit floating point with block scales (mk_quantize_fp8, mk_matmul_fp8).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mk.h"
#include "mk_launch_after.h"
#include "mk_mma.cuh"
#include "mk_paged.h"
#include "mk_tc.cuh"

namespace mkf8 {

using namespace mktc;

constexpr int kBlock = 128;

// ---------------------------------------------------------------------------
// Quantisation of rows: for each 128 of a row scale = largest / 448, code = x / scale rounded to e4m3.
//
// Bound by bytes: x read once, a byte an element and 4 a block written.  16 lanes have a block, 8 elements each; the
// quotient is fp32's (a bf16 element over its scale is often half way between two codes: a reciprocal's last place would
// decide which).
// ---------------------------------------------------------------------------

struct QuantParams {
  const void *x;
  uint8_t *codes;
  float *scales;
  int64_t x_row, codes_row, scales_row;
  int m, k, blocks;            // blocks of a row
  int64_t items;               // m * blocks
};

constexpr int kQuantThreads = 256;

__device__ __forceinline__ void load8(const float *p, bool hi, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = hi ? __ldcs(reinterpret_cast<const float4 *>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, bool, float (&x)[8]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float((&w.x)[i] << 16);
    x[2 * i + 1] = __uint_as_float((&w.x)[i] & 0xffff0000u);
  }
}

template <class T>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const __grid_constant__ QuantParams p) {
  mkw::follow_previous_kernel();
  const int lane = threadIdx.x & 15;
  const int64_t all = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 16);
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16) + (threadIdx.x >> 4); i0 - (threadIdx.x >> 4) < p.items; i0 += all) {
    const bool live = i0 < p.items;                        // (a warp's lanes stay together)
    const int64_t i = live ? i0 : 0;
    const int row = static_cast<int>(i / p.blocks), b = static_cast<int>(i - static_cast<int64_t>(row) * p.blocks);
    const int at = b * kBlock + lane * 8;                  // k is a multiple of 16: 8 elements are there or not
    float x[8] = {};
    const bool there = live && at < p.k;
    if (there) load8(static_cast<const T *>(p.x) + row * p.x_row + at, true, x);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float scale = __fdiv_rn(top, 448.f);
    if (!(scale > 0.f)) scale = 1.f;
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * e], scale), __fdiv_rn(x[4 * e + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[4 * e + 2], scale), __fdiv_rn(x[4 * e + 3], scale)), __NV_SATFINITE, __NV_E4M3);
      w[e] = a | c << 16;
    }
    if (there) *reinterpret_cast<uint2 *>(p.codes + row * p.codes_row + at) = make_uint2(w[0], w[1]);
    if (live && lane == 0) p.scales[row * p.scales_row + b] = scale;
  }
}

// ---------------------------------------------------------------------------
// y[t][j] = sum_b xs[t][b] ws[j / 128][b] sum_{k in b} x[t][k] w[j][k]  (+ residual)
//
// A CTA has 128 rows of w (one row of weight scales) and BN rows of x.  The inner sums of a block of 128 are four tensor
// instructions into one of two accumulators in tensor memory; eight warps take it out, multiply each column by its
// scale xs ws and add it to fp32 sums in registers while the next block is multiplied into the other.
// Roles: warp 0 asks for w and x by TMA, warp 1 multiplies, warps 2-9 add up, warps 10-11 bring the scales.
// Few rows (m): K is shared by the CTAs of a cluster, whose sums are added in order through their shared memory.
// ---------------------------------------------------------------------------

constexpr int kAddWarps = 8, kScaleWarps = 2, kWarps = 2 + kAddWarps + kScaleWarps, kThreads = 32 * kWarps;
constexpr int kScaleSlots = 8;
constexpr uint32_t kWTile = 128 * 128;
constexpr long long kWaitNs = 2000000000LL;

struct MatmulParams {
  const float *x_scale, *w_scale;
  const void *residual;
  void *y;
  int32_t *status;
  int64_t x_scale_row, residual_row, y_row;
  int m, n, kb;                // kb: blocks of K
  int tiles_n, tiles;          // tiles along n, in all
  int splits;                  // CTAs of a cluster that share a tile's K
};

template <int BN>
struct Cfg {
  static constexpr uint32_t XTILE = BN * 128, STAGE = kWTile + XTILE;
  static constexpr int STAGES = BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
  static constexpr uint32_t SCALES = STAGES * STAGE;                       // behind the stages: [slot][BN]
  static constexpr uint32_t CONTROL = SCALES + kScaleSlots * BN * 4;
  static constexpr int SMEM = static_cast<int>(1024 + CONTROL + 512);
  static constexpr int TCOLS = BN <= 16 ? 32 : 2 * BN;
  static constexpr int COLS = BN / 2;                                      // of an adding warp
  static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void fail(int32_t *status) {
  if (status) atomicCAS(status, 0, MK_ERR_TIMEOUT);
}
__device__ __forceinline__ float load_remote(uint32_t at) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

template <int BN, class T>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const __grid_constant__ MatmulParams p) {
  using C = Cfg<BN>;
  constexpr uint32_t kId = idesc_f32(128, BN);
  extern __shared__ unsigned char smraw[];
  mkw::follow_previous_kernel();
  unsigned char *sm = smraw + ((1024u - (smem_addr(smraw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::CONTROL), *empty = full + C::STAGES, *tfull = empty + C::STAGES, *tempty = tfull + 2,
           *sfull = tempty + 2, *sempty = sfull + kScaleSlots;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sempty + kScaleSlots);
  float *scales = reinterpret_cast<float *>(sm + C::SCALES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], kAddWarps);
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&sfull[i], kScaleWarps), mbar_init(&sempty[i], kAddWarps);
    fence_mbar_init();
    prefetch_tmap(&tw);
    prefetch_tmap(&tx);
  }
  if (warp == 1) tmem_alloc(tslot, C::TCOLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  const int rank = static_cast<int>(blockIdx.x) % p.splits, ctas = static_cast<int>(gridDim.x) / p.splits;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / p.splits), kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / p.splits);
  const int first = static_cast<int>(blockIdx.x) / p.splits;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += ctas) {
        const int j0 = tile % p.tiles_n * 128, t0 = tile / p.tiles_n * BN;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (it >= C::STAGES && !mbar_wait(&empty[s], (it / C::STAGES - 1) & 1, kWaitNs)) {
            fail(p.status);
            ok = false;
            break;
          }
          mbar_expect_tx(&full[s], C::STAGE);
          tma_load_2d(sm + s * C::STAGE, &tw, kb * kBlock, j0, &full[s]);
          tma_load_2d(sm + s * C::STAGE + kWTile, &tx, kb * kBlock, t0, &full[s]);
        }
      }
      // no copy may be on its way when the CTA ends
      for (int i = it - C::STAGES < 0 ? 0 : it - C::STAGES; i < it; ++i) mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, kWaitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += ctas)
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::STAGES, u = it & 1;
          if (!mbar_wait(&full[s], (it / C::STAGES) & 1, kWaitNs) || (it >= 2 && !mbar_wait(&tempty[u], (it / 2 - 1) & 1, kWaitNs))) {
            fail(p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_addr(sm + s * C::STAGE);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(tmem + u * BN, desc_sw128(a + 32 * k), desc_sw128(a + kWTile + 32 * k), kId, k != 0);
          mma_commit(&empty[s]);
          mma_commit(&tfull[u]);
        }
      // every product has been taken out (or abandoned, after the wait's limit) before tensor memory goes
      for (int i = it - 2 < 0 ? 0 : it - 2; i < it; ++i) mbar_wait(&tfull[i & 1], (i / 2) & 1, kWaitNs);
    }
  } else if (warp >= 2 + kAddWarps) {
    const int sw = warp - 2 - kAddWarps;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < p.tiles && ok; tile += ctas) {
      const int jb = tile % p.tiles_n, t0 = tile / p.tiles_n * BN;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % kScaleSlots;
        const float ws = p.w_scale[static_cast<int64_t>(jb) * p.kb + kb];
        float x[(BN + 63) / 64];
#pragma unroll
        for (int i = 0; i < (BN + 63) / 64; ++i) {
          const int t = t0 + i * 64 + sw * 32 + lane;
          x[i] = t < p.m ? p.x_scale[t * p.x_scale_row + kb] : 0.f;
        }
        if (it >= kScaleSlots && !__all_sync(0xffffffffu, mbar_wait(&sempty[s], (it / kScaleSlots - 1) & 1, kWaitNs))) {
          if (lane == 0) fail(p.status);
          ok = false;
          break;
        }
#pragma unroll
        for (int i = 0; i < (BN + 63) / 64; ++i)
          if (i * 64 + sw * 32 + lane < BN) scales[s * BN + i * 64 + sw * 32 + lane] = x[i] * ws;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[s]);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;        // lanes of tensor memory, half of the columns
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * C::COLS;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < p.tiles; tile += ctas) {
      const int j = tile % p.tiles_n * 128 + 32 * q + lane, t0 = tile / p.tiles_n * BN + half * C::COLS;
      float acc[C::COLS];
#pragma unroll
      for (int i = 0; i < C::COLS; ++i) acc[i] = 0.f;
      for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
        const int u = it & 1, s = it % kScaleSlots;
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[u], (it / 2) & 1, kWaitNs) && mbar_wait(&sfull[s], (it / kScaleSlots) & 1, kWaitNs))) {
          if (lane == 0) fail(p.status);
          ok = false;
          break;
        }
        tc_fence_after();
        const float *sc = scales + s * BN + half * C::COLS;
        constexpr int STEP = C::COLS < 32 ? C::COLS : 32;
#pragma unroll
        for (int c = 0; c < C::COLS; c += STEP) {
          uint32_t v[32];
          if constexpr (STEP == 32) {
            tmem_ld32(at + u * BN + c, v);
          } else if constexpr (STEP == 16) {
            float f[16];
            tmem_ld16(at + u * BN + c, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(f[i]);
          } else {
            tmem_ld8(at + u * BN + c, v);
          }
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < STEP; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(sc + c + i);
            acc[c + i] = fmaf(__uint_as_float(v[i]), f.x, acc[c + i]);
            acc[c + i + 1] = fmaf(__uint_as_float(v[i + 1]), f.y, acc[c + i + 1]);
            acc[c + i + 2] = fmaf(__uint_as_float(v[i + 2]), f.z, acc[c + i + 2]);
            acc[c + i + 3] = fmaf(__uint_as_float(v[i + 3]), f.w, acc[c + i + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tempty[u]);
          mbar_arrive(&sempty[s]);
        }
      }
      if (!ok) break;
      if (p.splits == 1) {
        if (j < p.n) {
#pragma unroll
          for (int i = 0; i < C::COLS; ++i) {
            const int t = t0 + i;
            if (t >= p.m) break;
            float y = acc[i];
            if (p.residual) y += static_cast<float>(static_cast<const T *>(p.residual)[t * p.residual_row + j]);
            static_cast<T *>(p.y)[t * p.y_row + j] = static_cast<T>(y);
          }
        }
      } else {
        // (one tile a cluster; its stages have been read)
        float *mine = reinterpret_cast<float *>(sm);
#pragma unroll
        for (int i = 0; i < C::COLS; ++i) mine[(half * C::COLS + i) * 128 + 32 * q + lane] = acc[i];
      }
    }
  }
  if (p.splits > 1) {
    mkw::cluster_arrive();
    mkw::cluster_wait();
    // columns rank, rank + splits, .. of the tile: the CTAs' sums in order
    const int j0 = first % p.tiles_n * 128, t0 = first / p.tiles_n * BN;
    for (int i = threadIdx.x; i < (BN - rank + p.splits - 1) / p.splits * 128; i += kThreads) {
      const int c = rank + i / 128 * p.splits, j = j0 + i % 128, t = t0 + c;
      if (c >= BN || t >= p.m || j >= p.n) continue;
      const float *own = reinterpret_cast<const float *>(sm) + c * 128 + i % 128;
      float y = 0.f;
      for (int r = 0; r < p.splits; ++r) y += load_remote(mkw::remote(own, r));
      if (p.residual) y += static_cast<float>(static_cast<const T *>(p.residual)[t * p.residual_row + j]);
      static_cast<T *>(p.y)[t * p.y_row + j] = static_cast<T>(y);
    }
    mkw::cluster_arrive();                                 // nobody leaves while its sums are read
    mkw::cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::TCOLS);
}

// ---- host side ---------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void *f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// rows of `inner` bytes, `row` apart, in boxes of 128 bytes by box_rows
bool byte_map(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t row, int box_rows) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(row)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, class T>
int launch(const mk_matmul_fp8_args *a, MatmulParams &p, int sms, int dev, cudaStream_t s) {
  using C = Cfg<BN>;
  static mkw::Ready ready[mkw::kMaxDevices];
  const auto fn = &matmul_kernel<BN, T>;
  mkw::Ready &r = ready[dev];
  if (!r.get(reinterpret_cast<const void *>(fn), kThreads, C::SMEM)) return MK_ERR_CUDA;
  CUtensorMap tw, tx;
  if (!byte_map(&tw, a->w, a->k, a->n, a->w_row, 128) || !byte_map(&tx, a->x, a->k, a->m, a->x_row, BN)) return MK_ERR_CUDA;
  const int64_t tiles_n = (a->n + 127) / 128, tiles = tiles_n * ((static_cast<int64_t>(a->m) + BN - 1) / BN);
  if (tiles > INT32_MAX - 65536) return MK_ERR_UNSUPPORTED;
  p.tiles_n = static_cast<int>(tiles_n), p.tiles = static_cast<int>(tiles);
  p.splits = 1;
  for (int i = 0; i < 3 && BN * 128 * 4 <= static_cast<int>(C::SCALES) && tiles * (2 << i) <= sms && p.kb >= 2 * (2 << i) && tiles <= r.clusters[i]; ++i)
    p.splits = 2 << i;
  const int ctas = p.splits > 1 ? p.tiles * p.splits : std::min(p.tiles, sms);
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fn, tw, tx, p) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

template <class T>
int launch_rows(const mk_matmul_fp8_args *a, MatmulParams &p, int sms, int dev, cudaStream_t s) {
  if (a->m <= 16) return launch<16, T>(a, p, sms, dev, s);
  if (a->m <= 64) return launch<64, T>(a, p, sms, dev, s);
  const int64_t tiles = (a->n + 127) / 128 * ((static_cast<int64_t>(a->m) + 255) / 256);
  return tiles < sms ? launch<128, T>(a, p, sms, dev, s) : launch<256, T>(a, p, sms, dev, s);
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
  p.m = a->m, p.k = a->k, p.blocks = (a->k - 1) / kBlock + 1;
  p.items = static_cast<int64_t>(p.m) * p.blocks;
  const int64_t ctas = (p.items - 1) / (kQuantThreads / 16) + 1;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ctas, 32 * sms)));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == MK_F32) return mkw::launch_after(&quantize_kernel<float>, grid, kQuantThreads, 0, s, p);
  return mkw::launch_after(&quantize_kernel<__nv_bfloat16>, grid, kQuantThreads, 0, s, p);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == MK_F32 ? launch_rows<float>(a, p, sms, dev, s) : launch_rows<__nv_bfloat16>(a, p, sms, dev, s);
}
