// Warp-level building blocks of the batched serving kernels: 16x8x16 matrix
// products of bf16 or fp16 operands with fp32 accumulators, matrix loads from
// shared memory, 16-byte asynchronous copies and the splitting of fp32 values
// into sums of 16-bit terms.
//
// Fragment layout of a 16x8x16 product (lane = 4 g + t): A holds rows g and
// g + 8 at k = 2t, 2t+1 (a0, a1) and 2t+8, 2t+9 (a2, a3); B column g at the same
// k (b0, b1); C rows g (c0, c1) and g + 8 (c2, c3) at columns 2t, 2t+1.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace mkw {

// division of 0 <= n < 2^31 by a constant of the call
struct Divisor {
  uint32_t value, mul;
  int shift;
  __host__ void set(int d) {
    value = d;
    shift = 0;
    while ((int64_t{1} << shift) < d) ++shift;
    // n mul / 2^(31 + shift) with mul = 2^(31 + shift) / d rounded up: exact below 2^31
    mul = d == 1 ? 0 : static_cast<uint32_t>(((uint64_t{1} << (31 + shift)) + d - 1) / d);
    --shift;
  }
  __device__ __forceinline__ int quotient(int n) const { return value == 1 ? n : static_cast<int>(__umulhi(n, mul) >> shift); }
};

struct BF16Op {};
struct FP16Op {};

__device__ __forceinline__ void mma(BF16Op, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(FP16Op, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same with a zero accumulator
__device__ __forceinline__ void mma_zero(BF16Op, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_zero(FP16Op, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// four 8x8 matrices of 16-bit elements; lane l passes the address of row l % 8 of matrix l / 8
__device__ __forceinline__ void ldmatrix4(uint32_t *r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t *r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// the transpose of an 8x8 matrix of 16-bit elements held a row a quad: lane 4 g + t has (g, 2t), (g, 2t + 1) before and
// (2t, g), (2t + 1, g) after
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 2^x to 2^-22, 0 for x below -126
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 16 bytes global -> shared; with valid false nothing is read and zeros are written
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// round a pair to 16 bits, the first in the low half, and leave what it lost
__device__ __forceinline__ uint32_t take_term(BF16Op, float &x, float &y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t take_term(FP16Op, float &x, float &y) {
  const __half2 h = __floats2half2_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// the same for values from outside, bf16 terms by truncation: the largest finite values stay finite, three terms hold
// all 24 bits of an fp32 value, and an infinity is its first term alone
__device__ __forceinline__ uint32_t take_input_term(BF16Op, float &x, float &y) {
  const uint32_t a = __float_as_uint(x) & 0xffff0000u, b = __float_as_uint(y) & 0xffff0000u;
  x = isinf(x) ? 0.f : x - __uint_as_float(a);
  y = isinf(y) ? 0.f : y - __uint_as_float(b);
  return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t take_input_term(FP16Op, float &x, float &y) {
  const __half2 h = __floats2half2_rn(x, y);
  x = isinf(x) ? 0.f : x - __low2float(h);
  y = isinf(y) ? 0.f : y - __high2float(h);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// a term, not the last, of a value that may meet an infinity: what remains of a value that is not zero is not zero either
// (an infinity times it would be NaN) but of its sign, 2^-30 of the term where nothing remains: below fp32's last place
// whatever the value is multiplied by.  Zero stays zero.
constexpr float kNothingLeft = 0x1p-30f;
__device__ __forceinline__ uint32_t take_query_term(BF16Op, float &x, float &y) {
  const uint32_t a = __float_as_uint(x) & 0xffff0000u, b = __float_as_uint(y) & 0xffff0000u;
  const float fa = __uint_as_float(a), fb = __uint_as_float(b);
  x = x == fa ? fa * kNothingLeft : x - fa;
  y = y == fb ? fb * kNothingLeft : y - fb;
  return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t take_query_term(FP16Op op, float &x, float &y) { return take_input_term(op, x, y); }
// a term of probabilities (>= 0), not the last: by truncation, so that no remainder is negative
__device__ __forceinline__ uint32_t take_weight_term(BF16Op, float &x, float &y) {
  const uint32_t a = __float_as_uint(x) & 0xffff0000u, b = __float_as_uint(y) & 0xffff0000u;
  const float fa = __uint_as_float(a), fb = __uint_as_float(b);
  x = fmaxf(x - fa, fa * kNothingLeft);
  y = fmaxf(y - fb, fb * kNothingLeft);
  return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t take_weight_term(FP16Op op, float &x, float &y) { return take_term(op, x, y); }

// four e4m3 values (lowest byte first) as two pairs of fp16 values: exact
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// 4 bytes; with valid false nothing is read and zeros are written
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}

// Programmatic dependent launch: the first statement of every kernel here, before it reads or writes anything.  The next
// kernel of the stream, if it is launched so too, may be set up from now on; what the previous one did is seen after it.
__device__ __forceinline__ void follow_previous_kernel() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

// the same in two parts, for what a kernel can set up before it looks at memory (not tensor memory: a CTA of the previous
// kernel may still have to get its own)
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// a cluster's CTAs: all their threads meet, shared memory written before is seen after
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the shared memory of the cluster's CTA `rank` at the place of `p` in this one, and a store there
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_remote(uint32_t at, float x) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory"); }

}  // namespace mkw
