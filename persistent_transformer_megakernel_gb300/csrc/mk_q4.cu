// mk_matvec_q4: the checks of a call, and the kernel for fp32 x.
#include "mk_q4.cuh"

#include "mk_paged.h"

namespace mkq {

constexpr int kMaxK = 32768;           // an fp32 row's two columns of this length still fit

int run_f32(Q4Params &p, int group, int sms, int dev, cudaStream_t s) { return run<float>(p, group, sms, dev, s); }

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
  p.m = a->m, p.n = a->n, p.k = a->k, p.groups = a->k / a->group;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == MK_F32 ? run_f32(p, a->group, sms, dev, s) : run_bf16(p, a->group, sms, dev, s);
}
