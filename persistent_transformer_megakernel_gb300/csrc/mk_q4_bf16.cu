// The 4-bit matrix-vector products' kernel for bf16 x.
#include "mk_q4.cuh"

namespace mkq {

int run_bf16(Q4Params &p, int group, int sms, int dev, cudaStream_t s) { return run<__nv_bfloat16>(p, group, sms, dev, s); }

}  // namespace mkq
