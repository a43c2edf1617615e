// verify_attn_scaled for heads of 128 (attn_scaled.cuh).
#include "attn_scaled.cuh"

namespace scaled_attn {
spec_status launch_d128(const Params& p, int rt, bool f16, cudaStream_t st) {
  return launch_d<128>(p, rt, f16, st);
}
}  // namespace scaled_attn
