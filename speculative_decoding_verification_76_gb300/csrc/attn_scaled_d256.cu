// verify_attn_scaled for heads of 256 (attn_scaled.cuh).
#include "attn_scaled.cuh"

namespace scaled_attn {
spec_status launch_d256(const Params& p, int rt, bool f16, cudaStream_t st) {
  return launch_d<256>(p, rt, f16, st);
}
}  // namespace scaled_attn
