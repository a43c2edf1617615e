// verify_attn_scaled for heads of 64 (attn_scaled.cuh).
#include "attn_scaled.cuh"

namespace scaled_attn {
spec_status launch_d64(const Params& p, int rt, bool f16, cudaStream_t st) {
  return launch_d<64>(p, rt, f16, st);
}
}  // namespace scaled_attn
