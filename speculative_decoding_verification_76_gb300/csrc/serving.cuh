// What the kernels of the cache's side of a decoding step share (tables.cu,
// append_tokens.cu, decode.cu).
#pragma once
#include "common.cuh"

// x / d for 0 <= x < 2^31 and a divisor the host knows: with 2^s >= d the
// multiplier m = ceil(2^(31+s) / d) errs by m d - 2^(31+s) < d <= 2^s, and
// x times that error stays below 2^(31+s), so floor(x m / 2^(31+s)) is exact.
// (The compiler's own division by a variable is some twenty instructions, and
// short kernels pay for code they have to fetch.)
struct FastDiv {
  uint32_t mul, shift;
  int d;
  FastDiv() = default;
  explicit FastDiv(int div) : d(div) {
    uint32_t s = 0;
    while (s < 31 && (1u << s) < (uint32_t)div) ++s;
    shift = 31 + s;
    mul = (uint32_t)(((1ull << shift) + div - 1) / div);
  }
  SPEC_DEV int quot(int x) const { return (int)(((uint64_t)(uint32_t)x * mul) >> shift); }
  SPEC_DEV int ceil_quot(int x) const {
    const int q = quot(x);
    return q + (q * d != x);
  }
};

// Programmatic dependent launch: a kernel started by launch_chained is set up while the
// kernel in front of it on the stream still runs, and chain_wait() holds it until that
// kernel is complete and its stores are visible.  EVERY thread runs it before it ends:
// the next operation on the stream waits for this kernel alone, so a grid that ends early
// would let it pass the kernel in front.  Every global access comes after it, but for
// join_kernel's (decode.cu) reads of the lengths: decode_kernel, which releases it, has
// itself waited for whatever wrote them.
// chain_next() lets the next such kernel start early.  It is worth having only where that
// one has work to do before its wait: blocks that merely wait slowed the ones they waited
// for (extend + release 8.4 against 9.7 us, one-token attention 13.1 against 14.1).
SPEC_DEV void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
SPEC_DEV void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename P>
static inline spec_status launch_chained(void (*kernel)(P), int grid, int block, size_t smem,
                                         cudaStream_t st, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) return SPEC_ECUDA;
  return launch_status();
}
