// spec_verify_attn_scaled -- attention of a verify block (or of single tokens) over an e4m3 cache
// with one scale for each block of tokens and KV head, on the 5th-generation tensor cores.
//
// Mathematics, for row i and the positions t it sees, with codes k_t, v_t and their blocks' scales
// a_t, c_t:
//   x_t = scale a_t (q . k_t),  out = sum_t e^(x_t) c_t v_t / l,  l = sum_t e^(x_t),  lse = ln l.
// V's scale goes into the weight, w_t = 2^(x_t + log2 c_t - m) with a reference m per row, and
// l = sum w_t / c_t.  So weights stay below 2^8 whatever the scales are, and a row's sum keeps the
// precision of its own largest contribution.  Parts of the positions give (m, l, sum w v) each and
// join by 2^(m_i - M) ("Speculative Token Decoupling: Asynchronous Verification via
// Flash-Decoding", section 03: split-K attention).
//
// What bounds it: HBM up to some 100 query rows per KV head (2 D bytes per position and head are
// read once); the tensor cores and the exponentials above that.
//
// Design.  Both products are taken transposed, positions (or dimensions) as the MMA's 128 rows and
// query rows as its columns, so that a few query rows cost a few columns:
//   S^T = K Q^T: a tile of 128 positions, as it lies in the cache: the codes go to the tensor cores
//     (tcgen05 kind::f8f6f4) as they are, without a conversion.  Q is a sum of e4m3 parts (two hold a
//     bf16 number's 8 bits, three an fp16's 11) under a power of two per row.
//   O^T = V^T W^T: A is the V tile, positions along K.  W is a sum of three 8-bit parts: two e4m3 (the
//     second times 2^4) and one e5m2 (times 2^15), 11 bits down to 2^-27 of a row's largest weight; the
//     parts are columns of their own and are added up at the end.
// In S^T a thread owns one position: its scales are two numbers, unseen positions one comparison,
// and the sum over positions is left to the end.  The reference of a row moves only when a weight
// passes 2^8 (one vote a tile); then O is rescaled in tensor memory.
//
// A CTA (one per SM) takes up to 64 query rows of a KV head and one contiguous range of (KV head, batch's
// positions), cut evenly in tiles of 128 over all SMs on the device, so that ragged batches, one long
// sequence and captured graphs whose lengths change fill the GPU alike.  Four copy warps stream K, V and
// their scales into a ring of stages (16-byte cp.async, zeros where nothing is seen) and run ahead
// over the ends of sequences; one thread issues the MMAs; eight warps turn scores into weights.
// Sequences cut over several CTAs leave parts, joined by a second kernel in their order.
//
// What is seen by some rows only (block rows, the edge of a window) gets weight 0 elsewhere; as 0 times a
// NaN code would be NaN, such tiles' NaN codes of V are zeroed and noted per row.
#pragma once
#include <cuda_fp16.h>

#include "scaled.cuh"
#include "tc_ptx.cuh"

namespace scaled_attn {

constexpr int kUnit = 128;                       // positions of a tile
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr int kMmaWarp = kSoftWarps, kCopyWarp0 = kMmaWarp + 1, kCopyWarps = 4;
constexpr int kCopy = 32 * kCopyWarps;
constexpr int kThreads = 32 * (kCopyWarp0 + kCopyWarps);
constexpr float kTop = 8.f;                      // weights stay at or below 2^8 ...
constexpr float kBelow = 2.f;                    // ... and begin at 2^2
constexpr float kNone = -1e30f;                  // the reference of a row that has seen nothing
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const char *q, *k, *v;
  const float *ks, *vs;
  const int32_t *table, *ctx;
  const uint64_t* mask;
  char* out;
  float *lse, *part_o, *part_ml;
  int32_t* err;
  long long q_stride_b, q_stride_r, q_stride_h;       // elements
  long long page_stride, token_stride, head_stride;   // bytes
  FastDiv P, block;
  int B, R, Hq, Hkv, G, num_pages, max_pages, window;
  int tiles, rows_per_tile, teams;   // row tiles of a KV head, their query rows; ranges
  float scale_log2;
  uint64_t wait_ns;
  int withhold_stage;
};

__device__ const float g_unseen = -INFINITY;  // K's scale of a position that is not there

struct Seq {  // positions first .. end - 1 of a sequence are looked at
  int ctx, first, end, units;
};

SPEC_DEV Seq seq_of(const Params& p, int b) {
  Seq s;
  s.ctx = p.ctx[b];
  const long long end = min((long long)s.ctx + p.R, (long long)p.max_pages * p.P.d);
  s.end = s.ctx < 0 ? 0 : (int)end;
  s.first = p.window > 0 && s.ctx > p.window ? s.ctx - p.window : 0;
  s.units = s.end > s.first ? (s.end - s.first + kUnit - 1) / kUnit : 0;
  return s;
}

// The ranges that `total` units are cut into: the first total % n have one more.
struct Ranges {
  int n, q, rem;
  SPEC_DEV Ranges(int total, int teams)
      : n(min(teams, total)), q(n ? total / n : 0), rem(n ? total - q * n : 0) {}
  SPEC_DEV int begin(int r) const { return r * q + min(r, rem); }
  SPEC_DEV int of(int unit) const {
    const int longer = rem * (q + 1);
    return unit < longer ? unit / (q + 1) : rem + (unit - longer) / q;
  }
};

// A walk over the segments (pieces of one sequence of one KV head) of a range.
struct Walk {
  int W, s, s1, kvh, b, at;  // batch's units; next unit and end; where it lies
  Seq seq;
  SPEC_DEV bool more() const { return s < s1; }
  SPEC_DEV int first_unit() const { return s - kvh * W - at; }
  SPEC_DEV int count() const { return min(seq.units - first_unit(), s1 - s); }
  SPEC_DEV void next(const Params& p) {
    s += count();
    if (s >= s1) return;
    at += seq.units;
    do {
      if (++b == p.B) b = 0, at = 0, ++kvh;
      seq = seq_of(p, b);
    } while (seq.units == 0);
  }
};

// ---------------------------------------------------------------- tensor-core pieces
// Shared-memory matrix descriptor with a layout type (0: none, 2: 128-byte, 4: 64-byte swizzle).
SPEC_DEV uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}

// kind::f8f6f4 with an e4m3 A and an fp32 accumulator; B e4m3 (0) or e5m2 (1).
constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool mn_major) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((mn_major ? 3u : 0u) << 15) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

SPEC_DEV void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
SPEC_DEV void tmem_ld(uint32_t addr, uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "columns");
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  else if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  else
    tmem_ld32(addr, *reinterpret_cast<uint32_t(*)[32]>(r));
}

SPEC_DEV void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// A barrier of the soft warps that ORs a predicate.
SPEC_DEV bool soft_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kSoft)
      : "memory");
  return r != 0;
}
SPEC_DEV void soft_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoft) : "memory"); }

// Columns combined over a warp's lanes in about N shuffles: lane holds column (lane * N / 32 ...)
// of the result, N = 8, 16 or 32; returns the column that this lane's result belongs to.
template <int N, class Op>
SPEC_DEV float over_lanes(float* x, int lane, Op op, int* column) {
  int col = 0;
#pragma unroll
  for (int n = N / 2, o = 16; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
      x[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
    col += up ? n : 0;
  }
#pragma unroll
  for (int o = 16 / N; o >= 1; o /= 2) x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], o));
  *column = col;
  return x[0];
}

SPEC_DEV uint32_t f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
SPEC_DEV uint32_t e4m3x2(uint32_t h2) {  // two halves to two codes (low 16 bits)
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
SPEC_DEV uint32_t e5m2x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
SPEC_DEV uint32_t halves_of(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
SPEC_DEV uint32_t sub_mul(uint32_t a, uint32_t b, uint32_t mul) {  // (a - b) * mul, halves
  uint32_t r;
  asm("{\n .reg .b32 t;\n sub.rn.f16x2 t, %1, %2;\n mul.rn.f16x2 %0, t, %3;\n}\n"
      : "=r"(r)
      : "r"(a), "r"(b), "r"(mul));
  return r;
}

SPEC_DEV uint32_t nan_bytes(uint32_t w) {  // bit 7 of every byte that is a NaN code
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// ---------------------------------------------------------------- shapes
template <int D, int RT, bool F16>
struct Shape {
  static constexpr int kRowBytes = D <= 128 ? D : 128;          // of a swizzled row
  static constexpr int kHalves = D / kRowBytes;                 // column halves of a tile
  static constexpr uint32_t kLayout = D == 64 ? 4 : 2;
  static constexpr uint32_t kGroup = 8 * kRowBytes;             // bytes of 8 rows
  static constexpr int kTileBytes = kUnit * D;
  static constexpr int kParts = F16 ? 3 : 2;                    // of Q
  static constexpr int kStageBytes = 2 * kTileBytes + 1024;     // V, K, scales
  static constexpr int kQBytes = kParts * RT * D;
  static constexpr int kPBytes = 3 * RT * kUnit;
  static constexpr int kPBufs = D == 256 && RT == 64 ? 1 : 2;
  static constexpr int kFixed = kQBytes + kPBufs * kPBytes + 1024;
  static constexpr int kRoom = 225 * 1024 - 8 * 1024 - kFixed;  // (static shared memory: < 8 KB)
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static_assert(kStages >= 2, "a ring needs two stages");
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static constexpr int kHalfCols = 3 * RT;                      // of O, per 128 dimensions
  static constexpr int kColS = 0, kColO = 2 * RT;
  static constexpr int kCols = kColO + kHalfCols * (D == 256 ? 2 : 1);
  static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "tensor memory");
};

// Byte of 16-byte chunk c of row r in a tile of `rows` rows.
template <int D>
SPEC_DEV uint32_t swizzled(int rows, int r, int c) {
  if constexpr (D == 64) return r * 64 + ((c ^ (r >> 1 & 3)) << 4);
  return (uint32_t)(c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <int D, int RT, bool F16>
__global__ void __launch_bounds__(kThreads, 1) attn_scaled_kernel(
    const __grid_constant__ Params p) {
  using S = Shape<D, RT, F16>;
  constexpr int NC = RT / 2;  // columns of a soft warp
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], s_full[2], p_full[2], pv_done[2], q_full, fin;
  __shared__ __align__(16) float sc_s[RT], neg_m[RT], fac_s[RT], red[kSoftWarps][NC];
  __shared__ uint64_t see_s[RT];
  __shared__ int from_s[RT];
  __shared__ uint32_t nan_s[RT][D / 32];
  __shared__ Walk start;
  __shared__ uint32_t tmem_base;
  __shared__ int part_w[kThreads / 32], any_nan;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;  // stages first: whole swizzle atoms
  const uint32_t q_at = base + NS * S::kStageBytes;
  uint8_t* const dyn0 = dyn + (base - smem_u32(dyn));

  chain_wait();
  // ---- this CTA's range, and the sequence it begins in: each thread sums consecutive sequences
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += seq_of(p, b).units;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part_w[warp] = x;
    __syncthreads();
    int before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += part_w[w];
      W += part_w[w];
    }
    const Ranges ranges(W * p.Hkv, p.teams);
    if (team >= ranges.n) return;
    const int s0 = ranges.begin(team), kvh = s0 / W, u = s0 - kvh * W;
    int at = before + x - mine;
    if (at <= u && u < at + mine) {
      int b = b0;
      Seq seq = seq_of(p, b);
#pragma unroll 1
      while (at + seq.units <= u) at += seq.units, seq = seq_of(p, ++b);
      start = {W, s0, ranges.begin(team + 1), kvh, b, at, seq};
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&full[i], kCopy);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], kSoft);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(&q_full, kSoft);
      mbar_init(&fin, 1);
      fence_mbar_init();
    }
    if (warp == kMmaWarp) {
      tmem_alloc(&tmem_base, S::kAlloc);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = tmem_base;
  const uint32_t p_at = q_at + S::kQBytes;

  if (warp >= kCopyWarp0) {
    // ================================================================ copy warps
    constexpr int L = D / 16, kRows = 32 / L;  // lanes of a row; rows of one instruction
    const int pt = threadIdx.x - 32 * kCopyWarp0, w = pt >> 5;
    const int sub = lane / L, chunk = lane % L;
    uint64_t pol;
    if (p.tiles == 1)  // the only reader of these rows
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    else
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    const int nb = p.P.d / p.block.d;
    int g = 0;
    bool ok = true;
    for (Walk walk = start; walk.more() && ok; walk.next(p)) {
      const int n = walk.count();
      int t = walk.seq.first + walk.first_unit() * kUnit + pt;
      const int32_t* bt = p.table + (size_t)walk.b * p.max_pages;
      const char* kh = p.k + walk.kvh * p.head_stride;
      const char* vh = p.v + walk.kvh * p.head_stride;
      int id = t < walk.seq.end ? bt[p.P.quot(t)] : -1;
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++g, t += kUnit) {
        const int stage = g % NS;
        const int off = t - p.P.quot(t) * p.P.d;
        const bool here = id >= 0 && id < p.num_pages;
        const long long row = here ? id * p.page_stride + off * p.token_stride : -1;
        const long long sc = here ? ((long long)id * nb + p.block.quot(off)) * p.Hkv + walk.kvh : 0;
        const int tn = t + kUnit;
        id = j + 1 < n && tn < walk.seq.end ? bt[p.P.quot(tn)] : -1;
        // (the warp as one: the shuffles below need every lane)
        if (g >= NS)
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], ((g / NS) - 1) & 1, p.err, p.wait_ns));
        if (!ok) break;
        const uint32_t v_at = base + stage * S::kStageBytes, k_at = v_at + S::kTileBytes;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const int r = i * kRows + sub;
          const long long from = __shfl_sync(0xffffffffu, row, r);
          const uint32_t to = swizzled<D>(kUnit, w * 32 + r, chunk), bytes = from >= 0 ? 16u : 0u;
          const long long at = (from >= 0 ? from : 0) + chunk * 16;
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(
                           k_at + to),
                       "l"(kh + at), "r"(bytes), "l"(pol)
                       : "memory");
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(
                           v_at + to),
                       "l"(vh + at), "r"(bytes), "l"(pol)
                       : "memory");
        }
        const uint32_t s_at = v_at + 2 * S::kTileBytes + pt * 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at),
                     "l"(here ? p.ks + sc : &g_unseen)
                     : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at + 512),
                     "l"(here ? p.vs + sc : &g_unseen)
                     : "memory");
        if (g != p.withhold_stage)  // (a test can withhold one: its waiters time out)
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&full[stage]))
                       : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kMmaWarp) {
    // ================================================================ the MMA thread
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_f8(128, RT, false, false);
      constexpr uint32_t kIdP = idesc_f8(128, 2 * RT, false, true);
      constexpr uint32_t kIdL = idesc_f8(128, RT, true, true);
      int g = 0, seg = 0;
      bool ok = true;
      // O^T (+)= V^T W^T of unit u
      auto pv = [&](int u, bool first) {
        if (!mbar_wait(&p_full[u & 1], u >> 1 & 1, p.err, p.wait_ns)) return false;
        tc_fence_after();
        const uint32_t v_at = base + u % NS * S::kStageBytes;
        const uint32_t w_at = p_at + (S::kPBufs == 2 ? u & 1 : 0) * S::kPBytes;
#pragma unroll
        for (int half = 0; half < (D == 256 ? 2 : 1); ++half)
#pragma unroll
          for (int k = 0; k < kUnit / 32; ++k) {
            // (D = 64: the rows behind the tile's 64 are the K tile's, and are not used)
            const uint64_t a = smem_desc(v_at + half * (kUnit * 128) + k * 4 * S::kGroup,
                                         D == 64 ? S::kTileBytes : 16384, S::kGroup, S::kLayout);
            const uint32_t d = tmem + S::kColO + half * S::kHalfCols;
            const uint32_t acc = !first || k > 0;
            mma_f8(d, a, smem_desc(w_at + k * 512, 128, 2048, 0), kIdP, acc);
            mma_f8(d + 2 * RT, a, smem_desc(w_at + 2 * RT * kUnit + k * 512, 128, 2048, 0), kIdL, acc);
          }
        tc_commit(&empty[u % NS]);
        tc_commit(&pv_done[u & 1]);
        return true;
      };
      for (Walk walk = start; walk.more() && ok; walk.next(p), ++seg) {
        const int n = walk.count();
        if (!mbar_wait(&q_full, seg & 1, p.err, p.wait_ns)) break;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j, ++g) {
          const int stage = g % NS;
          if (!(ok = mbar_wait(&full[stage], (g / NS) & 1, p.err, p.wait_ns))) break;
          fence_proxy_async();  // the copies' writes, for the tensor cores
          tc_fence_after();
          const uint32_t k_at = base + stage * S::kStageBytes + S::kTileBytes;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint32_t in = D == 64 ? k * 32 : (k & 3) * 32;
            const uint64_t a = smem_desc(k_at + (k >> 2) * (kUnit * 128) + in, 16, S::kGroup, S::kLayout);
#pragma unroll
            for (int part = 0; part < S::kParts; ++part)
              mma_f8(tmem + S::kColS + (g & 1) * RT, a,
                     smem_desc(q_at + part * RT * D + (k >> 2) * (RT * 128) + in, 16, S::kGroup,
                               S::kLayout),
                     kIdS, k > 0 || part > 0);
          }
          tc_commit(&s_full[g & 1]);
          if (j > 0) ok = pv(g - 1, j == 1);
        }
        if (ok) ok = pv(g - 1, n == 1);
      }
      // nothing of this thread's is in flight when the tensor memory goes
      tc_commit(&fin);
      mbar_wait(&fin, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ================================================================ scores into weights
    const int side = warp >> 2, c0 = side * NC;  // this warp's columns c0 .. c0 + NC - 1
    const int tok = (warp & 3) * 32 + lane;      // a position of the tile, a dimension of O
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const int rows = min(p.rows_per_tile, p.R * p.G - tile * p.rows_per_tile);
    int g = 0, seg = 0;
    bool ok = true;
    for (Walk walk = start; walk.more(); walk.next(p), ++seg) {
      const int b = walk.b, n_units = walk.count(), ctx = walk.seq.ctx;
      // ---- Q as sums of e4m3 parts under a power of two per row
      {
        constexpr int kPer = kSoft / RT;  // threads of a row
        const int n = threadIdx.x / kPer, x0 = threadIdx.x % kPer;
        const int row = tile * p.rows_per_tile + n, i = row / p.G;
        const bool real = n < rows;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (b * p.q_stride_b + (real ? i : 0) * p.q_stride_r +
                   (walk.kvh * p.G + (real ? row - i * p.G : 0)) * p.q_stride_h) * 2);
        auto values = [&](int c, float* x) {
          const uint4 w = real ? src[c] : make_uint4(0, 0, 0, 0);
          const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (F16) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(u + e));
              x[2 * e] = f.x, x[2 * e + 1] = f.y;
            } else {
              x[2 * e] = __uint_as_float(u[e] << 16);
              x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
          }
        };
        float big = 0.f;
        bool bad = false;
#pragma unroll 1
        for (int c = x0; c < D / 8; c += kPer) {
          float x[8];
          values(c, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            big = fmaxf(big, finite_abs(x[e]));
            bad = bad || !(fabsf(x[e]) < INFINITY);
          }
        }
#pragma unroll
        for (int o = 1; o < kPer; o <<= 1) {
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          bad = __shfl_xor_sync(0xffffffffu, (int)bad, o) || bad;
        }
        const float s = needed_scale(big), down = 1.f / s;
#pragma unroll 1
        for (int c = x0; c < D / 8; c += kPer) {
          float x[8];
          values(c, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= down;
          const uint32_t to = q_at - base + swizzled<D>(RT, n, c >> 1) + (c & 1) * 8;
#pragma unroll
          for (int part = 0; part < S::kParts; ++part) {
            const uint2 w = make_uint2(e4m3_word(x[0], x[1], x[2], x[3]),
                                       e4m3_word(x[4], x[5], x[6], x[7]));
            *reinterpret_cast<uint2*>(dyn0 + to + part * RT * D) = w;
            float y[8];
            e4m3_values(w.x, y);
            e4m3_values(w.y, y + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= y[e];
          }
        }
        if (x0 == 0) {
          sc_s[n] = bad ? NAN : real ? p.scale_log2 * s : 0.f;
          neg_m[n] = -kNone;
          uint64_t m = 0;
          if (real) {
            m = p.mask ? p.mask[(size_t)b * p.R + i] : i >= 63 ? ~0ull : (2ull << i) - 1;
            if (p.R < 64) m &= (1ull << p.R) - 1;
          }
          see_s[n] = m;
          from_s[n] = p.window > 0 ? ctx + __popcll(m) - p.window : 0;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) nan_s[n][e] = 0;
        }
        if (threadIdx.x == 0) any_nan = 0;
        fence_proxy_async();
        mbar_arrive(&q_full);
      }
      soft_sync();

      uint64_t l2[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l2[i] = 0ull;
      int t0 = walk.seq.first + walk.first_unit() * kUnit;
#pragma unroll 1
      for (int j = 0; j < n_units; ++j, ++g, t0 += kUnit) {
        const int stage = g % NS;
        ok = ok && mbar_wait(&full[stage], (g / NS) & 1, p.err, p.wait_ns) &&
             mbar_wait(&s_full[g & 1], g >> 1 & 1, p.err, p.wait_ns);
        tc_fence_after();
        uint32_t s[NC];
        tmem_ld<NC>(lanes + S::kColS + (g & 1) * RT + c0, s);
        const float* scales =
            reinterpret_cast<const float*>(dyn0 + stage * S::kStageBytes + 2 * S::kTileBytes);
        float ks = scales[tok], vs = scales[kUnit + tok];
        const bool here = ks != -INFINITY;
        vs = !here ? 1.f : vs < 0x1p-100f ? 0x1p-100f : vs;
        ks = here ? ks : 0.f;
        const float lvs = here ? log2f(vs) : -INFINITY, rvs = here ? 1.f / vs : 0.f;
        // positions that some rows see and others do not
        const bool mixed = (t0 + kUnit > ctx && (p.R > 1 || p.mask)) ||
                           (p.window > 0 && t0 < ctx + p.R - p.window);
        uint32_t see = 0xffffffffu;  // columns that see this thread's position
        if (mixed) {
          const int t = t0 + tok, jb = t - ctx;
          see = 0;
#pragma unroll 1
          for (int c = 0; c < NC; ++c)
            if (jb < 0 ? t >= from_s[c0 + c] : jb < 64 && (see_s[c0 + c] >> jb & 1)) see |= 1u << c;
          // NaN codes of V: noted for the rows that see them, then zeroed
          uint8_t* vrow = dyn0 + stage * S::kStageBytes;
          bool nan = false;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(vrow + swizzled<D>(kUnit, tok, c));
            if (nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w)) {
              nan = true;
              const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
              uint32_t bits = 0;
              for (int e = 0; e < 16; ++e) bits |= (nan_bytes(u[e >> 2]) >> (8 * (e & 3) + 7) & 1) << e;
              for (int x = 0; x < NC; ++x)
                if (see >> x & 1) atomicOr(&nan_s[c0 + x][c >> 1], bits << 16 * (c & 1));
            }
          }
          if (nan) any_nan = 1;
          soft_sync();
          if (nan && side == 0) {
            for (int c = 0; c < D / 16; ++c) {
              uint4* w = reinterpret_cast<uint4*>(vrow + swizzled<D>(kUnit, tok, c));
              uint32_t* u = reinterpret_cast<uint32_t*>(w);
              for (int e = 0; e < 4; ++e) u[e] &= ~((nan_bytes(u[e]) >> 7) * 255u);
            }
          }
        }
        tmem_wait_ld();
        // ---- exponents, relative to the rows' references
        const uint64_t ks2 = f2_pack(ks, ks), lvs2 = f2_pack(lvs, lvs);
        const uint64_t* sc2 = reinterpret_cast<const uint64_t*>(sc_s + c0);
        const uint64_t* nm2 = reinterpret_cast<const uint64_t*>(neg_m + c0);
        float a[NC];
        auto exponents = [&]() {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const uint64_t x =
                f2_mul(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2[i]);
            f2_unpack(f2_fma(x, ks2, f2_add(lvs2, nm2[i])), a[2 * i], a[2 * i + 1]);
            if (mixed) {
              a[2 * i] = see >> (2 * i) & 1 ? a[2 * i] : -INFINITY;
              a[2 * i + 1] = see >> (2 * i + 1) & 1 ? a[2 * i + 1] : -INFINITY;
            }
            top = fmax3(top, a[2 * i], a[2 * i + 1]);
          }
          return top;
        };
        const float top = exponents();
        if (soft_any(top > kTop || !ok)) {
          if (soft_any(!ok)) break;  // (the same for all: everyone leaves the tile loop)
          // ---- the references move: maxima over the tile's positions
          float x[NC];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            x[i] = __uint_as_float(s[i]) * sc_s[c0 + i] * ks + lvs;
            if (mixed && !(see >> i & 1)) x[i] = -INFINITY;
          }
          int col;
          const float m = over_lanes<NC>(x, lane, [](float u, float v) { return fmaxf(u, v); }, &col);
          red[warp][col] = m;
          soft_sync();
          if (threadIdx.x < RT) {
            const int n = threadIdx.x, w0 = n / NC * 4, c = n % NC;
            float m4 = fmaxf(fmaxf(red[w0][c], red[w0 + 1][c]), fmaxf(red[w0 + 2][c], red[w0 + 3][c]));
            const float old = -neg_m[n], now = m4 - old > kTop ? m4 - kBelow : old;
            fac_s[n] = fast_exp2(old - now);
            neg_m[n] = -now;
          }
          soft_sync();
#pragma unroll
          for (int i = 0; i < NC / 2; ++i)
            l2[i] = f2_mul(l2[i], reinterpret_cast<const uint64_t*>(fac_s + c0)[i]);
          if (j > 0) {
            ok = mbar_wait(&pv_done[(g - 1) & 1], (g - 1) >> 1 & 1, p.err, p.wait_ns);
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < (D == 256 ? 6 : 3); ++part)
#pragma unroll
              for (int c = 0; c < NC; c += 8) {
                const uint32_t at = lanes + S::kColO + part * RT + c0 + c;
                uint32_t o[8];
                tmem_ld<8>(at, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * fac_s[c0 + c + e]);
                tmem_st8(at, o);
              }
            tmem_wait_st();
          }
          exponents();
        }
        // ---- weights, their sums, and their three parts
        if constexpr (S::kPBufs == 1)
          if (j > 0)
            ok = ok && mbar_wait(&pv_done[(g - 1) & 1], (g - 1) >> 1 & 1, p.err, p.wait_ns);
        const uint64_t rvs2 = f2_pack(rvs, rvs);
        uint8_t* w_at = dyn0 + (p_at - base) + (S::kPBufs == 2 ? g & 1 : 0) * S::kPBytes +
                        (c0 >> 4) * 2048 + tok * 16 + (c0 & 15);
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint32_t p1[2], p2[2], p3[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = c + 2 * e;
            const float w0 = fast_exp2(a[i]), w1 = fast_exp2(a[i + 1]);
            l2[i / 2] = f2_fma(f2_pack(w0, w1), rvs2, l2[i / 2]);
            const uint32_t h = f16x2(w0, w1), x1 = e4m3x2(h);
            const uint32_t r1 = sub_mul(h, halves_of(x1), 0x4c004c00u);   // times 2^4
            const uint32_t x2 = e4m3x2(r1);
            const uint32_t x3 = e5m2x2(sub_mul(r1, halves_of(x2), 0x68006800u));  // times 2^11
            if (e & 1) {
              p1[e >> 1] |= x1 << 16, p2[e >> 1] |= x2 << 16, p3[e >> 1] |= x3 << 16;
            } else {
              p1[e >> 1] = x1, p2[e >> 1] = x2, p3[e >> 1] = x3;
            }
          }
          uint8_t* to = w_at + (c >> 4) * 2048 + (c & 15);
          *reinterpret_cast<uint2*>(to) = make_uint2(p1[0], p1[1]);
          *reinterpret_cast<uint2*>(to + RT * kUnit) = make_uint2(p2[0], p2[1]);
          *reinterpret_cast<uint2*>(to + 2 * RT * kUnit) = make_uint2(p3[0], p3[1]);
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&p_full[g & 1]);
      }
      // ---- the segment's sums and outputs
      ok = ok && mbar_wait(&pv_done[(g - 1) & 1], (g - 1) >> 1 & 1, p.err, p.wait_ns);
      if (soft_any(!ok)) break;
      tc_fence_after();
      {
        float l[NC];
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) f2_unpack(l2[i], l[2 * i], l[2 * i + 1]);
        int col;
        const float sum = over_lanes<NC>(l, lane, [](float u, float v) { return u + v; }, &col);
        red[warp][col] = sum;
      }
      soft_sync();
      const Ranges ranges(walk.W * p.Hkv, p.teams);
      const bool whole = n_units == walk.seq.units;
      const size_t part = ((size_t)team * 2 + (walk.s == ranges.begin(team) ? 0 : 1)) * p.tiles + tile;
#pragma unroll 1
      for (int c = 0; c < NC; c += 8) {
        if (c0 + c >= rows) break;
        float l8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          l8[e] = (red[side * 4][c + e] + red[side * 4 + 1][c + e]) +
                  (red[side * 4 + 2][c + e] + red[side * 4 + 3][c + e]);
#pragma unroll
        for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
          uint32_t o1[8], o2[8], o3[8];
          const uint32_t at = lanes + S::kColO + half * S::kHalfCols + c0 + c;
          tmem_ld<8>(at, o1);
          tmem_ld<8>(at + RT, o2);
          tmem_ld<8>(at + 2 * RT, o3);
          tmem_wait_ld();
          const int d = half * 128 + tok;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int n = c0 + c + e;
            if (n >= rows || d >= D) continue;
            float y = __uint_as_float(o1[e]) +
                      (__uint_as_float(o2[e]) * 0x1p-4f + __uint_as_float(o3[e]) * 0x1p-15f);
            if (any_nan && nan_s[n][d >> 5] >> (d & 31) & 1) y = NAN;
            if (whole) {
              const int row = tile * p.rows_per_tile + n, i = row / p.G;
              const size_t to = (((size_t)b * p.R + i) * p.Hq + walk.kvh * p.G + row - i * p.G) * D + d;
              y = l8[e] == 0.f ? 0.f : y / l8[e];
              if constexpr (F16) reinterpret_cast<__half*>(p.out)[to] = __float2half_rn(y);
              else reinterpret_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(y);
            } else {
              p.part_o[(part * RT + n) * D + d] = y;
            }
          }
        }
        if (tok < 8 && c0 + c + tok < rows) {
          const int n = c0 + c + tok;
          float lx = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) lx = e == tok ? l8[e] : lx;
          const float m = -neg_m[n];
          if (!whole) {
            *reinterpret_cast<float2*>(p.part_ml + (part * RT + n) * 2) = make_float2(m, lx);
          } else if (p.lse) {
            const int row = tile * p.rows_per_tile + n, i = row / p.G;
            p.lse[((size_t)b * p.R + i) * p.Hq + walk.kvh * p.G + row - i * p.G] =
                lx == 0.f ? -INFINITY : (m + log2f(lx)) * kLn2;
          }
        }
      }
      tc_fence_before();
      soft_sync();  // the rows' state is free
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, S::kAlloc);
}

// The sequences that lie in more than one range (and rows that see nothing): a warp joins a row's parts, in
// their order.
constexpr int kJoinWarps = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p, int RT) {
  constexpr int kPer = D / 32;
  __shared__ int sums[kJoinWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = (p.R * p.Hq + kJoinWarps - 1) / kJoinWarps;
  const int b = blockIdx.x / per_seq, r = blockIdx.x % per_seq * kJoinWarps + warp;
  chain_wait();
  int before = 0, W = 0;
  for (int x = threadIdx.x; x < p.B; x += 32 * kJoinWarps) {
    const int u = seq_of(p, x).units;
    W += u;
    if (x < b) before += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    W += __shfl_xor_sync(0xffffffffu, W, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) sums[warp][0] = W, sums[warp][1] = before;
  __syncthreads();
  W = before = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) W += sums[w][0], before += sums[w][1];
  if (r >= p.R * p.Hq) return;
  const int i = r / p.Hq, h = r % p.Hq, kvh = h / p.G, row = i * p.G + h % p.G;
  const size_t at = (size_t)b * p.R * p.Hq + r;
  const int units = seq_of(p, b).units;
  float acc[kPer], M = kNone, L = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
  if (units > 0) {
    const Ranges ranges(W * p.Hkv, p.teams);
    const int u0 = kvh * W + before, first = ranges.of(u0), np = ranges.of(u0 + units - 1) - first + 1;
    if (np == 1) return;  // written whole
    const int tile = row / p.rows_per_tile, n = row % p.rows_per_tile;
    const bool late = ranges.begin(first) != u0;
    auto part = [&](int x) {
      return (((size_t)(first + x) * 2 + (x == 0 && late)) * p.tiles + tile) * RT + n;
    };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    for (int x = lane; x < np; x += 32) M = fmaxf(M, __ldcg(ml + part(x)).x);
    M = warp_max(M);
    constexpr int kFlight = 8;
#pragma unroll 1
    for (int x0 = 0; x0 < np; x0 += kFlight) {
      float y[kFlight][kPer], e[kFlight];
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        const size_t from = part(min(x0 + x, np - 1));
        const float2 w = __ldcg(ml + from);
        e[x] = x0 + x < np ? fast_exp2(w.x - M) : 0.f;
        L += e[x] * w.y;
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(p.part_o + from * D + kPer * lane + c));
          y[x][c] = v.x, y[x][c + 1] = v.y;
        }
      }
#pragma unroll
      for (int x = 0; x < kFlight; ++x)
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] += x0 + x < np ? e[x] * y[x][c] : 0.f;
    }
  }
  const float f = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int c = 0; c < kPer; c += 2) {
    const float y0 = L == 0.f ? 0.f : acc[c] * f, y1 = L == 0.f ? 0.f : acc[c + 1] * f;
    reinterpret_cast<uint32_t*>(p.out)[(at * D + kPer * lane + c) / 2] =
        F16 ? f16x2(y0, y1) : pack_bf16(y0, y1);
  }
  if (lane == 0 && p.lse) p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------- host side
template <int D, int RT, bool F16>
spec_status launch_one(const Params& p, cudaStream_t st) {
  using S = Shape<D, RT, F16>;
  static PerDeviceOnce<int> once;
  const spec_status rc =
      ensure_smem_limit(once, (const void*)attn_scaled_kernel<D, RT, F16>, S::kSmem);
  if (rc != SPEC_OK) return rc;
  return launch_chained(attn_scaled_kernel<D, RT, F16>, p.teams * p.tiles, kThreads, S::kSmem, st, p);
}

// rt: 16, 32 or 64 query rows of a CTA.  Each D is a translation unit of its own.
template <int D>
spec_status launch_d(const Params& p, int rt, bool f16, cudaStream_t st) {
  spec_status rc;
  if (f16)
    rc = rt == 16 ? launch_one<D, 16, true>(p, st)
                  : rt == 32 ? launch_one<D, 32, true>(p, st) : launch_one<D, 64, true>(p, st);
  else
    rc = rt == 16 ? launch_one<D, 16, false>(p, st)
                  : rt == 32 ? launch_one<D, 32, false>(p, st) : launch_one<D, 64, false>(p, st);
  if (rc != SPEC_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * ((p.R * p.Hq + kJoinWarps - 1) / kJoinWarps), 1, 1);
  cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = f16 ? cudaLaunchKernelEx(&cfg, join_kernel<D, true>, p, rt)
                            : cudaLaunchKernelEx(&cfg, join_kernel<D, false>, p, rt);
  return e == cudaSuccess ? launch_status() : SPEC_ECUDA;
}

spec_status launch_d64(const Params& p, int rt, bool f16, cudaStream_t st);
spec_status launch_d128(const Params& p, int rt, bool f16, cudaStream_t st);
spec_status launch_d256(const Params& p, int rt, bool f16, cudaStream_t st);

}  // namespace scaled_attn
