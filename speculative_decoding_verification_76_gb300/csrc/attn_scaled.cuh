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
constexpr int kGroup = 128;                      // threads of a soft group: one per position
constexpr int kSoftWarps = 8, kSoft = 2 * kGroup;
constexpr int kScoreWarp = kSoftWarps, kSumWarp = kScoreWarp + 1;  // one thread each issues MMAs
constexpr int kCopyWarp0 = kSumWarp + 1, kCopyWarps = 2;
constexpr int kCopy = 32 * kCopyWarps;
constexpr int kThreads = 32 * (kCopyWarp0 + kCopyWarps);
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
// Shared-memory matrix descriptors as two words: the lower has the address / 16 (a step of n bytes adds
// n / 16) and the leading byte offset / 16, the upper the stride byte offset / 16, the version and the
// layout type (0: none, 2: 128-byte, 4: 64-byte swizzle).
SPEC_DEV uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return saddr >> 4 | (lbo >> 4) << 16; }
constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) { return sbo >> 4 | 1u << 14 | layout << 29; }

// kind::f8f6f4 with an e4m3 A and an fp32 accumulator; B e4m3 (0) or e5m2 (1).
constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool mn_major) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((mn_major ? 3u : 0u) << 15) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

SPEC_DEV void mma_f8(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                     uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " setp.ne.b32 p, %6, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// kind::f16 with fp16 operands, both with M / N contiguous, and an fp32 accumulator.
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (3u << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

SPEC_DEV void mma_f16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                      uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " setp.ne.b32 p, %6, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
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

// Barrier `id` of n threads that ORs a predicate; the soft groups have 1 and 2, both together 3.
SPEC_DEV bool any_of(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
SPEC_DEV void sync_of(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

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
  static constexpr uint32_t kLayout = D == 64 ? 4 : 2;
  static constexpr uint32_t kRows8 = 8 * kRowBytes;             // bytes of 8 rows
  static constexpr int kTileBytes = kUnit * D;
  static constexpr int kParts = F16 ? 3 : 2;                    // of Q
  // V as fp16, converted in shared memory, and the weights with it; else (no room at D = 256) V as it
  // lies, and the weights as three 8-bit parts
  static constexpr bool kHalfV = D <= 128;
  static constexpr int kSums = kHalfV ? 1 : 3;                  // columns of O per row and 128 dimensions
  static constexpr int kHalves = D == 256 ? 2 : 1;
  static constexpr int kOCols = kSums * RT * kHalves;
  // weights stay at or below 2^kTop and begin at 2^kBelow
  static constexpr float kTop = kHalfV ? 15.f : 8.f, kBelow = kHalfV ? 8.f : 2.f;
  // Q's parts as columns side by side, added up by the readers, where tensor memory has room: an
  // MMA of 128 x N x 32 takes 61 cycles up to N = 96, and N / 2 above that
  static constexpr bool kStack = 2 * kParts * RT + 2 * kOCols <= 512;
  static constexpr int kSCols = kStack ? kParts * RT : RT;      // of a score buffer
  static constexpr int kStageBytes = 2 * kTileBytes + 1024;     // V, K, scales
  static constexpr int kQBytes = kParts * RT * D;
  static constexpr int kPBytes = kHalfV ? RT * kUnit * 2 : 3 * RT * kUnit;
  static constexpr int kVBytes = kHalfV ? 2 * kTileBytes : 0;
  static constexpr int kFixed = kQBytes + 2 * kPBytes + 2 * kVBytes + 1024;
  static constexpr int kRoom = 225 * 1024 - 8 * 1024 - kFixed;  // (static shared memory: < 8 KB)
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static_assert(kStages >= 2, "a ring needs two stages");
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  // tensor memory: a score buffer and an O for each soft group
  static constexpr int kColO = 2 * kSCols, kCols = kColO + 2 * kOCols;
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
  constexpr int NS = S::kStages;
  constexpr int kC = 16;  // columns that a soft thread works on at a time
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], s_full[2], p_full[2], pv_done[2], q_full, o_full, fin;
  __shared__ __align__(16) float sc_s[RT], neg_m[2][RT], fac_s[2][RT], red[kSoftWarps][RT];
  __shared__ __align__(16) float inv_s[RT];
  __shared__ uint64_t see_s[RT];
  __shared__ long long out_s[RT];  // element of the row's output, or of its part's
  __shared__ int from_s[RT];
  __shared__ uint32_t nan_s[RT][D / 32];
  __shared__ Walk start;
  __shared__ uint32_t tmem_base;
  __shared__ int part_w[kThreads / 32], any_nan;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  // fp16 V, the stages, Q, the weights: whole swizzle atoms
  const uint32_t v16_at = (smem_u32(dyn) + 1023u) & ~1023u, base = v16_at + 2 * S::kVBytes;
  const uint32_t q_at = base + NS * S::kStageBytes, p_at = q_at + S::kQBytes;
  uint8_t* const v16_0 = dyn + (v16_at - smem_u32(dyn));
  uint8_t* const dyn0 = v16_0 + 2 * S::kVBytes;

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
        mbar_init(&empty[i], S::kHalfV ? kGroup : 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], kGroup);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(&q_full, kSoft);
      mbar_init(&o_full, 1);
      mbar_init(&fin, 2);
      fence_mbar_init();
    }
    if (warp == kScoreWarp) {
      tmem_alloc(&tmem_base, S::kAlloc);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = tmem_base;

  if (warp >= kCopyWarp0) {
    // ================================================================ copy warps
    // a lane copies chunks c and c + L of a row (L lanes of a row, 32 / L rows an instruction)
    constexpr int L = D / 32, kRows = 32 / L;
    constexpr int kMine = kUnit / kCopy;       // positions of a lane: 32 apart
    const int w = warp - kCopyWarp0, first = w * 32 * kMine;
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
      int t = walk.seq.first + walk.first_unit() * kUnit + first + lane;
      const int32_t* bt = p.table + (size_t)walk.b * p.max_pages;
      const char* kh = p.k + walk.kvh * p.head_stride;
      const char* vh = p.v + walk.kvh * p.head_stride;
      int id[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m)
        id[m] = t + 32 * m < walk.seq.end ? bt[p.P.quot(t + 32 * m)] : -1;
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++g, t += kUnit) {
        const int stage = g % NS;
        long long row[kMine], sc[kMine];
        uint32_t here[kMine];
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int tm = t + 32 * m, off = tm - p.P.quot(tm) * p.P.d;
          const bool ok_id = id[m] >= 0 && id[m] < p.num_pages;
          here[m] = __ballot_sync(0xffffffffu, ok_id);
          row[m] = ok_id ? id[m] * p.page_stride + off * p.token_stride : 0;
          sc[m] = ((long long)id[m] * nb + p.block.quot(off)) * p.Hkv + walk.kvh;
          const int tn = tm + kUnit;
          id[m] = j + 1 < n && tn < walk.seq.end ? bt[p.P.quot(tn)] : -1;
        }
        // (the warp as one: the shuffles below need every lane)
        if (g >= NS)
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], ((g / NS) - 1) & 1, p.err, p.wait_ns));
        if (!ok) break;
        const uint32_t v_at = base + stage * S::kStageBytes, k_at = v_at + S::kTileBytes;
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
#pragma unroll
          for (int i = 0; i < L; ++i) {
            const int r = i * kRows + sub;
            const long long from = __shfl_sync(0xffffffffu, row[m], r) + chunk * 16;
            const uint32_t bytes = here[m] >> r & 1 ? 16u : 0u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t to = swizzled<D>(kUnit, first + 32 * m + r, chunk + x * L);
              asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(
                               k_at + to),
                           "l"(kh + from + x * L * 16), "r"(bytes), "l"(pol)
                           : "memory");
              asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(
                               v_at + to),
                           "l"(vh + from + x * L * 16), "r"(bytes), "l"(pol)
                           : "memory");
            }
          }
          const uint32_t s_at = v_at + 2 * S::kTileBytes + (first + 32 * m + lane) * 4;
          const bool mine = here[m] >> lane & 1;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at),
                       "l"(mine ? p.ks + sc[m] : &g_unseen)
                       : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at + 512),
                       "l"(mine ? p.vs + sc[m] : &g_unseen)
                       : "memory");
        }
        if (g != p.withhold_stage)  // (a test can withhold one: its waiters time out)
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&full[stage]))
                       : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kScoreWarp) {
    // ================================================================ the scores' MMA thread
    if (lane == 0) {
      constexpr uint32_t kId = idesc_f8(128, S::kSCols, false, false);
      constexpr uint32_t kHi = desc_hi(S::kRows8, S::kLayout);
      // (a part is RT rows: stacked parts are kParts * RT rows of one operand)
      constexpr int kQRows = S::kStack ? S::kParts * RT : RT;
      const uint32_t q_lo = desc_lo(q_at, 16);
      int g = 0, seg = 0;
      bool ok = true;
      for (Walk walk = start; walk.more() && ok; walk.next(p), ++seg) {
        const int n = walk.count();
        if (!mbar_wait(&q_full, seg & 1, p.err, p.wait_ns)) break;
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          const int stage = g % NS;
          // the score buffer's last tile has been read, this tile has landed
          if (g >= 2 && !(ok = mbar_wait(&p_full[g & 1], (g - 2) >> 1 & 1, p.err, p.wait_ns))) break;
          if (!(ok = mbar_wait(&full[stage], (g / NS) & 1, p.err, p.wait_ns))) break;
          fence_proxy_async();  // the copies' writes, for the tensor cores
          tc_fence_after();
          const uint32_t k_lo = desc_lo(base + stage * S::kStageBytes + S::kTileBytes, 16);
          const uint32_t d = tmem + (g & 1) * S::kSCols;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            constexpr int kIn = D == 64 ? 2 : 4;  // steps within a swizzled row
#pragma unroll
            for (int part = 0; part < (S::kStack ? 1 : S::kParts); ++part)
              mma_f8(d, k_lo + ((k / kIn) * (kUnit * 128) + k % kIn * 32) / 16, kHi,
                     q_lo + (part * RT * D + (k / kIn) * (kQRows * 128) + k % kIn * 32) / 16, kHi, kId,
                     k > 0 || part > 0);
          }
          tc_commit(&s_full[g & 1]);
        }
      }
      // nothing of this thread's is in flight when the tensor memory goes
      tc_commit(&fin);
      mbar_wait(&fin, 0, nullptr);
    }
    __syncwarp();
  } else if (warp == kSumWarp) {
    // ================================================================ O^T += V^T W^T
    if (lane == 0) {
      constexpr uint32_t kHi = desc_hi(S::kRows8, S::kLayout), kHiW = desc_hi(2048, 0);
      int g = 0;
      bool ok = true;
      for (Walk walk = start; walk.more() && ok; walk.next(p)) {
        const int n = walk.count();
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          const int stage = g % NS;
          if constexpr (!S::kHalfV) ok = mbar_wait(&full[stage], (g / NS) & 1, p.err, p.wait_ns);
          ok = ok && mbar_wait(&p_full[g & 1], g >> 1 & 1, p.err, p.wait_ns);
          if (!ok) break;
          if constexpr (!S::kHalfV) fence_proxy_async();
          tc_fence_after();
          const uint32_t w_lo = desc_lo(p_at + (g & 1) * S::kPBytes, 128);
          const uint32_t o = tmem + S::kColO + (g & 1) * S::kOCols;
          const uint32_t later = j >= 2;  // this group's O holds something
          if constexpr (S::kHalfV) {
            // (D = 64: rows 64 .. 127 are what lies behind the tile, and are not used)
            constexpr uint32_t kId = idesc_f16(128, RT), kHiV = desc_hi(1024, 2);
            const uint32_t v_lo = desc_lo(v16_at + (g & 1) * S::kVBytes, kUnit * 128);
#pragma unroll
            for (int k = 0; k < kUnit / 16; ++k)
              mma_f16(o, v_lo + k * 2048 / 16, kHiV, w_lo + k * 256 / 16, kHiW, kId, k > 0 ? 1u : later);
          } else {
            constexpr uint32_t kIdP = idesc_f8(128, 2 * RT, false, true);
            constexpr uint32_t kIdL = idesc_f8(128, RT, true, true);
            const uint32_t v_lo = desc_lo(base + stage * S::kStageBytes, 16384);
#pragma unroll
            for (int half = 0; half < S::kHalves; ++half)
#pragma unroll
              for (int k = 0; k < kUnit / 32; ++k) {
                const uint32_t a = v_lo + (half * (kUnit * 128) + k * 4 * S::kRows8) / 16;
                const uint32_t d = o + half * 3 * RT;
                mma_f8(d, a, kHi, w_lo + k * 512 / 16, kHiW, kIdP, k > 0 ? 1u : later);
                mma_f8(d + 2 * RT, a, kHi, w_lo + (2 * RT * kUnit + k * 512) / 16, kHiW, kIdL,
                       k > 0 ? 1u : later);
              }
            tc_commit(&empty[stage]);
          }
          tc_commit(&pv_done[g & 1]);
        }
        if (ok) tc_commit(&o_full);
      }
      tc_commit(&fin);
      mbar_wait(&fin, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ================================================================ scores into weights
    // Two groups of four warps take the tiles in turn, each with references, sums and an O of its
    // own: one tile's chain of waits lies under the other's work.
    const int group = warp >> 2, bar = 1 + group;
    const int tok = (warp & 3) * 32 + lane;      // a position of the tile, a dimension of O
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const int rows = min(p.rows_per_tile, p.R * p.G - tile * p.rows_per_tile);
    const int range0 = start.s;
    int g = 0, seg = 0;
    bool ok = true;
    for (Walk walk = start; walk.more(); walk.next(p), ++seg) {
      const int b = walk.b, n_units = walk.count(), ctx = walk.seq.ctx;
      const bool whole = n_units == walk.seq.units;
      const int part = (team * 2 + (walk.s == range0 ? 0 : 1)) * p.tiles + tile;
      // ---- Q as sums of e4m3 parts under a power of two per row
      {
        constexpr int kPer = kSoft / RT;  // threads of a row
        const int n = threadIdx.x / kPer, x0 = threadIdx.x % kPer;
        const int row = tile * p.rows_per_tile + n, i = row / p.G;
        const bool real = n < rows;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (b * p.q_stride_b + (real ? i : 0) * p.q_stride_r +
                   (walk.kvh * p.G + (real ? row - i * p.G : 0)) * p.q_stride_h) * 2);
        constexpr int kMine = D / 8 / kPer > 0 ? D / 8 / kPer : 1;  // 16-byte chunks of a thread
        uint4 raw[kMine];
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int c = x0 + m * kPer;
          raw[m] = real && c < D / 8 ? src[c] : make_uint4(0, 0, 0, 0);
        }
        auto values = [&](int m, float* x) {
          const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw[m]);
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
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          float x[8];
          values(m, x);
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
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int c = x0 + m * kPer;
          if (c >= D / 8) break;
          float x[8];
          values(m, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= down;
#pragma unroll
          for (int part = 0; part < S::kParts; ++part) {
            const uint32_t to =
                S::kStack ? swizzled<D>(S::kParts * RT, part * RT + n, c >> 1)
                          : part * RT * D + swizzled<D>(RT, n, c >> 1);
            const uint2 w = make_uint2(e4m3_word(x[0], x[1], x[2], x[3]),
                                       e4m3_word(x[4], x[5], x[6], x[7]));
            *reinterpret_cast<uint2*>(dyn0 + (q_at - base) + to + (c & 1) * 8) = w;
            float y[8];
            e4m3_values(w.x, y);
            e4m3_values(w.y, y + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= y[e];
          }
        }
        if (x0 == 0) {
          sc_s[n] = bad ? NAN : real ? p.scale_log2 * s : 0.f;
          neg_m[0][n] = neg_m[1][n] = -kNone;
          uint64_t m = 0;
          if (real) {
            m = p.mask ? p.mask[(size_t)b * p.R + i] : i >= 63 ? ~0ull : (2ull << i) - 1;
            if (p.R < 64) m &= (1ull << p.R) - 1;
          }
          see_s[n] = m;
          out_s[n] = whole ? ((long long)b * p.R + i) * p.Hq + walk.kvh * p.G + row - i * p.G
                           : (long long)part * RT + n;
          from_s[n] = p.window > 0 ? ctx + __popcll(m) - p.window : 0;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) nan_s[n][e] = 0;
        }
        if (threadIdx.x == 0) any_nan = 0;
        fence_proxy_async();
        mbar_arrive(&q_full);
      }
      sync_of(3, kSoft);

      uint64_t l2[RT / 2];
#pragma unroll
      for (int i = 0; i < RT / 2; ++i) l2[i] = 0ull;
      bool begun = false;  // this group's O holds something
      const int t_seg = walk.seq.first + walk.first_unit() * kUnit;
#pragma unroll 1
      for (int j = (g ^ group) & 1; j < n_units; j += 2) {
        const int u = g + j, stage = u % NS, t0 = t_seg + j * kUnit;
        ok = ok && mbar_wait(&full[stage], (u / NS) & 1, p.err, p.wait_ns);
        const float* scales =
            reinterpret_cast<const float*>(dyn0 + stage * S::kStageBytes + 2 * S::kTileBytes);
        float ks = scales[tok], vs = scales[kUnit + tok];
        const bool here = ks != -INFINITY;
        vs = !here ? 1.f : vs < 0x1p-100f ? 0x1p-100f : vs;
        ks = here ? ks : 0.f;
        const float lvs = here ? __log2f(vs) : -INFINITY, rvs = here ? __fdividef(1.f, vs) : 0.f;
        // positions that some rows see and others do not
        const bool mixed = (t0 + kUnit > ctx && (p.R > 1 || p.mask)) ||
                           (p.window > 0 && t0 < ctx + p.R - p.window);
        uint64_t see = ~0ull;  // columns that see this thread's position
        if (mixed) {
          const int t = t0 + tok, jb = t - ctx;
          see = 0;
#pragma unroll 1
          for (int c = 0; c < RT; ++c)
            if (jb < 0 ? t >= from_s[c] : jb < 64 && (see_s[c] >> jb & 1)) see |= 1ull << c;
        }
        // the group's last product is complete: its O and its operands' buffers are free
        if (u >= 2) ok = ok && mbar_wait(&pv_done[group], (u - 2) >> 1 & 1, p.err, p.wait_ns);
        uint8_t* vrow = dyn0 + stage * S::kStageBytes;
        if (mixed) {  // NaN codes of V: noted for the rows that see them, and zeroed
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t* u4 = reinterpret_cast<uint32_t*>(vrow + swizzled<D>(kUnit, tok, c));
            if (nan_bytes(u4[0]) | nan_bytes(u4[1]) | nan_bytes(u4[2]) | nan_bytes(u4[3])) {
              uint32_t bits = 0;
              for (int e = 0; e < 16; ++e) bits |= (nan_bytes(u4[e >> 2]) >> (8 * (e & 3) + 7) & 1) << e;
              for (int x = 0; x < RT; ++x)
                if (see >> x & 1) atomicOr(&nan_s[x][c >> 1], bits << 16 * (c & 1));
              for (int e = 0; e < 4; ++e) u4[e] &= ~((nan_bytes(u4[e]) >> 7) * 255u);
              any_nan = 1;
            }
          }
        }
        if constexpr (S::kHalfV) {  // this position's V as fp16, 64 dimensions a row
          uint8_t* to = v16_0 + group * S::kVBytes + tok * 128;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(vrow + swizzled<D>(kUnit, tok, c));
            uint4 h0, h1;
            h0.x = halves_of(w.x), h0.y = halves_of(w.x >> 16);
            h0.z = halves_of(w.y), h0.w = halves_of(w.y >> 16);
            h1.x = halves_of(w.z), h1.y = halves_of(w.z >> 16);
            h1.z = halves_of(w.w), h1.w = halves_of(w.w >> 16);
            uint8_t* half = to + (c >> 2) * (kUnit * 128);
            const int c16 = 2 * (c & 3);
            *reinterpret_cast<uint4*>(half + ((c16 ^ (tok & 7)) << 4)) = h0;
            *reinterpret_cast<uint4*>(half + (((c16 + 1) ^ (tok & 7)) << 4)) = h1;
          }
        }
        ok = ok && mbar_wait(&s_full[group], u >> 1 & 1, p.err, p.wait_ns);
        tc_fence_after();
        // ---- exponents of kC columns, relative to the rows' references
        const uint64_t ks2 = f2_pack(ks, ks), lvs2 = f2_pack(lvs, lvs);
        const uint32_t s_at = lanes + group * S::kSCols;
        auto scores = [&](int c, uint32_t* s) {
          tmem_ld<kC>(s_at + c, s);
          if constexpr (S::kStack) {
            uint32_t y[S::kParts - 1][kC];
#pragma unroll
            for (int part = 1; part < S::kParts; ++part) tmem_ld<kC>(s_at + part * RT + c, y[part - 1]);
            tmem_wait_ld();
#pragma unroll
            for (int part = 1; part < S::kParts; ++part)
#pragma unroll
              for (int i = 0; i < kC; ++i)
                s[i] = __float_as_uint(__uint_as_float(s[i]) + __uint_as_float(y[part - 1][i]));
          } else {
            tmem_wait_ld();
          }
        };
        auto exponents = [&](int c, const uint32_t* s, float* a) {
          float top = -INFINITY;
          const uint64_t* sc2 = reinterpret_cast<const uint64_t*>(sc_s + c);
          const uint64_t* nm2 = reinterpret_cast<const uint64_t*>(neg_m[group] + c);
#pragma unroll
          for (int i = 0; i < kC / 2; ++i) {
            const uint64_t x =
                f2_mul(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2[i]);
            f2_unpack(f2_fma(x, ks2, f2_add(lvs2, nm2[i])), a[2 * i], a[2 * i + 1]);
            if (mixed) {
              a[2 * i] = see >> (c + 2 * i) & 1 ? a[2 * i] : -INFINITY;
              a[2 * i + 1] = see >> (c + 2 * i + 1) & 1 ? a[2 * i + 1] : -INFINITY;
            }
            top = fmax3(top, a[2 * i], a[2 * i + 1]);
          }
          return top;
        };
        // (K has been read, V and the scales have been taken over)
        if constexpr (S::kHalfV) mbar_arrive(&empty[stage]);
        // ---- weights and their sums; once more where a weight has passed 2^kTop
        const uint64_t rvs2 = f2_pack(rvs, rvs);
        uint8_t* w_at = dyn0 + (p_at - base) + group * S::kPBytes + tok * 16;
        bool failed = false;
#pragma unroll 1
        for (int pass = begun ? 0 : 1;; ++pass) {
          if (pass) {
            // ---- the references move: maxima over the tile's positions
#pragma unroll
            for (int c = 0; c < RT; c += kC) {
              uint32_t s[kC];
              float x[kC];
              scores(c, s);
#pragma unroll
              for (int i = 0; i < kC; ++i) {
                x[i] = __uint_as_float(s[i]) * sc_s[c + i] * ks + lvs;
                if (mixed && !(see >> (c + i) & 1)) x[i] = -INFINITY;
              }
              int col;
              const float m = over_lanes<kC>(x, lane, [](float u, float v) { return fmaxf(u, v); }, &col);
              red[warp][c + col] = m;
            }
            sync_of(bar, kGroup);
            if (tok < RT) {
              const int w0 = group * 4;
              const float m4 = fmaxf(fmaxf(red[w0][tok], red[w0 + 1][tok]),
                                     fmaxf(red[w0 + 2][tok], red[w0 + 3][tok]));
              const float old = -neg_m[group][tok], now = m4 - old > S::kTop ? m4 - S::kBelow : old;
              fac_s[group][tok] = fast_exp2(old - now);
              neg_m[group][tok] = -now;
            }
            sync_of(bar, kGroup);
            const float* fac = fac_s[group];
#pragma unroll
            for (int i = 0; i < RT / 2; ++i)
              l2[i] = f2_mul(l2[i], reinterpret_cast<const uint64_t*>(fac)[i]);
            if (begun) {
#pragma unroll 1
              for (int c = 0; c < S::kOCols; c += 8) {
                const uint32_t at = lanes + S::kColO + group * S::kOCols + c;
                uint32_t o[8];
                tmem_ld<8>(at, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * fac[c % RT + e]);
                tmem_st8(at, o);
              }
              tmem_wait_st();
            }
          }
          float top = -INFINITY;
          uint64_t t2[RT / 2];  // sums with this tile
#pragma unroll
          for (int c = 0; c < RT; c += kC) {
            uint32_t s[kC];
            float a[kC];
            scores(c, s);
            top = fmaxf(top, exponents(c, s, a));
            if constexpr (S::kHalfV) {
              uint32_t h[kC / 2];
#pragma unroll
              for (int e = 0; e < kC / 2; ++e) {
                const float w0 = fast_exp2(a[2 * e]), w1 = fast_exp2(a[2 * e + 1]);
                t2[c / 2 + e] = f2_fma(f2_pack(w0, w1), rvs2, l2[c / 2 + e]);
                h[e] = f16x2(w0, w1);
              }
#pragma unroll
              for (int x = 0; x < kC / 8; ++x)
                *reinterpret_cast<uint4*>(w_at + (c / 8 + x) * 2048) =
                    make_uint4(h[4 * x], h[4 * x + 1], h[4 * x + 2], h[4 * x + 3]);
            } else {
              uint32_t p1[4], p2[4], p3[4];
#pragma unroll
              for (int e = 0; e < kC / 2; ++e) {
                const float w0 = fast_exp2(a[2 * e]), w1 = fast_exp2(a[2 * e + 1]);
                t2[c / 2 + e] = f2_fma(f2_pack(w0, w1), rvs2, l2[c / 2 + e]);
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
              uint8_t* to = w_at + (c >> 4) * 2048;
              *reinterpret_cast<uint4*>(to) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
              *reinterpret_cast<uint4*>(to + RT * kUnit) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
              *reinterpret_cast<uint4*>(to + 2 * RT * kUnit) = make_uint4(p3[0], p3[1], p3[2], p3[3]);
            }
          }
          if (pass || !any_of(bar, kGroup, top > S::kTop || !ok)) {
#pragma unroll
            for (int i = 0; i < RT / 2; ++i) l2[i] = t2[i];
            break;
          }
          if ((failed = any_of(bar, kGroup, !ok))) break;  // (the same for all of the group)
        }
        if (failed) break;
        begun = true;
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&p_full[group]);
      }
      g += n_units;
      // ---- the segment's sums and outputs: the groups' states meet
      ok = ok && mbar_wait(&o_full, seg & 1, p.err, p.wait_ns);
      if (any_of(3, kSoft, !ok)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < RT; c += kC) {
        float l[kC];
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) f2_unpack(l2[c / 2 + i], l[2 * i], l[2 * i + 1]);
        int col;
        const float sum = over_lanes<kC>(l, lane, [](float u, float v) { return u + v; }, &col);
        red[warp][c + col] = sum;
      }
      sync_of(3, kSoft);
      if (threadIdx.x < RT) {  // weights of the two groups' states, the row's reference and sum
        const int n = threadIdx.x;
        const float m0 = -neg_m[0][n], m1 = -neg_m[1][n], m = fmaxf(m0, m1);
        const float la = (red[0][n] + red[1][n]) + (red[2][n] + red[3][n]);
        const float lb = (red[4][n] + red[5][n]) + (red[6][n] + red[7][n]);
        // (a state without weights holds nothing, or what was there before it)
        const float f0 = la == 0.f ? 0.f : fast_exp2(m0 - m), f1 = lb == 0.f ? 0.f : fast_exp2(m1 - m);
        const float l = (la == 0.f ? 0.f : la * f0) + (lb == 0.f ? 0.f : lb * f1);
        fac_s[0][n] = f0;
        fac_s[1][n] = f1;
        inv_s[n] = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        if (n < rows) {
          if (!whole)
            *reinterpret_cast<float2*>(p.part_ml + out_s[n] * 2) = make_float2(m, l);
          else if (p.lse)
            p.lse[out_s[n]] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      sync_of(3, kSoft);
#pragma unroll 1
      for (int c = group * 8; c < rows; c += 16) {  // (a group takes every other eight rows)
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          uint32_t o[2][S::kSums][8];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < S::kSums; ++y)
              tmem_ld<8>(lanes + S::kColO + x * S::kOCols + (half * S::kSums + y) * RT + c, o[x][y]);
          tmem_wait_ld();
          const int d = half * 128 + tok;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int n = c + e;
            if (n >= rows || d >= D) continue;
            float y = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float z = __uint_as_float(o[x][0][e]);
              if constexpr (!S::kHalfV)
                z += __uint_as_float(o[x][1][e]) * 0x1p-4f + __uint_as_float(o[x][2][e]) * 0x1p-15f;
              const float f = fac_s[x][n];
              y += f == 0.f ? 0.f : f * z;
            }
            if (any_nan && nan_s[n][d >> 5] >> (d & 31) & 1) y = NAN;
            const float inv = inv_s[n];
            y = inv == 0.f ? 0.f : y * inv;
            const long long to = out_s[n] * D + d;
            if (!whole) p.part_o[to] = y;
            else if constexpr (F16) reinterpret_cast<__half*>(p.out)[to] = __float2half_rn(y);
            else reinterpret_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(y);
          }
        }
      }
      tc_fence_before();
      sync_of(3, kSoft);  // the rows' state is free
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, S::kAlloc);
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

// Query rows that a CTA takes at most: what two O of 3 parts leave room for in tensor memory.
constexpr int most_rows(int D) { return D == 256 ? 32 : 64; }

// rt: 16, 32 or 64 query rows of a CTA.  Each D is a translation unit of its own.
template <int D>
spec_status launch_d(const Params& p, int rt, bool f16, cudaStream_t st) {
  constexpr int kMost = most_rows(D);
  spec_status rc;
  if (f16)
    rc = rt == 16 ? launch_one<D, 16, true>(p, st)
                  : rt == 32 ? launch_one<D, 32, true>(p, st) : launch_one<D, kMost, true>(p, st);
  else
    rc = rt == 16 ? launch_one<D, 16, false>(p, st)
                  : rt == 32 ? launch_one<D, 32, false>(p, st) : launch_one<D, kMost, false>(p, st);
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
