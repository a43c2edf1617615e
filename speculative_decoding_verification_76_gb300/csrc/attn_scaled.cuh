// spec_verify_attn_scaled -- attention of a verify block (or of single tokens) over an e4m3 cache
// with one scale for each block of tokens and KV head, on the 5th-generation tensor cores.
//
// Mathematics, for row i and the positions t it sees, with codes k_t, v_t and their blocks' scales
// a_t, c_t:
//   x_t = scale a_t (q . k_t),  out = sum_t e^(x_t) c_t v_t / l,  l = sum_t e^(x_t),  lse = ln l.
// V's scale goes into the weight, w_t = 2^(x_t + log2 c_t - m) with a reference m per row, and
// l = sum w_t / c_t.  So weights keep to a narrow range whatever the scales are, and a row's sum keeps the
// precision of its own largest contribution.  Parts of the positions give (m, l, sum w v) each and
// join by 2^(m_i - M) ("Speculative Token Decoupling: Asynchronous Verification via
// Flash-Decoding", section 03: split-K attention).
//
// What bounds it: HBM in principle up to some 100 query rows per KV head (2 D bytes per position and head
// are read once); measured, the chain of waits of a tile (below).
//
// Design.  Both products are taken transposed, positions (or dimensions) as the MMA's 128 rows and
// query rows as its columns, so that a few query rows cost a few columns:
//   S^T = K Q^T: a tile of 128 positions, as it lies in the cache: the codes go to the tensor cores
//     (tcgen05 kind::f8f6f4) as they are, without a conversion.  Q is a sum of e4m3 parts (two hold a
//     bf16 number's 8 bits, three an fp16's 11) under a power of two per row.
//   O^T = V^T W^T, with weights rounded to fp16, from 2^8 at a row's first maximum up to 2^15: 2^-11 relative down
//     to 2^-22 of the row's largest, and 2^-33 of it below that.  In one of two forms, both exact behind that
//     rounding.  V goes as it lies, and a weight is a sum of three e5m2 parts, the second times 2^4 and the third
//     times 2^8: e5m2 has fp16's exponents, and 3 bits, 3 behind a sign and 3 behind another are fp16's 11.  The parts
//     are columns of their own, added up at the end.  Or the V tile is converted to fp16 in shared memory.
//     The first costs three columns per row, the second conversions per code and room in shared memory: the second
//     is taken for 64 rows, where tensor memory has no room for three columns each, and at D = 64 (64 ragged chains
//     199 us against 214, with costlier parts than these), the first else (one row at D = 128 196 against 202, 5 rows
//     212 against 278).
// In S^T a lane owns four positions of eight columns: their scales are a few registers, unseen positions a
// bit, and the sum over positions is left to the end.  The reference of a row moves only when a weight
// would pass the largest (one vote a tile); then O is rescaled in tensor memory.
//
// A CTA (one per SM) takes up to 64 query rows of a KV head (32 at D = 256) and one contiguous range of (KV
// head, batch's positions), cut in tiles of 128 over all SMs on the device, so that ragged batches, one
// long sequence and captured graphs whose lengths change fill the GPU alike; the cut counts what a
// sequence's ends cost (8 tiles, 10 for 64 rows: 64 ragged chains 256 -> 244 us, one chain of 8 rows on 8192
// tokens 24.5 -> 20.5, a chain of 16 on 131072 168 -> 163).  Four warps stream K, V and their scales into a
// ring of stages (16-byte cp.async, zeros where nothing is seen), run ahead over the ends of sequences and
// make Q's parts behind a segment's first tile; one thread each issues the two products; two groups of four
// warps take the tiles in turn and turn scores into weights, each with references, sums and an O of its
// own, so that one tile's chain of waits lies under the other's work.  Sequences cut over several CTAs leave
// parts, joined by a second kernel in their order, which is set up early.
//
// What a tile costs (cycles of a group, at 32 rows with V as it lies): the wait for it 220, scales and who sees
// it 440, the wait for the scores 240, exponents and vote 950, weights 1000; 2980 with the rest, so 1490 a tile
// with both groups.  At 64 rows: 190, 510, V's conversion 1100, 150, 1600, 900; 4400, so 2200 a tile.  The products'
// arithmetic is 320 of the 1490 and 512 of the 2200 at the tensor cores' full rate, as their pipe's counter says
// (17 and 21 %); N = 64 columns do not reach that rate, and are under way for about twice as long.
// Issue slots are 42 to 52 % full: it is latency that is left.  Tried: three groups (96 registers a thread: 280 us
// against 244 for 64 ragged chains), two CTAs an SM (294), conversion by warps of its own beside two copy
// warps (draft trees 10 % faster, 64 ragged chains 13 % slower), one vote behind the weights instead of
// one in front (278), one score buffer a group instead of two (232 against 228), the rows that see a position
// by a thread's loop over them instead of votes (228 against 221, draft trees 562 against 551), outputs with
// twice the rows in flight (247 against 221).
//
// Measured (replays of a captured graph; bf16, 32/8 heads of 128 unless given): 64 ragged chains of 5 rows
// (540 K positions) 210 us, 5.3 TB/s (218 with weights in two e4m3 parts and one e5m2, of less range); one chain of 8
// on 8192 tokens 18.5; draft trees of 64 on 4 x 32768, 64/8 heads, 544, 505 TFLOP/s; a chain of 16 on 131072, 64/8
// heads, fp16, 154; single tokens of 37 sequences, window 1000, 16/4 heads of 64, fp16, 16.0.  (1 to 2 % from one
// GPU to the next.)
//
// What is seen by some rows only (block rows, the edge of a window) gets weight 0 elsewhere; as 0 times a
// NaN code would be NaN, such tiles' NaN codes of V are zeroed and noted per row.
#pragma once
#include <cuda_fp16.h>

#include "scaled.cuh"
#include "tc_ptx.cuh"

namespace scaled_attn {

constexpr int kUnit = 128;                       // positions of a tile
constexpr int kGroup = 128;                      // threads of a soft group
constexpr int kSoftWarps = 8, kSoft = 2 * kGroup;
constexpr int kLoadWarp0 = kSoftWarps, kLoadWarps = 4, kLoad = 32 * kLoadWarps;
constexpr int kScoreWarp = kLoadWarp0 + kLoadWarps, kSumWarp = kScoreWarp + 1;  // a thread each issues MMAs
constexpr int kThreads = 32 * (kSumWarp + 1);
static_assert(kLoad == kUnit, "a position of the tile for each");
constexpr float kNone = -1e30f;                  // the reference of a row that has seen nothing
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMostEnds = 10;                    // of Params::ends
// V's scales: a row's sum adds weights of up to 2^15 over them, of up to 2^31 positions (2^126 at the least scale);
// over the most, 2^120, a row's first weight of 2^8 or more still leaves 2^-112.  The most times the factor is the
// largest fp32 number.
constexpr float kLeastV = 0x1p-80f, kPastMostV = 0x1.fffffep7f;

struct Params {
  const char *q, *k, *v;
  const float *ks, *vs;
  const int32_t *table, *ctx;
  const uint64_t* mask;
  char* out;
  float *lse, *part_o, *part_ml;
  int32_t* err;
  long long q_stride_b, q_stride_r, q_stride_h;       // elements
  long long head_stride;             // bytes
  uint32_t token_stride, page_rows;  // bytes; page stride in token strides
  FastDiv P, block, per_head;        // page size, block, query heads of a KV head
  int B, R, Hq, Hkv, G, num_pages, max_pages, window;
  int tiles, rows_per_tile, teams;   // row tiles of a KV head, their query rows; ranges
  // What beginning and ending a segment costs (Q, sums, outputs), in tiles: a sequence counts as that many
  // more when the ranges are cut, so that those that meet an end take fewer.
  int ends;
  float scale_log2;
  uint32_t polls;                    // of a wait, before it gives up
  int withhold_stage;                // -1; a test sets a tile whose arrival the load warps withhold
};

__device__ const float g_unseen = -INFINITY;  // K's scale of a position that is not there

struct Seq {  // positions first .. end - 1 of a sequence are looked at
  int ctx, first, end, units, span;
};

SPEC_DEV Seq seq_of(const Params& p, int b) {
  Seq s;
  s.ctx = p.ctx[b];
  const long long end = min((long long)s.ctx + p.R, (long long)p.max_pages * p.P.d);
  s.end = s.ctx < 0 ? 0 : (int)end;
  s.first = p.window > 0 && s.ctx > p.window ? s.ctx - p.window : 0;
  s.units = s.end > s.first ? (s.end - s.first + kUnit - 1) / kUnit : 0;
  s.span = s.units > 0 ? s.units + p.ends : 0;
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
  int W, s, s1, kvh, b, at;  // batch's span; next unit and end; where it lies
  Seq seq;
  int s0;                    // the range's first unit
  SPEC_DEV bool more() const { return s < s1; }
  SPEC_DEV int first_unit() const { return s - kvh * W - at; }
  SPEC_DEV int count() const { return min(seq.units - first_unit(), s1 - s); }
  __device__ __noinline__ void next_seq(const Params& p) {
    at += seq.span;
    s = kvh * W + at;
    if (s >= s1) return;
#pragma unroll 1
    do {
      if (++b == p.B) b = 0, at = 0, ++kvh;
      seq = seq_of(p, b);
    } while (seq.units == 0);
  }
  SPEC_DEV void next(const Params& p) {
    s += count();
    if (s < s1) next_seq(p);
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

// 16 lanes x 8 N columns as accumulator fragments: registers 4 k, 4 k + 1 are columns 8 k + 2 (lane % 4),
// + 1 of lane / 4, registers 4 k + 2, + 3 those of lane / 4 + 8.
template <int N>
SPEC_DEV void tmem_ld_frag(uint32_t addr, uint32_t* r) {
  static_assert(N == 1 || N == 2 || N == 4, "column groups");
  if constexpr (N == 1)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

SPEC_DEV void tmem_ld2(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}

SPEC_DEV void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(addr));
}

// Four 8 x 8 fragments of 16-bit elements; lane i has the address of row i % 8 of fragment i / 8.
SPEC_DEV void store_frags(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
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

// mbar_wait with little code (what an instance holds in its loops has to stay in the SM's instruction cache:
// with waits, rare paths and unrolled loops written out, 64 ragged chains took 378 us against 293): suspended
// polls of up to 1 us, `polls` of them.  The roles set the error word when they end.
SPEC_DEV bool wait_for(uint64_t* bar, uint32_t parity, const Params& p) {
  uint32_t left = p.polls;
#pragma unroll 1
  while (!mbar_try_wait_ns(bar, parity, 1000))
    if (left-- == 0) return false;
  return true;
}
SPEC_DEV void report(bool ok, const Params& p) {
  if (!ok) set_error(p.err, SPEC_ERR_MBAR_TIMEOUT);
}

SPEC_DEV uint32_t f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two halves rounded to the nearest e5m2 number, which is a half whose lower byte is zero (ties away from zero;
// a NaN becomes a zero, and stays what the subtraction behind it makes).
SPEC_DEV uint32_t e5m2_of(uint32_t h2) { return (h2 + 0x00800080u) & 0xff00ff00u; }
SPEC_DEV void codes_to_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {  // bytes 0, 1 and 2, 3
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
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
  // V as fp16, converted in shared memory, and the weights with it; else V as it lies, and the weights as
  // three 8-bit parts (above)
  static constexpr bool kHalfV = D == 64 || (D == 128 && RT == 64);
  static constexpr int kSums = kHalfV ? 1 : 3;                  // columns of O per row and 128 dimensions
  static constexpr int kHalves = D == 256 ? 2 : 1;
  static constexpr int kOCols = kSums * RT * kHalves;
  // weights stay at or below 2^kTop and begin at 2^kBelow
  static constexpr float kTop = 15.f, kBelow = 8.f;
  static constexpr int kStageBytes = 2 * kTileBytes + 1024;     // V, K, scales
  static constexpr int kQBytes = kParts * RT * D;               // of one of two
  static constexpr int kPBytes = kHalfV ? RT * kUnit * 2 : 3 * RT * kUnit;
  static constexpr int kVBytes = kHalfV ? 2 * kTileBytes : 0;
  // buffers of Q (the next segment's is made while this one's is used) and of weights (with four, those
  // who write them need not wait for the product two tiles back), where there is room
  static constexpr int kQBufs = RT == 64 && F16 ? 1 : 2, kPBufs = 2;
  static constexpr int kFixed = kQBufs * kQBytes + kPBufs * kPBytes + 2 * kVBytes + 1024;
  static constexpr int kRoom = 225 * 1024 - 11 * 1024 - kFixed; // (static shared memory: < 11 KB)
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static_assert(kStages >= 1, "a ring needs a stage");
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  // tensor memory: two score buffers and an O for each soft group (the next tile's scores are made while one's
  // are read)
  static constexpr int kColO = 4 * RT, kCols = kColO + 2 * kOCols;
  static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "tensor memory");
};

// Byte of 16-byte chunk c of row r in a tile of `rows` rows.
template <int D>
SPEC_DEV uint32_t swizzled(int rows, int r, int c) {
  if constexpr (D == 64) return r * 64 + ((c ^ (r >> 1 & 3)) << 4);
  return (uint32_t)(c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <bool kWide>
struct RowBits {
  using T = uint32_t;
};
template <>
struct RowBits<true> {
  using T = uint64_t;
};

// Whether a position's V row has NaN codes.
template <int D>
SPEC_DEV bool has_nans(const uint8_t* tile, int tok) {
  uint32_t nan = 0;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    const uint4 w = *reinterpret_cast<const uint4*>(tile + swizzled<D>(kUnit, tok, c));
    nan |= nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w);
  }
  return nan != 0;
}

// NaN codes in a position's V row: noted for the query rows that see it, and zeroed (positions that only some
// rows see; hardly ever anything to do).
template <int D>
__device__ __noinline__ void note_nans(uint8_t* tile, int tok, uint64_t rows, uint32_t* notes) {
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t* u4 = reinterpret_cast<uint32_t*>(tile + swizzled<D>(kUnit, tok, c));
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      const uint32_t nan = nan_bytes(u4[e]);
      if (!nan) continue;
      const uint32_t bits = nan >> 7 & 1 | nan >> 14 & 2 | nan >> 21 & 4 | nan >> 28 & 8;
#pragma unroll 1
      for (uint64_t left = rows; left; left &= left - 1)
        atomicOr(&notes[(__ffsll((long long)left) - 1) * (D / 32) + (c >> 1)],
                 bits << (16 * (c & 1) + 4 * e));
      u4[e] &= ~((nan >> 7) * 255u);
    }
  }
}

template <int D, int RT, bool F16>
__global__ void __launch_bounds__(kThreads, 1) attn_scaled_kernel(
    const __grid_constant__ Params p) {
  using S = Shape<D, RT, F16>;
  constexpr int NS = S::kStages;
  constexpr int kGroups = RT / 8;                    // column groups of eight
  constexpr int kB = kGroups < 4 ? kGroups : 4;      // of them between two votes
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], s_full[4], p_full[4], pv_done[4], q_full[2],
      seg_done[2], o_full, fin;
  // per segment, two in flight: scale, block rows seen, first position, output row of a query row
  __shared__ __align__(16) float sc_s[2][RT];
  __shared__ uint64_t see_s[2][RT];
  __shared__ long long out_s[2][RT];
  __shared__ int from_s[2][RT], any_nan[2];
  __shared__ uint32_t nan_s[2][RT][D / 32];
  __shared__ __align__(16) float neg_m[2][RT], fac_s[2][RT], red[kSoftWarps][RT], inv_s[RT];
  // the rows that see a position, for tiles where not all of them do (a warp's positions are its own)
  using Rows = typename RowBits<(RT > 32)>::T;
  __shared__ Rows seen_by[2][kUnit];
  __shared__ Walk start;
  __shared__ uint32_t tmem_base;
  __shared__ int part_w[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  // fp16 V, the stages, Q, the weights: whole swizzle atoms
  const uint32_t v16_at = (smem_u32(dyn) + 1023u) & ~1023u, base = v16_at + 2 * S::kVBytes;
  const uint32_t q_at = base + NS * S::kStageBytes, p_at = q_at + S::kQBufs * S::kQBytes;
  uint8_t* const v16_0 = dyn + (v16_at - smem_u32(dyn));
  uint8_t* const dyn0 = v16_0 + 2 * S::kVBytes;
  uint8_t* const q_0 = dyn0 + NS * S::kStageBytes;
  const int rows = min(p.rows_per_tile, p.R * p.G - tile * p.rows_per_tile);

  chain_wait();
  chain_next();  // (the joining kernel may be set up)
  // ---- this CTA's range, and the sequence it begins in: each thread sums consecutive sequences
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += seq_of(p, b).span;
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
      while (at + seq.span <= u) at += seq.span, seq = seq_of(p, ++b);
      Walk walk{W, s0, ranges.begin(team + 1), kvh, b, at, seq, s0};
      if (walk.first_unit() >= seq.units) walk.next_seq(p);  // (nothing is left of this one)
      start = walk;
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&full[i], kLoad);
        mbar_init(&empty[i], kGroup + (S::kHalfV ? 1 : 2));  // scales (and V) taken, K's (and V's) product
      }
      for (int i = 0; i < 4; ++i) {  // tile u's is u & 3
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], kGroup);
        mbar_init(&pv_done[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], kLoad);
        mbar_init(&seg_done[i], kSoft);
      }
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

  if (warp >= kLoadWarp0 && warp < kScoreWarp) {
    // ================================================================ K, V, their scales, and Q
    // a thread looks up one position; a lane copies chunks c and c + L of a row (L lanes of a row)
    constexpr int L = D / 32, kRows = 32 / L;
    const int tid = threadIdx.x - 32 * kLoadWarp0, r0 = tid & ~31;
    const int sub = lane / L, chunk = lane % L;
    uint64_t pol;
    if (p.tiles == 1)  // the only reader of these rows
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    else
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    const int nb = p.P.d / p.block.d;
    int g = 0, seg = 0;
    bool ok = true;
    for (Walk walk = start; walk.more() && ok; walk.next(p), ++seg) {
      const int b = walk.b, n_units = walk.count(), ctx = walk.seq.ctx, end = walk.seq.end, sb = seg & 1;
      const bool whole = n_units == walk.seq.units;
      const int part_at = (team * 2 + (walk.s == walk.s0 ? 0 : 1)) * p.tiles + tile;
      const int32_t* bt = p.table + (size_t)b * p.max_pages;
      // a query row for kPer threads; what a thread has of it is on its way before anything else
      constexpr int kPer = kLoad / RT;
      constexpr int kMine = D / 8 / kPer > 0 ? D / 8 / kPer : 1;  // 16-byte chunks of a thread
      const int n = tid / kPer, x0 = tid % kPer;
      const int q_row = tile * p.rows_per_tile + n, i_row = p.per_head.quot(q_row);
      const bool real = n < rows;
      const uint4* const q_src = reinterpret_cast<const uint4*>(
          p.q + (b * p.q_stride_b + (real ? i_row : 0) * p.q_stride_r +
                 (walk.kvh * p.G + (real ? q_row - i_row * p.G : 0)) * p.q_stride_h) * 2);
      auto q_chunk = [&](int m) {
        const int c = x0 + m * kPer;
        return real && c < D / 8 ? q_src[c] : make_uint4(0, 0, 0, 0);
      };
      uint4 held[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) held[m] = q_chunk(m);
      int t = walk.seq.first + walk.first_unit() * kUnit + tid;
      int page = p.P.quot(t), off = t - page * p.P.d, id = t < end ? bt[page] : -1;
      const char* kh = p.k + walk.kvh * p.head_stride + chunk * 16;
      const char* vh = p.v + walk.kvh * p.head_stride + chunk * 16;
#pragma unroll 1
      for (int j = 0; j < n_units; ++j, ++g) {
        const int stage = g % NS;
        // (a position that is not there: zeros)
        const bool is_there = (uint32_t)id < (uint32_t)p.num_pages;
        const uint32_t there = __ballot_sync(0xffffffffu, is_there);
        const uint32_t row = is_there ? id * p.page_rows + off : 0;  // in token strides
        const long long sc = ((long long)id * nb + p.block.quot(off)) * p.Hkv + walk.kvh;
        t += kUnit;
        page = p.P.quot(t), off = t - page * p.P.d;
        id = j + 1 < n_units && t < end ? bt[page] : -1;
        // (the warp as one: the shuffles below need every lane)
        if (g >= NS) ok = __all_sync(0xffffffffu, wait_for(&empty[stage], ((g / NS) - 1) & 1, p));
        if (!ok) break;
        const uint32_t v_at = base + stage * S::kStageBytes, k_at = v_at + S::kTileBytes;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const int r = i * kRows + sub;
          const uint64_t from = (uint64_t)__shfl_sync(0xffffffffu, row, r) * p.token_stride;
          const uint32_t bytes = there >> r & 1 ? 16u : 0u;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t to = swizzled<D>(kUnit, r0 + r, chunk + x * L);
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
        const uint32_t s_at = v_at + 2 * S::kTileBytes + tid * 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at),
                     "l"(is_there ? p.ks + sc : &g_unseen)
                     : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at + 512),
                     "l"(is_there ? p.vs + sc : &g_unseen)
                     : "memory");
        if (g != p.withhold_stage)
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&full[stage]))
                       : "memory");
        if (j > 0) continue;
        // ---- behind the segment's first tile: Q as sums of e4m3 parts under a power of two per row
        // (the segment before the last is done with the places)
        if (seg >= S::kQBufs)
          ok = __all_sync(0xffffffffu,
                          wait_for(&seg_done[(seg - S::kQBufs) & 1], (seg - S::kQBufs) >> 1 & 1, p));
        if (!ok) break;
        {
          auto values = [&](const uint4& w, float* x) {
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
          // the largest magnitude, as bits; what is not finite has all exponent bits
          uint32_t big2 = 0;
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            const uint4 w = held[m];
            big2 = __vimax3_u16x2(big2, w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
            big2 = __vimax3_u16x2(big2, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
          }
#pragma unroll
          for (int o = 1; o < kPer; o <<= 1) big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, o));
          const uint32_t big = max(big2 & 0xffffu, big2 >> 16);
          const bool bad = big >= (F16 ? 0x7c00u : 0x7f80u);  // (then only the row's scale matters)
          const float s = needed_scale(F16 ? __half2float(__ushort_as_half((unsigned short)big))
                                           : __uint_as_float(big << 16));
          const float down = 1.f / s;
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            const int c = x0 + m * kPer;
            if (c >= D / 8) break;
            float x[8];
            values(held[m], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= down;
            uint8_t* to = q_0 + seg % S::kQBufs * S::kQBytes + swizzled<D>(RT, n, c >> 1) + (c & 1) * 8;
#pragma unroll 1
            for (int part = 0; part < S::kParts; ++part) {
              const uint2 w = make_uint2(e4m3_word(x[0], x[1], x[2], x[3]),
                                         e4m3_word(x[4], x[5], x[6], x[7]));
              *reinterpret_cast<uint2*>(to + part * RT * D) = w;
              float y[8];
              e4m3_values(w.x, y);
              e4m3_values(w.y, y + 4);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] -= y[e];
            }
          }
          if (x0 == 0) {
            sc_s[sb][n] = bad ? NAN : real ? p.scale_log2 * s : 0.f;
            uint64_t m = 0;
            if (real) {
              m = p.mask ? p.mask[(size_t)b * p.R + i_row] : i_row >= 63 ? ~0ull : (2ull << i_row) - 1;
              if (p.R < 64) m &= (1ull << p.R) - 1;
            }
            see_s[sb][n] = m;
            out_s[sb][n] = whole ? ((long long)b * p.R + i_row) * p.Hq + walk.kvh * p.G + q_row - i_row * p.G
                                 : (long long)part_at * RT + n;
            from_s[sb][n] = p.window > 0 ? ctx + __popcll(m) - p.window : 0;
#pragma unroll 1
            for (int e = 0; e < D / 32; ++e) nan_s[sb][n][e] = 0;
          }
          if (tid == 0) any_nan[sb] = 0;
          fence_proxy_async();
          mbar_arrive(&q_full[sb]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    report(ok, p);
  } else if (warp == kScoreWarp) {
    // ================================================================ S^T = K Q^T, one thread
    if (lane == 0) {
      constexpr uint32_t kId = idesc_f8(128, RT, false, false);
      constexpr uint32_t kHi = desc_hi(S::kRows8, S::kLayout);
      int g = 0, seg = 0;
      bool ok = true;
      for (Walk walk = start; walk.more() && ok; walk.next(p), ++seg) {
        const int n = walk.count();
        if (!(ok = wait_for(&q_full[seg & 1], seg >> 1 & 1, p))) break;
        const uint32_t q_lo = desc_lo(q_at + seg % S::kQBufs * S::kQBytes, 16);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          const int stage = g % NS;
          // the score buffer's last tile has been read, this tile has landed
          ok = (g < 4 || wait_for(&p_full[g & 3], (g - 4) >> 2 & 1, p)) &&
               wait_for(&full[stage], (g / NS) & 1, p);
          if (!ok) break;
          fence_proxy_async();  // the copies' writes, for the tensor cores
          tc_fence_after();
          const uint32_t k_lo = desc_lo(base + stage * S::kStageBytes + S::kTileBytes, 16);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            constexpr int kIn = D == 64 ? 2 : 4;  // steps within a swizzled row
            const uint32_t a = k_lo + ((k / kIn) * (kUnit * 128) + k % kIn * 32) / 16;
            uint32_t b = q_lo + ((k / kIn) * (RT * 128) + k % kIn * 32) / 16;
#pragma unroll
            for (int part = 0; part < S::kParts; ++part, b += RT * D / 16)
              mma_f8(tmem + (g & 3) * RT, a, kHi, b, kHi, kId, k > 0 || part > 0);
          }
          tc_commit(&s_full[g & 3]);
          tc_commit(&empty[stage]);
        }
      }
      // (nothing of this thread's is in flight when the tensor memory goes)
      report(ok, p);
      tc_commit(&fin);
      wait_for(&fin, 0, p);
    }
    __syncwarp();
  } else if (warp == kSumWarp) {
    // ================================================================ O^T += V^T W^T, one thread
    if (lane == 0) {
      constexpr uint32_t kHiW = desc_hi(2048, 0);
      int g = 0;
      bool ok = true;
      for (Walk walk = start; walk.more() && ok; walk.next(p)) {
        const int n = walk.count();
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          ok = wait_for(&p_full[g & 3], g >> 2 & 1, p);
          if (!ok) break;
          if constexpr (!S::kHalfV) fence_proxy_async();
          tc_fence_after();
          const uint32_t w_lo = desc_lo(p_at + g % S::kPBufs * S::kPBytes, 128);
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
            constexpr uint32_t kId = idesc_f8(128, 3 * RT, true, true);
            constexpr uint32_t kHi = desc_hi(S::kRows8, S::kLayout);
            const int stage = g % NS;
            const uint32_t v_lo = desc_lo(base + stage * S::kStageBytes, 16384);
#pragma unroll 1
            for (int half = 0; half < S::kHalves; ++half)
#pragma unroll 1
              for (int k = 0; k < kUnit / 32; ++k) {
                const uint32_t a = v_lo + (half * (kUnit * 128) + k * 4 * S::kRows8) / 16;
                mma_f8(o + half * 3 * RT, a, kHi, w_lo + k * 512 / 16, kHiW, kId, k > 0 ? 1u : later);
              }
            tc_commit(&empty[stage]);
          }
          tc_commit(&pv_done[g & 3]);
        }
        if (ok) tc_commit(&o_full);
      }
      report(ok, p);
      tc_commit(&fin);
      wait_for(&fin, 0, p);
    }
    __syncwarp();
  } else {
    // ================================================================ scores into weights
    // Two groups of four warps take the tiles in turn, each with references, sums and an O of its
    // own: one tile's chain of waits lies under the other's work.
    const int group = warp >> 2, bar = 1 + group, quad = warp & 3;
    const int tid = threadIdx.x & (kGroup - 1);       // in the group; a dimension of O
    const uint32_t lanes = tmem + ((uint32_t)quad << 21);
    const int c2 = 2 * (lane & 3), t_lane = quad * 32 + (lane >> 2);  // first column and position of this lane
    int g = 0, seg = 0;
    bool ok = true;
    for (Walk walk = start; walk.more(); walk.next(p), ++seg) {
      const int n_units = walk.count(), ctx = walk.seq.ctx, sb = seg & 1;
      const int t_seg = walk.seq.first + walk.first_unit() * kUnit;
      const bool whole = n_units == walk.seq.units;
      ok = ok && wait_for(&q_full[sb], seg >> 1 & 1, p);
      // columns 8 k + c2, + 1: their scales, references and sums (over this lane's positions)
      uint64_t sc2[kGroups], nm2[kGroups], l2[kGroups];
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        sc2[k] = *reinterpret_cast<const uint64_t*>(&sc_s[sb][8 * k + c2]);
        nm2[k] = 0ull;  // (the segment's first references come from its first exponents)
        l2[k] = 0ull;
      }
      if (tid < RT) neg_m[group][tid] = -kNone;
      bool begun = false;  // this group's O holds something
      bool failed = false;
#pragma unroll 1
      for (int j = (g ^ group) & 1; j < n_units; j += 2) {
        const int u = g + j, t0 = t_seg + j * kUnit;
        const int stage = u % NS;
        ok = ok && wait_for(&full[stage], (u / NS) & 1, p);
        // positions t_lane + 8 r: K's scale, the logarithm of V's and its inverse
        uint8_t* vrow = dyn0 + stage * S::kStageBytes;
        const float* scales = reinterpret_cast<const float*>(vrow + 2 * S::kTileBytes) + t_lane;
        float ks[4], lvs[4], rvs[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float stored = scales[kUnit + 8 * r], vs = fmaxf(stored, kLeastV);
          ks[r] = scales[8 * r];
          // (of a NaN scale, or one whose product passes fp32, the logarithm alone is NaN: where the weight is 0 the
          // inverse must not make the sum NaN.  Not a comparison and a select, which cost 1 to 2 % in every shape)
          lvs[r] = fmaf(stored * kPastMostV, 0.f, __log2f(vs)), rvs[r] = __fdividef(1.f, vs);
          if (ks[r] == -INFINITY) ks[r] = 0.f, lvs[r] = -INFINITY, rvs[r] = 0.f;  // not there
        }
        // positions that some rows see and others do not
        const bool mixed = (t0 + kUnit > ctx && (p.R > 1 || p.mask)) ||
                           (p.window > 0 && t0 < ctx + p.R - p.window);
        Rows* const seen = seen_by[group];
        if (mixed) {  // a lane holds a row (or two), a vote gives a position's (of 16 rows, two positions')
          constexpr int kAt = RT < 32 ? 16 : 32;  // positions from one of a vote to the next
          const int first = t0 + quad * 32;
          Rows m = 0;
          if (first + 31 < ctx && p.window == 0) {
            m = ~(Rows)0;
          } else if (first < ctx + p.R) {
            const int n0 = lane & (kAt - 1), n1 = RT > 32 ? lane + 32 : n0;
            const uint64_t see0 = see_s[sb][n0], see1 = see_s[sb][n1];
            const int from0 = from_s[sb][n0], from1 = from_s[sb][n1];
#pragma unroll 4
            for (int i = 0; i < kAt; ++i) {
              const int t = first + i + (lane & ~(kAt - 1)), jb = t - ctx;
              const bool sees0 = jb < 0 ? t >= from0 : jb < 64 && (see0 >> (jb & 63) & 1);
              Rows rows_of = __ballot_sync(0xffffffffu, sees0);
              if constexpr (RT > 32) {
                const bool sees1 = jb < 0 ? t >= from1 : jb < 64 && (see1 >> (jb & 63) & 1);
                rows_of |= (Rows)__ballot_sync(0xffffffffu, sees1) << 32;
              }
              if (n0 == i) m = kAt < 32 ? rows_of >> (lane & 16) : rows_of;
            }
          }
          if constexpr (RT < 32) m &= (1u << RT) - 1;
          __syncwarp();
          seen[tid] = m;
          if (has_nans<D>(vrow, tid)) {
            note_nans<D>(vrow, tid, m, nan_s[sb][0]);
            any_nan[sb] = 1;
          }
          __syncwarp();
        }
        if constexpr (S::kHalfV) {  // position tid's V as fp16, 64 dimensions a row
          // (the product that read the buffer last is complete)
          if (u >= 2) ok = ok && wait_for(&pv_done[(u - 2) & 3], (u - 2) >> 2 & 1, p);
          uint8_t* to = v16_0 + group * S::kVBytes + tid * 128;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(vrow + swizzled<D>(kUnit, tid, c));
            uint4 h0, h1;
            codes_to_halves(w.x, h0.x, h0.y);
            codes_to_halves(w.y, h0.z, h0.w);
            codes_to_halves(w.z, h1.x, h1.y);
            codes_to_halves(w.w, h1.z, h1.w);
            uint8_t* half = to + (c >> 2) * (kUnit * 128);
            const int c16 = 2 * (c & 3);
            *reinterpret_cast<uint4*>(half + ((c16 ^ (tid & 7)) << 4)) = h0;
            *reinterpret_cast<uint4*>(half + (((c16 + 1) ^ (tid & 7)) << 4)) = h1;
          }
        }
        ok = ok && wait_for(&s_full[u & 3], u >> 2 & 1, p);
        tc_fence_after();
        // (only what has been handed over is given back: a phase must not get more arrivals than it waits for)
        if (ok) mbar_arrive(&empty[stage]);
        const uint32_t s_at = lanes + (u & 3) * RT;
        const uint32_t w_at = p_at + u % S::kPBufs * S::kPBytes + (quad * 32 + lane) * 16;
#pragma unroll
        for (int h = 0; h < kGroups; h += kB) {
          if (8 * h >= rows) break;
          // ---- exponents relative to the rows' references; these move where a weight would pass
          // 2^kTop (column groups behind the last row are left out)
          float a[4][2 * kB];
          bool moved = false;
#pragma unroll 1
          while (true) {
            uint32_t s[2][4 * kB];
            tmem_ld_frag<kB>(s_at + 8 * h, s[0]);
            tmem_ld_frag<kB>(s_at + 8 * h + (16u << 16), s[1]);
            tmem_wait_ld();
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kB; ++k) {
              if (8 * (h + k) >= rows) break;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t* y = &s[r >> 1][4 * k + 2 * (r & 1)];
                const uint64_t x =
                    f2_mul(f2_pack(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2[h + k]);
                f2_unpack(f2_fma(x, f2_pack(ks[r], ks[r]), f2_add(f2_pack(lvs[r], lvs[r]), nm2[h + k])), a[r][2 * k],
                          a[r][2 * k + 1]);
              }
            }
            if (mixed) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t see = (uint32_t)(seen[t_lane + 8 * r] >> (8 * h + c2));
#pragma unroll
                for (int i = 0; i < 2 * kB; ++i)
                  a[r][i] = see >> (8 * (i >> 1) + (i & 1)) & 1 ? a[r][i] : -INFINITY;
              }
            }
            if (moved) break;
            if (!begun) {  // the first tile: references below the maxima of its positions
#pragma unroll
              for (int k = 0; k < kB; ++k) {
                if (8 * (h + k) >= rows) break;
                float m0 = fmaxf(fmaxf(a[0][2 * k], a[1][2 * k]), fmaxf(a[2][2 * k], a[3][2 * k]));
                float m1 = fmaxf(fmaxf(a[0][2 * k + 1], a[1][2 * k + 1]), fmaxf(a[2][2 * k + 1], a[3][2 * k + 1]));
#pragma unroll
                for (int o = 4; o <= 16; o *= 2) {
                  m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                  m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                }
                if (lane < 4) *reinterpret_cast<float2*>(&red[warp][8 * (h + k) + c2]) = make_float2(m0, m1);
              }
              sync_of(bar, kGroup);
              if (tid < 8 * kB && 8 * h + (tid & ~7) < rows) {
                const int w0 = group * 4, n = 8 * h + tid;
                const float m4 = fmaxf(fmaxf(red[w0][n], red[w0 + 1][n]), fmaxf(red[w0 + 2][n], red[w0 + 3][n]));
                neg_m[group][n] = m4 > kNone ? S::kBelow - m4 : -kNone;
              }
              sync_of(bar, kGroup);
#pragma unroll
              for (int k = 0; k < kB; ++k) {
                if (8 * (h + k) >= rows) break;
                nm2[h + k] = *reinterpret_cast<const uint64_t*>(&neg_m[group][8 * (h + k) + c2]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  f2_unpack(f2_add(f2_pack(a[r][2 * k], a[r][2 * k + 1]), nm2[h + k]), a[r][2 * k], a[r][2 * k + 1]);
              }
              break;
            }
#pragma unroll
            for (int k = 0; k < kB; ++k) {
              if (8 * (h + k) >= rows) break;
#pragma unroll
              for (int r = 0; r < 4; ++r) top = fmax3(top, a[r][2 * k], a[r][2 * k + 1]);
            }
            if (!any_of(bar, kGroup, top > S::kTop || !ok)) break;
            if ((failed = any_of(bar, kGroup, !ok))) break;  // (the same for all of the group)
            moved = true;
            // ---- maxima over the tile's positions
#pragma unroll 1
            for (int k = h; k < h + kB && 8 * k < rows; ++k) {
              uint32_t y[2][4];
              tmem_ld_frag<1>(s_at + 8 * k, y[0]);
              tmem_ld_frag<1>(s_at + 8 * k + (16u << 16), y[1]);
              tmem_wait_ld();
              const float2 sc = *reinterpret_cast<const float2*>(&sc_s[sb][8 * k + c2]);
              float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float z0 = __uint_as_float(y[r >> 1][2 * (r & 1)]) * sc.x * ks[r] + lvs[r];
                float z1 = __uint_as_float(y[r >> 1][2 * (r & 1) + 1]) * sc.y * ks[r] + lvs[r];
                if (mixed) {
                  const Rows see = seen[t_lane + 8 * r] >> (8 * k + c2);
                  if (!(see & 1)) z0 = -INFINITY;
                  if (!(see & 2)) z1 = -INFINITY;
                }
                m0 = fmaxf(m0, z0);
                m1 = fmaxf(m1, z1);
              }
#pragma unroll
              for (int o = 4; o <= 16; o *= 2) {
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
              }
              if (lane < 4) *reinterpret_cast<float2*>(&red[warp][8 * k + c2]) = make_float2(m0, m1);
            }
            sync_of(bar, kGroup);
            if (tid < 8 * kB && 8 * h + (tid & ~7) < rows) {
              const int w0 = group * 4, n = 8 * h + tid;
              const float m4 = fmaxf(fmaxf(red[w0][n], red[w0 + 1][n]), fmaxf(red[w0 + 2][n], red[w0 + 3][n]));
              const float old = -neg_m[group][n];
              const float now = m4 - old > S::kTop ? m4 - S::kBelow : old;
              fac_s[group][n] = fast_exp2(old - now);
              neg_m[group][n] = -now;
            }
            sync_of(bar, kGroup);
#pragma unroll
            for (int k = 0; k < kB; ++k) {
              if (8 * (h + k) >= rows) break;
              nm2[h + k] = *reinterpret_cast<const uint64_t*>(&neg_m[group][8 * (h + k) + c2]);
              l2[h + k] = f2_mul(l2[h + k],
                                 *reinterpret_cast<const uint64_t*>(&fac_s[group][8 * (h + k) + c2]));
            }
            // O, whose last product has to be complete
            ok = ok && wait_for(&pv_done[(u - 2) & 3], (u - 2) >> 2 & 1, p);
            tc_fence_after();
#pragma unroll 1
            for (int y = 0; y < S::kSums * S::kHalves; ++y)
#pragma unroll 1
              for (int k = h; k < h + kB && 8 * k < rows; ++k) {
                const uint32_t at = lanes + S::kColO + group * S::kOCols + y * RT;
                uint32_t o[8];
                if constexpr (S::kHalfV) {
                  tmem_ld8(at + 8 * k, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fac_s[group][8 * k + e]);
                  tmem_st8(at + 8 * k, o);
                } else {  // (columns in the parts' order, sixteen at a time)
                  if (k & 1) continue;
#pragma unroll 1
                  for (int x = 0; x < 2; ++x) {
                    tmem_ld8(at + 8 * k + 8 * x, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      const int q = 8 * x + e, n = 8 * k + 2 * (q >> 2) + (q & 1) + 8 * (q >> 1 & 1);
                      o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                             ((n & ~7) < rows ? fac_s[group][n] : 1.f));
                    }
                    tmem_st8(at + 8 * k + 8 * x, o);
                  }
                }
              }
            tmem_wait_st();
          }
          if (failed) break;
          // ---- weights and their sums
          if constexpr (S::kPBufs == 2 && !S::kHalfV)
            if (h == 0 && u >= 2) ok = ok && wait_for(&pv_done[(u - 2) & 3], (u - 2) >> 2 & 1, p);
          uint32_t w[kB][4];
#pragma unroll
          for (int k = 0; k < kB; ++k) {
            if (8 * (h + k) >= rows) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float w0 = fast_exp2(a[r][2 * k]), w1 = fast_exp2(a[r][2 * k + 1]);
              l2[h + k] = f2_fma(f2_pack(w0, w1), f2_pack(rvs[r], rvs[r]), l2[h + k]);
              w[k][r] = f16x2(w0, w1);
            }
            if constexpr (S::kHalfV) store_frags(w_at + (h + k) * 2048, w[k]);
          }
          if constexpr (!S::kHalfV) {  // three 8-bit parts, two column groups together
#pragma unroll
            for (int k = 0; k < kB; k += 2) {
              if (8 * (h + k) >= rows) break;
              uint32_t p1[4], p2[4], p3[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                uint32_t x1[2], x2[2], x3[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t y = 8 * (h + k + x) < rows ? w[k + x][r] : 0u;
                  x1[x] = e5m2_of(y);
                  const uint32_t r1 = sub_mul(y, x1[x], 0x4c004c00u);  // times 2^4
                  x2[x] = e5m2_of(r1);
                  x3[x] = sub_mul(r1, x2[x], 0x4c004c00u);             // (an e5m2 number as it is)
                }
                p1[r] = __byte_perm(x1[0], x1[1], 0x7531);  // the upper bytes
                p2[r] = __byte_perm(x2[0], x2[1], 0x7531);
                p3[r] = __byte_perm(x3[0], x3[1], 0x7531);
              }
              const uint32_t to = w_at + (h + k) / 2 * 2048;
              store_frags(to, p1);
              store_frags(to + RT * kUnit, p2);
              store_frags(to + 2 * RT * kUnit, p3);
            }
          }
        }
        if (failed) break;
        begun = true;
        fence_proxy_async();
        tc_fence_before();
        if (ok) mbar_arrive(&p_full[u & 3]);
      }
      g += n_units;
      // ---- the segment's sums and outputs: the groups' states meet
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        float l[2];
        f2_unpack(l2[k], l[0], l[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
          if (lane < 4) red[warp][8 * k + c2 + i] = l[i];
        }
      }
      ok = ok && wait_for(&o_full, seg & 1, p);
      if (any_of(3, kSoft, !ok)) break;
      tc_fence_after();
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
            *reinterpret_cast<float2*>(p.part_ml + out_s[sb][n] * 2) = make_float2(m, l);
          else if (p.lse)
            p.lse[out_s[sb][n]] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      sync_of(3, kSoft);
      // (a group takes every other two columns of O; of three 8-bit parts, a column and the next are rows n
      // and n + 1)
#pragma unroll(S::kHalfV ? 4 : 2)
      for (int c = 2 * group; c < RT; c += 4) {
        const int n0 = S::kHalfV ? c : (c & ~15) + 2 * (c >> 2 & 3) + 8 * (c >> 1 & 1);
        if (n0 >= rows) continue;
#pragma unroll 1
        for (int half = 0; half < S::kHalves; ++half) {
          uint32_t o[2][S::kSums][2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < S::kSums; ++y)
              tmem_ld2(lanes + S::kColO + x * S::kOCols + (half * S::kSums + y) * RT + c, o[x][y]);
          tmem_wait_ld();
          const int d = half * 128 + tid;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int n = n0 + e;
            if (n >= rows || d >= D) break;
            float y = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float z = __uint_as_float(o[x][0][e]);
              if constexpr (!S::kHalfV)
                z += __uint_as_float(o[x][1][e]) * 0x1p-4f + __uint_as_float(o[x][2][e]) * 0x1p-8f;
              const float f = fac_s[x][n];
              y += f == 0.f ? 0.f : f * z;
            }
            if (any_nan[sb] && nan_s[sb][n][d >> 5] >> (d & 31) & 1) y = NAN;
            const float inv = inv_s[n];
            y = inv == 0.f ? 0.f : y * inv;
            const long long to = out_s[sb][n] * D + d;
            if (!whole) p.part_o[to] = y;
            else if constexpr (F16) reinterpret_cast<__half*>(p.out)[to] = __float2half_rn(y);
            else reinterpret_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(y);
          }
        }
      }
      tc_fence_before();
      sync_of(3, kSoft);  // the rows' state is free
      mbar_arrive(&seg_done[sb]);
    }
    report(ok, p);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, S::kAlloc);
}

// The sequences that lie in more than one range (and rows that see nothing): a warp joins a row's parts, in
// their order.
constexpr int kJoinWarps = 8;

template <int D, bool F16, int kFlight>  // kFlight parts are on their way at once
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p, int RT) {
  constexpr int kPer = D / 32;
  __shared__ int sums[kJoinWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = (p.R * p.Hq + kJoinWarps - 1) / kJoinWarps;
  const int b = blockIdx.x / per_seq, r = blockIdx.x % per_seq * kJoinWarps + warp;
  // (in front of its wait it reads the lengths only: what wrote them the kernel in front has waited for)
  int before = 0, W = 0;
  for (int x = threadIdx.x; x < p.B; x += 32 * kJoinWarps) {
    const int u = seq_of(p, x).span;
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
  chain_wait();
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
#pragma unroll 1
    for (int x0 = 0; x0 < np; x0 += kFlight) {
      float2 w[kFlight], y[kFlight][kPer / 2];
      float now = M;
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        if (x0 + x >= np) break;
        const size_t from = part(x0 + x);
        w[x] = __ldcg(ml + from);
#pragma unroll
        for (int c = 0; c < kPer / 2; ++c)
          y[x][c] = __ldcg(reinterpret_cast<const float2*>(p.part_o + from * D + kPer * lane) + c);
      }
#pragma unroll
      for (int x = 0; x < kFlight; ++x)
        if (x0 + x < np) now = fmaxf(now, w[x].x);
      const float f = fast_exp2(M - now);
      M = now;
      L *= f;
#pragma unroll
      for (int c = 0; c < kPer; ++c) acc[c] *= f;
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        if (x0 + x >= np) break;
        const float e = fast_exp2(w[x].x - M);
        L += e * w[x].y;
#pragma unroll
        for (int c = 0; c < kPer / 2; ++c) {
          acc[2 * c] += e * y[x][c].x;
          acc[2 * c + 1] += e * y[x][c].y;
        }
      }
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
}  // namespace scaled_attn
void attn_fault_setting(int* withhold_stage, unsigned long long* wait_ns);  // spec_debug_attn_fault's
namespace scaled_attn {

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
  // Sequences in many parts: one round trip for sixteen (one chain 18.6 us against 19.4 with eight); else eight,
  // whose registers leave room for twice the rows (draft trees 5 us less).
  constexpr int kMany = D == 256 ? 8 : 16, kFew = kMany / 2;
  const bool many = p.teams > 8ll * p.B * p.Hkv;
  const auto join = f16 ? many ? join_kernel<D, true, kMany> : join_kernel<D, true, kFew>
                        : many ? join_kernel<D, false, kMany> : join_kernel<D, false, kFew>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join, p, rt);
  return e == cudaSuccess ? launch_status() : SPEC_ECUDA;
}

spec_status launch_d64(const Params& p, int rt, bool f16, cudaStream_t st);
spec_status launch_d128(const Params& p, int rt, bool f16, cudaStream_t st);
spec_status launch_d256(const Params& p, int rt, bool f16, cudaStream_t st);

}  // namespace scaled_attn
