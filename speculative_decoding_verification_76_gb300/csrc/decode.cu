// spec_decode_attn -- attention of one new token per sequence over the paged
// cache, split over the cache's length and joined.
//
// Mathematics: query head h of sequence b over the seen positions t:
//   x_t = scale * q . k_t,  out = sum_t e^(x_t - m) v_t / l,  l = sum_t e^(x_t - m),
//   lse = m + ln l  for any reference m.
// Parts of the positions give (m, l, sum) each, and parts join by e^(m_i - M)
// ("Speculative Token Decoupling: Asynchronous Verification via Flash-Decoding",
// section 03: split-K attention).  Everything runs in the log2 domain, in fp32.
//
// What bounds it: HBM.  Every K and V row is read once (512 bytes per position
// and KV head at D = 128 in bf16, 256 in e4m3) for 4 D flops per query head.
//
// Design.  A CTA (4 warps) takes one KV head (up to 8 or 16 of its query heads)
// and one contiguous range of the batch's positions; all CTAs of a launch are
// resident at once and the ranges are cut evenly over the whole batch (units of
// 64 or 128 positions, counted from seq_len on the device), so ragged batches, one long
// sequence and the launch of a captured graph whose lengths change all fill the
// GPU alike.  The CTAs of a range's heads are neighbours in the grid and walk the
// same token rows together.
// A warp streams its positions straight from HBM into registers: no shared
// memory ring, no barrier in the loop.  That works because both products are
// taken transposed, heads as the MMA's 8 columns (m16n8k16, fp32 accumulate):
//   S^T = K Q^T: rows are 16 positions; a lane's 16-byte pieces of a K row are
//     the A fragments of two (16-bit) or four (8-bit) k-steps, in an order of
//     the D dimensions that Q's fragments share;
//   O^T = V^T P^T: a lane holds 16-byte pieces of the four V rows that its
//     fragment columns want, and byte permutes pair the rows; the rows of the
//     output tile are whatever dimensions those pieces hold.
//   P^T's fragments are S^T's accumulators, packed and transposed by movmatrix.
// K's loads for the next tile go out as soon as a subtile's S has taken its registers,
// V's when its product has; the page lookups are two tiles ahead.
// P is a sum hi + lo of two parts of the cache's 16-bit type, or of fp16 beside e4m3 caches
// (which convert to fp16 exactly), so that rounding P adds nothing to the output's own
// rounding.  Beside bf16 queries an e4m3 cache takes one fp16 part: its 2^-11 is an eighth of
// what the bf16 output is rounded by.  (Two parts: 64 ragged sequences with 16 heads a CTA 118
// against 115 us, with 4 heads 176 both; fp16 outputs, whose error one part would double, pay
// it.)
// An infinite V must come out infinite, and lo V alone would be an infinity of the other sign
// or 0 Inf: in bf16 hi is the number next below P, so that lo is positive too (lo < 2^-7 P,
// rounded to 2^-16 P); in fp16, where such a lo may fall below the smallest number, lo
// multiplies V with its infinities made finite.
// The reference m of a row stays until a score exceeds it by 15 (it is set 7 below the
// maximum: P stays in fp16's range).
//
// Measured: 64 ragged sequences (540 K positions, 32 / 8 heads of 128) in bf16 320 us =
// 6.93 TB/s, in e4m3 176 us = 6.3; one request of 8192 13 us, of 131072 in e4m3 with 64
// query heads 53 us.  A short call is a chain of round trips (lengths, page ids, K and V,
// merge, join: 2, 1, 5, 1.5 and 3 us).
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "serving.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Ranges are cut in units of the positions that a CTA's warps take at once: 64 or 128.
constexpr int kMinUnit = 16 * kWarps;
// How far past a sequence's end positions are counted (the next two tiles of a warp, the last
// unit's rest), or past the batch's (a thread's share of the sequences).
constexpr int kPast = 512;
constexpr int kMaxHeadGroups = 4096;  // KV heads x head groups
constexpr int kMaxCounters = 2 * kMaxHeadGroups;  // two per CTA
constexpr int kMaxJoin = 64;          // parts that the last CTA joins; more: join_kernel
constexpr float kBelow = 7.f;         // the reference sits this far under the maximum
constexpr float kSlack = 15.f;        // a score may exceed the reference by this much
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  const char *q, *k, *v;
  const int32_t *table, *seq_len;
  const float *k_scale, *v_scale;
  char* out;
  float *lse, *part_o, *part_ml;
  int32_t* counters;                         // by a sequence's first part: zero between calls
  long long q_stride_b, q_stride_h;          // elements
  long long head_stride;                     // bytes
  uint32_t token_stride;                     // bytes
  uint32_t page_rows;                        // page stride in token strides
  FastDiv P;                                 // page size
  int B, Hq, Hkv, G, groups, hpg, num_pages, max_pages, window, ranges, q_bf16;
  int deep;                                  // join_kernel follows
  float scale_log2;
};

// What is read in the place of positions that are not seen: an address instead of
// a branch or a predicate around the loads, which made the compiler wait for them
// there or keep their registers live (64 ragged sequences: 415 against 318 us).
// One row per warp of a few hundred, so that the reads behind the last tiles do not
// all ask one L2 slice (one row for all: 4 us at the end of each CTA).
constexpr int kZeroRows = 512;
__device__ __align__(512) char g_zeros[kZeroRows * 512];

enum Cache { kBf16, kF16, kE4m3, kE4m3F16 };  // (e4m3 beside bf16 and beside fp16 queries)

template <int CT>
constexpr bool is_e4m3() { return CT == kE4m3 || CT == kE4m3F16; }
template <int CT>
constexpr int elem_bytes() { return is_e4m3<CT>() ? 1 : 2; }

// D = A(16x16, row) * B(16x8, col) + D (fp32), f16 or bf16 operands
template <bool BF>
SPEC_DEV void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                  uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

SPEC_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

SPEC_DEV uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two halves, infinities (and NaN) replaced by the largest finite number of their sign
SPEC_DEV uint32_t finite_f16(uint32_t x) {
  uint32_t r;
  asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7bff7bffu));
  return r;
}

SPEC_DEV void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {  // bytes 0, 1 and 2, 3
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// N words of the cache, read once: not kept in L1, first out of L2
template <int N>
SPEC_DEV void load_words(uint32_t* w, const char* p, uint64_t pol) {
  if constexpr (N == 8)
    asm volatile(
        "ld.global.nc.L1::no_allocate.L2::cache_hint.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7])
        : "l"(p), "l"(pol));
  else if constexpr (N == 4)
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.b32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p), "l"(pol));
  else
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v2.b32 {%0,%1}, [%2], %3;"
                 : "=r"(w[0]), "=r"(w[1])
                 : "l"(p), "l"(pol));
}

SPEC_DEV int seen_from(const DecodeParams& p, int n) {
  return p.window > 0 && n > p.window ? n - p.window : 0;
}

// stored tokens of sequence b (never more than its table row can name)
SPEC_DEV int stored(const DecodeParams& p, int b) {
  const int n = p.seq_len[b];
  return n < 0 ? 0 : min(n, p.max_pages * p.P.d);
}

template <int U>
SPEC_DEV int units_of(const DecodeParams& p, int n) {
  return (n - seen_from(p, n) + U - 1) / U;
}

template <int N>
struct Row {  // a lane's N consecutive floats of a part's row
  float x[N];
  SPEC_DEV void load(const float* row, int lane) {
    if constexpr (N == 2) {
      const float2 y = __ldcg(reinterpret_cast<const float2*>(row) + lane);
      x[0] = y.x, x[1] = y.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(row + N * lane + i));
        x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
      }
    }
  }
};

// The nr ranges that W units are cut into: the first W % nr have one unit more.
struct Cuts {
  int q, rem;
  SPEC_DEV Cuts(int W, int nr) : q((uint32_t)W / (uint32_t)nr), rem(W - q * nr) {}
  SPEC_DEV int begin(int r) const { return r * q + min(r, rem); }
  SPEC_DEV int range_of(int unit) const {
    const int longer = rem * (q + 1);  // units of the longer ranges
    return unit < longer ? (uint32_t)unit / (uint32_t)(q + 1)
                         : rem + (uint32_t)(unit - longer) / (uint32_t)q;
  }
};

template <int CT, int D, int NT>
struct Shape {
  static constexpr int kBytes = D * elem_bytes<CT>();           // of a row
  static constexpr int kTile = 16 * kBytes <= 2048 ? 32 : 16;   // positions of a warp's tile
  static constexpr int kSub = kTile / 16;
  static constexpr int kUnit = kTile * kWarps;
  static constexpr int kKPieces = kBytes / 64;                  // 16-byte pieces per lane and row
  static constexpr int kVWords = kBytes >= 128 ? 4 : kBytes / 32;  // words of a lane's V piece
  static constexpr int kVPieces = kBytes >= 128 ? kBytes / 128 : 1;
  static constexpr int kSteps = D / 16;
  // A lane's 16-byte pieces of a row, in pairs where the row is long enough (one 32-byte
  // load): byte of piece j of lane c of 4 (K) and of lane n of 8 (V).
  static constexpr bool kPairK = kBytes >= 128, kPairV = kBytes >= 256;
  SPEC_DEV static constexpr int k_byte(int j) { return kPairK ? (j >> 1) * 128 + (j & 1) * 16 : j * 64; }
  SPEC_DEV static constexpr int v_byte(int j) { return kPairV ? (j >> 1) * 256 + (j & 1) * 16 : j * 128; }
  static constexpr int kLaneK = kPairK ? 32 : 16, kLaneV = kPairV ? 32 : kVWords * 4;
};

// The np <= kMaxJoin parts of sequence b's head group, joined by one CTA in their order: a
// warp per head, kFlight parts' rows loaded together (a part's row is an L2 round
// trip away, and one after another 57 parts took 12 us).  `late`: the first part is
// its range's last segment (slot 1).
template <int D>
__device__ __forceinline__ void join(const DecodeParams& p, int b, int r_first, int np, bool late,
                                  int hv, int nh) {
  constexpr int kPer = D / 32, kFlight = kPer > 4 ? 16 : 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, HV = p.Hkv * p.groups;
  const int kvh = hv / p.groups, h0 = hv % p.groups * p.hpg;
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
#pragma unroll 1
  for (int h = warp; h < nh; h += kWarps) {
    // row of part 0 of head h (in slot 0), and the rows from part to part
    const size_t row0 = ((size_t)r_first * 2 * HV + hv) * p.hpg + h;
    const int step = 2 * HV * p.hpg, slot1 = late ? HV * p.hpg : 0;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row0;
    auto ml_of = [&](int i) {
      return i < np ? __ldcg(ml + (size_t)i * step + (i == 0 ? slot1 : 0))
                    : make_float2(-INFINITY, 0.f);
    };
    float M = -INFINITY, L = 0.f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < np; j0 += kFlight) {
      // (loads clamped, not skipped: a skipped load's registers stay live)
      Row<kPer> y[kFlight];
      const float* src = p.part_o + (row0 + (size_t)j0 * step) * D;
      const size_t first = j0 == 0 ? (size_t)slot1 * D : 0;
#pragma unroll
      for (int j = 0; j < kFlight; ++j)
        y[j].load(src + (size_t)(min(j, np - 1 - j0) * step) * D + (j == 0 ? first : 0), lane);
      const float2 mine = ml_of(j0 + min(lane, kFlight));
      if (j0 == 0) {  // the references and sums of all parts, under the first rows' loads
        static_assert(kMaxJoin <= 64, "two parts a lane");
        const float2 x0 = ml_of(lane), x1 = ml_of(lane + 32);
        M = warp_max(fmaxf(x0.x, x1.x));
        auto weigh = [&](float2 x) { L += (x.x == -INFINITY ? 0.f : fast_exp2(x.x - M)) * x.y; };
        weigh(x0);
        weigh(x1);
        L = warp_sum(L);
      }
      const float e = mine.x == -INFINITY ? 0.f : fast_exp2(mine.x - M);
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const float ej = __shfl_sync(0xffffffffu, e, j);
        if (j0 + j < np) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] += ej * y[j].x[i];
        }
      }
    }
    const float f = L == 0.f ? 0.f : vs / L;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const uint32_t y = p.q_bf16 ? pack_bf16(acc[i] * f, acc[i + 1] * f)
                                  : pack_f16(acc[i] * f, acc[i + 1] * f);
      *reinterpret_cast<uint32_t*>(
          p.out + (((size_t)b * p.Hq + kvh * p.G + h0 + h) * D + kPer * lane + i) * 2) = y;
    }
    if (lane == 0 && p.lse)
      p.lse[(size_t)b * p.Hq + kvh * p.G + h0 + h] =
          L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

template <int CT, int D, int NT, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) decode_kernel(
    const __grid_constant__ DecodeParams p) {
  using S = Shape<CT, D, NT>;
  constexpr int kUnit = S::kUnit;
  constexpr bool kBf = CT == kBf16, k8 = is_e4m3<CT>(), kTwo = CT != kE4m3;  // (P as two parts)
  constexpr int NS = S::kSub, KP = S::kKPieces, VW = S::kVWords, VP = S::kVPieces;
  constexpr int kHeads = 8 * NT;
  // row (h & 1) * 4 + (h >> 1 & 3) of each eight is head h, two words apart modulo the
  // banks: a warp's float2 stores touch each bank once per half
  __shared__ __align__(16) float so[kWarps][kHeads][D + 2];
  __shared__ float sml[kWarps][kHeads][2];
  __shared__ int ssum[kWarps];
  // the segment being worked on: in shared memory, read again behind the barriers,
  // so that it holds no registers while the positions stream through
  __shared__ struct {
    int W, nr, w, w1;  // the batch's units and ranges; this CTA's next unit and its end
    int b, at;         // the sequence, and the units in front of it
  } seg;
  __shared__ int s_last;

  const int hv = blockIdx.x % (p.Hkv * p.groups), r = blockIdx.x / (p.Hkv * p.groups);
  const int kvh = hv / p.groups, h0 = hv % p.groups * p.hpg;   // first query head within G
  const int nh = min(p.hpg, p.G - h0);                         // query heads of this CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n8 = lane >> 2, c4 = lane & 3;
  const int HV = p.Hkv * p.groups;

  chain_wait();
  if (p.deep) chain_next();  // join_kernel: it finds its sequence meanwhile

  // ---- this CTA's units of the batch's W, and the sequence that holds the first:
  // every thread takes `per` consecutive sequences of one running sum
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int mine = 0;
    bool idle = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int u = units_of<kUnit>(p, stored(p, b));
      mine += u;
      idle = idle || u == 0;
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ssum[warp] = x;
    const bool idles = __syncthreads_or(idle);
    int before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += ssum[w];
      W += ssum[w];
    }
    if (idles) {  // rows that see nothing: zeros and -inf for this CTA's heads
#pragma unroll 1
      for (int b = r; b < p.B; b += p.ranges) {
        if (units_of<kUnit>(p, stored(p, b)) != 0) continue;
        const size_t row = (size_t)b * p.Hq + kvh * p.G + h0;
#pragma unroll 1
        for (int i = threadIdx.x; i < nh * D; i += kThreads)
          reinterpret_cast<uint16_t*>(p.out)[row * D + i] = 0;
        if (p.lse && threadIdx.x < nh) p.lse[row + threadIdx.x] = -INFINITY;
      }
    }
    const int nr = min(p.ranges, W);
    if (r >= nr) return;
    const Cuts cuts(W, nr);
    const int w0 = cuts.begin(r);
    int at = before + x - mine;
    if (at <= w0 && w0 < at + mine) {
      int b = b0, u;
#pragma unroll 1
      while (b + 1 < b1 && at + (u = units_of<kUnit>(p, stored(p, b))) <= w0) at += u, ++b;
      seg = {W, nr, w0, cuts.begin(r + 1), b, at};
    }
    __syncthreads();
  }

  const char* zeros = g_zeros + ((blockIdx.x * kWarps + warp) % kZeroRows) * 512;
  uint64_t pol;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  const char* kh = p.k + kvh * p.head_stride + c4 * S::kLaneK;
  const char* vh = p.v + kvh * p.head_stride + n8 * S::kLaneV;

  while (true) {
    const int b = seg.b;
    int t_begin, t_end;
    {
      const int n = stored(p, b), first = seen_from(p, n);
      t_begin = first + (seg.w - seg.at) * kUnit;
      const int left = seg.w1 - seg.at;  // units of this sequence up to the range's end
      t_end = left < units_of<kUnit>(p, n) ? first + left * kUnit : n;
    }
    const int32_t* bt = p.table + (size_t)b * p.max_pages;

    // ---- Q fragments (column n8 of tile nt is query head h0 + 8 nt + n8)
    uint32_t qf[NT][S::kSteps][2];
    float sc[NT][2];   // log2-domain scale of this lane's accumulator columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = 8 * nt + n8;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + b * p.q_stride_b +
                            (kvh * p.G + h0 + min(g, nh - 1)) * p.q_stride_h;
      uint32_t raw[S::kSteps * 2];
      if constexpr (k8) {  // 16 dimensions per lane and piece
#pragma unroll
        for (int j = 0; j < KP; ++j) {
          const uint4* s4 = reinterpret_cast<const uint4*>(src + c4 * S::kLaneK + S::k_byte(j));
          const uint4 x = s4[0], y = s4[1];
          raw[8 * j] = x.x, raw[8 * j + 1] = x.y, raw[8 * j + 2] = x.z, raw[8 * j + 3] = x.w;
          raw[8 * j + 4] = y.x, raw[8 * j + 5] = y.y, raw[8 * j + 6] = y.z, raw[8 * j + 7] = y.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < KP; ++j) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + (c4 * S::kLaneK + S::k_byte(j)) / 2);
          raw[4 * j] = x.x, raw[4 * j + 1] = x.y, raw[4 * j + 2] = x.z, raw[4 * j + 3] = x.w;
        }
      }
      float up = 1.f;
      if constexpr (CT == kE4m3) {
        // bf16 q beside fp16 operands: scaled by a power of two that puts the
        // head's largest element at 2^14, so that nothing overflows and what
        // becomes subnormal is 2^-28 of the largest
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < S::kSteps * 2; ++i)
          big = fmaxf(big, fmaxf(fabsf(__uint_as_float(raw[i] << 16)),
                                 fabsf(__uint_as_float(raw[i] & 0xffff0000u))));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int e = (int)(__float_as_uint(big) >> 23) - 127;   // exponent of the largest
        if (!(big > 0.f) || e > 127) e = 14;               // zero, Inf or NaN: as it is
        e = max(e, -100);
        const float down = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        up = __uint_as_float((uint32_t)(127 + e - 14) << 23);
#pragma unroll
        for (int i = 0; i < S::kSteps * 2; ++i)
          raw[i] = pack_f16(__uint_as_float(raw[i] << 16) * down,
                            __uint_as_float(raw[i] & 0xffff0000u) * down);
      }
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) {
        qf[nt][i][0] = raw[2 * i];
        qf[nt][i][1] = raw[2 * i + 1];
      }
      const float mul = p.scale_log2 * (p.k_scale ? p.k_scale[kvh] : 1.f) * up;
      sc[nt][0] = __shfl_sync(0xffffffffu, mul, 8 * c4);       // head 2 c4 of the tile
      sc[nt][1] = __shfl_sync(0xffffffffu, mul, 8 * c4 + 4);   // head 2 c4 + 1
    }

    float o[NT][S::kSteps][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // page of this lane's position of the tile at t0: the raw table entry (-1: none)
    const int tl = lane % S::kTile;
    auto entry = [&](int t0) {
      const int t = t0 + tl;
      return t < t_end ? bt[p.P.quot(t)] : -1;
    };
    // cache row of that position, in token strides (-1: not seen)
    auto row_of = [&](int t0, int id) {
      const int t = t0 + tl;
      return id >= 0 && id < p.num_pages ? (int)(id * p.page_rows + (t - p.P.quot(t) * p.P.d)) : -1;
    };
    uint32_t kr[NS][2][KP][4], vr[NS][4][VP][VW];
    bool seen_next[NS][2];
    auto load_k = [&](int row, int s) {  // subtile s of the tile whose rows the lanes hold
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rr = __shfl_sync(0xffffffffu, row, 16 * s + 8 * x + n8);
          seen_next[s][x] = rr >= 0;
          const char* src = rr >= 0 ? kh + (uint64_t)(uint32_t)rr * p.token_stride : zeros;
#pragma unroll
          for (int j = 0; j < KP; j += S::kPairK ? 2 : 1)
            load_words<S::kPairK ? 8 : 4>(kr[s][x][j], src + S::k_byte(j), pol);
        }
    };
    auto load_v = [&](int row, int s) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int rr = __shfl_sync(0xffffffffu, row, 16 * s + 8 * (x >> 1) + 2 * c4 + (x & 1));
          const char* src = rr >= 0 ? vh + (uint64_t)(uint32_t)rr * p.token_stride : zeros;
#pragma unroll
          for (int j = 0; j < VP; j += S::kPairV ? 2 : 1)
            load_words<S::kPairV ? 8 : VW>(vr[s][x][j], src + S::v_byte(j), pol);
        }
    };

    constexpr int kStride = kWarps * S::kTile;
    static_assert(2 * kStride + 32 + kUnit <= kPast, "32-bit positions");
    int t0 = t_begin + warp * S::kTile;
    int row = row_of(t0, entry(t0));
#pragma unroll
    for (int s = 0; s < NS; ++s) load_k(row, s);
#pragma unroll
    for (int s = 0; s < NS; ++s) load_v(row, s);
    int id_next = entry(t0 + kStride);
    bool more = t0 < t_end;
#pragma unroll 1
    while (more) {
      // ---- S^T = K Q^T; a subtile's registers take the next tile's K at once (its
      // page ids came with the tile before)
      t0 += kStride;
      more = t0 < t_end;
      const int row_next = row_of(t0, id_next);
      id_next = entry(t0 + kStride);
      float x[NS][NT][4];
      bool seen[NS][2];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        seen[s][0] = seen_next[s][0];
        seen[s][1] = seen_next[s][1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[s][nt][0] = x[s][nt][1] = x[s][nt][2] = x[s][nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KP; ++j) {
          if constexpr (k8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a0, a1, a2, a3;
              e4m3_to_f16(kr[s][0][j][i], a0, a2);
              e4m3_to_f16(kr[s][1][j][i], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<false>(x[s][nt], a0, a1, a2, a3, qf[nt][4 * j + i][0], qf[nt][4 * j + i][1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<kBf>(x[s][nt], kr[s][0][j][2 * i], kr[s][1][j][2 * i], kr[s][0][j][2 * i + 1],
                         kr[s][1][j][2 * i + 1], qf[nt][2 * j + i][0], qf[nt][2 * j + i][1]);
          }
        }
        load_k(row_next, s);
      }
      // ---- scale, what is not seen, the reference
      bool over = false;
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = seen[s][e >> 1] ? x[s][nt][e] * sc[nt][e & 1] : -INFINITY;
            x[s][nt][e] = y;
            over = over || y > m[nt][e & 1] + kSlack;
          }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -INFINITY;
#pragma unroll
            for (int s = 0; s < NS; ++s) top = fmax3(top, x[s][nt][e], x[s][nt][e + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float now = fmaxf(m[nt][e], top - kBelow);
            const float a = m[nt][e] == -INFINITY ? 0.f : fast_exp2(m[nt][e] - now);
            m[nt][e] = now;
            l[nt][e] *= a;
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
              o[nt][i][e] *= a;
              o[nt][i][e + 2] *= a;
            }
          }
      }
      // ---- P^T fragments, then O^T += V^T P^T
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ref = m[nt][e & 1];
            y[e] = fast_exp2(x[s][nt][e] - (ref == -INFINITY ? 0.f : ref));
          }
          l[nt][0] += y[0] + y[2];
          l[nt][1] += y[1] + y[3];
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2) {
            const float y0 = y[2 * x2], y1 = y[2 * x2 + 1];
            if constexpr (kBf) {  // hi: the bf16 number next below, so that lo > 0
              const uint32_t u0 = max(__float_as_uint(y0), 1u) - 1, u1 = max(__float_as_uint(y1), 1u) - 1;
              ph[nt][x2] = transpose8x8(__byte_perm(u0, u1, 0x7632));
              pl[nt][x2] = transpose8x8(pack_bf16(y0 - __uint_as_float(u0 & 0xffff0000u),
                                                  y1 - __uint_as_float(u1 & 0xffff0000u)));
            } else {
              const uint32_t hi = pack_f16(y0, y1);
              ph[nt][x2] = transpose8x8(hi);
              if constexpr (kTwo) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                pl[nt][x2] = transpose8x8(pack_f16(y0 - f.x, y1 - f.y));
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < VP; ++j)
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const uint32_t v0 = vr[s][0][j][i], v1 = vr[s][1][j][i];
            const uint32_t v2 = vr[s][2][j][i], v3 = vr[s][3][j][i];
            if constexpr (k8) {
              const uint32_t a = __byte_perm(v0, v1, 0x5140), b2 = __byte_perm(v2, v3, 0x5140);
              const uint32_t c = __byte_perm(v0, v1, 0x7362), d = __byte_perm(v2, v3, 0x7362);
              const int t = 2 * (j * VW + i);
              uint32_t f[8];
              e4m3_to_f16(a, f[0], f[1]);
              e4m3_to_f16(b2, f[2], f[3]);
              e4m3_to_f16(c, f[4], f[5]);
              e4m3_to_f16(d, f[6], f[7]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<false>(o[nt][t], f[0], f[1], f[2], f[3], ph[nt][0], ph[nt][1]);
                mma<false>(o[nt][t + 1], f[4], f[5], f[6], f[7], ph[nt][0], ph[nt][1]);
                if constexpr (kTwo) {
                  mma<false>(o[nt][t], f[0], f[1], f[2], f[3], pl[nt][0], pl[nt][1]);
                  mma<false>(o[nt][t + 1], f[4], f[5], f[6], f[7], pl[nt][0], pl[nt][1]);
                }
              }
            } else {
              const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
              const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
              const int t = j * VW + i;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<kBf>(o[nt][t], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                if constexpr (kBf)
                  mma<kBf>(o[nt][t], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                else
                  mma<kBf>(o[nt][t], finite_f16(a0), finite_f16(a1), finite_f16(a2),
                           finite_f16(a3), pl[nt][0], pl[nt][1]);
              }
            }
          }
        load_v(row_next, s);
      }
    }

    // ---- the warps' parts meet in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nt][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        const int h = 8 * nt + 2 * c4 + e;
        if (n8 == 0) {
          sml[warp][h][0] = m[nt][e];
          sml[warp][h][1] = y;
        }
        // tile t of the output: dimensions (piece, word) of this lane's V bytes
#pragma unroll
        for (int t = 0; t < S::kSteps; ++t) {
          int d;
          if constexpr (k8)
            d = S::v_byte(t / (2 * VW)) + n8 * S::kLaneV + (t % (2 * VW)) * 2;
          else
            d = (S::v_byte(t / VW) + n8 * S::kLaneV) / 2 + (t % VW) * 2;
          *reinterpret_cast<float2*>(&so[warp][8 * nt + 4 * e + c4][d]) = make_float2(o[nt][t][e], o[nt][t][e + 2]);
        }
      }
    __syncthreads();

    // parts of this sequence: ranges r_first .. r_last
    const int at = seg.at, units = units_of<kUnit>(p, stored(p, b));
    const Cuts cuts(seg.W, seg.nr);
    int r_first = r, r_last = r;
    if (at < cuts.begin(r)) r_first = cuts.range_of(at);
    if (at + units > seg.w1) r_last = min(cuts.range_of(at + units - 1), p.ranges - 1);
    const bool whole = r_first == r_last;
    const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
    // slot 0: the segment a range begins with; slot 1: its last one, if another
    const bool begins = seg.w == cuts.begin(r);
    const size_t part = ((size_t)r * 2 + (begins ? 0 : 1)) * HV + hv;
#pragma unroll 1
    for (int h = warp; h < nh; h += kWarps) {
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sml[i][h][0]);
      float e[kWarps], L = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        e[i] = sml[i][h][0] == -INFINITY ? 0.f : fast_exp2(sml[i][h][0] - M);
        L += e[i] * sml[i][h][1];
      }
      const float f = whole ? (L == 0.f ? 0.f : vs / L) : 1.f;
      const int hr = (h & ~7) + 4 * (h & 1) + (h >> 1 & 3);
      for (int d = 2 * lane; d < D; d += 64) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 y = *reinterpret_cast<const float2*>(&so[i][hr][d]);
          a.x += e[i] * y.x;
          a.y += e[i] * y.y;
        }
        if (whole) {
          const uint32_t y = p.q_bf16 ? pack_bf16(a.x * f, a.y * f) : pack_f16(a.x * f, a.y * f);
          *reinterpret_cast<uint32_t*>(p.out + (((size_t)b * p.Hq + kvh * p.G + h0 + h) * D + d) * 2) = y;
        } else {
          *reinterpret_cast<float2*>(p.part_o + (part * p.hpg + h) * D + d) = a;
        }
      }
      if (lane == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + (part * p.hpg + h) * 2) = make_float2(M, L);
        else if (p.lse)
          p.lse[(size_t)b * p.Hq + kvh * p.G + h0 + h] =
              L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
      }
    }
    if (!whole) {
      // ---- the last CTA of the sequence's parts joins them, in their order (the
      // barriers carry the CTA's stores to, and the others' from, one thread's atomic)
      __syncthreads();
      if (threadIdx.x == 0) {
        s_last = 0;
        if (r_last - r_first < kMaxJoin) {  // (more parts: join_kernel's)
          int32_t* cnt =
              p.counters + ((size_t)r_first * 2 + (cuts.begin(r_first) != at)) * HV + hv;
          int before;
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(cnt)
                       : "memory");
          s_last = before == r_last - r_first;
          if (s_last) *cnt = 0;  // ready for the next call
        }
      }
      __syncthreads();
      if (s_last)
        join<D>(p, b, r_first, r_last - r_first + 1, cuts.begin(r_first) != at, hv, nh);
    }
    // ---- the next sequence that has units
    __syncthreads();  // the shared parts and the control block are free
    if (at + units >= seg.w1 || b + 1 >= p.B) return;
    __syncthreads();
    if (threadIdx.x == 0) {
      int nb = b + 1;  // (there is one: units are left)
      while (nb + 1 < p.B && units_of<kUnit>(p, stored(p, nb)) == 0) ++nb;
      seg.w = seg.at = at + units;
      seg.b = nb;
    }
    __syncthreads();
  }
}

// The sequences cut into more than kMaxJoin parts (one of a few KV heads over all the
// GPU: joining 304 parts of 16 heads in one CTA took 50 us): a CTA per head of the k-th
// such sequence.  Launched as a programmatic dependent of decode_kernel, and only where
// the batch may have one.  Neighbours share a range at most, so k such sequences span
// 64 k + 1 ranges or more: there are at most (ranges - 1) / kMaxJoin.
constexpr int kJoinWarps = 16;

template <int D, int kUnit>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kPer = D / 32, kFlight = 8;
  __shared__ float e[1024];  // parts' weights (ranges <= 1024)
  __shared__ __align__(16) float so[kJoinWarps][D];
  __shared__ int part[kJoinWarps];
  __shared__ float fpart[kJoinWarps];
  __shared__ int s_b, s_at, s_u;
  const int k = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, HV = p.Hkv * p.groups;
  const int kvh = hq / p.G, hv = kvh * p.groups + hq % p.G / p.hpg, h = hq % p.G % p.hpg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // exclusive running sum over the block; *all: the sum
  auto scan = [&](int v, int* all) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int before = 0;
    *all = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) before += part[w];
      *all += part[w];
    }
    return before + x - v;
  };
  auto reduce = [&](float v, auto op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) fpart[warp] = v;
    __syncthreads();
    v = fpart[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) v = op(v, fpart[w]);
    return v;
  };
  const int per = (p.B + 32 * kJoinWarps - 1) / (32 * kJoinWarps);
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  int mine = 0, W, many, deep = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += units_of<kUnit>(p, stored(p, b));
  const int pre = scan(mine, &W), nr = min(p.ranges, W);
  // No block ends without the wait: decode_kernel released this grid early, and what
  // follows on the stream is ordered behind this grid alone.
  if (nr <= kMaxJoin) return chain_wait();
  const Cuts cuts(W, nr);
  auto is_deep = [&](int at, int u) {
    return u >= kMaxJoin && cuts.range_of(at + u - 1) - cuts.range_of(at) >= kMaxJoin;
  };
  int at = pre;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int u = units_of<kUnit>(p, stored(p, b));
    deep += is_deep(at, u);
    at += u;
  }
  int nth = scan(deep, &many);
  if (k >= many) return chain_wait();
  at = pre;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int u = units_of<kUnit>(p, stored(p, b));
    if (is_deep(at, u) && nth++ == k) {
      s_b = b;
      s_at = at;
      s_u = u;
    }
    at += u;
  }
  __syncthreads();
  const int b = s_b, r_first = cuts.range_of(s_at);
  const int np = cuts.range_of(s_at + s_u - 1) - r_first + 1;
  const bool late = cuts.begin(r_first) != s_at;
  auto row_of = [&](int i) {  // part i of head h
    return (((size_t)(r_first + i) * 2 + (i == 0 && late)) * HV + hv) * p.hpg + h;
  };
  chain_wait();
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float2 x[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = threadIdx.x + u * 32 * kJoinWarps;
    x[u] = i < np ? __ldcg(ml + row_of(i)) : make_float2(-INFINITY, 0.f);
  }
  const float M = reduce(fmaxf(x[0].x, x[1].x), [](float a, float c) { return fmaxf(a, c); });
  float l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float w = x[u].x == -INFINITY ? 0.f : fast_exp2(x[u].x - M);
    l += w * x[u].y;
    e[threadIdx.x + u * 32 * kJoinWarps] = w;
  }
  const float L = reduce(l, [](float a, float c) { return a + c; });  // (and e is written)
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int i0 = warp; i0 < np; i0 += kJoinWarps * kFlight) {
    Row<kPer> y[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      y[j].load(p.part_o + row_of(min(i0 + j * kJoinWarps, np - 1)) * D, lane);
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int i = i0 + j * kJoinWarps;
      if (i < np) {
#pragma unroll
        for (int d = 0; d < kPer; ++d) acc[d] += e[i] * y[j].x[d];
      }
    }
  }
#pragma unroll
  for (int d = 0; d < kPer; d += 2)
    *reinterpret_cast<float2*>(&so[warp][kPer * lane + d]) = make_float2(acc[d], acc[d + 1]);
  __syncthreads();
  const size_t o = (size_t)b * p.Hq + hq;
  const float f = L == 0.f ? 0.f : (p.v_scale ? p.v_scale[kvh] : 1.f) / L;
  if (2 * threadIdx.x < D) {
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float2 y = *reinterpret_cast<const float2*>(&so[w][2 * threadIdx.x]);
      a.x += y.x;
      a.y += y.y;
    }
    *reinterpret_cast<uint32_t*>(p.out + (o * D + 2 * threadIdx.x) * 2) =
        p.q_bf16 ? pack_bf16(a.x * f, a.y * f) : pack_f16(a.x * f, a.y * f);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[o] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------ host side
// SMs of the current device, asked once per device (the query costs host time)
int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

struct DecodePlan {
  int G, groups, hpg, nt, ranges;
};

constexpr int kMostPerSm = 4;  // CTAs of any instance on an SM

// CTAs an SM holds at the instance's register bound.  Three of 168 registers take tiles of
// 8 KB a warp (four of 128 with smaller tiles or fewer loads in flight: e4m3 at D = 128
// 187 against 180 us on 64 ragged sequences, 16 bits at D = 64 178 against 172); D = 256
// and 16 heads a CTA need 255.
constexpr int per_sm(bool e4m3, int D, int nt) {
  return D == 256 || nt == 2 ? 2 : e4m3 && D == 64 ? 4 : 3;
}

// occ: CTAs an SM holds (0: of the instance that the shape selects)
bool make_plan(int B, int Hq, int Hkv, int D, bool e4m3, int occ, DecodePlan* pl) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv) return false;
  pl->G = Hq / Hkv;
  // query heads of a CTA: up to 16 share one read of K and V (8 where D = 256 fills the
  // registers; the other groups read the same rows from L2 at the same time)
  const int most = D == 256 ? 8 : 16;
  pl->groups = (pl->G + most - 1) / most;
  pl->hpg = (pl->G + pl->groups - 1) / pl->groups;
  pl->groups = (pl->G + pl->hpg - 1) / pl->hpg;
  pl->nt = pl->hpg > 8 ? 2 : 1;
  if (occ == 0) occ = per_sm(e4m3, D, pl->nt);
  pl->ranges = std::max(1, std::min(1024, num_sms() * occ / (Hkv * pl->groups)));
  return true;
}

size_t ws_layout(const DecodePlan& pl, int Hkv, int D, size_t* off_o, size_t* off_ml) {
  const size_t rows = (size_t)pl.ranges * 2 * Hkv * pl.groups * pl.hpg;
  size_t off = sizeof(WsHeader) + (size_t)kMaxCounters * sizeof(int32_t);
  *off_o = off;
  off += (rows * D * sizeof(float) + 255) / 256 * 256;
  *off_ml = off;
  off += (rows * 2 * sizeof(float) + 255) / 256 * 256;
  return off;
}

template <int CT, int D, int NT>
spec_status launch(DecodeParams p, cudaStream_t st) {
  constexpr int kOcc = per_sm(is_e4m3<CT>(), D, NT);
  // may a sequence be cut into more parts than its last CTA joins?  (Each holds a unit at
  // least, and the window or the table's width bounds its units.)
  const int row = p.max_pages * p.P.d, longest = p.window > 0 ? std::min(p.window, row) : row;
  p.deep = p.ranges > kMaxJoin && longest / kMinUnit + 1 > kMaxJoin;
  const spec_status rc = launch_chained(decode_kernel<CT, D, NT, kOcc>,
                                        p.ranges * p.Hkv * p.groups, kThreads, 0, st, p);
  if (rc != SPEC_OK || !p.deep) return rc;
  return launch_chained(join_kernel<D, Shape<CT, D, NT>::kUnit>, p.ranges / kMaxJoin * p.Hq,
                        32 * kJoinWarps, 0, st, p);
}

template <int CT>
spec_status launch_d(const DecodeParams& p, int D, int nt, cudaStream_t st) {
  if (D == 64) return nt == 1 ? launch<CT, 64, 1>(p, st) : launch<CT, 64, 2>(p, st);
  if (D == 128) return nt == 1 ? launch<CT, 128, 1>(p, st) : launch<CT, 128, 2>(p, st);
  return launch<CT, 256, 1>(p, st);
}

}  // namespace

extern "C" size_t spec_decode_attn_workspace_size(int B, int Hq, int Hkv, int D) {
  DecodePlan pl;
  if ((D != 64 && D != 128 && D != 256) || !make_plan(B, Hq, Hkv, D, false, kMostPerSm, &pl)) return 0;
  size_t a, c;
  return ws_layout(pl, Hkv, D, &a, &c);
}

extern "C" spec_status spec_decode_attn(const void* q, int64_t q_stride_b, int64_t q_stride_h,
                                        spec_dtype q_dtype, const void* k_cache,
                                        const void* v_cache, spec_dtype cache_dtype,
                                        const float* k_scale, const float* v_scale, int num_pages,
                                        int page_size, int64_t page_stride, int64_t token_stride,
                                        int64_t head_stride, const int32_t* block_table,
                                        int max_pages, const int32_t* seq_len, int B, int Hq,
                                        int Hkv, int D, int window, float scale, void* workspace,
                                        size_t workspace_bytes, void* out, float* lse_out,
                                        void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_pages < 1 || page_size < 1 || max_pages < 1 ||
      window < 0)
    return SPEC_EINVAL;
  if (q_dtype == SPEC_F32 || cache_dtype == SPEC_F32) return SPEC_EUNSUPPORTED;
  if (q_dtype != SPEC_BF16 && q_dtype != SPEC_F16) return SPEC_EINVAL;
  const bool e4m3 = cache_dtype == SPEC_E4M3;
  if (!e4m3 && cache_dtype != q_dtype) return SPEC_EINVAL;
  if (!e4m3 && (k_scale || v_scale)) return SPEC_EINVAL;
  if (D != 64 && D != 128 && D != 256) return SPEC_EUNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_len || !workspace || !out)
    return SPEC_EINVAL;
  const int es = e4m3 ? 1 : 2;
  if ((((uintptr_t)q | (uintptr_t)out) & 15) || (((uintptr_t)k_cache | (uintptr_t)v_cache) & 31))
    return SPEC_EINVAL;
  if ((uintptr_t)workspace & 255) return SPEC_EINVAL;
  if (q_stride_b < 0 || q_stride_h < 0 || page_stride < 0 || token_stride < 1 || head_stride < 0)
    return SPEC_EINVAL;
  if ((((q_stride_b | q_stride_h) * 2) & 15) ||
      (((page_stride | token_stride | head_stride) * es) & 31))
    return SPEC_EINVAL;
  // cache rows are numbered in token strides, in 31 bits
  if (page_stride % token_stride || token_stride * es > UINT32_MAX) return SPEC_EUNSUPPORTED;
  const int64_t page_rows = page_stride / token_stride;
  if (page_rows > INT32_MAX || (page_rows * (num_pages - 1) + page_size) > INT32_MAX ||
      (long long)max_pages * page_size > INT32_MAX - kPast || B > INT32_MAX - kPast)
    return SPEC_EUNSUPPORTED;
  // so are the batch's units
  if (((long long)max_pages * page_size / kMinUnit + 1) * B > INT32_MAX) return SPEC_EUNSUPPORTED;
  DecodePlan pl;
  if (!make_plan(B, Hq, Hkv, D, e4m3, 0, &pl)) return SPEC_EINVAL;
  if ((long long)Hkv * pl.groups > kMaxHeadGroups) return SPEC_EUNSUPPORTED;
  size_t off_o, off_ml;
  if (workspace_bytes < ws_layout(pl, Hkv, D, &off_o, &off_ml)) return SPEC_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeParams p{};
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k_cache);
  p.v = static_cast<const char*>(v_cache);
  p.table = block_table;
  p.seq_len = seq_len;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.out = static_cast<char*>(out);
  p.lse = lse_out;
  p.counters = reinterpret_cast<int32_t*>(ws + sizeof(WsHeader));
  p.part_o = reinterpret_cast<float*>(ws + off_o);
  p.part_ml = reinterpret_cast<float*>(ws + off_ml);
  p.q_stride_b = q_stride_b;
  p.q_stride_h = q_stride_h;
  p.head_stride = head_stride * es;
  p.token_stride = (uint32_t)(token_stride * es);
  p.page_rows = (uint32_t)page_rows;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = pl.G;
  p.groups = pl.groups;
  p.hpg = pl.hpg;
  p.P = FastDiv(page_size);
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.window = window;
  p.ranges = pl.ranges;
  p.q_bf16 = q_dtype == SPEC_BF16;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (e4m3)
    return p.q_bf16 ? launch_d<kE4m3>(p, D, pl.nt, st) : launch_d<kE4m3F16>(p, D, pl.nt, st);
  return p.q_bf16 ? launch_d<kBf16>(p, D, pl.nt, st) : launch_d<kF16>(p, D, pl.nt, st);
}
