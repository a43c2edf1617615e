// Rotary positions in the forms of spec_rope, shared by rotate.cu and append_scaled.cu.
//
// A pair's angle at position t is kept as a 64-bit fraction of a turn: F_i = f_i / 2 pi modulo
// one turn times 2^64, and t F_i modulo 2^64 is the angle with the whole turns gone, as exact as
// the double that f_i comes from, with integer multiplies and no FP64 (whose rate on this GPU is
// a small part of fp32's).
//
// Work items of a head: two chunks of 8 elements and the table entries of their 8 pairs.  Item j
// has entries 8 j .. 8 j + 7; entries behind the turning pairs are the identity, so a partly
// turned head needs no branch.
//   halves:     chunks j and j + dim/16 while 8 j < dim/2, behind that two neighbours that stay
//   neighbours: chunks 2 j and 2 j + 1
#pragma once
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_fp16.h>

#include "serving.cuh"

constexpr int kMaxRopePairs = 256;

template <int N = kMaxRopePairs>
struct RopeTable {
  uint64_t turn[N];  // 2^64 x turns per position, of each pair
  float magnitude;
  int pairs, interleaved;  // turning pairs (0: no rotation)
};

// Checks a spec_rope for heads of D elements and fills the table.  The last one's frequencies
// are kept per host thread: the powers cost more host time than a launch.
template <int N>
static inline spec_status rope_table(const spec_rope* r, int D, RopeTable<N>* out) {
  out->pairs = 0;
  out->interleaved = 0;
  out->magnitude = 1.f;
  if (!r || r->dim == 0) return SPEC_OK;
  if (r->dim < 0 || r->dim > D || r->dim > 2 * N || r->dim % 2 || r->reserved != 0)
    return SPEC_EINVAL;
  if (!r->interleaved && r->dim % 16) return SPEC_EUNSUPPORTED;
  if (!std::isfinite(r->magnitude)) return SPEC_EINVAL;
  const int n = r->dim;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  auto fraction = [&](double f) {  // of a turn, in units of 2^-64
    double t = f / kTwoPi;
    t -= std::floor(t);
    return (uint64_t)std::llround(t * 0x1p62) * 4;
  };
  out->pairs = n / 2;
  out->interleaved = r->interleaved != 0;
  out->magnitude = (float)r->magnitude;
  if (r->freqs) {
    for (int i = 0; i < n / 2; ++i) {
      if (!std::isfinite(r->freqs[i])) return SPEC_EINVAL;
      out->turn[i] = fraction(r->freqs[i]);
    }
    return SPEC_OK;
  }
  const bool scaled = r->scaling != SPEC_ROPE_NONE, parts = r->scaling == SPEC_ROPE_PARTS;
  if (r->scaling < SPEC_ROPE_NONE || r->scaling > SPEC_ROPE_PARTS) return SPEC_EINVAL;
  if (!(r->base > 1.0 && std::isfinite(r->base))) return SPEC_EINVAL;
  if (scaled && !(r->factor >= 1.0 && std::isfinite(r->factor))) return SPEC_EINVAL;
  if (r->scaling == SPEC_ROPE_NTK && n <= 2) return SPEC_EINVAL;
  if (parts && !(r->original_len > 0.0 && std::isfinite(r->original_len) && r->low < r->high &&
                 std::isfinite(r->low) && std::isfinite(r->high)))
    return SPEC_EINVAL;
  struct Key {
    int dim, scaling;
    double base, factor, original_len, low, high;
    bool operator==(const Key& o) const {
      return dim == o.dim && scaling == o.scaling && base == o.base && factor == o.factor &&
             original_len == o.original_len && low == o.low && high == o.high;
    }
  };
  const Key key{n,
                r->scaling,
                r->base,
                scaled ? r->factor : 1.0,
                parts ? r->original_len : 0.0,
                parts ? r->low : 0.0,
                parts ? r->high : 0.0};
  static thread_local struct {
    Key key;
    uint64_t turn[N];
  } last = {};
  if (!(last.key == key)) {
    double base = r->base;
    if (r->scaling == SPEC_ROPE_NTK) base *= std::pow(r->factor, (double)n / (n - 2));
    for (int i = 0; i < n / 2; ++i) {
      double f = std::pow(base, -2.0 * i / n);
      if (r->scaling == SPEC_ROPE_LINEAR) f /= r->factor;
      if (parts) {
        const double turns = r->original_len * f / kTwoPi;
        const double g = std::min(1.0, std::max(0.0, (turns - r->low) / (r->high - r->low)));
        f = f * g + f / r->factor * (1.0 - g);
      }
      last.turn[i] = fraction(f);
    }
    last.key = key;
  }
  std::memcpy(out->turn, last.turn, sizeof(uint64_t) * (n / 2));
  return SPEC_OK;
}

// Cosine and sine of a pair that turns by `turn` at position t, times the magnitude.
//
// The angle as a 32-bit fraction of a turn is split into the nearest quarter and a rest of at most an
// eighth of a turn, d + e with d what fp32 holds of it: sin and cos of d, and e (below 2^-26 of a turn)
// by the first term of its series.  An fp32 angle of up to half a turn alone would be off by 2^-24,
// twice what rounding the result costs, and shows in the codes of a cache that is written from it.
SPEC_DEV float2 rope_angle(uint64_t turn, float magnitude, int t) {
  const uint32_t frac = (uint32_t)(((uint64_t)(uint32_t)t * turn) >> 32);
  const uint32_t quarter = (frac + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(frac - (quarter << 30));
  const float d = (float)rest;
  const float e = (float)(rest - (int32_t)d) * (6.28318531f * 0x1p-32f);  // radians
  float s, c;
  sincospif(d * 0x1p-31f, &s, &c);
  const float s1 = fmaf(c, e, s), c1 = fmaf(-s, e, c);
  const float x = quarter & 1 ? -s1 : c1, y = quarter & 1 ? c1 : s1;
  const float m = quarter & 2 ? -magnitude : magnitude;
  return make_float2(x * m, y * m);
}

// The same of pair i (identity behind the pairs).  Lanes ask for different pairs, and constant memory serves them
// one after the other: where a thread needs a pair at many positions it reads its turn once.
template <int N>
SPEC_DEV float2 rope_entry(const RopeTable<N>& r, int t, int i) {
  return i < r.pairs ? rope_angle(r.turn[i], r.magnitude, t) : make_float2(1.f, 0.f);
}

// First and second chunk of item j.
template <int N>
SPEC_DEV int2 rope_chunks(const RopeTable<N>& r, int j) {
  const int half = r.interleaved ? 0 : r.pairs / 8;  // chunks of a half
  return j < half ? make_int2(j, j + half) : make_int2(2 * j, 2 * j + 1);
}

// A position's table of cosines (or sines) in shared memory, D / 2 of them: pairs 8 j + x of all items j with
// x < 4 lie in front of those with x >= 4, so that the lanes' 16-byte reads stand next to each other.
SPEC_DEV int rope_place(int items, int pair) {
  return (((pair >> 2 & 1) * items + (pair >> 3)) << 2) + (pair & 3);
}

// The pairs of item j of `items`, turned.
SPEC_DEV void rope_turn(bool interleaved, float* a, float* b, const float* cosines,
                        const float* sines, int items, int j) {
  float cs[8], sn[8];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    *reinterpret_cast<float4*>(cs + 4 * x) =
        *reinterpret_cast<const float4*>(cosines + ((x * items + j) << 2));
    *reinterpret_cast<float4*>(sn + 4 * x) =
        *reinterpret_cast<const float4*>(sines + ((x * items + j) << 2));
  }
  if (interleaved) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float* y = x < 4 ? a + 2 * x : b + 2 * (x - 4);
      const float p = y[0], q = y[1];
      y[0] = p * cs[x] - q * sn[x];
      y[1] = p * sn[x] + q * cs[x];
    }
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float p = a[x], q = b[x];
      a[x] = p * cs[x] - q * sn[x];
      b[x] = p * sn[x] + q * cs[x];
    }
  }
}

template <typename T>
struct Chunk8 {  // 8 elements of a row
  uint4 w[sizeof(T) / 2];
};

template <typename T>
SPEC_DEV void unpack_chunk(const Chunk8<T>& r, float* x) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.w[i].x);
      x[4 * i + 1] = __uint_as_float(r.w[i].y);
      x[4 * i + 2] = __uint_as_float(r.w[i].z);
      x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
  } else {
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(e[i]);
  }
}

template <typename T>
SPEC_DEV Chunk8<T> pack_chunk(const float* x) {
  Chunk8<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                          __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
  } else {
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = static_cast<T>(x[i]);
  }
  return r;
}
