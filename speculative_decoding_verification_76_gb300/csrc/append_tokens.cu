// spec_append_tokens -- packed K/V rows stored at their slots of the paged
// cache, keys (and queries) rotated for their positions, 16-bit rows optionally
// quantised to e4m3.
//
// Mathematics: pair (x_i, x_{i + D/2}) at position t turns by the angle
// t * base^(-2i/D) ("Speculative Decoding" (atlas), "Chains, trees and
// visibility": positions, not storage order).  The angle is kept as a 64-bit
// fraction of a turn: F_i = round(base^(-2i/D) / 2 pi * 2^64), and t * F_i
// modulo 2^64 is the angle with the whole turns gone, as exact as the double
// that F_i comes from (t * 2^-55 turns), with two integer multiplies and no FP64,
// whose rate on this GPU is a small part of fp32's.  Sine and cosine are fp32 of
// that fraction; a row rotates in fp32 and is rounded once.
//
// What bounds it: each row is read once and written once, so HBM, and for a verify
// block (a few hundred rows) the launch.  One thread takes 8 + 8 elements of one head,
// i and i + D/2 on: two 16-byte loads, the rotation in registers, two stores;
// consecutive threads take consecutive 16 bytes, and a thread has three such items'
// loads in flight.  A token's D/2 sines and cosines serve all its heads from shared
// memory.  A CTA of 128 threads takes two tokens, or one where there are few.
// Measured (32 / 8 heads of 128, bf16 rows): 16384 tokens into an e4m3 cache 58 us =
// 6.3 TB/s, into a bf16 one 63 us = 6.4 TB/s (one token a CTA 63 and 65; one item in
// flight 69 and 71); 320 tokens 3.2 us (two tokens a CTA 4.0).
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "serving.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kFlight = 3;        // work items of a thread in flight
constexpr int kFewTokens = 1216;  // up to eight per SM: a CTA per token
constexpr int kMaxD = 256;

struct AppendParams {
  const char *k, *v, *q;
  char *q_out, *kc, *vc;
  const float *k_scale, *v_scale;
  const int64_t* slots;
  const int32_t* pos;
  long long k_stride, v_stride, q_stride, q_out_stride;          // elements
  long long page_stride, token_stride, head_stride, num_slots;   // elements, slots
  FastDiv P, per;  // page size; work items of a token
  int T, Hq, Hkv, rotate;
  uint64_t turn[kMaxD / 2];  // 2^64 x turns per position, of each pair
};

template <typename T>
struct Vec8 {  // 8 elements of a row
  uint4 w[sizeof(T) / 2];
};

template <typename T>
SPEC_DEV void unpack8(const Vec8<T>& r, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f[i];
  } else {
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(e[i]);
  }
}

SPEC_DEV uint16_t e4m3_pair(float lo, float hi) {  // nearest even, limited to +-448
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Quotients by an e4m3 head's scale s.  x times the rounded 1 / s would put a quotient that is a
// midpoint of the grid beside it (and on the wrong side, one time in two).  With the reciprocal
// as a sum of two, inv + lo = 1 / s up to 2^-45, fma(x, inv, x lo) is rounded once: it is the
// quotient where that is an fp32 number, as every midpoint is (a product with a known divisor's
// two-part reciprocal: Brisebarre, Muller and Raina, "Accelerating correctly rounded
// floating-point division when the divisor is known in advance", 2004).  inv lies below 1 / s,
// so lo > 0 and infinities keep their sign; `up` brings scales whose reciprocal or its second
// part is no normal number into range.  (One rounded reciprocal: 16384 tokens 58.3 us, D = 64
// 24.8; a division per element 60.5 and 29.1.)
struct Quotient {
  float inv, lo, up;
  SPEC_DEV explicit Quotient(float s) {
    up = s < 0x1p-100f ? 0x1p100f : s > 0x1p100f ? 0x1p-100f : 1.f;
    s *= up;
    inv = __uint_as_float(__float_as_uint(1.f / s) - 1u);
    lo = fmaf(-inv, s, 1.f) * inv;
  }
  SPEC_DEV float operator()(float x) const { return fmaf(x, inv, x * lo); }
};

// 8 values rounded to the cache type and stored at element address p
template <typename C>
SPEC_DEV void store8(char* p, float* x, const Quotient& by) {
  if constexpr (sizeof(C) == 1) {
    if (by.up != 1.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= by.up;
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)e4m3_pair(by(x[4 * i]), by(x[4 * i + 1])) |
             (uint32_t)e4m3_pair(by(x[4 * i + 2]), by(x[4 * i + 3])) << 16;
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else if constexpr (sizeof(C) == 2) {
    C e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = static_cast<C>(x[i]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// T: type of the rows; C: of the cache (__nv_fp8_e4m3 or T); TB tokens a CTA
template <typename T, typename C, int D, int TB>
__global__ void __launch_bounds__(kThreads) append_tokens_kernel(
    const __grid_constant__ AppendParams p) {
  constexpr int kHalf = D / 2, kChunks = kHalf / 8;
  __shared__ __align__(16) float cs[TB][kHalf], sn[TB][kHalf];
  __shared__ long long dst[TB];  // element offset of the token's cache row; < 0: skipped
  const int t0 = blockIdx.x * TB;
  chain_wait();
  if (threadIdx.x < TB) {
    const int t = t0 + threadIdx.x;
    long long off = -1;
    if (t < p.T) {
      const long long slot = p.slots[t];
      if (slot >= 0 && slot < p.num_slots && !(p.rotate && p.pos[t] < 0))
        off = p.num_slots <= 1u << 31 ? p.P.quot((int)slot) * p.page_stride +
                                            ((int)slot - p.P.quot((int)slot) * p.P.d) * p.token_stride
                                      : slot / p.P.d * p.page_stride + slot % p.P.d * p.token_stride;
    }
    dst[threadIdx.x] = off;
  }
  if (p.rotate)
    for (int i = threadIdx.x; i < TB * kHalf; i += kThreads) {
      const int u = i / kHalf, j = i % kHalf;
      const int t = min(t0 + u, p.T - 1);
      // the angle as a signed 32-bit fraction of a turn, in half turns
      const int32_t frac = (int32_t)(((uint64_t)(uint32_t)p.pos[t] * p.turn[j]) >> 32);
      float s, c;
      sincospif((float)frac * 0x1p-31f, &s, &c);
      cs[u][j] = c;
      sn[u][j] = s;
    }
  __syncthreads();

  // kFlight work items a thread at a time, their loads together (items behind the last
  // and of skipped tokens load what is there and store nothing)
  const int per = (p.Hq + 2 * p.Hkv) * kChunks, n = TB * per;  // work items of a token, of all
  for (int i0 = threadIdx.x; i0 < n; i0 += kFlight * kThreads) {
    Vec8<T> lo[kFlight], hi[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = min(i0 + f * kThreads, n - 1), u = p.per.quot(i), r = i - u * per;
      const int h = r / kChunks, e = r % kChunks * 8, t = min(t0 + u, p.T - 1);
      const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
      const char* src = is_q ? p.q : is_k ? p.k : p.v;
      const long long stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
      const int hh = is_q ? h : is_k ? h - p.Hq : h - p.Hq - p.Hkv;
      src += (t * stride + (hh * D + e)) * (long long)sizeof(T);
      lo[f] = *reinterpret_cast<const Vec8<T>*>(src);
      hi[f] = *reinterpret_cast<const Vec8<T>*>(src + kHalf * sizeof(T));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + f * kThreads;
      if (i >= n) break;
      const int u = p.per.quot(i), r = i - u * per, h = r / kChunks, e = r % kChunks * 8;
      if (dst[u] < 0) continue;
      const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
      float a[8], b[8];
      unpack8(lo[f], a);
      unpack8(hi[f], b);
      if (p.rotate && (is_q || is_k)) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float c = cs[u][e + x], s = sn[u][e + x], y = a[x];
          a[x] = y * c - b[x] * s;
          b[x] = y * s + b[x] * c;
        }
      }
      if (is_q) {
        char* o = p.q_out + ((t0 + u) * p.q_out_stride + (h * D + e)) * (long long)sizeof(T);
        store8<T>(o, a, Quotient(1.f));
        store8<T>(o + kHalf * sizeof(T), b, Quotient(1.f));
      } else {
        const int hh = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
        const float* sc = is_k ? p.k_scale : p.v_scale;
        const Quotient by(sizeof(C) == 1 && sc ? sc[hh] : 1.f);
        char* o = (is_k ? p.kc : p.vc) +
                  (dst[u] + hh * p.head_stride + e) * (long long)sizeof(C);
        store8<C>(o, a, by);
        store8<C>(o + kHalf * sizeof(C), b, by);
      }
    }
  }
}

template <typename T, typename C, int D>
spec_status launch(const AppendParams& p, cudaStream_t st) {
  return p.T <= kFewTokens
             ? launch_chained(append_tokens_kernel<T, C, D, 1>, p.T, kThreads, 0, st, p)
             : launch_chained(append_tokens_kernel<T, C, D, 2>, (p.T + 1) / 2, kThreads, 0, st, p);
}

template <typename T, typename C>
spec_status launch_d(const AppendParams& p, int D, cudaStream_t st) {
  return D == 64 ? launch<T, C, 64>(p, st)
                 : D == 128 ? launch<T, C, 128>(p, st) : launch<T, C, 256>(p, st);
}

}  // namespace

extern "C" spec_status spec_append_tokens(
    const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, const void* q,
    int64_t q_stride, void* q_out, int64_t q_out_stride, spec_dtype new_dtype, void* k_cache,
    void* v_cache, spec_dtype cache_dtype, const float* k_scale, const float* v_scale,
    int num_pages, int page_size, int64_t page_stride, int64_t token_stride, int64_t head_stride,
    const int64_t* slot_map, const int32_t* positions, int T, int Hq, int Hkv, int D,
    double rope_base, void* stream) {
  if (T < 0 || Hq < 0 || Hkv < 1 || num_pages < 1 || page_size < 1) return SPEC_EINVAL;
  if (Hq > 4096 || Hkv > 4096 || T == INT32_MAX) return SPEC_EUNSUPPORTED;
  if (new_dtype != SPEC_F32 && new_dtype != SPEC_BF16 && new_dtype != SPEC_F16) return SPEC_EINVAL;
  const bool e4m3 = cache_dtype == SPEC_E4M3;
  if (!e4m3 && cache_dtype != new_dtype) return SPEC_EINVAL;
  if (!e4m3 && (k_scale || v_scale)) return SPEC_EINVAL;
  if (!(rope_base == 0.0 || (rope_base > 1.0 && std::isfinite(rope_base)))) return SPEC_EINVAL;
  if ((q == nullptr) != (q_out == nullptr) || (q && Hq < 1)) return SPEC_EINVAL;
  if (e4m3 && new_dtype == SPEC_F32) return SPEC_EUNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return SPEC_EUNSUPPORTED;
  if (T == 0) return SPEC_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_map || (rope_base != 0.0 && !positions))
    return SPEC_EINVAL;
  const int es = new_dtype == SPEC_F32 ? 4 : 2, ec = e4m3 ? 1 : es;
  const uintptr_t ptrs = (uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)q | (uintptr_t)q_out |
                         (uintptr_t)k_cache | (uintptr_t)v_cache;
  if (ptrs & 15) return SPEC_EINVAL;
  if (k_stride < 0 || v_stride < 0 || q_stride < 0 || q_out_stride < 0 || page_stride < 0 ||
      token_stride < 0 || head_stride < 0)
    return SPEC_EINVAL;
  if (((k_stride | v_stride) * es | (q ? (q_stride | q_out_stride) * es : 0) |
       (page_stride | token_stride | head_stride) * ec) & 15)
    return SPEC_EINVAL;
  if (q == q_out && q && q_stride != q_out_stride) return SPEC_EINVAL;
  AppendParams p{};
  p.k = static_cast<const char*>(k_new);
  p.v = static_cast<const char*>(v_new);
  p.q = static_cast<const char*>(q);
  p.q_out = static_cast<char*>(q_out);
  p.kc = static_cast<char*>(k_cache);
  p.vc = static_cast<char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slots = slot_map;
  p.pos = positions;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.num_slots = (long long)num_pages * page_size;
  p.P = FastDiv(page_size);
  p.T = T;
  p.Hq = q ? Hq : 0;
  p.Hkv = Hkv;
  p.rotate = rope_base != 0.0;
  p.per = FastDiv((p.Hq + 2 * Hkv) * (D / 16));
  if (p.rotate) {
    // turns per position as a 64-bit fraction (1 / 2 pi of a turn at i = 0); the
    // last base's frequencies are kept per host thread: D / 2 powers cost more
    // host time than the launch
    struct Freq {
      double base = 0.0;
      int D = 0;
      uint64_t turn[kMaxD / 2];
    };
    static thread_local Freq f;
    if (f.base != rope_base || f.D != D) {
      for (int i = 0; i < D / 2; ++i)
        f.turn[i] = (uint64_t)std::llround(std::pow(rope_base, -2.0 * i / D) * 0x1p62 /
                                           6.283185307179586476925286766559) * 4;
      f.base = rope_base;
      f.D = D;
    }
    std::copy(f.turn, f.turn + D / 2, p.turn);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (new_dtype == SPEC_F32) return launch_d<float, float>(p, D, st);
  if (new_dtype == SPEC_BF16)
    return e4m3 ? launch_d<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                : launch_d<__nv_bfloat16, __nv_bfloat16>(p, D, st);
  return e4m3 ? launch_d<__half, __nv_fp8_e4m3>(p, D, st)
              : launch_d<__half, __half>(p, D, st);
}
