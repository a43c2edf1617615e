// spec_verify_attn_scaled -- attention of a verify block (or of single tokens) over an e4m3 cache
// with one scale for each block of tokens and KV head.
//
// Mathematics, for row i and the positions t it sees, with codes k_t, v_t and their blocks' scales
// a_t, c_t:
//   x_t = scale a_t (q . k_t),  out = sum_t e^(x_t - m) c_t v_t / l,  l = sum_t e^(x_t - m),
//   lse = m + ln l.
// This is the plain form of it: a warp per query row, a tile of 32 positions in shared memory for
// the rows of a CTA, running maximum and sum per row.
#include <cuda_fp16.h>

#include "scaled.cuh"

namespace {

constexpr int kRowsPerCta = 8;
constexpr int kTile = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const char *q, *k, *v;
  const float *ks, *vs;
  const int32_t *table, *ctx;
  const uint64_t* mask;
  char* out;
  float* lse;
  long long q_stride_b, q_stride_r, q_stride_h;            // elements
  long long page_stride, token_stride, head_stride;        // bytes
  FastDiv P, block;
  int B, R, Hq, Hkv, G, num_pages, max_pages, window, q_bf16;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(32 * kRowsPerCta) attn_scaled_kernel(
    const __grid_constant__ Params p) {
  constexpr int kPer = D / 32;
  extern __shared__ float dyn[];
  float(*kt)[D + 1] = reinterpret_cast<float(*)[D + 1]>(dyn);
  float(*vt)[D] = reinterpret_cast<float(*)[D]>(dyn + kTile * (D + 1));
  float(*qt)[D] = reinterpret_cast<float(*)[D]>(dyn + kTile * (2 * D + 1));
  __shared__ int here[kTile];
  chain_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, kvh = blockIdx.y, n = blockIdx.x * kRowsPerCta + warp;
  const bool row = n < p.R * p.G;
  const int i = row ? n / p.G : 0, h = kvh * p.G + (row ? n % p.G : 0);
  const int ctx = p.ctx[b];
  const uint64_t m64 = !row ? 0 : p.mask ? p.mask[(size_t)b * p.R + i]
                       : i >= 63 ? ~0ull : (2ull << i) - 1;
  const uint64_t mask = p.R < 64 ? m64 & ((1ull << p.R) - 1) : m64;
  const int from = p.window ? max(0, ctx + __popcll(mask) - p.window) : 0;
  const long long width = (long long)p.max_pages * p.P.d;
  const int end = ctx < 0 ? 0 : (int)min((long long)ctx + p.R, width);
  for (int d = lane; d < D; d += 32) {
    const long long at = b * p.q_stride_b + i * p.q_stride_r + h * p.q_stride_h + d;
    qt[warp][d] = !row ? 0.f : p.q_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q)[at])
                                        : __half2float(reinterpret_cast<const __half*>(p.q)[at]);
  }
  float m = -INFINITY, l = 0.f, o[kPer] = {};
  for (int t0 = p.window ? max(0, ctx - p.window) : 0; t0 < end; t0 += kTile) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * (D / 16); e += blockDim.x) {
      const int u = e / (D / 16), x = e % (D / 16), t = t0 + u;
      int page = -1;
      if (t < end) page = p.table[(size_t)b * p.max_pages + p.P.quot(t)];
      const bool ok = page >= 0 && page < p.num_pages;
      float kv[16] = {}, vv[16] = {};
      if (ok) {
        const int off = t - p.P.quot(t) * p.P.d;
        const long long at = page * p.page_stride + off * p.token_stride + kvh * p.head_stride + x * 16;
        const long long sc = ((long long)page * (p.P.d / p.block.d) + p.block.quot(off)) * p.Hkv + kvh;
        const uint4 kw = *reinterpret_cast<const uint4*>(p.k + at);
        const uint4 vw = *reinterpret_cast<const uint4*>(p.v + at);
        const uint32_t *k4 = reinterpret_cast<const uint32_t*>(&kw), *v4 = reinterpret_cast<const uint32_t*>(&vw);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          e4m3_values(k4[w], kv + 4 * w);
          e4m3_values(v4[w], vv + 4 * w);
        }
#pragma unroll
        for (int w = 0; w < 16; ++w) kv[w] *= p.ks[sc], vv[w] *= p.vs[sc];
      }
#pragma unroll
      for (int w = 0; w < 16; ++w) kt[u][x * 16 + w] = kv[w], vt[u][x * 16 + w] = vv[w];
      if (x == 0) here[u] = ok;
    }
    __syncthreads();
    const int t = t0 + lane, j = t - ctx;
    const bool seen = row && here[lane] && (j < 0 ? t >= from : j < p.R && (mask >> j & 1));
    float x = 0.f;
    for (int d = 0; d < D; ++d) x += qt[warp][d] * kt[lane][d];
    x = seen ? x * p.scale_log2 : -INFINITY;
    const uint32_t who = __ballot_sync(0xffffffffu, seen);
    if (!who) continue;
    const float now = fmaxf(m, warp_max(x));
    const float ref = now == -INFINITY ? 0.f : now, a = m == -INFINITY ? 0.f : exp2f(m - ref);
    const float e = seen ? exp2f(x - ref) : 0.f;
    l = l * a + warp_sum(e);
    m = now;
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] *= a;
    for (int u = 0; u < kTile; ++u) {
      const float w = __shfl_sync(0xffffffffu, e, u);
      if (who >> u & 1)
#pragma unroll
        for (int c = 0; c < kPer; ++c) o[c] += w * vt[u][c * 32 + lane];
    }
  }
  if (!row) return;
  const size_t at = ((size_t)b * p.R + i) * p.Hq + h;
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float y = l == 0.f ? 0.f : o[c] / l;
    if (p.q_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[at * D + c * 32 + lane] = __float2bfloat16(y);
    else reinterpret_cast<__half*>(p.out)[at * D + c * 32 + lane] = __float2half(y);
  }
  if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

extern "C" size_t spec_verify_attn_scaled_workspace_size(int B, int R, int Hq, int Hkv, int D) {
  if (B < 0 || R < 1 || R > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256))
    return 0;
  return sizeof(WsHeader);
}

extern "C" spec_status spec_verify_attn_scaled(
    const void* q, int64_t q_stride_b, int64_t q_stride_r, int64_t q_stride_h, spec_dtype q_dtype,
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    int num_pages, int page_size, int block, int64_t page_stride, int64_t token_stride,
    int64_t head_stride, const int32_t* block_table, int max_pages, const int32_t* ctx_len,
    const uint64_t* anc_mask, int B, int R, int Hq, int Hkv, int D, int window, float scale,
    void* workspace, size_t workspace_bytes, void* out, float* lse_out, void* stream) {
  if (B < 0 || R < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_pages < 1 || page_size < 1 ||
      max_pages < 1 || block < 1 || page_size % block || window < 0)
    return SPEC_EINVAL;
  if (q_dtype == SPEC_F32) return SPEC_EUNSUPPORTED;
  if (q_dtype != SPEC_BF16 && q_dtype != SPEC_F16) return SPEC_EINVAL;
  if ((D != 64 && D != 128 && D != 256) || R > 64 || block > kMaxBlock) return SPEC_EUNSUPPORTED;
  if (window && window < R) return SPEC_EUNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !ctx_len || !workspace ||
      !out)
    return SPEC_EINVAL;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15)
    return SPEC_EINVAL;
  if ((uintptr_t)workspace & 255) return SPEC_EINVAL;
  if (q_stride_b < 0 || q_stride_r < 0 || q_stride_h < 0 || page_stride < 0 || token_stride < 0 ||
      head_stride < 0)
    return SPEC_EINVAL;
  if ((((q_stride_b | q_stride_r | q_stride_h) * 2) & 15) ||
      ((page_stride | token_stride | head_stride) & 15))
    return SPEC_EINVAL;
  if ((long long)max_pages * page_size > INT32_MAX - 512 || B > 65535 || Hkv > 65535)
    return SPEC_EUNSUPPORTED;
  if (workspace_bytes < spec_verify_attn_scaled_workspace_size(B, R, Hq, Hkv, D)) return SPEC_EINVAL;
  Params p{};
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k_cache);
  p.v = static_cast<const char*>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  p.table = block_table;
  p.ctx = ctx_len;
  p.mask = anc_mask;
  p.out = static_cast<char*>(out);
  p.lse = lse_out;
  p.q_stride_b = q_stride_b;
  p.q_stride_r = q_stride_r;
  p.q_stride_h = q_stride_h;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.P = FastDiv(page_size);
  p.block = FastDiv(block);
  p.B = B;
  p.R = R;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.window = window;
  p.q_bf16 = q_dtype == SPEC_BF16;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
  const dim3 grid((R * p.G + kRowsPerCta - 1) / kRowsPerCta, Hkv, B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto kernel = D == 64 ? attn_scaled_kernel<64> : D == 128 ? attn_scaled_kernel<128> : attn_scaled_kernel<256>;
  const int smem = (kTile * (2 * D + 1) + kRowsPerCta * D) * 4;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SPEC_ECUDA;
  kernel<<<grid, 32 * kRowsPerCta, smem, st>>>(p);
  return launch_status();
}
