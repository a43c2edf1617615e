// spec_logits_process -- the target logits as served: penalties over each row's own prefix,
// biases and grammar masks, every request with its own settings, in one pass.
//
// Mathematics, in fp32 and in this order: l -> l / r or l r for ids of the prompt or text
// (repetition), l - f n - p for ids that stand n > 0 times in the text (frequency, presence),
// l + bias, -inf where the mask's bit is clear ("Speculative Decoding" (atlas), "Greedy, sampling
// and the real sampler": p must include the transforms actually served).  A row's text is the
// history behind the prompt and the block tokens in front of the row.
//
// What bounds it: the logits are read once and written once, so HBM; what a mask forbids in
// groups of four is not read.
//
// Design: a CTA takes a slice of the vocabulary for some rows of one sequence.  It counts the
// history's ids of its slice in shared memory (integer atomics: the order does not matter), sums
// the biases there (ids are dealt to threads, each adds its own in the list's order), marks what
// either touches in a bitmap, and walks its rows: a thread takes four ids that are one 16-byte
// store, and looks at counts and biases only where the bitmap has a bit.  From row to row only the
// block tokens that differ are counted up or down.
#include <cuda_fp16.h>

#include "serving.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFlight = 4;                  // groups of four ids of a thread in flight
constexpr uint32_t kPrompt = 0x80000000u;   // of a count: the id stands in the prompt
constexpr int kHalo = 32;                   // ids behind a slice that its last group may touch

struct LogitsParams {
  const char* logits;
  float* out;
  const int32_t *history, *prompt_len, *tokens, *parent;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  const int32_t* mask_row;
  long long stride;  // elements
  int B, R, V, H, n_bias, n_masks, words, slice, rows, row_groups, counts, biases, in_place;
};

SPEC_DEV float to_float(float x) { return x; }
SPEC_DEV float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV float to_float(__half x) { return __half2float(x); }

template <typename T>
struct alignas(4 * sizeof(T)) Group {  // four logits, as they come
  T x[4];
};

// Four logits from src on: all of them in one load where the row has them and they are aligned, else
// those of `want`.
template <typename T>
SPEC_DEV void load_group(const T* src, uint32_t want, bool all, Group<T>& g) {
  if (all && ((uintptr_t)src & (4 * sizeof(T) - 1)) == 0) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(&g) = __ldcs(reinterpret_cast<const float4*>(src));
    else
      *reinterpret_cast<uint2*>(&g) = __ldcs(reinterpret_cast<const uint2*>(src));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (want >> i & 1) g.x[i] = src[i];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ __align__(16) uint32_t sm[];
  const int S = p.slice + kHalo;
  uint32_t* touched = sm;                                   // S / 32 + 1 words
  uint32_t* count = touched + (S / 32 + 1 + 3) / 4 * 4;      // S, if counts
  float* add = reinterpret_cast<float*>(count + (p.counts ? S : 0));  // S, if biases
  __shared__ uint64_t anc[64], here_s;
  __shared__ int32_t tok[64], list_id[kThreads];
  __shared__ float list_x[kThreads];
  __shared__ int warp_n[kWarps];
  const int b = blockIdx.y, base = blockIdx.x * p.slice;
  const int r0 = blockIdx.z * p.rows, r1 = min(r0 + p.rows, p.R);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int top = min(p.V - base, S);                        // ids of this CTA
  const bool any = p.counts || p.biases;
  if (any) {
    const int n = (int)((p.biases ? add + S : reinterpret_cast<float*>(count) + S) -
                        reinterpret_cast<float*>(sm));
    for (int i = threadIdx.x; i < n; i += kThreads) sm[i] = 0u;
  }
  chain_wait();
  __syncthreads();
  auto mark = [&](int i) { atomicOr(touched + (i >> 5), 1u << (i & 31)); };
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (p.counts) {
    rep = p.repetition ? p.repetition[b] : 1.f;
    freq = p.frequency ? p.frequency[b] : 0.f;
    pres = p.presence ? p.presence[b] : 0.f;
    const int prompt = p.prompt_len ? p.prompt_len[b] : 0;
    const int32_t* h = p.history + (size_t)b * p.H;
    for (int i = threadIdx.x; i < p.H; i += kThreads) {
      const uint32_t id = (uint32_t)h[i] - (uint32_t)base;
      if (id < (uint32_t)top) {
        if (i < prompt) atomicOr(count + id, kPrompt);
        else atomicAdd(count + id, 1u);
        mark(id);
      }
    }
    // the block's tokens and each row's ancestors
    if (threadIdx.x < p.R) {
      const int i = threadIdx.x;
      int t = -1;
      if (p.tokens && i > 0)
        t = p.parent ? p.tokens[(size_t)b * p.R + i] : p.tokens[(size_t)b * (p.R - 1) + i - 1];
      tok[i] = t;
      uint64_t m = 0;
      if (p.parent) {
        int v = i;
        while (v > 0) {
          m |= 1ull << v;
          const int u = p.parent[(size_t)b * p.R + v];
          v = u < v ? u : 0;
        }
      } else {
        m = (i >= 63 ? ~0ull : (2ull << i) - 1) & ~1ull;
      }
      anc[i] = m;
    }
    __syncthreads();
    if (warp == 0) {  // which of them are ids of this slice
      auto inside = [&](int i) {
        return i < p.R && tok[i] >= 0 && (uint32_t)tok[i] - (uint32_t)base < (uint32_t)top;
      };
      const uint32_t lo = __ballot_sync(0xffffffffu, inside(lane));
      const uint32_t hi = __ballot_sync(0xffffffffu, inside(lane + 32));
      if (lane == 0) here_s = (uint64_t)hi << 32 | lo;
    }
  }
  if (p.biases) {
    const int32_t* ids = p.bias_ids + (size_t)b * p.n_bias;
    const float* xs = p.bias + (size_t)b * p.n_bias;
    for (int i0 = 0; i0 < p.n_bias; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      const uint32_t id = i < p.n_bias ? (uint32_t)ids[i] - (uint32_t)base : ~0u;
      const bool in = id < (uint32_t)top;
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      if (lane == 0) warp_n[warp] = __popc(who);
      __syncthreads();
      int at = __popc(who & ((1u << lane) - 1)), n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += warp_n[w];
        n += warp_n[w];
      }
      if (in) {
        list_id[at] = (int)id;
        list_x[at] = xs[i];
      }
      __syncthreads();
      for (int e = 0; e < n; ++e)
        if ((list_id[e] & (kThreads - 1)) == (int)threadIdx.x) {
          add[list_id[e]] += list_x[e];
          mark(list_id[e]);
        }
    }
  }
  __syncthreads();

  uint64_t counted = 0;  // block tokens that the counts hold
  const uint64_t here = p.counts ? here_s : 0;
  for (int r = r0; r < r1; ++r) {
    const uint64_t want = p.counts ? anc[r] & here : 0, change = want ^ counted;
    if (change) {
      __syncthreads();
      if (threadIdx.x < 64 && change >> threadIdx.x & 1) {
        const int id = tok[threadIdx.x] - base;
        atomicAdd(count + id, want >> threadIdx.x & 1 ? 1u : ~0u);
        mark(id);
      }
      counted = want;
      __syncthreads();
    }
    const long long row = (long long)b * p.R + r;
    float* out = p.out + row * p.V;
    const T* src = reinterpret_cast<const T*>(p.logits) + row * p.stride;
    const uint32_t* mask = nullptr;
    if (p.mask) {
      const long long m = p.mask_row ? p.mask_row[row] : row;
      if (m >= 0 && m < p.n_masks) mask = p.mask + m * p.words;
    }
    if (p.in_place && !any && !mask) continue;
    // groups of four ids start where the store is aligned: at -off, 4 - off, ...
    const int off = (int)(((uintptr_t)out >> 2) & 3);
    const int k0 = base == 0 ? 0 : (base + off + 3) >> 2;
    const int end = min(base + p.slice, p.V);                 // groups that start in front of it
    const int k1 = (end + off + 3) >> 2;
    for (int k = k0 + threadIdx.x; k < k1; k += kThreads * kFlight) {
      Group<T> g[kFlight];
      uint32_t live[kFlight], hit[kFlight], ok[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int kk = k + f * kThreads, id = 4 * kk - off;
        live[f] = hit[f] = ok[f] = 0;
        if (kk >= k1) continue;
        live[f] = 15u;
        if (id < 0) live[f] = 15u << -id & 15u;
        if (id + 4 > p.V) live[f] &= (1u << (p.V - id)) - 1;
        auto bits = [&](const uint32_t* w, int at, int last) {  // four, from bit at on
          const int i = at < 0 ? 0 : at;
          uint32_t v = w[i >> 5] >> (i & 31);
          if ((i & 31) > 28 && (i >> 5) < last) v |= w[(i >> 5) + 1] << (32 - (i & 31));
          return at < 0 ? v << -at : v;
        };
        ok[f] = mask ? bits(mask, id, p.words - 1) & live[f] : live[f];
        if (any) hit[f] = bits(touched, id - base, S / 32) & ok[f];
        const uint32_t need = p.in_place ? hit[f] : ok[f];
        if (need) load_group(src + id, need, live[f] == 15u, g[f]);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (!live[f]) continue;
        const int id = 4 * (k + f * kThreads) - off;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = ok[f] >> i & 1 ? to_float(g[f].x[i]) : -INFINITY;
        if (hit[f]) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (hit[f] >> i & 1) {
              const int e = id + i - base;
              if (p.counts) {
                const uint32_t c = count[e], n = c & ~kPrompt;
                if (c && p.repetition) y[i] = y[i] > 0.f ? __fdiv_rn(y[i], rep) : y[i] * rep;
                if (n) {
                  if (p.frequency) y[i] = __fsub_rn(y[i], __fmul_rn(freq, (float)n));
                  if (p.presence) y[i] = __fsub_rn(y[i], pres);
                }
              }
              if (p.biases) y[i] += add[e];
            }
        }
        const uint32_t put = p.in_place ? hit[f] | (live[f] & ~ok[f]) : live[f];
        if (put == 15u)
          __stcs(reinterpret_cast<float4*>(out + id), make_float4(y[0], y[1], y[2], y[3]));
        else
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (put >> i & 1) out[id + i] = y[i];
      }
    }
  }
}

size_t smem_bytes(const LogitsParams& p) {
  const size_t S = p.slice + kHalo;
  return ((S / 32 + 1 + 3) / 4 * 4 + (p.counts ? S : 0) + (p.biases ? S : 0)) * 4;
}

template <typename T>
spec_status launch(const LogitsParams& p, cudaStream_t st) {
  const size_t smem = smem_bytes(p);
  static PerDeviceOnce<int> once;
  LogitsParams most = p;
  most.slice = 8192;
  most.counts = most.biases = 1;
  const spec_status rc =
      ensure_smem_limit(once, (const void*)logits_kernel<T>, (int)smem_bytes(most));
  if (rc != SPEC_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.V + p.slice - 1) / p.slice, p.B, p.row_groups);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, logits_kernel<T>, p) != cudaSuccess) return SPEC_ECUDA;
  return launch_status();
}

}  // namespace

extern "C" spec_status spec_logits_process(
    const void* logits, int64_t logits_stride, spec_dtype dtype, float* out, int B, int R, int V,
    const int32_t* history, int H, const int32_t* prompt_len, const int32_t* block_tokens,
    const int32_t* parent, const float* repetition, const float* frequency, const float* presence,
    const int32_t* bias_ids, const float* bias, int n_bias, const int32_t* mask, int n_masks,
    const int32_t* mask_row, void* stream) {
  if (B < 0 || R < 1 || R > 64 || V < 1 || H < 0 || n_bias < 0 || n_masks < 0) return SPEC_EINVAL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_EINVAL;
  if (V > INT32_MAX - 4096 || H > INT32_MAX - 4096 || n_bias > INT32_MAX - 4096 || B > 65535)
    return SPEC_EUNSUPPORTED;
  if ((H > 0 && !history) || (parent && !block_tokens) || (n_bias > 0 && (!bias_ids || !bias)) ||
      (n_masks > 0 && !mask))
    return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  if (!logits || !out || logits_stride < V) return SPEC_EINVAL;
  const bool in_place = logits == out;
  if (in_place && (dtype != SPEC_F32 || logits_stride != V)) return SPEC_EINVAL;
  if (((uintptr_t)logits & (dtype == SPEC_F32 ? 3 : 1)) || ((uintptr_t)out & 3)) return SPEC_EINVAL;
  LogitsParams p{};
  p.logits = static_cast<const char*>(logits);
  p.out = out;
  p.history = history;
  p.prompt_len = prompt_len;
  p.tokens = block_tokens;
  p.parent = parent;
  p.repetition = repetition;
  p.frequency = frequency;
  p.presence = presence;
  p.bias_ids = bias_ids;
  p.bias = bias;
  p.mask = reinterpret_cast<const uint32_t*>(n_masks > 0 ? mask : nullptr);
  p.mask_row = mask_row;
  p.stride = logits_stride;
  p.B = B;
  p.R = R;
  p.V = V;
  p.H = H;
  p.n_bias = n_bias;
  p.n_masks = n_masks;
  p.words = (V + 31) / 32;
  p.counts = (repetition || frequency || presence) && (H > 0 || block_tokens);
  p.biases = n_bias > 0;
  p.in_place = in_place;
  p.slice = 4096;
  p.rows = R;
  p.row_groups = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPEC_F32) return launch<float>(p, st);
  if (dtype == SPEC_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}
