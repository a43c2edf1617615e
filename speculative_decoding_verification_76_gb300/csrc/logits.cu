// spec_logits_process -- the target logits as served: penalties over each row's own prefix,
// biases and grammar masks, every request with its own settings, in one pass.
//
// Mathematics, in fp32 and in this order: l -> l / r or l r for ids of the prompt or text
// (repetition), l - f n - p for ids that stand n > 0 times in the text (frequency, presence),
// l + bias, -inf where the mask's bit is clear ("Speculative Decoding" (atlas), "Greedy, sampling
// and the real sampler": p must include the transforms actually served).  A row's text is the
// history behind the prompt and the block tokens in front of the row.
//
// What bounds it: the logits are read once and written once, so HBM (what a mask forbids in groups of
// eight is not read), and the counting in front of it where histories are long.
//
// Design: a CTA takes a slice of the vocabulary for some rows of one sequence.  It counts the
// history's ids of its slice in shared memory (integer atomics: the order does not matter), sums
// the biases there (ids are dealt to threads, each adds its own in the list's order) and lists what
// either touches; the first rows' logits and the lists' first ids are on their way meanwhile.  Rows are
// written as they come, eight ids a thread and store, with -inf where the mask forbids; behind them the
// touched ids, a thread each, are computed and written over it.  (Touched ids looked for within the
// stores: most warps met some, twice the instructions.)
//
// Measured: 64 sequences of 5 rows, fp32, 152064 ids, histories of 4099, a mask on a quarter 85.5 us, 4.6 TB/s
// (the copy alone 58.5, penalties 14 us more, biases 6, masks 6; simplest form 113, touched ids behind each
// row's stores 99, two rows in flight 89); one sequence of 8 rows, bf16, 128256 ids 5.7 us (19.4 before its
// rows were dealt out).  Copying first in every other wave of CTAs, so that not all count at once: 100 us.
#include <algorithm>

#include <cuda_fp16.h>

#include "serving.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kPrompt = 0x80000000u;   // of a count: the id stands in the prompt
constexpr uint32_t kBlock = 0x40000000u;    // a block token
constexpr int kRows = 2;                    // rows of a CTA in flight
constexpr int kFlight = 2;                  // units (of eight ids) of a thread
constexpr int kMostSlice = 8 * kFlight * kThreads;
constexpr int kHalo = 8;                    // ids in front of a slice that a row's first unit may hold

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
struct alignas(8 * sizeof(T)) Unit {  // eight logits, as they come
  T x[8];
};

template <typename T>
SPEC_DEV void load_unit(const T* src, Unit<T>& u) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
  if constexpr (sizeof(T) == 4)
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  else
    *reinterpret_cast<uint4*>(w) = __ldcs(reinterpret_cast<const uint4*>(src));
}

SPEC_DEV void store_unit(float* out, const float* y) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(y[0]),
               "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
               : "memory");
}

// Bits at .. at + 7 (at > -8; bits in front of the first and behind byte `last`: 0).
SPEC_DEV uint32_t eight_bits(const uint8_t* w, int at, int last) {
  const int i = at >> 3, sh = at & 7;
  uint32_t v = at >= 0 ? w[i] : 0u;
  if (sh && i < last) v |= (uint32_t)w[i + 1] << 8;
  return v >> sh & 255u;
}

__host__ __device__ constexpr int touched_words(int slice) {  // whole 16 bytes
  return ((slice + kHalo + 31) / 32 + 3) / 4 * 4;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ __align__(16) uint32_t sm[];
  const int S = p.slice + kHalo;
  uint32_t* touched = sm;                                   // a bit for each id: in the list
  uint32_t* count = touched + touched_words(p.slice);       // S, if counts
  float* add = reinterpret_cast<float*>(count + (p.counts ? S : 0));  // S, if biases
  uint16_t* list = reinterpret_cast<uint16_t*>(add + (p.biases ? S : 0));  // S
  __shared__ uint64_t anc[64];
  __shared__ int32_t tok[64], list_id[kThreads];
  __shared__ float list_x[kThreads];
  __shared__ int warp_n[kWarps], listed;
  const int b = blockIdx.y, first = blockIdx.x * p.slice;
  const int base = first - kHalo;                            // id of the first counter
  const int r0 = blockIdx.z * p.rows, r1 = min(r0 + p.rows, p.R);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool any = p.counts || p.biases;
  if (any) {
    const int n = (int)(reinterpret_cast<uint32_t*>(list) - sm);
    for (int i = threadIdx.x; i < n / 4; i += kThreads)
      reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) listed = 0;
  }
  chain_wait();

  // ---- a row, eight ids of it at a time: a unit is one aligned store of 32 bytes, so the CTA's units
  // start at ids first - off, first + 8 - off, ...
  struct Row {
    const T* src;
    float* out;
    const uint32_t* mask;
    int off;
  };
  auto row_of = [&](int r) {
    const long long at = (long long)b * p.R + r;
    Row row{reinterpret_cast<const T*>(p.logits) + at * p.stride, p.out + at * p.V, nullptr, 0};
    if (p.mask) {
      const long long m = p.mask_row ? p.mask_row[at] : at;
      if (m >= 0 && m < p.n_masks) row.mask = p.mask + m * p.words;
    }
    row.off = (int)(((uintptr_t)row.out >> 2) & 7);
    return row;
  };
  Unit<T> g[kRows][kFlight];
  uint32_t ok[kRows][kFlight];  // ids that may be drawn
  auto unit_id = [&](const Row& row, int f) {
    return first + 8 * (int)(threadIdx.x + f * kThreads) - row.off;
  };
  auto there = [&](int f, int id) {  // (id: the unit's first)
    return 8 * (threadIdx.x + f * kThreads) < p.slice && id < p.V;
  };
  auto load = [&](int r) {  // rows r .. r + kRows - 1
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      if (r + x >= r1) break;
      const Row row = row_of(r + x);
      const bool aligned = (((uintptr_t)row.src - row.off * sizeof(T)) & (8 * sizeof(T) - 1)) == 0;
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int id = unit_id(row, f);
        uint32_t m = 255u;
        if (row.mask && there(f, id))
          m = eight_bits(reinterpret_cast<const uint8_t*>(row.mask), id, 4 * p.words - 1);
        ok[x][f] = m;
        if (!m || p.in_place || !there(f, id)) continue;
        if (aligned && id >= 0 && id + 8 <= p.V) {
          load_unit(row.src + id, g[x][f]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((unsigned)(id + i) < (unsigned)p.V) g[x][f].x[i] = row.src[id + i];
        }
      }
    }
  };
  // ---- on their way while the ids are counted: the first rows; and the first ids of all lists
  load(r0);
  constexpr int kAtOnce = 8;
  const int32_t* const history = p.history + (size_t)b * p.H;
  int32_t past[kAtOnce], bias_id = -1, token = -1;
  float bias = 0.f;
  auto load_past = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x)
      past[x] = i0 + x * kThreads < p.H ? history[i0 + x * kThreads] : -1;
  };
  auto load_bias = [&](int i) {
    bias_id = i < p.n_bias ? p.bias_ids[(size_t)b * p.n_bias + i] : -1;
    bias = i < p.n_bias ? p.bias[(size_t)b * p.n_bias + i] : 0.f;
  };
  if (p.counts) {
    load_past(threadIdx.x);
    if (p.tokens && threadIdx.x > 0 && threadIdx.x < p.R)
      token = p.tokens[p.parent ? (size_t)b * p.R + threadIdx.x : (size_t)b * (p.R - 1) + threadIdx.x - 1];
  }
  if (p.biases) load_bias(threadIdx.x);

  auto mark = [&](int i) {
    const uint32_t bit = 1u << (i & 31);
    if (!(atomicOr(touched + (i >> 5), bit) & bit)) list[atomicAdd(&listed, 1)] = (uint16_t)i;
  };
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (any) __syncthreads();
  if (p.counts) {
    rep = p.repetition ? p.repetition[b] : 1.f;
    freq = p.frequency ? p.frequency[b] : 0.f;
    pres = p.presence ? p.presence[b] : 0.f;
    const int prompt = p.prompt_len ? p.prompt_len[b] : 0;
    auto index = [&](int32_t id) {  // of an id's counter, ~0 if there is none
      const uint32_t i = (uint32_t)id - (uint32_t)base;
      return i < (uint32_t)S && (uint32_t)id < (uint32_t)p.V ? i : ~0u;
    };
    for (int i0 = threadIdx.x; i0 < p.H; i0 += kAtOnce * kThreads) {
      if (i0 != threadIdx.x) load_past(i0);
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const uint32_t i = index(past[x]);
        if (i == ~0u) continue;
        if (i0 + x * kThreads < prompt) atomicOr(count + i, kPrompt);
        else atomicAdd(count + i, 1u);
        mark(i);
      }
    }
    // the block's tokens and each row's ancestors
    if (threadIdx.x < p.R) {
      const int i = threadIdx.x;
      const int t = (int)index(token);
      tok[i] = t;
      if (t >= 0) {
        atomicOr(count + t, kBlock);
        mark(t);
      }
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
  }
  if (p.biases) {
    for (int i0 = 0; i0 < p.n_bias; i0 += kThreads) {
      if (i0 > 0) load_bias(i0 + threadIdx.x);
      const bool in = (uint32_t)bias_id - (uint32_t)base < (uint32_t)S && (uint32_t)bias_id < (uint32_t)p.V;
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
        list_id[at] = bias_id - base;
        list_x[at] = bias;
      }
      __syncthreads();
      for (int e = 0; e < n; ++e)
        if ((list_id[e] & (kThreads - 1)) == (int)threadIdx.x) {
          add[list_id[e]] += list_x[e];
          mark(list_id[e]);
        }
    }
  }

  for (int r = r0; r < r1; r += kRows) {
    if (r > r0) load(r);
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      if (r + x >= r1) break;
      const long long at = (long long)b * p.R + r + x;
      float* out = p.out + at * p.V;
      const int off = (int)(((uintptr_t)out >> 2) & 7);
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int id = first + 8 * (int)(threadIdx.x + f * kThreads) - off;
        if (!there(f, id)) continue;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = !p.in_place && (ok[x][f] >> i & 1) ? to_float(g[x][f].x[i]) : -INFINITY;
        uint32_t put = 255u;
        if (id < 0) put = 255u << -id & 255u;
        if (id + 8 > p.V) put &= (1u << (p.V - id)) - 1;
        if (p.in_place) put &= ~ok[x][f];
        if (put == 255u) {
          store_unit(out + id, y);
        } else if (put) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (put >> i & 1) out[id + i] = y[i];
        }
      }
    }
  }
  if (!any) return;

  // ---- what the counts and biases touch, behind the stores of the other threads
  __syncthreads();
  const int n_listed = listed, n = n_listed * (r1 - r0);
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int u = j / n_listed, i = list[j - u * n_listed], id = base + i;
    const Row row = row_of(r0 + u);
    if ((unsigned)(id - first + row.off) >= (unsigned)p.slice) continue;  // (a neighbour's, in this row)
    if (row.mask && !(row.mask[id >> 5] >> (id & 31) & 1)) continue;
    float x = p.in_place ? row.out[id] : to_float(row.src[id]);
    if (p.counts) {
      const uint32_t c = count[i];
      uint64_t before = c & kBlock ? anc[r0 + u] : 0;  // rows of the block in front of this one
      int n = c & (kBlock - 1);
      for (; before; before &= before - 1) n += tok[__ffsll((long long)before) - 1] == i;
      if ((n > 0 || (c & kPrompt)) && p.repetition) x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      if (n > 0) {
        if (p.frequency) x = __fsub_rn(x, __fmul_rn(freq, (float)n));
        if (p.presence) x = __fsub_rn(x, pres);
      }
    }
    if (p.biases) x += add[i];
    row.out[id] = x;
  }
}

size_t smem_bytes(const LogitsParams& p) {
  if (!p.counts && !p.biases) return 0;
  const size_t S = p.slice + kHalo;
  return (touched_words(p.slice) + (p.counts ? S : 0) + (p.biases ? S : 0)) * 4 + S * 2;
}

template <typename T>
spec_status launch(const LogitsParams& p, cudaStream_t st) {
  const size_t smem = smem_bytes(p);
  static PerDeviceOnce<int> once;
  LogitsParams most = p;
  most.slice = kMostSlice;
  most.counts = most.biases = 1;
  const spec_status rc =
      ensure_smem_limit(once, (const void*)logits_kernel<T>, (int)smem_bytes(most));
  if (rc != SPEC_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.V + 7 + p.slice - 1) / p.slice, p.B, p.row_groups);
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
  if (V > INT32_MAX - 4 * kMostSlice || H >= (int)kBlock || n_bias > INT32_MAX - 4096 || B > 65535)
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
  // A CTA per sequence and slice walks all rows where that fills the GPU; else the rows are dealt out
  // too, and where even that leaves SMs idle the slices are shorter.
  const int sms = sm_count();
  p.slice = kMostSlice;
  while (p.slice > 1024 && (long long)B * R * ((V + p.slice - 1) / p.slice) < sms) p.slice /= 2;
  const long long ctas = (long long)B * ((V + p.slice - 1) / p.slice);
  p.rows = std::max<int>(1, (int)std::min<long long>(R, R * ctas / (2 * sms)));
  p.row_groups = (R + p.rows - 1) / p.rows;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPEC_F32) return launch<float>(p, st);
  if (dtype == SPEC_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}
