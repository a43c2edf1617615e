// Pages, block tables and slots of a step, built on the GPU from lengths alone.
//
//  spec_extend_tables -- with have = ceil(ctx / P), want = ceil((ctx + add) / P),
//    need = want - have and upto = the inclusive running sum of need over the
//    sequences, sequence b is served iff its lengths are valid and (need = 0 or
//    upto[b] <= free pages); its j-th new page is entry count - 1 -
//    (upto[b] - need[b] + j) of the free list.  Token t of the packed rows
//    belongs to the b with cu[b] <= t < cu[b + 1], sits at position
//    ctx[b] + t - cu[b] and at slot page * P + position % P.
//  spec_release_pages -- the same running sum over the pages behind the kept
//    ones gives each sequence its place at the free list's end.
//
// What bounds them: latency.  A step moves a few KB to a few MB (12 bytes a
// token, 8 a page), so the cost is the chain lengths -> running sums -> free
// list -> store.  One launch each, no workspace and no grid-wide wait: every
// CTA forms the running sums of ALL sequences again in its shared memory (at
// most 8192 lengths, from L2) and then writes its share, so nothing passes
// between CTAs.  A token's page comes from the old table entry or straight from
// the free list, never from an entry that this launch writes.  The counts are
// read from one word and written to another for the same reason.
#include <algorithm>
#include <climits>
#include <initializer_list>

#include "serving.cuh"

namespace {

constexpr int kMostCtas = 304;      // two per SM
// up to here blocks of 128 threads, else of 256 (extend + release of 64 sequences 7.4
// against 8.5 us, of 1000 11.5 against 10.5)
constexpr int kFewSeqs = 256;
constexpr int kMaxSeqs = 8192;      // two running sums of 4 bytes: 64 KB of shared memory
constexpr int kTokensPerThread = 4;
constexpr int kWarpPages = 64;      // more pages than this: the whole CTA writes the row
constexpr int kPast = 4096;         // how far past a row's end its entries are counted

// Sums of lengths and pages stop at 2^31 - 1 (nothing past the capacities matters).
SPEC_DEV int sat_add(int a, int b) {
  return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)INT_MAX);
}

// Exclusive running sum over the block of one value >= 0 per thread; *total: the sum.
template <int kThreads>
SPEC_DEV int block_scan(int v, int* total) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int part[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = sat_add(x, y);
  }
  __syncthreads();  // `part` of an earlier call is read no more
  if (lane == 31) part[warp] = x;
  x = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) x = 0;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = sum;
    sum = sat_add(sum, part[w]);
  }
  *total = sum;
  return sat_add(before, x);
}

// dst[j] = f(src[step j]) for j < n, a lane's ids loaded eight at a time (the compiler
// cannot move a load over a store here: 30000 ids of one request took 80 us one by one).
template <typename F>
SPEC_DEV void copy_ids(const int32_t* src, int step, int32_t* dst, int n, int lane, int lanes,
                       F f) {
#pragma unroll 1
  for (int j0 = lane; j0 < n; j0 += 8 * lanes) {
    int id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) id[u] = j0 + u * lanes < n ? src[step * (j0 + u * lanes)] : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j0 + u * lanes < n) dst[j0 + u * lanes] = f(id[u]);
  }
}

SPEC_DEV int clamp_count(int c, int n) { return c < 0 ? 0 : c > n ? n : c; }

struct ExtendParams {
  const int32_t *ctx, *add, *free_list, *free_count;
  int32_t *table, *positions, *cu, *new_len, *free_left, *status;
  int64_t* slots;
  FastDiv P;
  int B, max_pages, num_pages, cap;
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const ExtendParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ int32_t sm[];
  int32_t* tok = sm;             // [B + 1] first row of each sequence (at most cap + 1)
  int32_t* pg = sm + p.B + 1;    // [B] pages of the step in front of it; < 0: refused (-1 - bit)
  chain_wait();
  const int count = clamp_count(*p.free_count, p.num_pages);

  // ---- running sums; a thread holds `per` consecutive sequences
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  const uint32_t row_max = (uint32_t)p.max_pages * p.P.d;  // tokens a table row can name
  int sum = 0, total;
  for (int b = b0; b < b1; ++b) sum = sat_add(sum, max(p.add[b], 0));
  int at = block_scan<kThreads>(sum, &total);
  int need_sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = p.ctx[b], a = p.add[b];
    tok[b] = min(at, p.cap + 1);
    if (blockIdx.x == 0) p.cu[b] = at;
    at = sat_add(at, max(a, 0));
    const bool bad = c < 0 || a < 0 || (uint32_t)c + (uint32_t)a > row_max || at > p.cap;
    const int need = bad ? 0 : p.P.ceil_quot(c + a) - p.P.ceil_quot(c);
    pg[b] = bad ? INT_MIN : need;
    need_sum = sat_add(need_sum, need);
  }
  if (threadIdx.x == 0) {
    tok[p.B] = min(total, p.cap + 1);
    if (blockIdx.x == 0) p.cu[p.B] = total;
  }
  int unused;
  int pages = block_scan<kThreads>(need_sum, &unused);
  int taken = 0;   // the largest running sum that fits: what the step takes
  for (int b = b0; b < b1; ++b) {
    const int need = pg[b];
    if (need == INT_MIN) {
      pg[b] = -1 - SPEC_SEQ_BAD_LEN;
      continue;
    }
    const int upto = sat_add(pages, need);
    const bool fits = need == 0 || upto <= count;
    if (fits && need) taken = upto;
    pg[b] = fits ? pages : -1 - SPEC_SEQ_NO_PAGES;
    pages = upto;
  }
  if (blockIdx.x == 0) {  // the served sequences that take pages come first
    __shared__ int most;
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    if (taken) atomicMax(&most, taken);
    __syncthreads();
    if (threadIdx.x == 0) *p.free_left = count - most;
  }
  __syncthreads();

  // ---- new pages into the table rows, lengths and statuses
  auto row = [&](int b, int have, int need, int lane, int lanes) {
    int32_t* t = p.table + (size_t)b * p.max_pages;
    bool bad = false;
    if (lane == 0 && have * p.P.d != p.ctx[b] && p.add[b] > 0) {  // the first token's old page
      const int id = t[have - 1];
      bad = id < 0 || id >= p.num_pages;
    }
    const int32_t* from = p.free_list + (count - 1 - pg[b]);
    copy_ids(from, -1, t + have, need, lane, lanes, [&](int id) {
      bad = bad || id < 0 || id >= p.num_pages;
      return id;
    });
    return bad;
  };
  auto finish = [&](int b, bool bad) {
    p.status[b] = bad ? SPEC_SEQ_BAD_PAGE : 0;
    p.new_len[b] = bad ? p.ctx[b] : p.ctx[b] + p.add[b];
  };
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.B; b += gridDim.x * kWarps) {
    if (pg[b] < 0) {
      if (lane == 0) {
        p.status[b] = -1 - pg[b];
        p.new_len[b] = p.ctx[b];
      }
      continue;
    }
    const int have = p.P.ceil_quot(p.ctx[b]), need = p.P.ceil_quot(p.ctx[b] + p.add[b]) - have;
    if (need > kWarpPages) continue;
    const bool bad = __any_sync(0xffffffffu, row(b, have, need, lane, 32));
    if (lane == 0) finish(b, bad);
  }
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (pg[b] < 0) continue;
    const int have = p.P.ceil_quot(p.ctx[b]), need = p.P.ceil_quot(p.ctx[b] + p.add[b]) - have;
    if (need <= kWarpPages) continue;
    const bool bad = __syncthreads_or(row(b, have, need, threadIdx.x, kThreads));
    if (threadIdx.x == 0) finish(b, bad);
  }

  // ---- slots and positions: consecutive rows per thread, one search each
  for (long long t0 = ((long long)blockIdx.x * kThreads + threadIdx.x) * kTokensPerThread;
       t0 < p.cap; t0 += (long long)gridDim.x * kThreads * kTokensPerThread) {
    int lo = 0, hi = p.B;  // the last b with tok[b] <= t0 (rows behind the last: B)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tok[mid] <= t0)
        lo = mid;
      else
        hi = mid - 1;
    }
    int b = lo;
#pragma unroll
    for (int u = 0; u < kTokensPerThread; ++u) {
      const int t = (int)t0 + u;
      if (t >= p.cap) break;
      while (b < p.B && tok[b + 1] <= t) ++b;
      int64_t slot = -1;
      int pos = -1;
      if (b < p.B && pg[b] >= 0) {
        const int c = p.ctx[b];
        pos = c + (t - tok[b]);
        const int idx = p.P.quot(pos), have = p.P.ceil_quot(c);
        const int id = idx < have ? p.table[(size_t)b * p.max_pages + idx]
                                  : p.free_list[count - 1 - (pg[b] + idx - have)];
        if (id >= 0 && id < p.num_pages)
          slot = (int64_t)id * p.P.d + (pos - idx * p.P.d);
        else
          pos = -1;
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
  }
}

struct ReleaseParams {
  const int32_t *table, *len, *keep, *free_count;
  int32_t *free_list, *free_total, *status;
  FastDiv P;
  int B, max_pages, num_pages;
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads) release_pages_kernel(const ReleaseParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ int32_t sm[];
  int32_t* at = sm;  // [B] place of the sequence's first page on the list; < 0: refused
  chain_wait();
  const int count = clamp_count(*p.free_count, p.num_pages);
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  int sum = 0, unused;
  for (int b = b0; b < b1; ++b) {
    const int n = p.len[b], k = p.keep[b], held = n < 0 ? 0 : p.P.ceil_quot(n);
    const bool bad = n < 0 || k < 0 || k > held || held > p.max_pages;
    at[b] = bad ? INT_MIN : held - k;
    if (!bad) sum = sat_add(sum, held - k);
  }
  int pages = sat_add(count, block_scan<kThreads>(sum, &unused));
  int end = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = at[b];
    if (n == INT_MIN) {
      at[b] = -1 - SPEC_SEQ_BAD_LEN;
      continue;
    }
    const int upto = sat_add(pages, n);
    const bool fits = n == 0 || upto <= p.num_pages;
    if (fits && n) end = upto;
    at[b] = fits ? pages : -1 - SPEC_SEQ_NO_PAGES;
    pages = upto;
  }
  if (blockIdx.x == 0) {
    __shared__ int most;
    if (threadIdx.x == 0) most = count;
    __syncthreads();
    if (end) atomicMax(&most, end);
    __syncthreads();
    if (threadIdx.x == 0) *p.free_total = most;
  }
  __syncthreads();

  auto row = [&](int b, int n, int lane, int lanes) {
    const int32_t* t = p.table + (size_t)b * p.max_pages + p.keep[b];
    bool bad = false;
    copy_ids(t, 1, p.free_list + at[b], n, lane, lanes, [&](int id) {
      const bool ok = id >= 0 && id < p.num_pages;
      bad = bad || !ok;
      return ok ? id : -1;
    });
    return bad;
  };
  auto pages_of = [&](int b) { return p.P.ceil_quot(p.len[b]) - p.keep[b]; };
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.B; b += gridDim.x * kWarps) {
    int st = 0;
    if (at[b] < 0) {
      st = -1 - at[b];
    } else {
      const int n = pages_of(b);
      if (n > kWarpPages) continue;
      if (__any_sync(0xffffffffu, row(b, n, lane, 32))) st = SPEC_SEQ_BAD_PAGE;
    }
    if (lane == 0 && p.status) p.status[b] = st;
  }
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (at[b] < 0) continue;
    const int n = pages_of(b);
    if (n <= kWarpPages) continue;
    const bool bad = __syncthreads_or(row(b, n, threadIdx.x, kThreads));
    if (threadIdx.x == 0 && p.status) p.status[b] = bad ? SPEC_SEQ_BAD_PAGE : 0;
  }
}

// CTAs of `threads`: a warp per sequence, four rows per thread, at most two per SM
int grid_for(int B, long long tokens, int threads) {
  const int warps = threads / 32;
  const long long a = (B + warps - 1) / warps;
  const long long t = (tokens + threads * kTokensPerThread - 1) / (threads * kTokensPerThread);
  const long long g = a > t ? a : t;
  return (int)(g < 1 ? 1 : g > kMostCtas ? kMostCtas : g);
}

}  // namespace

extern "C" spec_status spec_extend_tables(const int32_t* ctx_len, const int32_t* add_len, int B,
                                          int page_size, int32_t* block_table, int max_pages,
                                          const int32_t* free_list, int num_pages,
                                          const int32_t* free_count, int max_tokens,
                                          int64_t* slot_map, int32_t* positions, int32_t* cu_len,
                                          int32_t* new_len, int32_t* free_left,
                                          int32_t* status_per_seq, void* stream) {
  if (B < 0 || page_size < 1 || max_pages < 1 || num_pages < 1 || max_tokens < 0)
    return SPEC_EINVAL;
  if (!free_list || !free_count || !cu_len || !free_left) return SPEC_EINVAL;
  if (B && (!ctx_len || !add_len || !block_table || !new_len || !status_per_seq))
    return SPEC_EINVAL;
  if (max_tokens && (!slot_map || !positions)) return SPEC_EINVAL;
  if (B > kMaxSeqs || (long long)max_pages * page_size > INT_MAX || max_pages > INT_MAX - kPast ||
      max_tokens == INT_MAX || num_pages == INT_MAX)
    return SPEC_EUNSUPPORTED;
  const size_t seqs = (size_t)B * 4, rows = (size_t)max_tokens;
  if (share({{block_table, seqs * max_pages}, {slot_map, rows * 8}, {positions, rows * 4},
             {cu_len, seqs + 4}, {new_len, seqs}, {free_left, 4}, {status_per_seq, seqs}},
            {{ctx_len, seqs}, {add_len, seqs}, {free_list, (size_t)num_pages * 4}, {free_count, 4}}))
    return SPEC_EINVAL;
  const size_t smem = (2 * (size_t)B + 1) * sizeof(int32_t);
  if (B > kFewSeqs) {  // (the default limit counts the kernel's static shared memory too)
    static PerDeviceOnce<int> smem_once;  // once per device, at the largest size
    const spec_status ra = ensure_smem_limit(smem_once, (const void*)extend_tables_kernel<256>,
                                             (2 * kMaxSeqs + 1) * (int)sizeof(int32_t));
    if (ra != SPEC_OK) return ra;
  }
  const ExtendParams p{ctx_len, add_len,   free_list, free_count, block_table, positions, cu_len,
                       new_len, free_left, status_per_seq, slot_map, FastDiv(page_size), B,
                       max_pages, num_pages, max_tokens};
  const int threads = B <= kFewSeqs ? 128 : 256;
  return launch_chained(B <= kFewSeqs ? extend_tables_kernel<128> : extend_tables_kernel<256>,
                        grid_for(B, max_tokens, threads), threads, smem, (cudaStream_t)stream, p);
}

extern "C" spec_status spec_release_pages(const int32_t* block_table, int max_pages,
                                          const int32_t* len, const int32_t* keep_pages, int B,
                                          int page_size, int32_t* free_list, int num_pages,
                                          const int32_t* free_count, int32_t* free_total,
                                          int32_t* status_per_seq, void* stream) {
  if (B < 0 || page_size < 1 || max_pages < 1 || num_pages < 1) return SPEC_EINVAL;
  if (!free_list || !free_count || !free_total) return SPEC_EINVAL;
  if (B && (!block_table || !len || !keep_pages)) return SPEC_EINVAL;
  if (B > kMaxSeqs || (long long)max_pages * page_size > INT_MAX || max_pages > INT_MAX - kPast ||
      num_pages == INT_MAX)
    return SPEC_EUNSUPPORTED;
  const size_t seqs = (size_t)B * 4;
  if (share({{free_list, (size_t)num_pages * 4}, {free_total, 4}, {status_per_seq, seqs}},
            {{block_table, seqs * max_pages}, {len, seqs}, {keep_pages, seqs}, {free_count, 4}}))
    return SPEC_EINVAL;
  const ReleaseParams p{block_table, len, keep_pages, free_count, free_list, free_total,
                        status_per_seq, FastDiv(page_size), B, max_pages, num_pages};
  const int threads = B <= kFewSeqs ? 128 : 256;
  // a CTA per sequence where rows may be long (a finished request gives all its pages)
  return launch_chained(B <= kFewSeqs ? release_pages_kernel<128> : release_pages_kernel<256>,
                        max_pages > kWarpPages ? std::max(1, std::min(B, kMostCtas))
                                               : grid_for(B, 0, threads),
                        threads, (size_t)B * sizeof(int32_t), (cudaStream_t)stream, p);
}
