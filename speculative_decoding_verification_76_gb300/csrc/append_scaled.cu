// spec_append_scaled, spec_read_scaled, spec_commit_scaled -- an e4m3 cache whose scales, one for
// each block of tokens and KV head, come from what is stored.
//
// Mathematics: a block needs the smallest power of two s with max |x| <= 448 s over the rows
// that a call stores to it; x is stored as x / s rounded to the nearest e4m3 number.  A block
// whose first token is stored begins anew; one that is only added to keeps the larger scale, and
// its other codes c become c s_old / s (scaled.cuh has why powers of two).  Keys turn for their
// positions first (rope.cuh).
//
// What bounds it: the rows are read once and the codes written once, so HBM, and for a verify
// block (a few hundred rows) a chain of round trips: slots, rows and scale, store.
//
// Design: the rows of a block stand next to each other in the call, so a block's rows are a run of
// at most `block` rows, and the run's first row tells who handles it.  A CTA takes the runs that
// begin among its W rows, of the keys or of the values; other CTAs turn the queries.  As many warps as hold a
// run of one head (16 rows of 128 each) take it, whole and read once -- maximum over the run's rows by
// shuffles and shared memory, no atomics, no second launch -- so every block has one writer and results do
// not depend on timing.  The first rows are on their way while the angles are worked out.
//
// Measured: 16384 prompt rows of 32/8 heads of 128 in bf16, blocks of 64: 71 us, 5.2 TB/s, and 18.4 to read
// them back as bf16 (144 together with one CTA's warps on all three kinds of rows; keys and values alone
// 43: two rotations of every key, one for the maximum and one for the codes, and waits between a run's
// load, maximum and store); 64 rows of a draft step and reading them 5.8 us.  Keys' CTAs and queries' in
// turn 2 % slower, a run's heads spread over more CTAs (angles worked out anew) 10 %, four CTAs an SM
// (spills) 9 %.
#include "rope.cuh"
#include "scaled.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;        // rows of a CTA where there are many
constexpr int kPasses = 4;       // row groups (items) that a warp (thread) keeps in registers

struct AppendParams {
  const char *k, *v, *q;
  char *q_out, *kc, *vc;
  float *ks, *vs;
  const int64_t* slots;
  const int32_t* pos;                                        // null: no rotation
  long long k_stride, v_stride, q_stride, q_out_stride;      // elements
  long long page_stride, token_stride, head_stride;          // bytes
  FastDiv P, block, heads, per;                              // KV heads; items of a row's queries
  int T, Hq, Hkv, W, Wq, kv_ctas, num_slots;                 // rows of a CTA; CTAs of keys and values
  RopeTable<128> rope;
};

SPEC_DEV long long slot_offset(const FastDiv& P, long long page_stride, long long token_stride,
                               int slot) {
  const int page = P.quot(slot);
  return page * page_stride + (slot - page * P.d) * token_stride;
}

SPEC_DEV void team_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The codes of a block's rows that are not in `written`, under a new scale: the work of `threads` threads
// (whole warps), of which this is number i.
template <int D>
SPEC_DEV void move_others(char* cache, long long token_stride, int block, uint64_t written,
                          float ratio, int i, int threads) {
  constexpr int kLanes = D / 16;
  for (int o = i / kLanes; o < block; o += threads / kLanes)
    if (!(written >> o & 1)) {
      uint4* p = reinterpret_cast<uint4*>(cache + o * token_stride + i % kLanes * 16);
      *p = moved_codes(*p, ratio);
    }
}

// Queries: a CTA turns Wq rows; what its threads hold at once is on its way while the angles are worked out.
template <typename T, int D>
SPEC_DEV void turn_queries(const AppendParams& p, int t0, float* table, int* live) {
  constexpr int kItems = D / 16;
  const int rows = min(p.Wq, p.T - t0), n = rows * p.per.d;
  uint4 raw[kPasses][2];
  auto load = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      const int i = i0 + x * kThreads, u = p.per.quot(i), y = i - u * p.per.d;
      if (i >= n) break;
      const int2 c = rope_chunks(p.rope, y % kItems);
      const uint4* row = reinterpret_cast<const uint4*>(
          reinterpret_cast<const T*>(p.q) + (t0 + u) * p.q_stride + y / kItems * D);
      raw[x][0] = __ldcs(row + c.x);
      raw[x][1] = __ldcs(row + c.y);
    }
  };
  load(threadIdx.x);
  const int j = threadIdx.x % (D / 2);
  const bool turns = j < p.rope.pairs;
  const uint64_t by = turns ? p.rope.turn[j] : 0;
  for (int u = threadIdx.x / (D / 2); u < rows; u += kThreads / (D / 2)) {
    const int at = p.pos ? p.pos[t0 + u] : 0;
    if (j == 0) {
      const int64_t slot = p.slots[t0 + u];
      live[u] = slot >= 0 && slot < p.num_slots && at >= 0;
    }
    if (p.rope.pairs == 0) continue;
    const float2 e = turns ? rope_angle(by, p.rope.magnitude, at) : make_float2(1.f, 0.f);
    float* to = table + u * D + rope_place(kItems, j);
    to[0] = e.x;
    to[D / 2] = e.y;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < n; i0 += kPasses * kThreads) {
    if (i0 != threadIdx.x) load(i0);
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      const int i = i0 + x * kThreads, u = p.per.quot(i), y = i - u * p.per.d, j = y % kItems;
      if (i >= n) break;
      if (!live[u]) continue;
      const int2 c = rope_chunks(p.rope, j);
      uint4* to = reinterpret_cast<uint4*>(
          reinterpret_cast<T*>(p.q_out) + (t0 + u) * p.q_out_stride + y / kItems * D);
      float a[8], e[8];
      unpack_chunk<T>(*reinterpret_cast<const Chunk8<T>*>(&raw[x][0]), a);
      unpack_chunk<T>(*reinterpret_cast<const Chunk8<T>*>(&raw[x][1]), e);
      if (p.rope.pairs > 0)
        rope_turn(p.rope.interleaved, a, e, table + u * D, table + u * D + D / 2, kItems, j);
      to[c.x] = pack_chunk<T>(a).w[0];
      to[c.y] = pack_chunk<T>(e).w[0];
    }
  }
}

// T: type of the rows
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3) append_scaled_kernel(
    const __grid_constant__ AppendParams p) {
  constexpr int kItems = D / 16;               // of a row
  constexpr int kRows = 32 / kItems;           // rows of a warp's pass
  constexpr int kWarpRows = kPasses * kRows;   // that a warp holds
  constexpr int kMost = kTile + kMaxBlock;     // rows looked at
  constexpr int kWords = kMost / 32 + 1;
  extern __shared__ __align__(16) float table[];  // [rows][2][D/2]: cosines, sines
  __shared__ int slot_s[kMost + 1];               // of row t0 - 1 + i; -1: none
  __shared__ int pos_s[kMost + 1];
  __shared__ long long at_s[kMost + 1];           // its place in a cache
  __shared__ uint32_t same[kWords];               // rows whose block is that of the row in front
  __shared__ int run_at[kTile], run_n[kTile];     // the runs that begin here
  __shared__ uint64_t run_to[kTile];              // places of their blocks that they write
  __shared__ int runs, rows_end, longest;
  __shared__ float big_s[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chain_wait();
  if ((int)blockIdx.x >= p.kv_ctas) {
    turn_queries<T, D>(p, (blockIdx.x - p.kv_ctas) * p.Wq, table, slot_s);
    return;
  }
  const bool is_k = (blockIdx.x & 1) == 0;
  const int t0 = (int)(blockIdx.x >> 1) * p.W, t1 = min(t0 + p.W, p.T);
  const int look = min(t1 - 1 + p.block.d, p.T);  // past the last row a run from here may have
  if (threadIdx.x <= kMost) {
    const int t = t0 - 1 + (int)threadIdx.x;
    int s = -1, at = 0;
    if (t >= 0 && t < look) {
      const int64_t slot = p.slots[t];
      at = p.pos ? p.pos[t] : 0;
      if (slot >= 0 && slot < p.num_slots && at >= 0) s = (int)slot;
    }
    slot_s[threadIdx.x] = s;
    pos_s[threadIdx.x] = at;
    at_s[threadIdx.x] = s < 0 ? 0 : slot_offset(p.P, p.page_stride, p.token_stride, s);
  }
  if (threadIdx.x == 0) rows_end = t0, longest = 0;
  __syncthreads();
  if (warp < kWords) {
    const int i = threadIdx.x;
    const bool joined = i > 0 && i <= kMost && slot_s[i] >= 0 && slot_s[i - 1] >= 0 &&
                        p.block.quot(slot_s[i]) == p.block.quot(slot_s[i - 1]);
    const uint32_t word = __ballot_sync(0xffffffffu, joined);
    if (lane == 0) same[warp] = word;
  }
  __syncthreads();
  // ---- the runs that begin in t0 .. t1 - 1, in order
  if (warp == 0) {
    const int i = lane + 1, t = t0 + lane;
    const bool first = t < t1 && slot_s[i] >= 0 && !(same[i >> 5] >> (i & 31) & 1u);
    const uint32_t who = __ballot_sync(0xffffffffu, first);
    if (first) {
      int n = 1;
      for (int y = i + 1; n < p.block.d && y <= kMost;) {
        const int left = 32 - (y & 31), more = __clz(__brev(~(same[y >> 5] >> (y & 31))));
        n += min(more, left), y += left;
        if (more < left) break;
      }
      n = min(n, p.block.d);  // (a slot that comes twice)
      const int r = __popc(who & ((1u << lane) - 1));
      run_at[r] = t;
      run_n[r] = n;
      atomicMax(&rows_end, t + n);
      atomicMax(&longest, n);
    }
    if (lane == 0) runs = __popc(who);
  }
  __syncthreads();
  if (runs == 0) return;
  for (int r = warp; r < runs; r += kWarps) {
    const int first = run_at[r] - t0 + 1, n = run_n[r], b0 = p.block.quot(slot_s[first]) * p.block.d;
    uint32_t lo = 0, hi = 0;
    for (int u = lane; u < n; u += 32) {
      const int o = slot_s[first + u] - b0;
      if (o < 32) lo |= 1u << o; else hi |= 1u << (o - 32);
    }
    lo = __reduce_or_sync(0xffffffffu, lo), hi = __reduce_or_sync(0xffffffffu, hi);
    if (lane == 0) run_to[r] = (uint64_t)hi << 32 | lo;
  }
  __syncthreads();
  // the heads of a row stand together and are used one after the other: on their way to L2 whole
  if (p.Hkv * D >= 512)
    for (int u = threadIdx.x; u < rows_end - t0; u += kThreads) {
      const char* row = (is_k ? p.k : p.v) + (t0 + u) * (is_k ? p.k_stride : p.v_stride) * (int)sizeof(T);
      if (slot_s[u + 1] >= 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row),
                     "r"(p.Hkv * D * (int)sizeof(T))
                     : "memory");
    }

  // ---- keys or values: a team of warps, as many as hold the longest run, takes a run of one head
  int team_warps = 1;
  while (team_warps * kWarpRows < longest) team_warps *= 2;
  const int team = warp / team_warps, mine = warp % team_warps, threads = 32 * team_warps;
  const int items = runs * p.Hkv, step = kWarps / team_warps;
  const int j = lane % kItems, sub = lane / kItems;   // item of a row, row of a pass
  const int2 c = is_k ? rope_chunks(p.rope, j) : make_int2(j, j + kItems);
  const bool turn = is_k && p.rope.pairs > 0;
  const int base = mine * kWarpRows;
  uint4 raw[kPasses][2];
  float stored = 0.f;
  auto load = [&](int i) {  // an item's rows (behind the last: the last again) and scale
    const int r = p.heads.quot(i), h = i - r * p.Hkv, at = run_at[r], n = run_n[r];
    const T* src = reinterpret_cast<const T*>(is_k ? p.k : p.v) + h * D;
    const long long stride = is_k ? p.k_stride : p.v_stride;
    stored = (is_k ? p.ks : p.vs)[(long long)p.block.quot(slot_s[at - t0 + 1]) * p.Hkv + h];
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      if (base + x * kRows >= n) break;
      const int t = at + min(base + x * kRows + sub, n - 1);
      const uint4* row = reinterpret_cast<const uint4*>(src + t * stride);
      raw[x][0] = __ldcs(row + c.x);
      raw[x][1] = __ldcs(row + c.y);
    }
  };
  if (team < items) load(team);  // (on its way while the angles are worked out)
  if (turn) {
    const int j = threadIdx.x % (D / 2), n = rows_end - t0;
    const bool turns = j < p.rope.pairs;
    const uint64_t by = turns ? p.rope.turn[j] : 0;
#pragma unroll 4
    for (int u = threadIdx.x / (D / 2); u < n; u += kThreads / (D / 2)) {
      const float2 e = turns ? rope_angle(by, p.rope.magnitude, pos_s[u + 1]) : make_float2(1.f, 0.f);
      float* to = table + u * D + rope_place(kItems, j);
      to[0] = e.x;
      to[D / 2] = e.y;
    }
    __syncthreads();
  }
  int buf = 0;
  for (int i = team; i < items; i += step, buf ^= 1) {
    const int r = p.heads.quot(i), h = i - r * p.Hkv;
    const int at = run_at[r], n = run_n[r], first = at - t0 + 1;
    const int b = p.block.quot(slot_s[first]);
    float* scale = (is_k ? p.ks : p.vs) + (long long)b * p.Hkv + h;
    if (i != team) load(i);
    auto values = [&](int x, float* a, float* e) {
      unpack_chunk<T>(*reinterpret_cast<const Chunk8<T>*>(&raw[x][0]), a);
      unpack_chunk<T>(*reinterpret_cast<const Chunk8<T>*>(&raw[x][1]), e);
      if (turn) {
        const float* cs = table + (first - 1 + min(base + x * kRows + sub, n - 1)) * D;
        rope_turn(p.rope.interleaved, a, e, cs, cs + D / 2, kItems, j);
      }
    };
    const uint64_t written = run_to[r];
    float big = 0.f;
    bool packed = !turn;
    if (packed) {  // magnitudes compare as their bits do, two at a time
      uint32_t m = 0;
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        if (base + x * kRows >= n) break;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint4 w = raw[x][y];
          m = __vimax3_u16x2(m, w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
          m = __vimax3_u16x2(m, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
        }
      }
      const unsigned short top = (unsigned short)max(m & 0xffffu, m >> 16);
      big = static_cast<float>(*reinterpret_cast<const T*>(&top));
      packed = big < INFINITY;  // (else some value is not finite, and does not count)
    }
    if (!packed) {
      big = 0.f;
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        if (base + x * kRows >= n) break;
        float a[8], e[8];
        values(x, a, e);
#pragma unroll
        for (int y = 0; y < 8; ++y) big = fmaxf(big, fmaxf(finite_abs(a[y]), finite_abs(e[y])));
      }
    }
    big = warp_max(big);
    if (team_warps > 1) {
      if (lane == 0) big_s[buf][warp] = big;
      team_sync(1 + team, threads);
      for (int w = 0; w < team_warps; ++w) big = fmaxf(big, big_s[buf][team * team_warps + w]);
    }
    const float held = written & 1 ? 0.f : held_scale(stored);  // (a block begun anew: its own)
    const float s = fmaxf(held, needed_scale(big));
    char* cache = (is_k ? p.kc : p.vc) + h * p.head_stride;
    if (held > 0.f && s != stored)
      move_others<D>(cache + slot_offset(p.P, p.page_stride, p.token_stride, b * p.block.d),
                     p.token_stride, p.block.d, written, stored / s, mine * 32 + lane, threads);
    if (mine == 0 && lane == 0 && s != stored) *scale = s;
    const float by = 1.f / s;  // (a power of two)
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      const int u = base + x * kRows + sub;
      if (base + x * kRows >= n) break;
      float a[8], e[8];
      values(x, a, e);
      if (u < n) {
        char* to = cache + at_s[first + u];
#pragma unroll
        for (int y = 0; y < 8; ++y) a[y] *= by, e[y] *= by;
        const uint2 first8 =
            make_uint2(e4m3_word(a[0], a[1], a[2], a[3]), e4m3_word(a[4], a[5], a[6], a[7]));
        const uint2 other8 =
            make_uint2(e4m3_word(e[0], e[1], e[2], e[3]), e4m3_word(e[4], e[5], e[6], e[7]));
        *reinterpret_cast<uint2*>(to + c.x * 8) = first8;
        *reinterpret_cast<uint2*>(to + c.y * 8) = other8;
      }
    }
  }
}

// ------------------------------------------------------------------ reading back
struct ReadParams {
  const char *kc, *vc;
  const float *ks, *vs;
  const int64_t* slots;
  char *k_out, *v_out;
  long long page_stride, token_stride, head_stride;  // bytes
  long long k_stride, v_stride;                      // elements
  FastDiv P, block, chunks, per;                     // 16-byte chunks of a row's head; of a row
  int T, Hkv, W, num_slots;                          // rows of a CTA
};

// A thread takes 16 codes of a key and of the value beside it.
template <typename O>
__global__ void __launch_bounds__(kThreads) read_scaled_kernel(const __grid_constant__ ReadParams p) {
  chain_wait();
  const int t0 = blockIdx.x * p.W, n = min(p.W, p.T - t0) * p.per.d;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int u = p.per.quot(i), y = i - u * p.per.d, h = p.chunks.quot(y), x = y - h * p.chunks.d;
    const int64_t slot = p.slots[t0 + u];
    if (slot < 0 || slot >= p.num_slots) continue;
    const long long from = slot_offset(p.P, p.page_stride, p.token_stride, (int)slot) +
                           h * p.head_stride + x * 16;
    const long long sc = (long long)p.block.quot((int)slot) * p.Hkv + h;
    uint4 w[2];
    float s[2];
    w[0] = *reinterpret_cast<const uint4*>(p.kc + from);
    s[0] = p.ks[sc];
    if (p.vc) {
      w[1] = *reinterpret_cast<const uint4*>(p.vc + from);
      s[1] = p.vs[sc];
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (kv && !p.vc) break;
      float v[16];
      e4m3_values(w[kv].x, v);
      e4m3_values(w[kv].y, v + 4);
      e4m3_values(w[kv].z, v + 8);
      e4m3_values(w[kv].w, v + 12);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= s[kv];
      Chunk8<O>* to = reinterpret_cast<Chunk8<O>*>(
          reinterpret_cast<O*>(kv ? p.v_out : p.k_out) +
          (t0 + u) * (kv ? p.v_stride : p.k_stride) + y * 16);
      to[0] = pack_chunk<O>(v);
      to[1] = pack_chunk<O>(v + 8);
    }
  }
}

// ------------------------------------------------------------------ commit
struct CommitParams {
  char *kc, *vc;
  float *ks, *vs;
  const int32_t *table, *ctx, *accepted, *path, *parent;
  int32_t *new_len, *keep, *status;
  FastDiv P, block;
  int num_pages, Hkv, max_pages, R;
};

// A CTA per sequence and KV head: every moving row is read into shared memory before any is
// written, then a warp takes each block that rows move to, of the keys and of the values.
template <int D>
__global__ void __launch_bounds__(kThreads) commit_scaled_kernel(
    const __grid_constant__ CommitParams p) {
  constexpr int kChunks = D / 16;
  __shared__ uint4 rows[2][64][kChunks];
  __shared__ float row_scale[2][64];
  __shared__ int ok;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chain_wait();
  const int c = p.ctx[b], a = p.accepted[b], P = p.P.d;
  const int32_t* bt = p.table + (size_t)b * p.max_pages;
  const int32_t* pth = p.path + (size_t)b * p.R;
  const int32_t* par = p.parent ? p.parent + (size_t)b * p.R : nullptr;
  if (threadIdx.x == 0) {
    bool good = c >= 0 && a >= 0 && a < p.R && (long long)c + p.R <= (long long)p.max_pages * P;
    int prev = 0;  // the anchor
    for (int i = 0; i < a && good; ++i) {
      const int v = pth[i];
      good = v > prev && v < p.R && (!par || par[v] == prev);
      prev = v;
      if (good) {
        const int ps = bt[(c + v) / P], pd = bt[(c + i + 1) / P];
        good = ps >= 0 && ps < p.num_pages && pd >= 0 && pd < p.num_pages;
      }
    }
    ok = good;
    if (h == 0) {
      const int n = good ? c + 1 + a : c;
      p.new_len[b] = n;
      if (p.keep) p.keep[b] = (int)(((long long)n + P - 1) / P);
      if (p.status) p.status[b] = good ? 0 : SPEC_SEQ_BAD_TREE;
    }
  }
  __syncthreads();
  if (!ok || a == 0) return;
  auto slot_of = [&](int t) { return (long long)bt[p.P.quot(t)] * P + (t - p.P.quot(t) * P); };
  auto code_at = [&](int kv, long long slot) {
    return (kv ? p.vc : p.kc) + (slot * p.Hkv + h) * D;
  };
  const int nb = P / p.block.d;
  auto scale_at = [&](int kv, int t) {
    const int page = p.P.quot(t);
    return (kv ? p.vs : p.ks) +
           ((long long)bt[page] * nb + p.block.quot(t - page * P)) * p.Hkv + h;
  };
  for (int i = threadIdx.x; i < 2 * a * kChunks; i += kThreads) {
    const int kv = i / (a * kChunks), r = i - kv * a * kChunks, k = r / kChunks, x = r % kChunks;
    rows[kv][k][x] = reinterpret_cast<const uint4*>(code_at(kv, slot_of(c + pth[k])))[x];
    if (x == 0) row_scale[kv][k] = *scale_at(kv, c + pth[k]);
  }
  __syncthreads();
  // blocks of positions c + 1 .. c + a (a page holds whole blocks)
  const int first = p.block.quot(c + 1), last = p.block.quot(c + a);
  for (int i = warp; i < 2 * (last - first + 1); i += kWarps) {
    const int kv = i & 1, blk = first + (i >> 1);
    const int begin = blk * p.block.d;
    const int lo = max(begin, c + 1), hi = min(begin + p.block.d, c + a + 1);  // written positions
    float big = 0.f;
    for (int u = lane; u < (hi - lo) * kChunks; u += 32) {
      const int k = lo - c - 1 + u / kChunks;
      const uint4 w = rows[kv][k][u % kChunks];
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x[4];
        e4m3_values(ww[e], x);
#pragma unroll
        for (int y = 0; y < 4; ++y) big = fmaxf(big, finite_abs(x[y] * row_scale[kv][k]));
      }
    }
    big = warp_max(big);
    float* scale = scale_at(kv, begin);
    const float stored = *scale, held = lo == begin ? 0.f : held_scale(stored);
    const float s = fmaxf(held, needed_scale(big));
    if (held > 0.f && s != stored) {
      const uint64_t written =
          (hi - lo == 64 ? ~0ull : (1ull << (hi - lo)) - 1) << (lo - begin);
      move_others<D>(code_at(kv, slot_of(begin)), (long long)p.Hkv * D, p.block.d, written,
                     stored / s, lane, 32);
    }
    __syncwarp();
    if (lane == 0 && s != stored) *scale = s;
    for (int u = lane; u < (hi - lo) * kChunks; u += 32) {
      const int k = lo - c - 1 + u / kChunks;
      reinterpret_cast<uint4*>(code_at(kv, slot_of(c + 1 + k)))[u % kChunks] =
          moved_codes(rows[kv][k][u % kChunks], row_scale[kv][k] / s);
    }
  }
}

// ------------------------------------------------------------------ host side
template <typename T, int D>
spec_status launch_append(const AppendParams& p, cudaStream_t st) {
  const size_t smem =
      p.rope.pairs ? (size_t)std::max(p.W - 1 + p.block.d, p.Wq) * D * sizeof(float) : 0;
  static PerDeviceOnce<int> once;
  const spec_status rc = ensure_smem_limit(once, (const void*)append_scaled_kernel<T, D>,
                                           (kTile - 1 + kMaxBlock) * D * (int)sizeof(float));
  if (rc != SPEC_OK) return rc;
  const int grid = p.kv_ctas + (p.Hq ? (p.T + p.Wq - 1) / p.Wq : 0);
  return launch_chained(append_scaled_kernel<T, D>, grid, kThreads, smem, st, p);
}

template <typename T>
spec_status launch_append_d(const AppendParams& p, int D, cudaStream_t st) {
  return D == 64 ? launch_append<T, 64>(p, st)
                 : D == 128 ? launch_append<T, 128>(p, st) : launch_append<T, 256>(p, st);
}

// What the calls ask of a scaled cache.
spec_status check_cache(const void* k_cache, const void* v_cache, int num_pages, int page_size,
                        int block, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                        int Hkv, int D) {
  if (num_pages < 1 || page_size < 1 || Hkv < 1 || block < 1 || page_size % block)
    return SPEC_EINVAL;
  if (block > kMaxBlock || Hkv > 4096 || (D != 64 && D != 128 && D != 256))
    return SPEC_EUNSUPPORTED;
  if ((long long)num_pages * page_size > INT32_MAX - kMaxBlock) return SPEC_EUNSUPPORTED;
  if (page_stride < 0 || token_stride < 0 || head_stride < 0) return SPEC_EINVAL;
  if ((((uintptr_t)k_cache | (uintptr_t)v_cache) & 15) ||
      ((page_stride | token_stride | head_stride) & 15))
    return SPEC_EINVAL;
  return SPEC_OK;
}

}  // namespace

extern "C" spec_status spec_append_scaled(
    const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, const void* q,
    int64_t q_stride, void* q_out, int64_t q_out_stride, spec_dtype new_dtype, void* k_cache,
    void* v_cache, float* k_scale, float* v_scale, int num_pages, int page_size, int block,
    int64_t page_stride, int64_t token_stride, int64_t head_stride, const int64_t* slot_map,
    const int32_t* positions, int T, int Hq, int Hkv, int D, const spec_rope* rope, void* stream) {
  if (T < 0 || Hq < 0) return SPEC_EINVAL;
  spec_status rc = check_cache(k_cache, v_cache, num_pages, page_size, block, page_stride,
                               token_stride, head_stride, Hkv, D);
  if (rc != SPEC_OK) return rc;
  if (new_dtype == SPEC_F32) return SPEC_EUNSUPPORTED;
  if (new_dtype != SPEC_BF16 && new_dtype != SPEC_F16) return SPEC_EINVAL;
  if (Hq > 4096 || T > INT32_MAX - kMaxBlock) return SPEC_EUNSUPPORTED;
  if ((q == nullptr) != (q_out == nullptr) || (q && Hq < 1)) return SPEC_EINVAL;
  AppendParams p{};
  rc = rope_table(rope, D, &p.rope);
  if (rc != SPEC_OK) return rc;
  if (T == 0) return SPEC_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !slot_map ||
      (rope && !positions))
    return SPEC_EINVAL;
  if (((uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)q | (uintptr_t)q_out) & 15)
    return SPEC_EINVAL;
  if (k_stride < 0 || v_stride < 0 || q_stride < 0 || q_out_stride < 0) return SPEC_EINVAL;
  if (((k_stride | v_stride | (q ? q_stride | q_out_stride : 0)) * 2) & 15) return SPEC_EINVAL;
  if (q && q == q_out && q_stride != q_out_stride) return SPEC_EINVAL;
  // (K's and V's caches may lie between one another; their scales are contiguous)
  const size_t scales = (size_t)num_pages * (page_size / block) * Hkv * sizeof(float);
  if (k_cache == v_cache || share({{k_scale, scales}, {v_scale, scales}}, {})) return SPEC_EINVAL;
  p.k = static_cast<const char*>(k_new);
  p.v = static_cast<const char*>(v_new);
  p.q = static_cast<const char*>(q);
  p.q_out = static_cast<char*>(q_out);
  p.kc = static_cast<char*>(k_cache);
  p.vc = static_cast<char*>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  p.slots = slot_map;
  p.pos = rope ? positions : nullptr;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.P = FastDiv(page_size);
  p.block = FastDiv(block);
  p.per = FastDiv(std::max(1, Hq * (D / 16)));
  p.T = T;
  p.Hq = q ? Hq : 0;
  p.Hkv = Hkv;
  // rows of a CTA: few where there are few, else a run's share of a block, and for the queries what its
  // threads hold at once
  const int sms = sm_count();
  p.W = std::min(kTile, std::max(1, T / (2 * sms)));
  p.heads = FastDiv(Hkv);
  p.kv_ctas = 2 * ((T + p.W - 1) / p.W);
  p.Wq = std::max(1, std::min({kPasses * kThreads / p.per.d, T / (2 * sms), kTile}));
  p.num_slots = num_pages * page_size;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return new_dtype == SPEC_BF16 ? launch_append_d<__nv_bfloat16>(p, D, st)
                                : launch_append_d<__half>(p, D, st);
}

extern "C" spec_status spec_read_scaled(const void* k_cache, const void* v_cache,
                                        const float* k_scale, const float* v_scale, int num_pages,
                                        int page_size, int block, int64_t page_stride,
                                        int64_t token_stride, int64_t head_stride,
                                        const int64_t* slot_map, int T, int Hkv, int D,
                                        void* k_out, int64_t k_out_stride, void* v_out,
                                        int64_t v_out_stride, spec_dtype out_dtype, void* stream) {
  if (T < 0) return SPEC_EINVAL;
  const spec_status rc = check_cache(k_cache, v_cache, num_pages, page_size, block, page_stride,
                                     token_stride, head_stride, Hkv, D);
  if (rc != SPEC_OK) return rc;
  if (out_dtype != SPEC_BF16 && out_dtype != SPEC_F16 && out_dtype != SPEC_F32) return SPEC_EINVAL;
  if ((v_out == nullptr) != (v_cache == nullptr) || (v_out == nullptr) != (v_scale == nullptr))
    return SPEC_EINVAL;
  if (T > INT32_MAX - kMaxBlock) return SPEC_EUNSUPPORTED;
  if (T == 0) return SPEC_OK;
  if (!k_cache || !k_scale || !slot_map || !k_out) return SPEC_EINVAL;
  if (((uintptr_t)k_out | (uintptr_t)v_out) & 15) return SPEC_EINVAL;
  const int es = out_dtype == SPEC_F32 ? 4 : 2;
  if (k_out_stride < 0 || v_out_stride < 0 ||
      (((k_out_stride | (v_out ? v_out_stride : 0)) * es) & 15))
    return SPEC_EINVAL;
  ReadParams p{};
  p.kc = static_cast<const char*>(k_cache);
  p.vc = static_cast<const char*>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  p.slots = slot_map;
  p.k_out = static_cast<char*>(k_out);
  p.v_out = static_cast<char*>(v_out);
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.k_stride = k_out_stride;
  p.v_stride = v_out_stride;
  p.P = FastDiv(page_size);
  p.block = FastDiv(block);
  p.chunks = FastDiv(D / 16);
  p.per = FastDiv(Hkv * (D / 16));
  p.T = T;
  p.Hkv = Hkv;
  p.W = std::max(1, kThreads / p.per.d);
  p.num_slots = num_pages * page_size;
  const int grid = (int)(((long long)T + p.W - 1) / p.W);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_dtype == SPEC_F32) return launch_chained(read_scaled_kernel<float>, grid, kThreads, 0, st, p);
  if (out_dtype == SPEC_BF16)
    return launch_chained(read_scaled_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
  return launch_chained(read_scaled_kernel<__half>, grid, kThreads, 0, st, p);
}

extern "C" spec_status spec_commit_scaled(void* k_cache, void* v_cache, float* k_scale,
                                          float* v_scale, int num_pages, int page_size, int block,
                                          int Hkv, int D, const int32_t* block_table,
                                          int max_pages, const int32_t* ctx_len,
                                          const int32_t* accepted_len, const int32_t* path,
                                          const int32_t* parent, int B, int R, int32_t* new_len,
                                          int32_t* keep_pages, int32_t* status_per_seq,
                                          void* stream) {
  if (B < 0 || R < 1 || R > 64 || max_pages < 1) return SPEC_EINVAL;
  const spec_status rc = check_cache(k_cache, v_cache, num_pages, page_size, block, 0, 0, 0, Hkv, D);
  if (rc != SPEC_OK) return rc;
  if ((long long)max_pages * page_size > INT32_MAX - kMaxBlock || (long long)B * Hkv > INT32_MAX)
    return SPEC_EUNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !ctx_len || !accepted_len ||
      !path || !new_len)
    return SPEC_EINVAL;
  // A sequence's lengths are read by the CTAs of all its heads and written by one.
  const size_t slots = (size_t)num_pages * page_size, seqs = (size_t)B * sizeof(int32_t);
  const size_t scales = slots / block * Hkv * sizeof(float);
  if (share({{k_cache, slots * Hkv * D}, {v_cache, slots * Hkv * D}, {k_scale, scales},
             {v_scale, scales}, {new_len, seqs}, {keep_pages, seqs}, {status_per_seq, seqs}},
            {{block_table, seqs * max_pages}, {ctx_len, seqs}, {accepted_len, seqs},
             {path, seqs * R}, {parent, seqs * R}}))
    return SPEC_EINVAL;
  CommitParams p{};
  p.kc = static_cast<char*>(k_cache);
  p.vc = static_cast<char*>(v_cache);
  p.ks = k_scale;
  p.vs = v_scale;
  p.table = block_table;
  p.ctx = ctx_len;
  p.accepted = accepted_len;
  p.path = path;
  p.parent = parent;
  p.new_len = new_len;
  p.keep = keep_pages;
  p.status = status_per_seq;
  p.P = FastDiv(page_size);
  p.block = FastDiv(block);
  p.num_pages = num_pages;
  p.Hkv = Hkv;
  p.max_pages = max_pages;
  p.R = R;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = B * Hkv;
  if (D == 64) return launch_chained(commit_scaled_kernel<64>, grid, kThreads, 0, st, p);
  if (D == 128) return launch_chained(commit_scaled_kernel<128>, grid, kThreads, 0, st, p);
  return launch_chained(commit_scaled_kernel<256>, grid, kThreads, 0, st, p);
}
