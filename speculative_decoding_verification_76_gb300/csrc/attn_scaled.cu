// spec_verify_attn_scaled -- the host side: checks, the plan of row tiles and ranges, the
// workspace.  The kernels and the reasons for them are in attn_scaled.cuh; each head size is a
// translation unit of its own.
#include <algorithm>

#include "attn_scaled.cuh"

namespace {

using scaled_attn::Params;

struct Plan {
  int tiles, rows_per_tile, rt, teams;
};

bool make_plan(int B, int R, int Hq, int Hkv, int D, Plan* pl) {
  if (B < 0 || R < 1 || R > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv ||
      (D != 64 && D != 128 && D != 256))
    return false;
  const long long rows = (long long)R * (Hq / Hkv);
  if (rows > 64ll * 65535) return false;
  const int most = scaled_attn::most_rows(D);
  pl->tiles = (int)((rows + most - 1) / most);
  pl->rows_per_tile = (int)((rows + pl->tiles - 1) / pl->tiles);
  pl->rt = pl->rows_per_tile <= 16 ? 16 : pl->rows_per_tile <= 32 ? 32 : 64;
  pl->teams = std::max(1, sm_count() / pl->tiles);
  return true;
}

size_t layout(const Plan& pl, int D, size_t* off_o, size_t* off_ml) {
  const size_t rows = (size_t)pl.teams * 2 * pl.tiles * pl.rt;
  size_t off = sizeof(WsHeader);
  *off_o = off;
  off += rows * D * sizeof(float);
  *off_ml = off;
  off += (rows * 2 * sizeof(float) + 255) / 256 * 256;
  return off;
}

}  // namespace

extern "C" size_t spec_verify_attn_scaled_workspace_size(int B, int R, int Hq, int Hkv, int D) {
  Plan pl;
  size_t a, b;
  return make_plan(B, R, Hq, Hkv, D, &pl) ? layout(pl, D, &a, &b) : 0;
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
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !ctx_len ||
      !workspace || !out)
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
  // cache rows are numbered in token strides, in 31 bits
  if (token_stride < 1) return SPEC_EINVAL;
  if (page_stride % token_stride || token_stride > UINT32_MAX) return SPEC_EUNSUPPORTED;
  const int64_t page_rows = page_stride / token_stride;
  if (page_rows > INT32_MAX || page_rows * (num_pages - 1) + page_size > INT32_MAX)
    return SPEC_EUNSUPPORTED;
  // so are positions, and the batch's tiles over all KV heads
  if ((long long)max_pages * page_size > INT32_MAX - 512 || B > INT32_MAX - 512)
    return SPEC_EUNSUPPORTED;
  const double units =
      ((double)max_pages * page_size / scaled_attn::kUnit + 1 + scaled_attn::kMostEnds) * B * Hkv;
  if (units > INT32_MAX - 1024.0) return SPEC_EUNSUPPORTED;
  if ((double)B * ((double)R * Hq / scaled_attn::kJoinWarps + 1) > INT32_MAX) return SPEC_EUNSUPPORTED;
  Plan pl;
  if (!make_plan(B, R, Hq, Hkv, D, &pl)) return SPEC_EUNSUPPORTED;
  if ((long long)Hkv * pl.tiles > 4096) return SPEC_EUNSUPPORTED;
  size_t off_o, off_ml;
  if (workspace_bytes < layout(pl, D, &off_o, &off_ml)) return SPEC_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
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
  p.part_o = reinterpret_cast<float*>(ws + off_o);
  p.part_ml = reinterpret_cast<float*>(ws + off_ml);
  p.err = &reinterpret_cast<WsHeader*>(ws)->error;
  p.q_stride_b = q_stride_b;
  p.q_stride_r = q_stride_r;
  p.q_stride_h = q_stride_h;
  p.head_stride = head_stride;
  p.token_stride = (uint32_t)token_stride;
  p.page_rows = (uint32_t)page_rows;
  p.P = FastDiv(page_size);
  p.block = FastDiv(block);
  p.per_head = FastDiv(Hq / Hkv);
  p.B = B;
  p.R = R;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.window = window;
  p.tiles = pl.tiles;
  p.rows_per_tile = pl.rows_per_tile;
  p.teams = pl.teams;
  p.ends = pl.rt == 64 ? scaled_attn::kMostEnds : 8;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  unsigned long long wait_ns;
  attn_fault_setting(&p.withhold_stage, &wait_ns);
  p.polls = (uint32_t)std::min<unsigned long long>(wait_ns / 1000 + 1, UINT32_MAX);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = q_dtype == SPEC_F16;
  return D == 64 ? scaled_attn::launch_d64(p, pl.rt, f16, st)
                 : D == 128 ? scaled_attn::launch_d128(p, pl.rt, f16, st)
                            : scaled_attn::launch_d256(p, pl.rt, f16, st);
}
