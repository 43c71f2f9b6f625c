// C ABI of the 8-bit KV cache (msa_cache.h): argument validation, workspace
// layout and launch.  As in msa_api.cu,
// everything is checked before anything is enqueued, and nothing allocates
// or synchronises.
#include "api_common.cuh"

namespace {

msa::CacheView view(const msa_kv_cache* c) {
  return {static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scale,
          c->v_scale, static_cast<__nv_bfloat16*>(c->k_mean), c->n_pages, c->Hkv, c->d, c->block,
          log2_of(c->block)};
}

// Attention workspace: the parts of the units that several CTAs share, and
// for weights every row's scores and lse.
struct AttnPlan {
  int n_ctas;
  size_t o, part_stat, scores, row_stat, total;
};

AttnPlan attn_plan(int Hkv, int d, int block, int batch, int n_q, int Hq, int max_blocks,
                   bool select, bool weights, int in_bf16) {
  const int g = Hq / Hkv;
  const int rows = select ? g : n_q * g;
  const int tile = msa::cache_attn_tile_rows(rows, in_bf16);
  const int64_t units =
      static_cast<int64_t>(select ? batch * n_q : batch) * Hkv * ((rows + tile - 1) / tile);
  const int64_t chunks = units * (static_cast<int64_t>(max_blocks) * block / msa::kChunk);
  AttnPlan p{};
  p.n_ctas = static_cast<int>(msa::max64(
      1, msa::min64(msa::cache_attn_max_ctas(tile, in_bf16),
                    msa::max64(units, (chunks + 3) / 4))));
  size_t at = 0;
  p.o = at;
  at += up(static_cast<size_t>(2) * p.n_ctas * tile * d * sizeof(float));
  p.part_stat = at;
  at += up(static_cast<size_t>(2) * p.n_ctas * tile * sizeof(float4));
  if (weights) {
    const size_t even = (static_cast<size_t>(rows) + 1) & ~static_cast<size_t>(1);
    p.scores = at;
    at += up(static_cast<size_t>(batch) * Hkv * max_blocks * block * even * sizeof(float));
    p.row_stat = at;
    at += up(static_cast<size_t>(batch) * Hkv * even * sizeof(float2));
  }
  p.total = at;
  return p;
}

struct SelectPlan {
  size_t score, err, exact, total;
};

SelectPlan select_plan(int Hkv, int batch, int n_q, int max_blocks) {
  const size_t n = static_cast<size_t>(batch) * n_q * Hkv * max_blocks;
  SelectPlan p{};
  p.exact = 0;
  p.score = up(n * sizeof(double));
  p.err = p.score + up(n * sizeof(float));
  p.total = p.err + up(n * sizeof(float));
  return p;
}

msa_status run_attn(const msa_kv_cache* c, const void* q, const int32_t* table, int max_blocks,
                    const int32_t* lens, int batch, int n_q, int Hq, int64_t window, float scale,
                    void* out, float* lse, const int32_t* sel, const int32_t* cnt, int top_k,
                    bool sel_from_kernel, float* weights, int64_t weights_ld, msa_dtype in_dt,
                    msa_dtype out_dt, uint8_t* ws, msa_stream_t stream) {
  const AttnPlan p = attn_plan(c->Hkv, c->d, c->block, batch, n_q, Hq, max_blocks, sel != nullptr,
                               weights != nullptr, in_dt == MSA_BF16);
  msa::CacheAttnArgs a{};
  a.c = view(c);
  a.s = {table, max_blocks, lens, batch};
  a.q = q;
  a.T = n_q;
  a.Hq = Hq;
  a.window = static_cast<int>(msa::min64(window, static_cast<int64_t>(max_blocks) * c->block));
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.sel = sel;
  a.cnt = cnt;
  a.sel_from_kernel = sel_from_kernel;
  a.top_k = top_k;
  a.weights = weights;
  a.weights_ld = weights_ld;
  a.o_part = reinterpret_cast<float*>(ws + p.o);
  a.part_stat = reinterpret_cast<float4*>(ws + p.part_stat);
  a.scores = reinterpret_cast<float*>(ws + p.scores);
  a.row_stat = reinterpret_cast<float2*>(ws + p.row_stat);
  a.n_ctas = p.n_ctas;
  a.in_bf16 = in_dt == MSA_BF16;
  a.out_bf16 = out_dt == MSA_BF16;
  msa_status st = msa::api_status_word(&a.status);
  if (st != MSA_OK) return st;
  return launched(msa::launch_cache_attn(a, reinterpret_cast<cudaStream_t>(stream)),
                  "cache attention");
}

msa_status run_select(const msa_kv_cache* c, const void* q, const int32_t* table, int max_blocks,
                      const int32_t* lens, int batch, int n_q, int Hq, int64_t window, int top_k,
                      int32_t* sel, int32_t* cnt, msa_dtype in_dt, uint8_t* ws,
                      msa_stream_t stream) {
  const SelectPlan p = select_plan(c->Hkv, batch, n_q, max_blocks);
  msa::CacheSelectArgs a{};
  a.c = view(c);
  a.s = {table, max_blocks, lens, batch};
  a.q = q;
  a.T = n_q;
  a.Hq = Hq;
  a.window = static_cast<int>(msa::min64(window, static_cast<int64_t>(max_blocks) * c->block));
  a.top_k = top_k;
  a.sel = sel;
  a.cnt = cnt;
  a.exact = reinterpret_cast<double*>(ws + p.exact);
  a.score = reinterpret_cast<float*>(ws + p.score);
  a.err = reinterpret_cast<float*>(ws + p.err);
  a.bf16 = in_dt == MSA_BF16;
  msa_status st = msa::api_status_word(&a.status);
  if (st != MSA_OK) return st;
  return launched(msa::launch_cache_select(a, reinterpret_cast<cudaStream_t>(stream)),
                  "cache block selection");
}

msa_status check_top_k(int top_k, int max_blocks) {
  if (top_k < 1 || top_k > max_blocks)
    return fail(MSA_ERR_INVALID_ARG, "top_k=%d must be in 1 .. max_blocks=%d", top_k, max_blocks);
  return MSA_OK;
}

}  // namespace

extern "C" {

msa_status msa_cache_append(const msa_kv_cache* cache, const void* k, const void* v,
                            const int32_t* cu, int64_t total, int64_t max_new,
                            const int32_t* table, int max_blocks, const int32_t* lens, int batch,
                            msa_dtype in_dt, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  if (!cu || !aligned(cu, 4)) return fail(MSA_ERR_INVALID_ARG, "cu null or not 4-byte aligned");
  if (total < 0 || total > INT32_MAX || max_new < 0 || max_new > total)
    return fail(MSA_ERR_INVALID_ARG, "total=%lld max_new=%lld (0 <= max_new <= total)",
                (long long)total, (long long)max_new);
  if (!valid_dtype(in_dt)) return fail(MSA_ERR_INVALID_ARG, "bad input dtype %d", (int)in_dt);
  if (max_new == 0) return msa::api_ok();
  if (!k || !v) return fail(MSA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(k, 16) || !aligned(v, 16))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointer not 16-byte aligned");
  const int64_t blocks = msa::min64((max_new + cache->block - 2) / cache->block + 1, max_blocks);
  if (blocks * cache->Hkv * 2 > INT32_MAX)
    return fail(MSA_ERR_UNSUPPORTED, "max_new=%lld too long for one call", (long long)max_new);
  msa::AppendArgs a{};
  a.c = view(cache);
  a.s = {table, max_blocks, lens, batch};
  a.k = k;
  a.v = v;
  a.cu = cu;
  a.total = total;
  a.max_new = max_new;
  a.blocks = static_cast<uint32_t>(blocks);
  a.bf16 = in_dt == MSA_BF16;
  MSA_TRY(msa::api_status_word(&a.status));
  return launched(msa::launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream)),
                  "cache append");
}

size_t msa_cache_attn_workspace_size(const msa_kv_cache* cache, int max_blocks, int batch, int n_q,
                                     int Hq, int with_weights, msa_dtype in_dt) {
  if (!cache ||
      check_sizes(cache->n_pages, cache->Hkv, cache->d, cache->block, batch, max_blocks) != MSA_OK ||
      check_query_sizes(cache, batch, n_q, Hq, max_blocks) != MSA_OK || !valid_dtype(in_dt))
    return 0;
  return attn_plan(cache->Hkv, cache->d, cache->block, batch, n_q, Hq, max_blocks, false,
                   with_weights != 0, in_dt == MSA_BF16)
      .total;
}

msa_status msa_cache_attn(const msa_kv_cache* cache, const void* q, const int32_t* table,
                          int max_blocks, const int32_t* lens, int batch, int n_q, int Hq,
                          int64_t window, float scale, void* out, float* lse, float* weights,
                          int64_t weights_ld, msa_dtype in_dt, msa_dtype out_dt, void* workspace,
                          size_t workspace_bytes, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_query_sizes(cache, batch, n_q, Hq, max_blocks));
  MSA_TRY(check_query(q, out, lse, window, scale, in_dt, out_dt));
  if (weights) {
    if (!aligned(weights, 4)) return fail(MSA_ERR_INVALID_ARG, "weights not 4-byte aligned");
    if (weights_ld < static_cast<int64_t>(max_blocks) * cache->block)
      return fail(MSA_ERR_INVALID_ARG, "weights_ld=%lld below max_blocks * block",
                  (long long)weights_ld);
    if (static_cast<int64_t>(batch) * cache->Hkv > 65535)
      return fail(MSA_ERR_UNSUPPORTED, "batch * Hkv above 65535 with weights");
  }
  const AttnPlan p = attn_plan(cache->Hkv, cache->d, cache->block, batch, n_q, Hq, max_blocks,
                               false, weights != nullptr, in_dt == MSA_BF16);
  MSA_TRY(check_workspace(workspace, workspace_bytes, p.total));
  return run_attn(cache, q, table, max_blocks, lens, batch, n_q, Hq, window, scale, out, lse,
                  nullptr, nullptr, 0, false, weights, weights_ld, in_dt, out_dt,
                  static_cast<uint8_t*>(workspace), stream);
}

size_t msa_cache_select_workspace_size(const msa_kv_cache* cache, int max_blocks, int batch,
                                       int n_q) {
  if (!cache ||
      check_sizes(cache->n_pages, cache->Hkv, cache->d, cache->block, batch, max_blocks) != MSA_OK ||
      check_query_sizes(cache, batch, n_q, cache->Hkv, max_blocks) != MSA_OK)
    return 0;
  return select_plan(cache->Hkv, batch, n_q, max_blocks).total;
}

msa_status msa_cache_select(const msa_kv_cache* cache, const void* q, const int32_t* table,
                            int max_blocks, const int32_t* lens, int batch, int n_q, int Hq,
                            int64_t window, int top_k, int32_t* sel, int32_t* cnt,
                            msa_dtype in_dt, void* workspace, size_t workspace_bytes,
                            msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_query_sizes(cache, batch, n_q, Hq, max_blocks));
  if (!q || !sel || !cnt) return fail(MSA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(q, 16) || !aligned(sel, 4) || !aligned(cnt, 4))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointer not aligned (q: 16 bytes, sel, cnt: 4)");
  if (!valid_dtype(in_dt)) return fail(MSA_ERR_INVALID_ARG, "bad input dtype %d", (int)in_dt);
  MSA_TRY(check_window(window));
  MSA_TRY(check_top_k(top_k, max_blocks));
  MSA_TRY(check_workspace(workspace, workspace_bytes,
                          select_plan(cache->Hkv, batch, n_q, max_blocks).total));
  return run_select(cache, q, table, max_blocks, lens, batch, n_q, Hq, window, top_k, sel, cnt,
                    in_dt, static_cast<uint8_t*>(workspace), stream);
}

size_t msa_cache_attn_select_workspace_size(const msa_kv_cache* cache, int max_blocks, int batch,
                                            int n_q, int Hq, msa_dtype in_dt) {
  if (!cache ||
      check_sizes(cache->n_pages, cache->Hkv, cache->d, cache->block, batch, max_blocks) != MSA_OK ||
      check_query_sizes(cache, batch, n_q, Hq, max_blocks) != MSA_OK || !valid_dtype(in_dt))
    return 0;
  return attn_plan(cache->Hkv, cache->d, cache->block, batch, n_q, Hq, max_blocks, true, false,
                   in_dt == MSA_BF16)
      .total;
}

msa_status msa_cache_attn_select(const msa_kv_cache* cache, const void* q, const int32_t* table,
                                 int max_blocks, const int32_t* lens, int batch, int n_q, int Hq,
                                 int64_t window, const int32_t* sel, const int32_t* cnt,
                                 int top_k, float scale, void* out, float* lse, msa_dtype in_dt,
                                 msa_dtype out_dt, void* workspace, size_t workspace_bytes,
                                 msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_query_sizes(cache, batch, n_q, Hq, max_blocks));
  MSA_TRY(check_query(q, out, lse, window, scale, in_dt, out_dt));
  if (!sel || !cnt || !aligned(sel, 4) || !aligned(cnt, 4))
    return fail(MSA_ERR_INVALID_ARG, "sel or cnt null or not 4-byte aligned");
  MSA_TRY(check_top_k(top_k, max_blocks));
  const AttnPlan p = attn_plan(cache->Hkv, cache->d, cache->block, batch, n_q, Hq, max_blocks,
                               true, false, in_dt == MSA_BF16);
  MSA_TRY(check_workspace(workspace, workspace_bytes, p.total));
  return run_attn(cache, q, table, max_blocks, lens, batch, n_q, Hq, window, scale, out, lse, sel,
                  cnt, top_k, false, nullptr, 0, in_dt, out_dt, static_cast<uint8_t*>(workspace), stream);
}

// Workspace of the one-call form: the attention's, the selection's, sel, cnt.
struct TopkPlan {
  size_t select, sel, cnt, total;
};
static TopkPlan topk_plan(const msa_kv_cache* c, int max_blocks, int batch, int n_q, int Hq,
                          int top_k, msa_dtype in_dt) {
  TopkPlan p{};
  const size_t units = static_cast<size_t>(batch) * n_q * c->Hkv;
  p.select = attn_plan(c->Hkv, c->d, c->block, batch, n_q, Hq, max_blocks, true, false,
                       in_dt == MSA_BF16)
                 .total;
  p.sel = p.select + select_plan(c->Hkv, batch, n_q, max_blocks).total;
  p.cnt = p.sel + up(units * top_k * sizeof(int32_t));
  p.total = p.cnt + up(units * sizeof(int32_t));
  return p;
}

size_t msa_cache_attn_topk_workspace_size(const msa_kv_cache* cache, int max_blocks, int batch,
                                          int n_q, int Hq, int top_k, msa_dtype in_dt) {
  if (!cache ||
      check_sizes(cache->n_pages, cache->Hkv, cache->d, cache->block, batch, max_blocks) != MSA_OK ||
      check_query_sizes(cache, batch, n_q, Hq, max_blocks) != MSA_OK || !valid_dtype(in_dt) ||
      check_top_k(top_k, max_blocks) != MSA_OK)
    return 0;
  return topk_plan(cache, max_blocks, batch, n_q, Hq, top_k, in_dt).total;
}

msa_status msa_cache_attn_topk(const msa_kv_cache* cache, const void* q, const int32_t* table,
                               int max_blocks, const int32_t* lens, int batch, int n_q, int Hq,
                               int64_t window, int top_k, float scale, void* out, float* lse,
                               msa_dtype in_dt, msa_dtype out_dt, void* workspace,
                               size_t workspace_bytes, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_query_sizes(cache, batch, n_q, Hq, max_blocks));
  MSA_TRY(check_query(q, out, lse, window, scale, in_dt, out_dt));
  MSA_TRY(check_top_k(top_k, max_blocks));
  const TopkPlan p = topk_plan(cache, max_blocks, batch, n_q, Hq, top_k, in_dt);
  MSA_TRY(check_workspace(workspace, workspace_bytes, p.total));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* sel = reinterpret_cast<int32_t*>(ws + p.sel);
  int32_t* cnt = reinterpret_cast<int32_t*>(ws + p.cnt);
  MSA_TRY(run_select(cache, q, table, max_blocks, lens, batch, n_q, Hq, window, top_k, sel, cnt,
                     in_dt, ws + p.select, stream));
  return run_attn(cache, q, table, max_blocks, lens, batch, n_q, Hq, window, scale, out, lse, sel,
                  cnt, top_k, true, nullptr, 0, in_dt, out_dt, ws, stream);
}

msa_status msa_cache_evict(const msa_kv_cache* cache, const int32_t* table, int max_blocks,
                           const int32_t* lens, int batch, const float* weights,
                           int64_t weights_ld, int64_t budget, int64_t recent,
                           const int32_t* dst_table, int dst_blocks, int32_t* new_lens,
                           int32_t* kept, float* new_weights, int64_t new_weights_ld,
                           msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  if (!weights || !dst_table || !new_lens || !kept || !new_weights)
    return fail(MSA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(weights, 4) || !aligned(dst_table, 4) || !aligned(new_lens, 4) ||
      !aligned(kept, 4) || !aligned(new_weights, 4))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointer not 4-byte aligned");
  if (weights_ld < static_cast<int64_t>(max_blocks) * cache->block)
    return fail(MSA_ERR_INVALID_ARG, "weights_ld=%lld below max_blocks * block",
                (long long)weights_ld);
  if (dst_blocks < 1 || static_cast<int64_t>(dst_blocks) * cache->block > kMaxSlots)
    return fail(MSA_ERR_INVALID_ARG, "dst_blocks=%d out of range", dst_blocks);
  if (budget < 1 || budget > static_cast<int64_t>(dst_blocks) * cache->block)
    return fail(MSA_ERR_INVALID_ARG, "budget=%lld must be in 1 .. dst_blocks * block",
                (long long)budget);
  if (recent < 0 || recent > budget)
    return fail(MSA_ERR_INVALID_ARG, "recent=%lld must be in 0 .. budget=%lld", (long long)recent,
                (long long)budget);
  if (new_weights_ld < budget || new_weights_ld > kMaxSlots)
    return fail(MSA_ERR_INVALID_ARG, "new_weights_ld=%lld below budget or too large",
                (long long)new_weights_ld);
  if (new_lens == lens || new_weights == weights)
    return fail(MSA_ERR_INVALID_ARG, "outputs must not be the inputs");
  const int64_t blocks = (budget + cache->block - 1) / cache->block;
  if (static_cast<int64_t>(batch) * cache->Hkv * 8 > INT32_MAX ||
      blocks * cache->Hkv > INT32_MAX)
    return fail(MSA_ERR_UNSUPPORTED, "batch, Hkv or budget too large for one call");
  msa::EvictArgs a{};
  a.c = view(cache);
  a.s = {table, max_blocks, lens, batch};
  a.weights = weights;
  a.weights_ld = weights_ld;
  a.budget = budget;
  a.recent = recent;
  a.new_lens = new_lens;
  a.kept = kept;
  a.new_weights = new_weights;
  a.new_ld = new_weights_ld;
  MSA_TRY(msa::api_status_word(&a.status));
  MSA_TRY(launched(msa::launch_cache_evict_select(a, reinterpret_cast<cudaStream_t>(stream)),
                   "cache eviction"));
  msa::GatherArgs g{};
  g.c = a.c;
  g.s = a.s;
  g.dst_table = dst_table;
  g.dst_blocks = dst_blocks;
  g.kept = kept;
  g.budget = budget;
  g.status = a.status;
  return launched(msa::launch_cache_gather(g, reinterpret_cast<cudaStream_t>(stream)),
                  "cache gather");
}

}  // extern "C"
