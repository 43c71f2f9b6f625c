// C ABI of the 4-bit KV cache and of reading either cache back (msa_cache4.h):
// argument validation, workspace layout and launch.  Everything is checked
// before anything is enqueued, and nothing allocates or synchronises.
#include "api_common.cuh"
#include "cache4.cuh"

namespace {

// Slots of a pool and head are counted in 32 bits.
template <class Cache>
msa_status check_pool(const Cache* c) {
  if (c->n_pages * c->Hkv * c->block >= int64_t(UINT32_MAX))
    return fail(MSA_ERR_UNSUPPORTED, "n_pages=%lld Hkv=%d block=%d: too large a pool",
                (long long)c->n_pages, c->Hkv, c->block);
  return MSA_OK;
}

msa_status check_cache4(const msa_kv_cache4* c, const int32_t* table, int max_blocks,
                        const int32_t* lens, int batch) {
  if (!c) return fail(MSA_ERR_INVALID_ARG, "null cache");
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !table || !lens)
    return fail(MSA_ERR_INVALID_ARG, "null cache, table or lens pointer");
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return fail(MSA_ERR_INVALID_ARG, "cache pointer not 16-byte aligned");
  if (!aligned(table, 4) || !aligned(lens, 4))
    return fail(MSA_ERR_INVALID_ARG, "table or lens pointer not 4-byte aligned");
  const msa_status st = check_sizes(c->n_pages, c->Hkv, c->d, c->block, batch, max_blocks);
  return st != MSA_OK ? st : check_pool(c);
}

// The rows of k and v that an append takes or a read writes.
msa_status check_rows(const int32_t* cu, int64_t total, int64_t most, const void* k, const void* v,
                      msa_dtype dt, int Hkv, int d) {
  if (!cu || !aligned(cu, 4)) return fail(MSA_ERR_INVALID_ARG, "cu null or not 4-byte aligned");
  if (total < 0 || total > INT32_MAX || most < 0 || most > total)
    return fail(MSA_ERR_INVALID_ARG, "total=%lld most=%lld (0 <= most <= total)", (long long)total,
                (long long)most);
  if (!valid_dtype(dt)) return fail(MSA_ERR_INVALID_ARG, "bad dtype %d", (int)dt);
  if (most == 0) return MSA_OK;
  if (!k || !v) return fail(MSA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(k, 16) || !aligned(v, 16))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointer not 16-byte aligned");
  if (msa::cache_rows_ctas(most, Hkv, d, dt == MSA_BF16) > INT32_MAX)
    return fail(MSA_ERR_UNSUPPORTED, "%lld rows: too many for one call", (long long)most);
  return MSA_OK;
}

template <class Cache>
msa_status rows_args(msa::RowsArgs* a, const Cache* c, const int32_t* cu, int64_t total,
                     int64_t most, const int32_t* table, int max_blocks, const int32_t* lens,
                     int batch, msa_dtype dt) {
  a->s = {table, max_blocks, lens, batch};
  a->cu = cu;
  a->total = total;
  a->most = most;
  a->Hkv = c->Hkv;
  a->d = c->d;
  a->block = c->block;
  a->lb = log2_of(c->block);
  a->n_pages = c->n_pages;
  a->bf16 = dt == MSA_BF16;
  return msa::api_status_word(&a->status);
}

template <class Cache>
msa_status run_read(const Cache* c, int bits, const int32_t* cu, int64_t total, int64_t most,
                    const int32_t* table, int max_blocks, const int32_t* lens, int batch, void* k,
                    void* v, msa_dtype dt, msa_stream_t stream) {
  msa_status st = check_rows(cu, total, most, k, v, dt, c->Hkv, c->d);
  if (st != MSA_OK) return st;
  if (most == 0) return msa::api_ok();
  msa::ReadArgs a{};
  st = rows_args(&a, c, cu, total, most, table, max_blocks, lens, batch, dt);
  if (st != MSA_OK) return st;
  a.k = k;
  a.v = v;
  a.k_codes = static_cast<const uint8_t*>(c->k_codes);
  a.v_codes = static_cast<const uint8_t*>(c->v_codes);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  return launched(msa::launch_cache_read(a, bits, reinterpret_cast<cudaStream_t>(stream)),
                  "cache read");
}

// Attention workspace: the parts of the units that several CTAs share.
struct AttnPlan4 {
  int n_ctas, tile;
  bool pairs;
  size_t part_stat, total;
};

// slots: the most that a sequence's rows attend.
AttnPlan4 attn_plan4(const msa_kv_cache4* c, int batch, int n_q, int Hq, int max_blocks, int tile,
                     int64_t slots, int in_bf16) {
  const int rows = n_q * (Hq / c->Hkv);
  const int64_t units = static_cast<int64_t>(batch) * c->Hkv * ((rows + tile - 1) / tile);
  const int64_t chunks = units * (static_cast<int64_t>(max_blocks) * c->block / msa::kChunk);
  AttnPlan4 p{};
  p.tile = tile;
  const int most = msa::cache4_attn_max_ctas(tile, in_bf16);
  p.n_ctas = static_cast<int>(
      msa::max64(1, msa::min64(most, msa::max64(units, (chunks + 3) / 4))));
  p.pairs = msa::cache4_attn_pairs(units * (slots / msa::kChunk), most);
  p.part_stat = up(static_cast<size_t>(2) * p.n_ctas * tile * c->d * sizeof(float));
  p.total = p.part_stat + up(static_cast<size_t>(2) * p.n_ctas * tile * sizeof(float4));
  return p;
}
AttnPlan4 attn_plan4(const msa_kv_cache4* c, int batch, int n_q, int Hq, int max_blocks,
                     int64_t window, int in_bf16) {
  const int64_t slots = msa::min64(window < kMaxSlots ? window + n_q : kMaxSlots,
                                   static_cast<int64_t>(max_blocks) * c->block);
  return attn_plan4(c, batch, n_q, Hq, max_blocks,
                    msa::cache4_attn_tile_rows(n_q * (Hq / c->Hkv), slots, in_bf16), slots,
                    in_bf16);
}

}  // namespace

extern "C" {

msa_status msa_cache4_append(const msa_kv_cache4* cache, const void* k, const void* v,
                             const int32_t* cu, int64_t total, int64_t max_new,
                             const int32_t* table, int max_blocks, const int32_t* lens, int batch,
                             msa_dtype in_dt, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache4(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_rows(cu, total, max_new, k, v, in_dt, cache->Hkv, cache->d));
  if (max_new == 0) return msa::api_ok();
  msa::Append4Args a{};
  MSA_TRY(rows_args(&a, cache, cu, total, max_new, table, max_blocks, lens, batch, in_dt));
  a.k = k;
  a.v = v;
  a.k_codes = static_cast<uint8_t*>(cache->k_codes);
  a.v_codes = static_cast<uint8_t*>(cache->v_codes);
  a.k_scale = static_cast<uint8_t*>(cache->k_scale);
  a.v_scale = static_cast<uint8_t*>(cache->v_scale);
  return launched(msa::launch_cache4_append(a, reinterpret_cast<cudaStream_t>(stream)),
                  "cache append");
}

size_t msa_cache4_attn_workspace_size(const msa_kv_cache4* cache, int max_blocks, int batch,
                                      int n_q, int Hq, msa_dtype in_dt) {
  if (!cache ||
      check_sizes(cache->n_pages, cache->Hkv, cache->d, cache->block, batch, max_blocks) != MSA_OK ||
      check_pool(cache) != MSA_OK ||
      check_query_sizes(cache, batch, n_q, Hq, max_blocks) != MSA_OK || !valid_dtype(in_dt))
    return 0;
  // Whatever the window: its tiles are those of one slot, or of all.
  const size_t few = attn_plan4(cache, batch, n_q, Hq, max_blocks, int64_t(1), in_dt == MSA_BF16).total;
  const size_t all = attn_plan4(cache, batch, n_q, Hq, max_blocks, kMaxSlots, in_dt == MSA_BF16).total;
  return few > all ? few : all;
}

msa_status msa_cache4_attn(const msa_kv_cache4* cache, const void* q, const int32_t* table,
                           int max_blocks, const int32_t* lens, int batch, int n_q, int Hq,
                           int64_t window, float scale, void* out, float* lse, msa_dtype in_dt,
                           msa_dtype out_dt, void* workspace, size_t workspace_bytes,
                           msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache4(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_query_sizes(cache, batch, n_q, Hq, max_blocks));
  MSA_TRY(check_query(q, out, lse, window, scale, in_dt, out_dt));
  const AttnPlan4 p = attn_plan4(cache, batch, n_q, Hq, max_blocks, window, in_dt == MSA_BF16);
  MSA_TRY(check_workspace(workspace, workspace_bytes, p.total));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  msa::Cache4AttnArgs a{};
  a.c = {static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->v_codes), nullptr,
         nullptr, nullptr, cache->n_pages, cache->Hkv, cache->d, cache->block,
         log2_of(cache->block)};
  a.s = {table, max_blocks, lens, batch};
  a.q = q;
  a.T = n_q;
  a.Hq = Hq;
  a.window = static_cast<int>(msa::min64(window, static_cast<int64_t>(max_blocks) * cache->block));
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.o_part = reinterpret_cast<float*>(ws);
  a.part_stat = reinterpret_cast<float4*>(ws + p.part_stat);
  a.n_ctas = p.n_ctas;
  a.tile = p.tile;
  a.pairs = p.pairs;
  a.in_bf16 = in_dt == MSA_BF16;
  a.out_bf16 = out_dt == MSA_BF16;
  a.k_exp = static_cast<const uint8_t*>(cache->k_scale);
  a.v_exp = static_cast<const uint8_t*>(cache->v_scale);
  MSA_TRY(msa::api_status_word(&a.status));
  return launched(msa::launch_cache4_attn(a, reinterpret_cast<cudaStream_t>(stream)),
                  "cache attention");
}

msa_status msa_cache_read(const msa_kv_cache* cache, const int32_t* cu, int64_t total,
                          int64_t max_rows, const int32_t* table, int max_blocks,
                          const int32_t* lens, int batch, void* k, void* v, msa_dtype out_dt,
                          msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache(cache, table, max_blocks, lens, batch));
  MSA_TRY(check_pool(cache));
  return run_read(cache, 8, cu, total, max_rows, table, max_blocks, lens, batch, k, v, out_dt,
                  stream);
}

msa_status msa_cache4_read(const msa_kv_cache4* cache, const int32_t* cu, int64_t total,
                           int64_t max_rows, const int32_t* table, int max_blocks,
                           const int32_t* lens, int batch, void* k, void* v, msa_dtype out_dt,
                           msa_stream_t stream) {
  MSA_NVTX_RANGE();
  MSA_TRY(check_cache4(cache, table, max_blocks, lens, batch));
  return run_read(cache, 4, cu, total, max_rows, table, max_blocks, lens, batch, k, v, out_dt,
                  stream);
}

}  // extern "C"
