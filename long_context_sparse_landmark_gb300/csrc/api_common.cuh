// What the C entry points of the caches and of the norms with rotation share:
// errors, argument checks, workspace rounding.
#pragma once

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "cache_common.cuh"

#include <nvtx3/nvToolsExt.h>

namespace msa {
// The error message, its reset and the device status word of msa_api.cu.
msa_status api_error(msa_status st, const char* message);
msa_status api_ok();
msa_status api_status_word(int** out);
}  // namespace msa

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
#define MSA_NVTX_RANGE() NvtxRange msa_nvtx_range_(__func__)

inline msa_status fail(msa_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return msa::api_error(st, buf);
}

inline msa_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(MSA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return msa::api_ok();
}

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
inline bool valid_dtype(msa_dtype d) { return d == MSA_F32 || d == MSA_BF16; }

constexpr int64_t kMaxSlots = (int64_t(1) << 31) - (1 << 16);
constexpr int kMaxBatch = 65535;  // a grid dimension
constexpr int kMaxHeads = 16384;
constexpr int kMaxRows = 4096;  // query rows of one sequence and KV head

inline msa_status check_sizes(int64_t n_pages, int Hkv, int d, int block, int batch,
                              int max_blocks) {
  if (n_pages < 1 || n_pages > INT32_MAX)
    return fail(MSA_ERR_INVALID_ARG, "n_pages=%lld out of range", (long long)n_pages);
  if (Hkv < 1 || Hkv > kMaxHeads)
    return fail(MSA_ERR_INVALID_ARG, "Hkv=%d out of range (1 .. %d)", Hkv, kMaxHeads);
  if (d != 64 && d != 128) return fail(MSA_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (block != 32 && block != 64 && block != 128 && block != 256)
    return fail(MSA_ERR_UNSUPPORTED, "block=%d (supported: 32, 64, 128, 256)", block);
  if (batch < 1 || batch > kMaxBatch)
    return fail(MSA_ERR_INVALID_ARG, "batch=%d out of range (1 .. %d)", batch, kMaxBatch);
  if (max_blocks < 1 || static_cast<int64_t>(max_blocks) * block > kMaxSlots)
    return fail(MSA_ERR_INVALID_ARG, "max_blocks=%d out of range", max_blocks);
  return MSA_OK;
}

inline msa_status check_cache(const msa_kv_cache* c, const int32_t* table, int max_blocks,
                              const int32_t* lens, int batch) {
  if (!c) return fail(MSA_ERR_INVALID_ARG, "null cache");
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->k_mean || !table || !lens)
    return fail(MSA_ERR_INVALID_ARG, "null cache, table or lens pointer");
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_mean, 16))
    return fail(MSA_ERR_INVALID_ARG, "cache pointer not 16-byte aligned");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(table, 4) ||
      !aligned(lens, 4))
    return fail(MSA_ERR_INVALID_ARG, "scale, table or lens pointer not 4-byte aligned");
  return check_sizes(c->n_pages, c->Hkv, c->d, c->block, batch, max_blocks);
}

template <class Cache>
msa_status check_query_sizes(const Cache* c, int batch, int n_q, int Hq, int max_blocks) {
  const int Hkv = c->Hkv, block = c->block;
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MSA_ERR_INVALID_ARG, "Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (n_q < 1) return fail(MSA_ERR_INVALID_ARG, "n_q=%d must be >= 1", n_q);
  const int64_t rows = static_cast<int64_t>(n_q) * (Hq / Hkv);
  if (rows > kMaxRows)
    return fail(MSA_ERR_UNSUPPORTED, "%lld query rows of a sequence and KV head (at most %d)",
                (long long)rows, kMaxRows);
  if (static_cast<int64_t>(batch) * n_q * Hq > INT32_MAX)
    return fail(MSA_ERR_UNSUPPORTED, "batch=%d n_q=%d Hq=%d: too many rows", batch, n_q, Hq);
  // Chunks of 32 slots of every 8 rows are counted in 32 bits.
  if (static_cast<int64_t>(batch) * n_q * Hkv * ((Hq / Hkv + 7) / 8) >
      INT32_MAX / (static_cast<int64_t>(max_blocks) * block / msa::kChunk + 1))
    return fail(MSA_ERR_UNSUPPORTED, "batch=%d n_q=%d Hq=%d max_blocks=%d: too much for one call",
                batch, n_q, Hq, max_blocks);
  return MSA_OK;
}

inline msa_status check_window(int64_t window) {
  if (window < 1) return fail(MSA_ERR_INVALID_ARG, "window=%lld must be >= 1", (long long)window);
  return MSA_OK;
}

inline msa_status check_query(const void* q, const void* out, const float* lse, int64_t window,
                              float scale, msa_dtype in_dt, msa_dtype out_dt) {
  if (!q || !out || !lse) return fail(MSA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointer not 16-byte aligned (lse: 4)");
  if (!(scale > 0.f) || !isfinite(scale))
    return fail(MSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!valid_dtype(in_dt)) return fail(MSA_ERR_INVALID_ARG, "bad input dtype %d", (int)in_dt);
  if (!valid_dtype(out_dt)) return fail(MSA_ERR_INVALID_ARG, "bad output dtype %d", (int)out_dt);
  return check_window(window);
}

inline msa_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return MSA_OK;
  if (!ws || !aligned(ws, 256))
    return fail(MSA_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (bytes < need)
    return fail(MSA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", bytes, need);
  return MSA_OK;
}

inline int log2_of(int block) { return block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : 8; }

inline size_t up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

#define MSA_TRY(x)                          \
  do {                                      \
    const msa_status msa_try_st_ = (x);     \
    if (msa_try_st_ != MSA_OK) return msa_try_st_; \
  } while (0)

