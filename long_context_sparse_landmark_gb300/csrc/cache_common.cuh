// The 8-bit KV cache: what its kernels share.
//
// A page holds one block of `block` token slots of one sequence for every KV
// head: K and V codes (e4m3) [Hkv, block, d], one fp32 scale per (block, KV
// head) for K and one for V, and the mean key of the block in bf16 (the
// block's landmark, written when the block is full).  A slot stands for
// code * scale.  Scales are powers of two: e4m3 has the same relative
// precision at every scale, so nothing is lost against an arbitrary scale
// but up to one binade of range at the bottom; in return x / scale,
// code * scale and a change of scale are exact in fp32 (below e4m3's
// subnormal range excepted), and a block appended token by token ends with
// the codes of one written at once.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "msa_cache.h"
#include "msa_common.cuh"

namespace msa {

struct CacheView {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  __nv_bfloat16* k_mean;
  int64_t n_pages;
  int Hkv, d, block;
  int lb;  // log2 of block
};

// Batch of sequences in a cache: table [batch][max_blocks] page of each
// block, lens [batch].
struct CacheBatch {
  const int32_t* table;
  int max_blocks;
  const int32_t* lens;
  int batch;
};

constexpr int kSms = 152;  // of a GB300: grids of persistent kernels

// Keys a warp takes at a time; every block is a whole number of them.
constexpr int kChunkLog2 = 5;
constexpr int kChunk = 1 << kChunkLog2;

// Length of sequence b, clamped to what its table row can hold.
__device__ __forceinline__ int cache_len(const CacheBatch& s, int b, int block, int* status) {
  const int n = s.lens[b];
  const int most = s.max_blocks * block;  // fits: the entry points check
  if (n < 0 || n > most) {
    record_status(status, MSA_ERR_INVALID_ARG);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Page of block j of sequence b; -1 (and the status recorded) if the table
// names none that exists.
__device__ __forceinline__ int64_t cache_page(const CacheBatch& s, int b, int64_t j,
                                              int64_t n_pages, int* status) {
  if (!MSA_IN_RANGE(static_cast<int64_t>(b) * s.max_blocks + j, 1,
                    static_cast<int64_t>(s.batch) * s.max_blocks, status))
    return -1;
  const int64_t p = s.table[static_cast<int64_t>(b) * s.max_blocks + j];
  if (p < 0 || p >= n_pages) {
    record_status(status, MSA_ERR_INVALID_ARG);
    return -1;
  }
  return p;
}

// Two e4m3 codes (low 16 bits of w) to two halves: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t w) {
  const uint32_t h = e4m3x2_to_half2(w);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four codes of a word to floats.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float* f) {
  const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w));
  const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(w >> 16));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// Least e >= -126 with amax <= 448 * 2^e (amax finite, > 0): 448 is
// 1.75 * 2^8, so e is amax's exponent less 8, one more above 1.75.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2i(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A kernel of a chain starts while the one before it drains: what it does
// before this call must not depend on that kernel.  The wait ends when the
// kernel before has finished and its writes are visible, so every kernel of
// a chain makes it on every path, before it exits; without a kernel to wait
// for it returns at once.
__device__ __forceinline__ void wait_for_inputs() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets the next kernel of a chain start as soon as every CTA of this one has.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel; with `chained`, as the dependent of the kernel that the
// same call has just put on the stream (programmatic stream serialization).
template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                                cudaStream_t st, bool chained, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launchers of the cache kernels (return the launch's cudaError_t).
struct AppendArgs {
  CacheView c;
  CacheBatch s;
  const void* k;  // [total, Hkv, d]
  const void* v;
  const int32_t* cu;  // [batch + 1] rows of each sequence's new tokens
  int64_t total, max_new;
  uint32_t blocks;  // blocks that a range of max_new tokens can touch
  int bf16;
  int* status;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);

struct GatherArgs {
  CacheView c;
  CacheBatch s;
  const int32_t* dst_table;  // [batch][dst_blocks]
  int dst_blocks;
  const int32_t* kept;  // [batch][Hkv][budget] ascending slots, -1 past the last
  int64_t budget;
  int* status;
};
cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t st);

struct CacheAttnArgs {
  CacheView c;
  CacheBatch s;
  const void* q;  // [batch, T, Hq, d]
  int T, Hq;
  int window;
  float scale;
  void* out;   // [batch, T, Hq, d]
  float* lse;  // [batch, Hq, T]
  const int32_t* sel;  // [batch, T, Hkv, top_k], null: dense
  const int32_t* cnt;  // [batch, T, Hkv]
  int sel_from_kernel;  // sel was put on the stream just before, by the same call
  int top_k;
  float* weights;  // [batch, Hkv, weights_ld], null: none
  int64_t weights_ld;
  // workspace
  float* o_part;    // [2 * n_ctas][tile rows][d], in units of 2^(r + u)
  float4* part_stat;  // [2 * n_ctas][tile rows]: a score m (log2 units), sum of 2^(s - m), r, u
  float* scores;    // [batch, Hkv, max_blocks * block, rows padded to even] (log2 units)
  float2* row_stat;  // [batch, Hkv, rows padded to even]: m, 1 / sum of 2^(s - m)
  int n_ctas;
  int in_bf16, out_bf16;
  int* status;
};
// Query rows of one (sequence, KV head) that a CTA takes together.
int cache_attn_tile_rows(int rows, int in_bf16);
// CTAs that fill the device; the launch uses at most this many.
int cache_attn_max_ctas(int tile_rows, int in_bf16);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t st);

struct CacheSelectArgs {
  CacheView c;
  CacheBatch s;
  const void* q;
  int T, Hq;
  int window;
  int top_k;
  int32_t* sel;
  int32_t* cnt;
  float* score;   // [batch, T, Hkv, max_blocks]
  float* err;     // [batch, T, Hkv, max_blocks] bound of each score's rounding
  double* exact;  // [batch, T, Hkv, max_blocks] scores in 64 bits, where the order needs them
  int bf16;
  int* status;
};
cudaError_t launch_cache_select(const CacheSelectArgs& a, cudaStream_t st);

struct EvictArgs {
  CacheView c;
  CacheBatch s;
  const float* weights;  // [batch, Hkv, weights_ld]
  int64_t weights_ld;
  int64_t budget, recent;
  int32_t* new_lens;   // [batch]
  int32_t* kept;       // [batch, Hkv, budget]
  float* new_weights;  // [batch, Hkv, new_ld]
  int64_t new_ld;
  int* status;
};
cudaError_t launch_cache_evict_select(const EvictArgs& a, cudaStream_t st);

}  // namespace msa
