// The 4-bit KV cache (msa_cache4.h): what its kernels share.  Pages, block
// tables and lengths are the 8-bit cache's; a slot of one head is d / 2 bytes of
// e2m1 codes and d / 32 bytes of e8m0 scales for K, and as many for V.
#pragma once

#include "cache_common.cuh"
#include "msa_cache4.h"

namespace msa {

constexpr int kGroup4 = 32;  // values of one scale

// Largest magnitude a group may hold, as bits of a float: 1.75 * 2^127 =
// 7 * 2^125.  Its codes stand for at most 6 * 2^125, a finite float; rounded
// codes of what is above (up to 2 * 2^127) would not.
constexpr uint32_t kMost4 = 0x7f600000u;

// Exponent of a group's scale, its largest magnitude given as the bits of a
// float (<= kMost4): the least e >= -126 with amax <= 7 * 2^e, 7 = 1.75 * 2^2.
__device__ __forceinline__ int group_exponent4(uint32_t b) {
  const int e = static_cast<int>(b >> 23) - 127 - 2 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Two codes (a byte) to two halves, exactly; the low four bits' value first.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Eight values to a word of codes, rounded to the nearest, ties to even,
// magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t floats_to_e2m1x8(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// The value of a scale's byte.
__device__ __forceinline__ float e8m0_to_float(uint32_t x) {
  return __uint_as_float(x == 255 ? 0x7fc00000u : x == 0 ? 0x00400000u : x << 23);
}

// Rows of tokens and slots of a cache: sequence b's rows cu[b] .. cu[b+1]-1
// are its last slots.
struct RowsArgs {
  CacheBatch s;
  const int32_t* cu;
  int64_t total, most;  // rows of k and v, and most of one sequence
  int Hkv, d, block, lb;
  int64_t n_pages;
  int bf16;  // of k and v
  int* status;
};
struct Append4Args : RowsArgs {
  const void* k;
  const void* v;
  uint8_t *k_codes, *v_codes, *k_scale, *v_scale;
};
struct ReadArgs : RowsArgs {
  void* k;
  void* v;
  const uint8_t *k_codes, *v_codes;  // 4 or 8 bits
  const void *k_scale, *v_scale;     // bytes [.., d / 32], or floats of a block
};
cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t st);
// CTAs along x that most * Hkv rows take (the entry points check that they fit).
int64_t cache_rows_ctas(int64_t most, int Hkv, int d, bool bf16);
cudaError_t launch_cache_read(const ReadArgs& a, int bits, cudaStream_t st);

struct Cache4AttnArgs : CacheAttnArgs {  // its cache's scales are not looked at
  const uint8_t *k_exp, *v_exp;  // [n_pages, Hkv, block, d / 32]
  int tile;                      // query rows that a CTA takes together
  bool pairs;                    // a warp two chunks (8 bf16 rows)
};
// slots: the most that a sequence's rows attend.
int cache4_attn_tile_rows(int rows, int64_t slots, int in_bf16);
// chunks: the most of all units.
bool cache4_attn_pairs(int64_t chunks, int max_ctas);
int cache4_attn_max_ctas(int tile_rows, int in_bf16);
cudaError_t launch_cache4_attn(const Cache4AttnArgs& a, cudaStream_t st);

}  // namespace msa
