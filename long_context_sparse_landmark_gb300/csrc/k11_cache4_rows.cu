// K11: tokens' rows and cache slots -- writing the 4-bit KV cache, and reading
// it or the 8-bit one back.
//
// A row is the d values of one token and KV head; a thread takes 16 of them, so
// a row is 8 lanes (d = 128) or 4, and a group of 32 values 2 neighbouring
// lanes.  Writing: the group's largest magnitude m, its scale 2^e, the least
// with m <= 7 * 2^e, and codes of x * 2^-e, exact but for one rounding.
// Reading: code * 2^e, rounded once.  Both move every byte once, and HBM bounds
// them: 131072 tokens of 8 heads of 128 in bf16 (679 MB) are appended in about 100 us,
// 6.8 TB/s (DRAM 82 % of its peak, issue slots 59 %, integer pipe 58 %), and read
// back in 104.8, 6.5 TB/s (DRAM 76 %, issue slots 61 %).
// A thread has 128 bytes of rows under way, 4 rows in bf16 or 2 in fp32, K and V in
// CTAs of their own.  Append and then read of 131072 tokens in bf16: 2 rows 207 us, 8
// rows 237, 4 rows 202, 8 values a thread 238; of 8192 tokens 2 rows 14.7 us, 4 rows
// 13.8; fp32, 24 ragged prompts of up to 501 tokens, 4 heads of 64: 2 rows 9.0, 4 rows
// 10.7 (in CTAs of 256 threads 10.3 and 12.7; the same prompts over and over, which L2
// holds: new ones each time, in blocks of 32, take 11.3, and 13.4 with 4 rows and 256).
#include "cache4.cuh"

namespace msa {
namespace {

constexpr int kThreads = 128;
constexpr int kPer = 16;  // values a thread
__host__ __device__ constexpr int thread_rows(bool bf16) { return bf16 ? 4 : 2; }

// Rows (token, head) that a CTA takes.
constexpr int cta_rows(int d, bool bf16) { return kThreads / (d / kPer) * thread_rows(bf16); }

// The rows of a sequence, or none (and the status recorded) where the device
// data cannot be.
struct Span {
  int r0, n;   // first row, tokens
  int first;   // first token's slot
};
__device__ __forceinline__ bool span_of(const RowsArgs& a, int b, Span* s) {
  const int r0 = a.cu[b], r1 = a.cu[b + 1];
  const int len = cache_len(a.s, b, a.block, a.status);
  if (r0 == r1 || len != a.s.lens[b]) return false;
  if (r0 < 0 || r1 < r0 || r1 > a.total || r1 - r0 > a.most || r1 - r0 > len) {
    if (threadIdx.x == 0) record_status(a.status, MSA_ERR_INVALID_ARG);
    return false;
  }
  s->r0 = r0;
  s->n = r1 - r0;
  s->first = len - s->n;
  return true;
}

// This thread's rows: kRows of the CTA's, kStep apart, in the order of k and v.
constexpr uint32_t kNoSlot = 0xffffffffu;
template <int D, int kRows>
struct Rows {
  static constexpr int kLanes = D / kPer, kStep = kThreads / kLanes;
  static_assert(kRows <= kLanes, "a lane looks up one row");
  int64_t row0;          // first row of the CTA, of all rows of k and v
  int left;              // rows of the CTA
  uint32_t slot[kRows];  // row in the pool ([n_pages * Hkv * block], fewer than 2^32 - 1: the
                         // entry points check), kNoSlot: no such page

  __device__ __forceinline__ bool in(int i) const {
    return static_cast<int>(threadIdx.x) / kLanes + i * kStep < left;
  }
  // Offset of row i's values in k and v.
  __device__ __forceinline__ int64_t at(int i) const {
    return (row0 + threadIdx.x / kLanes + i * kStep) * D;
  }
  // The CTA's rows of the sequence; false: none.
  __device__ __forceinline__ bool find(const RowsArgs& a, const Span& s, uint32_t cta) {
    const int64_t from = static_cast<int64_t>(cta) * (kStep * kRows);
    const int64_t all = static_cast<int64_t>(s.n) * a.Hkv;
    row0 = static_cast<int64_t>(s.r0) * a.Hkv + from;
    left = static_cast<int>(min64(all - from, kStep * kRows));
    return all > from;
  }
  // Each lane of a row looks up one of its kRows rows for the others.
  __device__ __forceinline__ void look_up(const RowsArgs& a, int b, const Span& s, uint32_t cta) {
    const int lane = threadIdx.x & (kLanes - 1), i = lane % kRows;
    const int64_t from = static_cast<int64_t>(cta) * (kStep * kRows);
    // Most launches have fewer than 2^32 rows: one 32-bit division for the CTA.
    const int64_t t0 = from >> 32 ? from / a.Hkv
                                  : static_cast<uint32_t>(from) / static_cast<uint32_t>(a.Hkv);
    const uint32_t x = static_cast<uint32_t>(from - t0 * a.Hkv) + threadIdx.x / kLanes + i * kStep;
    const uint32_t up = x / static_cast<uint32_t>(a.Hkv);
    uint32_t mine = kNoSlot;
    if (in(i)) {
      const int at = s.first + static_cast<int>(t0) + static_cast<int>(up);
      const int64_t page = cache_page(a.s, b, at >> a.lb, a.n_pages, a.status);
      if (page >= 0)
        mine = (static_cast<uint32_t>(page * a.Hkv + (x - up * a.Hkv)) << a.lb) +
               (at & (a.block - 1));
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      slot[k] = __shfl_sync(0xffffffffu, mine, k, kLanes);
  }
};

// 16 values of a row, as they are in memory.
template <bool kBf16>
struct Raw;
template <>
struct Raw<true> {
  uint32_t w[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void* src, int64_t off) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + off);
    const uint4 x = __ldcs(p), y = __ldcs(p + 1);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
  // The largest magnitude, as bits of a float: two halves of a word at a time.
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      x = __vimax3_u16x2(x, w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu);
    return max(x << 16, x & 0xffff0000u);
  }
  // Codes of the values times inv, a power of two that leaves none above 7: exact
  // in fp32.  The products are mixed multiply-adds, which widen bf16 on the way:
  // the integer pipe, where widening and the conversions to codes run at half
  // rate, bounds the append.
  __device__ __forceinline__ uint2 encode(float inv) const {
    const uint16_t f = static_cast<uint16_t>(__float_as_uint(inv) >> 16);
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
          "fma.rn.f32.bf16 %0, l, %3, %4;\n\tfma.rn.f32.bf16 %1, h, %3, %4;\n\t}"
          : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
          : "r"(w[i]), "h"(f), "f"(-0.f));
    return make_uint2(floats_to_e2m1x8(v), floats_to_e2m1x8(v + 8));
  }
};
template <>
struct Raw<false> {
  float v[16];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void load(const void* src, int64_t off) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = __ldcs(p + i);
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      m = __vimax3_u32(m, __float_as_uint(v[i]) & 0x7fffffffu,
                       __float_as_uint(v[i + 1]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ uint2 encode(float inv) const {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = v[i] * inv;
    return make_uint2(floats_to_e2m1x8(y), floats_to_e2m1x8(y + 8));
  }
};

// blockIdx.x = (rows, K or V), blockIdx.y = sequence.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) cache4_append_kernel(const Append4Args a) {
  constexpr int kLanes = D / kPer;
  const int b = blockIdx.y, kv = blockIdx.x & 1;
  Span s;
  if (!span_of(a, b, &s)) return;
  constexpr int kRows = thread_rows(kBf16);
  Rows<D, kRows> rows;
  if (!rows.find(a, s, blockIdx.x >> 1)) return;
  const int lane = threadIdx.x & (kLanes - 1);
  const void* src = kv ? a.v : a.k;
  Raw<kBf16> v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t off = rows.at(i) + lane * kPer;
    if (rows.in(i) && MSA_IN_RANGE(off, kPer, a.total * a.Hkv * D, a.status))
      v[i].load(src, off);
    else
      v[i].clear();
  }
  rows.look_up(a, b, s, blockIdx.x >> 1);
  uint8_t* codes = kv ? a.v_codes : a.k_codes;
  uint8_t* scale = kv ? a.v_scale : a.k_scale;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t m = v[i].max_bits();
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    // A group of the warp holds zeros only, or what no code stands for.
    bool poisoned = false;
    if (__any_sync(0xffffffffu, m - 1u >= kMost4)) {
      uint32_t most = m;
#pragma unroll
      for (int o = 2; o < kLanes; o <<= 1)
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      poisoned = most > kMost4;
      if (m == 0) m = most;
    }
    const int e = poisoned ? 0 : group_exponent4(m);
    uint2 w = v[i].encode(pow2i(-e));
    if (poisoned) w = make_uint2(0, 0);
    const int64_t at = rows.slot[i];
    if (rows.slot[i] == kNoSlot ||
        !MSA_IN_RANGE(at, 1, a.n_pages * a.Hkv << a.lb, a.status))
      continue;
    *reinterpret_cast<uint2*>(codes + at * (D / 2) + lane * (kPer / 2)) = w;
    if ((lane & 1) == 0)
      scale[at * (D / kGroup4) + (lane >> 1)] =
          static_cast<uint8_t>(poisoned ? 255 : e + 127);
  }
}

// blockIdx.x = (rows, K or V), blockIdx.y = sequence.  A thread's 16 values are runs
// of 16 bytes of output, so that a row's lanes write whole lines side by side (as one
// run of 32 bytes a lane, every store left half sectors: 130 us for 128K tokens of 8
// heads of 128, now 104).
template <int D, int kBits, bool kBf16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
  constexpr int kLanes = D / kPer;
  constexpr int kRun = kBf16 ? 8 : 4, kRuns = kPer / kRun;  // values of a run
  constexpr int kRunBytes = kRun * kBits / 8;               // of codes: 2, 4 or 8
  const int b = blockIdx.y, kv = blockIdx.x & 1;
  Span s;
  if (!span_of(a, b, &s)) return;
  constexpr int kRows = thread_rows(kBf16);
  Rows<D, kRows> rows;
  if (!rows.find(a, s, blockIdx.x >> 1)) return;
  rows.look_up(a, b, s, blockIdx.x >> 1);
  const int lane = threadIdx.x & (kLanes - 1);
  const uint8_t* codes = kv ? a.v_codes : a.k_codes;
  const void* scale = kv ? a.v_scale : a.k_scale;
  uint2 w[kRows][kRuns];
  uint32_t f[kRows][kBits == 4 ? kRuns : 1];  // bytes, or a float
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t at = rows.slot[i];
    const bool on = rows.slot[i] != kNoSlot && MSA_IN_RANGE(at, 1, a.n_pages * a.Hkv << a.lb, a.status);
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int v = r * (D / kRuns) + lane * kRun;  // first value
      w[i][r] = make_uint2(0, 0);
      if constexpr (kBits == 4) {
        f[i][r] = 127;
        const uint8_t* p = codes + at * (D / 2) + v / 2;
        if (on) {
          w[i][r].x = kRunBytes == 4 ? __ldcs(reinterpret_cast<const uint32_t*>(p))
                                     : __ldcs(reinterpret_cast<const uint16_t*>(p));
          f[i][r] = static_cast<const uint8_t*>(scale)[at * (D / kGroup4) + v / kGroup4];
        }
      } else {
        const uint8_t* p = codes + at * D + v;
        if (on && kRunBytes == 8) w[i][r] = __ldcs(reinterpret_cast<const uint2*>(p));
        if (on && kRunBytes == 4) w[i][r].x = __ldcs(reinterpret_cast<const uint32_t*>(p));
      }
    }
    if constexpr (kBits == 8)
      f[i][0] = on ? __float_as_uint(static_cast<const float*>(scale)[at >> a.lb]) : 0;
  }
  void* dst = kv ? a.v : a.k;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!rows.in(i)) continue;
    const int64_t row = rows.at(i);
    if (!MSA_IN_RANGE(row, D, a.total * a.Hkv * D, a.status)) continue;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      float v[8];
      if constexpr (kBits == 4) {
        uint32_t h[4];
        e2m1x8_to_half2(w[i][r].x, h);
#pragma unroll
        for (int k = 0; k < kRun / 2; ++k) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
          v[2 * k] = x.x;
          v[2 * k + 1] = x.y;
        }
      } else {
        e4m3x4_to_float(w[i][r].x, v);
        if (kRun == 8) e4m3x4_to_float(w[i][r].y, v + 4);
      }
      const float g = kBits == 4 ? e8m0_to_float(f[i][kBits == 4 ? r : 0]) : __uint_as_float(f[i][0]);
#pragma unroll
      for (int k = 0; k < kRun; ++k) v[k] *= g;
      const int64_t off = row + r * (D / kRuns) + lane * kRun;
      if constexpr (kBf16) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
          o[k] = *reinterpret_cast<const uint32_t*>(&x);
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off),
               make_uint4(o[0], o[1], o[2], o[3]));
      } else {
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(dst) + off),
               make_float4(v[0], v[1], v[2], v[3]));
      }
    }
  }
}

}  // namespace

int64_t cache_rows_ctas(int64_t most, int Hkv, int d, bool bf16) {
  const int rows = cta_rows(d, bf16);
  return (most * Hkv + rows - 1) / rows * 2;
}

cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(cache_rows_ctas(a.most, a.Hkv, a.d, a.bf16)), a.s.batch);
  const auto kernel = a.d == 128 ? (a.bf16 ? cache4_append_kernel<128, true>
                                           : cache4_append_kernel<128, false>)
                                 : (a.bf16 ? cache4_append_kernel<64, true>
                                           : cache4_append_kernel<64, false>);
  return launch_after(kernel, grid, kThreads, 0, st, false, a);
}

cudaError_t launch_cache_read(const ReadArgs& a, int bits, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(cache_rows_ctas(a.most, a.Hkv, a.d, a.bf16)), a.s.batch);
  void (*kernel)(ReadArgs);
  if (bits == 4)
    kernel = a.d == 128 ? (a.bf16 ? cache_read_kernel<128, 4, true> : cache_read_kernel<128, 4, false>)
                        : (a.bf16 ? cache_read_kernel<64, 4, true> : cache_read_kernel<64, 4, false>);
  else
    kernel = a.d == 128 ? (a.bf16 ? cache_read_kernel<128, 8, true> : cache_read_kernel<128, 8, false>)
                        : (a.bf16 ? cache_read_kernel<64, 8, true> : cache_read_kernel<64, 8, false>);
  return launch_after(kernel, grid, kThreads, 0, st, false, a);
}

}  // namespace msa
