// K7: writing the 8-bit KV cache -- appending new tokens, and gathering kept
// tokens into fresh blocks after an eviction.
//
// Both write whole (block, KV head) pairs: a CTA takes the values of one block
// of one head, finds their largest magnitude, forms the power-of-two scale
// (cache_common.cuh), and stores the codes.  Every thread keeps its values in
// registers (64 of them: 4 rows of 16 columns), all their loads under way at
// once, so the data is read once and written once.  HBM bounds a long append:
// 128K tokens of 8 heads of 128 (bf16) in 128 us, 6.3 TB/s, 93 % of a measured
// copy; with 32 values a thread the instructions did (182 us), and a loop over
// tasks with copies under way in shared memory, one barrier a task, took 296.
// The gather is bound by its chain of lookups and by some 900 instructions a
// thread: 2273 to 4096 slots of each of 64 (sequence, head) pairs, 51 MB read and
// as much written, in 24 us.
#include "cache_common.cuh"

namespace msa {
namespace {

constexpr int kVec = 16;  // values of one 16-byte code store

constexpr int kRows = 4;  // groups of 16 values a thread has, block / 4 rows apart

__host__ __device__ inline int write_threads(int block, int d) {
  return block * d / (kRows * kVec);  // 32 .. 512
}

// Largest of the CTA's magnitudes, as the bits of non-negative floats (which
// order as unsigned integers; a NaN or infinity is 0x7f800000 and above).
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* smem) {
  x = __reduce_max_sync(0xffffffffu, x);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) smem[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < nw ? smem[lane] : 0u);
}

constexpr uint32_t kNanBits = 0x7fc00000u;

// Scale of a block whose largest magnitude has these bits: 0 for a block of
// zeros, NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ float scale_for(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(kNanBits);
  return amax ? pow2i(block_exponent(__uint_as_float(amax))) : 0.f;
}
// 1 / scale (0 for a scale of 0 or NaN: codes of 0).  Exponents end at 120.
__device__ __forceinline__ float inverse(float s) {
  return s > 0.f ? pow2i(127 - static_cast<int>(__float_as_uint(s) >> 23)) : 0.f;
}

// Two values times inv (a power of two: exact), rounded once to codes.
__device__ __forceinline__ uint32_t encode2(float x, float y, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x * inv, y * inv), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t encode4(float x, float y, float z, float w, float inv) {
  return encode2(x, y, inv) | encode2(z, w, inv) << 16;
}

// 16 input values of a thread as they are in memory.
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
  // The larger of m and the magnitudes' bits: two 16-bit halves at a time.
  __device__ __forceinline__ uint32_t max_bits(uint32_t m) const {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      x = __vimax3_u16x2(x, w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu);
    return max(m, max(x << 16, x & 0xffff0000u));
  }
  __device__ __forceinline__ uint4 encode(float inv) const {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = encode4(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i] & 0xffff0000u),
                     __uint_as_float(w[2 * i + 1] << 16),
                     __uint_as_float(w[2 * i + 1] & 0xffff0000u), inv);
    return make_uint4(c[0], c[1], c[2], c[3]);
  }
};
template <>
struct Raw<false> {
  float v[kVec];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void load(const void* src, int64_t off) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = __ldcs(p + i);
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
  __device__ __forceinline__ uint32_t max_bits(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < kVec; i += 2)
      m = __vimax3_u32(m, __float_as_uint(v[i]) & 0x7fffffffu,
                       __float_as_uint(v[i + 1]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ uint4 encode(float inv) const {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = encode4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
    return make_uint4(c[0], c[1], c[2], c[3]);
  }
};

// Codes of scale s rounded again to the scale 1 / inv, in halves: code * 2^-k
// is exact in them down to 2^-24, and what is smaller than that is far below
// the 2^-10 at which e4m3 rounds to its least value.  The new scale is the
// smaller one, by up to 2^17, where the slots kept of a block are all tiny: a
// factor that halves do not hold is applied in two steps, each exact.  Slots of
// zeros say nothing of the new scale: there the factor may be anything, and is
// bounded, since 0 times an infinity is none.
__device__ __forceinline__ uint4 rescale(const uint4& x, float s, float inv) {
  float by = fminf(s * inv, 0x1p17f);
  const bool twice = by > 32768.f;
  if (twice) by *= 1.f / 256.f;
  const __half2 f = __float2half2_rn(by);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = e4m3x2_to_half2(static_cast<uint16_t>(w[i]));
    const uint32_t b = e4m3x2_to_half2(static_cast<uint16_t>(w[i] >> 16));
    __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
    __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&b), f);
    if (twice) {
      y = __hmul2(y, __float2half2_rn(256.f));
      z = __hmul2(z, __float2half2_rn(256.f));
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
        : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t*>(&z)));
    c[i] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// Mean key of a full block from its codes, rounded to bf16 once.  Codes are
// whole multiples of 2^-9, so a lane's sums are exact in fp32 (up to 32 rows:
// 32 * 448 * 512 < 2^24) and a column's in 32-bit integers (256 * 448 * 512 <
// 2^26); the conversion to fp32 keeps a sticky bit, and the scaling by 2^e /
// block (a power of two) is exact.
__device__ __forceinline__ void column_sums(const uint4& c, float* part) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    e4m3x4_to_float(w[i], f);
#pragma unroll
    for (int k = 0; k < 4; ++k) part[4 * i + k] += f[k];
  }
}
__device__ __forceinline__ __nv_bfloat16 mean_of(int sum, float scale, int block) {
  float f = __int2float_rz(sum);
  if (static_cast<int>(f) != sum) f = __uint_as_float(__float_as_uint(f) | 1u);
  return __float2bfloat16_rn(f * (1.f / (512.f * static_cast<float>(block))) * scale);
}

// Adds the thread's 16 column sums to sums[d] (integers: any order gives the
// same result).  Lanes of the same columns are d/16 apart; after the joins a
// lane of each column group has its 2 * 512 / d rows' sums.
__device__ __forceinline__ void add_columns(float* part, int* sums, int col, int d) {
  for (int o = 16; o >= d / kVec; o >>= 1) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[i] += __shfl_xor_sync(0xffffffffu, part[i], o);
  }
  if ((threadIdx.x & 31) < d / kVec) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      atomicAdd(&sums[col * kVec + i], static_cast<int>(part[i] * 512.f));
  }
}
__device__ __forceinline__ void store_mean(const CacheView& c, int64_t head, const int* sums,
                                           float s) {
  for (int e = threadIdx.x; e < c.d; e += blockDim.x)
    c.k_mean[head * c.d + e] =
        isnan(s) ? __float2bfloat16_rn(s) : mean_of(sums[e], s, c.block);
}

// blockIdx.x = (block of the new range, head, K or V), blockIdx.y = sequence.
template <bool kBf16, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 512 ? 1 : kBf16 ? 8 : 4)
    cache_append_kernel(const AppendArgs a) {
  __shared__ uint32_t red[32];
  __shared__ int sums[128];
  const int d = a.c.d, block = a.c.block, lb = a.c.lb, Hkv = a.c.Hkv;
  const int b = blockIdx.y;
  const int kv = blockIdx.x & 1;
  const int jh = blockIdx.x >> 1;
  const int jj = jh / Hkv, h = jh - jj * Hkv;
  const int r0 = a.cu[b], r1 = a.cu[b + 1];
  const int len = cache_len(a.s, b, block, a.status);
  if (r0 == r1 || len != a.s.lens[b]) return;  // nothing new, or a length that cannot be
  if (r0 < 0 || r1 < r0 || r1 > a.total || r1 - r0 > a.max_new || r1 - r0 > len) {
    if (threadIdx.x == 0) record_status(a.status, MSA_ERR_INVALID_ARG);
    return;
  }
  const int first = len - (r1 - r0);  // slot of the first new token
  const int j = (first >> lb) + jj;
  if (j > (len - 1) >> lb) return;

  const int slot0 = j << lb;
  const int old = max(0, first - slot0);    // slots held before
  const int end = min(block, len - slot0);  // slots held after
  const int cols = d / kVec, apart = block / kRows;
  const int col = threadIdx.x & (cols - 1);
  const int row = threadIdx.x / cols;       // and + apart, + 2 apart, + 3 apart
  Raw<kBf16> v[kRows];
  {
    const int64_t off =
        ((static_cast<int64_t>(r0) + (slot0 - first) + row) * Hkv + h) * d + col * kVec;
    const int64_t step = static_cast<int64_t>(apart) * Hkv * d;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row + i * apart;
      if (r >= old && r < end &&
          MSA_IN_RANGE(off + i * step, kVec, a.total * Hkv * d, a.status))
        v[i].load(kv ? a.v : a.k, off + i * step);
      else
        v[i].clear();
    }
  }
  const int64_t page = cache_page(a.s, b, j, a.c.n_pages, a.status);
  if (page < 0) return;
  const int64_t head = page * Hkv + h;
  float* scale_p = (kv ? a.c.v_scale : a.c.k_scale) + head;
  const float s_old = old > 0 ? *scale_p : 0.f;
  const bool mean = end == block && kv == 0;
  if (mean)
    for (int e = threadIdx.x; e < d; e += blockDim.x) sums[e] = 0;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) m = v[i].max_bits(m);
  m = block_max(m, red);  // its barrier is also between the reads of the old scale and the write
  const float s_new = scale_for(m);
  // NaN stays; otherwise the larger of the two.
  const float s = isnan(s_old) || isnan(s_new) ? __uint_as_float(kNanBits) : fmaxf(s_old, s_new);
  const float inv = inverse(s);
  const bool poisoned = isnan(s);
  const bool grown = old > 0 && !(s == s_old);

  float part[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[i] = 0.f;
  uint8_t* codes = (kv ? a.c.v_codes : a.c.k_codes) + ((head << lb) + row) * d + col * kVec;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row + i * apart;
    uint4* at = reinterpret_cast<uint4*>(codes + static_cast<int64_t>(i * apart) * d);
    uint4 c = make_uint4(0, 0, 0, 0);
    bool put = r >= old && r < end;
    if (put) {
      if (!poisoned) c = v[i].encode(inv);
    } else if (r < old && (grown || mean)) {
      c = *at;
      if (grown) {  // the old values, rounded again to the larger scale
        c = poisoned ? make_uint4(0, 0, 0, 0) : rescale(c, s_old, inv);
        put = true;
      }
    }
    if (put && MSA_IN_RANGE(((head << lb) + r) * d + col * kVec, kVec,
                            (a.c.n_pages * Hkv << lb) * d, a.status))
      *at = c;
    if (mean) column_sums(c, part);
  }
  if (threadIdx.x == 0) *scale_p = s;
  if (mean) {
    add_columns(part, sums, col, d);
    __syncthreads();
    store_mean(a.c, head, sums, s);
  }
}

// Kept slots of one (sequence, head) into block j of its new pages, K and V:
// blockIdx.x = (j, head), blockIdx.y = sequence.
template <int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 512 ? 1 : 7)
    cache_gather_kernel(const GatherArgs a) {
  __shared__ uint32_t red[2][32];
  __shared__ int sums[128];
  __shared__ int64_t src[256];   // source row of each slot in the codes
  const int d = a.c.d, block = a.c.block, lb = a.c.lb, Hkv = a.c.Hkv;
  const int b = blockIdx.y;
  const int j = blockIdx.x / Hkv, h = blockIdx.x - j * Hkv;
  const int len = cache_len(a.s, b, block, a.status);
  const int held = static_cast<int>(min64(len, a.budget));
  wait_for_inputs();
  if (static_cast<int64_t>(j) << lb >= held) return;
  CacheBatch dst = a.s;
  dst.table = a.dst_table;
  dst.max_blocks = a.dst_blocks;
  const int64_t page = cache_page(dst, b, j, a.c.n_pages, a.status);
  if (page < 0) return;
  const int end = min(block, held - (j << lb));
  const int32_t* kept =
      a.kept + (static_cast<int64_t>(b) * Hkv + h) * a.budget + (static_cast<int64_t>(j) << lb);
  for (int r = threadIdx.x; r < block; r += blockDim.x) {
    int64_t at = -1;
    if (r < end) {
      const int slot = kept[r];
      const int64_t sp =
          slot >= 0 && slot < len ? cache_page(a.s, b, slot >> lb, a.c.n_pages, a.status) : -1;
      if (sp >= 0) at = ((sp * Hkv + h) << lb) + (slot & (block - 1));
    }
    src[r] = at;
  }
  for (int e = threadIdx.x; e < d; e += blockDim.x) sums[e] = 0;
  __syncthreads();

  const int cols = d / kVec;
  const int col = threadIdx.x & (cols - 1), row = threadIdx.x / cols, apart = block / kRows;
  uint4 c[2][kRows];  // [K, V][row + i * apart]
  float scale[2][kRows];
  uint32_t m[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t at = src[row + i * apart];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      c[kv][i] = make_uint4(0, 0, 0, 0);
      scale[kv][i] = 0.f;
      if (at >= 0 && MSA_IN_RANGE(at, 1, a.c.n_pages * Hkv << lb, a.status)) {
        c[kv][i] = __ldcs(reinterpret_cast<const uint4*>(
            (kv ? a.c.v_codes : a.c.k_codes) + at * d + col * kVec));
        scale[kv][i] = (kv ? a.c.v_scale : a.c.k_scale)[at >> lb];
      }
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      // The largest code's magnitude, then its value.
      const uint32_t w[4] = {c[kv][i].x, c[kv][i].y, c[kv][i].z, c[kv][i].w};
      uint32_t x = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x = __vimax3_u16x2(x, w[k] & 0x007f007fu, (w[k] >> 8) & 0x007f007fu);
      x = max(x >> 16, x & 0xffffu);
      const float s = scale[kv][i];
      const float top = e4m3x2_to_float2(static_cast<uint16_t>(x)).x * s;
      m[kv] = max(m[kv], isnan(s) ? kNanBits : __float_as_uint(top));
    }
  {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      m[kv] = __reduce_max_sync(0xffffffffu, m[kv]);
      if (lane == 0) red[kv][threadIdx.x >> 5] = m[kv];
    }
    __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      m[kv] = __reduce_max_sync(0xffffffffu, lane < nw ? red[kv][lane] : 0u);
  }
  const int64_t head = page * Hkv + h;
  const bool mean = end == block;
  float k_scale = 0.f;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float s = scale_for(m[kv]), inv = inverse(s);
    if (kv == 0) k_scale = s;
    float part[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row + i * apart;
      if (r >= end) continue;
      const float s0 = scale[kv][i];
      uint4 x = c[kv][i];
      if (isnan(s))
        x = make_uint4(0, 0, 0, 0);
      else if (s0 != s)  // codes of the same scale stay as they are
        x = rescale(x, s0, inv);
      if (MSA_IN_RANGE((head << lb) + r, 1, a.c.n_pages * Hkv << lb, a.status))
        *reinterpret_cast<uint4*>((kv ? a.c.v_codes : a.c.k_codes) + ((head << lb) + r) * d +
                                  col * kVec) = x;
      if (kv == 0 && mean) column_sums(x, part);
    }
    if (threadIdx.x == 0) (kv ? a.c.v_scale : a.c.k_scale)[head] = s;
    if (kv == 0 && mean) add_columns(part, sums, col, d);
  }
  if (mean) {
    __syncthreads();
    store_mean(a.c, head, sums, k_scale);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  const dim3 grid(a.blocks * a.c.Hkv * 2, a.s.batch);
  const int threads = write_threads(a.c.block, a.c.d);
  const auto kernel =
      threads <= 128
          ? (a.bf16 ? cache_append_kernel<true, 128> : cache_append_kernel<false, 128>)
          : (a.bf16 ? cache_append_kernel<true, 512> : cache_append_kernel<false, 512>);
  return launch_after(kernel, grid, threads, 0, st, false, a);
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.budget + a.c.block - 1) / a.c.block;
  const dim3 grid(static_cast<unsigned>(blocks * a.c.Hkv), a.s.batch);
  const int threads = write_threads(a.c.block, a.c.d);
  return launch_after(threads <= 128 ? cache_gather_kernel<128> : cache_gather_kernel<512>, grid,
                      threads, 0, st, true, a);
}

}  // namespace msa
