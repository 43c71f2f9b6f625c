// K7: writing the 8-bit KV cache -- appending new tokens, and gathering kept
// tokens into fresh blocks after an eviction.
//
// Both write whole (block, KV head) pairs, K and V apart: one CTA takes the
// values of one block of one head of K or of V, finds their largest
// magnitude, forms the power-of-two scale (cache_common.cuh), and stores the
// codes.  Every thread keeps its 2 x 16 values in registers, so the data is
// read once and written once: nothing but HBM bounds a long write.
#include "cache_common.cuh"

namespace msa {
namespace {

constexpr int kVec = 16;  // values of one 16-byte code store

// Threads of a CTA: each takes two groups of 16 values of the same columns.
__host__ __device__ inline int write_threads(int block, int d) { return block * d / (2 * kVec); }

__device__ __forceinline__ float block_max(float x, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  const int warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
  if ((threadIdx.x & 31) == 0) smem[warp] = x;
  __syncthreads();
  x = smem[0];
  for (int w = 1; w < nw; ++w) x = fmaxf(x, smem[w]);
  return x;
}

// Largest finite magnitude of the thread's values, +inf where one is not
// finite (fmaxf would drop a NaN).
__device__ __forceinline__ float group_max(const float* v, float m) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const float a = fabsf(v[i]);
    m = fmaxf(m, a <= 3.402823466e38f ? a : INFINITY);
  }
  return m;
}

__device__ __forceinline__ uint4 encode(const float* v, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // One rounding, to nearest even: the product is exact (inv is 2^-e).
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void decode(const uint4& x, float s, float* v) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e4m3x4_to_float(w[i], v + 4 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * i + k] *= s;
  }
}

// Scale of a block whose largest magnitude is amax: 0 for a block of zeros,
// NaN for one that holds a NaN or an infinity.
__device__ __forceinline__ float scale_for(float amax) {
  if (isinf(amax)) return __uint_as_float(0x7fc00000u);
  return amax > 0.f ? pow2i(block_exponent(amax)) : 0.f;
}
// 1 / scale (0 for a scale of 0 or NaN: codes of 0).  An exponent of 127 and
// more cannot come up: block_exponent ends at 120.
__device__ __forceinline__ float inverse(float s) {
  return s > 0.f ? pow2i(127 - static_cast<int>(__float_as_uint(s) >> 23)) : 0.f;
}

// Mean key of a full block from its codes, rounded to bf16 once.  Codes are
// whole multiples of 2^-9, so a column sums exactly in 32-bit integers (at
// most 256 * 448 * 512 < 2^26); the conversion to fp32 keeps a sticky bit,
// and the scaling by 2^e / block (a power of two) is exact.
__device__ __forceinline__ void column_sums(const uint4& c, int* part) {
  float v[kVec];
  decode(c, 512.f, v);
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[i] += static_cast<int>(v[i]);
}
__device__ __forceinline__ __nv_bfloat16 mean_of(int sum, float scale, int block) {
  float f = __int2float_rz(sum);
  if (static_cast<int>(f) != sum) f = __uint_as_float(__float_as_uint(f) | 1u);
  // scale / (512 * block) in two exact steps unless the result is subnormal
  return __float2bfloat16_rn(f * (1.f / (512.f * static_cast<float>(block))) * scale);
}

// Adds the thread's 16 column sums to sums[d] (integers: any order gives the
// same result).  Lanes of the same columns are d/16 apart.
__device__ __forceinline__ void add_columns(int* part, int* sums, int col, int d) {
  for (int o = 16; o >= d / kVec; o >>= 1) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[i] += __shfl_xor_sync(0xffffffffu, part[i], o);
  }
  if ((threadIdx.x & 31) < d / kVec) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) atomicAdd(&sums[col * kVec + i], part[i]);
  }
}

template <bool kBf16>
__device__ __forceinline__ void load_values(const void* src, int64_t off, float* v) {
  if constexpr (kBf16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + off);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 x = __ldcs(p + h);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float4 x = __ldcs(p + h);
      v[4 * h] = x.x;
      v[4 * h + 1] = x.y;
      v[4 * h + 2] = x.z;
      v[4 * h + 3] = x.w;
    }
  }
}

// blockIdx.x = (block of the new range, head, K or V), blockIdx.y = sequence.
template <bool kBf16>
__global__ void __launch_bounds__(1024) cache_append_kernel(const AppendArgs a) {
  __shared__ float red[32];
  __shared__ int sums[128];
  const int d = a.c.d, block = a.c.block, Hkv = a.c.Hkv;
  const int b = blockIdx.y;
  const int kv = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % Hkv;
  const int64_t r0 = a.cu[b], r1 = a.cu[b + 1];
  const int64_t len = cache_len(a.s, b, block, a.status), n_new = r1 - r0;
  if (n_new == 0) return;
  if (r0 < 0 || r1 > a.total || n_new < 0 || n_new > a.max_new || n_new > len) {
    if (threadIdx.x == 0) record_status(a.status, MSA_ERR_INVALID_ARG);
    return;
  }
  const int64_t first = len - n_new;  // slot of the first new token
  const int64_t j = first / block + (blockIdx.x >> 1) / Hkv;
  if (j * block >= len) return;
  const int64_t page = cache_page(a.s, b, j, a.c.n_pages, a.status);
  if (page < 0) return;

  const int64_t slot0 = j * block;
  const int old = static_cast<int>(max64(0, first - slot0));           // slots held before
  const int end = static_cast<int>(min64(block, len - slot0));         // slots held after
  const bool full = end == block;
  const int cols = d / kVec;
  const int col = threadIdx.x % cols, row = threadIdx.x / cols;  // and row + block/2
  const int64_t head = (page * Hkv + h);
  uint8_t* codes = (kv ? a.c.v_codes : a.c.k_codes) + head * block * d;
  float* scale_p = (kv ? a.c.v_scale : a.c.k_scale) + head;
  const void* src = kv ? a.v : a.k;
  if (kv == 0)
    for (int e = threadIdx.x; e < d; e += blockDim.x) sums[e] = 0;

  float v[2][kVec];
  float m = 0.f;
  bool fresh[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row + i * (block / 2);
    fresh[i] = r >= old && r < end;
    if (fresh[i]) {
      const int64_t off = ((r0 + slot0 + r - first) * Hkv + h) * d + col * kVec;
      if (MSA_IN_RANGE(off, kVec, a.total * Hkv * d, a.status)) load_values<kBf16>(src, off, v[i]);
      m = group_max(v[i], m);
    }
  }
  const float s_old = old > 0 ? *scale_p : 0.f;
  m = block_max(m, red);
  const float s_new = scale_for(m);
  // NaN stays; otherwise the larger of the two.
  const float s = isnan(s_old) || isnan(s_new) ? __uint_as_float(0x7fc00000u) : fmaxf(s_old, s_new);
  const float inv = inverse(s);
  const bool grown = old > 0 && !(s == s_old);
  const bool mean = full && kv == 0;

  int part[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[i] = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row + i * (block / 2);
    uint4* at = reinterpret_cast<uint4*>(codes + static_cast<int64_t>(r) * d + col * kVec);
    uint4 c;
    bool put = fresh[i];
    if (r < old && (grown || mean)) {
      c = *at;
      if (grown) {
        // The old values, rounded again to the larger scale.
        decode(c, isnan(s_old) ? 0.f : s_old, v[i]);
        put = true;
      }
    }
    if (put) {
      c = encode(v[i], inv);
      if (isnan(s)) c = make_uint4(0, 0, 0, 0);
      if (MSA_IN_RANGE(head * block * d + static_cast<int64_t>(r) * d + col * kVec, kVec,
                       a.c.n_pages * Hkv * block * d, a.status))
        *at = c;
    }
    if (mean && r < end) column_sums(c, part);
  }
  // Every read of the old scale is before block_max's barrier.
  if (threadIdx.x == 0) *scale_p = s;
  if (mean) {
    add_columns(part, sums, col, d);
    __syncthreads();
    for (int e = threadIdx.x; e < d; e += blockDim.x)
      a.c.k_mean[head * d + e] =
          isnan(s) ? __float2bfloat16_rn(s) : mean_of(sums[e], s, block);
  }
}

// Kept slots of one (sequence, head) into block j of its new pages.
__global__ void __launch_bounds__(1024) cache_gather_kernel(const GatherArgs a) {
  __shared__ float red[32];
  __shared__ int sums[128];
  const int d = a.c.d, block = a.c.block, Hkv = a.c.Hkv;
  const int b = blockIdx.y;
  const int kv = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % Hkv;
  const int64_t j = (blockIdx.x >> 1) / Hkv;
  const int64_t len = cache_len(a.s, b, block, a.status);
  const int64_t held = min64(len, a.budget);
  if (j * block >= held) return;
  CacheBatch dst = a.s;
  dst.table = a.dst_table;
  dst.max_blocks = a.dst_blocks;
  const int64_t page = cache_page(dst, b, j, a.c.n_pages, a.status);
  if (page < 0) return;
  const int end = static_cast<int>(min64(block, held - j * block));
  const int cols = d / kVec;
  const int col = threadIdx.x % cols, row = threadIdx.x / cols;
  const uint8_t* codes = kv ? a.c.v_codes : a.c.k_codes;
  const float* scales = kv ? a.c.v_scale : a.c.k_scale;
  const int32_t* kept = a.kept + (static_cast<int64_t>(b) * Hkv + h) * a.budget + j * block;
  if (kv == 0)
    for (int e = threadIdx.x; e < d; e += blockDim.x) sums[e] = 0;

  float v[2][kVec];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row + i * (block / 2);
    if (r < end) {
      const int64_t slot = kept[r];
      const int64_t sp = slot >= 0 && slot < len
                             ? cache_page(a.s, b, slot / block, a.c.n_pages, a.status)
                             : -1;
      if (sp >= 0) {
        const int64_t hd = sp * Hkv + h;
        const float s = scales[hd];
        const uint4 c = *reinterpret_cast<const uint4*>(codes + (hd * block + slot % block) * d +
                                                        col * kVec);
        decode(c, s, v[i]);
        if (isnan(s)) m = INFINITY;
      } else {
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[i][k] = 0.f;
      }
      m = group_max(v[i], m);
    }
  }
  m = block_max(m, red);
  const float s = scale_for(m), inv = inverse(s);
  const bool mean = end == block && kv == 0;
  const int64_t head = page * Hkv + h;
  uint8_t* to = (kv ? a.c.v_codes : a.c.k_codes) + head * block * d;
  int part[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) part[i] = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row + i * (block / 2);
    if (r < end) {
      uint4 c = encode(v[i], inv);
      if (isnan(s)) c = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(to + static_cast<int64_t>(r) * d + col * kVec) = c;
      if (mean) column_sums(c, part);
    }
  }
  if (threadIdx.x == 0) (kv ? a.c.v_scale : a.c.k_scale)[head] = s;
  if (mean) {
    add_columns(part, sums, col, d);
    __syncthreads();
    for (int e = threadIdx.x; e < d; e += blockDim.x)
      a.c.k_mean[head * d + e] =
          isnan(s) ? __float2bfloat16_rn(s) : mean_of(sums[e], s, block);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  // A range of max_new tokens touches at most this many blocks.
  const int64_t blocks = (a.max_new + a.c.block - 2) / a.c.block + 1;
  const dim3 grid(static_cast<unsigned>(min64(blocks, a.s.max_blocks) * a.c.Hkv * 2), a.s.batch);
  const int threads = write_threads(a.c.block, a.c.d);
  if (a.bf16)
    cache_append_kernel<true><<<grid, threads, 0, st>>>(a);
  else
    cache_append_kernel<false><<<grid, threads, 0, st>>>(a);
  return cudaPeekAtLastError();
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.budget + a.c.block - 1) / a.c.block;
  const dim3 grid(static_cast<unsigned>(blocks * a.c.Hkv * 2), a.s.batch);
  cache_gather_kernel<<<grid, write_threads(a.c.block, a.c.d), 0, st>>>(a);
  return cudaPeekAtLastError();
}

}  // namespace msa
