// K11: tokens' rows and cache slots -- writing the 4-bit KV cache, and reading
// it or the 8-bit one back.
//
// A row is the d values of one token and KV head; a thread takes 8 of them, so
// a row is 16 lanes (d = 128) or 8, and a group of 32 values 4 neighbouring
// lanes.  Writing: the group's largest magnitude m (two shuffles), its scale
// 2^e, the least with m <= 7 * 2^e, and codes of x * 2^-e, exact but for one
// rounding.  Reading: code * 2^e, rounded once.  Both move every byte once, and
// HBM bounds them; a thread has kRows rows under way, K and V in CTAs of their
// own.
#include "cache4.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;   // values a thread
constexpr int kRows = 4;  // rows a thread

// Rows (token, head) that a CTA takes.
constexpr int cta_rows(int d) { return kThreads / (d / kPer) * kRows; }

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

// This thread's rows: token and head of each, and the slot's row in the pool
// ([n_pages * Hkv * block]; -1: no such page).
template <int D>
struct Rows {
  int token[kRows];   // within the sequence; -1: past its end
  int head[kRows];
  int64_t slot[kRows];

  __device__ __forceinline__ bool find(const RowsArgs& a, int b, const Span& s, int64_t cta) {
    constexpr int kLanes = D / kPer, kStep = kThreads / kLanes;
    const int64_t row0 = cta * (kStep * kRows);
    const int64_t t0 = row0 / a.Hkv;
    if (t0 >= s.n) return false;
    const int h0 = static_cast<int>(row0 - t0 * a.Hkv) + threadIdx.x / kLanes;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int x = h0 + i * kStep, up = x / a.Hkv;
      const int64_t t = t0 + up;
      token[i] = t < s.n ? static_cast<int>(t) : -1;
      head[i] = x - up * a.Hkv;
    }
    return true;
  }
  __device__ __forceinline__ void look_up(const RowsArgs& a, int b, const Span& s) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      slot[i] = -1;
      if (token[i] < 0) continue;
      const int at = s.first + token[i];
      const int64_t page = cache_page(a.s, b, at >> a.lb, a.n_pages, a.status);
      if (page >= 0) slot[i] = ((page * a.Hkv + head[i]) << a.lb) + (at & (a.block - 1));
    }
  }
};

// 8 values of a row.
template <bool kBf16>
__device__ __forceinline__ void load8(const void* src, int64_t off, float* v) {
  if constexpr (kBf16) {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + off));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
    const float4 x = __ldcs(p), y = __ldcs(p + 1);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}
template <bool kBf16>
__device__ __forceinline__ void store8(void* dst, int64_t off, const float* v) {
  if constexpr (kBf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off),
           make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off);
    __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
}

// blockIdx.x = (rows, K or V), blockIdx.y = sequence.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) cache4_append_kernel(const Append4Args a) {
  constexpr int kLanes = D / kPer;
  const int b = blockIdx.y, kv = blockIdx.x & 1;
  Span s;
  if (!span_of(a, b, &s)) return;
  Rows<D> rows;
  if (!rows.find(a, b, s, blockIdx.x >> 1)) return;
  const int lane = threadIdx.x & (kLanes - 1);
  const void* src = kv ? a.v : a.k;
  float v[kRows][kPer];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t off =
        ((static_cast<int64_t>(s.r0) + max(rows.token[i], 0)) * a.Hkv + rows.head[i]) * D +
        lane * kPer;
    if (rows.token[i] >= 0 && MSA_IN_RANGE(off, kPer, a.total * a.Hkv * D, a.status)) {
      load8<kBf16>(src, off, v[i]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[i][k] = 0.f;
    }
  }
  rows.look_up(a, b, s);
  uint8_t* codes = kv ? a.v_codes : a.k_codes;
  uint8_t* scale = kv ? a.v_scale : a.k_scale;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) m = max(m, __float_as_uint(v[i][k]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // A lane of the row holds what no code stands for.
    const uint32_t bad = __ballot_sync(0xffffffffu, m > kMost4);
    const uint32_t mine = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
    const bool poisoned = bad & mine;
    const int e = poisoned ? 0 : group_exponent4(m);
    const float inv = pow2i(-e);
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[i][k] = poisoned ? 0.f : v[i][k] * inv;
    const uint32_t w = floats_to_e2m1x8(v[i]);
    if (rows.slot[i] < 0 || !MSA_IN_RANGE(rows.slot[i], 1, a.n_pages * a.Hkv << a.lb, a.status)) continue;
    *reinterpret_cast<uint32_t*>(codes + rows.slot[i] * (D / 2) + lane * (kPer / 2)) = w;
    if ((lane & 3) == 0)
      scale[rows.slot[i] * (D / kGroup4) + (lane >> 2)] =
          static_cast<uint8_t>(poisoned ? 255 : e + 127);
  }
}

// blockIdx.x = (rows, K or V), blockIdx.y = sequence.
template <int D, int kBits, bool kBf16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
  constexpr int kLanes = D / kPer;
  const int b = blockIdx.y, kv = blockIdx.x & 1;
  Span s;
  if (!span_of(a, b, &s)) return;
  Rows<D> rows;
  if (!rows.find(a, b, s, blockIdx.x >> 1)) return;
  rows.look_up(a, b, s);
  const int lane = threadIdx.x & (kLanes - 1);
  const uint8_t* codes = kv ? a.v_codes : a.k_codes;
  const void* scale = kv ? a.v_scale : a.k_scale;
  uint2 w[kRows];
  float f[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    w[i] = make_uint2(0, 0);
    f[i] = 0.f;
    const int64_t at = rows.slot[i];
    if (at < 0 || !MSA_IN_RANGE(at, 1, a.n_pages * a.Hkv << a.lb, a.status)) continue;
    if constexpr (kBits == 4) {
      w[i].x = *reinterpret_cast<const uint32_t*>(codes + at * (D / 2) + lane * 4);
      f[i] = e8m0_to_float(static_cast<const uint8_t*>(scale)[at * (D / kGroup4) + (lane >> 2)]);
    } else {
      w[i] = *reinterpret_cast<const uint2*>(codes + at * D + lane * 8);
      f[i] = static_cast<const float*>(scale)[at >> a.lb];
    }
  }
  void* dst = kv ? a.v : a.k;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (rows.token[i] < 0) continue;
    float v[kPer];
    if constexpr (kBits == 4) {
      uint32_t h[4];
      e2m1x8_to_half2(w[i].x, h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        v[2 * k] = x.x;
        v[2 * k + 1] = x.y;
      }
    } else {
      e4m3x4_to_float(w[i].x, v);
      e4m3x4_to_float(w[i].y, v + 4);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] *= f[i];
    const int64_t off =
        ((static_cast<int64_t>(s.r0) + rows.token[i]) * a.Hkv + rows.head[i]) * D + lane * kPer;
    if (MSA_IN_RANGE(off, kPer, a.total * a.Hkv * D, a.status)) store8<kBf16>(dst, off, v);
  }
}

}  // namespace

int64_t cache_rows_ctas(int64_t most, int Hkv, int d) {
  return (most * Hkv + cta_rows(d) - 1) / cta_rows(d) * 2;
}

cudaError_t launch_cache4_append(const Append4Args& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(cache_rows_ctas(a.most, a.Hkv, a.d)), a.s.batch);
  const auto kernel = a.d == 128 ? (a.bf16 ? cache4_append_kernel<128, true>
                                           : cache4_append_kernel<128, false>)
                                 : (a.bf16 ? cache4_append_kernel<64, true>
                                           : cache4_append_kernel<64, false>);
  return launch_after(kernel, grid, kThreads, 0, st, false, a);
}

cudaError_t launch_cache_read(const ReadArgs& a, int bits, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(cache_rows_ctas(a.most, a.Hkv, a.d)), a.s.batch);
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
