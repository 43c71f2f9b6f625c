// K13: norms of queries and keys for each head with the rotary position
// embedding, and their gradients.
//
// Of a row x (one token and head): z = x r w, r = (mean(x^2) + eps)^-1/2, and y
// = R z, R turning every pair of dims by the token's angles.  Backward, of g =
// R^T dy and u = w g: dx = r (u - x r^2 mean(x u)), dw = the sum over tokens
// and heads of g x r.  Everything is fp32 between one read and one rounding.
//
// Each value is read and written once, and HBM bounds a long call.  A thread
// takes 16 values of a row, two runs of 8 half a row apart, so that both
// members of a pair are its own in either pairing; a row is d / 16 lanes.  The
// angles are the same for all heads of a token: the CTA computes them once for
// a tile of tokens, as 64-bit integers that wrap around at a full turn, reduced
// to an eighth of a turn before they become floats.
#include "rope.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;  // tokens whose angles a CTA holds

// cos and sin (times m) of position * f / 2^64 turns.  Products wrap at whole
// turns; the nearest quarter turn is taken off as an integer, so the rest, at
// most an eighth of a turn, loses 2^-27 of a turn at most as a float.
__device__ __forceinline__ float2 turn_of(int64_t position, int64_t f, float m) {
  const uint64_t phase = static_cast<uint64_t>(position) * static_cast<uint64_t>(f);
  const uint32_t hi = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int rest = static_cast<int>(hi - (quarter << 30));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * m, s * m);
}

// 16 values of a row: 8 at `p`, 8 half a row on.
template <int D, bool kBf16>
struct Piece {
  float v[16];
  __device__ __forceinline__ void load(const void* src, int64_t off) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kBf16) {
        const uint4 x = __ldcs(reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(src) + off + h * (D / 2)));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
          v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
        const float4* p =
            reinterpret_cast<const float4*>(static_cast<const float*>(src) + off + h * (D / 2));
        const float4 x = __ldcs(p), y = __ldcs(p + 1);
        v[8 * h + 0] = x.x, v[8 * h + 1] = x.y, v[8 * h + 2] = x.z, v[8 * h + 3] = x.w;
        v[8 * h + 4] = y.x, v[8 * h + 5] = y.y, v[8 * h + 6] = y.z, v[8 * h + 7] = y.w;
      }
    }
  }
  __device__ __forceinline__ void store(void* dst, int64_t off) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kBf16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off + h * (D / 2)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off + h * (D / 2));
        p[0] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
        p[1] = make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
      }
    }
  }
  // Turns the pairs by the angles of cs (of pair i: [i] the cosine, [D / 2 + i]
  // the sine), or back.
  template <bool kInterleaved, bool kBack>
  __device__ __forceinline__ void turn(const float* cs, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // 4 pairs: of halves a run apart, dims 4h .. 4h + 3 of both; of
      // neighbours, the 8 dims of run h.
      const int i0 = kInterleaved ? h * (D / 4) + lane * 4 : lane * 8 + 4 * h;
      const float4 c4 = *reinterpret_cast<const float4*>(cs + i0);
      const float4 s4 = *reinterpret_cast<const float4*>(cs + D / 2 + i0);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float& a = kInterleaved ? v[8 * h + 2 * k] : v[4 * h + k];
        float& b = kInterleaved ? v[8 * h + 2 * k + 1] : v[8 + 4 * h + k];
        const float sn = kBack ? -s[k] : s[k];
        const float x = a * c[k] - b * sn, y = a * sn + b * c[k];
        a = x;
        b = y;
      }
    }
  }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float weight_at(const void* w, int bf16, int i) {
  return bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(w)[i])
              : static_cast<const float*>(w)[i];
}

// The angles of a tile's tokens: [token][cosines, sines].
template <int D>
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t t0, int tokens, float* cs) {
  for (int i = threadIdx.x; i < tokens * (D / 2); i += kThreads) {
    const int t = i / (D / 2), f = i - t * (D / 2);
    const float2 x = turn_of(a.positions[t0 + t], a.freqs[f], a.mscale);
    cs[t * D + f] = x.x;
    cs[t * D + D / 2 + f] = x.y;
  }
}

// A CTA takes tiles of tokens, all heads of queries and keys.
template <int D, bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
  __shared__ __align__(16) float cs[kMaxTile * D];
  __shared__ __align__(16) float weight[2][D];
  const int lane = threadIdx.x & (kLanes - 1), H = a.heads[0] + a.heads[1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (a.weight[i])
      for (int k = threadIdx.x; k < D; k += kThreads) weight[i][k] = weight_at(a.weight[i], a.w_bf16, k);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile; t0 < a.n;
       t0 += static_cast<int64_t>(gridDim.x) * a.tile) {
    const int tokens = static_cast<int>(min64(a.tile, a.n - t0));
    __syncthreads();
    angles<D>(a, t0, tokens, cs);
    __syncthreads();
    const int rows = tokens * H;
    for (int r0 = 0; r0 < rows; r0 += kStep) {  // whole warps, for the sums
      const int r = r0 + threadIdx.x / kLanes;
      const bool in = r < rows;
      const int t = in ? r / H : 0, hh = in ? r - t * H : 0;
      const int side = hh >= a.heads[0];
      const int h = side ? hh - a.heads[0] : hh;
      Piece<D, kBf16> x;
      const int64_t from = (t0 + t) * a.stride[side] + h * D + lane * 8;
      if (in) {
        x.load(a.x[side], from);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) x.v[k] = 0.f;
      }
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) ss = fmaf(x.v[k], x.v[k], ss);
      ss = row_sum<kLanes>(ss);
      if (!in) continue;
      if (a.weight[side]) {
        const float s = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          x.v[k] = x.v[k] * s * weight[side][(k >> 3) * (D / 2) + lane * 8 + (k & 7)];
      }
      x.template turn<kInterleaved, false>(cs + t * D, lane);
      const int64_t to = ((t0 + t) * a.heads[side] + h) * D + lane * 8;
      if (MSA_IN_RANGE(to, D / 2 + 8, a.n * a.heads[side] * D, a.status)) x.store(a.out[side], to);
    }
  }
}

// The first ctas[0] CTAs take the queries' rows, the others the keys'.
template <int D, bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
  __shared__ __align__(16) float cs[kMaxTile * D];
  __shared__ __align__(16) float weight[D];
  const int side = static_cast<int>(blockIdx.x) >= a.ctas[0];
  const int cta = blockIdx.x - (side ? a.ctas[0] : 0), ctas = a.ctas[side];
  const int lane = threadIdx.x & (kLanes - 1), H = a.heads[side];
  const bool norm = a.weight[side] != nullptr;
  let_next_start();
  if (norm)
    for (int k = threadIdx.x; k < D; k += kThreads) weight[k] = weight_at(a.weight[side], a.w_bf16, k);
  float dw[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) dw[k] = 0.f;
  for (int64_t t0 = static_cast<int64_t>(cta) * a.tile; t0 < a.n;
       t0 += static_cast<int64_t>(ctas) * a.tile) {
    const int tokens = static_cast<int>(min64(a.tile, a.n - t0));
    __syncthreads();
    angles<D>(a, t0, tokens, cs);
    __syncthreads();
    const int rows = tokens * H;
    for (int r0 = 0; r0 < rows; r0 += kStep) {
      const int r = r0 + threadIdx.x / kLanes;
      const bool in = r < rows;
      const int t = in ? r / H : 0, h = in ? r - t * H : 0;
      Piece<D, kBf16> x, g;
      if (in) {
        g.load(a.dy[side], (t0 + t) * a.dy_stride[side] + h * D + lane * 8);
        if (norm) x.load(a.x[side], (t0 + t) * a.stride[side] + h * D + lane * 8);
      }
      if (!in || !norm) {
#pragma unroll
        for (int k = 0; k < 16; ++k) x.v[k] = 0.f;
      }
      if (!in) {
#pragma unroll
        for (int k = 0; k < 16; ++k) g.v[k] = 0.f;
      }
      g.template turn<kInterleaved, true>(cs + t * D, lane);
      if (norm) {
        float ss = 0.f, xu = 0.f, w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          w[k] = weight[(k >> 3) * (D / 2) + lane * 8 + (k & 7)];
          ss = fmaf(x.v[k], x.v[k], ss);
          xu = fmaf(x.v[k] * w[k], g.v[k], xu);
        }
        ss = row_sum<kLanes>(ss);
        xu = row_sum<kLanes>(xu);
        const float s = rsqrtf(ss * (1.f / D) + a.eps);
        const float f = s * s * (xu * (1.f / D));
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          if (in) dw[k] = fmaf(g.v[k], x.v[k] * s, dw[k]);
          g.v[k] = s * (w[k] * g.v[k] - x.v[k] * f);
        }
      }
      const int64_t to = ((t0 + t) * H + h) * D + lane * 8;
      if (in && MSA_IN_RANGE(to, D / 2 + 8, a.n * H * D, a.status)) g.store(a.out[side], to);
    }
  }
  if (!norm) return;
  // Lanes of the same dims are kLanes apart, then the warps, in order.
#pragma unroll
  for (int k = 0; k < 16; ++k)
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
  __syncthreads();
  if ((threadIdx.x & 31) < kLanes) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      cs[(threadIdx.x >> 5) * D + (k >> 3) * (D / 2) + lane * 8 + (k & 7)] = dw[k];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += cs[w * D + threadIdx.x];
    a.part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = sum;
  }
}

// The weights' gradients from the CTAs' sums: blockIdx.x the side, a thread a
// column of every kSlices-th CTA.
constexpr int kSlices = 8;
template <int D>
__global__ void __launch_bounds__(D * kSlices) norm_rope_dw_kernel(const RopeArgs a) {
  __shared__ float sums[kSlices][D];
  const int side = blockIdx.x, k = threadIdx.x % D, slice = threadIdx.x / D;
  wait_for_inputs();
  if (!a.dweight[side]) return;
  const float* part = a.part + (side ? static_cast<int64_t>(a.ctas[0]) * D : 0) + k;
  float sum = 0.f;
  if (a.n > 0)
    for (int c = slice; c < a.ctas[side]; c += kSlices) sum += part[static_cast<int64_t>(c) * D];
  sums[slice][k] = sum;
  __syncthreads();
  if (slice) return;
#pragma unroll
  for (int i = 1; i < kSlices; ++i) sum += sums[i][k];
  if (a.w_bf16)
    static_cast<__nv_bfloat16*>(a.dweight[side])[k] = __float2bfloat16_rn(sum);
  else
    static_cast<float*>(a.dweight[side])[k] = sum;
}

// Tokens a CTA takes at a time: enough rows for some passes of its threads, and
// a tile for every CTA.
int tile_of(int64_t n, int heads, int d, int ctas) {
  const int step = kThreads / (d / 16);
  const int64_t t = min64(kMaxTile, max64(1, 8 * step / max64(1, heads)));
  return static_cast<int>(max64(1, min64(t, (n + ctas - 1) / ctas)));
}

constexpr int kPerSm = 4;

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a0, cudaStream_t st) {
  RopeArgs a = a0;
  a.tile = tile_of(a.n, a.heads[0] + a.heads[1], a.d, kSms * kPerSm);
  const dim3 grid(static_cast<unsigned>(min64((a.n + a.tile - 1) / a.tile, kSms * kPerSm)));
  void (*kernel)(RopeArgs);
  if (a.d == 128)
    kernel = a.bf16 ? (a.interleaved ? norm_rope_kernel<128, true, true>
                                     : norm_rope_kernel<128, true, false>)
                    : (a.interleaved ? norm_rope_kernel<128, false, true>
                                     : norm_rope_kernel<128, false, false>);
  else
    kernel = a.bf16 ? (a.interleaved ? norm_rope_kernel<64, true, true>
                                     : norm_rope_kernel<64, true, false>)
                    : (a.interleaved ? norm_rope_kernel<64, false, true>
                                     : norm_rope_kernel<64, false, false>);
  return launch_after(kernel, grid, kThreads, 0, st, false, a);
}

void norm_rope_bwd_ctas(int64_t n, const int* heads, int d, int* ctas) {
  const int64_t all = kSms * kPerSm;
  const int H = heads[0] + heads[1];
  ctas[1] = heads[1] ? static_cast<int>(max64(1, min64(n, all * heads[1] / H))) : 0;
  ctas[0] = static_cast<int>(max64(1, min64(n, all - ctas[1])));
}

cudaError_t launch_norm_rope_bwd(const RopeArgs& a0, cudaStream_t st) {
  RopeArgs a = a0;
  const bool norm = a.weight[0] || a.weight[1];
  if (a.n > 0) {
    const int t0 = tile_of(a.n, a.heads[0], a.d, a.ctas[0]);
    const int t1 = a.heads[1] ? tile_of(a.n, a.heads[1], a.d, a.ctas[1]) : 1;
    a.tile = t0 > t1 ? t0 : t1;
    const dim3 grid(static_cast<unsigned>(a.ctas[0] + a.ctas[1]));
    void (*kernel)(RopeArgs);
    if (a.d == 128)
      kernel = a.bf16 ? (a.interleaved ? norm_rope_bwd_kernel<128, true, true>
                                       : norm_rope_bwd_kernel<128, true, false>)
                      : (a.interleaved ? norm_rope_bwd_kernel<128, false, true>
                                       : norm_rope_bwd_kernel<128, false, false>);
    else
      kernel = a.bf16 ? (a.interleaved ? norm_rope_bwd_kernel<64, true, true>
                                       : norm_rope_bwd_kernel<64, true, false>)
                      : (a.interleaved ? norm_rope_bwd_kernel<64, false, true>
                                       : norm_rope_bwd_kernel<64, false, false>);
    const cudaError_t e = launch_after(kernel, grid, kThreads, 0, st, false, a);
    if (e != cudaSuccess) return e;
  }
  if (!norm) return cudaSuccess;
  return launch_after(a.d == 128 ? norm_rope_dw_kernel<128> : norm_rope_dw_kernel<64>, dim3(2),
                      a.d * kSlices, 0, st, a.n > 0, a);
}

}  // namespace msa
