// K9: which blocks of the cache each query token attends -- the decode-time
// form of the landmark-scored selection (msa_block_select takes 128 rows
// together).
//
// For query token t of sequence b and KV group c, block l (full, wholly
// before the window) scores sum over the group's heads h of <q_h, kmean_l>;
// the top_k best are chosen, ties to the lower block.  The result is that of
// the sum in 64 bits: the scores are computed in fp32 with a bound of their
// rounding each, E_l = (g + 48) 2^-24 sum_d (sum_h |q_h|) |kmean_l| (a lane
// adds D/4 <= 32 products one by one, two more additions join four lanes,
// and the sum over g heads rounds g times); only the blocks whose score is
// within 2 max E of the k-th are computed again in 64 bits.  So the choice
// does not depend on the order of any fp32 sum.
//
// The block means are read once for all query tokens of a sequence: 2 d
// bytes a block and KV head, four lanes a block with four 16-byte loads in
// flight each; HBM (or L2) bounds the scores.  The choice is one CTA a
// (token, group): a radix selection of the k-th score over the CTA's list.
#include <math.h>

#include "cache_common.cuh"

namespace msa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = kScoreThreads / 4;  // blocks a CTA scores at a time
constexpr int kScoreT = 4;                       // query tokens taken together
constexpr int kPickThreads = 512;
constexpr int kListMax = 1024;  // near-ties ranked in shared memory

__device__ __forceinline__ int candidates(const CacheSelectArgs& a, int len, int t) {
  const int p = len - a.T + t;
  return p >= a.window ? (p - a.window + 1) >> a.c.lb : 0;
}

template <bool kBf16>
__device__ __forceinline__ float q_at(const void* q, int64_t i) {
  if constexpr (kBf16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]);
  else
    return static_cast<const float*>(q)[i];
}

// blockIdx = (tile of 64 blocks, KV head, sequence).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const CacheSelectArgs a) {
  __shared__ __align__(16) float qs[kScoreT][D], qa[kScoreT][D];
  let_next_start();
  const int c = blockIdx.y, b = blockIdx.z, g = a.Hq / a.c.Hkv;
  const int len = cache_len(a.s, b, a.c.block, a.status);
  const int most = candidates(a, len, a.T - 1);  // the last token sees the most
  const int l = blockIdx.x * kScoreBlocks + (threadIdx.x >> 2), lane4 = threadIdx.x & 3;
  if (static_cast<int>(blockIdx.x) * kScoreBlocks >= most) return;
  // Four 16-byte pieces of the block's mean a lane: d = 32 i + 8 lane4 + 0..7.
  uint4 km[D / 32];
  if (l < most) {
    int64_t page = cache_page(a.s, b, l, a.c.n_pages, a.status);
    page = page < 0 ? 0 : page;
    const uint4* src = reinterpret_cast<const uint4*>(a.c.k_mean + (page * a.c.Hkv + c) * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) km[i] = __ldg(src + 4 * i + lane4);
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) km[i] = make_uint4(0, 0, 0, 0);
  }
  const float eps = (g + 48) * 5.9604645e-8f;
  for (int t0 = 0; t0 < a.T; t0 += kScoreT) {
    const int nt = min(kScoreT, a.T - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * D; i += kScoreThreads) {
      const int t = i / D, e = i - t * D;
      const int64_t at = ((static_cast<int64_t>(b) * a.T + t0 + t) * a.Hq + c * g) * D + e;
      float s = 0.f, m = 0.f;
      for (int h = 0; h < g; ++h) {
        const float x = q_at<kBf16>(a.q, at + static_cast<int64_t>(h) * D);
        s += x;
        m += fabsf(x);
      }
      qs[t][e] = s;
      qa[t][e] = m;
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {km[i].x, km[i].y, km[i].z, km[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
          const int e = 32 * i + 8 * lane4 + 2 * k;
          const float2 qv = *reinterpret_cast<const float2*>(&qs[t][e]);
          const float2 av = *reinterpret_cast<const float2*>(&qa[t][e]);
          s = fmaf(qv.x, lo, s);
          s = fmaf(qv.y, hi, s);
          m = fmaf(av.x, fabsf(lo), m);
          m = fmaf(av.y, fabsf(hi), m);
        }
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      m += __shfl_xor_sync(0xffffffffu, m, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      m += __shfl_xor_sync(0xffffffffu, m, 2);
      if (lane4 == 0 && l < most) {
        const int64_t at =
            ((static_cast<int64_t>(b) * a.T + t0 + t) * a.c.Hkv + c) * a.s.max_blocks + l;
        // NaN ranks last, as -inf; a bound that is not finite asks for 64 bits.
        a.score[at] = s;
        a.err[at] = m * eps;
      }
    }
  }
}

// Unsigned keys that order as the values do; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  x = isnan(x) ? -INFINITY : x + 0.f;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {
  x = isnan(x) ? -INFINITY : x + 0.0;
  const uint64_t u = __double_as_longlong(x);
  return u >> 63 ? ~u : u | (1ull << 63);
}

struct PickShared {
  int hist[256];
  int warp[kPickThreads / 32];
  int base, digit, left;
  int n_list;
  int list[kListMax];
  double val[kListMax];
  float emax[kPickThreads / 32];
};

// The `need`-th largest of the keys get(0..n): by bytes from the top, a
// histogram of the keys that share the bytes found so far.
template <typename K, typename Get>
__device__ __forceinline__ K kth_largest(int n, int need, Get get, PickShared& sh) {
  constexpr int kBytes = sizeof(K);
  K prefix = 0, mask = 0;
  int left = need;
  for (int byte = kBytes - 1; byte >= 0; --byte) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      K k;
      if (get(i, &k) && (k & mask) == prefix)
        atomicAdd(&sh.hist[static_cast<int>(k >> (8 * byte)) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // Lane l sums digits 255 - 8 l .. 248 - 8 l, then the lanes scan.
      int s = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += sh.hist[255 - 8 * threadIdx.x - i];
      int upto = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (threadIdx.x >= o) upto += y;
      }
      int before = upto - s;
      if (before < left && left <= upto) {
        for (int i = 0; i < 8; ++i) {
          const int dgt = 255 - 8 * threadIdx.x - i, h = sh.hist[dgt];
          if (left <= before + h) {
            sh.digit = dgt;
            sh.left = left - before;
            break;
          }
          before += h;
        }
      }
    }
    __syncthreads();
    prefix |= static_cast<K>(sh.digit) << (8 * byte);
    mask |= static_cast<K>(255) << (8 * byte);
    left = sh.left;
  }
  return prefix;
}

// Score of block l in 64 bits, by one warp: the products of bf16 are exact,
// so what rounds is a sum of g * D / 32 terms a lane and five joins.
template <bool kBf16>
__device__ __forceinline__ double exact_score(const CacheSelectArgs& a, int b, int t, int c,
                                              int l) {
  const int lane = threadIdx.x & 31, g = a.Hq / a.c.Hkv, d = a.c.d;
  int64_t page = cache_page(a.s, b, l, a.c.n_pages, a.status);
  page = page < 0 ? 0 : page;
  const __nv_bfloat16* km = a.c.k_mean + (page * a.c.Hkv + c) * d;
  const int64_t q0 = ((static_cast<int64_t>(b) * a.T + t) * a.Hq + c * g) * d;
  double s = 0.0;
  for (int e = lane; e < d; e += 32) {
    double x = 0.0;
    for (int h = 0; h < g; ++h)
      x += static_cast<double>(q_at<kBf16>(a.q, q0 + static_cast<int64_t>(h) * d + e));
    s += x * static_cast<double>(__bfloat162float(km[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One CTA a (token, KV head).
template <bool kBf16>
__global__ void __launch_bounds__(kPickThreads) cache_pick_kernel(const CacheSelectArgs a) {
  __shared__ PickShared sh;
  const int c = blockIdx.x % a.c.Hkv, bt = blockIdx.x / a.c.Hkv;
  const int b = bt / a.T, t = bt - b * a.T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t u = static_cast<int64_t>(bt) * a.c.Hkv + c;
  const int n = candidates(a, cache_len(a.s, b, a.c.block, a.status), t);
  int32_t* sel = a.sel + u * a.top_k;
  const int k = min(a.top_k, n);
  let_next_start();
  wait_for_inputs();
  if (threadIdx.x == 0) a.cnt[u] = k;
  for (int i = k + threadIdx.x; i < a.top_k; i += kPickThreads) sel[i] = -1;
  if (k == n) {
    for (int i = threadIdx.x; i < n; i += kPickThreads) sel[i] = i;
    return;
  }
  const float* score = a.score + u * a.s.max_blocks;
  const float* err = a.err + u * a.s.max_blocks;
  double* exact = a.exact + u * a.s.max_blocks;

  float em = 0.f;
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const float e = err[i];
    em = fmaxf(em, isnan(e) ? INFINITY : e);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) em = fmaxf(em, __shfl_xor_sync(0xffffffffu, em, o));
  if (lane == 0) sh.emax[warp] = em;
  if (threadIdx.x == 0) sh.n_list = 0;
  const float kth = value_of(kth_largest<uint32_t>(
      n, k,
      [&](int i, uint32_t* key) {
        *key = key_of(score[i]);
        return true;
      },
      sh));
  em = sh.emax[0];
  for (int w = 1; w < kPickThreads / 32; ++w) em = fmaxf(em, sh.emax[w]);
  // Twice the bound on either side, widened for the roundings of these two.
  const float room = 2.0001f * em + fabsf(kth) * 2.4e-7f + 1e-38f;
  const float above = kth + room, below = kth - room;
  // 2: chosen whatever the rest, 1: near the k-th, 0: not chosen.
  auto cls = [&](float s) {
    s = isnan(s) ? -INFINITY : s;
    if (s > above) return 2;
    return s < below ? 0 : 1;
  };
  int sure = 0;
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const int x = cls(score[i]);
    sure += x == 2;
    if (x == 1) {
      const int at = atomicAdd(&sh.n_list, 1);
      if (at < kListMax) sh.list[at] = i;  // in any order: ranked by value, then block
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sure += __shfl_xor_sync(0xffffffffu, sure, o);
  if (lane == 0) sh.warp[warp] = sure;
  __syncthreads();
  sure = 0;
  for (int w = 0; w < kPickThreads / 32; ++w) sure += sh.warp[w];
  const int near = sh.n_list, need = k - sure;
  __syncthreads();

  // Which of the near ones: all; by rank in shared memory; or, for more than
  // a list of them (equal blocks), by another radix selection.
  double cut = 0.0;   // near values above are taken
  int ties = 0;       // of those equal to it, the lowest so many
  const bool listed = near <= kListMax;
  if (near > need) {
    if (listed) {
      for (int i = warp; i < near; i += kPickThreads / 32) {
        const double s = exact_score<kBf16>(a, b, t, c, sh.list[i]);
        if (lane == 0) sh.val[i] = isnan(s) ? -INFINITY : s;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < near; i += kPickThreads) {
        const double s = sh.val[i];
        const int me = sh.list[i];
        int rank = 0;
        for (int j = 0; j < near; ++j)
          rank += sh.val[j] > s || (sh.val[j] == s && sh.list[j] < me);
        exact[me] = rank < need ? 1.0 : 0.0;
      }
      __syncthreads();
    } else {
      for (int i = warp; i < n; i += kPickThreads / 32) {
        if (cls(score[i]) != 1) continue;
        const double s = exact_score<kBf16>(a, b, t, c, i);
        if (lane == 0) exact[i] = isnan(s) ? -INFINITY : s + 0.0;
      }
      __syncthreads();
      const uint64_t key = kth_largest<uint64_t>(
          n, need,
          [&](int i, uint64_t* kk) {
            if (cls(score[i]) != 1) return false;
            *kk = key_of(exact[i]);
            return true;
          },
          sh);
      cut = __longlong_as_double(key >> 63 ? key & ~(1ull << 63) : ~key);
      ties = sh.left;
    }
  }
  // Ascending: scan the flags, kPickThreads blocks at a time.
  if (threadIdx.x == 0) sh.base = 0;
  int tied = 0;  // blocks equal to the cut in earlier rounds
  for (int i0 = 0; i0 < n; i0 += kPickThreads) {
    const int i = i0 + threadIdx.x;
    const int x = i < n ? cls(score[i]) : 0;
    bool take = x == 2;
    bool tie = false;
    if (x == 1) {
      if (near <= need)
        take = true;
      else if (listed)
        take = exact[i] != 0.0;
      else {
        take = exact[i] > cut;
        tie = exact[i] == cut;
      }
    }
    if (!listed && near > need) {
      const uint32_t m = __ballot_sync(0xffffffffu, tie);
      if (lane == 0) sh.warp[warp] = __popc(m);
      __syncthreads();
      int before = tied, all = 0;
      for (int w = 0; w < kPickThreads / 32; ++w) {
        before += w < warp ? sh.warp[w] : 0;
        all += sh.warp[w];
      }
      tied += all;
      take |= tie && before + __popc(m & ((1u << lane) - 1u)) < ties;
      __syncthreads();
    }
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (lane == 0) sh.warp[warp] = __popc(m);
    __syncthreads();
    int before = sh.base, all = 0;
    for (int w = 0; w < kPickThreads / 32; ++w) {
      before += w < warp ? sh.warp[w] : 0;
      all += sh.warp[w];
    }
    const int at = before + __popc(m & ((1u << lane) - 1u));
    if (take && at < k) sel[at] = i;
    __syncthreads();
    if (threadIdx.x == 0) sh.base += all;
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_scores(const CacheSelectArgs& a, cudaStream_t st) {
  const dim3 grid((a.s.max_blocks + kScoreBlocks - 1) / kScoreBlocks, a.c.Hkv, a.s.batch);
  if (a.bf16)
    cache_score_kernel<D, true><<<grid, kScoreThreads, 0, st>>>(a);
  else
    cache_score_kernel<D, false><<<grid, kScoreThreads, 0, st>>>(a);
  return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_cache_select(const CacheSelectArgs& a, cudaStream_t st) {
  cudaError_t e = a.c.d == 128 ? launch_scores<128>(a, st) : launch_scores<64>(a, st);
  if (e != cudaSuccess) return e;
  const dim3 units(static_cast<unsigned>(a.s.batch) * a.T * a.c.Hkv);
  return launch_after(a.bf16 ? cache_pick_kernel<true> : cache_pick_kernel<false>, units,
                      kPickThreads, 0, st, true, a);
}

}  // namespace msa
