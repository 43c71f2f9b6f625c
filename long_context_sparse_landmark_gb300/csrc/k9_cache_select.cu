// K9: which blocks of the cache each query token attends -- the decode-time
// form of the landmark-scored selection (msa_block_select takes 128 rows
// together).
//
// For query token t of sequence b and KV group c, block l (full, wholly
// before the window) scores sum over the group's heads h of <q_h, kmean_l>;
// the top_k best are chosen, ties to the lower block.  The result is that of
// the sum in 64 bits: the scores are computed in fp32 with a bound of their
// rounding each, E_l = (g + 16) 2^-24 |sum_h |q_h||_2 |kmean_l|_2 (the sum over
// g heads rounds g times, a lane's 8 products of each 32 dims 8 times, and
// four joins follow; each is relative to sum_d (sum_h |q_h|) |kmean_l| at most,
// which the norms bound, each with kNormLost more for the squares that
// fall below fp32); only the blocks whose score is
// within 2 max E of the k-th are computed again in 64 bits.  So the choice
// does not depend on the order of any fp32 sum.
//
// The block means are read once for all query tokens of a sequence: 2 d
// bytes a block and KV head, four lanes a block with four 16-byte loads in
// flight each.  The choice is one CTA a (token, group), whose warps have
// contiguous runs of the blocks with their keys in shared memory: a radix
// selection of the k-th score by 11 + 11 + 10 bits, then a pass of ballots
// that writes the chosen in order; what bounds it is the chain of barriers.
// 508 blocks of 8 heads: scores 3.9 us, choice 5.6 (5.0 and 7.7 one by one with
// cold caches); 104104 blocks and heads (16 sequences of 38K to 65K slots, 2 tokens
// each, 27 MB of means): 15 and 12, of which 2 for the CTAs that have to score in
// 64 bits.
#include <math.h>

#include "cache_common.cuh"

namespace msa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = kScoreThreads / 4;  // blocks a CTA scores at a time
constexpr int kScoreT = 4;                       // query tokens taken together
// What a norm of 128 values may lack by squares that are flushed or rounded below
// 2^-126: sqrt(128 * 2^-126).
constexpr float kNormLost = 0x1p-59f;
constexpr int kPickWarpsMax = 16;
constexpr int kBins = 2048;
constexpr int kListMax = 512;          // near-ties ranked in shared memory
constexpr int kStagedMax = 40 * 1024;  // keys in shared memory; more are kept in the workspace
constexpr int kFewMax = 4096;          // blocks of a list that 256 threads take

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

// blockIdx = (share of the tiles of 64 blocks, KV head, sequence).  A tile's
// means are under way while the one before is scored, and its pages are looked
// up one tile earlier still.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const CacheSelectArgs a) {
  __shared__ __align__(16) float qs[kScoreT][D], qa[kScoreT][D];
  __shared__ float norm[kScoreT];  // of qa, times the bound's factor
  let_next_start();
  const int c = blockIdx.y, b = blockIdx.z, g = a.Hq / a.c.Hkv;
  const int step = gridDim.x * kScoreBlocks;
  const int l0 = blockIdx.x * kScoreBlocks + (threadIdx.x >> 2), lane4 = threadIdx.x & 3;
  const float eps = (g + 16) * 5.9604645e-8f * 1.001f;  // with room for its own rounding
  const int32_t* table = a.s.table + static_cast<int64_t>(b) * a.s.max_blocks;
  const auto entry = [&](int l) { return l < a.s.max_blocks ? table[l] : -1; };
  int32_t page1 = entry(l0);  // not looked at unless the block is a candidate
  const int len = cache_len(a.s, b, a.c.block, a.status);
  const int most = candidates(a, len, a.T - 1);  // the last token sees the most
  if (static_cast<int>(blockIdx.x) * kScoreBlocks >= most) return;
  struct Mean {
    uint4 x[D / 32];  // 16-byte pieces of a mean: d = 32 i + 8 lane4 + 0..7
  };
  const auto fetch = [&](int l, int32_t page) {
    Mean k;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) k.x[i] = make_uint4(0, 0, 0, 0);
    if (l < most) {
      if (page < 0 || page >= a.c.n_pages) {
        record_status(a.status, MSA_ERR_INVALID_ARG);
        page = 0;
      }
      const uint4* src = reinterpret_cast<const uint4*>(
          a.c.k_mean + (static_cast<int64_t>(page) * a.c.Hkv + c) * D);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) k.x[i] = __ldg(src + 4 * i + lane4);
    }
    return k;
  };
  for (int t0 = 0; t0 < a.T; t0 += kScoreT) {
    const int nt = min(kScoreT, a.T - t0);
    if (t0 > 0) page1 = entry(l0);
    Mean next = fetch(l0, page1);
    page1 = entry(l0 + step);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * D; i += kScoreThreads) {
      const int t = i / D, e = i - t * D;
      const int64_t at = ((static_cast<int64_t>(b) * a.T + t0 + t) * a.Hq + c * g) * D + e;
      float s = 0.f, m = 0.f;
#pragma unroll 8
      for (int h = 0; h < g; ++h) {
        const float x = q_at<kBf16>(a.q, at + static_cast<int64_t>(h) * D);
        s += x;
        m += fabsf(x);
      }
      qs[t][e] = s;
      qa[t][e] = m;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x >> 5) < nt) {
      const int t = threadIdx.x >> 5;
      float n2 = 0.f;
      for (int e = threadIdx.x & 31; e < D; e += 32) n2 = fmaf(qa[t][e], qa[t][e], n2);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      if ((threadIdx.x & 31) == 0) norm[t] = (sqrtf(n2) + kNormLost) * eps;
    }
    __syncthreads();
    for (int l = l0; l - (static_cast<int>(threadIdx.x) >> 2) < most; l += step) {
      const Mean km = next;
      next = fetch(l + step, page1);
      page1 = entry(l + 2 * step);
      float k2 = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {km.x[i].x, km.x[i].y, km.x[i].z, km.x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = __uint_as_float(w[k] << 16);
          const float hi = __uint_as_float(w[k] & 0xffff0000u);
          k2 = fmaf(lo, lo, fmaf(hi, hi, k2));
        }
      }
      k2 += __shfl_xor_sync(0xffffffffu, k2, 1);
      k2 += __shfl_xor_sync(0xffffffffu, k2, 2);
      const float k_norm = sqrtf(k2) + kNormLost;
      for (int t = 0; t < nt; ++t) {
        float s[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const float4 q0 = *reinterpret_cast<const float4*>(&qs[t][32 * i + 8 * lane4]);
          const float4 q1 = *reinterpret_cast<const float4*>(&qs[t][32 * i + 8 * lane4 + 4]);
          const uint4 w = km.x[i];
          s[i] = q0.x * __uint_as_float(w.x << 16);
          s[i] = fmaf(q0.y, __uint_as_float(w.x & 0xffff0000u), s[i]);
          s[i] = fmaf(q0.z, __uint_as_float(w.y << 16), s[i]);
          s[i] = fmaf(q0.w, __uint_as_float(w.y & 0xffff0000u), s[i]);
          s[i] = fmaf(q1.x, __uint_as_float(w.z << 16), s[i]);
          s[i] = fmaf(q1.y, __uint_as_float(w.z & 0xffff0000u), s[i]);
          s[i] = fmaf(q1.z, __uint_as_float(w.w << 16), s[i]);
          s[i] = fmaf(q1.w, __uint_as_float(w.w & 0xffff0000u), s[i]);
        }
        float sum = s[0] + s[1];
        if constexpr (D == 128) sum += s[2] + s[3];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (lane4 == 0 && l < most && MSA_IN_RANGE(l, 1, a.s.max_blocks, a.status)) {
          const int64_t at =
              ((static_cast<int64_t>(b) * a.T + t0 + t) * a.c.Hkv + c) * a.s.max_blocks + l;
          a.score[at] = sum;
          a.err[at] = k_norm * norm[t];  // not finite: asks for 64 bits
        }
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
  int hist[3][kBins];
  int warp[kPickWarpsMax], warp2[kPickWarpsMax];
  int digit, left;
  int n_list;
  int list[kListMax];
  double val[kListMax];
  float emax[kPickWarpsMax];
};

// In hist, the bin that holds the `left`-th largest key (bins fall as keys
// do); sh.digit and sh.left, the keys still wanted of that bin.
template <int kThreads>
__device__ __forceinline__ void find_bin(const int* hist, int left, PickShared& sh) {
  constexpr int kOwn = kBins / kThreads;  // bins of a thread, the first has the highest
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = kOwn * (kThreads - 1 - threadIdx.x);
  int bin[kOwn], sum = 0;
#pragma unroll
  for (int i = 0; i < kOwn; i += 4) {
    const int4 s = *reinterpret_cast<const int4*>(hist + at + i);
    bin[i] = s.x;
    bin[i + 1] = s.y;
    bin[i + 2] = s.z;
    bin[i + 3] = s.w;
    sum += s.x + s.y + s.z + s.w;
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sh.warp[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kThreads / 32; ++v) upto += v < warp ? sh.warp[v] : 0;
  int before = upto - sum;
  if (before < left && left <= upto) {
#pragma unroll
    for (int k = kOwn - 1; k >= 0; --k) {
      if (before < left && left <= before + bin[k]) {
        sh.digit = at + k;
        sh.left = left - before;
      }
      before += bin[k];
    }
  }
  __syncthreads();
}

// kN consecutive values of a row as floats, in one load.
template <int kN, bool kBf16>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float* v) {
  if constexpr (kBf16) {
    const uint16_t* src = static_cast<const uint16_t*>(p) + at;
    uint32_t w[kN / 2];
    if constexpr (kN == 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(src);
      w[0] = x.x;
      w[1] = x.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(src);
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at + i);
      v[i] = x.x;
      v[i + 1] = x.y;
    }
  }
}

// Score of block l in 64 bits, by one warp, a lane D/32 dims.  The sum over
// the heads is kept as an fp32 value and the exact error of each addition (the
// error-free sum of two floats); the errors' own sum may round, 2^-48 g of the
// sum of magnitudes at most, where heads differ by many binades.  That spares
// most of the 64-bit operations, each 16 cycles of an SM for a warp; left are
// the products, their sum, and heads whose sum is beyond fp32.  Eight heads'
// loads go together.
template <int D, bool kBf16>
__device__ __forceinline__ double exact_score(const CacheSelectArgs& a, int b, int t, int c,
                                              int l) {
  constexpr int kN = D / 32;
  const int lane = threadIdx.x & 31, g = a.Hq / a.c.Hkv;
  int64_t page = cache_page(a.s, b, l, a.c.n_pages, a.status);
  page = page < 0 ? 0 : page;
  float km[kN];
  load_row<kN, true>(a.c.k_mean, (page * a.c.Hkv + c) * D + kN * lane, km);
  const int64_t q0 = ((static_cast<int64_t>(b) * a.T + t) * a.Hq + c * g) * D + kN * lane;
  float sum[kN], rest[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) sum[i] = rest[i] = 0.f;
  for (int h0 = 0; h0 < g; h0 += 8) {
    float q[8][kN];
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h0 + h < g) load_row<kN, kBf16>(a.q, q0 + static_cast<int64_t>(h0 + h) * D, q[h]);
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h0 + h < g)
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float x = q[h][i], t = sum[i] + x, b = t - sum[i];
          rest[i] += (sum[i] - (t - b)) + (x - b);
          sum[i] = t;
        }
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const double k = km[i];
    double x = sum[i];
    if (!isfinite(sum[i])) {
      x = 0.0;
      for (int h = 0; h < g; ++h)
        x += static_cast<double>(q_at<kBf16>(a.q, q0 + static_cast<int64_t>(h) * D + i));
    }
    s += x * k;
    if (rest[i] != 0.f && isfinite(sum[i])) s += static_cast<double>(rest[i]) * k;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One CTA a (token, KV head).  kStaged: the keys are in shared memory, else
// in the place of the scores' error bounds in the workspace.
template <int D, bool kBf16, bool kStaged, int kPickThreads>
__global__ void __launch_bounds__(kPickThreads, 1024 / kPickThreads)
    cache_pick_kernel(const CacheSelectArgs a) {
  constexpr int kPickWarps = kPickThreads / 32;
  __shared__ __align__(16) PickShared sh;
  extern __shared__ uint32_t staged[];
  const int c = blockIdx.x % a.c.Hkv, bt = blockIdx.x / a.c.Hkv;
  const int b = bt / a.T, t = bt - b * a.T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t u = static_cast<int64_t>(bt) * a.c.Hkv + c;
  let_next_start();
  const int n = candidates(a, cache_len(a.s, b, a.c.block, a.status), t);
  int32_t* sel = a.sel + u * a.top_k;
  const int k = min(a.top_k, n);
#pragma unroll
  for (int i = 0; i < 3 * kBins; i += 4 * kPickThreads)
    *reinterpret_cast<int4*>(&sh.hist[0][i + 4 * threadIdx.x]) = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) sh.n_list = 0;
  wait_for_inputs();
  if (threadIdx.x == 0) a.cnt[u] = k;
  for (int i = k + threadIdx.x; i < a.top_k; i += kPickThreads) sel[i] = -1;
  if (k == n) {
    for (int i = threadIdx.x; i < n; i += kPickThreads) sel[i] = i;
    return;
  }
  const float* score = a.score + u * a.s.max_blocks;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.err + u * a.s.max_blocks);
  uint32_t* keys = kStaged ? staged : err;
  // The warp's blocks [i0, i1): whole groups of 32, the last of all cut short.
  const int per = ((n + kPickWarps - 1) / kPickWarps + 31) & ~31;
  const int i0 = min(n, warp * per), i1 = min(n, i0 + per);

  float em = 0.f;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const float e = __uint_as_float(err[i]);
    em = fmaxf(em, isnan(e) ? INFINITY : e);
    keys[i] = key_of(score[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) em = fmaxf(em, __shfl_xor_sync(0xffffffffu, em, o));
  if (lane == 0) sh.emax[warp] = em;
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
  int left = k;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bits = pass == 2 ? 0x3ffu : 0x7ffu;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint32_t key = keys[i];
      if ((key & mask) == prefix) atomicAdd(&sh.hist[pass][(key >> shift) & bits], 1);
    }
    __syncthreads();
    find_bin<kPickThreads>(sh.hist[pass], left, sh);
    prefix |= static_cast<uint32_t>(sh.digit) << shift;
    mask |= bits << shift;
    left = sh.left;
    __syncthreads();
  }
  const float kth = value_of(prefix);
  em = sh.emax[0];
#pragma unroll
  for (int w = 1; w < kPickWarps; ++w) em = fmaxf(em, sh.emax[w]);
  // Twice the bound on either side, widened for the roundings of these two;
  // keys above `above` are chosen whatever the rest, keys from `below` on are
  // near the k-th.  Where a side is not a number (infinite scores or bounds)
  // all are near.
  const float room = 2.0001f * em + fabsf(kth) * 2.4e-7f + 1e-38f;
  const float hi = kth + room, lo = kth - room;
  const uint32_t above = isnan(hi) ? 0xffffffffu : key_of(hi);
  const uint32_t below = isnan(lo) ? 0u : key_of(lo);
  int sure = 0, near = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t key = keys[i];
    sure += key > above;
    if (key <= above && key >= below) {
      const int at = atomicAdd(&sh.n_list, 1);
      if (at < kListMax) sh.list[at] = i;  // in any order: ranked by value, then block
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  if (lane == 0) sh.warp[warp] = sure;
  __syncthreads();
  sure = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) sure += sh.warp[w];
  near = sh.n_list;
  const int need = k - sure;
  // Keys from `from` on are chosen; near ones get the key of one that is, or
  // 0, where not all of them are.
  uint32_t from = below;
  if (near > need) {
    constexpr uint32_t kTaken = 0xffffffffu;
    from = above == kTaken ? kTaken : above + 1;
    if (near <= kListMax) {
      for (int i = warp; i < near; i += kPickWarps) {
        const double s = exact_score<D, kBf16>(a, b, t, c, sh.list[i]);
        if (lane == 0) sh.val[i] = isnan(s) ? -INFINITY : s;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < near; i += kPickThreads) {
        const double s = sh.val[i];
        const int me = sh.list[i];
        int rank = 0;
        for (int j = 0; j < near; ++j)
          rank += sh.val[j] > s || (sh.val[j] == s && sh.list[j] < me);
        keys[me] = rank < need ? kTaken : 0u;
      }
    } else {
      // More than the list holds (equal blocks): 64-bit scores in the
      // workspace, and a selection among them by six digits.
      double* exact = a.exact + u * a.s.max_blocks;
      for (int i = i0; i < i1; ++i) {
        if (keys[i] > above || keys[i] < below) continue;
        const double s = exact_score<D, kBf16>(a, b, t, c, i);
        if (lane == 0) exact[i] = isnan(s) ? -INFINITY : s + 0.0;
      }
      uint64_t found = 0, known = 0;
      int want = need;
      for (int shift = 55; shift >= 0; shift -= 11) {
        constexpr uint64_t bits = 0x7ff;
        __syncthreads();
        for (int i = 4 * threadIdx.x; i < kBins; i += 4 * kPickThreads)
          *reinterpret_cast<int4*>(&sh.hist[0][i]) = make_int4(0, 0, 0, 0);
        __syncthreads();
        for (int i = i0 + lane; i < i1; i += 32)
          if (keys[i] <= above && keys[i] >= below) {
            const uint64_t key = key_of(exact[i]);
            if ((key & known) == found)
              atomicAdd(&sh.hist[0][static_cast<int>((key >> shift) & bits)], 1);
          }
        __syncthreads();
        find_bin<kPickThreads>(sh.hist[0], want, sh);
        found |= static_cast<uint64_t>(sh.digit) << shift;
        known |= bits << shift;
        want = sh.left;
      }
      // Of the scores equal to the last one in, the `want` lowest blocks.
      int ties = 0;
      for (int i = i0 + lane; i < i1; i += 32)
        ties += keys[i] <= above && keys[i] >= below && key_of(exact[i]) == found;
      ties = __reduce_add_sync(0xffffffffu, ties);
      __syncthreads();
      if (lane == 0) sh.warp2[warp] = ties;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += sh.warp2[w];
      for (int j = i0; j < i1; j += 32) {
        const int i = j + lane;
        const bool is_near = i < i1 && keys[i] <= above && keys[i] >= below;
        const uint64_t key = is_near ? key_of(exact[i]) : 0;
        const bool tie = is_near && key == found;
        const uint32_t m = __ballot_sync(0xffffffffu, tie);
        if (is_near) {
          const bool take =
              key > found || (tie && before + __popc(m & ((1u << lane) - 1u)) < want);
          keys[i] = take ? kTaken : 0u;
        }
        before += __popc(m);
      }
    }
    __syncthreads();
  }
  // Ascending: each warp's run starts after those of the warps before.
  int mine = 0;
  for (int i = i0 + lane; i < i1; i += 32) mine += keys[i] >= from;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sh.warp2[warp] = mine;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) at += w < warp ? sh.warp2[w] : 0;
  for (int j = i0; j < i1; j += 32) {
    const int i = j + lane;
    const bool take = i < i1 && keys[i] >= from;
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    const int to = at + __popc(m & ((1u << lane) - 1u));
    if (take && to < k && MSA_IN_RANGE(u * a.top_k + to, 1,
                                       static_cast<int64_t>(gridDim.x) * a.top_k, a.status))
      sel[to] = i;
    at += __popc(m);
  }
}

template <int D>
cudaError_t launch_scores(const CacheSelectArgs& a, cudaStream_t st) {
  // CTAs that the device holds at once, each with as many tiles as that leaves.
  const int64_t tiles = (a.s.max_blocks + kScoreBlocks - 1) / kScoreBlocks;
  const int64_t others = static_cast<int64_t>(a.c.Hkv) * a.s.batch;
  const int64_t x = min64(tiles, max64(1, kSms * 3 / others));
  const dim3 grid(static_cast<unsigned>(x), a.c.Hkv, a.s.batch);
  return launch_after(a.bf16 ? cache_score_kernel<D, true> : cache_score_kernel<D, false>, grid,
                      kScoreThreads, 0, st, false, a);
}

template <int D, bool kBf16>
cudaError_t launch_pick(const CacheSelectArgs& a, cudaStream_t st) {
  // 256 threads up to kFewMax blocks, whose few keys leave most instructions to
  // the bins and barriers, 512 above.
  const bool few = a.s.max_blocks <= kFewMax, staged = a.s.max_blocks <= kStagedMax;
  const int smem = staged ? a.s.max_blocks * 4 : 0;
  const auto kernel = few      ? cache_pick_kernel<D, kBf16, true, 256>
                      : staged ? cache_pick_kernel<D, kBf16, true, 512>
                               : cache_pick_kernel<D, kBf16, false, 512>;
  static_assert(sizeof(PickShared) + kFewMax * 4 <= 48 * 1024, "few: no leave needed");
  if (staged && !few) {
    // More than 48 KB needs leave: for the kernel's most, not this call's, since
    // the limit is the function's and another host thread may launch between
    // this and the launch below.
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedMax * 4);
    if (e != cudaSuccess) return e;
  }
  const dim3 units(static_cast<unsigned>(a.s.batch) * a.T * a.c.Hkv);
  return launch_after(kernel, units, few ? 256 : 512, smem, st, true, a);
}

}  // namespace

cudaError_t launch_cache_select(const CacheSelectArgs& a, cudaStream_t st) {
  cudaError_t e = a.c.d == 128 ? launch_scores<128>(a, st) : launch_scores<64>(a, st);
  if (e != cudaSuccess) return e;
  if (a.c.d == 128) return a.bf16 ? launch_pick<128, true>(a, st) : launch_pick<128, false>(a, st);
  return a.bf16 ? launch_pick<64, true>(a, st) : launch_pick<64, false>(a, st);
}

}  // namespace msa
