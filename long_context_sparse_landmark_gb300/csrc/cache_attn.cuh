// Attention of a few query tokens over a paged KV cache: what the kernels of the
// 8-bit and the 4-bit cache share -- the list of chunks and its cut, the output,
// and the join of the units that several CTAs take.
#pragma once

#include <math.h>

#include "cache_common.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPBits = 14.f;  // log2 of the largest half weight
// log2 of a value scale of 0 (finite: no difference of two is a NaN).  Such a
// block counts in the denominator; its values weigh nothing beside any others,
// and what they leave where there are no others is scaled to 0 in the end.
constexpr float kLogZero = -0x1p126f;

// ---- the list of chunks ----------------------------------------------------

// Entry i of the outer list: a sequence (dense), or a query token of one
// (selected blocks).  Its Hkv * n_tiles units have the same chunks.
struct Entry {
  int b, t;      // sequence, query token (dense: 0)
  int len;       // slots held, the query tokens' own among them
  int win0;      // first slot of the window part, a multiple of kChunk
  int n_sel;     // selected blocks
  int n_cand;    // blocks that may be selected
  int n_chunks;  // of selected blocks, then of the window
};

__device__ __forceinline__ Entry entry_at(const CacheAttnArgs& a, int i) {
  Entry e;
  e.b = a.sel ? i / a.T : i;
  e.t = a.sel ? i - e.b * a.T : 0;
  e.len = cache_len(a.s, e.b, a.c.block, a.status);
  const int p0 = e.len - a.T + e.t;       // first row's position
  const int p1 = a.sel ? p0 : e.len - 1;  // last row's
  const int lo = max(0, p0 - a.window + 1);
  e.win0 = lo / kChunk * kChunk;
  e.n_cand = e.n_sel = 0;
  if (a.sel && p0 >= a.window) {
    e.n_cand = (p0 - a.window + 1) >> a.c.lb;
    e.n_sel = min(a.top_k, e.n_cand);
  }
  e.n_chunks = p1 < 0 ? 0 : (e.n_sel << (a.c.lb - kChunkLog2)) + (p1 - e.win0) / kChunk + 1;
  return e;
}

struct Plan {
  int n_entries, units;  // units an entry: Hkv * n_tiles
  int rows, n_tiles;     // query rows of a unit's entry, and their tiles
};

__device__ __forceinline__ Plan plan_of(const CacheAttnArgs& a, int tile) {
  Plan p;
  const int g = a.Hq / a.c.Hkv;
  p.n_entries = a.sel ? a.s.batch * a.T : a.s.batch;
  p.rows = a.sel ? g : a.T * g;
  p.n_tiles = (p.rows + tile - 1) / tile;
  p.units = a.c.Hkv * p.n_tiles;
  return p;
}

// Inclusive sum over the CTA's kNw warps; all threads get the total in *total.
template <int kNw>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* smem, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kNw; ++w) {
    before += w < warp ? smem[w] : 0;
    all += smem[w];
  }
  *total = all;
  return x + before;
}

// The chunks of all entries; up to a CTA of them are read once.
struct Scan {
  uint32_t total;   // chunks of one unit of every entry
  uint32_t first;   // this thread's entry: chunks before it (one unit an entry)
  uint32_t n;       // and its own
};
template <int kNw>
__device__ __forceinline__ Scan scan_entries(const CacheAttnArgs& a, const Plan& p, uint32_t* smem) {
  Scan r;
  uint32_t more = 0;
  r.n = static_cast<int>(threadIdx.x) < p.n_entries ? entry_at(a, threadIdx.x).n_chunks : 0;
  for (int i = threadIdx.x + 32 * kNw; i < p.n_entries; i += 32 * kNw)
    more += entry_at(a, i).n_chunks;
  uint32_t first_total, rest = 0;
  r.first = block_scan<kNw>(r.n, smem, &first_total) - r.n;
  if (p.n_entries > 32 * kNw) block_scan<kNw>(more, smem, &rest);
  r.total = first_total + rest;
  return r;
}

// Calls hit(i, before, n) in the thread of each entry: its index, the chunks
// (one unit an entry) before it and its own.
template <int kNw, typename Hit>
__device__ __forceinline__ void each_entry(const CacheAttnArgs& a, const Plan& p, const Scan& s,
                                           uint32_t* smem, Hit hit) {
  if (static_cast<int>(threadIdx.x) < p.n_entries) hit(threadIdx.x, s.first, s.n);
  if (p.n_entries <= 32 * kNw) return;
  uint32_t before = 0;
  for (int i0 = 0; i0 < p.n_entries; i0 += 32 * kNw) {
    const int i = i0 + threadIdx.x;
    const uint32_t n = i < p.n_entries ? entry_at(a, i).n_chunks : 0;
    uint32_t total;
    const uint32_t upto = before + block_scan<kNw>(n, smem, &total);
    if (i0 > 0 && i < p.n_entries) hit(i, upto - n, n);
    before += total;
  }
}

// The W chunks of all units, cut into P ranges, one a CTA: the first W % P
// have one chunk more.  A CTA's warps take at least one chunk each in fp32, two
// in bf16, where a second chunk costs less than the parts to join (one sequence
// of 32K slots, one KV head: 13.1 us with one, 11.7 with two; fp32 with 2K
// slots: 13.8 with one, 17.2 with two) -- unless that is more than a unit: a
// unit's rows and sums cost a CTA more than its chunks (200 units of one chunk,
// 24 rows: 84 us at eight units a CTA, 14 at one).  W fits 31 bits (the entry
// points check).
struct Cut {
  uint32_t P, each, more;
};
__device__ __forceinline__ Cut cut_of(const CacheAttnArgs& a, const Plan& p, uint32_t W) {
  Cut k;
  const uint32_t least = a.in_bf16 ? 2 * kWarps : kWarps;
  const uint32_t units = static_cast<uint32_t>(p.n_entries) * p.units;
  k.P = max(1u, min(static_cast<uint32_t>(a.n_ctas), min(W, max((W + least - 1) / least, units))));
  k.each = W / k.P;
  k.more = W - k.each * k.P;
  return k;
}
__device__ __forceinline__ uint32_t cta_begin(const Cut& k, uint32_t p) {
  return p * k.each + min(p, k.more);
}
// The CTA whose range holds chunk x.
__device__ __forceinline__ uint32_t cta_of(const Cut& k, uint32_t x) {
  const uint32_t longer = k.more * (k.each + 1);
  return x < longer ? x / (k.each + 1) : k.more + (x - longer) / k.each;
}

__device__ __forceinline__ void copy_async16(void* smem, const void* global) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
}

// ---- pieces of the tensor-core body ---------------------------------------

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^x, within 2 ulp; results below the normal range are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// 2^x as a product, applied one after the other (and apart from a denominator
// of up to 2^91): for x down to -226, where a result in fp32's range is left of
// a sum times 2^x although 2^x is not.
struct Pow2 {
  float a, b;
};
__device__ __forceinline__ Pow2 pow2_of(float x) {
  return {ex2(fmaxf(x, -100.f)), ex2(fminf(x + 100.f, 0.f))};
}

// Row m of an entry: its query token and head.
__device__ __forceinline__ void row_of(const CacheAttnArgs& a, const Entry& e, int c, int m,
                                       int* t, int* h) {
  const int g = a.Hq / a.c.Hkv;
  *t = a.sel ? e.t : m / g;
  *h = c * g + (a.sel ? m : m % g);
}

// The joined result of a CTA's warps for one unit's range, or a whole unit.
// Row r: osum[w][r][dim] holds warp w's sum in units of 2^{M + D}, stat[w][r]
// its references and denominator, l in units of 2^M.
struct Stat {
  float M, D, l;
};

// Writes row m's lse and, for the weights pass, its reference and denominator.
__device__ __forceinline__ void store_lse(const CacheAttnArgs& a, const Plan& p, const Entry& e,
                                          int c, int m, float mx, float l) {
  int t, h;
  row_of(a, e, c, m, &t, &h);
  const int64_t at = (static_cast<int64_t>(e.b) * a.Hq + h) * a.T + t;
  if (MSA_IN_RANGE(at, 1, static_cast<int64_t>(a.s.batch) * a.Hq * a.T, a.status))
    a.lse[at] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
  if (a.weights) {
    const int even = (p.rows + 1) & ~1;
    a.row_stat[(static_cast<int64_t>(e.b) * a.c.Hkv + c) * even + m] =
        make_float2(mx, l == 0.f ? 0.f : 1.f / l);
  }
}
__device__ __forceinline__ void store_out(const CacheAttnArgs& a, const Entry& e, int c, int m,
                                          int dim, float4 v) {
  int t, h;
  row_of(a, e, c, m, &t, &h);
  const int64_t at = ((static_cast<int64_t>(e.b) * a.T + t) * a.Hq + h) * a.c.d + dim;
  if (!MSA_IN_RANGE(at, 4, static_cast<int64_t>(a.s.batch) * a.T * a.Hq * a.c.d, a.status)) return;
  if (a.out_bf16) {
    __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<uint32_t*>(&x);
    w.y = *reinterpret_cast<uint32_t*>(&y);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
  }
}

// kN dims of a row, times f.
template <int kN>
__device__ __forceinline__ void store_dims(const CacheAttnArgs& a, const Entry& e, int c, int m,
                                           int dim, const float* v, float f) {
  if constexpr (kN == 4) {
    store_out(a, e, c, m, dim, make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f));
  } else {
    int t, h;
    row_of(a, e, c, m, &t, &h);
    const int64_t at = ((static_cast<int64_t>(e.b) * a.T + t) * a.Hq + h) * a.c.d + dim;
    if (!MSA_IN_RANGE(at, 2, static_cast<int64_t>(a.s.batch) * a.T * a.Hq * a.c.d, a.status))
      return;
    if (a.out_bf16)
      *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          __floats2bfloat162_rn(v[0] * f, v[1] * f);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) =
          make_float2(v[0] * f, v[1] * f);
  }
}

// Place of a row's dim in the warps' sums [warp][row][D]: rows padded by 4
// floats, and every second group of D/8 dims with neighbouring 16-byte pieces
// swapped, so that the fragments' stores meet no bank twice.
template <int D>
__device__ __forceinline__ int sum_at(int row, int dim) {
  const int piece = dim >> 2;
  return row * (D + 4) + ((piece ^ (piece / (D / 32) & 1)) << 2) + (dim & 3);
}

// Joins the warps' sums of a unit's range and writes them: a thread a row for
// the statistics, which become each warp's factor, then all of them the dims.
// Of a range that is not whole the sums stay in units of their own: over its
// denominator, a range of little weight and great values would be lost when the
// ranges' weights are compared.
template <int D, int kTile>
__device__ __forceinline__ void join_warps(const CacheAttnArgs& a, const Plan& p, const Entry& e,
                                           int c, int rt, const float* osum, Stat* stat,
                                           bool whole, int64_t slot) {
  const int left = p.rows - rt * kTile;  // rows from the tile's first on
  if (static_cast<int>(threadIdx.x) < min(kTile, left)) {
    const int r = threadIdx.x;
    Stat s[kWarps];
    float mx = -INFINITY, l = 0.f, M = -INFINITY, D0 = 0.f;  // (M, D0): the largest M + D
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s[w] = stat[w * kTile + r];
      mx = fmaxf(mx, s[w].M);
      if ((s[w].M - M) + (s[w].D - D0) > 0.f) {
        M = s[w].M;
        D0 = s[w].D;
      }
    }
    mx = finite_or_0(mx);
    M = finite_or_0(M);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (!(s[w].M == -INFINITY && s[w].l == 0.f)) l += s[w].l * ex2(s[w].M - mx);
    const float unit = D0 - kPBits;
    const Pow2 to = pow2_of((M - mx) + unit);
    // l == 0: no slot attended.
    const float f = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      stat[w * kTile + r].l = s[w].M == -INFINITY && s[w].l == 0.f
                                  ? 0.f
                                  : ex2((finite_or_0(s[w].M) - M) + (s[w].D - D0)) * f;
    stat[r].M = whole ? to.a : 1.f;
    stat[r].D = whole ? to.b : 1.f;
    if (whole)
      store_lse(a, p, e, c, rt * kTile + r, mx, l);
    else
      // (a part that attends nothing: references below any other's)
      a.part_stat[slot * kTile + r] =
          l == 0.f ? make_float4(-INFINITY, 0.f, -1e38f, 0.f) : make_float4(mx, l, M, unit);
  }
  __syncthreads();
#pragma unroll 2
  for (int i = threadIdx.x; i < kTile * (D / 4); i += kThreads) {
    const int r = i / (D / 4), dim = (i - r * (D / 4)) * 4;
    if (r >= left) break;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = stat[w * kTile + r].l;
      const float4 x = *reinterpret_cast<const float4*>(osum + sum_at<D>(w * kTile + r, dim));
      v.x += x.x * f;
      v.y += x.y * f;
      v.z += x.z * f;
      v.w += x.w * f;
    }
    const Pow2 to{stat[r].M, stat[r].D};
    v.x = v.x * to.a * to.b;
    v.y = v.y * to.a * to.b;
    v.z = v.z * to.a * to.b;
    v.w = v.w * to.a * to.b;
    if (whole)
      store_out(a, e, c, rt * kTile + r, dim, v);
    else
      *reinterpret_cast<float4*>(a.o_part + (slot * kTile + r) * D + dim) = v;
  }
}

// Joins the parts of the units that several CTAs share, and writes the rows
// that attend nothing.  kWpr warps a row: 1 where a unit has a few parts (and
// 4 rows a CTA), 16 where it has many, every 16th part each (32K tokens of one
// KV head: 128 parts in 5.2 us; 256 parts took 5 with 16 warps, 12 with 4); a
// lane has D/32 dims.
constexpr int kJoinMany = 16;

template <int D, int kTile, int kWpr>
__global__ void __launch_bounds__(kWpr == 1 ? kThreads : 32 * kWpr)
    cache_attn_join_kernel(const CacheAttnArgs a) {
  constexpr int kDl = D / 32;
  constexpr int kWarpsJ = kWpr == 1 ? kWarps : kWpr, kRows = kWarpsJ / kWpr;
  __shared__ uint32_t scan[kWarpsJ];
  __shared__ uint32_t found[kRows];
  __shared__ float4 red[kWarpsJ];
  __shared__ __align__(16) float osum[kWarpsJ][kWpr == 1 ? 1 : D];
  const Plan p = plan_of(a, kTile);
  const int rows = a.c.Hkv * p.rows;  // of an entry, all KV heads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * kRows, all = p.n_entries * rows;  // fit: the entry points check
  const Scan sc = scan_entries<kWarpsJ>(a, p, scan);
  each_entry<kWarpsJ>(a, p, sc, scan, [&](int k, uint32_t before, uint32_t) {
#pragma unroll
    for (int w = 0; w < kRows; ++w)
      if ((row0 + w) / rows == k) found[w] = before;
  });
  __syncthreads();
  const int mine = kWpr == 1 ? warp : 0, part = kWpr == 1 ? 0 : warp;
  wait_for_inputs();  // every path: whoever waits for this kernel waits for the parts too
  if (row0 + mine >= all) return;
  const int i = (row0 + mine) / rows, cm = row0 + mine - i * rows;
  const int c = cm / p.rows, m = cm - c * p.rows, rt = m / kTile, r = m - rt * kTile;
  const Entry e = entry_at(a, i);
  if (e.n_chunks == 0) {
    if (part == 0 && lane < D / 4) store_out(a, e, c, m, 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f));
    if (part == 0 && lane == 0) store_lse(a, p, e, c, m, 0.f, 0.f);
    return;
  }
  const Cut cut = cut_of(a, p, sc.total * p.units);
  const uint32_t u0 = found[mine] * p.units + (c * p.n_tiles + rt) * e.n_chunks;
  const int c0 = cta_of(cut, u0), c1 = cta_of(cut, u0 + e.n_chunks - 1);
  if (c0 == c1) return;  // written whole
  const auto at = [&](int x) { return (2 * static_cast<int64_t>(x) + (x == c0)) * kTile + r; };
  // A warp's parts, kAhead of them loaded at once: the denominators in units of
  // 2^mx, the sums in units of 2^(ref + unit).
  constexpr int kAhead = kWpr == 1 ? 4 : 8;
  float mx = -INFINITY, l = 0.f, ref = -INFINITY, unit = 0.f, v[kDl];
#pragma unroll
  for (int k = 0; k < kDl; ++k) v[k] = 0.f;
#pragma unroll 1
  for (int x0 = c0 + part; x0 <= c1; x0 += kAhead * kWpr) {
    float4 of[kAhead], best[kAhead];
    float y[kAhead][kDl];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int x = x0 + j * kWpr;
      of[j] = make_float4(-INFINITY, 0.f, -1e38f, 0.f);
#pragma unroll
      for (int k = 0; k < kDl; ++k) y[j][k] = 0.f;
      if (x <= c1) {
        const int64_t s = at(x);
        of[j] = a.part_stat[s];
        const float* src = a.o_part + s * D + lane * kDl;
        if constexpr (kDl == 4) {
          const float4 z = *reinterpret_cast<const float4*>(src);
          y[j][0] = z.x, y[j][1] = z.y, y[j][2] = z.z, y[j][3] = z.w;
        } else {
          const float2 z = *reinterpret_cast<const float2*>(src);
          y[j][0] = z.x, y[j][1] = z.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) best[j] = of[j];
#pragma unroll
    for (int n = 1; n < kAhead; n *= 2)
#pragma unroll
      for (int j = 0; j < kAhead; j += 2 * n) {
        best[j].x = fmaxf(best[j].x, best[j + n].x);
        if ((best[j + n].z - best[j].z) + (best[j + n].w - best[j].w) > 0.f) {
          best[j].z = best[j + n].z;
          best[j].w = best[j + n].w;
        }
      }
    const float mn = fmaxf(mx, best[0].x), mu = finite_or_0(mn);
    l *= ex2(mx - mu);
    mx = mn;
    const float up = (best[0].z - ref) + (best[0].w - unit);
    if (up > 0.f) {
      const float down = ex2(-up);
#pragma unroll
      for (int k = 0; k < kDl; ++k) v[k] *= down;
      ref = best[0].z;
      unit = best[0].w;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      l += of[j].y * ex2(of[j].x - mu);
      const float f = ex2((of[j].z - ref) + (of[j].w - unit));
#pragma unroll
      for (int k = 0; k < kDl; ++k) v[k] += y[j][k] * f;
    }
  }
  if (kWpr > 1) {
#pragma unroll
    for (int k = 0; k < kDl; ++k) osum[warp][lane * kDl + k] = v[k];
    if (lane == 0) red[warp] = make_float4(mx, l, ref, unit);
    __syncthreads();
    if (warp > 0) return;
    const float4 own = red[lane < kWpr ? lane : 0];
    mx = own.x;
    ref = own.z;
    unit = own.w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float ref2 = __shfl_xor_sync(0xffffffffu, ref, o);
      const float unit2 = __shfl_xor_sync(0xffffffffu, unit, o);
      if ((ref2 - ref) + (unit2 - unit) > 0.f) {
        ref = ref2;
        unit = unit2;
      }
    }
    const float mu = finite_or_0(mx);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < kDl; ++k) v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kWpr; ++w) {
      const float4 of = red[w];
      l += of.y * ex2(of.x - mu);
      // No part (a warp without any): no reference.
      const float f = of.z == -INFINITY ? 0.f : ex2((of.z - ref) + (of.w - unit));
#pragma unroll
      for (int k = 0; k < kDl; ++k) v[k] += osum[w][lane * kDl + k] * f;
    }
  }
  mx = finite_or_0(mx);
  const Pow2 to = pow2_of((ref - mx) + unit);
  const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < kDl; ++k) v[k] = v[k] * f * to.a;
  store_dims<kDl>(a, e, c, m, lane * kDl, v, to.b);
  if (lane == 0) store_lse(a, p, e, c, m, mx, l);
}

// Puts the join behind the attention kernel.
template <int D, int kTile>
cudaError_t launch_join(const CacheAttnArgs& a, cudaStream_t st) {
  const int g = a.Hq / a.c.Hkv;
  const int rows = a.sel ? g : a.T * g;
  const int64_t all = static_cast<int64_t>(a.s.batch) * a.T * a.Hq;
  // Parts of a unit: at most about the CTAs over the units (all of them where
  // one sequence is long and the others are not).
  const int64_t units = static_cast<int64_t>(a.sel ? a.s.batch * a.T : a.s.batch) * a.c.Hkv *
                        ((rows + kTile - 1) / kTile);
  if (a.n_ctas > kJoinMany * units)
    return launch_after(cache_attn_join_kernel<D, kTile, kJoinMany>,
                        dim3(static_cast<unsigned>(all)), 32 * kJoinMany, 0, st, true, a);
  return launch_after(cache_attn_join_kernel<D, kTile, 1>,
                      dim3(static_cast<unsigned>((all + kWarps - 1) / kWarps)), kThreads, 0, st,
                      true, a);
}

}  // namespace
}  // namespace msa
