// K10: which slots an eviction keeps -- for each sequence and KV head the
// last `recent` slots and, of the others, those that drew the most
// attention, min(len, budget) in all, ties to the lower slot.  K7 then
// gathers them into fresh blocks.
//
// One cluster of CTAs a (sequence, KV head), each with a contiguous part of
// the slots, whose keys it keeps in shared memory: a radix selection of the
// least kept weight by 11 + 11 + 10 bits (histograms joined through the
// cluster's shared memory), then one pass of ballots that puts the kept slots
// in order.  Weights compare as they are: the choice is exact.  The first
// digit is sign, exponent and two bits of the mantissa, so that weights of a
// few binades do not all meet at a few counters.  The weights are read once
// (parts too long for shared memory: once a digit, from L2): 4 bytes a slot,
// against the 2 d bytes a kept slot costs in the gather.  A call is bound by
// latency: of the warps a scheduler has waiting per issue 4.7 wait for loads from
// global or another CTA's shared memory, 2.0 for fixed latencies, 1.6 at the ten or
// so barriers.  2273 to 4160 slots of 64 (sequence, head) pairs take 9.4 us,
// 131072 and 76276 of 8 heads each (clusters of 8) 29.
#include <math.h>

#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kKeysMax = 48 * 1024;  // of a CTA, in shared memory
constexpr int kBins = 2048;

// Unsigned key that orders as the weight does; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// And back (a -0 comes back as 0, a NaN as the standard one).
__device__ __forceinline__ float key_weight(uint32_t k) {
  if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// kStaged: the keys stay in shared memory (kKeysMax of them at most).
template <bool kStaged>
__global__ void __launch_bounds__(kEvictThreads) cache_evict_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ int digit, left_s;
  __shared__ int counts[2];  // this CTA's slots above the least kept weight, and equal to it
  __shared__ int wsum[2][kEvictWarps];
  let_next_start();
  cg::cluster_group cl = cg::this_cluster();
  const int ranks = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const auto sync_all = [&] {
    if (ranks > 1)
      cl.sync();
    else
      __syncthreads();
  };
  const int u = blockIdx.x / ranks;
  const int b = u / a.c.Hkv, h = u - b * a.c.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = cache_len(a.s, b, a.c.block, a.status);
  const int kept = static_cast<int>(min64(len, a.budget));
  const int recent = static_cast<int>(min64(kept, a.recent));
  const int n = len - recent;       // slots that compete
  const int need = kept - recent;   // and how many of them stay
  const float* w = a.weights + static_cast<int64_t>(u) * a.weights_ld;
  int32_t* out = a.kept + static_cast<int64_t>(u) * a.budget;
  float* out_w = a.new_weights + static_cast<int64_t>(u) * a.new_ld;
  // The warp's slots [i0, i1): whole groups of 32, the last of all cut short.
  // The launcher's kKeysMax covers what the rounding adds.
  const int warps = ranks * kEvictWarps;
  const int per = ((n + warps - 1) / warps + 31) & ~31;
  const int64_t from = static_cast<int64_t>(rank * kEvictWarps + warp) * per;
  const int i0 = static_cast<int>(min64(n, from)), i1 = static_cast<int>(min64(n, from + per));
  uint32_t* mine = keys + warp * per;

  const bool all = need == n;
  const bool pick = need > 0 && !all;  // the same for the whole cluster
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<int4*>(&hist[k][4 * threadIdx.x]) = make_int4(0, 0, 0, 0);
  if constexpr (kStaged) {
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) mine[i - i0] = weight_key(w[i]);
  }
  const auto key_at = [&](int i) { return kStaged ? mine[i - i0] : weight_key(w[i]); };
  // The warp's keys in any order, four a lane at a time from shared memory (a
  // run starts on a multiple of 32 keys).
  const auto each_key = [&](auto f) {
    if constexpr (kStaged) {
      const int n4 = (i1 - i0) & ~127;
#pragma unroll 2
      for (int i = 4 * lane; i < n4; i += 128) {
        const uint4 k = *reinterpret_cast<const uint4*>(mine + i);
        f(k.x);
        f(k.y);
        f(k.z);
        f(k.w);
      }
      for (int i = n4 + lane; i < i1 - i0; i += 32) f(mine[i]);
    } else {
      for (int i = i0 + lane; i < i1; i += 32) f(weight_key(w[i]));
    }
  };

  if (rank == 0 && threadIdx.x == 0 && h == 0) a.new_lens[b] = kept;
  // Past the kept: -1 and 0.
  for (int64_t i = kept + static_cast<int64_t>(rank) * kEvictThreads + threadIdx.x; i < a.new_ld;
       i += static_cast<int64_t>(ranks) * kEvictThreads) {
    if (i < a.budget) out[i] = -1;
    out_w[i] = 0.f;
  }
  // The recent ones.
  for (int i = rank * kEvictThreads + threadIdx.x; i < recent; i += ranks * kEvictThreads) {
    out[need + i] = n + i;
    out_w[need + i] = w[n + i];
  }

  uint32_t prefix = 0, mask = 0;
  int left = need;
  __syncthreads();
  if (pick) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bits = pass == 2 ? 0x3ffu : 0x7ffu;
      each_key([&](uint32_t k) {
        if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> shift) & bits], 1);
      });
      sync_all();
      // Thread t sums the bins 4 * (511 - t) + 3 .. + 0 of all ranks: the
      // threads' order is that of falling keys.
      const int at = 4 * (kEvictThreads - 1 - threadIdx.x);
      int4 s = *reinterpret_cast<const int4*>(&hist[pass][at]);
      if (ranks > 1) {
        int4 y[kClusterMax - 1];  // all under way at once
#pragma unroll
        for (int r = 1; r < kClusterMax; ++r)
          y[r - 1] = r < ranks ? *reinterpret_cast<const int4*>(
                                     cl.map_shared_rank(&hist[pass][0], (rank + r) & (ranks - 1)) + at)
                               : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 1; r < kClusterMax; ++r) {
          s.x += y[r - 1].x;
          s.y += y[r - 1].y;
          s.z += y[r - 1].z;
          s.w += y[r - 1].w;
        }
      }
      const int sum = s.x + s.y + s.z + s.w;
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) wsum[0][warp] = upto;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < kEvictWarps; ++v) upto += v < warp ? wsum[0][v] : 0;
      int before = upto - sum;
      if (before < left && left <= upto) {
        const int bin[4] = {s.w, s.z, s.y, s.x};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (before < left && left <= before + bin[k]) {
            digit = at + 3 - k;
            left_s = left - before;
          }
          before += bin[k];
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(digit) << shift;
      mask |= bits << shift;
      left = left_s;
      __syncthreads();
    }
  }
  // How many of this warp's slots lie above the least kept weight, and at it.
  int above = 0, equal = 0;
  if (need > 0) {
    each_key([&](uint32_t k) {
      above += all || k > prefix;
      equal += !all && k == prefix;
    });
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    wsum[0][warp] = above;
    wsum[1][warp] = equal;
  }
  __syncthreads();
  int before_above = 0, before_equal = 0, t_above = 0, t_equal = 0;
#pragma unroll
  for (int v = 0; v < kEvictWarps; ++v) {
    before_above += v < warp ? wsum[0][v] : 0;
    before_equal += v < warp ? wsum[1][v] : 0;
    t_above += wsum[0][v];
    t_equal += wsum[1][v];
  }
  if (ranks > 1) {
    if (threadIdx.x == 0) {
      counts[0] = t_above;
      counts[1] = t_equal;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      before_above += cl.map_shared_rank(counts, r)[0];
      before_equal += cl.map_shared_rank(counts, r)[1];
    }
    cl.sync();  // no CTA leaves while another reads its counts or histograms
  }
  if (need == 0) return;
  // `left` of the equal ones stay, the lowest slots first.  Position of a
  // kept slot: kept above before it, and kept equals before it.
#pragma unroll 4
  for (int j = i0; j < i1; j += 32) {
    const int i = j + lane;
    const uint32_t k = i < i1 ? key_at(i) : 0u;
    const bool up = i < i1 && (all || k > prefix), eq = i < i1 && !all && k == prefix;
    const uint32_t mu = __ballot_sync(0xffffffffu, up), me = __ballot_sync(0xffffffffu, eq);
    const int au = before_above + __popc(mu & ((1u << lane) - 1u));
    const int ae = before_equal + __popc(me & ((1u << lane) - 1u));
    if (up || (eq && ae < left)) {
      const int at = au + min(ae, left);
      if (MSA_IN_RANGE(at, 1, kept, a.status)) {
        out[at] = i;
        out_w[at] = key_weight(k);
      }
    }
    before_above += __popc(mu);
    before_equal += __popc(me);
  }
}

}  // namespace

cudaError_t launch_cache_evict_select(const EvictArgs& a, cudaStream_t st) {
  // 8192 slots a CTA up to a cluster of 8 while every CTA has an SM, else 32768
  // a CTA: a cluster's barriers cost more than the counting that it shares (256
  // lists of 60000 slots: 158 us with clusters of 8, 65 with 2; 128 of 12000:
  // 13.9 with 2, 11.1 without; but 16 of 30000: 13.2 with 4, 14.7 with 2).
  // Then up to kKeysMax a CTA; longer rows are read again for each digit.
  const int64_t slots = static_cast<int64_t>(a.s.max_blocks) * a.c.block;
  const int64_t lists = static_cast<int64_t>(a.s.batch) * a.c.Hkv;
  int ranks = 1;
  while (ranks < kClusterMax && slots > ranks * 8192 &&
         (lists * ranks * 2 <= kSms || slots > ranks * 32768))
    ranks *= 2;
  const int64_t each = (slots / ranks + 1) + 32 * kEvictWarps;
  const bool staged = each <= kKeysMax;
  const auto kernel = staged ? cache_evict_kernel<true> : cache_evict_kernel<false>;
  const int smem = staged ? static_cast<int>(each) * 4 : 0;
  if (staged) {
    // The kernel's most, not this call's: the limit is the function's, and
    // another host thread may launch between this and the launch below.
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.batch) * a.c.Hkv * ranks);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace msa
