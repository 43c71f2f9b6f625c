// K10: which slots an eviction keeps -- for each sequence and KV head the
// last `recent` slots and, of the others, those that drew the most
// attention, min(len, budget) in all, ties to the lower slot.  K7 then
// gathers them into fresh blocks.
//
// One cluster of CTAs a (sequence, KV head), each with a contiguous part of
// the slots: a radix selection of the least kept weight by bytes (histograms
// in shared memory, joined through the cluster's), then one pass that counts
// and one that writes the kept slots in order.  Weights compare as they are:
// the choice is exact.  The weights are read once from HBM and again, twice
// to five times more, from L2: 4 bytes a slot, against the 2 d bytes a kept
// slot costs in the gather.
#include <math.h>

#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kClusterMax = 8;

// Unsigned key that orders as the weight does; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) cache_evict_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int total[256];
  __shared__ int digit, left_s;
  __shared__ int counts[2];  // this CTA's slots above the least kept weight, and equal to it
  __shared__ int wsum[2][kEvictWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int ranks = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
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
  const int per = (n + ranks - 1) / ranks;
  const int i0 = min(n, rank * per), i1 = min(n, i0 + per);

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
  if (need > 0 && need < n) {  // the same for the whole cluster
    for (int byte = 3; byte >= 0; --byte) {
      for (int i = threadIdx.x; i < 256; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int i = i0 + threadIdx.x; i < i1; i += kEvictThreads) {
        const uint32_t k = weight_key(w[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> (8 * byte)) & 255], 1);
      }
      cl.sync();
      if (threadIdx.x < 256) {
        int s = 0;
        for (int r = 0; r < ranks; ++r) s += cl.map_shared_rank(hist, r)[threadIdx.x];
        total[threadIdx.x] = s;
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += total[255 - 8 * threadIdx.x - i];
        int upto = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        int before = upto - s;
        if (before < left && left <= upto) {
          for (int i = 0; i < 8; ++i) {
            const int dgt = 255 - 8 * threadIdx.x - i;
            if (left <= before + total[dgt]) {
              digit = dgt;
              left_s = left - before;
              break;
            }
            before += total[dgt];
          }
        }
      }
      // All ranks have read this histogram before any clears it again.
      cl.sync();
      prefix |= static_cast<uint32_t>(digit) << (8 * byte);
      mask |= 255u << (8 * byte);
      left = left_s;
    }
  }
  const bool all = need == n;
  // How many of this CTA's slots lie above the least kept weight, and at it.
  int above = 0, equal = 0;
  if (need > 0) {
    for (int i = i0 + threadIdx.x; i < i1; i += kEvictThreads) {
      const uint32_t k = weight_key(w[i]);
      above += all || k > prefix;
      equal += !all && k == prefix;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (lane == 0) {
    wsum[0][warp] = above;
    wsum[1][warp] = equal;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int x = 0, y = 0;
    for (int i = 0; i < kEvictWarps; ++i) {
      x += wsum[0][i];
      y += wsum[1][i];
    }
    counts[0] = x;
    counts[1] = y;
  }
  cl.sync();
  int before_above = 0, before_equal = 0;
  for (int r = 0; r < rank; ++r) {
    before_above += cl.map_shared_rank(counts, r)[0];
    before_equal += cl.map_shared_rank(counts, r)[1];
  }
  cl.sync();  // no CTA leaves while another reads its counts
  if (need == 0) return;
  // `left` of the equal ones stay, the lowest slots first.  Position of a
  // kept slot: kept above before it, and kept equals before it.
  for (int j0 = i0; j0 < i1; j0 += kEvictThreads) {
    const int i = j0 + threadIdx.x;
    const float x = i < i1 ? w[i] : 0.f;
    const uint32_t k = weight_key(x);
    const bool up = i < i1 && (all || k > prefix), eq = i < i1 && !all && k == prefix;
    const uint32_t mu = __ballot_sync(0xffffffffu, up), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(mu);
      wsum[1][warp] = __popc(me);
    }
    __syncthreads();
    int au = before_above, ae = before_equal, tu = 0, te = 0;
#pragma unroll
    for (int v = 0; v < kEvictWarps; ++v) {
      au += v < warp ? wsum[0][v] : 0;
      ae += v < warp ? wsum[1][v] : 0;
      tu += wsum[0][v];
      te += wsum[1][v];
    }
    au += __popc(mu & ((1u << lane) - 1u));
    ae += __popc(me & ((1u << lane) - 1u));
    if (up || (eq && ae < left)) {
      const int at = au + min(ae, all ? 0 : left);
      out[at] = i;
      out_w[at] = x;
    }
    before_above += tu;
    before_equal += te;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_cache_evict_select(const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  // A CTA reads 16K weights a pass in about a microsecond; more than that is
  // split over a cluster.
  const int64_t slots = static_cast<int64_t>(a.s.max_blocks) * a.c.block;
  const int ranks = slots <= 16384 ? 1 : kClusterMax;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.batch) * a.c.Hkv * ranks);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_evict_kernel, a);
}

}  // namespace msa
