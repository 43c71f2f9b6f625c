// Norms of queries and keys for each head with the rotary position embedding
// (msa_rope.h): launchers.
#pragma once

#include "cache_common.cuh"
#include "msa_rope.h"

namespace msa {

struct RopeArgs {
  const void* x[2];      // queries, keys: [n][heads][d], stride[i] elements a token
  int64_t stride[2];
  const void* dy[2];     // backward: gradients of the outputs
  int64_t dy_stride[2];
  void* out[2];          // outputs, or the gradients of x: [n][heads][d]
  int heads[2];
  const void* weight[2];  // [d], null: no norm
  void* dweight[2];       // backward: [d]
  float2* part;           // backward: [ctas][d] sums of the weights' gradients in two floats,
                          // queries' CTAs first
  int ctas[2];            // of queries, of keys
  int64_t n;
  int d;
  const int64_t* positions;
  const int64_t* freqs;
  float eps, mscale;
  int interleaved, bf16, w_bf16;
  int* status;
};
cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t st);
// CTAs of the backward's two sides.
void norm_rope_bwd_ctas(int64_t n, const int* heads, int d, int* ctas);
cudaError_t launch_norm_rope_bwd(const RopeArgs& a, cudaStream_t st);

}  // namespace msa
