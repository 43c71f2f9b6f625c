// C ABI of the norms of queries and keys with the rotary position embedding
// (msa_rope.h): argument validation, workspace layout and launch.
#include "api_common.cuh"
#include "rope.cuh"

namespace {

msa_status check_rope_sizes(int64_t n, int Hq, int Hkv, int d) {
  if (n < 0 || n > INT32_MAX) return fail(MSA_ERR_INVALID_ARG, "n=%lld out of range", (long long)n);
  if (Hq < 1 || Hq > kMaxHeads || Hkv < 0 || Hkv > kMaxHeads)
    return fail(MSA_ERR_INVALID_ARG, "Hq=%d Hkv=%d out of range", Hq, Hkv);
  if (d != 64 && d != 128) return fail(MSA_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (n * (Hq > Hkv ? Hq : Hkv) > int64_t(1) << 38)  // a CTA's rows are counted in 32 bits
    return fail(MSA_ERR_UNSUPPORTED, "n=%lld Hq=%d Hkv=%d: too many rows", (long long)n, Hq, Hkv);
  return MSA_OK;
}

// [n, heads, d] at p, tokens `stride` elements apart.
msa_status check_tokens(const void* p, int64_t stride, int heads, int d, msa_dtype dt,
                        const char* what) {
  if (!p || !aligned(p, 16))
    return fail(MSA_ERR_INVALID_ARG, "%s null or not 16-byte aligned", what);
  const int64_t per = dt == MSA_BF16 ? 8 : 4;
  if (stride < static_cast<int64_t>(heads) * d || stride % per || stride > (int64_t(1) << 31))
    return fail(MSA_ERR_INVALID_ARG, "%s: stride=%lld (at least heads * d, a multiple of 16 bytes)",
                what, (long long)stride);
  return MSA_OK;
}

// What both directions take; with n = 0 the tensors are not looked at.
msa_status check_rope(msa::RopeArgs* a, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, int64_t n, int Hq, int Hkv, int d,
                      const int64_t* positions, const int64_t* freqs, const void* q_weight,
                      const void* k_weight, float eps, float mscale, int interleaved,
                      void* q_out, void* k_out, msa_dtype dt, msa_dtype w_dt) {
  MSA_TRY(check_rope_sizes(n, Hq, Hkv, d));
  if (!valid_dtype(dt)) return fail(MSA_ERR_INVALID_ARG, "bad dtype %d", (int)dt);
  if ((q_weight || k_weight) && !valid_dtype(w_dt))
    return fail(MSA_ERR_INVALID_ARG, "bad weight dtype %d", (int)w_dt);
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4))
    return fail(MSA_ERR_INVALID_ARG, "weight not 4-byte aligned");
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(MSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!isfinite(mscale)) return fail(MSA_ERR_INVALID_ARG, "mscale must be finite");
  if (n > 0) {
    if (!positions || !freqs || !aligned(positions, 8) || !aligned(freqs, 8))
      return fail(MSA_ERR_INVALID_ARG, "positions or freqs null or not 8-byte aligned");
    MSA_TRY(check_tokens(q, q_stride, Hq, d, dt, "q"));
    MSA_TRY(check_tokens(q_out, static_cast<int64_t>(Hq) * d, Hq, d, dt, "q's output"));
    if (Hkv) {
      MSA_TRY(check_tokens(k, k_stride, Hkv, d, dt, "k"));
      MSA_TRY(check_tokens(k_out, static_cast<int64_t>(Hkv) * d, Hkv, d, dt, "k's output"));
    }
  }
  a->x[0] = q;
  a->x[1] = k;
  a->stride[0] = q_stride;
  a->stride[1] = k_stride;
  a->out[0] = q_out;
  a->out[1] = k_out;
  a->heads[0] = Hq;
  a->heads[1] = Hkv;
  a->weight[0] = q_weight;
  a->weight[1] = k_weight;
  a->n = n;
  a->d = d;
  a->positions = positions;
  a->freqs = freqs;
  a->eps = eps;
  a->mscale = mscale;
  a->interleaved = interleaved != 0;
  a->bf16 = dt == MSA_BF16;
  a->w_bf16 = w_dt == MSA_BF16;
  return MSA_OK;
}

size_t bwd_bytes(int64_t n, int Hq, int Hkv, int d, int* ctas) {
  const int heads[2] = {Hq, Hkv};
  msa::norm_rope_bwd_ctas(n, heads, d, ctas);
  return up(static_cast<size_t>(ctas[0] + ctas[1]) * d * sizeof(float2));
}

}  // namespace

extern "C" {

msa_status msa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            int64_t n, int Hq, int Hkv, int d, const int64_t* positions,
                            const int64_t* freqs, const void* q_weight, const void* k_weight,
                            float eps, float mscale, int interleaved, void* q_out, void* k_out,
                            msa_dtype dt, msa_dtype w_dt, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  msa::RopeArgs a{};
  MSA_TRY(check_rope(&a, q, q_stride, k, k_stride, n, Hq, Hkv, d, positions, freqs, q_weight,
                     k_weight, eps, mscale, interleaved, q_out, k_out, dt, w_dt));
  if (n == 0) return msa::api_ok();
  MSA_TRY(msa::api_status_word(&a.status));
  return launched(msa::launch_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)),
                  "norm and rotation");
}

size_t msa_qk_norm_rope_bwd_workspace_size(int64_t n, int Hq, int Hkv, int d) {
  if (check_rope_sizes(n, Hq, Hkv, d) != MSA_OK) return 0;
  int ctas[2];
  return bwd_bytes(n, Hq, Hkv, d, ctas);
}

msa_status msa_qk_norm_rope_bwd(const void* dq_out, int64_t dq_out_stride, const void* dk_out,
                                int64_t dk_out_stride, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, int64_t n, int Hq, int Hkv, int d,
                                const int64_t* positions, const int64_t* freqs,
                                const void* q_weight, const void* k_weight, float eps,
                                float mscale, int interleaved, void* dq, void* dk,
                                void* dq_weight, void* dk_weight, msa_dtype dt, msa_dtype w_dt,
                                void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  MSA_NVTX_RANGE();
  msa::RopeArgs a{};
  MSA_TRY(check_rope(&a, q, q_stride, k, k_stride, n, Hq, Hkv, d, positions, freqs, q_weight,
                     k_weight, eps, mscale, interleaved, dq, dk, dt, w_dt));
  if (n > 0) {
    MSA_TRY(check_tokens(dq_out, dq_out_stride, Hq, d, dt, "dq_out"));
    if (Hkv) MSA_TRY(check_tokens(dk_out, dk_out_stride, Hkv, d, dt, "dk_out"));
  }
  if ((q_weight && !dq_weight) || (k_weight && !dk_weight) || !aligned(dq_weight, 4) ||
      !aligned(dk_weight, 4))
    return fail(MSA_ERR_INVALID_ARG, "a weight's gradient null or not 4-byte aligned");
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.dy_stride[0] = dq_out_stride;
  a.dy_stride[1] = dk_out_stride;
  a.dweight[0] = q_weight ? dq_weight : nullptr;
  a.dweight[1] = k_weight ? dk_weight : nullptr;
  const size_t need = bwd_bytes(n, Hq, Hkv, d, a.ctas);
  if (q_weight || k_weight) MSA_TRY(check_workspace(workspace, workspace_bytes, need));
  a.part = static_cast<float2*>(workspace);
  MSA_TRY(msa::api_status_word(&a.status));
  return launched(msa::launch_norm_rope_bwd(a, reinterpret_cast<cudaStream_t>(stream)),
                  "norm and rotation backward");
}

}  // extern "C"
