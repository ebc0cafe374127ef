// Internal declarations of the decoder operators around the MoE layer.
#pragma once

#include <cmath>

#include "moe_internal.h"

namespace moe {

// ---------------------------------------------------------------------------
// E4M3 quantisation of a group of values (one scale per group)
// ---------------------------------------------------------------------------
// Smallest largest-magnitude that is quantised: 448 / a stays finite.
constexpr uint32_t kQuantMinBits = 0x05000000u;  // 2^-117

// From the bits of a group's largest magnitude: the factor v -> code, which
// is 448 times the rounded reciprocal (what tensor programs compute for
// 448 / a, so that activations quantised by one agree code for code), and the
// scale code -> v, a times the rounded 1 / 448 (0 for a group that holds
// nothing).
__device__ __forceinline__ void quant_factors(uint32_t maxbits, float& to_code, float& scale) {
  const float a = __uint_as_float(maxbits);
  const bool any = maxbits >= kQuantMinBits;
  to_code = any ? __fmul_rn(448.f, __frcp_rn(a)) : 0.f;
  scale = any ? __fmul_rn(a, 1.f / 448.f) : 0.f;
}
// Two floats -> two E4M3 codes (lo in bits 0..7), nearest even, saturated.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// All launchers enqueue on `s`.
// logits: `slices` arrays of [T, row_stride], slice_stride apart, which are
// added in order, then logit_bias (may be NULL).  found (may be NULL): a status
// word of the kernels before, whose bits are raised in status as well.
cudaError_t launch_select_experts(const float* logits, long long row_stride, int slices,
                                  long long slice_stride, const float* logit_bias,
                                  const float* bias, const moe_select_rule& rule, int T, int E,
                                  int k, int32_t* topk_idx, float* topk_w, const int32_t* found,
                                  int32_t* status, cudaStream_t s);

cudaError_t launch_qk_norm_rope(const uint16_t* qkv, const float* q_norm, const float* k_norm,
                                const float* cos_sin, const int32_t* pos, const int64_t* slots,
                                const moe_qk_dims& d, const moe_kv_cache& cache, uint16_t* q_out,
                                int32_t* status, cudaStream_t s);

// Whether the work units that the block table has room for fit 31 bits.
bool paged_attention_fits(const moe_attn_dims& d, const moe_kv_cache& cache);
// Scratch bytes of one attention call: two partial results per CTA.
size_t paged_attention_workspace(const moe_attn_dims& d, int D);
cudaError_t launch_paged_attention(const uint16_t* q, const moe_kv_cache& cache,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const moe_attn_dims& d, uint16_t* out, void* ws,
                                   int32_t* status, cudaStream_t s);

// Whether the work units that the block table has room for fit 31 bits.
bool draft_attention_fits(const moe_draft_dims& d, const moe_kv_cache& cache);
// Scratch bytes of one call: two partial results per CTA, and where each
// segment's begin.
size_t draft_attention_workspace(const moe_draft_dims& d, int Hkv, int DV);
// latent: cache has one head whose values are its keys' leading DV dimensions.
cudaError_t launch_draft_attention(const uint16_t* q, const moe_kv_cache& cache, bool latent,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const int64_t* mask, const int32_t* draft_lens,
                                   const moe_draft_dims& d, int DV, uint16_t* out, void* ws,
                                   int32_t* status, cudaStream_t s);

cudaError_t launch_latent_store(const uint16_t* kv, const float* norm, const float* cos_sin,
                                const int32_t* pos, const int64_t* slots, const uint16_t* q,
                                const moe_latent_dims& d, const moe_latent_cache& cache,
                                uint16_t* q_out, uint16_t* rows, int32_t* status, cudaStream_t s);

// Whether the grid fits 31 bits.
bool expanded_attention_fits(const moe_expanded_dims& d);
cudaError_t launch_expanded_attention(const uint16_t* q, const uint16_t* k_nope, const uint16_t* k_rope,
                                      const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                                      const moe_expanded_dims& d, uint16_t* out, int32_t* status,
                                      cudaStream_t s);

size_t linear_fp8_workspace(const moe_linear_dims& d);
cudaError_t launch_linear_fp8(const uint16_t* x, const moe_fp8_mat& w, const float* bias,
                              const moe_linear_dims& d, uint16_t* out, void* ws, int32_t* status,
                              cudaStream_t s);

}  // namespace moe
