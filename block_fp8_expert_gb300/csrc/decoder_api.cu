// The C ABI of the decoder operators around the MoE layer (include/moe_fp8.h):
// argument checks and launches.
#include "api_check.h"
#include "decoder_internal.h"

namespace moe {
namespace {

moe_status check_stride(long long stride, long long least, int multiple, const char* name) {
  if (stride < least || stride % multiple)
    return fail(MOE_ERR_INVALID_ARG, "%s = %lld: need at least %lld and a multiple of %d", name,
                stride, least, multiple);
  return MOE_OK;
}

moe_status check_cache(const moe_kv_cache& c) {
  moe_status s;
  if (c.format != MOE_KV_BF16 && c.format != MOE_KV_E4M3)
    return fail(MOE_ERR_INVALID_ARG, "cache format %d", c.format);
  if (c.D != 64 && c.D != 128 && c.D != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head size D = %d: need 64, 128 or 256", c.D);
  if (c.Hkv < 1 || c.Hkv > 1024)
    return fail(MOE_ERR_UNSUPPORTED, "Hkv = %d outside [1, 1024]", c.Hkv);
  if (c.pages < 1 || c.page_size < 1)
    return fail(MOE_ERR_INVALID_ARG, "cache of %d pages of %d tokens", c.pages, c.page_size);
  REQUIRE_PTR(c.k);
  REQUIRE_PTR(c.v);
  const bool f8 = c.format == MOE_KV_E4M3;
  const int m = f8 ? 16 : 8;  // 16 bytes
  if ((s = check_stride(c.page_stride, 0, m, "page_stride")) != MOE_OK) return s;
  if ((s = check_stride(c.head_stride, 0, m, "head_stride")) != MOE_OK) return s;
  if ((s = check_stride(c.token_stride, 0, m, "token_stride")) != MOE_OK) return s;
  if (f8) {
    REQUIRE_ELEMENTS(c.k_scale);
    REQUIRE_ELEMENTS(c.v_scale);
    if ((s = check_stride(c.scale_page_stride, 0, 1, "scale_page_stride")) != MOE_OK) return s;
    if ((s = check_stride(c.scale_head_stride, 0, 1, "scale_head_stride")) != MOE_OK) return s;
    if ((s = check_stride(c.scale_token_stride, 0, 1, "scale_token_stride")) != MOE_OK) return s;
  } else if (c.k_scale || c.v_scale) {
    return fail(MOE_ERR_INVALID_ARG, "a bf16 cache has no scales");
  }
  return MOE_OK;
}

moe_status check_attn(const moe_attn_dims& d, int D) {
  if (D != 64 && D != 128 && D != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head size D = %d: need 64, 128 or 256", D);
  if (d.B < 0 || d.window < 0 || d.table_width < 0)
    return fail(MOE_ERR_INVALID_ARG, "B = %d, window = %d, table_width = %d", d.B, d.window,
                d.table_width);
  if (d.Hq < 1 || d.Hq > 1024) return fail(MOE_ERR_UNSUPPORTED, "Hq = %d outside [1, 1024]", d.Hq);
  if ((long long)d.B * d.Hq >= (1ll << 31)) return fail(MOE_ERR_UNSUPPORTED, "B * Hq too large");
  return MOE_OK;
}

moe_status check_rule(const moe_select_rule& rule, int E, int k) {
  if (rule.score != MOE_SCORE_SOFTMAX && rule.score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "score %d", rule.score);
  if (rule.groups < 1 || rule.groups > 32 || E % rule.groups)
    return fail(MOE_ERR_UNSUPPORTED, "groups = %d: need 1 to 32 that divide E = %d", rule.groups, E);
  if (rule.top_groups < 1 || rule.top_groups > rule.groups)
    return fail(MOE_ERR_INVALID_ARG, "top_groups = %d outside [1, %d]", rule.top_groups, rule.groups);
  const int n = E / rule.groups;
  if (rule.group_top < 1 || rule.group_top > 2 || (rule.groups > 1 && rule.group_top > n))
    return fail(MOE_ERR_INVALID_ARG, "group_top = %d: need 1 or 2, at most the group's %d experts",
                rule.group_top, n);
  if (k < 1 || k > 32 || k > rule.top_groups * n)
    return fail(MOE_ERR_UNSUPPORTED, "k = %d outside [1, min(%d experts of the kept groups, 32)]", k,
                rule.top_groups * n);
  return MOE_OK;
}

moe_status check_linear(const moe_linear_dims& d) {
  if (d.M < 0) return fail(MOE_ERR_INVALID_ARG, "M = %d < 0", d.M);
  if (d.M > (1 << 22)) return fail(MOE_ERR_UNSUPPORTED, "M = %d: at most 2^22 rows", d.M);
  if (d.N < 8 || d.N > 65536 || d.N % 8)
    return fail(MOE_ERR_UNSUPPORTED, "N = %d: need a multiple of 8 in [8, 65536]", d.N);
  if (d.K < 16 || d.K > 65536 || d.K % 16)
    return fail(MOE_ERR_UNSUPPORTED, "K = %d: need a multiple of 16 in [16, 65536]", d.K);
  moe_status s;
  if ((s = check_stride(d.x_stride, d.K, 8, "x_stride")) != MOE_OK) return s;
  return check_stride(d.out_stride, d.N, 8, "out_stride");
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_select_experts(const float* logits, int64_t row_stride, const float* bias,
                              moe_select_rule rule, int32_t T, int32_t E, int32_t k,
                              int32_t* topk_idx, float* topk_w, void* stream) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", T);
  if (E < 1 || E > kMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "E = %d outside [1, %d]", E, kMaxExperts);
  const moe_status s = check_rule(rule, E, k);
  if (s != MOE_OK) return s;
  if ((long long)T * k >= (1ll << 31)) return fail(MOE_ERR_UNSUPPORTED, "T*k too large");
  if (row_stride < E) return fail(MOE_ERR_INVALID_ARG, "row_stride = %lld < E", (long long)row_stride);
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(logits);
  REQUIRE_OPT_PTR(bias);
  REQUIRE_ELEMENTS(topk_idx);
  REQUIRE_ELEMENTS(topk_w);
  CUDA_CHECK(launch_select_experts(logits, row_stride, 1, 0, nullptr, bias, rule, T, E, k, topk_idx,
                                   topk_w, nullptr, nullptr, (cudaStream_t)stream),
             "moe_select_experts");
  return MOE_OK;
}

moe_status moe_route_select(const uint16_t* x, const float* Wr, const float* logit_bias,
                            const float* bias, moe_select_rule rule, moe_dims d,
                            int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                            void* stream) {
  return moe_route_select_status(x, Wr, logit_bias, bias, rule, d, topk_idx, topk_w, ws, ws_bytes,
                                 nullptr, stream);
}

moe_status moe_route_select_status(const uint16_t* x, const float* Wr, const float* logit_bias,
                                   const float* bias, moe_select_rule rule, moe_dims d,
                                   int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                                   int32_t* status, void* stream) {
  size_t need = 0;
  moe_status s = moe_workspace_bytes(d, &need);  // checks the dims
  if (s != MOE_OK) return s;
  if ((s = check_rule(rule, d.E, d.k)) != MOE_OK) return s;
  REQUIRE_OPT_PTR(status);
  if (d.T == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(Wr);
  REQUIRE_OPT_PTR(logit_bias);
  REQUIRE_OPT_PTR(bias);
  REQUIRE_ELEMENTS(topk_idx);
  REQUIRE_ELEMENTS(topk_w);
  REQUIRE_PTR(ws);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  const WsLayout L = ws_layout(d);
  float* part = at<float>(ws, L.logits);
  const cudaStream_t st = (cudaStream_t)stream;
  int32_t* found = at<int32_t>(ws, L.status);
  CUDA_CHECK(launch_router_logits(x, Wr, d.T, d.H, d.E, part, at<uint16_t>(ws, L.wr_planes), nullptr,
                                  nullptr, found, st, true),
             "moe_route_select");
  CUDA_CHECK(launch_select_experts(part, d.E, route_kslices(d.T, d.H, d.E), (long long)d.T * d.E,
                                   logit_bias, bias, rule, d.T, d.E, d.k, topk_idx, topk_w,
                                   status ? found : nullptr, status, st),
             "moe_route_select");
  return MOE_OK;
}

moe_status moe_qk_norm_rope(const uint16_t* qkv, const float* q_norm, const float* k_norm,
                            const float* cos_sin, const int32_t* pos, const int64_t* slots,
                            moe_qk_dims d, moe_kv_cache cache, uint16_t* q_out, int32_t* status,
                            void* stream) {
  moe_status s;
  if (d.T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", d.T);
  if (d.Hq < 1 || d.Hq > 1024) return fail(MOE_ERR_UNSUPPORTED, "Hq = %d outside [1, 1024]", d.Hq);
  if ((s = check_cache(cache)) != MOE_OK) return s;
  const int D = cache.D;
  if (d.rot < 0 || d.rot > D || d.rot % 16)
    return fail(MOE_ERR_UNSUPPORTED, "rot = %d: need a multiple of 16 in [0, %d]", d.rot, D);
  if ((s = check_stride(d.qkv_stride, (long long)(d.Hq + 2 * cache.Hkv) * D, 8, "qkv_stride")) != MOE_OK)
    return s;
  if ((s = check_stride(d.q_stride, (long long)d.Hq * D, 8, "q_stride")) != MOE_OK) return s;
  REQUIRE_OPT_PTR(q_norm);
  REQUIRE_OPT_PTR(k_norm);
  if (d.rot > 0 && d.n_pos < 1) return fail(MOE_ERR_INVALID_ARG, "n_pos = %d", d.n_pos);
  REQUIRE_OPT_PTR(status);
  if (d.T == 0) return MOE_OK;
  REQUIRE_PTR(qkv);
  if (d.rot > 0) {
    REQUIRE_PTR(cos_sin);
    REQUIRE_ELEMENTS(pos);
  } else if (cos_sin || pos) {
    return fail(MOE_ERR_INVALID_ARG, "rot = 0 takes no cos_sin and no pos");
  }
  REQUIRE_ELEMENTS(slots);
  REQUIRE_PTR(q_out);
  CUDA_CHECK(launch_qk_norm_rope(qkv, q_norm, k_norm, cos_sin, pos, slots, d, cache, q_out, status,
                                 (cudaStream_t)stream),
             "moe_qk_norm_rope");
  return MOE_OK;
}

moe_status moe_paged_attention_workspace_bytes(moe_attn_dims d, int32_t D, size_t* bytes) {
  moe_status s = check_attn(d, D);
  if (s != MOE_OK) return s;
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = align_up(paged_attention_workspace(d, D));
  return MOE_OK;
}

moe_status moe_paged_attention(const uint16_t* q, moe_kv_cache cache, const int32_t* block_table,
                               const int32_t* seq_lens, moe_attn_dims d, uint16_t* out, void* ws,
                               size_t ws_bytes, int32_t* status, void* stream) {
  moe_status s;
  if ((s = check_cache(cache)) != MOE_OK) return s;
  if ((s = check_attn(d, cache.D)) != MOE_OK) return s;
  if (d.Hq % cache.Hkv)
    return fail(MOE_ERR_UNSUPPORTED, "Hq = %d is no multiple of Hkv = %d", d.Hq, cache.Hkv);
  if (d.table_stride < d.table_width)
    return fail(MOE_ERR_INVALID_ARG, "table_stride = %lld < table_width", (long long)d.table_stride);
  if ((s = check_stride(d.q_stride, (long long)d.Hq * cache.D, 8, "q_stride")) != MOE_OK) return s;
  if ((s = check_stride(d.out_stride, (long long)d.Hq * cache.D, 8, "out_stride")) != MOE_OK) return s;
  if (!paged_attention_fits(d, cache))
    return fail(MOE_ERR_UNSUPPORTED, "B * Hkv * (table_width * page_size / 16 + 9) too large");
  REQUIRE_OPT_PTR(status);
  if (d.B == 0) return MOE_OK;
  REQUIRE_PTR(q);
  if (d.table_width > 0) REQUIRE_ELEMENTS(block_table);
  REQUIRE_ELEMENTS(seq_lens);
  REQUIRE_PTR(out);
  REQUIRE_PTR(ws);
  const size_t need = align_up(paged_attention_workspace(d, cache.D));
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  CUDA_CHECK(launch_paged_attention(q, cache, block_table, seq_lens, d, out, ws, status,
                                    (cudaStream_t)stream),
             "moe_paged_attention");
  return MOE_OK;
}

moe_status moe_linear_fp8_workspace_bytes(moe_linear_dims d, size_t* bytes) {
  moe_status s = check_linear(d);
  if (s != MOE_OK) return s;
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = align_up(linear_fp8_workspace(d));
  return MOE_OK;
}

moe_status moe_linear_fp8(const uint16_t* x, moe_fp8_mat w, const float* bias, moe_linear_dims d,
                          uint16_t* out, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  moe_status s;
  if ((s = check_linear(d)) != MOE_OK) return s;
  REQUIRE_PTR(w.codes);
  REQUIRE_PTR(w.scales);
  REQUIRE_OPT_PTR(bias);
  REQUIRE_OPT_PTR(status);
  if (d.M == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(out);
  REQUIRE_PTR(ws);
  const size_t need = align_up(linear_fp8_workspace(d));
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  CUDA_CHECK(launch_linear_fp8(x, w, bias, d, out, ws, status, (cudaStream_t)stream),
             "moe_linear_fp8");
  return MOE_OK;
}

}  // extern "C"
