// Expert selection from router logits: softmax or sigmoid scores, a balance
// bias that only steers the choice, groups of experts, top-k and the weights
// (moe_select_experts).
#include <climits>

#include "decoder_internal.h"

namespace moe {

namespace {

// Order-preserving integer of a key: a larger key gives a larger integer, -0
// and +0 the same one, and any NaN the largest.  INT_MIN is below every key.
__device__ __forceinline__ int order_key(float v) {
  if (v != v) return INT_MAX;
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_value(int key) {
  return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace

// A warp per token; lane l holds experts l EPL .. l EPL + EPL - 1, so the
// logits arrive in whole rows, all loads in flight at once, a group of experts
// is a run of lanes, and nothing touches memory again before the k results.
//   scores   softmax: the row maximum and sum over the warp;
//   groups   a lane's two largest keys, then the group's by a butterfly over
//            its lanes (ALIGNED: groups of 2^i EPL experts); other group sizes:
//            per group two warp-wide integer max reductions.  A group's
//            score is ranked against the others'; the kept groups are a mask;
//   top-k    per round a max reduction over the lanes' best remaining keys;
//            the lowest lane that holds it wins (ties to the lower expert) and
//            rescans its own experts.
template <int EPL, bool ALIGNED>
__global__ void __launch_bounds__(128)
k_select_experts(const float* __restrict__ logits, long long row_stride,
                 const float* __restrict__ bias, const moe_select_rule rule, int T, int E, int k,
                 int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr unsigned kAll = 0xffffffffu;
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  const int e0 = lane * EPL;
  const float* row = logits + (size_t)t * row_stride;
  float l[EPL];
  int key[EPL];
  // 16-byte loads where rows and lanes allow them
  if (EPL % 4 == 0 && (row_stride & 3) == 0 && (E & 3) == 0) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const float4 v = e0 + i < E ? __ldg(reinterpret_cast<const float4*>(row + e0 + i))
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      l[i] = v.x;
      l[(i + 1) % EPL] = v.y;  // (% EPL: no such lane where EPL = 2)
      l[(i + 2) % EPL] = v.z;
      l[(i + 3) % EPL] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = e0 + i < E ? __ldg(row + e0 + i) : -INFINITY;
  }
  const bool sigmoid = rule.score == MOE_SCORE_SIGMOID;
  float vmax = 0.f, inv_sum = 0.f;  // softmax statistics
  if (!sigmoid) {
    vmax = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) vmax = fmaxf(vmax, l[i]);
    vmax = order_value(__reduce_max_sync(kAll, order_key(vmax)));
    if (vmax == -INFINITY) vmax = 0.f;  // every expert off: all scores 0
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s += expf(l[i] - vmax);
    s = warp_sum(s);
    inv_sum = s == 0.f ? 0.f : 1.f / s;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float s;
    if (sigmoid) {
      s = __frcp_rn(1.f + expf(-l[i]));
      l[i] = s;  // the weight's source: the score itself
    } else {
      s = expf(l[i] - vmax) * inv_sum;
    }
    const bool real = e0 + i < E;
    if (bias && real) s += __ldg(bias + e0 + i);
    key[i] = real ? order_key(s) : INT_MIN;
  }
  if (rule.groups > 1) {
    const int n = E / rule.groups;
    auto sum_of = [&](int first, int second) {  // a group's score
      float v = first == INT_MAX ? NAN : order_value(first);
      if (rule.group_top == 2) v += second == INT_MAX ? NAN : order_value(second);
      return order_key(v);
    };
    if (ALIGNED) {
      int a = INT_MIN, b = INT_MIN;  // the two largest keys: the lane's, then the group's
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        b = max(b, min(a, key[i]));
        a = max(a, key[i]);
      }
      const int span = n / EPL;  // lanes of a group
      for (int o = 1; o < span; o <<= 1) {
        const int oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
        b = max(max(b, ob), min(a, oa));
        a = max(a, oa);
      }
      const int g = e0 / n, sk = g < rule.groups ? sum_of(a, b) : INT_MIN;
      int better = 0;
      for (int h = 0; h < rule.groups; ++h) {
        const int o = __shfl_sync(kAll, sk, h * span);
        better += o > sk || (o == sk && h < g);
      }
      if (better >= rule.top_groups) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = INT_MIN;
      }
    } else {
      int sk = INT_MIN;  // lane g: group g's score
      for (int g = 0; g < rule.groups; ++g) {
        int a = INT_MIN, b = INT_MIN;  // this lane's two largest keys of the group
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int x = (unsigned)(e0 + i - g * n) < (unsigned)n ? key[i] : INT_MIN;
          b = max(b, min(a, x));
          a = max(a, x);
        }
        const int first = __reduce_max_sync(kAll, a);
        const unsigned holders = __ballot_sync(kAll, a == first);
        const int second = __reduce_max_sync(kAll, lane == __ffs(holders) - 1 ? b : a);
        if (lane == g) sk = sum_of(first, second);
      }
      int better = 0;
      for (int g = 0; g < rule.groups; ++g) {
        const int o = __shfl_sync(kAll, sk, g);
        better += o > sk || (o == sk && g < lane);
      }
      const unsigned kept = __ballot_sync(kAll, lane < rule.groups && better < rule.top_groups);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i < E && !((kept >> ((e0 + i) / n)) & 1u)) key[i] = INT_MIN;
    }
  }
  int hk, hs;  // the lane's best remaining key and its place
  float hv;
  auto rescan = [&]() {
    hk = key[0];
    hs = 0;
    hv = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      const bool up = key[i] > hk;  // the first (lowest) expert of equal keys
      hk = up ? key[i] : hk;
      hs = up ? i : hs;
      hv = up ? l[i] : hv;
    }
  };
  rescan();
  int my_idx = 0;
  float my_v = 0.f;
  for (int j = 0; j < k; ++j) {
    const int wk = __reduce_max_sync(kAll, hk);
    const int src = __ffs(__ballot_sync(kAll, hk == wk)) - 1;
    const int we = __shfl_sync(kAll, e0 + hs, src);
    const float wv = __shfl_sync(kAll, hv, src);
    if (lane == j) {
      my_idx = we;
      my_v = wv;
    }
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = i == hs ? INT_MIN : key[i];
      rescan();
    }
  }
  // weights: the chosen scores, renormalised softmax as the softmax over the
  // chosen logits (the normaliser over all experts cancels)
  float w;
  if (sigmoid) {
    w = lane < k ? my_v : 0.f;
  } else if (rule.renorm) {
    float m = lane < k ? my_v : -INFINITY;
    m = order_value(__reduce_max_sync(kAll, order_key(m)));
    if (m == -INFINITY) m = 0.f;
    w = lane < k ? expf(my_v - m) : 0.f;
  } else {
    w = lane < k ? expf(my_v - vmax) * inv_sum : 0.f;
  }
  if (rule.renorm) {
    const float s = warp_sum(w);
    w = s == 0.f ? 0.f : w / s;
  }
  if (lane < k) {
    topk_idx[(size_t)t * k + lane] = my_idx;
    topk_w[(size_t)t * k + lane] = w * rule.scale;
  }
}

cudaError_t launch_select_experts(const float* logits, long long row_stride, const float* bias,
                                  const moe_select_rule& rule, int T, int E, int k,
                                  int32_t* topk_idx, float* topk_w, cudaStream_t s) {
  const dim3 grid(cdiv(T, 4)), blk(128);
  int epl = 2;
  while (epl * 32 < E) epl *= 2;
  const int n = E / rule.groups, span = n / epl;
  const bool aligned = n % epl == 0 && (span & (span - 1)) == 0;
#define MOE_SELECT(EPLV)                                                                        \
  return aligned ? launch_k(k_select_experts<EPLV, true>, grid, blk, 0, s, true, logits,        \
                            row_stride, bias, rule, T, E, k, topk_idx, topk_w)                  \
                 : launch_k(k_select_experts<EPLV, false>, grid, blk, 0, s, true, logits,       \
                            row_stride, bias, rule, T, E, k, topk_idx, topk_w)
  if (epl <= 2) MOE_SELECT(2);
  if (epl <= 4) MOE_SELECT(4);
  if (epl <= 8) MOE_SELECT(8);
  if (epl <= 16) MOE_SELECT(16);
  MOE_SELECT(32);
#undef MOE_SELECT
}

}  // namespace moe
