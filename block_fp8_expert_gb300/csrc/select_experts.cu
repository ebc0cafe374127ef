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

// A warp per token; lane l holds experts l, l + 32, ... (EPL of them), so the
// logits arrive in coalesced rows, all loads in flight at once, and nothing
// touches memory again before the k results.
//   scores   softmax: the row maximum and sum over the warp;
//   groups   per group two integer max reductions (redux.sync): the largest
//            key, then the largest of the rest with one instance of it taken
//            out; lane g keeps group g's score and ranks it against the
//            others, the kept groups are a ballot;
//   top-k    per round a max reduction over the lanes' best remaining keys
//            and a min reduction over the expert indices that hold it (ties
//            to the lower expert); only the winning lane rescans its own.
template <int EPL>
__global__ void __launch_bounds__(128)
k_select_experts(const float* __restrict__ logits, long long row_stride,
                 const float* __restrict__ bias, const moe_select_rule rule, int T, int E, int k,
                 int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  const float* row = logits + (size_t)t * row_stride;
  float l[EPL];
  int key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? __ldg(row + e) : -INFINITY;
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
    const int e = lane + 32 * i;
    float s;
    if (sigmoid) {
      s = 1.f / (1.f + expf(-l[i]));
      l[i] = s;  // the weight's source: the score itself
    } else {
      s = expf(l[i] - vmax) * inv_sum;
    }
    const float b = (bias && e < E) ? __ldg(bias + e) : 0.f;
    key[i] = e < E ? order_key(s + b) : INT_MIN;
  }
  if (rule.groups > 1) {
    const int n = E / rule.groups;
    float score = -INFINITY;  // lane g: group g's score
    for (int g = 0; g < rule.groups; ++g) {
      int a = INT_MIN, b = INT_MIN;  // this lane's two largest keys of the group
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * n && e < g * n + n) {
          b = max(b, min(a, key[i]));
          a = max(a, key[i]);
        }
      }
      const int first = __reduce_max_sync(kAll, a);
      float v = first == INT_MAX ? NAN : order_value(first);
      if (rule.group_top == 2) {
        const unsigned holders = __ballot_sync(kAll, a == first);
        const int mine = lane == __ffs(holders) - 1 ? b : a;
        const int second = __reduce_max_sync(kAll, mine);
        v += second == INT_MAX ? NAN : order_value(second);
      }
      if (lane == g) score = v;
    }
    const int sk = lane < rule.groups ? order_key(score) : INT_MIN;
    int better = 0;
    for (int g = 0; g < rule.groups; ++g) {
      const int o = __shfl_sync(kAll, sk, g);
      better += o > sk || (o == sk && g < lane);
    }
    const unsigned kept = __ballot_sync(kAll, lane < rule.groups && better < rule.top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((kept >> (e / n)) & 1u)) key[i] = INT_MIN;
    }
  }
  int hk, he;
  float hv;
  auto rescan = [&]() {
    hk = INT_MIN;
    he = INT_MAX;
    hv = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (key[i] > hk) {  // the first (lowest) expert of equal keys
        hk = key[i];
        he = lane + 32 * i;
        hv = l[i];
      }
    }
  };
  rescan();
  int my_idx = 0;
  float my_v = 0.f;
  for (int j = 0; j < k; ++j) {
    const int wk = __reduce_max_sync(kAll, hk);
    const int we = __reduce_min_sync(kAll, hk == wk ? he : INT_MAX);
    const float wv = __shfl_sync(kAll, hv, we & 31);
    if (lane == j) {
      my_idx = we;
      my_v = wv;
    }
    if (he == we) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i == we) key[i] = INT_MIN;
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
  const int epl = cdiv(E, 32);
#define MOE_SELECT(EPLV)                                                                      \
  return launch_k(k_select_experts<EPLV>, grid, blk, 0, s, false, logits, row_stride, bias, rule, \
                  T, E, k, topk_idx, topk_w)
  if (epl <= 2) MOE_SELECT(2);
  if (epl <= 4) MOE_SELECT(4);
  if (epl <= 8) MOE_SELECT(8);
  if (epl <= 16) MOE_SELECT(16);
  MOE_SELECT(32);
#undef MOE_SELECT
}

}  // namespace moe
