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

// 1 / (1 + exp(-l)); the reciprocal to 1 ulp, subnormal ones too on this GPU
// (logits from -87.3 down to -88.7; tested).
__device__ __forceinline__ float sigmoid_of(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-l)));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace

// A warp per token; every group of experts (all of them, where there is one
// group) has a run of 2^span_log2 lanes, which hold EPL consecutive experts
// each while there are some: the logits arrive in whole rows, all loads in
// flight at once, and nothing touches memory again before the k results.
//   scores   softmax: the row maximum and sum over the warp;
//   groups   a lane's two largest keys, then the group's by a butterfly over
//            its lanes; its score is ranked against the others';
//   top-k    the k-th largest of the lanes' best keys (k max reductions) bounds
//            the k-th largest key from below.  The keys that reach it, seldom
//            many more than k, are gathered one per lane and ranked against
//            one another, ties to the lower expert; a lane's rank is its slot.
//            Where more than 32 reach it (many equal keys), k rounds pick the
//            largest remaining key each: a max reduction, the lowest lane that
//            holds it wins and looks its experts through again.
// Bound by instruction issue, not by the 4 E bytes a token reads: T 8192, E
// 256, sigmoid, 8 groups, k 8: 7.1 us (8.9 MB would take 1.3 at the copy
// rate), of which 1.1 for the groups and 0.9 for k 8 instead of 1; an earlier
// version took 13.5 with k rounds for the top-k alone and 11.0 as it is here.
// T 5: 2.8 us, launch and one warp's latency, so the code is kept short: what
// is rare (NaN keys, lanes with fewer experts) stands in branches of its own,
// and a group's lanes share its comparisons with the other groups.
template <int EPL>
__global__ void __launch_bounds__(128)
k_select_experts(const float* __restrict__ logits, long long row_stride, int slices,
                 long long slice_stride, const float* __restrict__ logit_bias,
                 const float* __restrict__ bias, const moe_select_rule rule, int n, int span_log2,
                 int T, int k, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
                 const int32_t* found, int32_t* status) {
  constexpr unsigned kAll = 0xffffffffu;
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  // what the kernels before found, where the caller keeps it
  if (found && t == 0 && lane == 0) {
    const int32_t bits = __ldcg(found);
    if (bits) raise_status(status, bits);
  }
  const int g = lane >> span_log2, place = (lane & ((1 << span_log2) - 1)) * EPL;
  const int e0 = g * n + place, count = g < rule.groups ? n - place : 0;  // (may be over EPL, or below 0)
  const float* row = logits + (size_t)t * row_stride;
  float l[EPL];
  int key[EPL];
  // 16-byte loads where rows and lanes allow them
  if (EPL % 4 == 0 && (row_stride & 3) == 0 && (n & 3) == 0) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const float4 v = i < count ? __ldg(reinterpret_cast<const float4*>(row + e0 + i))
                                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      l[i] = v.x;
      l[(i + 1) % EPL] = v.y;  // (% EPL: no such lane where EPL = 2)
      l[(i + 2) % EPL] = v.z;
      l[(i + 3) % EPL] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < count ? __ldg(row + e0 + i) : -INFINITY;
  }
  // the router's partial sums in order, then its bias
#pragma unroll 1
  for (int ks = 1; ks < slices; ++ks)
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < count) l[i] += __ldg(row + ks * slice_stride + e0 + i);
  if (logit_bias) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < count) l[i] += __ldg(logit_bias + e0 + i);
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
    for (int i = 0; i < EPL; ++i) {
      l[i] = expf(l[i] - vmax);
      s += l[i];
    }
    s = warp_sum(s);
    inv_sum = s == 0.f ? 0.f : 1.f / s;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = sigmoid ? sigmoid_of(l[i]) : l[i] * inv_sum;
  if (bias) {
    if (EPL % 4 == 0 && (n & 3) == 0) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4)
        if (i < count) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(bias + e0 + i));
          l[i] += v.x;
          l[(i + 1) % EPL] += v.y;
          l[(i + 2) % EPL] += v.z;
          l[(i + 3) % EPL] += v.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i < count) l[i] += __ldg(bias + e0 + i);
    }
  }
  // order_key() of the keys, which are never -0, with what is rare set apart
  bool nan = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int b = __float_as_int(l[i]);
    key[i] = b ^ ((b >> 31) & 0x7FFFFFFF);
    nan |= l[i] != l[i];
  }
  if (nan) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l[i] != l[i]) key[i] = INT_MAX;
  }
  if (count < EPL) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i >= count) key[i] = INT_MIN;
  }
  int hk = INT_MIN;  // the lane's best key
  if (rule.groups > 1) {
    auto sum_of = [&](int first, int second) {  // a group's score
      float v = first == INT_MAX ? NAN : order_value(first);
      if (rule.group_top == 2) v += second == INT_MAX ? NAN : order_value(second);
      return order_key(v);
    };
    int a = INT_MIN, b = INT_MIN;  // the two largest keys: the lane's, then the group's
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      b = max(b, min(a, key[i]));
      a = max(a, key[i]);
    }
    hk = a;
    for (int o = 1; o < 1 << span_log2; o <<= 1) {
      const int oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = max(max(b, ob), min(a, oa));
      a = max(a, oa);
    }
    const int sk = g < rule.groups ? sum_of(a, b) : INT_MIN;
    // the group's lanes share the comparisons with the others
    int better = 0;
    const int j = lane & ((1 << span_log2) - 1);
    for (int h0 = 0; h0 < rule.groups; h0 += 1 << span_log2) {
      const int h = h0 + j, o = __shfl_sync(kAll, sk, h << span_log2);
      better += h < rule.groups && (o > sk || (o == sk && h < g));
    }
    for (int o = 1; o < 1 << span_log2; o <<= 1) better += __shfl_xor_sync(kAll, better, o);
    if (better >= rule.top_groups) {
      hk = INT_MIN;
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = INT_MIN;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) hk = max(hk, key[i]);
  }
  __shared__ int4 s_key[4][8];
  __shared__ int s_expert[4][32];
  int* pool = reinterpret_cast<int*>(s_key[threadIdx.x >> 5]);
  int* expert = s_expert[threadIdx.x >> 5];
  int my_idx = 0;
  // a bound: the k-th largest best key (lower where lanes tie; INT_MIN where
  // fewer lanes have one)
  int head = hk, bound = INT_MIN;
  for (int j = 0; j < k; ++j) {
    bound = __reduce_max_sync(kAll, head);
    if (head == bound) head = INT_MIN;
  }
  bound = max(bound, INT_MIN + 1);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) mine += key[i] >= bound;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += v;
  }
  const int n_pool = __shfl_sync(kAll, upto, 31);
  if (n_pool <= 32) {
    pool[lane] = INT_MIN;
    __syncwarp();
    int w = upto - mine;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] >= bound) {
        pool[w] = key[i];
        expert[w++] = e0 + i;
      }
    __syncwarp();
    const int me = pool[lane], my_expert = expert[lane];
    int rank = 0;  // (the pool is in ascending order of experts: of equal keys the earlier one wins)
    for (int q = 0; 4 * q < n_pool; ++q) {
      const int4 o = s_key[threadIdx.x >> 5][q];
      rank += (o.x > me || (o.x == me && 4 * q < lane)) + (o.y > me || (o.y == me && 4 * q + 1 < lane)) +
              (o.z > me || (o.z == me && 4 * q + 2 < lane)) + (o.w > me || (o.w == me && 4 * q + 3 < lane));
    }
    __syncwarp();
    if (lane < n_pool && rank < k) expert[rank] = my_expert;
    __syncwarp();
    if (lane < k) my_idx = expert[lane];
  } else {
    for (int j = 0; j < k; ++j) {
      const int wk = __reduce_max_sync(kAll, hk);
      const int src = __ffs(__ballot_sync(kAll, hk == wk)) - 1;
      int hs = 0;  // (of equal keys the lower expert)
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i) hs = key[i] == hk ? i : hs;
      const int we = __shfl_sync(kAll, e0 + hs, src);
      if (lane == j) my_idx = we;
      if (lane == src) {
        hk = INT_MIN;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (i == hs) key[i] = INT_MIN;
          hk = max(hk, key[i]);
        }
      }
    }
  }
  // the chosen experts' logits again (cheaper than carrying them along)
  float my_v = lane < k ? __ldg(row + my_idx) : -INFINITY;
  if (lane < k) {
    for (int ks = 1; ks < slices; ++ks) my_v += __ldg(row + ks * slice_stride + my_idx);
    if (logit_bias) my_v += __ldg(logit_bias + my_idx);
  }
  if (sigmoid) my_v = sigmoid_of(my_v);
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
    if (inv_sum != inv_sum) w = inv_sum;  // a NaN anywhere in the row: every score is one
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

cudaError_t launch_select_experts(const float* logits, long long row_stride, int slices,
                                  long long slice_stride, const float* logit_bias,
                                  const float* bias, const moe_select_rule& rule, int T, int E,
                                  int k, int32_t* topk_idx, float* topk_w, const int32_t* found,
                                  int32_t* status, cudaStream_t s) {
  const dim3 grid(cdiv(T, 4)), blk(128);
  const int n = E / rule.groups;  // experts of a group
  int span_log2 = 0;
  while (rule.groups * (2 << span_log2) <= 32) ++span_log2;
#define MOE_SELECT(EPL)                                                                          \
  if ((EPL << span_log2) >= n)                                                                   \
  return launch_k(k_select_experts<EPL>, grid, blk, 0, s, true, logits, row_stride, slices,      \
                  slice_stride, logit_bias, bias, rule, n, span_log2, T, k, topk_idx, topk_w,    \
                  found, status)
  MOE_SELECT(2);
  MOE_SELECT(4);
  MOE_SELECT(8);
  MOE_SELECT(16);
  MOE_SELECT(32);
  MOE_SELECT(64);  // (1024 experts in 17 groups: 60 for a lane)
#undef MOE_SELECT
  return cudaErrorInvalidValue;
}

}  // namespace moe
