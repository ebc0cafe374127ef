// Causal attention over ragged sequences with heads of 128 + 64 query and key
// dimensions, the 64 shared by the keys of all heads, and values of 128
// (moe_expanded_attention: latent attention in its expanded form).
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),  s_t = scale log2(e) q . k_t
//
// in one pass over the keys with a running maximum m and sum l.
//
// A CTA has 256 rows of a head, two query tiles that take turns: while one's
// softmax runs, the tensor cores work for the other.  S = Q K^T of 128 rows by 64
// keys from shared memory, O += P V with the weights P as bf16 in tensor memory,
// in the place of their scores; the scores are made two key tiles ahead.  A thread
// owns a row, so maxima and sums need no exchange; the maximum moves once it is
// exceeded by 2^8 and only then are the outputs rescaled.
//
// Bound by the tensor pipe where prompts are long: one of 8192 tokens and 32 heads
// 497 us, 1.38 PFLOP/s of the half that is not masked, 0.71 of the measured bf16
// rate.  64 keys of both query tiles take 1650 cycles, which is what the MMAs need
// (an S of 128 x 64 x 16 takes 48 cycles for 32 of math: its keys and queries come
// from shared memory; with 128 keys it would take 64 for 64, but then two buffers
// of scores per query tile do not fit next to the outputs: 633 us against 520).
// Short ones are bound by the start and the chain of key tiles, all of which one CTA
// walks: 3 chunks of 9 tokens on contexts of 700, 32 heads: 14.3 us of the GPU; 200
// tokens on a context of 8000, 8 or 32 heads: 117.
// Weights are rounded to bf16 once, as the products take them, and summed as rounded; a
// second part would add 31% to the MMAs.
#include <algorithm>

#include "attention_tc.cuh"

namespace moe {

namespace {

using namespace attn;

constexpr int kNope = 128, kRope = 64, kVd = 128;
constexpr int kBlock = 128;         // rows of a query tile
constexpr int kKeys = 64;           // tokens of a key tile
constexpr int kQChunk = kBlock * 128, kSlot = kKeys * 128;  // rows or tokens x 64 dimensions, 128-byte swizzled
constexpr int kQChunks = (kNope + kRope) / 64, kVChunks = kVd / 64;
constexpr int kStages = 3;          // tiles of keys, and of values, in shared memory
constexpr int kKBytes = kQChunks * kSlot, kVBytes = kVChunks * kSlot;
constexpr int kSoftWarps = 8;       // four per query tile
constexpr int kThreads = (kSoftWarps + 3) * 32;  // then one per query tile for its MMAs, one for the loads
constexpr int kSmem = 2 * kQChunks * kQChunk + kStages * (kKBytes + kVBytes) + 1024;
// TMEM: two buffers of scores (then weights) per query tile, then their outputs
constexpr int kOCol = 4 * kKeys;
constexpr int kHeads = 32;          // heads whose blocks are in one order
constexpr int kHeld = 4;            // sequences per lane up to which blocks are ordered by size

struct ExpandedArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  moe_expanded_dims d;
  int blocks;  // of 256 rows, at most, per head
  int by_size;
  float scale2;
  uint16_t* out;
  int32_t* status;
};

struct ExpandedShared {
  uint64_t q_full[2], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2];
  uint32_t tmem_base;
  volatile int abort_flag;
  int seq, blk;
};

// The rows and keys of a sequence, within the tensors.
struct Seq {
  int q0, lq, k0, lk;
};
__device__ __forceinline__ Seq seq_of(const ExpandedArgs& a, int b, bool* bad = nullptr) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  Seq s;
  s.q0 = min(max(q0, 0), a.d.Tq);
  s.lq = min(max(q1, s.q0), a.d.Tq) - s.q0;
  s.k0 = min(max(k0, 0), a.d.Tk);
  s.lk = min(max(k1, s.k0), a.d.Tk) - s.k0;
  if (bad) *bad = s.q0 != q0 || s.q0 + s.lq != q1 || s.k0 != k0 || s.k0 + s.lk != k1;
  return s;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
k_expanded_attention(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap,
                     const ExpandedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandedShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~(uintptr_t)1023);
  uint8_t* const sm_k = smem + 2 * kQChunks * kQChunk;
  uint8_t* const sm_v = sm_k + kStages * kKBytes;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 2);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.q_full[x], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh.s_full[x][b], 1);
        mbar_init(&sh.p_full[x][b], kSoftWarps / 2);
      }
      mbar_init(&sh.pv_done[x], 1);
    }
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSoftWarps) {
    tc::tmem_alloc(&sh.tmem_base, 512);
    tc::tmem_relinquish();
  }
  griddep_wait();
  griddep_trigger();
  // In groups of kHeads heads, the blocks of the last places in their sequences
  // first, which see the most, and of one place all heads: small blocks are left
  // for the end, and the CTAs at work share few heads' keys.  (One prompt of 8192,
  // 32 heads: 497 us; 7 ragged ones, 20 heads: 63.7; head after head 521 and 76.3.
  // All heads at once: 8192, 128 heads 1915 against 1800.)  Where CTAs are so many
  // that their end does not count, or sequences more than a warp's registers hold:
  // head after head, in the order of the sequences.  (The limit of 32 CTAs per SM, by
  // size against head after head: 40 ragged ones up to 900, 18 per SM 184 us, 192; 16
  // up to 1024, 16 per SM 178.5, 180, 25 per SM 264, 262, 33 per SM 352, 344.5; one of
  // 8192, 28 per SM 1943, 1910; 40 up to 900, 37 per SM 371, 369, 74 per SM 738, 724;
  // 100 short ones up to 300, 29 per SM 194, 206, 58 per SM 392, 406.)
  const int group = a.by_size ? min(kHeads, a.d.H) : 1, span = a.blocks * group;
  const int h0 = (int)(blockIdx.x / span) * group, at = blockIdx.x % span;
  const int heads = min(group, a.d.H - h0), h = h0 + at % heads;
  if (warp == 0) {
    int want = at / heads, seq = -1, blk = 0;
    if (a.by_size) {
      int n[kHeld];  // blocks of the sequences lane, lane + 32, ...
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        n[k] = 0;
        if (32 * k + lane < a.d.B) {
          bool bad;
          n[k] = cdiv(seq_of(a, 32 * k + lane, &bad).lq, 2 * kBlock);
          if (bad && blockIdx.x == 0) raise_status(a.status, MOE_DEV_BAD_POSITION);
        }
      }
      auto from = [&](int place) {  // blocks of this place or later
        int f = 0;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) f += max(n[k] - place, 0);
        return __reduce_add_sync(kAll, f);
      };
      int most = 0;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) most = max(most, n[k]);
      int lo = 0, hi = __reduce_max_sync(kAll, most), later = 0;
      if (want < from(0)) {
        while (hi - lo > 1) {  // from(lo) > want >= from(hi) = later
          const int mid = (lo + hi) / 2, f = from(mid);
          if (f > want) {
            lo = mid;
          } else {
            hi = mid;
            later = f;
          }
        }
        blk = lo;
        want -= later;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const unsigned have = __ballot_sync(kAll, n[k] > lo);
          const bool me = n[k] > lo && __popc(have & ((1u << lane) - 1)) == want;
          const unsigned it = __ballot_sync(kAll, me);
          if (it) seq = 32 * k + __ffs(it) - 1;
          want -= __popc(have);
        }
      }
    } else {
      // (the first CTA checks every sequence)
      for (int b0 = 0; b0 < a.d.B && (seq < 0 || blockIdx.x == 0); b0 += 32) {
        const int b = b0 + lane;
        int n = 0;
        if (b < a.d.B) {
          bool bad;
          n = cdiv(seq_of(a, b, &bad).lq, 2 * kBlock);
          if (bad && blockIdx.x == 0) raise_status(a.status, MOE_DEV_BAD_POSITION);
        }
        if (seq >= 0) continue;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(kAll, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned here = __ballot_sync(kAll, want < incl);
        if (here) {
          const int l = __ffs(here) - 1;
          seq = b0 + l;
          blk = __shfl_sync(kAll, incl, l) - 1 - want;  // (counted from the last)
        } else {
          want -= __shfl_sync(kAll, incl, 31);
        }
      }
    }
    if (lane == 0) {
      sh.seq = seq;
      sh.blk = blk;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  volatile int* const dead = &sh.abort_flag;
  const bool any = sh.seq >= 0;
  const Seq s = any ? seq_of(a, sh.seq) : Seq{0, 0, 0, 0};
  const int row0 = sh.blk * 2 * kBlock, off = s.lk - s.lq;
  // key tiles of either query tile: up to what its last row sees
  auto tiles_of = [&](int x) {
    const int r0 = row0 + x * kBlock;
    if (!any || r0 >= s.lq) return 0;
    return cdiv(max(0, min(r0 + kBlock, s.lq) + off), kKeys);
  };
  const int nt[2] = {tiles_of(0), tiles_of(1)}, n = max(nt[0], nt[1]);

  if (warp == kSoftWarps + 2) {
    // ---- loads, by one thread: queries, then the next tile's keys and this one's
    // values in turn, as scores are made ahead
    if (tc::elect_one()) {
      for (int x = 0; x < 2; ++x)
        if (nt[x] > 0) {
          mbar_arrive_expect_tx(&sh.q_full[x], kQChunks * kQChunk);
          for (int c = 0; c < kQChunks; ++c)
            tma_load_3d(smem + (x * kQChunks + c) * kQChunk, &qmap, 64 * c, h, s.q0 + row0 + x * kBlock,
                        &sh.q_full[x]);
        }
      for (int j = -1; j < n && !*dead; ++j) {
        if (const int k = j + 1, st = k % kStages; k < n) {
          if (k >= kStages) lane_wait(dead, &sh.k_empty[st], (uint32_t)((k / kStages - 1) & 1), a.status);
          if (*dead) break;
          mbar_arrive_expect_tx(&sh.k_full[st], kKBytes);
          uint8_t* to = sm_k + st * kKBytes;
          for (int c = 0; c < 2; ++c)
            tma_load_3d(to + c * kSlot, &kmap, 64 * c, h, s.k0 + k * kKeys, &sh.k_full[st]);
          tc::tma_load_2d(to + 2 * kSlot, &rmap, 0, s.k0 + k * kKeys, &sh.k_full[st]);
        }
        if (j >= 0) {
          const int st = j % kStages;
          if (j >= kStages) lane_wait(dead, &sh.v_empty[st], (uint32_t)((j / kStages - 1) & 1), a.status);
          if (*dead) break;
          mbar_arrive_expect_tx(&sh.v_full[st], kVBytes);
          for (int c = 0; c < kVChunks; ++c)
            tma_load_3d(sm_v + st * kVBytes + c * kSlot, &vmap, 64 * c, h, s.k0 + j * kKeys, &sh.v_full[st]);
        }
      }
      // every copy has landed and been read before the CTA's memory goes
      for (int j = max(0, n - kStages); j < n; ++j) {
        const int st = j % kStages;
        const uint32_t parity = (uint32_t)((j / kStages) & 1);
        mbar_wait(&sh.k_full[st], parity);
        mbar_wait(&sh.v_full[st], parity);
        if (!*dead) {
          mbar_wait(&sh.k_empty[st], parity);
          mbar_wait(&sh.v_empty[st], parity);
        }
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    // ---- the products, a warp per query tile: O += P V of a key tile, then S = Q
    // K^T of the next but one, into the buffer of the weights P
    const int x = warp - kSoftWarps;
    const uint32_t q0 = desc_k(smem_u32(smem) + x * kQChunks * kQChunk);
    const uint32_t kd = desc_k(smem_u32(sm_k)), vd = desc_mn(smem_u32(sm_v), 0);
    const uint32_t t_s = tmem + 2 * x * kKeys, t_o = tmem + kOCol + x * kVd;
    constexpr uint32_t idesc_s = idesc_bf16(kBlock, kKeys, false, false);
    constexpr uint32_t idesc_o = idesc_bf16(kBlock, 64, false, true);
    if (nt[x] > 0) role_wait(dead, &sh.q_full[x], 0, a.status);
    for (int j = -2; j < n; ++j) {
      const int kj = j + 2, jv = max(j, 0);  // the tile whose scores are made, and whose values are added
      const int vs = jv % kStages, ks = kj % kStages;
      const uint32_t u = uniform(vs | ks << 4 | (j & 1) << 8);
      // (a stage that it does not read is given back no sooner either; what there
      // is none of is a wait for what has been waited for)
      const bool pv = j >= 0 && j < nt[x];
      uint64_t* const kb = &sh.k_full[kj < n ? ks : (n - 1) % kStages];
      const uint32_t kp = (uint32_t)(((kj < n ? kj : n - 1) / kStages) & 1);
      if (j >= 0) {
        uint64_t* const vb = &sh.v_full[vs];
        const uint32_t vp = (uint32_t)((jv / kStages) & 1);
        role_wait3(dead, kb, kp, vb, vp, pv ? &sh.p_full[x][j & 1] : vb, pv ? (uint32_t)((j / 2) & 1) : vp, a.status);
      } else if (kj < n) {
        role_wait(dead, kb, kp, a.status);
      }
      tc::fence_after_sync();
      const uint32_t uv = u & 15, uk = u >> 4 & 15, buf = u >> 8;
      if (tc::elect_one() && !*dead) {
        if (j >= 0) {
          if (pv) {
#pragma unroll
            for (int c = 0; c < kVChunks; ++c)
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(t_o + 64 * c, t_s + buf * kKeys + 8 * kk, vd + (uv * kVBytes + c * kSlot + kk * 2048) / 16,
                       idesc_o, 1u);
            tc::commit(&sh.pv_done[x]);
          }
          tc::commit(&sh.v_empty[uv]);
        }
        if (kj < n) {
          if (kj < nt[x]) {
#pragma unroll
            for (int c = 0; c < kQChunks; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(t_s + buf * kKeys, q0 + c * (kQChunk / 16) + 2 * kk, kd + (uk * kKBytes + c * kSlot) / 16 + 2 * kk,
                       idesc_s, c | kk ? 1u : 0u);
            tc::commit(&sh.s_full[x][buf]);
          }
          tc::commit(&sh.k_empty[uk]);
        }
      }
      __syncwarp();
    }
  } else {
    // ---- softmax.  A thread owns a row.
    const int x = warp >> 2, r = 32 * (warp & 3) + lane, i = row0 + x * kBlock + r;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_s = lanes + 2 * x * kKeys, t_o = lanes + kOCol + x * kVd;
    const int limit = i < s.lq ? max(0, i + off + 1) : 0;  // keys that the row sees: the first ones
    // tiles that every row of the warp, or of the CTA, sees whole
    const int whole = (i - lane < s.lq ? max(0, i - lane + off + 1) : s.lk) / kKeys;
    const int whole_cta = max(0, row0 + off + 1) / kKeys;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const bool mine = j < nt[x];
      const uint32_t t_p = t_s + (j & 1) * kKeys;
      float2 v[kKeys / 2];
      if (mine) {
        role_wait(dead, &sh.s_full[x][j & 1], (uint32_t)((j / 2) & 1), a.status);
        tc::fence_after_sync();
        uint32_t raw[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tc::ld_32x32b_x32(t_p + 32 * c, raw[c]);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c)
          v[c] = make_float2(__uint_as_float(raw[c / 16][2 * c % 32]), __uint_as_float(raw[c / 16][2 * c % 32 + 1]));
        if (j >= whole) {
          const int left = limit - j * kKeys;
#pragma unroll
          for (int c = 0; c < kKeys / 2; ++c) {
            if (2 * c >= left) v[c].x = -INFINITY;
            if (2 * c + 1 >= left) v[c].y = -INFINITY;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) mx[c & 3] = max3(mx[c & 3], v[c].x, v[c].y);
        const float top = a.scale2 * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));  // (scale > 0)
        // (-inf + slack is -inf: a row's first score moves its maximum)
        if (__any_sync(kAll, top > m + kMaxSlack)) {
          const float mn = fmaxf(m, top);
          const float f = m == mn ? 1.f : exp2_fast(m - mn);
          l *= f;
          m = mn;
          if (j > 0) {
            role_wait(dead, &sh.pv_done[x], (uint32_t)((j - 1) & 1), a.status);
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < kVd; c += 16) {
              uint32_t o[16];
              ld_32x32b_x16(t_o + c, o);
              tc::wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
              st_32x32b_x16(t_o + c, o);
            }
            tc::wait_st();
          }
        }
        if (j == 0) {  // the products are added to zeros
          const uint32_t zero[16] = {};
#pragma unroll 1
          for (int c = 0; c < kVd; c += 16) st_32x32b_x16(t_o + c, zero);
        }
        const float ms = m == -INFINITY ? 0.f : m;
        float2 sum = make_float2(0.f, 0.f);
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          const float2 e = fma2(v[u], make_float2(a.scale2, a.scale2), make_float2(-ms, -ms));
          w[u] = pack_bf16x2(exp2_fast(e.x), exp2_fast(e.y));
          sum = add2(sum, make_float2(bf16_lo(w[u]), bf16_hi(w[u])));
        }
        tc::st_32x32b_x32(t_p, w);
        l += sum.x + sum.y;
        tc::wait_st();
      }
      if (j >= whole_cta) {
        // Tokens that some rows do not see, or that are another sequence's: a
        // value that is not finite reaches the rows that see it and no other.  It
        // is added to their outputs, and the tile holds 0 in its place (times a
        // weight of 0 it would be NaN).
        uint8_t* chunk[kVChunks];
        bool odd = false;
#pragma unroll
        for (int c = 0; c < kVChunks; ++c) {
          chunk[c] = sm_v + j % kStages * kVBytes + c * kSlot;
          if (c == 0) role_wait(dead, &sh.v_full[j % kStages], (uint32_t)((j / kStages) & 1), a.status);
          for (int e = tid; e < kSlot / 16; e += kSoftWarps * 32) {
            const uint4 w = *reinterpret_cast<const uint4*>(chunk[c] + e * 16);
            odd |= nonfinite_16x2<false>(w.x) || nonfinite_16x2<false>(w.y) || nonfinite_16x2<false>(w.z) ||
                   nonfinite_16x2<false>(w.w);
          }
        }
        if (bar_any(1, kSoftWarps * 32, odd)) {
          if (mine) {
            if (j > 0) role_wait(dead, &sh.pv_done[x], (uint32_t)((j - 1) & 1), a.status);
            tc::fence_after_sync();
#pragma unroll 1
            for (int d0 = 0; d0 < kVd; d0 += 16) {
              uint32_t o[16];
              ld_32x32b_x16(t_o + d0, o);
              tc::wait_ld();
#pragma unroll 1
              for (int t = 0; t < kKeys; ++t) {
                const uint8_t* row = chunk[0] + (d0 >> 6) * (chunk[1] - chunk[0]);
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                  const uint32_t w = *reinterpret_cast<const uint16_t*>(
                      row + tc::sw128_off(t, ((d0 + u) >> 3) & 7) + 2 * (u & 7));
                  if ((w & 0x7F80u) == 0x7F80u && j * kKeys + t < limit)
                    o[u] = __float_as_uint(__uint_as_float(o[u]) + __uint_as_float(w << 16));
                }
              }
              st_32x32b_x16(t_o + d0, o);
            }
            tc::wait_st();
          }
          named_bar(1, kSoftWarps * 32);  // every thread has read the values
#pragma unroll
          for (int c = 0; c < kVChunks; ++c)
            for (int e = tid; e < kSlot / 2; e += kSoftWarps * 32) {
              uint16_t* w = reinterpret_cast<uint16_t*>(chunk[c]) + e;
              if ((*w & 0x7F80u) == 0x7F80u) *w = 0;
            }
          tc::fence_proxy_async();
          named_bar(1, kSoftWarps * 32);  // none is left
        }
      }
      if (mine) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[x][j & 1]);
      }
    }
    // ---- the rows' outputs, through the query tile's shared memory (whose last
    // product has been made), so that a row is written by neighbouring lanes
    const int r_warp = row0 + x * kBlock + 32 * (warp & 3);
    if (any && r_warp < s.lq) {
      uint8_t* const stage = smem + x * kQChunks * kQChunk + (warp & 3) * 32 * 2 * kVd;
      if (nt[x] > 0) {
        role_wait(dead, &sh.pv_done[x], (uint32_t)((nt[x] - 1) & 1), a.status);
        tc::fence_after_sync();
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (nt[x] > 0) {
          tc::ld_32x32b_x32(t_o + 32 * c, o);
          tc::wait_ld();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[8 * u + 2 * e]) * inv, __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
          if (l == 0.f) w[0] = w[1] = w[2] = w[3] = 0u;  // a row that sees nothing
          const int k = 4 * c + u;  // the row's 16-byte chunk
          *reinterpret_cast<uint4*>(stage + lane * 256 + ((k ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      for (int y = 0; y < 32; y += 2) {
        const int row = y + (lane >> 4), k = lane & 15;
        if (r_warp + row < s.lq)
          *reinterpret_cast<uint4*>(a.out + (long long)(s.q0 + r_warp + row) * a.d.out_stride +
                                    h * a.d.out_head_stride + 8 * k) =
              *reinterpret_cast<const uint4*>(stage + row * 256 + ((k ^ (row & 7)) << 4));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kSoftWarps) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

namespace {

long long expanded_blocks(const moe_expanded_dims& d) { return (long long)d.Tq / (2 * kBlock) + d.B; }

}  // namespace

bool expanded_attention_fits(const moe_expanded_dims& d) { return expanded_blocks(d) * d.H < (1ll << 31); }

cudaError_t launch_expanded_attention(const uint16_t* q, const uint16_t* k_nope, const uint16_t* k_rope,
                                      const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                                      const moe_expanded_dims& d, uint16_t* out, int32_t* status,
                                      cudaStream_t s) {
  CUtensorMap qmap, kmap, rmap, vmap;
  cudaError_t err;
  const int Tk = std::max(1, d.Tk);  // (without keys nothing is loaded)
  if (d.Tk == 0) k_nope = k_rope = v = q;
  if ((err = make_tensor_map_3d(&qmap, q, d.Tq, d.H, kNope + kRope, d.q_stride, d.q_head_stride, 64, kBlock)) !=
          cudaSuccess ||
      (err = make_tensor_map_3d(&kmap, k_nope, Tk, d.H, kNope, d.k_stride, d.k_head_stride, 64, kKeys)) !=
          cudaSuccess ||
      (err = make_tensor_map_2d(&rmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k_rope, Tk, kRope, 64, kKeys, 128,
                                d.rope_stride)) != cudaSuccess ||
      (err = make_tensor_map_3d(&vmap, v, Tk, d.H, kVd, d.v_stride, d.v_head_stride, 64, kKeys)) != cudaSuccess)
    return err;
  if ((err = ensure_smem((const void*)k_expanded_attention, kSmem)) != cudaSuccess) return err;
  const long long ctas = expanded_blocks(d) * d.H;
  const ExpandedArgs a{cu_q, cu_k, d, (int)expanded_blocks(d), d.B <= 32 * kHeld && ctas <= 32ll * num_sms(),
                       d.scale * kLog2e, out, status};
  return launch_k(k_expanded_attention, dim3((unsigned)ctas), dim3(kThreads), kSmem, s, true,
                  qmap, kmap, rmap, vmap, a);
}

}  // namespace moe
