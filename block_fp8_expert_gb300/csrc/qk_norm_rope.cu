// Query/key head norms, rotary positions and the store into the paged cache
// in one pass over a token's projected heads (moe_qk_norm_rope).
#include <algorithm>

#include "decoder_internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kRing = 4;
constexpr int kCtasPerSm = 6;  // of 4 warps, as many as the registers allow

struct QkArgs {
  const uint16_t* qkv;
  const float* q_norm;
  const float* k_norm;
  const float* cos_sin;
  const int32_t* pos;
  const int64_t* slots;
  moe_qk_dims d;
  moe_kv_cache c;
  uint16_t* q_out;
  int32_t* status;
  int chunks;  // warps that share a token's heads
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint2 pack_e4m3x8(const float* f, float m) {
  return make_uint2(f32x2_to_e4m3x2(f[0] * m, f[1] * m) | (f32x2_to_e4m3x2(f[2] * m, f[3] * m) << 16),
                    f32x2_to_e4m3x2(f[4] * m, f[5] * m) | (f32x2_to_e4m3x2(f[6] * m, f[7] * m) << 16));
}
__device__ __forceinline__ void load_f32x8(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

}  // namespace

// A lane owns 16 dimensions of one head in two runs of 8 (two 16-byte loads,
// and two stores), so D / 16 lanes make a head and a warp takes 512 / D heads
// per step.  In the half layout the runs of a rotated lane p are 8 p .. and
// rot / 2 + 8 p .., which holds both partners of each pair; otherwise they are
// neighbours, which holds the interleaved pairs: a rotation needs no shuffle.
// The mean of squares and the E4M3 maximum are butterflies over the head's
// lanes.  A token's steps, those of the query heads before the key heads'
// before the value heads', are dealt to `chunks` warps.  A lane's loads go
// through a ring of its own in shared memory (cp.async: registers would hold
// two steps ahead, the ring holds kRing), the first ones on their way before
// the token's position and slot are known.
// Bound by HBM from some thousand tokens on: T 8192, 32 + 4 + 4 heads of 128,
// bf16: 172 MB in 30.9 us, 5.6 TB/s, 0.82 of the copy rate (with eight
// dimensions per lane and shuffles for the partners 64.9; the loads in
// registers 37.6; warps that walk over several tokens 39.7; a ring of 3 or
// 6, or fewer registers for more warps, 34 to 47).  T 8: 2.2 us,
// latency: the token's place, then its heads.  T 517, 16 + 2 + 2 heads of 256,
// E4M3: 5.7 us, the latency and 6.4 ns per token, which bf16 takes as well.
template <int D>
__global__ void __launch_bounds__(128, kCtasPerSm)
k_qk_norm_rope(const QkArgs a) {
  constexpr int LPH = D / 16;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp and step
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ uint4 ring[kRing][2][128];
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / a.chunks), ch = (int)(unit % a.chunks);
  if (t >= a.d.T) return;  // warp-uniform
  const int sub = lane / LPH, p = lane % LPH;
  const int Hq = a.d.Hq, Hkv = a.c.Hkv, rot = a.d.rot, half = rot / 2;
  const bool rotated = 16 * p < rot;
  const bool split = rotated && !a.d.interleaved;
  const int oa = split ? 8 * p : 16 * p, ob = split ? half + 8 * p : 16 * p + 8;
  const int sq = cdiv(Hq, HPW), sk = cdiv(Hkv, HPW), steps = sq + 2 * sk;
  const uint16_t* row = a.qkv + (size_t)t * a.d.qkv_stride;

  // this lane's head of step s, counted within its kind, and its loads
  auto head_of = [&](int s) { return (s < sq ? s : s < sq + sk ? s - sq : s - sq - sk) * HPW + sub; };
  struct Raw {
    uint4 a, b;
  };
  auto fetch = [&](int i) {  // the i-th of this warp's steps
    const int s = ch + i * a.chunks;
    if (s < steps) {
      const int h = head_of(s);
      const bool real = h < (s < sq ? Hq : Hkv);
      const uint16_t* x = row + (real ? (size_t)(h + (s < sq ? 0 : s < sq + sk ? Hq : Hq + Hkv)) * D : 0);
      tc::cp_async16_zfill(&ring[i % kRing][0][threadIdx.x], x + oa, real);
      tc::cp_async16_zfill(&ring[i % kRing][1][threadIdx.x], x + ob, real);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(i);

  // the token's place: its position's rotation row and its cache slot
  const long long slot = a.slots[t];
  bool pos_ok = true;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (rot > 0) {
    const int pos = a.pos[t];
    pos_ok = pos >= 0 && pos < a.d.n_pos;
    if (pos_ok && rotated) {
      const float* tab = a.cos_sin + (size_t)pos * rot + 8 * p;
      load_f32x8(tab, cs);
      load_f32x8(tab + half, sn);
    }
  }
  const long long cap = (long long)a.c.pages * a.c.page_size;
  const bool slot_ok = slot < cap;
  const bool store = slot >= 0 && slot_ok && pos_ok;
  if (lane == 0 && ch == 0) {
    if (!pos_ok) raise_status(a.status, MOE_DEV_BAD_POSITION);
    if (!slot_ok) raise_status(a.status, MOE_DEV_BAD_PAGE);
  }
  long long at = 0, sat = 0;  // the slot's elements of head 0
  if (store) {
    long long page, off;
    if (cap < (1ll << 31)) {
      const unsigned pg = (unsigned)slot / (unsigned)a.c.page_size;
      page = pg;
      off = (unsigned)slot - pg * (unsigned)a.c.page_size;
    } else {
      page = slot / a.c.page_size;
      off = slot % a.c.page_size;
    }
    at = page * a.c.page_stride + off * a.c.token_stride;
    sat = page * a.c.scale_page_stride + off * a.c.scale_token_stride;
  }

  // x = norm and rotation of this lane's run of a head
  auto norm_rope = [&](const Raw& r, const float* weight, float (&x)[16]) {
    unpack_bf16x8(r.a, x);
    unpack_bf16x8(r.b, x + 8);
    if (weight) {
      float ss = 0.f, w[16];
      load_f32x8(weight + oa, w);
      load_f32x8(weight + ob, w + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(kAll, ss, o);
      const float f = rsqrtf(ss * (1.f / D) + a.d.eps);  // (2 ulp)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= f * w[i];
    }
    if (rotated) {
      if (a.d.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * cs[i] - v * sn[i];
          x[2 * i + 1] = v * cs[i] + u * sn[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i], v = x[8 + i];
          x[i] = u * cs[i] - v * sn[i];
          x[8 + i] = v * cs[i] + u * sn[i];
        }
      }
    }
  };
  // codes and scale of a head's run into the cache
  auto store_e4m3 = [&](const float (&x)[16], int h, void* codes, float* scales) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    float f, scale;
    quant_factors(m, f, scale);
    if (h < Hkv) {
      uint8_t* c = static_cast<uint8_t*>(codes) + at + h * a.c.head_stride;
      *reinterpret_cast<uint2*>(c + oa) = pack_e4m3x8(x, f);
      *reinterpret_cast<uint2*>(c + ob) = pack_e4m3x8(x + 8, f);
      if (p == 0) scales[sat + h * a.c.scale_head_stride] = scale;
    }
  };
  const bool e4m3 = a.c.format == MOE_KV_E4M3;
#pragma unroll 1
  for (int s = ch, i = 0; s < steps; s += a.chunks, ++i) {
    fetch(i + kRing - 1);
    cp_async_wait<kRing - 1>();  // (a lane reads what it copied itself)
    const Raw r{ring[i % kRing][0][threadIdx.x], ring[i % kRing][1][threadIdx.x]};
    const int h = head_of(s);
    float x[16];
    if (s < sq) {
      norm_rope(r, a.q_norm, x);
      if (h < Hq) {
        if (!pos_ok) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = NAN;
        }
        uint16_t* q = a.q_out + (size_t)t * a.d.q_stride + (size_t)h * D;
        *reinterpret_cast<uint4*>(q + oa) = pack_bf16x8(x);
        *reinterpret_cast<uint4*>(q + ob) = pack_bf16x8(x + 8);
      }
    } else if (store) {
      if (s < sq + sk) {
        norm_rope(r, a.k_norm, x);
        if (e4m3) {
          store_e4m3(x, h, a.c.k, a.c.k_scale);
        } else if (h < Hkv) {
          uint16_t* c = static_cast<uint16_t*>(a.c.k) + at + h * a.c.head_stride;
          *reinterpret_cast<uint4*>(c + oa) = pack_bf16x8(x);
          *reinterpret_cast<uint4*>(c + ob) = pack_bf16x8(x + 8);
        }
      } else if (e4m3) {
        unpack_bf16x8(r.a, x);
        unpack_bf16x8(r.b, x + 8);
        store_e4m3(x, h, a.c.v, a.c.v_scale);
      } else if (h < Hkv) {  // values are copied as they are
        uint16_t* c = static_cast<uint16_t*>(a.c.v) + at + h * a.c.head_stride;
        *reinterpret_cast<uint4*>(c + oa) = r.a;
        *reinterpret_cast<uint4*>(c + ob) = r.b;
      }
    }
  }
}

cudaError_t launch_qk_norm_rope(const uint16_t* qkv, const float* q_norm, const float* k_norm,
                                const float* cos_sin, const int32_t* pos, const int64_t* slots,
                                const moe_qk_dims& d, const moe_kv_cache& cache, uint16_t* q_out,
                                int32_t* status, cudaStream_t s) {
  QkArgs a{qkv, q_norm, k_norm, cos_sin, pos, slots, d, cache, q_out, status, 1};
  const int hpw = 512 / cache.D, steps = cdiv(d.Hq, hpw) + 2 * cdiv(cache.Hkv, hpw);
  // one step per warp while all of the warps run at once, then as many as keep
  // it so, the same number for each; at most 16 steps per warp.  (32 + 4 + 4
  // heads of 128: T 8 2.2 us, against 5.6 with all of a token's steps in one
  // warp; T 8192 31.1, against 58.5 with one step per warp; T 700 4.1, against
  // 5.6 with uneven warps, T 1000 5.4 against 7.0 with warps for a third more
  // than can run.)
  const long long resident = (long long)num_sms() * kCtasPerSm * 4;
  a.chunks = (int)std::min<long long>(steps, std::max<long long>(cdiv(steps, 16), resident / d.T));
  a.chunks = cdiv(steps, cdiv(steps, a.chunks));
  const long long warps = (long long)d.T * a.chunks;
  const dim3 grid((unsigned)((warps + 3) / 4)), blk(128);
  if (cache.D == 64) return launch_k(k_qk_norm_rope<64>, grid, blk, 0, s, true, a);
  if (cache.D == 128) return launch_k(k_qk_norm_rope<128>, grid, blk, 0, s, true, a);
  return launch_k(k_qk_norm_rope<256>, grid, blk, 0, s, true, a);
}

}  // namespace moe
