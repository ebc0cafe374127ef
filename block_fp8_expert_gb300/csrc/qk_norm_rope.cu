// Query/key head norms, rotary positions and the store into the paged cache
// in one pass over a token's projected heads (moe_qk_norm_rope).
#include <algorithm>

#include "decoder_internal.h"

namespace moe {

namespace {

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

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void load_f32x8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

}  // namespace

// A lane owns 8 consecutive dimensions of one head (one 16-byte load and, for
// bf16, one 16-byte store), so LPH = D / 8 lanes make a head and a warp works
// on 32 / LPH heads at once.  A token's heads are dealt to `chunks` warps; a
// warp loads its lanes' cos, sin and norm values once and keeps kAhead head
// loads in flight.  The mean of squares and the E4M3 maximum are butterflies
// over the head's lanes.  Rotation: interleaved pairs sit inside a lane; in
// the half layout the partner of dimension i is rot / 2 away, which is rot /
// 16 lanes (rot a multiple of 16), one shuffle per value.
template <int D>
__global__ void __launch_bounds__(128)
k_qk_norm_rope(const QkArgs a) {
  constexpr int LPH = D / 8;         // lanes per head
  constexpr int HPW = 32 / LPH;      // heads per warp and step
  constexpr int kAhead = 4;
  constexpr unsigned kAll = 0xffffffffu;
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / a.chunks), ch = (int)(unit % a.chunks);
  if (t >= a.d.T) return;  // warp-uniform
  const int sub = lane / LPH, part = lane % LPH, d0 = 8 * part;
  const int Hq = a.d.Hq, Hkv = a.c.Hkv, heads = Hq + 2 * Hkv;
  const int steps = cdiv(heads, HPW);
  const int rot = a.d.rot, half = rot / 2;

  // the first heads are on their way while the token's place is found
  const uint16_t* row = a.qkv + (size_t)t * a.d.qkv_stride;
  uint4 raw[kAhead];
  auto load_heads = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = (s0 + u * a.chunks) * HPW + sub;
      raw[u] = h < heads ? ldg_stream16(row + (size_t)h * D + d0) : make_uint4(0, 0, 0, 0);
    }
  };
  load_heads(ch);

  // the token's place: its position's rotation row and its cache slot
  const long long slot = a.slots[t];
  bool pos_ok = true;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  const bool rotated = d0 < rot;
  const int partner = rotated ? (d0 < half ? part + rot / 16 : part - rot / 16) : part;
  if (rot > 0) {
    const int p = a.pos[t];
    pos_ok = p >= 0 && p < a.d.n_pos;
    if (pos_ok && rotated) {
      const float* row = a.cos_sin + (size_t)p * rot;
      if (a.d.interleaved) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + d0 / 2));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + d0 / 2));
        cs[0] = c4.x; cs[1] = c4.y; cs[2] = c4.z; cs[3] = c4.w;
        sn[0] = s4.x; sn[1] = s4.y; sn[2] = s4.z; sn[3] = s4.w;
      } else {
        const int i0 = d0 < half ? d0 : d0 - half;
        load_f32x8(row + i0, cs);
        load_f32x8(row + half + i0, sn);
      }
    }
  }
  const long long cap = (long long)a.c.pages * a.c.page_size;
  const bool slot_ok = slot < cap;
  const bool store = slot >= 0 && slot_ok && pos_ok;
  if (lane == 0 && ch == 0) {
    if (!pos_ok) raise_status(a.status, MOE_DEV_BAD_POSITION);
    if (!slot_ok) raise_status(a.status, MOE_DEV_BAD_PAGE);
  }
  const long long page = store ? slot / a.c.page_size : 0;
  const long long off = store ? slot % a.c.page_size : 0;
  float qn[8], kn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qn[i] = kn[i] = 1.f;
  if (a.q_norm) load_f32x8(a.q_norm + d0, qn);
  if (a.k_norm) load_f32x8(a.k_norm + d0, kn);

  for (int s0 = ch; s0 < steps; s0 += kAhead * a.chunks) {
    if (s0 != ch) load_heads(s0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int st = s0 + u * a.chunks;
      if (st >= steps) break;  // warp-uniform
      const int h = st * HPW + sub;
      const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
      float x[8];
      unpack_bf16x8(raw[u], x);
      if (st * HPW < Hq + Hkv) {  // warp-uniform: some head here is a query or a key
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(kAll, ss, o);
        const bool normed = is_q ? a.q_norm != nullptr : (!is_v && a.k_norm != nullptr);
        if (normed) {
          const float r = 1.f / sqrtf(ss * (1.f / D) + a.d.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (is_q ? qn[i] : kn[i]);
        }
        if (a.d.interleaved) {
          if (rotated && !is_v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = x[2 * i], q = x[2 * i + 1];
              x[2 * i] = p * cs[i] - q * sn[i];
              x[2 * i + 1] = q * cs[i] + p * sn[i];
            }
          }
        } else if (rot > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(kAll, x[i], sub * LPH + partner);
            if (rotated && !is_v) x[i] = d0 < half ? x[i] * cs[i] - o * sn[i] : x[i] * cs[i] + o * sn[i];
          }
        }
      }
      if (is_q) {
        if (!pos_ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = NAN;
        }
        *reinterpret_cast<uint4*>(a.q_out + (size_t)t * a.d.q_stride + (size_t)h * D + d0) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      }
      if (st * HPW + HPW <= Hq || !store) continue;  // warp-uniform: no key or value to store
      const int kvh = h - Hq - (is_v ? Hkv : 0);
      const long long at = page * a.c.page_stride + kvh * a.c.head_stride + off * a.c.token_stride + d0;
      if (a.c.format == MOE_KV_E4M3) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
        float f, scale;
        quant_factors(m, f, scale);
        if (!is_q && h < heads) {
          uint2 codes;
          codes.x = f32x2_to_e4m3x2(x[0] * f, x[1] * f) | (f32x2_to_e4m3x2(x[2] * f, x[3] * f) << 16);
          codes.y = f32x2_to_e4m3x2(x[4] * f, x[5] * f) | (f32x2_to_e4m3x2(x[6] * f, x[7] * f) << 16);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + at) = codes;
          if (part == 0) {
            float* sc = is_v ? a.c.v_scale : a.c.k_scale;
            sc[page * a.c.scale_page_stride + kvh * a.c.scale_head_stride +
               off * a.c.scale_token_stride] = scale;
          }
        }
      } else if (!is_q && h < heads) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      }
    }
  }
}

cudaError_t launch_qk_norm_rope(const uint16_t* qkv, const float* q_norm, const float* k_norm,
                                const float* cos_sin, const int32_t* pos, const int64_t* slots,
                                const moe_qk_dims& d, const moe_kv_cache& cache, uint16_t* q_out,
                                int32_t* status, cudaStream_t s) {
  QkArgs a{qkv, q_norm, k_norm, cos_sin, pos, slots, d, cache, q_out, status, 1};
  const int steps = cdiv(d.Hq + 2 * cache.Hkv, 32 / (cache.D / 8));
  // one head step per warp while that leaves the SMs short of warps, then
  // more steps per warp, which saves the repeated loads of the token's
  // rotation row
  const long long want = (long long)num_sms() * 32;
  a.chunks = (int)std::min<long long>(steps, std::max<long long>(cdiv(steps, 8), want / d.T));
  const long long warps = (long long)d.T * a.chunks;
  const dim3 grid((unsigned)((warps + 3) / 4)), blk(128);
  if (cache.D == 64) return launch_k(k_qk_norm_rope<64>, grid, blk, 0, s, true, a);
  if (cache.D == 128) return launch_k(k_qk_norm_rope<128>, grid, blk, 0, s, true, a);
  return launch_k(k_qk_norm_rope<256>, grid, blk, 0, s, true, a);
}

}  // namespace moe
