// The latent vector of every token: norm, rotation of its shared key part, the
// store into the paged cache, and the rotation of the queries' heads on the way
// (moe_latent_store).
#include <algorithm>

#include "decoder_internal.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kRot = 64;  // rotated dimensions: of the shared key part and of every query head
constexpr int kRing = 4;
constexpr int kCtasPerSm = 6;  // of 4 warps (T 8192, 128 heads: 8 68.6 us, 4 63.6)

struct StoreArgs {
  const uint16_t* kv;
  const float* norm;
  const float* cos_sin;
  const int32_t* pos;
  const int64_t* slots;
  const uint16_t* q;
  moe_latent_dims d;
  moe_latent_cache c;
  uint16_t* q_out;
  uint16_t* rows;
  int32_t* status;
  int chunks;  // warps that share a token's steps
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

}  // namespace

// Step 0 of a token is its latent vector, R / 32 dimensions per lane (runs of
// 8), the mean of squares a butterfly over the warp.  The other steps are
// eight heads of 64 each, four lanes to a head, of which the last is the shared
// key part: a lane owns 16 dimensions in two runs of 8, in the half layout 8 p ..
// and 32 + 8 p .., which holds both partners of each pair, otherwise
// neighbours, which holds the interleaved pairs, so a rotation needs no shuffle.
// A token's steps are dealt to `chunks` warps; a lane's loads go through a ring
// of its own in shared memory (cp.async), the first ones on their way before the
// token's position and slot are known.
// Bound by bytes (8192 tokens with 128 heads: 299 MB read and written in 62 us in
// the interleaved layout, 0.71 of the copy rate, 56 us in the half layout, 0.79:
// interleaved, an access of a warp has halves of 32-byte sectors, as a lane's two runs
// are neighbours; every token's 16 KB of queries are 64-element runs of strided heads)
// and for few tokens by the launch (T 5: 2.2 us in a graph).
template <int R>
__global__ void __launch_bounds__(128, kCtasPerSm) k_latent_store(const StoreArgs a) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kRuns = R / 256;  // runs of 8 dimensions per lane of the latent vector
  __shared__ uint4 ring[kRing][2][128];
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / a.chunks), ch = (int)(unit % a.chunks);
  if (t >= a.d.T) return;  // warp-uniform
  const int p = lane & 3, H = a.d.H, steps = 1 + cdiv(H + 1, 8);
  const int oa = a.d.interleaved ? 16 * p : 8 * p, ob = a.d.interleaved ? 16 * p + 8 : 32 + 8 * p;
  const uint16_t* kv = a.kv + t * a.d.kv_stride;
  auto head_of = [&](int s) { return 8 * (s - 1) + (lane >> 2); };
  auto fetch = [&](int i) {  // the i-th of this warp's steps
    const int s = ch + i * a.chunks;
    uint4* const to = &ring[i % kRing][0][threadIdx.x];
    if (s == 0) {
#pragma unroll
      for (int u = 0; u < kRuns; ++u) tc::cp_async16_zfill(to + 128 * u, kv + 256 * u + 8 * lane, true);
    } else if (s < steps) {
      const int h = head_of(s);
      const uint16_t* x = h < H ? a.q + t * a.d.q_stride + h * a.d.q_head_stride : kv + R;
      tc::cp_async16_zfill(to, x + oa, h <= H);
      tc::cp_async16_zfill(to + 128, x + ob, h <= H);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(i);

  const long long slot = a.slots[t];
  const int pos = a.pos[t];
  const bool pos_ok = pos >= 0 && pos < a.d.n_pos;
  const long long cap = (long long)a.c.pages * a.c.page_size;
  const bool slot_ok = slot < cap, store = slot >= 0 && slot_ok && pos_ok;
  if (lane == 0 && ch == 0) {
    if (!pos_ok) raise_status(a.status, MOE_DEV_BAD_POSITION);
    if (!slot_ok) raise_status(a.status, MOE_DEV_BAD_PAGE);
  }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = sn[i] = NAN;  // a position outside the table
  if (pos_ok) {
    load8(a.cos_sin + (size_t)pos * kRot + 8 * p, cs);
    load8(a.cos_sin + (size_t)pos * kRot + kRot / 2 + 8 * p, sn);
  }
  uint16_t* const row = a.rows ? a.rows + t * a.d.rows_stride : nullptr;
  uint16_t* place = nullptr;
  if (store) {
    const long long page = slot / a.c.page_size;
    place = static_cast<uint16_t*>(a.c.data) + page * a.c.page_stride +
            (slot - page * a.c.page_size) * a.c.token_stride;
  }

#pragma unroll 1
  for (int s = ch, i = 0; s < steps; s += a.chunks, ++i) {
    fetch(i + kRing - 1);
    cp_async_wait<kRing - 1>();  // (a lane reads what it copied itself)
    const uint4 v0 = ring[i % kRing][0][threadIdx.x], v1 = ring[i % kRing][1][threadIdx.x];
    float x[16];
    unpack8(v0, x);
    if (s > 0 || kRuns > 1) unpack8(v1, x + 8);
    if (s == 0) {
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < 8 * kRuns; ++u) ss = fmaf(x[u], x[u], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
        const float f = rsqrtf(ss * (1.f / R) + a.d.eps);  // (2 ulp)
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
          float w[8];
          load8(a.norm + 256 * u + 8 * lane, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[8 * u + e] *= f * w[e];
        }
      }
      if (!pos_ok) {
#pragma unroll
        for (int e = 0; e < 8 * kRuns; ++e) x[e] = NAN;
      }
#pragma unroll
      for (int u = 0; u < kRuns; ++u) {
        const uint4 o = pack8(x + 8 * u);
        if (place) *reinterpret_cast<uint4*>(place + 256 * u + 8 * lane) = o;
        if (row) *reinterpret_cast<uint4*>(row + 256 * u + 8 * lane) = o;
      }
    } else {
      if (a.d.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[2 * e], v = x[2 * e + 1];
          x[2 * e] = u * cs[e] - v * sn[e];
          x[2 * e + 1] = v * cs[e] + u * sn[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[e], v = x[8 + e];
          x[e] = u * cs[e] - v * sn[e];
          x[8 + e] = v * cs[e] + u * sn[e];
        }
      }
      const int h = head_of(s);
      const uint4 o0 = pack8(x), o1 = pack8(x + 8);
      if (h < H) {
        uint16_t* q = a.q_out + t * a.d.q_out_stride + h * a.d.q_out_head_stride;
        *reinterpret_cast<uint4*>(q + oa) = o0;
        *reinterpret_cast<uint4*>(q + ob) = o1;
      } else if (h == H) {
        if (place) {
          *reinterpret_cast<uint4*>(place + R + oa) = o0;
          *reinterpret_cast<uint4*>(place + R + ob) = o1;
        }
        if (row) {
          *reinterpret_cast<uint4*>(row + R + oa) = o0;
          *reinterpret_cast<uint4*>(row + R + ob) = o1;
        }
      }
    }
  }
}

cudaError_t launch_latent_store(const uint16_t* kv, const float* norm, const float* cos_sin,
                                const int32_t* pos, const int64_t* slots, const uint16_t* q,
                                const moe_latent_dims& d, const moe_latent_cache& cache,
                                uint16_t* q_out, uint16_t* rows, int32_t* status, cudaStream_t s) {
  StoreArgs a{kv, norm, cos_sin, pos, slots, q, d, cache, q_out, rows, status, 1};
  const int steps = 1 + cdiv(d.H + 1, 8);
  // one step per warp while all of the warps run at once, then as many as keep
  // it so, the same number for each, at most 3 (T 8192, 128 heads, 18 steps: 62.0
  // us; 9 steps per warp 65.0, 18 73.8, 1 86.0)
  const long long resident = (long long)num_sms() * kCtasPerSm * 4;
  a.chunks = (int)std::min<long long>(steps, std::max<long long>(cdiv(steps, 3), resident / d.T));
  a.chunks = cdiv(steps, cdiv(steps, a.chunks));
  const long long warps = (long long)d.T * a.chunks;
  const dim3 grid((unsigned)((warps + 3) / 4)), blk(128);
  if (cache.R == 512) return launch_k(k_latent_store<512>, grid, blk, 0, s, true, a);
  return launch_k(k_latent_store<256>, grid, blk, 0, s, true, a);
}

}  // namespace moe
