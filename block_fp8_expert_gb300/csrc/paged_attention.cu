// Attention of one new token per sequence over a paged key/value cache
// (moe_paged_attention).
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),  s_t = scale log2(e) q . k_t
//
// in one pass over the cache with a running maximum m and sum l; the query
// heads of one key/value head (padded to 16) share every cache element read.
#include <algorithm>

#include "decoder_internal.h"

namespace moe {

namespace {

constexpr int kTile = 16;     // tokens per tile: one MMA K step of the second product
constexpr int kWarps = 4;     // warps per CTA, each with its own tiles and pipeline
constexpr int kRows = 16;     // query heads per CTA segment (MMA M)
// E4M3: the largest weight times value scale is held as 2^15, so that fp16
// keeps weights down to 2^-39 of it (a long cache's many small ones)
constexpr float kWTop = 15.f;
constexpr int kMinTiles = 8;  // least tiles per CTA: shorter shares cost more in joining

template <int D, bool E4M3>
struct AttnShape {
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kStage = 2 * kTile * kRowBytes + (E4M3 ? 2 * kTile * 4 : 0);
  static constexpr int kStages = kStage >= 8192 ? 3 : (24576 / kStage < 8 ? 24576 / kStage : 8);
  static constexpr int kWarpBytes = kStages * kStage;
  // the query fragments of D = 256 live in shared memory: with them in
  // registers next to 128 accumulators a thread would need more than 255
  static constexpr bool kQShared = D == 256;
  static constexpr int kQBytes = kQShared ? (D / 16) * 32 * 16 : 0;
  static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
  static constexpr int kCtasPerSm = kSmem > 113 * 1024 ? 1 : 2;
  static_assert(kWarpBytes >= kRows * D * 4, "the join of the warps reuses the stages");
};

struct AttnArgs {
  const uint16_t* q;
  moe_kv_cache c;
  const int32_t* block_table;
  const int32_t* seq_lens;
  moe_attn_dims d;
  int G, gtiles, HG;  // query heads per kv head, 16-head tiles of them, Hkv * gtiles
  uint16_t* out;
  float* part_o;   // [2 * grid][16][D]
  float* part_ml;  // [2 * grid][2][16]
  int grid;
  int32_t* status;
};

// Tokens [lo, len) of sequence b that are attended to, and their tiles.
struct Span {
  int lo, len, first, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  const int len0 = a.seq_lens[b];
  const long long cap = min((long long)a.d.table_width * a.c.page_size, 0x7fffffffll);
  Span s;
  s.len = (int)min((long long)max(len0, 0), cap);
  s.lo = a.d.window > 0 ? max(0, s.len - a.d.window) : 0;
  s.first = s.lo / kTile;
  s.tiles = (int)(((long long)s.len + kTile - 1) / kTile) - s.first;
  if (s.len <= 0) s.tiles = 0;
  return s;
}

// The tiles of all sequences and heads in one row, sequence-major, then head:
// CTA c takes tiles [c share, (c + 1) share).  A sequence's tiles for one
// head are a segment; one that crosses CTAs is joined by k_attn_join.  Every
// thread of the CTA calls this; it returns the sequence that holds tile
// `want` and the tiles (times heads) before it, and the total.
struct Place {
  int b;
  long long before;
};
__device__ __forceinline__ long long plan(const AttnArgs& a, long long* s_scan, Place* s_place,
                                          bool by_share, long long want, Place& at,
                                          long long& share) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
  const int per = cdiv(a.d.B, n), b0 = min(tid * per, a.d.B), b1 = min(b0 + per, a.d.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of(a, b).tiles;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid == 0) *s_place = Place{a.d.B, 0};
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < n / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  total *= a.HG;
  share = max((long long)kMinTiles, (total + a.grid - 1) / a.grid);
  if (by_share) {
    const long long t0 = want * share;
    if (before * a.HG <= t0 && t0 < (before + mine) * a.HG) {
      long long at0 = before;
      int b = b0;
      for (; b < b1; ++b) {
        const int k = span_of(a, b).tiles;
        if (t0 < (at0 + k) * a.HG) break;
        at0 += k;
      }
      *s_place = Place{b, at0 * a.HG};
    }
  } else if (want >= b0 && want < b1) {
    long long at0 = before;
    for (int b = b0; b < (int)want; ++b) at0 += span_of(a, b).tiles;
    *s_place = Place{(int)want, at0 * a.HG};
  }
  __syncthreads();
  at = *s_place;
  return total;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cp_async16_z(uint32_t smem, const void* gmem, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4_z(uint32_t smem, const void* gmem, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem), "l"(gmem),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where 16-byte chunk j of token row r lies in its tile.  bf16: the eight
// rows of one ldmatrix fall on eight different chunks of a 128-byte line.
// E4M3 keys: a quarter-warp reads four neighbouring chunks of two rows;
// values: two neighbouring chunks of four even (or odd) rows.
template <int D, bool E4M3>
__device__ __forceinline__ int k_chunk(int r, int j) {
  if (!E4M3) return j ^ (r & 7);
  return D == 64 ? j : j ^ ((r & 1) << 2);
}
template <int D, bool E4M3>
__device__ __forceinline__ int v_chunk(int r, int j) {
  if (!E4M3) return j ^ (r & 7);
  return D == 64 ? j ^ ((r >> 1) & 3) : j ^ (((r >> 1) & 3) << 1);
}

}  // namespace

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, AttnShape<D, E4M3>::kCtasPerSm)
k_paged_attention(const AttnArgs a) {
  using S = AttnShape<D, E4M3>;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int LPR = S::kRowBytes / 16;       // lanes (16-byte chunks) per token row
  constexpr int NI = kTile * LPR / 32;         // copies per lane and matrix
  constexpr int DPL = D == 64 ? 8 : 16;        // E4M3: dimensions per lane of the second product
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps];
  __shared__ Place s_place;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ unsigned s_seen[kWarps][S::kStages];  // tokens of each stage that exist
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t stages = smem_u32(smem) + warp * S::kWarpBytes;
  uint8_t* const qshared = smem + kWarps * S::kWarpBytes;

  Place at;
  long long share;
  const long long total = plan(a, s_scan, &s_place, true, blockIdx.x, at, share);
  long long cur = (long long)blockIdx.x * share;
  const long long end = min(total, cur + share);
  if (cur >= end) return;
  int b = at.b;
  Span sp = span_of(a, b);
  const long long first_tile = cur;

  while (cur < end) {
    while (cur >= at.before + (long long)sp.tiles * a.HG) {  // next sequence with a token
      at.before += (long long)sp.tiles * a.HG;
      sp = span_of(a, ++b);
    }
    if (tid == 0 && a.seq_lens[b] != sp.len) raise_status(a.status, MOE_DEV_BAD_PAGE);
    const int hg = (int)((cur - at.before) / sp.tiles);
    const long long s0 = at.before + (long long)hg * sp.tiles, s1 = s0 + sp.tiles;
    const long long stop = min(s1, end);
    const int i0 = (int)(cur - s0), i1 = (int)(stop - s0);  // tiles of the segment
    const int hkv = hg / a.gtiles, row0 = (hg % a.gtiles) * kRows;
    const int rows = min(kRows, a.G - row0);

    // ---- this warp's tiles: i0 + warp, + kWarps, ...
    const int n = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;
    const int32_t* table = a.block_table + (size_t)b * a.d.table_stride;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k);
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v);
    // lane i (and i + 16) looks up token i of tile j: its page, or -1
    auto token_of = [&](int j) { return (sp.first + i0 + warp + j * kWarps) * kTile + (lane & 15); };
    auto page_of = [&](int j) {
      if (j >= n) return -1;
      const int tok = token_of(j);
      if (tok < sp.lo || tok >= sp.len) return -1;
      const int p = __ldg(table + (unsigned)tok / (unsigned)a.c.page_size);
      if (p >= 0 && p < a.c.pages) return p;
      raise_status(a.status, MOE_DEV_BAD_PAGE);
      return -1;
    };
    auto issue = [&](int j, int page) {
      if (j < n) {
        const int inpage = (int)((unsigned)token_of(j) % (unsigned)a.c.page_size);
        const long long off =
            page < 0 ? -1
                     : (long long)page * a.c.page_stride + (long long)hkv * a.c.head_stride +
                           (long long)inpage * a.c.token_stride;
        const uint32_t kt = stages + (j % S::kStages) * S::kStage, vt = kt + kTile * S::kRowBytes;
        const unsigned seen = __ballot_sync(kAll, page >= 0);
        if (lane == 0) s_seen[warp][j % S::kStages] = seen;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = i * (32 / LPR) + lane / LPR, ch = lane % LPR;
          const long long o = __shfl_sync(kAll, off, r);
          const bool ok = o >= 0;
          const long long byte = (ok ? o * (E4M3 ? 1 : 2) : 0) + ch * 16;
          cp_async16_z(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, ch) * 16, kbase + byte, ok);
          cp_async16_z(vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, ch) * 16, vbase + byte, ok);
        }
        if (E4M3) {  // lanes 0-15 the keys' scales, 16-31 the values'
          const long long so = page < 0 ? 0
                                        : (long long)page * a.c.scale_page_stride +
                                              (long long)hkv * a.c.scale_head_stride +
                                              (long long)inpage * a.c.scale_token_stride;
          cp_async4_z(vt + kTile * S::kRowBytes + lane * 4,
                      (lane < 16 ? a.c.k_scale : a.c.v_scale) + so, page >= 0);
        }
      }
      cp_async_commit();
    };
    int page = page_of(0);
#pragma unroll 1
    for (int j = 0; j < S::kStages - 1; ++j) {
      const int next = page_of(j + 1);
      issue(j, page);
      page = next;
    }

    // ---- queries: the A operand, rows g and g + 8
    const uint16_t* q0 = a.q + (size_t)b * a.d.q_stride + (size_t)(hkv * a.G + row0) * D;
    float qf[2] = {a.d.scale * 1.44269504088896341f, a.d.scale * 1.44269504088896341f};
    float qn[2] = {1.f, 1.f};
    if (E4M3) {
      // fp16 operands: each row times a power of two that puts its largest
      // magnitude into [2^14, 2^15), undone on the scores (exact)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t m = 0;
        if (g + 8 * h < rows)
          for (int i = c * 8; i < D; i += 32) {
            const uint4 v = ldg16(q0 + (size_t)(g + 8 * h) * D + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) m = max(m, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
          }
        m = max(m, __shfl_xor_sync(kAll, m, 1));
        m = max(m, __shfl_xor_sync(kAll, m, 2));
        const int E = min(exp_of_bits(m << 16), 126);
        qn[h] = pow2f(kGroupTop - E);
        qf[h] *= pow2f(E - kGroupTop);
      }
    }
    auto q_frag = [&](int ks) {
      uint32_t f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = g + 8 * (u & 1);
        int d0;
        if (E4M3)  // chunk of 64 columns ks / 4, step ks % 4: columns 16 c + 4 step + {0,1}, {2,3}
          d0 = 64 * (ks >> 2) + 16 * c + 4 * (ks & 3) + 2 * (u >> 1);
        else
          d0 = 16 * ks + 2 * c + 8 * (u >> 1);
        uint32_t v = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + (size_t)r * D + d0)) : 0u;
        if (E4M3) v = pack_f16x2(bf16_lo(v) * qn[u & 1], bf16_hi(v) * qn[u & 1]);
        f[u] = v;
      }
      return make_uint4(f[0], f[1], f[2], f[3]);
    };
    uint4 qr[S::kQShared ? 1 : D / 16];
    if (S::kQShared) {
      for (int ks = warp; ks < D / 16; ks += kWarps)
        reinterpret_cast<uint4*>(qshared)[ks * 32 + lane] = q_frag(ks);
      __syncthreads();
    } else {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) qr[S::kQShared ? 0 : ks] = q_frag(ks);
    }

    // ---- one pass over the tiles
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) o[i][u] = 0.f;
    // m: running maximum of the scores; w: of score + log2(value scale), the
    // exponent the accumulators are kept at (bf16: the same as m)
    float m[2] = {-INFINITY, -INFINITY}, w[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int next = page_of(j + S::kStages);
      issue(j + S::kStages - 1, page);
      page = next;
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t kt = stages + (j % S::kStages) * S::kStage, vt = kt + kTile * S::kRowBytes;
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int u = 0; u < 4; ++u) s[nt][u] = 0.f;
      auto q_at = [&](int ks) {
        return S::kQShared ? reinterpret_cast<const uint4*>(qshared)[ks * 32 + lane]
                           : qr[S::kQShared ? 0 : ks];
      };
      if (E4M3) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t kb[2][8];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int r = 8 * nt + g;
            decode16_f16(lds128(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, 4 * h + c) * 16), kb[nt]);
          }
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint4 qv = q_at(4 * h + st);
            const uint32_t av[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const uint32_t bv[2] = {kb[nt][2 * st], kb[nt][2 * st + 1]};
              mma_f16_16x8x16(s[nt], av, bv);
            }
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint4 qv = q_at(ks);
          const uint32_t av[4] = {qv.x, qv.y, qv.z, qv.w};
          const int mi = lane >> 3, r = (mi >> 1) * 8 + (lane & 7);
          uint32_t kb[4];
          ldmatrix_x4(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, 2 * ks + (mi & 1)) * 16, kb);
          const uint32_t b0[2] = {kb[0], kb[1]}, b1[2] = {kb[2], kb[3]};
          mma_bf16_16x8x16(s[0], av, b0);
          mma_bf16_16x8x16(s[1], av, b1);
        }
      }
      // scores of tokens 8 nt + 2 c + {0, 1}; -inf where there is none
      float lv[2][2];  // E4M3: log2 of the values' scales
      const unsigned seen = s_seen[warp][j % S::kStages];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tt = 8 * nt + 2 * c + u;
          float ks = 1.f;
          lv[nt][u] = 0.f;
          if (E4M3) {
            const float* sc = reinterpret_cast<const float*>(
                smem + (vt - smem_u32(smem)) + kTile * S::kRowBytes);
            ks = sc[tt];
            lv[nt][u] = __log2f(sc[16 + tt]);
          }
          const bool ok = (seen >> tt) & 1u;
          s[nt][u] = ok ? s[nt][u] * (qf[0] * ks) : -INFINITY;
          s[nt][2 + u] = ok ? s[nt][2 + u] * (qf[1] * ks) : -INFINITY;
        }
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = m[h], wx = w[h];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mx = fmaxf(mx, s[nt][2 * h + u]);
            if (E4M3) wx = fmaxf(wx, s[nt][2 * h + u] + lv[nt][u]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
        if (E4M3) {
          wx = fmaxf(wx, __shfl_xor_sync(kAll, wx, 1));
          wx = fmaxf(wx, __shfl_xor_sync(kAll, wx, 2));
        } else {
          wx = mx;
        }
        // the maxima moved: the sums so far are scaled down to them
        const float ms = mx == -INFINITY ? 0.f : mx, ws = wx == -INFINITY ? 0.f : wx;
        if (mx != m[h]) l[h] *= exp2_fast(m[h] - ms);
        if (__any_sync(kAll, wx != w[h])) {
          const float f = exp2_fast(w[h] - ws);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][2 * h] *= f;
            o[i][2 * h + 1] *= f;
          }
        }
        m[h] = mx;
        w[h] = wx;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float s_a = s[nt][2 * h], s_b = s[nt][2 * h + 1];
          uint32_t p;
          if (E4M3) {
            l[h] += exp2_fast(s_a - ms) + exp2_fast(s_b - ms);
            p = pack_f16x2(exp2_fast(s_a + lv[nt][0] - ws + kWTop),
                           exp2_fast(s_b + lv[nt][1] - ws + kWTop));
          } else {
            p = pack_bf16x2(exp2_fast(s_a - ms), exp2_fast(s_b - ms));
            l[h] += bf16_lo(p) + bf16_hi(p);  // the weights as they are multiplied
          }
          pa[2 * nt + h] = p;
        }
      }
      if (E4M3) {
#pragma unroll
        for (int blk = 0; blk < (D == 256 ? 2 : 1); ++blk) {
          // codes of tokens 2c, 2c + 1, 2c + 8, 2c + 9, this lane's DPL dimensions
          uint32_t v[4][DPL / 4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = 2 * c + (u & 1) + 8 * (u >> 1);
            if (D == 64) {
              const uint32_t addr = vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, g >> 1) * 16 + (g & 1) * 8;
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n"
                           : "=r"(v[u][0]), "=r"(v[u][1])
                           : "r"(addr)
                           : "memory");
            } else {
              const uint4 x = lds128(vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, 8 * blk + g) * 16);
              v[u][0] = x.x;
              v[u][1] = x.y;
              v[u][DPL / 4 - 2] = x.z;
              v[u][DPL / 4 - 1] = x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < DPL / 4; ++i) {
            // bytes (token a, token b) of dimensions 4 i .. 4 i + 3
            const uint32_t lo01 = __byte_perm(v[0][i], v[1][i], 0x5140);
            const uint32_t lo23 = __byte_perm(v[0][i], v[1][i], 0x7362);
            const uint32_t hi01 = __byte_perm(v[2][i], v[3][i], 0x5140);
            const uint32_t hi23 = __byte_perm(v[2][i], v[3][i], 0x7362);
            const uint32_t lo[4] = {lo01 & 0xffffu, lo01 >> 16, lo23 & 0xffffu, lo23 >> 16};
            const uint32_t hi[4] = {hi01 & 0xffffu, hi01 >> 16, hi23 & 0xffffu, hi23 >> 16};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t bv[2] = {e4m3x2_to_f16x2(lo[u]), e4m3x2_to_f16x2(hi[u])};
              mma_f16_16x8x16(o[DPL * blk + 4 * i + u], pa, bv);
            }
          }
        }
      } else {
#pragma unroll
        for (int jj = 0; jj < D / 16; ++jj) {
          const int mi = lane >> 3, r = (mi & 1) * 8 + (lane & 7);
          uint32_t vb[4];
          ldmatrix_x4_trans(vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, 2 * jj + (mi >> 1)) * 16, vb);
          const uint32_t b0[2] = {vb[0], vb[1]}, b1[2] = {vb[2], vb[3]};
          mma_bf16_16x8x16(o[2 * jj], pa, b0);
          mma_bf16_16x8x16(o[2 * jj + 1], pa, b1);
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- join the four warps (their stages are drained)
    float* mine = reinterpret_cast<float*>(smem + warp * S::kWarpBytes);  // [16][D]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kAll, l[h], 1);
      l[h] += __shfl_xor_sync(kAll, l[h], 2);
      if (c == 0) {
        s_m[warp][g + 8 * h] = m[h];
        s_l[warp][g + 8 * h] = l[h];
      }
      // accumulators from exponent w to exponent m
      const float f = (E4M3 && w[h] != -INFINITY) ? exp2f(w[h] - m[h] - kWTop) : 1.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        int d0, d1;
        if (E4M3) {
          d0 = 128 * (i / DPL) * (D == 64 ? 0 : 1) + DPL * 2 * c + i % DPL;
          d1 = d0 + DPL;
        } else {
          d0 = 8 * i + 2 * c;
          d1 = d0 + 1;
        }
        mine[(g + 8 * h) * D + d0] = o[i][2 * h] * f;
        mine[(g + 8 * h) * D + d1] = o[i][2 * h + 1] * f;
      }
    }
    __syncthreads();
    const bool whole = cur == s0 && stop == s1;
    const int slot = 2 * blockIdx.x + (s0 <= first_tile ? 0 : 1);
    for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
      const int r = e / (D / 4), d4 = e % (D / 4);
      float M = s_m[0][r];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) M = fmaxf(M, s_m[x][r]);
      const float Ms = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = exp2f(s_m[x][r] - Ms);
        const float4 v = *reinterpret_cast<const float4*>(smem + x * S::kWarpBytes + ((size_t)r * D + 4 * d4) * 4);
        L = fmaf(s_l[x][r], f, L);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint2 r2;
        r2.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        r2.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(a.out + (size_t)b * a.d.out_stride +
                                  (size_t)(hkv * a.G + row0 + r) * D + 4 * d4) = r2;
      } else {
        *reinterpret_cast<float4*>(a.part_o + ((size_t)slot * kRows + r) * D + 4 * d4) = acc;
        if (d4 == 0) {
          a.part_ml[(size_t)slot * 2 * kRows + r] = M;
          a.part_ml[(size_t)slot * 2 * kRows + kRows + r] = L;
        }
      }
    }
    __syncthreads();
    cur = stop;
  }
}

// Joins the parts of every segment that crosses CTAs, in CTA order, and
// writes the zeros of empty sequences.  One CTA per (sequence, head tile) and
// query head: the parts' maxima and sums first, then their outputs, D / 4
// threads per part and several parts at a time.
template <int D>
__global__ void __launch_bounds__(128)
k_attn_join(const AttnArgs a) {
  constexpr int TP = D / 4, PP = 128 / TP;  // threads per part, parts at a time
  extern __shared__ float s_f[];            // [grid] factor of each part
  __shared__ long long s_scan[4];
  __shared__ Place s_place;
  __shared__ float s_red[4], s_l[PP];
  __shared__ float4 s_acc[PP][TP];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.HG, hg = blockIdx.x % a.HG, r = blockIdx.y;
  const int hkv = hg / a.gtiles, row0 = (hg % a.gtiles) * kRows;
  Place at;
  long long share;
  plan(a, s_scan, &s_place, false, b, at, share);
  const Span sp = span_of(a, b);
  if (row0 + r >= a.G) return;  // uniform
  uint16_t* out = a.out + (size_t)b * a.d.out_stride + (size_t)(hkv * a.G + row0 + r) * D;
  if (sp.tiles == 0) {
    if (tid < TP) *reinterpret_cast<uint2*>(out + 4 * tid) = make_uint2(0, 0);
    if (tid == 0 && a.seq_lens[b] != sp.len) raise_status(a.status, MOE_DEV_BAD_PAGE);
    return;
  }
  const long long s0 = at.before + (long long)hg * sp.tiles, s1 = s0 + sp.tiles;
  const int c0 = (int)(s0 / share), c1 = (int)((s1 - 1) / share);
  if (c0 == c1) return;  // written by its CTA
  griddep_wait();
  const int n = c1 - c0 + 1;
  auto slot_of = [&](int i) { return 2 * (c0 + i) + (s0 <= (c0 + i) * share ? 0 : 1); };
  float M = -INFINITY;
  for (int i = tid; i < n; i += 128) M = fmaxf(M, __ldcg(a.part_ml + (size_t)slot_of(i) * 2 * kRows + r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_red[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  const float Ms = M == -INFINITY ? 0.f : M;
  for (int i = tid; i < n; i += 128)
    s_f[i] = exp2f(__ldcg(a.part_ml + (size_t)slot_of(i) * 2 * kRows + r) - Ms);
  __syncthreads();
  const int p = tid / TP, d4 = tid % TP;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
#pragma unroll 4
  for (int i = p; i < n; i += PP) {
    const float f = s_f[i];
    const size_t sl = (size_t)slot_of(i);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (sl * kRows + r) * D + 4 * d4));
    L = fmaf(__ldcg(a.part_ml + sl * 2 * kRows + kRows + r), f, L);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  s_acc[p][d4] = acc;
  if (d4 == 0) s_l[p] = L;
  __syncthreads();
  if (p == 0) {
    float Lt = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < PP; ++x) {
      Lt += s_l[x];
      const float4 v = s_acc[x][d4];
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
    uint2 r2;
    r2.x = pack_bf16x2(t.x * inv, t.y * inv);
    r2.y = pack_bf16x2(t.z * inv, t.w * inv);
    *reinterpret_cast<uint2*>(out + 4 * d4) = r2;
  }
}

namespace {

int attn_head_tiles(const moe_attn_dims& d, int Hkv) { return Hkv * cdiv(d.Hq / Hkv, kRows); }

// The least CTAs per SM over the shapes bounds nothing: the workspace is
// sized for the most, two.
int attn_max_grid() { return 2 * num_sms(); }

template <int D, bool E4M3>
cudaError_t launch_attn(AttnArgs& a, cudaStream_t s) {
  using S = AttnShape<D, E4M3>;
  cudaError_t err = ensure_smem((const void*)k_paged_attention<D, E4M3>, S::kSmem);
  if (err != cudaSuccess) return err;
  // no more CTAs than the table could give least shares
  const long long most = (long long)a.d.B * a.HG *
                         (((long long)a.d.table_width * a.c.page_size + kTile - 1) / kTile + 1);
  a.grid = (int)std::max(1ll, std::min((long long)S::kCtasPerSm * num_sms(),
                                       (most + kMinTiles - 1) / kMinTiles));
  err = launch_k(k_paged_attention<D, E4M3>, dim3(a.grid), dim3(kWarps * 32), S::kSmem, s, false, a);
  if (err != cudaSuccess) return err;
  return launch_k(k_attn_join<D>, dim3(a.d.B * a.HG, std::min(a.G, kRows)), dim3(128),
                  (size_t)a.grid * sizeof(float), s, true, a);
}

}  // namespace

size_t paged_attention_workspace(const moe_attn_dims&, int D) {
  const size_t slots = 2 * (size_t)attn_max_grid();
  return slots * kRows * ((size_t)D + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const uint16_t* q, const moe_kv_cache& cache,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const moe_attn_dims& d, uint16_t* out, void* ws,
                                   int32_t* status, cudaStream_t s) {
  AttnArgs a{};
  a.q = q;
  a.c = cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.d = d;
  a.G = d.Hq / cache.Hkv;
  a.gtiles = cdiv(a.G, kRows);
  a.HG = attn_head_tiles(d, cache.Hkv);
  a.out = out;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + 2 * (size_t)attn_max_grid() * kRows * cache.D;
  a.status = status;
  const bool f8 = cache.format == MOE_KV_E4M3;
  if (cache.D == 64) return f8 ? launch_attn<64, true>(a, s) : launch_attn<64, false>(a, s);
  if (cache.D == 128) return f8 ? launch_attn<128, true>(a, s) : launch_attn<128, false>(a, s);
  return f8 ? launch_attn<256, true>(a, s) : launch_attn<256, false>(a, s);
}

}  // namespace moe
