// Attention of one new token per sequence over a paged key/value cache
// (moe_paged_attention).
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),  s_t = scale log2(e) q . k_t
//
// in one pass over the cache with a running maximum m and sum l; the query
// heads of one key/value head (up to eight, padded to 8, or 16 of them, padded
// to 16, at a time) share every cache element read.
#include <unistd.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "decoder_internal.h"

namespace moe {

namespace {

constexpr int kWarps = 4;     // warps per CTA, each with its own tiles and pipeline
constexpr int kMaxRows = 16;  // query heads per CTA segment at most
constexpr int kMinTiles = 8;  // least share of a CTA (one user, 8000 tokens: 11.2 us; 16: 12.9)
// What a segment costs a CTA beside its tiles (table and query loads, filling
// and draining the pipeline, the join), in tiles (0 would make 24.5 us, of 48
// ragged sequences up to 4096, 35.7; 16: 27.9).
constexpr int kSegCost = 8;
constexpr int kManySegments = 16;  // CTAs per segment at most for even parts (plan)
// E4M3: the largest weight times value scale is held as 2^15, so that fp16
// keeps weights down to 2^-39 of it (a long cache's many small ones)
constexpr float kWTop = 15.f;

// NH: groups of 8 query heads per CTA segment (the MMA's N).  The figures are
// of 48 ragged E4M3 sequences up to 4096 tokens, 32 + 4 heads of 128 (24.5 us),
// and of two of 131072 with heads of 64 (33.5 us).
template <int D, bool E4M3, int NH>
struct AttnShape {
  static constexpr int kRows = 8 * NH;
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  // 16-token MMA tiles per step: about 8 KB of keys and values (half of that,
  // MT = 1: 31.0 and 48.4 us)
  static constexpr int MT = kRowBytes >= 256 ? 1 : 2;
  static constexpr int kTile = 16 * MT;
  static constexpr int kStage = 2 * kTile * kRowBytes + (E4M3 ? 2 * kTile * 4 : 0);
  // as many as the registers allow (two instead of three: 27.7 and 37.5 us)
  static constexpr int kCtasPerSm = D == 256 ? (E4M3 ? 2 : 1) : (NH == 1 ? 3 : 2);
  static constexpr int kStagesFit = (220 * 1024 / kCtasPerSm - (D == 256 ? 8192 * NH : 0)) / (kWarps * kStage);
  static constexpr int kStages = kStagesFit < 2 ? 2 : (kStagesFit > 6 ? 6 : kStagesFit);
  static constexpr int kWarpBytes = kStages * kStage;
  // the query fragments of D = 256 live in shared memory: with them in
  // registers next to its accumulators a thread would need more than 255
  static constexpr bool kQShared = D == 256;
  static constexpr int kQBytes = kQShared ? (D / 16) * NH * 32 * 8 : 0;
  static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
  static_assert(kWarpBytes >= kRows * D * 4, "the join of the warps reuses the stages");
  static_assert(kSmem + 2048 <= 227 * 1024 / kCtasPerSm, "shared memory");
};

struct AttnArgs {
  const uint16_t* q;
  moe_kv_cache c;
  const int32_t* block_table;
  const int32_t* seq_lens;
  moe_attn_dims d;
  int G, gtiles, HG;  // query heads per kv head; segments per kv head, in all
  int tile;                 // tokens per tile
  uint32_t ps_mul, ps_shift;  // t / page_size = umulhi(t, ps_mul) >> ps_shift (page_size > 1)
  uint16_t* out;
  float* part_o;   // [2 * grid][kMaxRows][D]
  float* part_ml;  // [2 * grid][2][kMaxRows]
  unsigned long long* arrived;  // [3][grid], of any content
  unsigned long long call;      // this launch's number << 8
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
  s.first = s.lo / a.tile;
  s.tiles = (int)(((long long)s.len + a.tile - 1) / a.tile) - s.first;
  if (s.len <= 0) s.tiles = 0;
  return s;
}

// A sequence's tiles for one tile of heads are a segment of tiles + kSegCost
// units; empty sequences have none.  All segments lie in one row, sequence-
// major, then head.  Where there are CTAs enough to give every segment its own
// parts of at most kMinTiles tiles, or else, where there may be a segment for
// every 16 of them (kManySegments), of an even share and a little more, a CTA
// takes one such part: no CTA pays for two segments (with 4 key/value heads of
// 128, bf16: 8 sequences of 2000 tokens 13.9 us against 18.6, 24 up to 2000
// 16.6 against 21.8, 8 of 8000 31.1 against 34.3, but 8 of 65536 168.5 against
// 167.4; with fewer segments the parts are long and their number leaves CTAs
// idle: 2 of 131072 91.8 against 90.7, E4M3 heads of 64 1 of 32000 13.8 against
// 12.1, 2 of 131072 35.3 against 32.6).  Otherwise CTA c takes units [c share, (c + 1)
// share) of the row, and with them the same part of each segment's tiles, so
// ragged batches, many short sequences and a few long ones alike, give every
// CTA the same time.  A segment that several CTAs hold is joined by the last
// of them to be done.  (Units fit 31 bits: the host checks.)
__device__ __forceinline__ int units_of(const Span& s) { return s.tiles ? s.tiles + kSegCost : 0; }
__device__ __forceinline__ int parts_of(int tiles, int most) { return cdiv(tiles, most); }
// The tile at which unit u of a segment begins, in fp32: the CTAs on either
// side get the same answer, and it never falls as u grows.
__device__ __forceinline__ int tile_at(const Span& s, int u) {
  const int units = units_of(s);
  return u <= 0 ? 0 : u >= units ? s.tiles : min(s.tiles, (int)(u * ((float)s.tiles / (float)units)));
}

// A CTA's range of units, the sequence that holds its first one, and where
// that sequence begins; and whether sequence number blockIdx.x is empty (its
// output is zeros, written by this CTA).
struct Place {
  int b, before, cur, end, part;  // part: which one of its segment, where a CTA has one part
  Span span;
  int empty;
};
// Every thread of the CTA calls this.  share: 0 where each CTA has one part,
// of at most `most` tiles.
__device__ __forceinline__ Place plan(const AttnArgs& a, uint2* s_scan, Place* s_place, int& share,
                                      int& most) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = cdiv(a.d.B, kWarps * 32), b0 = min(tid * per, a.d.B), b1 = min(b0 + per, a.d.B);
  if (tid == 0) *s_place = Place{a.d.B, 0, 0, 0, 0, Span{0, 0, 0, 0}, 0};
  uint2 mine = make_uint2(0u, 0u);  // units, parts
  Span span{0, 0, 0, 0};            // of the last of this thread's sequences
  bool empty = false;
  for (int b = b0; b < b1; ++b) {
    span = span_of(a, b);
    empty |= b == (int)blockIdx.x && span.tiles == 0;
    const int u = units_of(span);
    mine.x += u;
    mine.y += parts_of(span.tiles, kMinTiles);
  }
  uint2 before, total;
  auto scan = [&](uint2* s) {
    uint2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x += x;
        incl.y += y;
      }
    }
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    before = make_uint2(incl.x - mine.x, incl.y - mine.y);
    total = make_uint2(0u, 0u);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint2 v = s[w];
      if (w < warp) {
        before.x += v.x;
        before.y += v.y;
      }
      total.x += v.x;
      total.y += v.y;
    }
    total.x *= a.HG;
    total.y *= a.HG;
  };
  scan(s_scan);
  most = kMinTiles;
  share = max((uint32_t)kMinTiles, (total.x + a.grid - 1) / a.grid);
  bool own = total.y <= (uint32_t)a.grid;
  if (!own && a.d.B * a.HG >= cdiv(a.grid, kManySegments)) {  // (the same for every thread)
    most = share + max(kSegCost, share / 6);
    mine.y = 0;
    for (int b = b0; b < b1; ++b) mine.y += parts_of(per > 1 ? span_of(a, b).tiles : span.tiles, most);
    scan(s_scan + kWarps);
    own = total.y <= (uint32_t)a.grid;
  }
  if (own) share = 0;
  // the first unit, or the part, that this CTA looks for
  const uint32_t want = own ? blockIdx.x : min((uint32_t)blockIdx.x * share, total.x);
  const uint32_t from = own ? before.y : before.x, len = own ? mine.y : mine.x;
  if (empty) s_place->empty = 1;
  if (from * a.HG <= want && want < (from + len) * a.HG) {
    uint32_t at = from;
    int b = b0, u = 0, k = 0;
    for (; b < b1; ++b) {
      if (per > 1) span = span_of(a, b);
      u = units_of(span);
      k = own ? parts_of(span.tiles, most) : u;
      if (want < (at + k) * a.HG) break;
      at += k;
      before.x += u;
    }
    const int first = (int)(before.x * a.HG);
    s_place->b = b;
    s_place->before = first;
    s_place->span = span;
    if (own) {
      const int hg = (int)(want - at * a.HG) / k, part = (int)(want - at * a.HG) - hg * k;
      const int s0 = first + hg * u;
      s_place->part = part;
      const int each = u / k, more = u - each * k;  // the first `more` parts have a unit more
      s_place->cur = s0 + part * each + min(part, more);
      s_place->end = s0 + (part + 1) * each + min(part + 1, more);
    } else {
      s_place->cur = (int)want;
      s_place->end = (int)min(want + share, total.x);
    }
  }
  __syncthreads();
  return *s_place;
}

// The counters of arrivals lie in the workspace, which may hold anything.  A
// counter counts while its upper 56 bits are this launch's number, which no
// other launch of the process has, and which what else is there meets with a
// chance of 2^-56.  Every CTA that will arrive readies the counter early: one
// exchange is enough, for if it fails, another CTA's has succeeded.  The last
// one to arrive leaves 0, which is no launch's number, for the next replay of
// the same launch.
__device__ __forceinline__ void ready_counter(unsigned long long* counter, unsigned long long call) {
  const unsigned long long seen = __ldcg(counter);
  if ((seen & ~0xFFull) != call) atomicCAS(counter, seen, call);
}
__device__ __forceinline__ bool last_of(unsigned long long* counter, unsigned n) {
  const bool last = (atomicAdd(counter, 1ull) & 0xFFu) == n - 1;
  if (last) __stcg(counter, 0ull);
  return last;
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
// An 8 x 8 matrix of 16-bit values held as one MMA fragment, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
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

// Two softmax weights as the sum of two bf16 pairs: hi their leading 8 bits, lo
// the rest, rounded (2^-16 of the weight).  The lo of a weight that is not zero
// is at least 2^-126, so that an infinite value meets no zero.
__device__ __forceinline__ float low_part(float a) {
  return fmaxf(a - bf16_hi(__float_as_uint(a)), fminf(a, 0x1p-126f));
}
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  lo = pack_bf16x2(low_part(a), low_part(b));
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

// Joins `count` parts, base, base + step, ..., of the segment that begins in
// CTA c0: to `out` (count is all there is), or into the first one's slot.  A
// thread owns four dimensions of a row, the parts are added in order.
template <int D>
__device__ __forceinline__ void add_parts(const AttnArgs& a, int c0, int slot0, int base, int step,
                                          int count, int rows, uint16_t* out) {
  constexpr int kAhead = 8, kBoth = 2;  // parts, and elements of a thread, on their way at once
  constexpr int kThreads = kWarps * 32;
  const int n = rows * (D / 4);
  auto slot_of = [&](int i) { return (size_t)(base + i == 0 ? slot0 : 2 * (c0 + base + i * step)); };
  for (int e0 = threadIdx.x; e0 < cdiv(n, kThreads) * kThreads; e0 += kBoth * kThreads) {
    float M[kBoth], L[kBoth];
    float4 acc[kBoth];
#pragma unroll
    for (int x = 0; x < kBoth; ++x) {
      M[x] = -INFINITY;
      L[x] = 0.f;
      acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i0 = 0; i0 < count; i0 += kAhead) {
      float4 v[kBoth][kAhead];
      float m[kBoth][kAhead], l[kBoth][kAhead];
#pragma unroll
      for (int x = 0; x < kBoth; ++x)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int e = e0 + x * kThreads, r = e / (D / 4), d4 = e % (D / 4);
          m[x][u] = -INFINITY;
          l[x][u] = 0.f;
          v[x][u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + u < count && e < n) {
            const size_t sl = slot_of(i0 + u);
            const float* ml = a.part_ml + sl * 2 * kMaxRows + r;
            m[x][u] = __ldcg(ml);
            l[x][u] = __ldcg(ml + kMaxRows);
            v[x][u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (sl * kMaxRows + r) * D + 4 * d4));
          }
        }
#pragma unroll
      for (int x = 0; x < kBoth; ++x) {
        float M2 = M[x];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) M2 = fmaxf(M2, m[x][u]);
        const float Ms = M2 == -INFINITY ? 0.f : M2, f0 = exp2f(M[x] - Ms);
        L[x] *= f0;
        acc[x].x *= f0;
        acc[x].y *= f0;
        acc[x].z *= f0;
        acc[x].w *= f0;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float f = exp2f(m[x][u] - Ms);
          L[x] = fmaf(l[x][u], f, L[x]);
          acc[x].x = fmaf(v[x][u].x, f, acc[x].x);
          acc[x].y = fmaf(v[x][u].y, f, acc[x].y);
          acc[x].z = fmaf(v[x][u].z, f, acc[x].z);
          acc[x].w = fmaf(v[x][u].w, f, acc[x].w);
        }
        M[x] = M2;
      }
    }
    if (!out) __syncthreads();  // the rows' other threads have read their m and l
#pragma unroll
    for (int x = 0; x < kBoth; ++x) {
      const int e = e0 + x * kThreads, r = e / (D / 4), d4 = e % (D / 4);
      if (e >= n) continue;
      if (out) {
        const float inv = L[x] == 0.f ? 0.f : 1.f / L[x];
        *reinterpret_cast<uint2*>(out + (size_t)r * D + 4 * d4) =
            make_uint2(pack_bf16x2(acc[x].x * inv, acc[x].y * inv), pack_bf16x2(acc[x].z * inv, acc[x].w * inv));
      } else {
        const size_t sl = slot_of(0);
        *reinterpret_cast<float4*>(a.part_o + (sl * kMaxRows + r) * D + 4 * d4) = acc[x];
        if (d4 == 0) {
          a.part_ml[sl * 2 * kMaxRows + r] = M[x];
          a.part_ml[sl * 2 * kMaxRows + kMaxRows + r] = L[x];
        }
      }
    }
  }
}

// A segment's parts are in their slots.  The last CTA of each kFan neighbouring
// parts adds these up, and the last of those the groups: few parts to read for
// any one, and the same sums whoever comes last.  A CTA begins one segment that
// goes on and continues one at most, so the counters of first groups, of other
// groups and of segments never meet.  (A second kernel for the joins: 27.4
// against 24.5 us for 48 ragged sequences, 7.5 against 5.9 for 30 up to 200,
// and 2 us of the host's time; but 10.0 against 11.2 for one user with 8000
// tokens, whose 32 parts take two rounds here.  Groups of 16: 12.7.)
constexpr int kFan = 8;
struct Parts {
  int c0, slot0;     // the segment's first CTA, the slot of its part
  int parts, first;  // its parts, the first one of this CTA's group
  __device__ __forceinline__ int groups() const { return cdiv(parts, kFan); }
  __device__ __forceinline__ int size() const { return min(kFan, parts - first); }
  __device__ __forceinline__ unsigned long long* group_counter(const AttnArgs& a) const {
    return a.arrived + (first ? a.grid : 0) + c0 + first;
  }
  __device__ __forceinline__ unsigned long long* segment_counter(const AttnArgs& a) const {
    return a.arrived + 2 * a.grid + c0;
  }
};
template <int D>
__device__ __forceinline__ void join_parts(const AttnArgs& a, const Parts& p, int rows,
                                           uint16_t* out, int* s_last) {
  const int groups = p.groups(), size = p.size();
  auto arrive = [&](unsigned long long* counter, int n) {
    __syncthreads();  // (one thread's fences around the arrival hold for what the barriers order)
    if (threadIdx.x == 0) {
      __threadfence();
      *s_last = last_of(counter, n);
      __threadfence();
    }
    __syncthreads();
    return *s_last != 0;
  };
  if (size > 1) {
    if (!arrive(p.group_counter(a), size)) return;
    add_parts<D>(a, p.c0, p.slot0, p.first, 1, size, rows, groups == 1 ? out : nullptr);
    if (groups == 1) return;
  }
  if (!arrive(p.segment_counter(a), groups)) return;
  add_parts<D>(a, p.c0, p.slot0, 0, kFan, groups, rows, out);
}

}  // namespace

// Both products take tokens or dimensions as the MMA's M and the query heads
// as its N = 8, so up to eight heads of a key/value head waste nothing:
//   scores   S^T[token, head] = K Q^T     A = 16 tokens x 16 dimensions
//   outputs  O^T[dim, head]  += V^T P^T   A = 16 dimensions x 16 tokens
// The weights P^T leave the first product as accumulators with a token per
// row and enter the second as its B operand with a token per k: one 8 x 8
// transposition (movmatrix) per 8 tokens.  bf16 operands come out of shared
// memory by ldmatrix; E4M3 codes by 16-byte loads of a permuted order of the
// dimensions (the same for q and k; free for the output) and an exact
// conversion to fp16, the values' codes of two tokens paired by byte permutes.
// A weight rounded to bf16 once would be as far off as the output's own
// rounding (2 x 131072 tokens: 1.95e-3 of the 64-bit result instead of 1.64e-3),
// so bf16 values are multiplied by it in two parts (90.1 -> 90.6 us, 64 ragged
// sequences 59.5 -> 59.7).  Next to E4M3 values one fp16 part stays: it rounds
// eight times finer than the output, and a second one costs more there (48
// ragged sequences 24.6 -> 25.7 us, 16 of 8000 with 16 heads of 256 41.7 -> 46.5).
//
// Bound by HBM once its pipelines are full: 2 x 131072 tokens, 4 heads of 128,
// bf16: 537 MB in 90.6 us, 5.9 TB/s, 0.88 of the copy rate; what is lost is
// the first 5.6 us (lengths, page numbers, rows: loads that wait for one
// another), the SMs' uneven rates (the last ends 12% after the mean) and the
// join.  64 ragged sequences up to 12000: 59.8 us; 48 up to 4096, E4M3: 24.5
// us, 0.51 of the copy rate (the bytes alone take 12).  (With the heads as the
// MMA's M, half of it empty for eight heads, an earlier version took 93, 66.7
// and 56.9 us, and 90, 61 and 41 as it is here.)  One user with 777 tokens: 7.7
// us, all latency (100 tokens, which need no join: 5.1).  A warp runs its tiles
// without any barrier: its own copies, its own maximum, one join per segment.
template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kWarps * 32, AttnShape<D, E4M3, NH>::kCtasPerSm)
k_paged_attention(const AttnArgs a) {
  using S = AttnShape<D, E4M3, NH>;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int MT = S::MT, kTile = S::kTile, kRows = S::kRows;
  constexpr int LPR = S::kRowBytes / 16;       // lanes (16-byte chunks) per token row
  constexpr int NI = kTile * LPR / 32;         // copies per lane and matrix
  constexpr int DPL = D == 64 ? 8 : 16;        // E4M3: dimensions per lane of the second product
  constexpr int kParts = E4M3 ? 1 : 2;         // of a weight
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint2 s_scan[2 * kWarps];
  __shared__ int s_last;
  __shared__ Place s_place;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ unsigned s_seen[kWarps][S::kStages];  // tokens of each stage that exist
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t stages = smem_u32(smem) + warp * S::kWarpBytes;
  uint2* const qshared = reinterpret_cast<uint2*>(smem + kWarps * S::kWarpBytes);

  int share, most;
  Place at = plan(a, s_scan, &s_place, share, most);
  int cur = at.cur;
  const int end = at.end;
  // empty sequences answer zeros: the one of this CTA's number, and those
  // beyond the grid
  for (int e = at.empty ? blockIdx.x : blockIdx.x + a.grid; e < a.d.B; e += a.grid) {
    if (e != (int)blockIdx.x && span_of(a, e).tiles) continue;
    uint4* row = reinterpret_cast<uint4*>(a.out + (size_t)e * a.d.out_stride);
    for (int i = tid; i < a.d.Hq * D / 8; i += kWarps * 32) row[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0 && a.seq_lens[e] != 0) raise_status(a.status, MOE_DEV_BAD_PAGE);
  }
  if (cur >= end) return;
  int b = at.b;
  Span sp = at.span;
  const int first_unit = cur;
  const float scale2 = a.d.scale * 1.44269504088896341f;

  while (cur < end) {
    while (cur >= at.before + units_of(sp) * a.HG) {  // next sequence with a token
      at.before += units_of(sp) * a.HG;
      sp = span_of(a, ++b);
    }
    if (tid == 0 && a.seq_lens[b] != sp.len) raise_status(a.status, MOE_DEV_BAD_PAGE);
    const int units = units_of(sp);
    const int hg = (cur - at.before) / units;
    const int s0 = at.before + hg * units, s1 = s0 + units, stop = min(s1, end);
    const int i0 = tile_at(sp, cur - s0), i1 = tile_at(sp, stop - s0);  // tiles of the segment
    const int hkv = hg / a.gtiles, row0 = (hg % a.gtiles) * kRows;
    const int rows = min(kRows, a.G - row0);

    // ---- this warp's tiles: i0 + warp, + kWarps, ...
    const int n = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;
    const int32_t* table = a.block_table + (size_t)b * a.d.table_stride;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) +
                           (long long)hkv * a.c.head_stride * (E4M3 ? 1 : 2);
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) +
                           (long long)hkv * a.c.head_stride * (E4M3 ? 1 : 2);
    // lane i (and i + 16 of a 16-token tile) looks up token i of tile j: its
    // page (-1: no such token) and its place in the page
    struct Spot {
      int page, inpage;
    };
    auto look_up = [&](int j) {
      Spot r{-1, 0};
      if (j >= n) return r;
      const int tok = (sp.first + i0 + warp + j * kWarps) * kTile + (lane & (kTile - 1));
      if (tok < sp.lo || tok >= sp.len) return r;
      const uint32_t idx = a.c.page_size > 1 ? __umulhi((uint32_t)tok, a.ps_mul) >> a.ps_shift : tok;
      r.inpage = tok - (int)(idx * (uint32_t)a.c.page_size);
      const int p = __ldg(table + idx);
      if (p >= 0 && p < a.c.pages)
        r.page = p;
      else
        raise_status(a.status, MOE_DEV_BAD_PAGE);
      return r;
    };
    auto issue = [&](int j, const Spot& sl) {
      if (j < n) {
        const bool real = sl.page >= 0;
        const long long off = real ? ((long long)sl.page * a.c.page_stride +
                                      (long long)sl.inpage * a.c.token_stride) *
                                         (E4M3 ? 1 : 2)
                                   : -1;
        const uint32_t kt = stages + (j % S::kStages) * S::kStage, vt = kt + kTile * S::kRowBytes;
        const unsigned seen = __ballot_sync(kAll, real);
        if (lane == 0) s_seen[warp][j % S::kStages] = seen;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = i * (32 / LPR) + lane / LPR, ch = lane % LPR;
          const long long o = __shfl_sync(kAll, off, r);
          const bool ok = o >= 0;
          const long long byte = (ok ? o : 0) + ch * 16;
          cp_async16_z(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, ch) * 16, kbase + byte, ok);
          cp_async16_z(vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, ch) * 16, vbase + byte, ok);
        }
        if (E4M3) {  // the scales: kTile of the keys, then kTile of the values
          const long long so = real ? (long long)sl.page * a.c.scale_page_stride +
                                          (long long)hkv * a.c.scale_head_stride +
                                          (long long)sl.inpage * a.c.scale_token_stride
                                    : 0;
          const uint32_t sc = vt + kTile * S::kRowBytes + lane * 4;
          if (MT == 1) {  // lanes 0-15 the keys', 16-31 the values'
            cp_async4_z(sc, (lane < 16 ? a.c.k_scale : a.c.v_scale) + so, real);
          } else {
            cp_async4_z(sc, a.c.k_scale + so, real);
            cp_async4_z(sc + kTile * 4, a.c.v_scale + so, real);
          }
        }
      }
      cp_async_commit();
    };
    Spot spot = look_up(0);

    // ---- queries: the B operand, head 8 nh + g, loaded beside the first page
    // numbers.  E4M3: chunk of 64 columns ks / 4, step ks % 4: columns 16 c +
    // 4 step + {0,1}, {2,3}; the four lanes of a quad hold a whole head.
    const uint16_t* q0 = a.q + (size_t)b * a.d.q_stride + (size_t)(hkv * a.G + row0) * D;
    uint2 qr[D / 16][NH];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const bool real = 8 * nh + g < rows;
      const uint16_t* p = q0 + (real ? (size_t)(8 * nh + g) * D : 0);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (E4M3) {
          qr[ks][nh] = __ldg(reinterpret_cast<const uint2*>(p + 64 * (ks >> 2) + 16 * c + 4 * (ks & 3)));
        } else {
          qr[ks][nh].x = __ldg(reinterpret_cast<const uint32_t*>(p + 16 * ks + 2 * c));
          qr[ks][nh].y = __ldg(reinterpret_cast<const uint32_t*>(p + 16 * ks + 2 * c + 8));
        }
        if (!real) qr[ks][nh] = make_uint2(0u, 0u);
      }
    }
#pragma unroll 1
    for (int j = 0; j < S::kStages - 1; ++j) {
      const Spot next = look_up(j + 1);
      issue(j, spot);
      spot = next;
    }
    const bool whole = cur == s0 && stop == s1;
    auto part_of = [&]() {
      Parts p;
      p.c0 = share ? s0 / share : (int)blockIdx.x - at.part;
      p.slot0 = 2 * p.c0 + (share && s0 > p.c0 * share ? 1 : 0);
      p.parts = share ? (s1 - 1) / share - p.c0 + 1 : parts_of(sp.tiles, most);
      p.first = ((int)blockIdx.x - p.c0) / kFan * kFan;
      return p;
    };
    if (!whole && warp == kWarps - 1 && lane < 2) {  // (its loads are on their way)
      const Parts p = part_of();
      if (lane == 0 ? p.size() > 1 : p.groups() > 1)
        ready_counter(lane == 0 ? p.group_counter(a) : p.segment_counter(a), a.call);
    }
    float qf[NH][2];  // factor on the scores of heads 8 nh + 2 c + {0, 1}
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      qf[nh][0] = qf[nh][1] = scale2;
      if (E4M3) {
        // fp16 operands: each head times a power of two that puts its largest
        // magnitude into [2^14, 2^15), undone on the scores (exact)
        uint32_t m = 0;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint2 v = qr[ks][nh];
          m = max(m, max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu)));
        }
        m = max(m, __shfl_xor_sync(kAll, m, 1));
        m = max(m, __shfl_xor_sync(kAll, m, 2));
        const int E = min(exp_of_bits(m << 16), 126);
        const float f = pow2f(kGroupTop - E), back = pow2f(E - kGroupTop);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint2& v = qr[ks][nh];
          v.x = pack_f16x2(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
          v.y = pack_f16x2(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) qf[nh][u] *= __shfl_sync(kAll, back, 4 * (2 * c + u));
      }
    }
    if (S::kQShared) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
          if ((ks * NH + nh) % kWarps == warp) qshared[(ks * NH + nh) * 32 + lane] = qr[ks][nh];
      __syncthreads();
    }
    auto q_at = [&](int ks, int nh) {
      return S::kQShared ? qshared[(ks * NH + nh) * 32 + lane] : qr[ks][nh];
    };

    // ---- one pass over the tiles
    float o[D / 16][NH][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[i][nh][u] = 0.f;
    // per head 8 nh + 2 c + u: m, the running maximum of the scores, w, that of
    // score + log2(value scale), the exponent the accumulators are kept at
    // (bf16: the same as m), and l, this lane's part of the weights' sum
    float m[NH][2], w[NH][2], l[NH][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[nh][u] = w[nh][u] = -INFINITY;
        l[nh][u] = 0.f;
      }
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const Spot next = look_up(j + S::kStages);
      issue(j + S::kStages - 1, spot);
      spot = next;
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t kt = stages + (j % S::kStages) * S::kStage, vt = kt + kTile * S::kRowBytes;
      float s[MT][NH][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[mt][nh][u] = 0.f;
      if (E4M3) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t lo[8], hi[8];  // tokens 16 mt + g and + 8
            const int r = 16 * mt + g;
            decode16_f16(lds128(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, 4 * h + c) * 16), lo);
            decode16_f16(lds128(kt + (r + 8) * S::kRowBytes + k_chunk<D, E4M3>(r + 8, 4 * h + c) * 16), hi);
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              const uint32_t av[4] = {lo[2 * st], hi[2 * st], lo[2 * st + 1], hi[2 * st + 1]};
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) {
                const uint2 qv = q_at(4 * h + st, nh);
                const uint32_t bv[2] = {qv.x, qv.y};
                mma_f16_16x8x16(s[mt][nh], av, bv);
              }
            }
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // matrices: tokens 0-7 and 8-15 of dimensions 0-7, then of 8-15
            const int mi = lane >> 3, r = 16 * mt + (mi & 1) * 8 + (lane & 7);
            uint32_t av[4];
            ldmatrix_x4(kt + r * S::kRowBytes + k_chunk<D, E4M3>(r, 2 * ks + (mi >> 1)) * 16, av);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              const uint2 qv = q_at(ks, nh);
              const uint32_t bv[2] = {qv.x, qv.y};
              mma_bf16_16x8x16(s[mt][nh], av, bv);
            }
          }
      }
      // scores of tokens 16 mt + g + 8 x; -inf where there is none
      const unsigned seen = s_seen[warp][j % S::kStages];
      float lv[MT][2];  // E4M3: log2 of the values' scales
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int tt = 16 * mt + 8 * x + g;
          float ks = 1.f;
          lv[mt][x] = 0.f;
          if (E4M3) {
            const float* sc = reinterpret_cast<const float*>(
                smem + (vt - smem_u32(smem)) + kTile * S::kRowBytes);
            ks = sc[tt];
            lv[mt][x] = __log2f(sc[kTile + tt]);
          }
          const bool ok = (seen >> tt) & 1u;
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float& v = s[mt][nh][2 * x + u];
              v = ok ? v * (E4M3 ? qf[nh][u] * ks : qf[nh][u]) : -INFINITY;
            }
        }
      uint32_t pb[kParts][MT][NH][2];  // the weights as the second product's B operand
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float mx[2], wx[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mx[u] = m[nh][u];
          wx[u] = w[nh][u];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float v = s[mt][nh][2 * x + u];
              mx[u] = fmaxf(mx[u], v);
              if (E4M3) wx[u] = fmaxf(wx[u], v + lv[mt][x]);
            }
        }
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(kAll, mx[u], sh));
            if (E4M3) wx[u] = fmaxf(wx[u], __shfl_xor_sync(kAll, wx[u], sh));
          }
        float ms[2], ws[2];
        bool moved = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!E4M3) wx[u] = mx[u];
          ms[u] = mx[u] == -INFINITY ? 0.f : mx[u];
          ws[u] = wx[u] == -INFINITY ? 0.f : wx[u];
          moved |= mx[u] != m[nh][u] || wx[u] != w[nh][u];
        }
        if (__any_sync(kAll, moved)) {  // the sums so far are scaled to the new maxima
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float f = exp2_fast(w[nh][u] - ws[u]);
            l[nh][u] *= E4M3 ? exp2_fast(m[nh][u] - ms[u]) : f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[i][nh][u] *= f;
              o[i][nh][2 + u] *= f;
            }
            m[nh][u] = mx[u];
            w[nh][u] = wx[u];
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float sa = s[mt][nh][2 * x], sb = s[mt][nh][2 * x + 1];
            const float pa = exp2_fast(sa - ms[0]), pc = exp2_fast(sb - ms[1]);
            l[nh][0] += pa;
            l[nh][1] += pc;
            uint32_t p[kParts];
            if (E4M3)
              p[0] = pack_f16x2(exp2_fast(sa + lv[mt][x] - ws[0] + kWTop),
                                exp2_fast(sb + lv[mt][x] - ws[1] + kWTop));
            else
              split_weights(pa, pc, p[0], p[kParts - 1]);
#pragma unroll
            for (int y = 0; y < kParts; ++y) pb[y][mt][nh][x] = transpose8x8(p[y]);
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (E4M3) {
#pragma unroll
          for (int blk = 0; blk < (D == 256 ? 2 : 1); ++blk) {
            // codes of tokens 2c, 2c + 1, 2c + 8, 2c + 9, this lane's DPL dimensions
            uint32_t v[4][DPL / 4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int r = 16 * mt + 2 * c + (u & 1) + 8 * (u >> 1);
              if (D == 64) {
                const uint32_t addr =
                    vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, g >> 1) * 16 + (g & 1) * 8;
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
            for (int i = 0; i < DPL / 2; ++i) {
              // dimensions 2 i and 2 i + 1: bytes (token a, token b) of each
              const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
              const uint32_t ta = __byte_perm(v[0][i / 2], v[1][i / 2], sel);
              const uint32_t tb = __byte_perm(v[2][i / 2], v[3][i / 2], sel);
              const uint32_t av[4] = {e4m3x2_to_f16x2(ta & 0xffffu), e4m3x2_to_f16x2(ta >> 16),
                                      e4m3x2_to_f16x2(tb & 0xffffu), e4m3x2_to_f16x2(tb >> 16)};
#pragma unroll
              for (int nh = 0; nh < NH; ++nh)
                mma_f16_16x8x16(o[(DPL / 2) * blk + i][nh], av, pb[0][mt][nh]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            // matrices: dimensions 0-7 and 8-15 of tokens 0-7, then of 8-15
            const int mi = lane >> 3, r = 16 * mt + (mi >> 1) * 8 + (lane & 7);
            uint32_t av[4];
            ldmatrix_x4_trans(vt + r * S::kRowBytes + v_chunk<D, E4M3>(r, 2 * i + (mi & 1)) * 16, av);
#pragma unroll
            for (int y = 0; y < kParts; ++y)
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma_bf16_16x8x16(o[i][nh], av, pb[y][mt][nh]);
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- join the four warps (their stages are drained)
    float* mine = reinterpret_cast<float*>(smem + warp * S::kWarpBytes);  // [kRows][D]
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 8 * nh + 2 * c + u;
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[nh][u] += __shfl_xor_sync(kAll, l[nh][u], sh);
        if (g == 0) {
          s_m[warp][r] = m[nh][u];
          s_l[warp][r] = l[nh][u];
        }
        // accumulators from exponent w to exponent m
        const float f = (E4M3 && w[nh][u] != -INFINITY) ? exp2f(w[nh][u] - m[nh][u] - kWTop) : 1.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          int d0, d1;
          if (E4M3) {
            d0 = 128 * (i / (DPL / 2)) * (D == 64 ? 0 : 1) + DPL * g + 2 * (i % (DPL / 2));
            d1 = d0 + 1;
          } else {
            d0 = 16 * i + g;
            d1 = d0 + 8;
          }
          mine[r * D + d0] = o[i][nh][u] * f;
          mine[r * D + d1] = o[i][nh][2 + u] * f;
        }
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + (s0 <= first_unit ? 0 : 1);
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
        *reinterpret_cast<float4*>(a.part_o + ((size_t)slot * kMaxRows + r) * D + 4 * d4) = acc;
        if (d4 == 0) {
          a.part_ml[(size_t)slot * 2 * kMaxRows + r] = M;
          a.part_ml[(size_t)slot * 2 * kMaxRows + kMaxRows + r] = L;
        }
      }
    }
    __syncthreads();
    if (!whole)
      join_parts<D>(a, part_of(), rows,
                    a.out + (size_t)b * a.d.out_stride + (size_t)(hkv * a.G + row0) * D, &s_last);
    cur = stop;
  }
}

namespace {

// The workspace is sized for the most CTAs per SM that any shape runs.
int attn_max_grid() { return 3 * num_sms(); }

// A number of 56 bits for a launch, counted up from where the process began.
unsigned long long call_number() {
  static std::atomic<unsigned long long> next{[] {
    // (a mix of the time and the process, so that processes begin far apart)
    unsigned long long x = (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() +
                           ((unsigned long long)getpid() << 40);
    x = (x ^ (x >> 31)) * 0xD6E8FEB86659FD93ull;
    return x ^ (x >> 29);
  }()};
  unsigned long long n;
  do {
    n = next.fetch_add(1) & ((1ull << 56) - 1);
  } while (n == 0);
  return n;
}

// The most units that the block table has room for, with `rows` heads per
// segment and `tile` tokens per tile.
long long attn_units(const moe_attn_dims& d, const moe_kv_cache& c, int rows, int tile) {
  const long long tokens = std::min((long long)d.table_width * c.page_size, 0x7fffffffll);
  const long long seg = (tokens + tile - 1) / tile + 1 + kSegCost;
  return (long long)d.B * c.Hkv * cdiv(d.Hq / c.Hkv, rows) * seg;
}

template <int D, bool E4M3, int NH>
cudaError_t launch_attn_nh(AttnArgs& a, cudaStream_t s) {
  using S = AttnShape<D, E4M3, NH>;
  static_assert(S::kCtasPerSm <= 3, "attn_max_grid");
  cudaError_t err = ensure_smem((const void*)k_paged_attention<D, E4M3, NH>, S::kSmem);
  if (err != cudaSuccess) return err;
  a.tile = S::kTile;
  a.gtiles = cdiv(a.G, S::kRows);
  a.HG = a.c.Hkv * a.gtiles;
  // no more CTAs than the table could give parts
  const long long most = attn_units(a.d, a.c, S::kRows, S::kTile) / kMinTiles + (long long)a.d.B * a.HG;
  a.grid = (int)std::max(1ll, std::min((long long)S::kCtasPerSm * num_sms(), most));
  return launch_k(k_paged_attention<D, E4M3, NH>, dim3(a.grid), dim3(kWarps * 32), S::kSmem, s, true, a);
}

template <int D, bool E4M3>
cudaError_t launch_attn(AttnArgs& a, cudaStream_t s) {
  return a.G <= 8 ? launch_attn_nh<D, E4M3, 1>(a, s) : launch_attn_nh<D, E4M3, 2>(a, s);
}

}  // namespace

bool paged_attention_fits(const moe_attn_dims& d, const moe_kv_cache& cache) {
  return attn_units(d, cache, 8, 16) + (1ll << 24) < (1ll << 31);
}

size_t paged_attention_workspace(const moe_attn_dims&, int D) {
  const size_t slots = 2 * (size_t)attn_max_grid();
  return slots * kMaxRows * ((size_t)D + 2) * sizeof(float) +
         3 * attn_max_grid() * sizeof(unsigned long long);
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
  a.out = out;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + 2 * (size_t)attn_max_grid() * kMaxRows * cache.D;
  a.arrived = reinterpret_cast<unsigned long long*>(a.part_ml + 2 * (size_t)attn_max_grid() * 2 * kMaxRows);
  a.call = call_number() << 8;
  a.status = status;
  // t / page_size for 0 <= t < 2^31: with 2^(e-1) < page_size <= 2^e and mul =
  // ceil(2^(31+e) / page_size) < 2^32, floor(t mul / 2^(31+e)) is exact
  int e = 0;
  while ((1ll << e) < cache.page_size) ++e;
  a.ps_mul = (uint32_t)(((1ull << (31 + e)) + cache.page_size - 1) / cache.page_size);
  a.ps_shift = e > 0 ? e - 1 : 0;
  const bool f8 = cache.format == MOE_KV_E4M3;
  if (cache.D == 64) return f8 ? launch_attn<64, true>(a, s) : launch_attn<64, false>(a, s);
  if (cache.D == 128) return f8 ? launch_attn<128, true>(a, s) : launch_attn<128, false>(a, s);
  return f8 ? launch_attn<256, true>(a, s) : launch_attn<256, false>(a, s);
}

}  // namespace moe
