// Attention of several new tokens per sequence, which see each other as a tree,
// over a paged cache: of grouped key/value heads (moe_tree_attention), or of
// one latent vector per token that is key and value of every head
// (moe_latent_attention).
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),  s_t = scale log2(e) q . k_t
//
// in one pass over the cache with a running maximum m and sum l.  The rows of a
// key/value head are its query heads times the new tokens: up to 64 or 128 of
// them share a CTA's pass over the tokens.
//
// Products (tcgen05, fp32 sums in tensor memory): S = Q K^T with the rows as M and
// a tile's 64 tokens as N, the scores of up to two tiles ahead of the softmax;
// O^T += V^T P^T with the value dimensions as M and the rows, rounded up to 16, as
// N.  So few rows cost few cycles in the second product, keys and values are read
// as they lie in the cache (K-major for the first, M-major for the second), and a
// latent vector's tile in shared memory serves both.  P goes through shared
// memory.  The maximum that the weights refer to moves once it is exceeded by 2^8
// (2^5 next to E4M3), which rarely rescales the outputs.
//
// What bounds it: bytes in the middle of a long sequence, otherwise the latency of a
// tile's chain (loads, scores, softmax, weights, outputs) and what stands around the
// tiles: 5 us until the first one is there, a part's end, its outputs through L2 and
// the join.  (GPU times of calls in a graph.)
// Latent vectors of 576, 2 sequences, 64 heads: 131072 tokens 68 us, 262144 114, so
// that a further token costs its bytes at 6.55 TB/s (0.96 of the copy rate) and 22 us
// are around them.  40 sequences of 128 heads: 3000 tokens 71 us, 6000 109.5 (866
// TFLOP/s between them, 32 us around); ragged up to 6000, 56 to 67 us by their lengths.
// Trees of 16 for 32 sequences, 32 / 4 heads of 128, E4M3: 4096 tokens 109 us, 8192
// 190, so a tile of 64 tokens and 128 rows takes 1.5 us, of which 27% of the cycles
// issue and 8% have the tensor pipe at work: latency (28 us are around the tiles); bf16
// 94 and 165.  One sequence of 777 or 900 tokens 11 us.
// Pages that boxes do not divide: 2 x 131072 in pages of 24 75 us, of 1 84, of 8 (eight
// boxes per chunk) 101; the 32 trees, bf16, pages of 16 51 us, of 24 or 1 65; E4M3 65
// and 102 to 107.
// Measured and left out: prefetching later tiles to L2 (2 x 131072: 74.6 us with,
// 71.3 without), one warp that polls the pieces side by side (73.9 against 68.5),
// two CTAs per SM for E4M3 of 128 dimensions (129 us against 114 on the 32 trees).
#include <algorithm>

#include "attention_tc.cuh"

namespace moe {

namespace {

using namespace attn;

constexpr int kTile = 64;      // tokens per tile
constexpr int kChunk = 8192;   // 64 tokens or rows x 64 dimensions, 128-byte swizzled
// What a segment costs a CTA beside its tiles, in tiles.  (32 ragged trees of 16: bf16
// 61 us with 1, 55 with 2, 51 with 3, 52 with 4 or 6; E4M3 89, 74, 69, 62, 61; 40
// ragged latent sequences 67.6, 67.6, 66.8, 66.8, 66.9; 200 short sequences of 2 heads
// 26.2, 25.4, 26.4, 25.9, 27.1.)
constexpr int kSegCost = 3;
constexpr int kNoRow = 0x7fffffff;
// Tiles per part, where there are columns for smaller ones.  (One latent sequence of
// 777 tokens: 13.1 us with 1, 11.8 with 2, 12.7 with 3, 13.9 with 4; 4 of 1000, trees
// of 3, E4M3: 14.8, 14.0, 14.9, 16.3.)
constexpr int kMinTiles = 2;
constexpr int kOCol = 2 * kTile;  // TMEM: two buffers of scores, then the outputs
constexpr long long kMaxTokens = 0x7fffff80;  // of a sequence: its tiles' ends fit 31 bits
// Tiles whose tokens' notes (which are there, their scales) are kept: the codes
// of a tile may be on their way while the softmax reads the notes of the sixth
// before it (two tiles of codes ahead of the stages, two stages, two scores).
constexpr int kNotes = 8;

// LATENT: the values are the leading DV dimensions of the keys.  A stage (64
// tokens) consists of pieces that are loaded, waited for and given back one by
// one: the keys and the values, or, of latent vectors, the 128 dimensions that
// one block of the outputs reads (the first piece with the shared key part).
// TMA: pages of 8, 16, 32 or a multiple of 64 tokens are copied as boxes, E4M3
// codes into a ring of their own, from where warps take them to the stages as
// fp16; other page sizes are gathered token by token.
// ROWS: rows (query head x new token) of a CTA at most, 64 or 128.
template <int DK, int DV, bool LATENT, bool E4M3, bool TMA, int ROWS>
struct DraftShape {
  static constexpr bool kRaw = E4M3 && TMA;
  static constexpr int kKChunks = DK / 64, kVChunks = LATENT ? 0 : DV / 64;
  // Parts of a softmax weight: bf16, next to E4M3 fp16.  One bf16 part next to latent
  // vectors, because a second one has no room: queries (72 KB), two stages (144 KB)
  // and weights (8 KB) of 576 dimensions fill the shared memory, and smaller vectors
  // round alike.  The sums are of the rounded weights, so equal values come out whole.
  static constexpr int kParts = LATENT || E4M3 ? 1 : 2;
  static constexpr int kQChunk = ROWS * 128;  // the rows x 64 dimensions, or tokens
  static constexpr int kQ = kKChunks * kQChunk, kP = kParts * kQChunk;
  static constexpr int kCtas = ROWS == 64 && DK <= (kRaw ? 64 : 128) ? 2 : 1;  // per SM
  static constexpr int kBlocks = DV >= 128 ? DV / 128 : 1;  // of the outputs' dimensions
  static constexpr int kPieces = LATENT ? kBlocks : 2;
  // barriers and small arrays, the tiles' E4M3 scales, and the tiles' alignment
  static constexpr int kFixed = (ROWS == 64 ? 2048 : 4096) + (E4M3 ? kNotes * 2 * kTile * 4 + 256 : 0) + 1024;
  static constexpr int kRoom = 227 * 1024 / kCtas - kFixed - kQ - kP;
  // tiles of keys and of values in shared memory, keys first
  static constexpr int kStages = LATENT && kRoom / (kKChunks * kChunk) >= 4 ? 4 : 2;
  static constexpr int kVStages = LATENT ? kStages : kRaw && kCtas == 2 ? 1 : kRoom / kChunk >= 4 * kKChunks ? 2 : 1;
  static constexpr int kStage = kKChunks * kChunk, kVStage = LATENT ? kStage : kVChunks * kChunk;
  static constexpr int kV = LATENT ? 0 : kStages * kStage;  // where the values begin
  static constexpr int kStaged = kStages * kStage + (LATENT ? 0 : kVStages * kVStage);
  // the ring of codes, each slot 64 tokens' keys or values
  static constexpr int kSlot = kTile * DK;
  static constexpr int kSlotsFit = (kRoom - kStaged) / kSlot;
  // (an even number: a slot is always the keys' or always the values')
  static constexpr int kSlots = !kRaw ? 0 : kSlotsFit >= 4 ? 4 : 2;
  static_assert(kRoom >= kStaged && (!kRaw || kSlotsFit >= 2), "shared memory");
  // softmax warps per 16 rows: they share the tile's tokens
  static constexpr int kSplit = kCtas == 1 && (LATENT || kRaw || ROWS == 128) ? 2 : 1;
  // softmax warps; then two for MMAs; then the loading warps: one for the boxes
  // and those that convert, or one per piece and stage
  static constexpr int kSoft = 4 * kSplit;
  static constexpr int kConvert = kRaw ? 4 * kSplit : 0;
  static constexpr int kWarps = kSoft + 2 + (TMA ? 1 + kConvert : kStages * kPieces);
  static constexpr int kSmem = kQ + kP + kStaged + kSlots * kSlot + 1024;
  static constexpr int kCols = kOCol + kBlocks * ROWS;
  static constexpr int kTmem = kCols <= 256 ? 256 : 512;
  static_assert(kTmem * kCtas <= 512, "TMEM");
};

struct DraftArgs {
  const uint16_t* q;
  moe_kv_cache c;  // the latent cache: one head, v = k
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int64_t* mask;        // NULL: every new token sees those before it
  const int32_t* draft_lens;  // NULL: d.n
  moe_draft_dims d;
  int G, rows, gtiles;  // query heads per key/value head; n G; CTAs that share them
  int tile_rows;        // rows of a CTA at most
  int cols;             // columns of the grid
  int box, box_shift;  // tokens of a page that one copy takes (TMA), a power of two
  uint32_t ps_mul, ps_shift;  // t / page_size = umulhi(t, ps_mul) >> ps_shift (page_size > 1)
  uint16_t* out;
  float* part_o;   // [2 cols][gtiles][tile_rows][DV]
  float* part_ml;  // [2 cols][gtiles][2][tile_rows]
  int2* info;      // [B][Hkv]: the segment's first slot, its parts
  int32_t* status;
};

// A sequence's cached tokens [lo, len), of which those from ctx on are new.
struct Span {
  int lo, len, ctx, first, tiles;
};
__device__ __forceinline__ int drafted(const DraftArgs& a, int b) {
  return a.draft_lens ? a.draft_lens[b] : a.d.n;
}
__device__ __forceinline__ Span span_of(const DraftArgs& a, int b, bool* bad = nullptr) {
  const int len0 = a.seq_lens[b], n0 = drafted(a, b);
  const long long cap = min((long long)a.d.table_width * a.c.page_size, kMaxTokens);
  Span s;
  s.len = (int)min((long long)max(len0, 0), cap);
  const int n = min(min(max(n0, 0), a.d.n), s.len);
  if (bad) *bad = s.len != len0 || (a.draft_lens || s.len > 0 ? n != n0 : false);
  s.ctx = s.len - n;
  s.lo = a.d.window > 0 ? max(0, s.ctx + 1 - a.d.window) : 0;
  s.first = s.lo / kTile;
  s.tiles = n > 0 ? (int)(((long long)s.len + kTile - 1) / kTile) - s.first : 0;
  return s;
}

// A sequence's tiles for one key/value head are a segment; sequences without new
// tokens have none.  All segments lie in one row, sequence-major, then head.
// Where there are columns of the grid enough, each takes one part of one segment
// (share 0): the segments are cut into parts of at most `most` tiles, the least
// of a few sizes with which the parts are no more than the columns.  Otherwise a
// segment counts as tiles + kSegCost units, and column c takes units [c share,
// (c + 1) share) of the row, and with them the same part of each segment's tiles.
// The CTAs of a column do so for different rows of queries: they read the same
// tiles at about the same time, so HBM gives them once.
__device__ __forceinline__ int units_of(const Span& s) { return s.tiles ? s.tiles + kSegCost : 0; }
// The tile at which unit u of a segment begins, in fp32: the columns on either
// side get the same answer, and it never falls as u grows.
__device__ __forceinline__ int tile_at(const Span& s, int u) {
  const int units = units_of(s);
  return u <= 0 ? 0 : u >= units ? s.tiles : min(s.tiles, (int)(u * ((float)s.tiles / (float)units)));
}

// x / y, 0 <= x, 0 < y: a guess in fp32, put right (an integer division takes
// several times as long, and several of them stand before the first load).
__device__ __forceinline__ int quotient(int x, int y) {
  int q = (int)__fdividef((float)x, (float)y);
  while ((long long)q * y > x) --q;
  while ((long long)(q + 1) * y <= x) ++q;
  return q;
}

// What a column does, one segment's part after the other.
struct Part {
  int b, hkv, tile, n;  // tiles [tile, tile + n), in tiles of the sequence
  int slot;             // of a part's results; -1: the whole segment
  int first, parts;     // whether the segment begins here, and then of how many parts it is
  Span sp;
};
struct Walk {
  int b, before, cur, end, first, share, col;
  int part, parts;  // share 0: which part of the segment, of how many
  Span sp;
  __device__ __forceinline__ bool next(const DraftArgs& a, Part& p) {
    if (cur >= end) return false;
    p.sp = sp;
    p.b = b;
    if (!share) {  // cur: the key/value head
      p.hkv = cur++;
      const int each = quotient(sp.tiles, parts), more = sp.tiles - each * parts;
      const int i0 = part * each + min(part, more);  // the first `more` parts have a tile more
      p.tile = sp.first + i0;
      p.n = each + (part < more);
      p.slot = parts == 1 ? -1 : 2 * col;
      p.first = part == 0;
      p.parts = parts;
      return true;
    }
    while (cur >= before + units_of(sp) * a.c.Hkv) {
      before += units_of(sp) * a.c.Hkv;
      sp = span_of(a, ++b);
    }
    const int units = units_of(sp);
    p.sp = sp;
    p.b = b;
    p.hkv = a.c.Hkv == 1 ? 0 : quotient(cur - before, units);
    const int s0 = before + p.hkv * units, s1 = s0 + units, stop = min(s1, end);
    const int i0 = tile_at(sp, cur - s0), i1 = tile_at(sp, stop - s0);
    p.tile = sp.first + i0;
    p.n = i1 - i0;
    p.slot = cur == s0 && stop == s1 ? -1 : 2 * col + (cur == first ? 0 : 1);
    p.first = cur == s0;
    p.parts = p.slot < 0 || !p.first ? 1 : quotient(s1 - 1, share) - col + 1;
    cur = stop;
    return true;
  }
  // The next part that has tiles.
  __device__ __forceinline__ bool next_tiles(const DraftArgs& a, Part& p) {
    while (next(a, p))
      if (p.n > 0) return true;
    return false;
  }
};

// Tiles per part to try, in eighths of an even share.
constexpr int kTries = 5;
__device__ __forceinline__ int most_of(int even, int i) {
  return max(kMinTiles, (even * (8 + i + i / 4 * 4) + 7) / 8);  // 8, 9, 10, 11, 16
}
// Every thread of the CTA calls this.
template <int WARPS>
__device__ __forceinline__ Walk plan(const DraftArgs& a, int col, unsigned (*s_scan)[WARPS], Walk* s_walk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Hkv = a.c.Hkv;
  const int per = cdiv(a.d.B, WARPS * 32), b0 = min(tid * per, a.d.B), b1 = min(b0 + per, a.d.B);
  if (a.d.B == 1 && Hkv <= a.cols) {  // every thread on its own
    Walk w{0, 0, 0, 0, 0, 0, col, 0, 1, span_of(a, 0)};
    const int each = quotient(a.cols, Hkv);  // columns of a head: no more parts than these
    const int most = max(kMinTiles, quotient(w.sp.tiles + each - 1, each));
    w.parts = max(1, quotient(w.sp.tiles + most - 1, most));
    w.cur = quotient(col, w.parts);
    w.part = col - w.cur * w.parts;
    w.end = w.sp.tiles ? min(w.cur + 1, Hkv) : 0;
    return w;
  }
  if (tid == 0) *s_walk = Walk{0, 0, 0, 0, 0, 1, col, 0, 1, Span{0, 0, 0, 0, 0}};
  // Loops that stay loops: what runs once is paid for by the fetch of its code.
  Span span{0, 0, 0, 0, 0};  // of the last of this thread's sequences
  unsigned mine, before, total;
  int most = 0, even = 0, turn = 0;
#pragma unroll 1
  for (int i = -1; i <= kTries; ++i) {
    // i = -1: tiles; then parts with sizes to try; at last units
    const int m = i >= 0 && i < kTries ? most_of(even, i) : 1;
    if (i > 0 && i < kTries && m > even + 2 * kSegCost) continue;  // (a share has two segments at most)
    mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      if (per > 1 || i < 0) span = span_of(a, b);
      mine += i < 0 ? span.tiles : i == kTries ? units_of(span) : quotient(span.tiles + m - 1, m);
    }
    unsigned incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += x;
    }
    unsigned* const s = s_scan[turn ^= 1];  // (some of the sizes are skipped: not by i)
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    const unsigned v = lane < WARPS ? s[lane] : 0;
    total = __reduce_add_sync(kAll, v) * Hkv;
    before = __reduce_add_sync(kAll, lane < warp ? v : 0) + incl - mine;
    // (tiles fit 31 bits: the host checks)
    if (i < 0) {
      even = quotient((int)total + a.cols - 1, a.cols);
    } else if (i < kTries && total <= (unsigned)a.cols) {
      most = m;
      break;
    }
  }
  Walk w;
  w.col = col;
  if (most) {
    if (before * Hkv <= (unsigned)col && (unsigned)col < (before + mine) * Hkv) {
      for (w.b = b0; w.b < b1; ++w.b) {
        w.sp = per > 1 ? span_of(a, w.b) : span;
        w.parts = quotient(w.sp.tiles + most - 1, most);
        if ((unsigned)col < (before + w.parts) * Hkv) break;
        before += w.parts;
      }
      const int k = col - (int)(before * Hkv);
      w.cur = quotient(k, w.parts);
      w.part = k - w.cur * w.parts;
      w.end = w.cur + 1;
      w.before = w.first = w.share = 0;
      *s_walk = w;
    }
  } else {
    const unsigned share = quotient((int)(total + a.cols - 1), a.cols);
    const unsigned want = min((unsigned)col * share, total);
    if (before * Hkv <= want && want < (before + mine) * Hkv) {
      for (w.b = b0; w.b < b1; ++w.b) {
        w.sp = per > 1 ? span_of(a, w.b) : span;
        const unsigned u = units_of(w.sp);
        if (want < (before + u) * Hkv) break;
        before += u;
      }
      w.before = (int)(before * Hkv);
      w.cur = w.first = (int)want;
      w.end = (int)min(want + share, total);
      w.share = (int)share;
      w.part = 0;
      w.parts = 1;
      *s_walk = w;
    }
  }
  __syncthreads();
  return *s_walk;
}

template <int ROWS, int STAGES, int PIECES, int SLOTS, int WARPS, bool E4M3>
struct DraftShared {
  uint64_t raw_full[SLOTS ? SLOTS : 1], raw_empty[SLOTS ? SLOTS : 1];
  uint64_t full[STAGES][PIECES], empty[STAGES][PIECES], s_full[2], s_empty[2], p_full, pv_done, q_full;
  uint32_t tmem_base;
  volatile int abort_flag;
  uint32_t exists[kNotes][2];  // tokens of the tile that are there
  alignas(16) float scale[E4M3 ? kNotes : 1][2][E4M3 ? kTile : 1];  // of its keys and values
  float factor[ROWS];  // on the outputs of a row, when its maximum moves
  int vexp[kNotes];    // E4M3: exponents of the tiles' largest value scales
  float q_scale[2][E4M3 ? ROWS : 1];  // E4M3: of the rows' queries, this part's and the next one's
  union {
    float top[2][ROWS];  // the largest score of a row, by halves of the tile; after the last tile [1]: half of its sum
    float inv[ROWS];     // after the last tile: 1 / the row's sum, E4M3: times what its weights were held at
  };
  union {
    unsigned scan[2][WARPS];
    uint64_t seen[ROWS];  // tokens of the tile that a row sees
    long long at[ROWS];   // after the last tile: the rows' outputs, in elements; -1: none
  };
  Walk walk;
};

// E4M3 codes -> fp16, exact (every E4M3 value is an fp16 value).
__device__ __forceinline__ uint4 e4m3x8_to_f16(uint32_t lo, uint32_t hi) {
  return make_uint4(e4m3x2_to_f16x2(lo & 0xFFFFu), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi & 0xFFFFu),
                    e4m3x2_to_f16x2(hi >> 16));
}
// Next to E4M3 codes the products are of fp16.  Weights times their value's scale
// are held as w 2^(kWTop - e), e one less than the exponent of the largest scale so
// far (so that 2^-e is a normal number for every finite scale); as a maximum moves
// here once it is exceeded by 2^5 (kHalfSlack), they stay below 2^(8 + 5 + 2), and
// fp16 keeps eleven bits down to 2^-23 of the largest, and steps of 2^-33 of it
// below.  (Less slack keeps more of them, but maxima of 128 rows then move in half
// of the tiles: 32 trees of 16: 83.1 us with 2^2.)
constexpr float kWTop = 8.f, kHalfSlack = 5.f;
constexpr int kExpMin = -126;
// e of a scale, for the largest: at most 126 (what is not finite counts as none).
__device__ __forceinline__ int scale_exp(float v) {
  const uint32_t bits = __float_as_uint(v) & 0x7fffffffu;
  return bits >= 0x7f800000u ? kExpMin : max((int)(bits >> 23) - 128, kExpMin);
}
// The largest of 16 scales, of the tokens that a row sees.
__device__ __noinline__ float seen_top(const float* scales, uint32_t seen) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(scales + 4 * i);
    const float f[4] = {fabsf(v.x), fabsf(v.y), fabsf(v.z), fabsf(v.w)};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if ((seen >> (4 * i + u) & 1) && f[u] < INFINITY) top = fmaxf(top, f[u]);
  }
  return top;
}

}  // namespace

template <int DK, int DV, bool LATENT, bool E4M3, bool TMA, int ROWS>
__global__ void __launch_bounds__(DraftShape<DK, DV, LATENT, E4M3, TMA, ROWS>::kWarps * 32,
                                  DraftShape<DK, DV, LATENT, E4M3, TMA, ROWS>::kCtas)
k_draft_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const DraftArgs a) {
  using S = DraftShape<DK, DV, LATENT, E4M3, TMA, ROWS>;
  constexpr int kRows = ROWS;
  constexpr int ST = S::kStages, VST = S::kVStages, NP = S::kPieces, kSoft = S::kSoft, kSoftThreads = kSoft * 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ DraftShared<ROWS, ST, NP, S::kSlots, S::kWarps, E4M3> sh;
  static_assert(sizeof(sh) + 1024 <= S::kFixed, "shared memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~(uintptr_t)1023);
  uint8_t* const sm_q = smem;
  uint8_t* const sm_p = smem + S::kQ;
  uint8_t* const sm_kv = smem + S::kQ + S::kP;
  uint8_t* const sm_raw = sm_kv + S::kStaged;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i)
      for (int x = 0; x < NP; ++x) {
        mbar_init(&sh.full[i][x], S::kRaw ? S::kConvert / 2 : 1);
        mbar_init(&sh.empty[i][x], 1);
      }
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&sh.raw_full[i], 1 + 32);  // the codes, and every lane's scales
      mbar_init(&sh.raw_empty[i], S::kConvert / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], kSoft);
    }
    mbar_init(&sh.p_full, kSoft);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.q_full, kSoft);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (TMA && tid == 32) {
    prefetch_map(&kmap);
    if (!LATENT) prefetch_map(&vmap);
  }
  if (warp == kSoft) {
    tc::tmem_alloc(&sh.tmem_base, S::kTmem);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  griddep_wait();
  griddep_trigger();

  const int col = blockIdx.x / a.gtiles, rt = blockIdx.x % a.gtiles;
  const int row0 = rt * kRows, rows = min(kRows, a.rows - row0);
  const int npad = cdiv(rows, 16) * 16;
  Walk walk = plan<S::kWarps>(a, col, sh.scan, &sh.walk);
  volatile int* const dead = &sh.abort_flag;

  if (TMA && warp == kSoft + 2) {
    // ---- loading: every lane one box of tokens (a page, or 64 tokens of it)
    Part p{};
    struct Box {
      int in, page;  // -1: no token of the box is attended to
    };
    const int shift = a.box_shift, boxes = kTile >> shift;
    // the page number of this lane's box, which nothing waits for yet
    auto look_up = [&](int tile) {
      Box x{0, -1};
      const int t0 = tile * kTile + (lane << shift);
      if (lane < boxes && t0 < p.sp.len && t0 + a.box > p.sp.lo) {
        const uint32_t idx = a.c.page_size > 1 ? __umulhi((uint32_t)t0, a.ps_mul) >> a.ps_shift : t0;
        x.in = t0 - (int)(idx * (uint32_t)a.c.page_size);
        x.page = __ldg(a.block_table + (size_t)p.b * a.d.table_stride + idx);
        if (x.page < 0) x.page = 0x7fffffff;
      }
      return x;
    };
    int j = 0;
    // Until a wait has run out; the same in every lane.  (No copy is started after
    // that: the parities of later waits mean nothing, and what had been started has
    // long landed.)
    bool alive = true;
    while (walk.next_tiles(a, p)) {
      // the tile's boxes, and those of the next two
      Box x, x1 = look_up(p.tile), x2 = look_up(p.tile + 1);
      for (int i = 0; i < p.n; ++i, ++j) {
        x = x1;
        x1 = x2;
        x2 = look_up(p.tile + i + 2);
        const int st = j % ST, note = j % kNotes;
        uint64_t there = 0;  // the box's tokens, as the tile's
        if (x.page >= 0) {
          const int t0 = (p.tile + i) * kTile + (lane << shift);
          if (x.page < a.c.pages)
            there = (low_bits(min(a.box, p.sp.len - t0)) & ~low_bits(p.sp.lo - t0)) << (lane << shift);
          else
            raise_status(a.status, MOE_DEV_BAD_PAGE);
        }
        if ((uint32_t)x.page >= (uint32_t)a.c.pages) x.page = a.c.pages;  // which reads as zeros
        const uint32_t there_lo = __reduce_or_sync(kAll, (uint32_t)there);
        const uint32_t there_hi = __reduce_or_sync(kAll, (uint32_t)(there >> 32));
#pragma unroll
        for (int y = 0; y < NP; ++y) {
          uint64_t* full = &sh.full[st][y];
          if (S::kRaw) {
            const int k = 2 * j + y, slot = k % (S::kSlots ? S::kSlots : 1);
            full = &sh.raw_full[slot];
            if (k >= S::kSlots)
              alive = alive && role_wait(dead, &sh.raw_empty[slot],
                                         (uint32_t)((k / (S::kSlots ? S::kSlots : 1) - 1) & 1), a.status);
          } else if (j >= ST) {  // (as many stages for every piece)
            alive = alive && role_wait(dead, &sh.empty[st][y], (uint32_t)((j / ST - 1) & 1), a.status);
          }
          if (y == 0 && lane == 0) {
            sh.exists[note][0] = there_lo;
            sh.exists[note][1] = there_hi;
          }
          if (!alive) continue;
          constexpr int kFirst = (LATENT ? 3 : S::kKChunks) * kChunk;  // bytes of piece 0
          __syncwarp();
          if (lane == 0)
            mbar_arrive_expect_tx(full, S::kRaw ? S::kSlot : y == 0 ? kFirst : LATENT ? 2 * kChunk : S::kVChunks * kChunk);
          __syncwarp();
          if (lane < boxes) {
            const CUtensorMap* map = !LATENT && y ? &vmap : &kmap;
            if (S::kRaw) {
              uint8_t* to = sm_raw + (2 * j + y) % (S::kSlots ? S::kSlots : 1) * S::kSlot + (lane << shift) * DK;
              tma_load_4d(to, map, 0, x.in, p.hkv, x.page, full);
            } else {
              uint8_t* to = sm_kv + (y && !LATENT ? S::kV + st * S::kVStage : st * S::kStage) + (lane << shift) * 128;
              if (LATENT) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tma_load_4d(to + (2 * y + c) * kChunk, map, 64 * (2 * y + c), x.in, 0, x.page, full);
                if (y == 0) tma_load_4d(to + (S::kKChunks - 1) * kChunk, map, DV, x.in, 0, x.page, full);
              } else {
#pragma unroll
                for (int c = 0; c < S::kKChunks; ++c)
                  tma_load_4d(to + c * kChunk, map, 64 * c, x.in, p.hkv, x.page, full);
              }
            }
          }
          __syncwarp();
          if (S::kRaw) {
            // the tokens' scales, 0 where there is none
            const float* src = y ? a.c.v_scale : a.c.k_scale;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int t = 32 * u + lane, l = t >> shift;
              const int page = __shfl_sync(kAll, x.page, l), in = __shfl_sync(kAll, x.in, l) + (t & (a.box - 1));
              const bool ok = (u ? there_hi : there_lo) >> lane & 1;
              const long long at = ok ? page * a.c.scale_page_stride + p.hkv * a.c.scale_head_stride +
                                            in * a.c.scale_token_stride
                                      : 0;
              cp_async4_zfill(&sh.scale[E4M3 ? note : 0][y][E4M3 ? t : 0], src + at, ok);
            }
            cp_async_arrive(full);
          }
        }
      }
    }
    // every copy has landed before the CTA's memory goes
    cp_async_wait<0>();
    if (lane == 0 && j > 0 && !S::kRaw)
      for (int y = 0; y < NP; ++y)
        for (int k = max(0, j - ST); k < j; ++k) mbar_wait(&sh.full[k % ST][y], (uint32_t)((k / ST) & 1));
    if (lane == 0 && S::kRaw)
      for (int k = max(0, 2 * j - S::kSlots); k < 2 * j; ++k)
        mbar_wait(&sh.raw_full[k % (S::kSlots ? S::kSlots : 1)], (uint32_t)((k / (S::kSlots ? S::kSlots : 1)) & 1));
    __syncwarp();
  } else if (TMA && warp > kSoft + 2) {
    // ---- E4M3 codes to fp16: half of the warps the keys', half the values' (one
    // does not wait for the other's stage), a warp its share of the tokens
    constexpr int kSlots = S::kSlots ? S::kSlots : 1, kTok = kTile / (S::kConvert ? S::kConvert / 2 : 1);
    constexpr int LPR = DK / 16;           // lanes (16-byte chunks) per token row
    constexpr int NI = kTok * LPR / 32;    // chunks per lane
    const int y = (warp - kSoft - 3) & 1, w = (warp - kSoft - 3) >> 1, ch = lane % LPR, jj = 2 * (lane & 3);
    Part p;
    int j = 0;
    while (walk.next_tiles(a, p))
      for (int i = 0; i < p.n; ++i, ++j) {
        const int k = 2 * j + y, slot = k % kSlots, held = y ? VST : ST, st = j % held;
        role_wait(dead, &sh.raw_full[slot], (uint32_t)((k / kSlots) & 1), a.status);
        const uint8_t* src = sm_raw + slot * S::kSlot + w * kTok * DK + lane * 16;
        uint4 codes[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n) codes[n] = *reinterpret_cast<const uint4*>(src + n * 512);
        if (j >= held) role_wait(dead, &sh.empty[st][y], (uint32_t)((j / held - 1) & 1), a.status);
        uint8_t* const to = sm_kv + (y ? S::kV + st * S::kVStage : st * S::kStage) + (ch >> 2) * kChunk;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int r = w * kTok + n * (32 / LPR) + lane / LPR;
          *reinterpret_cast<uint4*>(to + tc::sw128_off(r, jj)) = e4m3x8_to_f16(codes[n].x, codes[n].y);
          *reinterpret_cast<uint4*>(to + tc::sw128_off(r, jj + 1)) = e4m3x8_to_f16(codes[n].z, codes[n].w);
        }
        if (y && w == 0) {
          const float* sc = sh.scale[E4M3 ? j % kNotes : 0][1];
          const int e = max(scale_exp(sc[E4M3 ? lane : 0]), scale_exp(sc[E4M3 ? 32 + lane : 0]));
          sh.vexp[j % kNotes] = __reduce_max_sync(kAll, e);
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.raw_empty[slot]);
          mbar_arrive(&sh.full[st][y]);
        }
      }
  } else if (!TMA && warp > kSoft + 1) {
    // ---- loading, token by token: a warp per piece and stage, so that waiting for
    // one piece's copies holds up no other
    const int stage = (warp - kSoft - 2) / NP, piece = (warp - kSoft - 2) % NP;
    uint64_t* const full = &sh.full[stage][piece];
    uint64_t* const empty = &sh.empty[stage][piece];
    uint8_t* const dst = sm_kv + (piece && !LATENT ? S::kV + stage * S::kVStage : stage * S::kStage);
    struct Tok {
      long long at;   // elements from the head's first; -1: no such token
      long long sat;  // E4M3: of its scales
    };
    Part p;
    bool more = walk.next_tiles(a, p);
    int i = stage;  // the tile of this part
    auto settle = [&]() {
      while (more && i >= p.n) {
        i -= p.n;
        more = walk.next_tiles(a, p);
      }
    };
    auto look_up = [&](Tok (&tk)[2]) {  // of tokens lane and lane + 32
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        tk[u].at = -1;
        tk[u].sat = 0;
        const int tok = (p.tile + i) * kTile + 32 * u + lane;
        if (!more || tok < p.sp.lo || tok >= p.sp.len) continue;
        const uint32_t idx = a.c.page_size > 1 ? __umulhi((uint32_t)tok, a.ps_mul) >> a.ps_shift : tok;
        const int in = tok - (int)(idx * (uint32_t)a.c.page_size);
        const int page = __ldg(a.block_table + (size_t)p.b * a.d.table_stride + idx);
        if (page < 0 || page >= a.c.pages) {
          raise_status(a.status, MOE_DEV_BAD_PAGE);
          continue;
        }
        tk[u].at = page * a.c.page_stride + p.hkv * a.c.head_stride + in * a.c.token_stride;
        if (E4M3)
          tk[u].sat = page * a.c.scale_page_stride + p.hkv * a.c.scale_head_stride +
                      in * a.c.scale_token_stride;
      }
    };
    settle();
    Tok tk[2];
    look_up(tk);
    for (int round = 0; more; ++round) {
      const int note = (round * ST + stage) % kNotes;
      const uint32_t there[2] = {__ballot_sync(kAll, tk[0].at >= 0), __ballot_sync(kAll, tk[1].at >= 0)};
      if (E4M3) {
        // codes to registers, and as fp16 into the stage once it is free
        constexpr int LPR = DK / 16;          // lanes (16-byte chunks) per token row
        constexpr int NI = kTile * LPR / 32;  // loads per lane
        const uint8_t* const src = static_cast<const uint8_t*>(piece ? a.c.v : a.c.k);
        const float* const scales = piece ? a.c.v_scale : a.c.k_scale;
        uint4 codes[NI];
        float sc[2];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int r = n * (32 / LPR) + lane / LPR;
          const long long o = __shfl_sync(kAll, tk[n * (32 / LPR) / 32].at, r & 31);
          codes[n] = make_uint4(0, 0, 0, 0);
          if (o >= 0) codes[n] = ldg_stream16(src + o + (lane % LPR) * 16);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) sc[u] = tk[u].at >= 0 ? __ldg(scales + tk[u].sat) : 0.f;
        i += ST;
        settle();
        look_up(tk);
        if (round > 0) role_wait(dead, empty, (uint32_t)((round - 1) & 1), a.status);
        uint8_t* const to = dst + ((lane % LPR) >> 2) * kChunk;
        const int j = 2 * (lane & 3);
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int r = n * (32 / LPR) + lane / LPR;
          *reinterpret_cast<uint4*>(to + tc::sw128_off(r, j)) = e4m3x8_to_f16(codes[n].x, codes[n].y);
          *reinterpret_cast<uint4*>(to + tc::sw128_off(r, j + 1)) = e4m3x8_to_f16(codes[n].z, codes[n].w);
        }
        sh.scale[note][piece][lane] = sc[0];
        sh.scale[note][piece][32 + lane] = sc[1];
        if (piece) sh.vexp[note] = __reduce_max_sync(kAll, max(scale_exp(sc[0]), scale_exp(sc[1])));
      } else {
        if (round > 0) role_wait(dead, empty, (uint32_t)((round - 1) & 1), a.status);
        // this lane's 16-byte chunk of the 128-byte rows of the piece's chunks
        const int j = lane & 7;
        const uint16_t* src = static_cast<const uint16_t*>(a.c.k) + 8 * j;
        uint8_t* to = dst;
        if (LATENT) {
          src += 128 * piece;
          to += 2 * piece * kChunk;
        } else if (piece) {
          src = static_cast<const uint16_t*>(a.c.v) + 8 * j;
        }
        constexpr int kOwn = LATENT ? 2 : S::kKChunks;
#pragma unroll 4
        for (int r4 = 0; r4 < kTile; r4 += 4) {
          const int r = r4 + (lane >> 3);
          const long long o = __shfl_sync(kAll, r4 < 32 ? tk[0].at : tk[1].at, r & 31);
          const bool ok = o >= 0;
          const uint16_t* x = src + (ok ? o : 0);
          const uint32_t at = tc::sw128_off(r, j);
#pragma unroll
          for (int c = 0; c < kOwn; ++c) tc::cp_async16_zfill(to + c * kChunk + at, x + 64 * c, ok);
          if (LATENT && piece == 0)
            tc::cp_async16_zfill(to + (S::kKChunks - 1) * kChunk + at, x + DV, ok);
        }
        cp_async_commit();
        i += ST;
        settle();
        look_up(tk);
        cp_async_wait<0>();
      }
      if (piece == 0 && lane < 2) sh.exists[note][lane] = there[lane];
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    cp_async_wait<0>();
  } else if (warp == kSoft) {
    // ---- scores: S = Q K^T (rows x tokens), up to two tiles ahead of the softmax
    const uint32_t q0 = desc_k(smem_u32(sm_q)), kv0 = desc_k(smem_u32(sm_kv));
    constexpr uint32_t idesc = idesc_bf16<E4M3>(kRows, kTile, false, false);
    constexpr int kKeys = LATENT ? NP : 1;  // pieces with keys
    Part p;
    int j = 0, parts = 0;
    while (walk.next_tiles(a, p)) {
      role_wait(dead, &sh.q_full, (uint32_t)(parts & 1), a.status);
      ++parts;
      for (int i = 0; i < p.n; ++i, ++j) {
        if (j >= 2) role_wait(dead, &sh.s_empty[j & 1], (uint32_t)((j / 2 - 1) & 1), a.status);
        const uint32_t st = uniform(j % ST), buf = uniform(j & 1);
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
          role_wait(dead, &sh.full[st][x], (uint32_t)((j / ST) & 1), a.status);
          tc::fence_after_sync();
          if (tc::elect_one() && !*dead) {
            const uint32_t k = kv0 + st * (S::kStage / 16), d = tmem + buf * kTile;
            auto chunk = [&](int c, uint32_t add) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(d, q0 + c * (S::kQChunk / 16) + 2 * kk, k + c * (kChunk / 16) + 2 * kk, idesc, kk ? 1u : add);
            };
            if (LATENT) {
              chunk(2 * x, x);
              chunk(2 * x + 1, 1);
              if (x == 0) chunk(S::kKChunks - 1, 1);
            } else {
#pragma unroll
              for (int c = 0; c < S::kKChunks; ++c) chunk(c, c);
              tc::commit(&sh.empty[st][0]);
            }
            if (x == kKeys - 1) tc::commit(&sh.s_full[buf]);
          }
          __syncwarp();
        }
      }
    }
    // every product has been made before the CTA's memory goes
    if (j > 0 && lane == 0) mbar_wait(&sh.s_full[(j - 1) & 1], (uint32_t)(((j - 1) / 2) & 1));
    __syncwarp();
  } else if (warp == kSoft + 1) {
    // ---- outputs: O^T += V^T P^T (dimensions x rows).  A warp of their own: a
    // warp's MMAs wait for its own checks, not for the other's.
    const uint32_t p0 = desc_k(smem_u32(sm_p)), v0 = desc_mn(smem_u32(sm_kv) + S::kV, kChunk);
    const uint32_t idesc = idesc_bf16<E4M3>(DV >= 128 ? 128 : 64, npad, true, false);
    Part p;
    int j = 0;
    while (walk.next_tiles(a, p))
      for (int i = 0; i < p.n; ++i, ++j) {
        const uint32_t st = uniform(j % VST);
        if (!LATENT) role_wait(dead, &sh.full[st][NP - 1], (uint32_t)((j / VST) & 1), a.status);
        role_wait(dead, &sh.p_full, (uint32_t)(j & 1), a.status);
        tc::fence_after_sync();
        if (tc::elect_one() && !*dead) {
          const uint32_t v = v0 + st * (S::kVStage / 16);
#pragma unroll
          for (int mb = 0; mb < S::kBlocks; ++mb) {
#pragma unroll
            for (int y = 0; y < S::kParts; ++y)
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                mma_ss(tmem + kOCol + mb * kRows, v + (2 * mb * kChunk + kk * 2048) / 16,
                       p0 + (y * S::kQChunk + kk * 32) / 16, idesc, 1u);
            if (LATENT) tc::commit(&sh.empty[st][mb]);
          }
          if (!LATENT) tc::commit(&sh.empty[st][NP - 1]);
          tc::commit(&sh.pv_done);
        }
        __syncwarp();
      }
    if (j > 0 && lane == 0) mbar_wait(&sh.pv_done, (uint32_t)((j - 1) & 1));
    __syncwarp();
  } else {
    // ---- softmax.  Of 128 rows, a thread (times kSplit) has one, of 64 a quad of
    // lanes has rows ra and ra + 8: a thread holds kE tokens of kX rows.
    constexpr int kMine = kTile / S::kSplit;  // tokens of a warp
    constexpr int kX = ROWS == 64 ? 2 : 1, kE = ROWS == 64 ? kMine / 4 : kMine;
    const int c = lane & 3, quad = warp & 3, half = warp >> 2;
    const int ra = ROWS == 64 ? 16 * quad + (lane >> 2) : 32 * quad + lane;
    const int c0 = half * kMine;  // the warp's first token
    const bool writes = ROWS == 128 || c == 0;  // what a row has once
    // the token of element e, from the warp's first on
    auto token = [&](int e) { return ROWS == 64 ? 8 * (e / 2) + 2 * c + (e & 1) : e; };
    const uint32_t quadrant = tmem + ((uint32_t)(32 * quad) << 16);
    const float scale2 = a.d.scale * kLog2e;
    Walk ahead = walk;
    Part p;
    auto load_q = [&](const Part& x, int buf) {
      // a warp: kRows / kSoft rows, four at a time, eight lanes to a row
      constexpr int kOwn = kRows / kSoft;
      const int R = row0 + warp * kOwn + (lane & (kOwn - 1)), n = R / a.G;
      const long long mine = warp * kOwn + (lane & (kOwn - 1)) < rows
                                 ? x.b * a.d.q_stride + n * a.d.q_row_stride + (long long)(x.hkv * a.G + R - n * a.G) * DK
                                 : -1;
      const int j = lane & 7;
#pragma unroll 1
      for (int r4 = 0; r4 < kOwn; r4 += 4) {
        const int r = r4 + (lane >> 3);
        const long long o = __shfl_sync(kAll, mine, r);
        const bool ok = o >= 0;
        const uint16_t* src = a.q + (ok ? o : 0) + 8 * j;
        uint8_t* to = sm_q + tc::sw128_off(warp * kOwn + r, j);
        if (!E4M3) {
#pragma unroll
          for (int k = 0; k < S::kKChunks; ++k) tc::cp_async16_zfill(to + k * S::kQChunk, src + 64 * k, ok);
        } else {
          // as fp16, the row times a power of two that puts its largest magnitude
          // into [2^14, 2^15): exact but for what is below 2^-28 of it
          uint4 v[S::kKChunks];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < S::kKChunks; ++k) {
            v[k] = ok ? ldg16(src + 64 * k) : make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) top = max(top, max(u[y] & 0x7FFFu, (u[y] >> 16) & 0x7FFFu));
          }
#pragma unroll
          for (int y = 1; y < 8; y <<= 1) top = max(top, __shfl_xor_sync(kAll, top, y));
          const int E = min(exp_of_bits(top << 16), 126);
          const float f = pow2f(kGroupTop - E);
#pragma unroll
          for (int k = 0; k < S::kKChunks; ++k) {
            uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) u[y] = pack_f16x2(bf16_lo(u[y]) * f, bf16_hi(u[y]) * f);
            *reinterpret_cast<uint4*>(to + k * S::kQChunk) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (j == 0) sh.q_scale[buf][E4M3 ? warp * kOwn + r : 0] = scale2 * pow2f(E - kGroupTop);
        }
      }
      cp_async_commit();
    };
    bool more = ahead.next_tiles(a, p);
    if (more) load_q(p, 0);
    int j = 0, buf = 0;
    while (walk.next(a, p)) {
      if (rt == 0 && tid == 0 && p.first) a.info[p.b * a.c.Hkv + p.hkv] = make_int2(2 * col + (p.slot & 1), p.parts);
      const size_t slot = (size_t)max(p.slot, 0) * a.gtiles + rt;
      float* const part_ml = a.part_ml + slot * 2 * kRows;
      if (p.n == 0) {  // (a part of fewer units than a tile)
        if (tid < kRows) {
          part_ml[tid] = -INFINITY;
          part_ml[kRows + tid] = 0.f;
        }
        continue;
      }
      cp_async_wait<0>();
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      // what the thread's two rows see: the context from `low` on, and the new
      // tokens of `tree`
      uint64_t tree[kX];
      int low[kX];
      const int drafts = p.sp.len - p.sp.ctx;
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        const int R = row0 + ra + 8 * x, n = R / a.G;
        tree[x] = 0;
        low[x] = kNoRow;
        if (ra + 8 * x < rows && n < drafts) {
          const uint64_t m = a.mask ? (uint64_t)a.mask[p.b * a.d.mask_stride + n] : low_bits(n + 1);
          tree[x] = m & low_bits(drafts);
          low[x] = a.d.window > 0 ? p.sp.ctx + max(1, __popcll(tree[x])) - a.d.window : 0;
        }
      }
      float m[kX], l[kX], qf[kX];  // the maximum, the sum, the factor on the scores
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
        qf[x] = scale2;
      }
      // E4M3: the exponents that the rows' weights are held at, and what every
      // row's is at least (the same in every thread)
      int vexp[kX], vlow = kExpMin;
#pragma unroll
      for (int x = 0; x < kX; ++x) vexp[x] = kExpMin;
      for (int i = 0; i < p.n; ++i, ++j) {
        const int st = j % VST, t0 = (p.tile + i) * kTile;
        role_wait(dead, &sh.s_full[j & 1], (uint32_t)((j / 2) & 1), a.status);
        tc::fence_after_sync();
        float s[kX][kE];
        {
          uint32_t raw[kX * kE];
          const uint32_t at = quadrant + (j & 1) * kTile + c0;
          if constexpr (ROWS == 64 && kMine == 64)
            ld_16x256b_x8(at, raw);
          else if constexpr (ROWS == 64)
            ld_16x256b_x4(at, raw);
          else
            tc::ld_32x32b_x32(at, raw);
          tc::wait_ld();
#pragma unroll
          for (int x = 0; x < kX; ++x)
#pragma unroll
            for (int e = 0; e < kE; ++e)
              s[x][e] = __uint_as_float(raw[ROWS == 64 ? 4 * (e / 2) + 2 * x + (e & 1) : e]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty[j & 1]);
        if (i == p.n - 1) {  // the queries have been read for the last time
          Part x;
          more = ahead.next_tiles(a, x);
          if (more) load_q(x, buf ^ 1);
        }
        const int note = j % kNotes;
        const uint64_t exists = (uint64_t)sh.exists[note][1] << 32 | sh.exists[note][0];
        // a tile that some rows see more of than others
        const bool mixed = t0 + kTile > p.sp.ctx ||
                           (a.d.window > 0 && t0 < p.sp.ctx + drafts - a.d.window);
        if (E4M3 && i == 0) {  // (with the first scores the queries' factors are there)
#pragma unroll
          for (int x = 0; x < kX; ++x) qf[x] = sh.q_scale[buf][E4M3 ? ra + 8 * x : 0];
        }
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
          float2 f = make_float2(1.f, 1.f);
          if (E4M3) f = *reinterpret_cast<const float2*>(&sh.scale[note][0][c0 + token(e)]);
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            const float2 g = E4M3 ? mul2(f, make_float2(qf[x], qf[x])) : make_float2(qf[x], qf[x]);
            const float2 v = mul2(make_float2(s[x][e], s[x][e + 1]), g);
            s[x][e] = v.x;
            s[x][e + 1] = v.y;
          }
        }
        if (mixed || ~exists) {
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            uint64_t seen = low_bits(p.sp.ctx - t0) & ~low_bits(min(low[x], t0 + kTile) - t0);
            const int sft = p.sp.ctx - t0;
            if (sft > -64 && sft < 64) seen |= sft >= 0 ? tree[x] << sft : tree[x] >> -sft;
            seen &= exists;
            if (writes && half == 0) sh.seen[ra + 8 * x] = seen;
            const uint64_t mine = seen >> (ROWS == 64 ? c0 + 2 * c : c0);
#pragma unroll
            for (int e = 0; e < kE; ++e)
              if (!(mine >> (ROWS == 64 ? 8 * (e / 2) + (e & 1) : e) & 1)) s[x][e] = -INFINITY;
          }
        }
        float mx[kX];
        bool above = false;
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kE; e += 2) top[e / 2 & 1] = max3(top[e / 2 & 1], s[x][e], s[x][e + 1]);
          mx[x] = fmaxf(top[0], top[1]);
          if (ROWS == 64) {
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(kAll, mx[x], 1));
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(kAll, mx[x], 2));
          }
          if (S::kSplit > 1 && writes) sh.top[half][ra + 8 * x] = mx[x];
          above |= mx[x] > m[x] + (E4M3 ? kHalfSlack : kMaxSlack);  // (a row's first score moves its maximum from -inf)
        }
        bool moved = bar_any(1, kSoftThreads, above);
        int tile_top = kExpMin;
        if (E4M3) {
          role_wait(dead, &sh.full[st][NP - 1], (uint32_t)((j / VST) & 1), a.status);  // the values' scales
          tile_top = sh.vexp[note];
          moved |= tile_top > vlow;  // (the same in every thread)
        }
        if (j > 0) role_wait(dead, &sh.pv_done, (uint32_t)((j - 1) & 1), a.status);
        tc::fence_after_sync();
        if (i == 0) {  // the products are added to zeros
          const uint32_t zero[16] = {};
#pragma unroll 1
          for (int mb = 0; mb < S::kBlocks; ++mb)
#pragma unroll 1
            for (int r0 = 16 * half; r0 < npad; r0 += 16 * S::kSplit)
              st_32x32b_x16(quadrant + kOCol + mb * kRows + r0, zero);
          tc::wait_st();
        }
        if (moved) {
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            if (S::kSplit > 1) mx[x] = fmaxf(mx[x], sh.top[half ^ 1][ra + 8 * x]);
            const float mn = fmaxf(m[x], mx[x]);
            const float f = m[x] == mn ? 1.f : exp2_fast(m[x] - mn);
            l[x] *= f;
            m[x] = mn;
            float vmove = 1.f;
            if (E4M3 && tile_top > vlow) {
              int top = tile_top;
              if (mixed) {
                // The scales of what the row sees: what it does not see takes no bits
                // from its weights.  (A row's four lanes look at 16 tokens each.)
                const uint64_t seen = sh.seen[ra + 8 * x];
                float v = 0.f;
#pragma unroll 1
                for (int t = ROWS == 64 ? 16 * c : 0; t < (ROWS == 64 ? 16 * c + 16 : kTile); t += 16)
                  v = fmaxf(v, seen_top(&sh.scale[note][1][E4M3 ? t : 0], (uint32_t)(seen >> t)));
                if (ROWS == 64) {
                  v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
                  v = fmaxf(v, __shfl_xor_sync(kAll, v, 2));
                }
                top = scale_exp(v);
              }
              if (top > vexp[x]) {
                vmove = ldexp2f(1.f, vexp[x] - top);
                vexp[x] = top;
              }
            }
            if (writes && half == 0) sh.factor[ra + 8 * x] = f * vmove;
          }
          if (!mixed) vlow = max(vlow, tile_top);
          named_bar(1, kSoftThreads);  // (before the halves' tops are written again, too)
          if (i > 0) {
#pragma unroll 1
            for (int mb = 0; mb < S::kBlocks; ++mb)
#pragma unroll 1
              for (int r0 = 16 * half; r0 < npad; r0 += 16 * S::kSplit) {
                uint32_t o[16];
                const uint32_t at = quadrant + kOCol + mb * kRows + r0;
                ld_32x32b_x16(at, o);
                tc::wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u)
                  o[u] = __float_as_uint(__uint_as_float(o[u]) * sh.factor[r0 + u]);
                st_32x32b_x16(at, o);
              }
            tc::wait_st();
          }
        }
        // weights, as the second product's operand: row, then token
        float vdown[kX];
#pragma unroll
        for (int x = 0; x < kX; ++x) vdown[x] = pow2f(-vexp[x]);
        uint32_t w[S::kParts][ROWS == 64 ? 1 : 4];
        float2 sum[kX];
#pragma unroll
        for (int x = 0; x < kX; ++x) sum[x] = make_float2(0.f, 0.f);
        {
#pragma unroll
          for (int e = 0; e < kE; e += 2) {
            float2 vs = make_float2(1.f, 1.f);
            if (E4M3)
              vs = *reinterpret_cast<const float2*>(&sh.scale[note][1][c0 + token(e)]);
#pragma unroll
            for (int x = 0; x < kX; ++x) {
              const float ms = (m[x] == -INFINITY ? 0.f : m[x]) - (E4M3 ? kWTop : 0.f);
              const float2 d = add2(make_float2(s[x][e], s[x][e + 1]), make_float2(-ms, -ms));
              float2 v = make_float2(exp2_fast(d.x), exp2_fast(d.y));
              const int k = ROWS == 64 ? 0 : e / 2 % 4;
              if (E4M3) {
                sum[x] = add2(sum[x], v);
                float2 t = mul2(v, mul2(vs, make_float2(vdown[x], vdown[x])));
                t.x = v.x == 0.f ? 0.f : t.x;  // (a token that is not seen may have any scale)
                t.y = v.y == 0.f ? 0.f : t.y;
                w[0][k] = pack_f16x2(t.x, t.y);
              } else if (S::kParts == 1) {
                w[0][k] = pack_bf16x2(v.x, v.y);
                sum[x] = add2(sum[x], make_float2(bf16_lo(w[0][k]), bf16_hi(w[0][k])));
              } else {
                sum[x] = add2(sum[x], v);
                w[0][k] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
                const float2 r = add2(v, make_float2(-bf16_lo(w[0][k]), -bf16_hi(w[0][k])));
                w[S::kParts - 1][k] = pack_bf16x2(r.x, r.y);
              }
#pragma unroll
              for (int y = 0; y < S::kParts; ++y) {
                if (ROWS == 64)
                  *reinterpret_cast<uint32_t*>(sm_p + y * S::kQChunk + tc::sw128_off(ra + 8 * x, c0 / 8 + e / 2) +
                                               4 * c) = w[y][0];
                else if (k == 3)
                  *reinterpret_cast<uint4*>(sm_p + y * S::kQChunk + tc::sw128_off(ra, (c0 + e) / 8)) =
                      make_uint4(w[y][0], w[y][ROWS == 64 ? 0 : 1], w[y][ROWS == 64 ? 0 : 2], w[y][k]);
              }
            }
          }
        }
#pragma unroll
        for (int x = 0; x < kX; ++x) l[x] += sum[x].x + sum[x].y;
        if (mixed) {
          // A value that is not finite reaches the rows that see its token and no
          // other: it is added to their outputs, and the tile holds 0 in its place
          // (times a weight of 0 it would be NaN).
          if (!LATENT) role_wait(dead, &sh.full[st][NP - 1], (uint32_t)((j / VST) & 1), a.status);
          uint8_t* const v = sm_kv + S::kV + st * S::kVStage;
          bool odd = false;
          for (int e = tid; e < kTile * (DV / 8); e += kSoftThreads) {
            const uint4 w = *reinterpret_cast<const uint4*>(v + e * 16);
            odd |= nonfinite_16x2<E4M3>(w.x) || nonfinite_16x2<E4M3>(w.y) || nonfinite_16x2<E4M3>(w.z) ||
                   nonfinite_16x2<E4M3>(w.w);
          }
          if (bar_any(1, kSoftThreads, odd)) {
#pragma unroll 1
            for (int mb = 0; mb < S::kBlocks; ++mb) {
              const int d = DV >= 128 ? mb * 128 + 32 * quad + lane : 16 * quad + (lane & 15);
#pragma unroll 1
              for (int r0 = 16 * half; r0 < npad; r0 += 16 * S::kSplit) {
                uint32_t o[16];
                const uint32_t at = quadrant + kOCol + mb * kRows + r0;
                ld_32x32b_x16(at, o);
                tc::wait_ld();
#pragma unroll 1
                for (int t = 0; t < kTile; ++t) {
                  const uint32_t w = *reinterpret_cast<const uint16_t*>(
                      v + (d >> 6) * kChunk + tc::sw128_off(t, (d >> 3) & 7) + 2 * (d & 7));
                  const bool bad = nonfinite_16x2<E4M3>(w);
                  const float add = E4M3 ? NAN : __uint_as_float(w << 16);  // (E4M3 has no infinity)
#pragma unroll
                  for (int u = 0; u < 16; ++u) {
                    if (bad && (sh.seen[r0 + u] >> t & 1))
                      o[u] = __float_as_uint(__uint_as_float(o[u]) + add);
                  }
                }
                st_32x32b_x16(at, o);
              }
            }
            tc::wait_st();
            named_bar(1, kSoftThreads);  // every thread has read the values
            for (int e = tid; e < kTile * DV; e += kSoftThreads) {
              uint16_t* w = reinterpret_cast<uint16_t*>(v) + e;
              if (nonfinite_16x2<E4M3>(*w)) *w = 0;
            }
          }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full);
      }
      // ---- the part's results
      if (tid < kRows) {
        const int R = row0 + tid, n = R / a.G;
        sh.at[tid] = tid < rows ? p.b * a.d.out_stride + n * a.d.out_row_stride +
                                      (long long)(p.hkv * a.G + R - n * a.G) * DV
                                : -1;
      }
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        if (ROWS == 64) {
          l[x] += __shfl_xor_sync(kAll, l[x], 1);
          l[x] += __shfl_xor_sync(kAll, l[x], 2);
        }
        if (S::kSplit > 1 && writes && half == 1) sh.top[1][ra + 8 * x] = l[x];  // (factors may be in use still)
      }
      if (S::kSplit > 1) named_bar(1, kSoftThreads);
#pragma unroll
      for (int x = 0; x < kX; ++x)
        if (writes && half == 0) {
          const int r = ra + 8 * x;
          if (S::kSplit > 1) l[x] += sh.top[1][r];
          // (a row that is none has taken in the tiles that all rows see alike)
          const bool real = low[x] != kNoRow;
          sh.inv[r] = l[x] == 0.f || !real ? 0.f : E4M3 ? ldexp2f(1.f / l[x], vexp[x]) : 1.f / l[x];
          if (p.slot >= 0) {
            part_ml[r] = real ? m[x] : -INFINITY;
            part_ml[kRows + r] = real ? l[x] : 0.f;
          }
        }
      role_wait(dead, &sh.pv_done, (uint32_t)((j - 1) & 1), a.status);
      tc::fence_after_sync();
      named_bar(1, kSoftThreads);
      float* const part_o = a.part_o + slot * kRows * DV;
      const bool lives = DV >= 128 || lane < 16;
#pragma unroll 1
      for (int mb = 0; mb < S::kBlocks; ++mb) {
        const int d = DV >= 128 ? mb * 128 + 32 * quad + lane : 16 * quad + (lane & 15);
#pragma unroll 1
        for (int r0 = 16 * half; r0 < npad; r0 += 16 * S::kSplit) {
          uint32_t o[16];
          ld_32x32b_x16(quadrant + kOCol + mb * kRows + r0, o);
          tc::wait_ld();
          if (p.slot >= 0) {
            // (next to E4M3 divided by the part's sum: with large scales the undivided
            // outputs leave fp32 where the answers do not)
#pragma unroll
            for (int u = 0; u < 16; ++u)
              if (lives && r0 + u < rows)
                part_o[(r0 + u) * DV + d] = __uint_as_float(o[u]) * (E4M3 ? sh.inv[r0 + u] : 1.f);
          } else {
            // two neighbouring lanes trade, and each writes two dimensions of a row
            const int odd = lane & 1;
#pragma unroll
            for (int u = 0; u < 16; u += 2) {
              const float f0 = sh.inv[r0 + u], f1 = sh.inv[r0 + u + 1];
              const float v0 = f0 == 0.f ? 0.f : __uint_as_float(o[u]) * f0;
              const float v1 = f1 == 0.f ? 0.f : __uint_as_float(o[u + 1]) * f1;
              const float got = __shfl_xor_sync(kAll, odd ? v0 : v1, 1);
              const long long at = sh.at[r0 + u + odd];
              if (lives && at >= 0)
                *reinterpret_cast<uint32_t*>(a.out + at + (d - odd)) =
                    odd ? pack_bf16x2(got, v1) : pack_bf16x2(v0, got);
            }
          }
        }
      }
      tc::fence_before_sync();
      buf ^= 1;
      named_bar(1, kSoftThreads);  // the next part may write factors and places
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kSoft) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, S::kTmem);
  }
}

// Joins the parts of the segments that several columns hold, in order, and
// answers zeros for sequences without new tokens: out = sum_i 2^(m_i - M) o_i /
// sum_i 2^(m_i - M) l_i.  DIVIDED: the o_i are divided by their l_i already; what is
// joined so far is kept divided, so that nothing in between is larger than they are.
// Bound by latency (its parts come from L2, 76 of them for 2 x 131072 tokens): DV /
// 4 threads have a row's four dimensions each, and enough groups of them share a
// row's parts for four rounds of loads, in which `kAhead` parts of a thread are on
// their way at once.  4 to 5 us of a call.
template <int DV, int THREADS, int kAhead, bool DIVIDED>
__global__ void __launch_bounds__(THREADS) k_draft_join(const DraftArgs a) {
  constexpr int kLanes = DV / 4, kGroups = THREADS / kLanes;  // threads per row; rows, or shares of the parts
  __shared__ float4 s_acc[kGroups][kLanes];
  __shared__ float s_m[kGroups], s_l[kGroups];
  griddep_wait();
  griddep_trigger();
  const int kRows = a.tile_rows;
  const int rt = blockIdx.x % a.gtiles, seg = blockIdx.x / a.gtiles, b = seg / a.c.Hkv, hkv = seg % a.c.Hkv;
  const int row0 = rt * kRows, rows = min(kRows, a.rows - row0);
  const int d4 = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  int2 info = a.info[seg];  // (of no meaning for a sequence without new tokens)
  bool bad;
  const Span sp = span_of(a, b, &bad);
  if (bad && threadIdx.x == 0 && blockIdx.y == 0 && hkv == 0 && rt == 0) raise_status(a.status, MOE_DEV_BAD_PAGE);
  if (!sp.tiles) info = make_int2(0, 0);
  if (info.y == 1) return;  // its column has written it
  // enough threads for a row to fetch its parts in four rounds
  int shares = 1;
  while (shares < kGroups && shares * 4 * kAhead < info.y) shares *= 2;
  const int at_once = kGroups / shares, mine = grp % shares;
  for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
    const int r = r0 + grp / shares, R = row0 + r, n = R / a.G;
    uint16_t* out = a.out + b * a.d.out_stride + n * a.d.out_row_stride +
                    (long long)(hkv * a.G + R - n * a.G) * DV + 4 * d4;
    if (info.y == 0) {
      if (r < rows) *reinterpret_cast<uint2*>(out) = make_uint2(0u, 0u);
      continue;
    }
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int each = cdiv(info.y, shares), i1 = r < rows ? min(info.y, (mine + 1) * each) : 0;
    for (int i0 = mine * each; i0 < i1; i0 += kAhead) {
      float m[kAhead], l[kAhead];
      float4 v[kAhead];
      float M2 = M;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u;
        m[u] = -INFINITY;
        l[u] = 0.f;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < i1) {
          const size_t slot = (size_t)(i == 0 ? info.x : 2 * (info.x / 2 + i)) * a.gtiles + rt;
          m[u] = __ldcg(a.part_ml + slot * 2 * kRows + r);
          l[u] = __ldcg(a.part_ml + slot * 2 * kRows + kRows + r);
          v[u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot * kRows + r) * DV) + d4);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) M2 = fmaxf(M2, m[u]);
      const float Ms = M2 == -INFINITY ? 0.f : M2, f0 = M == M2 ? 1.f : exp2f(M - Ms);
      const float kept = L * f0;
      L = kept;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        // A part with nothing of this row: its outputs may hold anything.  (Not told by
        // the maximum: a row of nothing but NaN scores leaves it at -inf, its sum is NaN.)
        if (l[u] == 0.f) continue;
        m[u] = exp2f(m[u] - Ms);
        L = fmaf(l[u], m[u], L);
      }
      const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);  // (a sum is below 2^46)
      const float fa = DIVIDED ? kept * inv : f0;
      acc = make_float4(acc.x * fa, acc.y * fa, acc.z * fa, acc.w * fa);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (l[u] == 0.f) continue;
        const float f = DIVIDED ? l[u] * m[u] * inv : m[u];
        acc.x = fmaf(v[u].x, f, acc.x);
        acc.y = fmaf(v[u].y, f, acc.y);
        acc.z = fmaf(v[u].z, f, acc.z);
        acc.w = fmaf(v[u].w, f, acc.w);
      }
      M = M2;
    }
    if (shares > 1) {
      s_acc[grp][d4] = acc;
      if (d4 == 0) {
        s_m[grp] = M;
        s_l[grp] = L;
      }
      __syncthreads();
      if (mine == 0) {
        for (int x = 1; x < shares; ++x) M = fmaxf(M, s_m[grp + x]);
        const float Ms = M == -INFINITY ? 0.f : M;
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (DIVIDED)
          for (int x = 0; x < shares; ++x)
            if (s_l[grp + x] != 0.f) L = fmaf(s_l[grp + x], exp2f(s_m[grp + x] - Ms), L);
        const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
        for (int x = 0; x < shares; ++x) {
          if (s_l[grp + x] == 0.f) continue;
          float f = exp2f(s_m[grp + x] - Ms);
          const float4 v = s_acc[grp + x][d4];
          if (DIVIDED)
            f *= s_l[grp + x] * inv;
          else
            L = fmaf(s_l[grp + x], f, L);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
      }
      __syncthreads();
    }
    if (mine == 0 && r < rows) {
      const float inv = L == 0.f ? 0.f : DIVIDED ? 1.f : 1.f / L;
      *reinterpret_cast<uint2*>(out) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
  }
}

namespace {

// Partial results of a call: two per CTA of one wave, counted in 64 rows (a CTA
// of 128 rows has an SM for itself).
size_t draft_slots(const moe_draft_dims& d, int Hkv) {
  return 2 * (size_t)std::max(2 * num_sms(), 2 * cdiv(d.n * (d.Hq / Hkv), 128));
}

template <int DK, int DV, bool LATENT, bool E4M3, bool TMA, int ROWS>
cudaError_t launch_draft(DraftArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  using S = DraftShape<DK, DV, LATENT, E4M3, TMA, ROWS>;
  cudaError_t err = ensure_smem((const void*)k_draft_attention<DK, DV, LATENT, E4M3, TMA, ROWS>, S::kSmem);
  if (err != cudaSuccess) return err;
  a.tile_rows = ROWS;
  a.gtiles = cdiv(a.rows, ROWS);
  const long long tiles = (std::min((long long)a.d.table_width * a.c.page_size, kMaxTokens) + kTile - 1) / kTile + 1;
  const long long units = (long long)a.d.B * a.c.Hkv * (tiles + kSegCost);
  a.cols = (int)std::max(1ll, std::min<long long>(S::kCtas * num_sms() / a.gtiles, units));
  err = launch_k(k_draft_attention<DK, DV, LATENT, E4M3, TMA, ROWS>, dim3(a.cols * a.gtiles), dim3(S::kWarps * 32),
                 S::kSmem, s, true, kmap, vmap, a);
  if (err != cudaSuccess) return err;
  // many parts per segment: as many of a row's as a CTA's registers hold at
  // once; few: more CTAs (2 x 131072 latent vectors, 76 parts: 73.5 us in all
  // against 79.9 with the other form; 32 trees of 16, E4M3: 104.5 against 113.8)
  const int segs = a.d.B * a.c.Hkv * a.gtiles;
  if (a.cols >= 8 * a.d.B * a.c.Hkv)
    return launch_k(k_draft_join<DV, 512, 8, E4M3>, dim3(segs, std::min(ROWS, cdiv(4 * num_sms(), segs))), dim3(512), 0,
                    s, true, a);
  return launch_k(k_draft_join<DV, 256, 4, E4M3>, dim3(segs, ROWS / (1024 / DV)), dim3(256), 0, s, true, a);
}

// A cache of pages that tile boxes divide is copied by maps of [pages, heads,
// tokens, dimensions]; any other is gathered.
template <int DK, int DV, bool LATENT, bool E4M3>
cudaError_t launch_draft(DraftArgs& a, cudaStream_t s) {
  CUtensorMap kmap{}, vmap{};
  const int ps = a.c.page_size;
  bool boxes = ps >= 8 && (ps % kTile == 0 || kTile % ps == 0);
  a.box = std::min(ps, kTile);
  while (boxes && 1 << a.box_shift < a.box) ++a.box_shift;
  if (boxes) {
    const long long strides[3] = {a.c.token_stride, a.c.head_stride, a.c.page_stride};
    const int extents[3] = {ps, a.c.Hkv, a.c.pages};
    boxes = make_cache_map(&kmap, a.c.k, E4M3, DK, extents, strides, a.box) == cudaSuccess &&
            (LATENT || make_cache_map(&vmap, a.c.v, E4M3, DV, extents, strides, a.box) == cudaSuccess);
  }
  // more than 64 rows go through the cache once, not twice
  if constexpr (!LATENT && DK <= 128)
    if (boxes && a.rows > 64) return launch_draft<DK, DV, LATENT, E4M3, true, 128>(a, kmap, vmap, s);
  return boxes ? launch_draft<DK, DV, LATENT, E4M3, true, 64>(a, kmap, vmap, s)
               : launch_draft<DK, DV, LATENT, E4M3, false, 64>(a, kmap, vmap, s);
}

}  // namespace

bool draft_attention_fits(const moe_draft_dims& d, const moe_kv_cache& c) {
  const long long tokens = std::min((long long)d.table_width * c.page_size, kMaxTokens);
  return (long long)d.B * c.Hkv * (tokens / kTile + 2 + kSegCost) + (1ll << 24) < (1ll << 31);
}

size_t draft_attention_workspace(const moe_draft_dims& d, int Hkv, int DV) {
  return draft_slots(d, Hkv) * 64 * ((size_t)DV + 2) * sizeof(float) + (size_t)d.B * Hkv * sizeof(int2);
}

cudaError_t launch_draft_attention(const uint16_t* q, const moe_kv_cache& cache, bool latent,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const int64_t* mask, const int32_t* draft_lens,
                                   const moe_draft_dims& d, int DV, uint16_t* out, void* ws,
                                   int32_t* status, cudaStream_t s) {
  DraftArgs a{};
  a.q = q;
  a.c = cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.mask = mask;
  a.draft_lens = draft_lens;
  a.d = d;
  a.G = d.Hq / cache.Hkv;
  a.rows = d.n * a.G;
  a.out = out;
  a.part_o = static_cast<float*>(ws);
  const size_t slots = draft_slots(d, cache.Hkv);
  a.part_ml = a.part_o + slots * 64 * DV;
  a.info = reinterpret_cast<int2*>(a.part_ml + slots * 2 * 64);
  a.status = status;
  // t / page_size for 0 <= t < 2^31: with 2^(e-1) < page_size <= 2^e and mul =
  // ceil(2^(31+e) / page_size) < 2^32, floor(t mul / 2^(31+e)) is exact
  int e = 0;
  while ((1ll << e) < cache.page_size) ++e;
  a.ps_mul = (uint32_t)(((1ull << (31 + e)) + cache.page_size - 1) / cache.page_size);
  a.ps_shift = e > 0 ? e - 1 : 0;
  if (latent) {
    return DV == 512 ? launch_draft<576, 512, true, false>(a, s) : launch_draft<320, 256, true, false>(a, s);
  }
  const bool f8 = cache.format == MOE_KV_E4M3;
  if (DV == 64) return f8 ? launch_draft<64, 64, false, true>(a, s) : launch_draft<64, 64, false, false>(a, s);
  if (DV == 128) return f8 ? launch_draft<128, 128, false, true>(a, s) : launch_draft<128, 128, false, false>(a, s);
  return f8 ? launch_draft<256, 256, false, true>(a, s) : launch_draft<256, 256, false, false>(a, s);
}

}  // namespace moe
