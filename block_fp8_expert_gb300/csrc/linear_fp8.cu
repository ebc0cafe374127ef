// Block-FP8 linear layer on E4M3 activations (moe_linear_fp8):
//   out[m, n] = sum_b Sx[m, b] Sw[n / 128, b] P_b[m, n] + bias[n],
//   P_b[m, n] = sum over the 128 columns of block b of code_x code_w.
#include <algorithm>

#include "decoder_internal.h"
#include "per_device.h"
#include "tcgen05.cuh"

namespace moe {

namespace {
struct LinArgs {
  const uint16_t* x;
  long long x_stride;
  const uint8_t* codes;
  const float* scales;
  const float* bias;
  uint16_t* out;
  long long out_stride;
  int M, N, K;
  int32_t* status;
};
}  // namespace

// Few rows: the weights are streamed once and the activations quantised on
// the way, in one launch.  A CTA owns 16 output features and 8 NT rows; its
// warps take the 128-wide blocks in turn.  Thread (g, c) of a warp holds 2 x
// 16 consecutive codes of weight rows g and g + 8 and the same columns of
// activation rows 8 nt + g, so the four threads of a quad hold a row's whole
// group: its maximum is two shuffles.  Codes become fp16 (exactly) and feed
// mma.sync with fp32 accumulation; the block's two scales are applied to its
// sums, and the warps' sums are added in a fixed order.
// One row, N 5120, K 2048: 4.5 us in a graph (10.5 MB of codes take 1.6 at the
// copy rate): launch, one round of loads per warp, the exchange.  8 rows 4.8,
// 16 rows 7.3 us: every CTA quantises all of x for itself, which is what
// hands over to the tensor-core kernel beyond.  All four blocks' loads of a
// warp at once take as long; a ring of cp.async copies twice as long, since
// every CTA then brings its x in from L2 instead of the SM's first level.
template <int NT, int kLinWarps>
__global__ void __launch_bounds__(kLinWarps * 32)
k_linear_stream(const LinArgs a) {
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ float red[kLinWarps][NT][4][32];
  griddep_wait();
  griddep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * (8 * NT);
  const int nkb = cdiv(a.K, kScaleBlock);
  const bool lo_ok = n0 + g < a.N, hi_ok = n0 + g + 8 < a.N;
  const uint8_t* w_lo = a.codes + (size_t)(lo_ok ? n0 + g : 0) * a.K;
  const uint8_t* w_hi = a.codes + (size_t)(hi_ok ? n0 + g + 8 : 0) * a.K;
  const float* sw = a.scales + (size_t)(n0 / kScaleBlock) * nkb;  // 16 divides 128
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[nt][u] = 0.f;
  bool bad = false;
#pragma unroll 2
  for (int kb = warp; kb < nkb; kb += kLinWarps) {
    uint4 wl[2], wh[2], xv[NT][2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = kb * kScaleBlock + 64 * h + 16 * c;
      const bool in = col < a.K;
      wl[h] = in && lo_ok ? ldg_stream16(w_lo + col) : zero;
      wh[h] = in && hi_ok ? ldg_stream16(w_hi + col) : zero;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int m = m0 + 8 * nt + g;
        const uint16_t* p = a.x + (size_t)m * a.x_stride + col;
        const bool real = in && m < a.M;
        xv[nt][h][0] = real ? ldg16(p) : zero;
        xv[nt][h][1] = real ? ldg16(p + 8) : zero;
      }
    }
    const float s_w = __ldg(sw + kb);
    uint32_t al[2][8], ah[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      decode16_f16(wl[h], al[h]);
      decode16_f16(wh[h], ah[h]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t w4[4] = {xv[nt][h][v].x, xv[nt][h][v].y, xv[nt][h][v].z, xv[nt][h][v].w};
#pragma unroll
          for (int u = 0; u < 4; ++u) m = max(m, max(w4[u] & 0x7FFFu, (w4[u] >> 16) & 0x7FFFu));
        }
      m = max(m, __shfl_xor_sync(kAll, m, 1));
      m = max(m, __shfl_xor_sync(kAll, m, 2));
      if (m >= 0x7F80u) bad = true;
      float f, s_x;
      quant_factors(m << 16, f, s_x);
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t xr[8];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t w4[4] = {xv[nt][h][v].x, xv[nt][h][v].y, xv[nt][h][v].z, xv[nt][h][v].w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            xr[4 * v + u] = e4m3x2_to_f16x2(f32x2_to_e4m3x2(bf16_lo(w4[u]) * f, bf16_hi(w4[u]) * f));
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t A[4] = {al[h][2 * s], ah[h][2 * s], al[h][2 * s + 1], ah[h][2 * s + 1]};
          const uint32_t B[2] = {xr[2 * s], xr[2 * s + 1]};
          mma_f16_16x8x16(part, A, B);
        }
      }
      // this thread's sums are of rows 2c and 2c + 1 of the group of 8
      const float s0 = s_w * __shfl_sync(kAll, s_x, 8 * c);
      const float s1 = s_w * __shfl_sync(kAll, s_x, 8 * c + 4);
      acc[nt][0] = fmaf(part[0], s0, acc[nt][0]);
      acc[nt][1] = fmaf(part[1], s1, acc[nt][1]);
      acc[nt][2] = fmaf(part[2], s0, acc[nt][2]);
      acc[nt][3] = fmaf(part[3], s1, acc[nt][3]);
    }
  }
  if (bad) raise_status(a.status, MOE_DEV_NONFINITE);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int u = 0; u < 4; ++u) red[warp][nt][u][lane] = acc[nt][u];
  __syncthreads();
  // two features (n, n + 1) of one row per thread
  for (int e = tid; e < NT * 64; e += kLinWarps * 32) {
    const int np = e & 7, r = (e >> 3) & 7, nt = e >> 6;
    const int n = n0 + 2 * np, m = m0 + 8 * nt + r;
    if (n >= a.N || m >= a.M) continue;
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 2 * np + i;  // feature inside the CTA's 16
      const int u = (r & 1) + 2 * (row >> 3), L = 4 * (row & 7) + (r >> 1);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kLinWarps; ++w) s += red[w][nt][u][L];
      v[i] = a.bias ? s + __ldg(a.bias + n + i) : s;
    }
    *reinterpret_cast<uint32_t*>(a.out + (size_t)m * a.out_stride + n) = pack_bf16x2(v[0], v[1]);
  }
}

// ---------------------------------------------------------------------------
// Many rows: tcgen05
// ---------------------------------------------------------------------------
// Activations to E4M3: 16 lanes per group of 128 columns, 8 columns per lane.
// codes [M][K]; scales transposed, sxt [ceil(K / 128)][ld], so that the GEMM's
// lanes, which hold a row each, read them side by side.
__global__ void __launch_bounds__(256)
k_linear_quant(const uint16_t* __restrict__ x, long long x_stride, int M, int K,
               uint8_t* __restrict__ codes, float* __restrict__ sxt, int ld,
               int32_t* __restrict__ status) {
  griddep_wait();
  griddep_trigger();  // (after the wait: the GEMM reads weights before its own)
  const int nkb = cdiv(K, kScaleBlock);
  const long long unit = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int part = threadIdx.x & 15;
  const bool in = unit < (long long)M * nkb;
  const int m = in ? (int)(unit / nkb) : 0, kb = in ? (int)(unit % nkb) : 0;
  const int col = kb * kScaleBlock + 8 * part;
  const bool real = in && col < K;
  const uint4 v = real ? ldg_stream16(x + (size_t)m * x_stride + col) : make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t mx = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) mx = max(mx, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (mx >= 0x7F80u && part == 0) raise_status(status, MOE_DEV_NONFINITE);
  float f, scale;
  quant_factors(mx << 16, f, scale);
  uint32_t c[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    c[u] = f32x2_to_e4m3x2(bf16_lo(w[2 * u]) * f, bf16_hi(w[2 * u]) * f) |
           (f32x2_to_e4m3x2(bf16_lo(w[2 * u + 1]) * f, bf16_hi(w[2 * u + 1]) * f) << 16);
  if (real) *reinterpret_cast<uint2*>(codes + (size_t)m * K + col) = make_uint2(c[0], c[1]);
  if (in && part == 0) sxt[(size_t)kb * ld + m] = scale;
}

namespace {
constexpr int GM = 128, GN = 128;        // rows (TMEM lanes) x features (TMEM columns) per CTA
constexpr int GSTAGES = 3;
constexpr int G_TILE = 128 * 128;        // bytes of one operand's 128 rows x 128 K
constexpr int G_STAGE = 2 * G_TILE;
constexpr int G_PITCH = GN + 4;          // floats per row of the split's exchange
constexpr int G_EXCHANGE = GM * G_PITCH * 4;
constexpr int g_smem(int split) { return GSTAGES * G_STAGE + (split > 1 ? G_EXCHANGE : 0) + 1024; }
// The activation scales of a block's 128 rows ride with its stage, into a ring
// of their own that is two slots longer: a stage is refilled once its MMAs are
// done, when the sums of all but the last two blocks have been read (p_empty).
constexpr int GSX_SLOTS = GSTAGES + 2;
constexpr int kProWarps = 8;
constexpr int kGemmThreads = (2 + kProWarps) * 32;
static_assert(kProWarps * 4096 <= GSTAGES * G_STAGE, "the output is staged in the ring");

struct GemmArgs {
  const float* sxt;
  int ld;
  const float* sw;
  const float* bias;
  uint16_t* out;
  long long out_stride;
  int M, N, nkb;
  int32_t* status;
};

struct GemmShared {
  alignas(16) float sx[GSX_SLOTS][128];
  uint64_t full[GSTAGES], empty[GSTAGES], p_full[2], p_empty[2];
  uint32_t tmem_base;
  volatile int abort_flag;
};

// Warp-uniform bounded wait: the warp gives up together once the budget is
// spent or another role has given up.
__device__ __forceinline__ bool gwait(GemmShared& sh, uint64_t* bar, uint32_t parity,
                                      int32_t* status) {
  constexpr unsigned kAll = 0xffffffffu;
  bool done = mbar_try_wait(bar, parity);
  if (__all_sync(kAll, done)) return true;
  const WaitBudget b = wait_budget();
  for (uint32_t n = 1;; ++n) {
    if (__any_sync(kAll, done)) {
      for (int r = 0; !done && r < (1 << 16); ++r) done = mbar_try_wait(bar, parity);
      if (__all_sync(kAll, done)) return true;
      break;
    }
    if ((n & 31) == 0) {
      const bool give_up = sh.abort_flag != 0 || budget_spent(b);
      if (__any_sync(kAll, give_up)) break;
    }
    done = mbar_try_wait(bar, parity);
  }
  if ((threadIdx.x & 31) == 0 && !sh.abort_flag) {
    sh.abort_flag = 1;
    raise_status(status, MOE_DEV_WAIT_TIMEOUT);
  }
  __syncwarp();
  return false;
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// (a.x, a.y) += (p.x, p.y) * (f, f)
__device__ __forceinline__ void fma2(float2& a, uint32_t p0, uint32_t p1, float f) {
  asm("{\n .reg .b64 A, P, F;\n mov.b64 A, {%0, %1};\n mov.b64 P, {%2, %3};\n mov.b64 F, {%4, %4};\n"
      " fma.rn.f32x2 A, P, F, A;\n mov.b64 {%0, %1}, A;\n}\n"
      : "+f"(a.x), "+f"(a.y)
      : "r"(p0), "r"(p1), "f"(f));
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "f"(a), "f"(b), "f"(c),
               "f"(d)
               : "memory");
}
// A warp's 32 rows x 64 features (a row per lane) as bf16 into a 4 KB tile of
// shared memory, 128-byte swizzled as the TMA store reads it: a thread's own
// stores would touch 32 rows at a time, half a sector of each.
__device__ __forceinline__ void stage_rows(uint8_t* tile, float2 (&acc)[32], const float* bias,
                                           int n0, int N, int lane) {
  if (bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int n = min(n0 + 2 * j, N - 2);  // (features past the matrix are not stored)
      acc[j].x += __ldg(bias + n);
      acc[j].y += __ldg(bias + n + 1);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 v = make_uint4(pack_bf16x2(acc[4 * j].x, acc[4 * j].y),
                               pack_bf16x2(acc[4 * j + 1].x, acc[4 * j + 1].y),
                               pack_bf16x2(acc[4 * j + 2].x, acc[4 * j + 2].y),
                               pack_bf16x2(acc[4 * j + 3].x, acc[4 * j + 3].y));
    *reinterpret_cast<uint4*>(tile + tc::sw128_off(lane, j)) = v;
  }
}
// A tile row of weight scales, block kb of kb0 .. kb1 in lane (kb - kb0) % 32:
// one load per 32 blocks, handed round by shuffles.
struct BlockScales {
  const float* p;
  int n, lane;
  float v;
  __device__ __forceinline__ void start(const float* p_, int n_, int lane_) {
    p = p_;
    n = n_;
    lane = lane_;
    v = lane < n ? __ldg(p + lane) : 0.f;
  }
  __device__ __forceinline__ float at(int i) {
    if (i > 0 && (i & 31) == 0) v = i + lane < n ? __ldg(p + i + lane) : 0.f;
    return __shfl_sync(0xffffffffu, v, i & 31);
  }
};
__device__ __forceinline__ float bias_at(const GemmArgs& a, int n) {
  return a.bias ? __ldg(a.bias + n) : 0.f;
}
}  // namespace

// One 128 x 128 tile of the output per cluster, the K blocks divided over its
// CTAs.  Warp 0 fills a ring of stages by TMA (128 rows x 128 K of either
// operand, 128-byte swizzled; what lies outside the matrices reads as zero),
// one thread of warp 1 issues the four K = 32 MMAs of a block into one of two
// TMEM buffers, and warps 2-9 add the block's sums, times Sx of their row and
// Sw of the tile, to fp32 sums in registers (a thread: one row, 64 features).
// The weights' first stages are on their way before the quantisation ends: only
// warp 0 waits for the kernel before, and only for what it wrote.  The kernel
// before that has ended by then, as this one may only follow a kernel that
// triggers it after its own wait (k_linear_quant).
// A cluster's sums meet in shared memory: each CTA owns a share of the rows, the
// others store theirs for it straight from registers, and it adds them in the
// CTAs' order and writes the result.
//
// What bounds it, at M 4096, N 5120, K 2048 (53 us with the quantisation, 1.62
// PFLOP/s): an SM takes in about 64 bytes per cycle, so the 32 KB of a block
// take 500 cycles (the MMAs 256), 555 measured with two CTAs per SM, and 1280
// equal tiles make five rounds of 304 where 4.2 would do.  Measured instead,
// and left out: 128 x 256 tiles, one persistent CTA per SM (48 KB per block of
// twice the features; 940 cycles a block, the copies' latency with three
// stages: 51.7 us, and slower below 150 tiles), the same with W multicast to a
// cluster of two (52.8 us), and 256 x 256 tiles of CTA pairs (32 KB per block,
// but 880 cycles for the two buffers' way from MMA to registers and back
// across the pair: 52.5 us).
template <int SPLIT>
__global__ void __launch_bounds__(kGemmThreads, SPLIT > 1 ? 1 : 2)
k_linear_gemm(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
              const __grid_constant__ CUtensorMap omap, const GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ GemmShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = SPLIT > 1 ? blockIdx.x : 0;
  const int n0 = blockIdx.y * GN, m0 = blockIdx.z * GM;
  const int kb0 = rank * a.nkb / SPLIT, kb1 = (rank + 1) * a.nkb / SPLIT, nk = kb1 - kb0;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  if (tid == 0) {
    for (int s = 0; s < GSTAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.p_full[b], 1);
      mbar_init(&sh.p_empty[b], kProWarps);
    }
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&sh.tmem_base, 2 * GN);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (SPLIT > 1) cluster_arrive();  // (waited for before the exchange: every CTA has begun)
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  float2 acc[32];  // warps 2-9

  if (warp == 0) {
    const int ahead = min(nk, GSTAGES);
    const uint32_t sx_bytes = 4u * min(128, a.ld - m0);  // ld: the rows, up to a multiple of 32
    auto load_x = [&](int i) {
      const int s = i % GSTAGES;
      bulk_g2s(sh.sx[i % GSX_SLOTS], a.sxt + (size_t)(kb0 + i) * a.ld + m0, sx_bytes, &sh.full[s]);
      tc::tma_load_2d(smem + s * G_STAGE, &xmap, (kb0 + i) * kScaleBlock, m0, &sh.full[s]);
    };
    if (tc::elect_one())
      for (int i = 0; i < ahead; ++i) {
        mbar_arrive_expect_tx(&sh.full[i], G_STAGE + sx_bytes);
        tc::tma_load_2d(smem + i * G_STAGE + G_TILE, &wmap, (kb0 + i) * kScaleBlock, n0, &sh.full[i]);
      }
    __syncwarp();
    griddep_wait();  // the codes and scales of x
    if (tc::elect_one())
      for (int i = 0; i < ahead; ++i) load_x(i);
    __syncwarp();
    int i = ahead;
    for (; i < nk; ++i) {
      const int s = i % GSTAGES;
      if (!gwait(sh, &sh.empty[s], (uint32_t)((i / GSTAGES - 1) & 1), a.status)) break;
      if (tc::elect_one()) {
        mbar_arrive_expect_tx(&sh.full[s], G_STAGE + sx_bytes);
        tc::tma_load_2d(smem + s * G_STAGE + G_TILE, &wmap, (kb0 + i) * kScaleBlock, n0, &sh.full[s]);
        load_x(i);
      }
      __syncwarp();
    }
    // every copy has landed and every commit has arrived before the stages are
    // reused or the CTA ends
    if (lane == 0)
      for (int j = max(0, i - GSTAGES); j < i; ++j) {
        mbar_wait(&sh.full[j % GSTAGES], (uint32_t)((j / GSTAGES) & 1));
        if (!sh.abort_flag) mbar_wait(&sh.empty[j % GSTAGES], (uint32_t)((j / GSTAGES) & 1));
      }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16_f32(GM, GN);  // the same fields; format 0 is E4M3 here
    int i = 0;
    for (; i < nk; ++i) {
      const int s = i % GSTAGES, b = i & 1;
      if (!gwait(sh, &sh.full[s], (uint32_t)((i / GSTAGES) & 1), a.status)) break;
      if (i >= 2 && !gwait(sh, &sh.p_empty[b], (uint32_t)((i / 2 - 1) & 1), a.status)) break;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint32_t xa = smem_u32(smem) + s * G_STAGE, wa = xa + G_TILE;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_f8(tmem + b * GN, tc::sw128_desc(xa + 32 * k), tc::sw128_desc(wa + 32 * k), idesc, k > 0);
        tc::commit(&sh.empty[s]);
        tc::commit(&sh.p_full[b]);
      }
      __syncwarp();
    }
    if (lane == 0 && i > 0) mbar_wait(&sh.p_full[(i - 1) & 1], (uint32_t)(((i - 1) / 2) & 1));
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16) + 64 * half;
    BlockScales sw;
    sw.start(a.sw + (size_t)(n0 / kScaleBlock) * a.nkb + kb0, nk, lane);
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = make_float2(0.f, 0.f);
    for (int i = 0; i < nk; ++i) {
      const int b = i & 1;
      const float w = sw.at(i);
      if (!gwait(sh, &sh.p_full[b], (uint32_t)((i / 2) & 1), a.status)) break;
      tc::fence_after_sync();
      const float f0 = w * sh.sx[i % GSX_SLOTS][32 * q + lane];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t p[16];
        ld_32x32b_x16(t_lane + b * GN + 16 * h, p);
        tc::wait_ld();
        if (h == 3) {  // the next block but one may overwrite the buffer
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_empty[b]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) fma2(acc[8 * h + j], p[2 * j], p[2 * j + 1], f0);
      }
    }
  }
  __syncthreads();  // every stage's copies have landed and every MMA has read them
  if (SPLIT == 1) {
    if (warp >= 2) {
      const int n = n0 + 64 * ((warp - 2) >> 2), m = m0 + 32 * (warp & 3);
      uint8_t* tile = smem + (warp - 2) * 4096;
      stage_rows(tile, acc, a.bias, n, a.N, lane);
      tc::fence_proxy_async();
      __syncwarp();
      if (n < a.N && m < a.M && tc::elect_one()) {
        tc::tma_store_2d(&omap, n, m, tile);
        tc::bulk_commit();
        tc::bulk_wait_all();
      }
      __syncwarp();
    }
  } else {
    constexpr int kRowsOf = GM / SPLIT;  // rows a CTA owns
    float* ex = reinterpret_cast<float*>(smem + GSTAGES * G_STAGE);  // [SPLIT][kRowsOf][G_PITCH]
    cluster_wait();
    if (warp >= 2) {
      const int row = 32 * (warp & 3) + lane, col = 64 * ((warp - 2) >> 2);
      const uint32_t to = in_cta(ex + (rank * kRowsOf + row % kRowsOf) * G_PITCH + col, row / kRowsOf);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        st_cluster(to + 16 * j, acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int e = tid; e < kRowsOf * (GN / 8); e += kGemmThreads) {
      const int lr = e / (GN / 8), r = rank * kRowsOf + lr, c8 = 8 * (e % (GN / 8));
      if (m0 + r >= a.M || n0 + c8 >= a.N) continue;
      float v[8] = {};
#pragma unroll
      for (int p = 0; p < SPLIT; ++p) {
        const float4* src = reinterpret_cast<const float4*>(ex + (p * kRowsOf + lr) * G_PITCH + c8);
        const float4 lo = src[0], hi = src[1];
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
      }
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        o[u] = pack_bf16x2(v[2 * u] + bias_at(a, n0 + c8 + 2 * u), v[2 * u + 1] + bias_at(a, n0 + c8 + 2 * u + 1));
      *reinterpret_cast<uint4*>(a.out + (size_t)(m0 + r) * a.out_stride + n0 + c8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 2 * GN);
  }
}

namespace {

// The streamed kernel up to 8 rows (N 5120, K 2048: 4.6 - 4.8 us against 8.5 on
// tcgen05), up to 16 where the weights are few (N 5120, K 2048: 7.3 against 8.6,
// but K 4096: 13.0 against 11.6 - 12.3, and N 10240, K 2048: 11.4 against 9.5),
// and with more where its CTAs of 16 features x 32 rows all run at once over a
// short K (M 64, N 640, K 512: 3.2 against 5.4 us; but M 24, N 2048, K 4096: 9.4
// against 9.0, M 24, N 5120, K 2048: 14.6 against 8.5).
bool linear_streams(const moe_linear_dims& d) {
  return d.M <= 8 || (d.M <= 16 && (long long)d.N * d.K <= (1 << 24)) ||
         (d.K <= 2048 && cdiv(d.N, 16) * (long long)cdiv(d.M, 32) <= num_sms());
}

template <int NT>
cudaError_t launch_stream(const LinArgs& a, cudaStream_t s) {
  const dim3 grid(cdiv(a.N, 16), cdiv(a.M, 8 * NT));
  // a warp per block of K, up to 16 where an SM has one CTA, up to 8 where it
  // has two, otherwise 4; more than 8 rows take 8, whose quantisation hides
  // (N x K, 1 row: 2048 x 4096 5.4 / 4.0 / 3.5 us with 4 / 8 / 16 warps, 4096 x
  // 2048 3.9 / 3.5 / 4.1, 5120 x 2048 4.5 / 4.8 / 5.5; 16 rows, 5120 x 2048:
  // 8.7 / 7.3 / 8.9)
  const int nkb = cdiv(a.K, kScaleBlock), ctas = grid.x * grid.y;
  if (ctas <= num_sms() && nkb > 8)
    return launch_k(k_linear_stream<NT, 16>, grid, dim3(512), 0, s, true, a);
  if ((ctas <= 2 * num_sms() || NT > 1) && nkb > 4)
    return launch_k(k_linear_stream<NT, 8>, grid, dim3(256), 0, s, true, a);
  return launch_k(k_linear_stream<NT, 4>, grid, dim3(128), 0, s, true, a);
}

struct LinWs {
  size_t codes, sxt, total;
  int ld;
};
LinWs lin_ws(const moe_linear_dims& d) {
  LinWs w{};
  if (linear_streams(d)) {
    w.total = 256;
    return w;
  }
  const size_t nkb = cdiv(d.K, kScaleBlock);
  w.ld = cdiv(d.M, 32) * 32;
  w.codes = 0;
  w.sxt = ((size_t)d.M * d.K + 255) & ~size_t(255);
  w.total = w.sxt + nkb * w.ld * sizeof(float);
  return w;
}

// One launch of the GEMM, attributes and all.
struct GemmLaunch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  GemmLaunch(int split, int tiles_n, int tiles_m, cudaStream_t s) {
    cfg.gridDim = dim3(split, tiles_n, tiles_m);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = g_smem(split);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
  }
};
template <int SPLIT>
cudaError_t launch_gemm(const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& omap,
                        const GemmArgs& a, cudaStream_t s) {
  cudaError_t err = ensure_smem((const void*)k_linear_gemm<SPLIT>, g_smem(SPLIT));
  if (err != cudaSuccess) return err;
  count_launch();
  const GemmLaunch l(SPLIT, cdiv(a.N, GN), cdiv(a.M, GM), s);
  return cudaLaunchKernelEx(&l.cfg, k_linear_gemm<SPLIT>, xmap, wmap, omap, a);
}
// Clusters of SPLIT that the current GPU holds at once (fewer than its SMs /
// SPLIT, where its clusters of SMs are no multiples of it).
template <int SPLIT>
int clusters_at_once() {
  static PerDevice known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return known.get(dev, [] {
    int most = 0;
    GemmLaunch l(SPLIT, 1, 1, nullptr);
    l.cfg.numAttrs = 1;
    l.cfg.attrs = l.attr + 1;
    if (ensure_smem((const void*)k_linear_gemm<SPLIT>, g_smem(SPLIT)) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&most, k_linear_gemm<SPLIT>, &l.cfg) == cudaSuccess)
      return most;
    cudaGetLastError();
    return -1;
  });
}

}  // namespace

size_t linear_fp8_workspace(const moe_linear_dims& d) { return lin_ws(d).total; }

cudaError_t launch_linear_fp8(const uint16_t* x, const moe_fp8_mat& w, const float* bias,
                              const moe_linear_dims& d, uint16_t* out, void* ws, int32_t* status,
                              cudaStream_t s) {
  if (linear_streams(d)) {
    const LinArgs a{x, d.x_stride, w.codes, w.scales, bias, out, d.out_stride, d.M, d.N, d.K, status};
    if (d.M <= 8) return launch_stream<1>(a, s);
    if (d.M <= 16) return launch_stream<2>(a, s);
    return launch_stream<4>(a, s);
  }
  const LinWs l = lin_ws(d);
  uint8_t* codes = static_cast<uint8_t*>(ws) + l.codes;
  float* sxt = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.sxt);
  const int nkb = cdiv(d.K, kScaleBlock);
  CUtensorMap xmap, wmap, omap;
  cudaError_t err;
  if ((err = make_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, d.M, d.K,
                                kScaleBlock, GM, 128)) != cudaSuccess ||
      (err = make_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w.codes, d.N, d.K,
                                kScaleBlock, GN, 128)) != cudaSuccess ||
      // stored 64 features x 32 rows at a time
      (err = make_tensor_map_2d(&omap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, d.M, d.N, 64, 32, 128,
                                d.out_stride)) != cudaSuccess)
    return err;
  const long long groups = (long long)d.M * nkb;
  err = launch_k(k_linear_quant, dim3((unsigned)((groups + 15) / 16)), dim3(256), 0, s, true, x,
                 (long long)d.x_stride, d.M, d.K, codes, sxt, l.ld, status);
  if (err != cudaSuccess) return err;
  const GemmArgs a{sxt, l.ld, w.scales, bias, out, d.out_stride, d.M, d.N, nkb, status};
  const int tiles = cdiv(d.M, GM) * cdiv(d.N, GN);
  // K divided while all clusters run at once, one CTA per SM, and a CTA has four
  // blocks: clusters of four, two CTAs per SM take longer to place than they
  // save (M 203, N 2048, K 4096: 15.8 / 12.7 / 11.7 / 19.3 us with 1 / 2 / 4 / 8
  // CTAs per tile; M 1000, N 2048, K 2048, 128 tiles: 11.4 / 13.8 us with 1 / 2;
  // M 64, N 4864, K 2048, 38 tiles: 9.1 / 14.5 with 2 / 4, as 38 clusters of 4
  // do not fit)
  int split = 1;
  if (tiles <= clusters_at_once<2>() && nkb >= 8) split = 2;
  if (tiles <= clusters_at_once<4>() && nkb >= 16) split = 4;
  if (split == 1) return launch_gemm<1>(xmap, wmap, omap, a, s);
  if (split == 2) return launch_gemm<2>(xmap, wmap, omap, a, s);
  return launch_gemm<4>(xmap, wmap, omap, a, s);
}

}  // namespace moe
