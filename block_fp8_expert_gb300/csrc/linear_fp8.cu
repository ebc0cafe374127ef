// Block-FP8 linear layer on E4M3 activations (moe_linear_fp8):
//   out[m, n] = sum_b Sx[m, b] Sw[n / 128, b] P_b[m, n] + bias[n],
//   P_b[m, n] = sum over the 128 columns of block b of code_x code_w.
#include "decoder_internal.h"

namespace moe {

namespace {
constexpr int kLinWarps = 8;

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
template <int NT>
__global__ void __launch_bounds__(kLinWarps * 32)
k_linear_stream(const LinArgs a) {
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ float red[kLinWarps][NT][4][32];
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

size_t linear_fp8_workspace(const moe_linear_dims&) { return 256; }

cudaError_t launch_linear_fp8(const uint16_t* x, const moe_fp8_mat& w, const float* bias,
                              const moe_linear_dims& d, uint16_t* out, void* ws, int32_t* status,
                              cudaStream_t s) {
  const LinArgs a{x, d.x_stride, w.codes, w.scales, bias, out, d.out_stride, d.M, d.N, d.K, status};
  const dim3 blk(kLinWarps * 32);
  const int nt = d.M <= 8 ? 1 : d.M <= 16 ? 2 : 4;
  const dim3 grid(cdiv(d.N, 16), cdiv(d.M, 8 * nt));
  if (nt == 1) return launch_k(k_linear_stream<1>, grid, blk, 0, s, false, a);
  if (nt == 2) return launch_k(k_linear_stream<2>, grid, blk, 0, s, false, a);
  return launch_k(k_linear_stream<4>, grid, blk, 0, s, false, a);
}

}  // namespace moe
