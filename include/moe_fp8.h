/*
 * moe_fp8.h - C ABI of a block-FP8 (E4M3) Mixture-of-Experts FFN layer for
 * NVIDIA GB300 (sm_103a).
 *
 * The layer, as the colizig README states its parts (model table under "What
 * this project is trying to prove": experts, top-k routing, an optional shared
 * expert; "Features": block-FP8 E4M3 expert weights evaluated with a fused
 * decode+FMA dot product, MoE per-expert evaluation):
 *
 *   l[t,e]  = sum_h x[t,h] Wr[e,h] (+ b[e])                       router GEMM
 *   p[t,:]  = softmax(l[t,:]) over the E experts
 *   idx,w   = the k largest p[t,e] (descending, ties to the lower e),
 *             w_j = p_j / sum_{selected} p                        top-k, renorm
 *   rows    = the (t,j) pairs sorted by expert, ascending t inside an expert
 *   W[r,c]  = dec(C[r,c]) * S[r/128, c/128]                       block-FP8
 *   hid     = silu(x Wg^T) * (x Wu^T),  silu(z) = z/(1+exp(-z))   SwiGLU
 *   y       = hid Wd^T                                            down proj.
 *   out[t]  = sum_j w[t,j] y[row(t,j)] (+ shared(x[t]))           combine
 *
 * Conventions shared by every call:
 *  - Every pointer is a DEVICE pointer the caller owns (allocated, for
 *    example, by PyTorch); the library allocates no memory.  Every array must
 *    start on a 16-byte boundary.
 *  - bf16 arrays are passed as uint16_t bit patterns (IEEE binary32 top half).
 *  - `stream` is a cudaStream_t passed as void*; every call only enqueues
 *    work on it and returns without synchronising the host, so a sequence of
 *    calls can be captured into a CUDA graph.  Host-side argument errors are
 *    returned before anything is enqueued.
 *  - `ws` is a caller-owned device workspace of at least the size returned
 *    by moe_workspace_bytes() for the same dims; its contents on entry do not
 *    matter.  Calls that overlap on the GPU must not share one workspace.
 *  - T = 0 is valid: the call checks its dims and returns MOE_OK without
 *    touching any array (moe_permute still writes the E+1 zero offsets), so
 *    token-sized pointers may then be NULL.
 *  - Supported shapes: H, I and I_shared (when non-zero) multiples of 64 and
 *    at most 16384; 1 <= E <= 1024; 1 <= k <= min(E, 32); 0 <= T and
 *    T*k < 2^31.  Other shapes return MOE_ERR_UNSUPPORTED.
 *  - Errors are never silent.  A call returns MOE_OK only after every check
 *    it can make on the host; errors the kernels detect (for example an
 *    expert index out of range given to moe_permute) set a status word in the
 *    workspace that moe_read_device_status() returns.  There is no CPU
 *    fallback: without a usable GPU every call fails with MOE_ERR_CUDA.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status;

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG 1     /* null or misaligned pointer, bad value  */
#define MOE_ERR_UNSUPPORTED 2     /* shape outside the supported set        */
#define MOE_ERR_WORKSPACE 3       /* workspace smaller than required        */
#define MOE_ERR_CUDA 4            /* a CUDA launch or runtime call failed   */
#define MOE_ERR_DEVICE_STATUS 5   /* a kernel flagged bad input on device   */
#define MOE_ERR_TIMEOUT 6         /* a bounded device wait gave up          */
#define MOE_ERR_NOT_IMPLEMENTED 7

/* Device status bits (moe_read_device_status). */
#define MOE_DEV_BAD_EXPERT_INDEX 1 /* moe_permute saw idx < 0 or idx >= E   */
#define MOE_DEV_WAIT_TIMEOUT 2     /* a kernel's bounded wait ran out       */
#define MOE_DEV_FP16_RANGE 4       /* an fp16 intermediate left its range   */
#define MOE_DEV_NONFINITE 8        /* an input (x, a block scale) or an
                                      intermediate was infinite or NaN      */
#define MOE_DEV_BAD_PAGE 16        /* a cache slot, page number or sequence
                                      length outside the cache or its table */
#define MOE_DEV_BAD_POSITION 32    /* a position outside the cos/sin table  */

/* Layer dimensions. T tokens, hidden size H, routed-expert intermediate I,
 * E routed experts, top-k, shared-expert intermediate I_shared (0 = none). */
typedef struct {
  int32_t T, H, I, E, k, I_shared;
} moe_dims;

/* One block-FP8 weight stack: codes are E4M3 bytes, scales one float per
 * 128x128 block.  For a stack of n matrices of shape [rows, cols] (rows =
 * output features, cols = input features, cols contiguous):
 *   codes  uint8 [n, rows, cols]
 *   scales float [n, ceil(rows/128), ceil(cols/128)]                       */
typedef struct {
  const uint8_t* codes;
  const float* scales;
} moe_fp8_mat;

/* The three projections of n experts: gate and up [n, I, H], down [n, H, I]. */
typedef struct {
  moe_fp8_mat gate, up, down;
} moe_fp8_ffn;

/* Short text for a status code (static storage). */
const char* moe_status_string(moe_status s);

/* Text of the most recent failure on the calling host thread ("" if none). */
const char* moe_last_error_message(void);

/* Library version string, e.g. "moe_fp8 0.1 sm_103a". */
const char* moe_version(void);

/* Diagnostic: kernel launches this library has issued in this process (all
 * host threads; a launch recorded into a CUDA graph counts once, at capture).
 * No counterpart in the pages: it lets a caller count the kernels of one
 * call, e.g. around the capture of one moe_layer_forward. */
unsigned long long moe_kernel_launches(void);

/* Diagnostic: 1 if the routed experts of a layer call with dimensions d run
 * on the tensor-core grouped GEMM, 0 if on the streamed GEMV (the regime rule
 * documented at moe_layer_forward, including the MOE_FP8_EXPERT_PATH
 * override); -1 if d is invalid.  No GPU work, no counterpart in the pages. */
int moe_expert_uses_gemm(moe_dims d);

/* Workspace size in bytes that every call below needs for dims d. */
moe_status moe_workspace_bytes(moe_dims d, size_t* bytes);

/*
 * Router: logits, softmax over experts, top-k with renormalisation (colizig
 * README, model table under "What this project is trying to prove": 128
 * experts top-8, or 512 experts top-10, per MoE layer).
 *   x        bf16  [T, H]
 *   Wr       float [E, H]
 *   bias     float [E] or NULL
 *   topk_idx int32 [T, k]  out: experts in descending probability, ties to
 *                          the lower expert index
 *   topk_w   float [T, k]  out: p_j / sum of the k selected p
 * Logits are accumulated in fp32.  The renormalised weights equal the softmax
 * over the k selected logits, which is how they are computed.  Clears the
 * workspace's device status word.
 */
moe_status moe_route(const uint16_t* x, const float* Wr, const float* bias,
                     moe_dims d, int32_t* topk_idx, float* topk_w, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * Permutation of the T*k (token, slot) pairs into expert-contiguous rows, so
 * that each selected expert is evaluated once over all of its tokens
 * (colizig README, "Features": MoE per-expert evaluation).
 *   topk_idx     int32 [T, k]   in
 *   expert_off   int32 [E + 1]  out: segment e is rows [off[e], off[e+1]),
 *                               off[0] = 0, off[E] = T*k
 *   row_token    int32 [T*k]    out: token of each permuted row; inside one
 *                               segment tokens ascend
 *   tok_slot_row int32 [T*k]    out: row of pair (t, j) at index t*k + j
 * The result is unique and deterministic (no atomics decide an order).  An
 * index outside [0, E) sets MOE_DEV_BAD_EXPERT_INDEX; its pair gets no row
 * (tok_slot_row = -1) and off[E] counts only valid pairs.
 */
moe_status moe_permute(const int32_t* topk_idx, moe_dims d,
                       int32_t* expert_off, int32_t* row_token,
                       int32_t* tok_slot_row, void* ws, size_t ws_bytes,
                       void* stream);

/*
 * Routed experts: for every permuted row r of expert e,
 *   y_perm[r] = (silu(x[row_token[r]] Wg_e^T) * (x[row_token[r]] Wu_e^T)) Wd_e^T
 * with W = dec(codes) * block scale (colizig README, "Features": block-FP8
 * E4M3 weights dequantised inside a fused decode+FMA dot product, MoE
 * per-expert evaluation).
 *   x          bf16  [T, H]
 *   expert_off int32 [E + 1], row_token int32 [T*k]  (from moe_permute)
 *   w          the E routed experts
 *   y_perm     float [T*k, H] out (rows past off[E] are left untouched)
 * d.T and d.k size the row space; d.I_shared is ignored.
 * Precision and range: the products run on fp16 operands with fp32
 * accumulation.  Every fp16 operand and intermediate (activations, scaled
 * weights, the SwiGLU output hid) is normalised by an exact power of two
 * that the fp32 side undoes, so block scales and activations of any
 * magnitude keep fp16's relative precision; the remaining roundings are
 * one fp16 rounding of each scaled weight (tensor-core GEMM) and of hid.
 * Flags: MOE_DEV_NONFINITE for an infinite or NaN activation, block scale
 * or result; on the tensor-core GEMM (many rows per expert), whose hid uses
 * a fixed power of two per expert, MOE_DEV_FP16_RANGE when a hid value
 * exceeds fp16's range or a token's values of 32 features all fall below
 * 2^-12 of the normalised scale (weights whose codes are far smaller or
 * larger than their block scale suggests).  Clears the device status word
 * first.
 */
moe_status moe_expert_ffn_fp8(const uint16_t* x, const int32_t* expert_off,
                              const int32_t* row_token, moe_fp8_ffn w,
                              moe_dims d, float* y_perm, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * Combine of the expert outputs back to token order, weighted by the
 * renormalised routing weights (colizig README, model table: top-k routed
 * experts plus, for the 512-expert family, one shared expert):
 * out[t] = sum_j topk_w[t,j] y_perm[tok_slot_row[t*k+j]]
 *                   (+ shared_y[t] when shared_y is not NULL),
 * summed in fp32 in slot order and rounded once to bf16 (nearest-even).
 * Pairs with tok_slot_row < 0 contribute nothing.
 *   y_perm float [T*k, H], tok_slot_row int32 [T*k], topk_w float [T, k],
 *   shared_y float [T, H] or NULL, out bf16 [T, H].
 */
moe_status moe_combine(const float* y_perm, const int32_t* tok_slot_row,
                       const float* topk_w, const float* shared_y, moe_dims d,
                       uint16_t* out, void* stream);

/*
 * The whole layer (colizig README, model table under "What this project is
 * trying to prove" and "Status": MoE (+shared expert) with block-FP8
 * weights): route, permute, routed experts, the shared expert when
 * d.I_shared > 0 (applied to every token with weight 1), combine.  The
 * expert outputs stay in the workspace as fp16 with one power-of-two
 * exponent per row and 32 columns, so they too have no range limit; the
 * precision and flags are those of moe_expert_ffn_fp8.
 *   shared       NULL when d.I_shared == 0, else one expert (n = 1) with
 *                gate/up [I_shared, H] and down [H, I_shared]
 *   out          bf16 [T, H]
 *   topk_idx_out int32 [T, k] or NULL: the routing, for inspection
 *   topk_w_out   float [T, k] or NULL
 * The regime (few tokens per expert: streamed grouped GEMV; many tokens per
 * expert: tensor-core grouped GEMM) is chosen on the host from T*k/E only:
 * the GEMM (tcgen05, needs H % 256 == 0, I % 128 == 0, H, I <= 4096) from 1
 * row per routed expert on average (T*k >= E) when H*I >= 2^20, else from
 * 32 rows per expert; the shared expert: from 32 tokens.  The
 * environment variable MOE_FP8_EXPERT_PATH=gemm or =gemv overrides the choice
 * (diagnostics and tests; read on every call).  The GEMM runs its gate/up
 * and down tiles in one launch when gate/up tiles alone fill the SMs and
 * there are at most 16 tiles per SM (bounded from the shapes), else in two;
 * MOE_FP8_GEMM_LAUNCHES=1 or =2 forces either.  Two more diagnostic
 * variables, read on every call of the tensor-core GEMM, exist to test the
 * failure path: MOE_FP8_WAIT_LIMIT_US shortens its bounded device waits
 * (default 2 s), and MOE_FP8_TEST_STALL=down makes its down projection wait
 * for one more finished gate/up tile than exists, so that the wait runs out
 * and MOE_DEV_WAIT_TIMEOUT is set (the output is then not valid).
 */
moe_status moe_layer_forward(const uint16_t* x, const float* Wr,
                             const float* bias, moe_fp8_ffn routed,
                             const moe_fp8_ffn* shared, moe_dims d,
                             uint16_t* out, int32_t* topk_idx_out,
                             float* topk_w_out, void* ws, size_t ws_bytes,
                             void* stream);

/*
 * The layer with a gated shared expert: as moe_layer_forward, except that
 * the shared expert's output for token t is scaled by
 * sigmoid(sum_h x[t,h] shared_gate[h]) before it is added.  This variant is
 * not on the colizig README (its 512-expert family lists "top-10 + 1 shared"
 * without a gate); it is the sigmoid-gated form of that shared expert.
 *   shared_gate float [H]; the layer must have a shared expert
 *               (d.I_shared > 0, shared not NULL).
 * The gate is computed by the routing kernels in fp32 and applied in the
 * combine.
 */
moe_status moe_layer_forward_gated(const uint16_t* x, const float* Wr,
                                   const float* bias, moe_fp8_ffn routed,
                                   const moe_fp8_ffn* shared,
                                   const float* shared_gate, moe_dims d,
                                   uint16_t* out, int32_t* topk_idx_out,
                                   float* topk_w_out, void* ws, size_t ws_bytes,
                                   void* stream);

/*
 * The layer with E4M3 activations in the routed experts.  The pages' block-FP8
 * format covers the weights only; this variant also feeds the experts' inputs
 * to the tensor cores as E4M3 (tcgen05.mma kind::f8f6f4), so the weight
 * codes are multiplied without a decode.  Routing and combine are those of
 * moe_layer_forward.  The inputs of each projection (x, then the SwiGLU
 * output hid in fp32) are quantised per row and group of 128 input features
 * (the weights' scale-block width): with a the group's largest magnitude,
 * code = E4M3(v * fp32(448 / a)) rounded to nearest even and saturated to
 * +-448, scale = fp32(a / 448); a = 0 gives zero codes and scale.  Each
 * 128-wide K block's E4M3 product sums are scaled by the weight and
 * activation scales in fp32 and accumulated in fp32.
 * Accuracy: the quantisation of x and hid costs about 4.5% of the output's
 * rms against the bf16-activation layer (measured on the synthetic
 * workloads; largest elements up to about 20%), so the layer is checked
 * against its own definition, not against moe_layer_forward's tolerance.
 * Shapes: H % 256 == 0, I % 128 == 0, H, I <= 2048, any T; other shapes
 * and layers with a shared expert (d.I_shared > 0) return
 * MOE_ERR_UNSUPPORTED.  Arguments as moe_layer_forward without `shared`.
 */
moe_status moe_layer_forward_act8(const uint16_t* x, const float* Wr,
                                  const float* bias, moe_fp8_ffn routed,
                                  moe_dims d, uint16_t* out,
                                  int32_t* topk_idx_out, float* topk_w_out,
                                  void* ws, size_t ws_bytes, void* stream);

/*
 * moe_permute without a workspace, for callers that cannot allocate device
 * memory: for example a plugin whose host framework passes it only the input
 * and output buffers of each call, or a serving loop whose device memory is
 * fixed at start-up.  The paper has no counterpart to this call.
 *
 * Same arguments, results and determinism as moe_permute, minus ws/ws_bytes.
 * Its scratch is one array compiled into the library (about 1.3 MB, held on
 * every GPU that loads the library until the process exits), sized for
 * T*k <= 65536 and E <= 512; larger sizes return MOE_ERR_UNSUPPORTED before
 * anything is enqueued.  It calls no allocator.
 *  - The first call on a device looks up the array's device address with
 *    that device current (cudaGetSymbolAddress) and caches it; make that
 *    first call before any stream capture on the device.
 *  - All calls on a device share the array, and it keeps the last call's
 *    contents: calls that overlap on the GPU race and give undefined
 *    results; order them on one stream (or with events).  Each call clears
 *    the status word it uses before its kernels run; every other scratch
 *    value is written before it is read.
 *  - An expert index outside [0, E) gives its pair tok_slot_row = -1 and no
 *    row, as in moe_permute, and sets MOE_DEV_BAD_EXPERT_INDEX in the fixed
 *    array's status word: moe_read_device_status(NULL, ...) reads it.
 */
moe_status moe_permute_static_scratch(const int32_t* topk_idx, moe_dims d,
                                      int32_t* expert_off, int32_t* row_token,
                                      int32_t* tok_slot_row, void* stream);

/*
 * Runtime cross-check of a layer call on sampled tokens, the GPU counterpart
 * of the colizig README's --cuda-verify (CLI reference), which checks the
 * CUDA path against the CPU path.  It recomputes the layer output of each
 * listed token on an arithmetic path independent of the layer kernels
 * (plain fp32 dot products, the E4M3 codes decoded from their bit fields
 * times their block scale, no tensor cores, no power-of-two normalisation),
 * from the routing the layer call produced, and compares it with `out`.
 *   x, routed, shared, shared_gate, d   as given to the layer call
 *                  (shared_gate NULL for moe_layer_forward)
 *   out            bf16 [T, H], the layer call's output
 *   topk_idx, topk_w  the layer call's routing ([T, k]; pass topk_idx_out /
 *                  topk_w_out of the layer call)
 *   tokens         int32 [n_tokens], token indices in [0, T); 1 <= n_tokens
 *                  <= 64
 *   result         float [3] out (device): worst |out - ref| / (1e-2 (|ref| +
 *                  rms(ref))) over the sampled outputs (<= 1: within the
 *                  layer tolerance; infinite for a NaN or an expert index
 *                  outside [0, E)), worst |out - ref|, rms(ref)
 *   ws, ws_bytes   scratch of at least moe_verify_workspace_bytes(d, n_tokens)
 * Enqueued on `stream` like every call; read `result` after synchronising.
 */
moe_status moe_verify_workspace_bytes(moe_dims d, int n_tokens, size_t* bytes);
moe_status moe_verify_layer(const uint16_t* x, moe_fp8_ffn routed,
                            const moe_fp8_ffn* shared, const float* shared_gate,
                            moe_dims d, const uint16_t* out,
                            const int32_t* topk_idx, const float* topk_w,
                            const int32_t* tokens, int n_tokens, float* result,
                            void* ws, size_t ws_bytes, void* stream);

/*
 * Copy the workspace's device status word to *status (MOE_DEV_* bits) after
 * synchronising `stream`.  Returns MOE_ERR_DEVICE_STATUS when any bit is set.
 * The word is cleared at the start of moe_route, moe_permute,
 * moe_expert_ffn_fp8 and moe_layer_forward.  With ws == NULL it reads the
 * status word of moe_permute_static_scratch's fixed array on the current
 * device instead (this does no allocation; on a device where that call has
 * not run yet it looks up the array's address first).  An unfinished or
 * invalid result is reported here rather than returned as a plausible
 * number (colizig README, "What this project is trying to prove" and
 * "Status": an incomplete subsystem returns an error, not a wrong number).
 */
moe_status moe_read_device_status(const void* ws, int32_t* status,
                                  void* stream);

/*
 * ---------------------------------------------------------------------------
 * The rest of a decoder layer around the MoE layer: expert selection with
 * balance bias and groups, query/key norms with rotary positions into a paged
 * key/value cache, attention of one new token per sequence or of several
 * drafted ones over that cache, a paged cache of latent vectors with the
 * attention over it, and the block-FP8 linear layers between them.  None of these has a
 * counterpart in the pages, which state the MoE layer only.
 *
 * They follow the conventions above, with two additions:
 *  - `status` (may be NULL) is a device array of 16 int32 that the caller
 *    zeroes once.  A call ORs MOE_DEV_* bits into word 0 and never clears
 *    them; moe_read_device_status(status, ...) reads it.
 *  - Rows may be strided.  A row stride counts elements and is at least the
 *    row's length; the elements inside a row are contiguous, and every row
 *    starts on a 16-byte boundary where noted.
 *  - topk_idx, topk_w, pos, slots, block_table, seq_lens, draft_lens, mask,
 *    cu_q, cu_k, k_scale and v_scale need the alignment of their elements only
 *    (a step's part of a longer array will do); every other pointer is 16-byte
 *    aligned.
 * ---------------------------------------------------------------------------
 */

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/* How moe_select_experts scores and picks. */
typedef struct {
  int32_t score;      /* MOE_SCORE_*                                         */
  int32_t groups;     /* equal groups of consecutive experts; 1: no groups   */
  int32_t top_groups; /* groups that stay in the running                     */
  int32_t group_top;  /* 1 or 2: a group's score is the sum of that many of
                         its largest keys                                    */
  int32_t renorm;     /* 1: divide the weights by their sum                  */
  float scale;        /* factor on the weights                               */
} moe_select_rule;

/*
 * Experts from router logits:
 *   s[t,e] = softmax(logits[t,:])[e] or 1 / (1 + exp(-logits[t,e]))
 *   key    = s + bias          (bias balances the load; it only steers the
 *                               choice and never enters the weights)
 *   the top_groups groups of the largest group score are kept (ties: the
 *   lower group), then the k largest keys among their experts are chosen
 *   (descending, ties: the lower expert)
 *   topk_w = scale * s (renorm: divided by the sum of the k chosen s)
 * logits float [T, row_stride >= E]; bias float [E] or NULL; topk_idx int32
 * [T, k], topk_w float [T, k], as moe_permute and moe_combine take them.
 * 1 <= E <= 1024, 1 <= k <= 32, groups <= 32 divides E, E / groups >=
 * group_top, k <= top_groups * (E / groups).  Everything is fp32.  A logit of
 * -inf (an expert that is switched off) scores 0; where the chosen scores sum
 * to 0 the weights are 0, not NaN.  A NaN key counts as the largest key, and
 * NaN logits give NaN weights; the indices are valid whatever the logits.
 */
moe_status moe_select_experts(const float* logits, int64_t row_stride,
                              const float* bias, moe_select_rule rule,
                              int32_t T, int32_t E, int32_t k,
                              int32_t* topk_idx, float* topk_w, void* stream);

/*
 * moe_select_experts on the router's own logits: x Wr^T (+ logit_bias), as in
 * moe_route (x bf16 [T, H], Wr float [E, H], logit_bias float [E] or NULL,
 * workspace and status as there), then the selection by `rule`.
 */
moe_status moe_route_select(const uint16_t* x, const float* Wr,
                            const float* logit_bias, const float* bias,
                            moe_select_rule rule, moe_dims d,
                            int32_t* topk_idx, float* topk_w, void* ws,
                            size_t ws_bytes, void* stream);

/* moe_route_select that also ORs what it finds into `status` (may be NULL),
 * where it stays: the workspace's word is cleared by the next call on it. */
moe_status moe_route_select_status(const uint16_t* x, const float* Wr,
                                   const float* logit_bias, const float* bias,
                                   moe_select_rule rule, moe_dims d,
                                   int32_t* topk_idx, float* topk_w, void* ws,
                                   size_t ws_bytes, int32_t* status,
                                   void* stream);

/*
 * The layer after its router: the experts on a routing made elsewhere, by
 * moe_select_experts for example.  moe_layer_forward's permutation, routed
 * experts, shared expert and combine with its arguments, workspace, precision
 * and flags, except that topk_idx int32 [T, k] and topk_w float [T, k] are
 * given (the alignment of their elements will do), shared_gate float [H] may be
 * NULL (no gate), and the flags go to `status`; the workspace's own status word
 * is neither read nor written.
 * An index outside [0, E) raises MOE_DEV_BAD_EXPERT_INDEX and its pair adds
 * nothing.  With moe_route's routing the result is moe_layer_forward's.
 */
moe_status moe_experts_forward(const uint16_t* x, const int32_t* topk_idx,
                               const float* topk_w, moe_fp8_ffn routed,
                               const moe_fp8_ffn* shared,
                               const float* shared_gate, moe_dims d,
                               uint16_t* out, void* ws, size_t ws_bytes,
                               int32_t* status, void* stream);

#define MOE_KV_BF16 0
#define MOE_KV_E4M3 1

/* A paged key/value cache.  Token slot n (n = page * page_size + offset) of
 * head h starts at element page * page_stride + h * head_stride + offset *
 * token_stride of k and of v, D contiguous elements each; the strides are
 * multiples of 16 bytes.  MOE_KV_BF16: bf16 elements, k_scale and v_scale
 * NULL.  MOE_KV_E4M3: E4M3 codes, and one float per token and head at
 * element page * scale_page_stride + h * scale_head_stride + offset *
 * scale_token_stride of k_scale and of v_scale; the value is code * scale, a
 * scale being 0 or positive. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int32_t pages, page_size, Hkv, D, format;
  int64_t page_stride, head_stride, token_stride;
  int64_t scale_page_stride, scale_head_stride, scale_token_stride;
} moe_kv_cache;

/* One moe_qk_norm_rope call.  rot: leading dimensions of each head that are
 * rotated (0: none), a multiple of 16 and at most D; interleaved: 1 rotates
 * the pairs (2i, 2i + 1), 0 the pairs (i, i + rot / 2).  n_pos: rows of
 * cos_sin.  Strides in elements, multiples of 8. */
typedef struct {
  int32_t T, Hq, rot, interleaved, n_pos;
  float eps;
  int64_t qkv_stride, q_stride;
} moe_qk_dims;

/*
 * Per token t, on row t of qkv (bf16: Hq query heads, then Hkv key heads,
 * then Hkv value heads, D elements each, D = 64, 128 or 256):
 *   x' = x / sqrt(mean(x^2) + eps) * norm      query and key heads; norm NULL:
 *                                              x' = x
 *   (a, b) -> (a cos - b sin, b cos + a sin)   the rotated pairs i, with
 *                                              cos = cos_sin[pos[t]][i],
 *                                              sin = cos_sin[pos[t]][rot/2 + i]
 * in fp32, rounded once.  Queries go to q_out bf16 [T, q_stride >= Hq * D].
 * Keys and values go to slot slots[t] of the cache (slots[t] < 0: a padding
 * token, nothing is stored); two tokens of one call must not share a slot.
 * MOE_KV_E4M3: per token and head with a = the largest magnitude, code =
 * E4M3(v * fp32(448 * fp32(1 / a))) to nearest even, scale = fp32(a *
 * fp32(1 / 448)); a = 0 gives zero codes and scale; 0 < a < 2^-117 is treated
 * as a = 0.
 * q_norm, k_norm float [D] or NULL; cos_sin float [n_pos, rot], pos int32 [T]
 * (both NULL iff rot == 0); slots int64 [T].
 * A position outside [0, n_pos) raises MOE_DEV_BAD_POSITION: the token's
 * queries are NaN and it stores nothing.  A slot past the cache raises
 * MOE_DEV_BAD_PAGE and stores nothing.
 */
moe_status moe_qk_norm_rope(const uint16_t* qkv, const float* q_norm,
                            const float* k_norm, const float* cos_sin,
                            const int32_t* pos, const int64_t* slots,
                            moe_qk_dims d, moe_kv_cache cache, uint16_t* q_out,
                            int32_t* status, void* stream);

/* One moe_paged_attention call: B sequences, Hq query heads (a multiple of
 * the cache's Hkv; query head h reads key/value head h / (Hq / Hkv)).
 * table_width: page numbers per sequence in block_table, table_stride apart.
 * window > 0: only the last `window` tokens are attended to; 0: all.
 * q_stride, out_stride: elements between sequences, multiples of 8. */
typedef struct {
  int32_t B, Hq, table_width, window;
  float scale;
  int64_t table_stride, q_stride, out_stride;
} moe_attn_dims;

/*
 * Attention of one new token per sequence over the paged cache:
 *   out[b,h] = sum_t softmax_t(scale * q[b,h] . k[b,t]) v[b,t],
 *   t in [max(0, len - window), len), len = seq_lens[b]
 * q bf16 [B, q_stride] (Hq heads of D), block_table int32 [B, table_stride]:
 * token t of sequence b is offset t % page_size of page block_table[b][t /
 * page_size]; seq_lens int32 [B]; out bf16 [B, out_stride].  The cache's
 * length splits over the GPU and the parts are joined in a fixed order, so
 * equal calls give equal bits.  A sequence of length 0 gives zeros.  Cache
 * elements outside [max(0, len - window), len) are never read: they may
 * hold anything, and the pages of a window's past may be reused.
 * Scores, maxima, sums and outputs are fp32; the softmax weights enter the
 * product with the values as two bf16 parts next to bf16 values (2^-16 of the
 * weight), rounded to fp16 next to E4M3 values.  D = 64, 128 or 256; up to 2^31 - 1 tokens per sequence,
 * and about 2^31 tiles of 16 tokens in all (B * Hkv * the table's room).
 * A page number outside [0, pages) or a length outside [0, table_width *
 * page_size] raises MOE_DEV_BAD_PAGE; the tokens of such a page are left
 * out, and such a length is clamped.
 */
moe_status moe_paged_attention_workspace_bytes(moe_attn_dims d, int32_t D,
                                               size_t* bytes);
moe_status moe_paged_attention(const uint16_t* q, moe_kv_cache cache,
                               const int32_t* block_table,
                               const int32_t* seq_lens, moe_attn_dims d,
                               uint16_t* out, void* ws, size_t ws_bytes,
                               int32_t* status, void* stream);

/* One moe_linear_fp8 call: x [M, K] -> out [M, N].  M at most 2^22; N a
 * multiple of 8 and K of 16, both at most 65536; x_stride, out_stride:
 * elements between rows, multiples of 8. */
typedef struct {
  int32_t M, N, K;
  int64_t x_stride, out_stride;
} moe_linear_dims;

/*
 * out = x_q W^T + bias on E4M3 tensor-core products, W = dec(codes) * block
 * scale (w: one matrix [N, K] with scales [ceil(N/128), ceil(K/128)]).  The
 * activations are quantised in the call per row and group of 128 columns,
 * with a the group's largest magnitude:
 *   code = E4M3(x * fp32(448 * fp32(1 / a))) to nearest even,
 *   scale = fp32(a * fp32(1 / 448)); a = 0, or below 2^-117, gives zero codes
 *   and scale.
 * Each 128-wide block's products are summed and scaled by both scales in
 * fp32, the blocks are summed in fp32, and the result is rounded once.
 * x bf16 [M, x_stride], bias float [N] or NULL, out bf16 [M, out_stride].
 * An infinite or NaN activation raises MOE_DEV_NONFINITE (its output row is
 * then NaN or infinite).
 */
moe_status moe_linear_fp8_workspace_bytes(moe_linear_dims d, size_t* bytes);
moe_status moe_linear_fp8(const uint16_t* x, moe_fp8_mat w, const float* bias,
                          moe_linear_dims d, uint16_t* out, void* ws,
                          size_t ws_bytes, int32_t* status, void* stream);

/* One moe_tree_attention or moe_latent_attention call: B sequences with n new
 * tokens each at most, Hq query heads (moe_tree_attention: a multiple of the
 * cache's Hkv).  n in [1, 64], n * Hq / Hkv at most 8192.  table_width: page
 * numbers per sequence in block_table, table_stride apart.  window > 0 (at
 * least n; moe_tree_attention only): tokens further back are not attended to.
 * q_stride, out_stride: elements between sequences, q_row_stride,
 * out_row_stride between a sequence's tokens, multiples of 8 (the heads of a
 * token are contiguous); mask_stride: between the sequences' masks, 0 where
 * they share one. */
typedef struct {
  int32_t B, n, Hq, table_width, window;
  float scale;
  int64_t table_stride, q_stride, q_row_stride, out_stride, out_row_stride,
      mask_stride;
} moe_draft_dims;

/*
 * Attention of several new tokens per sequence, a tree of drafted ones or the
 * next few of a chain, over the paged cache that already holds them:
 *   out[b,i,h] = sum_t softmax_t(scale * q[b,i,h] . k[b,t]) v[b,t]
 * Sequence b has seq_lens[b] tokens in the cache, of which the last
 * draft_lens[b] (NULL: n; none of an empty sequence) are its new tokens 0, 1,
 * ...; those before are its context.  New token i sees the context, and new
 * token j where bit j of mask[b][i] is set (its ancestors and itself; bits from
 * draft_lens[b] on are ignored).  mask NULL: j <= i.  With a window, token i
 * stands c = max(1, number of new tokens that it sees) places after the
 * context's end and sees the last window - c tokens of the context.
 * q bf16 [B, n, Hq, D] and out bf16 [B, n, Hq, D] by their strides; block_table
 * as in moe_paged_attention; seq_lens, draft_lens int32 [B]; mask int64 [B, n].
 * Rows from draft_lens[b] on, and rows that see nothing, are zeros.  Pages
 * outside a sequence's length and window are not read; within a page that is
 * used anything may be, as what a row does not see does not reach it (NaN,
 * infinities and huge scales included).  What it sees does: a NaN score makes
 * the row NaN.  A score of -infinity has no weight, and a row that sees no other
 * is zeros, too.
 * The cache's length splits over the GPU and the parts are joined in a fixed
 * order, so equal calls give equal bits.  Scores, maxima, sums and outputs are
 * fp32; the softmax weights enter the product with the values as two bf16 parts
 * next to bf16 values (2^-15 of the weight), times the value's scale and rounded
 * to fp16 next to E4M3 values: 2^-11 of the product down to 2^-23 of the largest
 * weight times the largest value scale that the row has seen so far, and below
 * that steps of 2^-33 of it (so a token of tiny weight and a scale many orders
 * above the others takes bits from them).  Value scales may be any finite
 * numbers; outputs next to tiny ones are within 2^-126 times the number of
 * tokens.  A page number outside [0, pages), a
 * length outside [0, table_width * page_size] or a draft_lens[b] outside [0,
 * min(n, seq_lens[b])] raises MOE_DEV_BAD_PAGE; the tokens of such a page are
 * left out, and such a length is clamped.
 */
moe_status moe_tree_attention_workspace_bytes(moe_draft_dims d, int32_t Hkv,
                                              int32_t D, size_t* bytes);
moe_status moe_tree_attention(const uint16_t* q, moe_kv_cache cache,
                              const int32_t* block_table,
                              const int32_t* seq_lens, const int64_t* mask,
                              const int32_t* draft_lens, moe_draft_dims d,
                              uint16_t* out, void* ws, size_t ws_bytes,
                              int32_t* status, void* stream);

/* A paged cache of latent vectors, bf16: token slot n (n = page * page_size +
 * offset) is R elements of the vector and rot of the shared key part, R + rot
 * contiguous elements at page * page_stride + offset * token_stride of data.
 * R is 256 or 512, rot 64; the strides are multiples of 8. */
typedef struct {
  void* data;
  int32_t pages, page_size, R, rot;
  int64_t page_stride, token_stride;
} moe_latent_cache;

/* One moe_latent_store call: T tokens, H query heads (0: none).  interleaved:
 * 1 rotates the pairs (2i, 2i + 1), 0 the pairs (i, i + rot / 2).  n_pos: rows
 * of cos_sin.  Strides in elements, multiples of 8: between tokens, and
 * between the heads of q and q_out. */
typedef struct {
  int32_t T, H, interleaved, n_pos;
  float eps;
  int64_t kv_stride, q_stride, q_head_stride, q_out_stride, q_out_head_stride,
      rows_stride;
} moe_latent_dims;

/*
 * Per token t, on row t of kv (bf16: R elements of the latent vector, then rot
 * of the shared key part):
 *   c' = c / sqrt(mean(c^2) + eps) * norm      norm NULL: c' = c
 *   (a, b) -> (a cos - b sin, b cos + a sin)   the shared key part's pairs i, and
 *                                              those of the rot elements of each
 *                                              of the H heads of q, with
 *                                              cos = cos_sin[pos[t]][i],
 *                                              sin = cos_sin[pos[t]][rot/2 + i]
 * in fp32, rounded once.  The vector and the key part go to slot slots[t] of
 * the cache (slots[t] < 0: a padding token, nothing is stored; two tokens of
 * one call must not share a slot) and, where rows is given, to row t of rows;
 * the heads go to q_out, which may be q itself with its strides.
 * norm float [R]; cos_sin float [n_pos, rot]; pos int32 [T]; slots int64 [T];
 * q, q_out bf16 [T, H, rot] by their strides (NULL iff H == 0); rows bf16
 * [T, R + rot] or NULL.  A position outside [0, n_pos) raises
 * MOE_DEV_BAD_POSITION: the token's heads and its row are NaN and it stores
 * nothing.  A slot past the cache raises MOE_DEV_BAD_PAGE and stores nothing.
 */
moe_status moe_latent_store(const uint16_t* kv, const float* norm,
                            const float* cos_sin, const int32_t* pos,
                            const int64_t* slots, const uint16_t* q,
                            moe_latent_dims d, moe_latent_cache cache,
                            uint16_t* q_out, uint16_t* rows, int32_t* status,
                            void* stream);

/*
 * moe_tree_attention over latent vectors c[t] (latent attention in its absorbed
 * form: the queries have been taken through the heads' key projections, and
 * the outputs go through their value projections):
 *   out[b,i,h] = sum_t softmax_t(scale * q[b,i,h] . c[b,t]) c[b,t][0 .. R)
 * q bf16 [B, n, Hq, R + rot], out bf16 [B, n, Hq, R]; the rest as in
 * moe_tree_attention, without a window.  The softmax weights are rounded to
 * bf16 (2^-8 of the weight) before both the product and their sum.
 */
moe_status moe_latent_attention_workspace_bytes(moe_draft_dims d, int32_t R,
                                                size_t* bytes);
moe_status moe_latent_attention(const uint16_t* q, moe_latent_cache cache,
                                const int32_t* block_table,
                                const int32_t* seq_lens, const int64_t* mask,
                                const int32_t* draft_lens, moe_draft_dims d,
                                uint16_t* out, void* ws, size_t ws_bytes,
                                int32_t* status, void* stream);

/* One moe_expanded_attention call: B sequences of Tq query tokens and Tk key
 * tokens in all, H heads.  Strides in elements, multiples of 8: between tokens
 * and between heads, at least what they step over.  scale > 0. */
typedef struct {
  int32_t B, Tq, Tk, H;
  float scale;
  int64_t q_stride, q_head_stride, k_stride, k_head_stride, rope_stride,
      v_stride, v_head_stride, out_stride, out_head_stride;
} moe_expanded_dims;

/*
 * Latent attention in its expanded form, for prompts: every head has keys of
 * 128 dimensions of its own and 64 that all heads share, and values of 128:
 *   out[i,h] = sum_t softmax_t(scale * (q[i,h,:128] . k_nope[t,h]
 *                                       + q[i,h,128:] . k_rope[t])) v[t,h]
 * Sequence b has query tokens cu_q[b] .. cu_q[b+1] - 1 and key tokens cu_k[b]
 * .. cu_k[b+1] - 1, of which the last are its query tokens: query token i of lq
 * sees the keys t <= i + lk - lq (a row that sees none, or none but scores of
 * -infinity, answers zeros; one that sees a NaN score is NaN).
 * q bf16 [Tq, H, 192], k_nope [Tk, H, 128], k_rope [Tk, 64], v [Tk, H, 128]
 * and out [Tq, H, 128] by their strides; cu_q, cu_k int32 [B + 1], which do not
 * fall.  Rows of no sequence are left as they were, and keys and values that a
 * row does not see do not reach it, whatever they are.
 * Scores, maxima, sums and outputs are fp32; the softmax weights are rounded
 * to bf16 (2^-8 of the weight) before both the product and their sum.
 * Offsets outside the tensors, or falling ones, raise MOE_DEV_BAD_POSITION and
 * are clamped.
 */
moe_status moe_expanded_attention(const uint16_t* q, const uint16_t* k_nope,
                                  const uint16_t* k_rope, const uint16_t* v,
                                  const int32_t* cu_q, const int32_t* cu_k,
                                  moe_expanded_dims d, uint16_t* out,
                                  int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
