/* moe.h — C ABI of the MI355X (gfx950) DeepSeekMoE layer-forward library (libmoe.so).
 *
 * The layer is the one of the page "DeepSeek-V3 技術報告"
 * (xyznot.com/zh-tw/paper/2412.19437), section 方法 §2:
 *
 *   h'_t = u_t + sum_{i<=N_s} FFN^(s)_i(u_t) + sum_{i<=N_r} g_{i,t} FFN^(r)_i(u_t)
 *   s_{i,t} = Sigmoid(u_t^T e_i)
 *   g'_{i,t} = s_{i,t} if s_{i,t} + b_i is among the K_r largest {s_{j,t} + b_j}, else 0
 *   g_{i,t} = g'_{i,t} / sum_j g'_{j,t}
 *   end of step: b_i <- b_i - gamma if expert i is overloaded, + gamma if underloaded
 *
 * with every expert FFN a bias-free SwiGLU, FFN(x) = (SiLU(x Wg^T) * (x Wu^T)) Wd^T,
 * and, for MOE_DTYPE_FP8_B128, the FP8 scheme of the same page's 核心概念 list:
 * E4M3 values with one fp32 scale per 1x128 activation tile and per 128x128
 * weight block, accumulated in fp32.
 *
 * Conventions shared by every entry point:
 *  - Every tensor pointer is DEVICE memory owned by the caller.  The library
 *    never allocates device memory and never synchronises: work is enqueued on
 *    `stream` (which must belong to the calling thread's current device) and
 *    results are valid once the stream has completed it.  Scratch memory is the
 *    caller's workspace.  Between calls the library keeps only per-device facts
 *    set up once per device (its CU count and the kernels' LDS limits), under
 *    std::call_once / a mutex, so host threads may call it concurrently.
 *  - Arguments are validated on the host before anything is enqueued; on an
 *    error nothing is launched and the outputs are untouched.  A failed launch
 *    returns MOE_ERR_HIP.  No C++ exception crosses the ABI.
 *  - Row-major layouts throughout.  Expert weights are stored like
 *    nn.Linear weights, [out_features, in_features]:
 *        gate/up projections  [N, I, d]   (row n of expert e = output feature n)
 *        down projection      [N, d, I]
 *  - Results are bit-reproducible run to run (no floating-point atomics).
 *  - Calls that share a workspace must be ordered on one stream.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* null pointer, negative size, K_r > N_r, ... */
  MOE_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels handle (see each call) */
  MOE_ERR_WORKSPACE = 3,    /* workspace smaller than moe_workspace_size() */
  MOE_ERR_HIP = 4           /* a HIP launch or runtime call failed */
} moe_status;

typedef enum moe_dtype {
  MOE_DTYPE_F32 = 0,       /* u, weights, out: fp32 */
  MOE_DTYPE_BF16 = 1,      /* u, weights, out: bf16 */
  MOE_DTYPE_FP8_B128 = 2   /* u, out: bf16; weights E4M3 codes + fp32 128x128 block scales */
} moe_dtype;

/* Layer shape.  Limits: tokens >= 0; 1 <= n_routed <= 512; 1 <= top_k <= min(n_routed, 32);
 * 0 <= n_shared <= 64; hidden, inter >= 1 and multiples of 8 (bf16) or of 128 (fp8);
 * tokens * top_k < 2^31; fp8 also tokens * hidden, (padded permuted rows) * inter and
 * hidden * inter below 2^32 (the FP8 GEMMs' 32-bit byte offsets).  Outside them the calls
 * return MOE_ERR_INVALID_ARG (malformed) or MOE_ERR_UNSUPPORTED. */
typedef struct moe_shape {
  int32_t tokens;    /* T   */
  int32_t hidden;    /* d   */
  int32_t n_routed;  /* N_r */
  int32_t top_k;     /* K_r */
  int32_t n_shared;  /* N_s */
  int32_t inter;     /* I   */
  int32_t dtype;     /* moe_dtype */
} moe_shape;

/* Expert weights.  Element type: fp32 (F32), bf16 (BF16) or E4M3FN bytes (FP8_B128).
 * The shared pointers may be NULL when n_shared == 0.  The *_scale pointers are
 * read only for FP8_B128: one fp32 per 128x128 block of each stored matrix,
 * laid out [N, out/128, in/128] (as written by moe_quantize_weights). */
typedef struct moe_weights {
  const void* w_gate;       /* [N_r, I, d] */
  const void* w_up;         /* [N_r, I, d] */
  const void* w_down;       /* [N_r, d, I] */
  const void* sh_gate;      /* [N_s, I, d] */
  const void* sh_up;        /* [N_s, I, d] */
  const void* sh_down;      /* [N_s, d, I] */
  const float* w_gate_scale;   /* [N_r, I/128, d/128] */
  const float* w_up_scale;     /* [N_r, I/128, d/128] */
  const float* w_down_scale;   /* [N_r, d/128, I/128] */
  const float* sh_gate_scale;  /* [N_s, I/128, d/128] */
  const float* sh_up_scale;    /* [N_s, I/128, d/128] */
  const float* sh_down_scale;  /* [N_s, d/128, I/128] */
} moe_weights;

/* Number of stage boundaries moe_forward_profiled() records events at. */
#define MOE_FORWARD_EVENTS 6

/* Bytes of device workspace that moe_route and moe_forward need for `shape`
 * (one buffer serves both).  Never fails for a shape within the limits above. */
moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes);

/* Routing: sigmoid affinities, biased top-K_r selection, normalised gates, per-expert load
 * (方法 §2: the s_{i,t} and g'_{i,t} equations).
 *   u          [T, d]     fp32 (F32) or bf16 (BF16, FP8_B128)
 *   centroids  [N_r, d]   fp32 (e_i)
 *   bias       [N_r]      fp32 (b_i; only ranks experts, never enters a gate)
 *   topk_idx   [T, K_r]   int32 out: selected experts ordered by s+b descending, ties to the
 *                         lower index; NaN scores rank below every number
 *   topk_gate  [T, K_r]   fp32 out: s_{i,t} / sum of the selected s, in topk_idx order
 *   expert_load[N_r]      int32 out: number of (token, slot) picks of each expert
 * Affinities are computed fp32-accurately (the contraction over d is exact products
 * accumulated in fp32).  T == 0 writes expert_load = 0 and launches nothing else. */
moe_status moe_route(const moe_shape* shape, const void* u, const float* centroids,
                     const float* bias, int32_t* topk_idx, float* topk_gate,
                     int32_t* expert_load, void* workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* Size of the fixed device array that holds moe_route_noalloc's scratch (one per GPU). */
#define MOE_ROUTE_NOALLOC_SCRATCH_BYTES (64u << 20)

/* moe_route without a workspace, for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation).  Same arguments,
 * outputs, errors and results as moe_route, bit for bit.  The routing's scratch lives in a
 * file-scope device array of MOE_ROUTE_NOALLOC_SCRATCH_BYTES (64 MiB): each GPU the library
 * runs on holds its own copy from the library's load until the process ends, and its address is
 * looked up once per device on the first call there.  The call allocates nothing.
 *   - A shape whose routing scratch exceeds the array (at d=7168, N_r=256 that is T > 52330)
 *     returns MOE_ERR_WORKSPACE before anything touches the GPU.
 *   - `stream` must belong to the calling thread's current device (else MOE_ERR_INVALID_ARG).
 *   - Every call on one GPU shares that GPU's array: calls that overlap on one GPU (two streams,
 *     two host threads, or a call overlapping a graph replay that contains one) race on it and
 *     must be ordered by the caller.  Nothing in the array needs clearing between calls. */
moe_status moe_route_noalloc(const moe_shape* shape, const void* u, const float* centroids,
                             const float* bias, int32_t* topk_idx, float* topk_gate,
                             int32_t* expert_load, hipStream_t stream);

/* moe_route with a per-token group limit.  The page's cross-node all-to-all section limits
 * every token to experts on at most 4 nodes and prints no rule for choosing them; the reading
 * here: the N_r experts form n_groups equal contiguous groups (expert i is in group
 * i / (N_r / n_groups)), a group's score is the highest s+b among its experts, the
 * topk_groups groups with the highest scores (ties to the lower group index; NaN below every
 * number) stay eligible, and the K_r experts are then picked among the eligible ones exactly as
 * in moe_route.  Gates and expert_load as in moe_route.  n_groups == 1 or
 * topk_groups == n_groups is moe_route.
 * Errors: MOE_ERR_INVALID_ARG unless 1 <= topk_groups <= n_groups <= 64, N_r % n_groups == 0 and
 * topk_groups * N_r / n_groups >= K_r (plus moe_route's checks); nothing is launched then. */
moe_status moe_route_grouped(const moe_shape* shape, int32_t n_groups, int32_t topk_groups,
                             const void* u, const float* centroids, const float* bias,
                             int32_t* topk_idx, float* topk_gate, int32_t* expert_load,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* moe_route plus the sequence-wise balance statistic.  The page (方法 §2, last paragraph) adds
 * a tiny sequence-level balance loss (alpha = 0.0001) to the bias rule and prints no formula;
 * the reading here: for each of the T / seq_len sequences of consecutive tokens,
 *   f_i = N_r / (K_r seq_len) * (the sequence's picks of expert i),
 *   P_i = mean over the sequence's tokens of s_{i,t} / sum_j s_{j,t},
 *   seq_loss[q] = alpha * sum_i f_i P_i          (fp32 out, [T / seq_len]).
 * Routing outputs as in moe_route.  Errors: MOE_ERR_INVALID_ARG unless 1 <= seq_len <= 16384
 * divides T and seq_loss is non-null (plus moe_route's checks); nothing is launched then. */
moe_status moe_route_balance(const moe_shape* shape, int32_t seq_len, float alpha, const void* u,
                             const float* centroids, const float* bias, int32_t* topk_idx,
                             float* topk_gate, int32_t* expert_load, float* seq_loss,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Expert half of the layer (方法 §2, the h'_t equation): permutes tokens into per-expert
 * segments, runs every routed expert on its tokens and every shared expert on all tokens
 * (grouped SwiGLU GEMMs), and combines out_t = u_t + sum_s FFN_s(u_t) + sum_k gate FFN(u_t).
 *   u          [T, d]     fp32 (F32) or bf16 (BF16, FP8_B128; FP8 quantises it per 1x128 tile)
 *   topk_idx   [T, K_r]   int32 from moe_route (entries outside [0, N_r) are ignored)
 *   topk_gate  [T, K_r]   fp32 from moe_route
 *   out        [T, d]     fp32 (F32) or bf16 (BF16, FP8_B128); may not alias u
 * FP8_B128 needs d % 128 == 0 and I % 128 == 0 (else MOE_ERR_UNSUPPORTED). */
moe_status moe_forward(const moe_shape* shape, const void* u, const moe_weights* weights,
                       const int32_t* topk_idx, const float* topk_gate, void* out,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* moe_forward, recording events[0..MOE_FORWARD_EVENTS) on `stream` at its stage boundaries:
 * [0] start, [1] after the token->expert permutation, [2] after activation quantisation
 * (FP8 only; else right after [1]), [3] after the gate/up GEMM with SwiGLU, [4] after the
 * down GEMM, [5] after the combine.  events must hold MOE_FORWARD_EVENTS created events
 * (hipEvent_t); they are recorded, never created or destroyed, by the library. */
moe_status moe_forward_profiled(const moe_shape* shape, const void* u, const moe_weights* weights,
                                const int32_t* topk_idx, const float* topk_gate, void* out,
                                void* workspace, size_t workspace_bytes, hipStream_t stream,
                                hipEvent_t* events, int32_t n_events);

/* Weight gradients written by moe_backward: bf16, same layouts as the weights
 * (gate/up [N, I, d], down [N, d, I], N = N_r or N_s).  Owned by the caller. */
typedef struct {
  void* w_gate;
  void* w_up;
  void* w_down;
  void* sh_gate;
  void* sh_up;
  void* sh_down;
} moe_weight_grads;

/* Bytes of device workspace moe_backward needs for `shape` (BF16 or FP8_B128; d and I multiples
 * of 128).  MOE_ERR_UNSUPPORTED for other shapes. */
moe_status moe_backward_workspace_size(const moe_shape* shape, size_t* bytes);

/* Layer backward (方法 §2, the h'_t, s_{i,t} and g'_{i,t} equations): gradients of
 * L = <dout, h'> with the routing (topk_idx) held fixed — the Topk is piecewise constant — and
 * none for the bias, which never enters a gate.  With g_k = s_k / S (S = sum of the selected
 * s) the gate gradient flows through the unbiased s into u and the centroids.
 *   u, centroids, weights, topk_idx, topk_gate   as given to moe_route / moe_forward
 *   dout        [T, d]   bf16 dL/dh'
 *   du          [T, d]   bf16 out: dL/du (residual + every expert's input gradient + router term)
 *   d_centroids [N_r, d] fp32 out (rows of experts no token picked are zero)
 *   dw          bf16 out, every routed and shared expert's gate/up/down gradient (zero for
 *               experts no token picked)
 * FP8_B128 (section 方法, FP8 Mixed Precision Training: the forward and both backward GEMM
 * kinds in FP8; 核心概念, FP8 item: E4M3, 1x128 activation tiles, 128x128 weight blocks): the
 * weights are the E4M3 codes and block scales of moe_forward; every product runs on E4M3
 * operands with fp32 accumulation: dout and u in 1x128 tiles along d, [dA dB] along 2I, the
 * weights transposed per 128x128 block (codes and scales carry over), and for the weight
 * gradients the transposed activations in runs of 128 of each expert's rows (token order);
 * quantised from bf16 (u, dout, H, dA, dB) or fp32 (gate * dout).  Gates, router and residual
 * stay unquantised, and every output is bf16 / fp32 as for BF16.
 * Errors: MOE_ERR_UNSUPPORTED unless dtype is BF16 or FP8_B128, d % 128 == 0, I % 128 == 0;
 * MOE_ERR_INVALID_ARG for a null pointer (FP8_B128: also a null weight scale) or du aliasing
 * u or dout; MOE_ERR_WORKSPACE if workspace_bytes < moe_backward_workspace_size.  Nothing is
 * launched on an error. */
moe_status moe_backward(const moe_shape* shape, const void* u, const float* centroids,
                        const moe_weights* weights, const int32_t* topk_idx, const float* topk_gate,
                        const void* dout, void* du, float* d_centroids, const moe_weight_grads* dw,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Saved-input training pair (BF16 and FP8_B128).  The backward's gate/up step needs the SwiGLU inputs
 * a = x W_gate^T and b = x W_up^T of every (token, expert) row (方法 §2, the h'_t equation: the
 * expert FFN is SwiGLU).  moe_backward recomputes them with a second gate/up product; this pair
 * keeps them from the forward instead, trading [max_rows, 2I] bf16 of device memory for that
 * product.  The results equal moe_forward / moe_backward up to the rounding of a and b to bf16
 * before the backward's SwiGLU derivative (FP8_B128: a and b of the FP8 forward product, kept
 * in bf16; the backward's other FP8 products are unchanged).
 *
 * moe_saved_inputs_size: bytes of the saved buffer for `shape` (bf16 [max_rows, 2I] for both
 * dtypes).  Errors as for moe_backward_workspace_size. */
moe_status moe_saved_inputs_size(const moe_shape* shape, size_t* bytes);

/* moe_forward (same arguments, same workspace, same out) that also writes the SwiGLU inputs
 * [a b] of every row of the permuted token->expert layout to `saved` (bf16, row r at
 * saved + r * 2I: a then b; the layout is private to the library and fixed by topk_idx).  The
 * caller owns `saved` and passes it, unchanged, with the same topk_idx to moe_backward_saved.
 * Errors: those of moe_forward and moe_backward_workspace_size (so MOE_ERR_UNSUPPORTED for
 * F32); MOE_ERR_INVALID_ARG for a null `saved` (T > 0) or one aliasing u or out;
 * MOE_ERR_WORKSPACE if saved_bytes < moe_saved_inputs_size. */
moe_status moe_forward_train(const moe_shape* shape, const void* u, const moe_weights* weights,
                             const int32_t* topk_idx, const float* topk_gate, void* out, void* saved,
                             size_t saved_bytes, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* moe_backward (same arguments and outputs, same workspace) reading the SwiGLU inputs that
 * moe_forward_train saved for the same shape, weights and topk_idx in place of recomputing
 * them.  Errors: those of moe_backward; MOE_ERR_INVALID_ARG for a null `saved` or one aliasing du; MOE_ERR_WORKSPACE if
 * saved_bytes < moe_saved_inputs_size. */
moe_status moe_backward_saved(const moe_shape* shape, const void* u, const float* centroids,
                              const moe_weights* weights, const int32_t* topk_idx, const float* topk_gate,
                              const void* saved, size_t saved_bytes, const void* dout, void* du,
                              float* d_centroids, const moe_weight_grads* dw, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* Auxiliary-loss-free bias update (方法 §2, last paragraph), in place on bias[N_r] (fp32):
 * expert i is overloaded when load_i * N_r > total_assignments (= T * K_r, i.e. above the
 * step mean), underloaded when below; b_i <- b_i - gamma resp. b_i + gamma as one fp32 add;
 * equal to the mean: unchanged. */
moe_status moe_update_bias(int32_t n_routed, int64_t total_assignments, const int32_t* expert_load,
                           float* bias, float gamma, hipStream_t stream);

/* One-time weight preparation for moe_forward and moe_backward (untimed, outside the hot path).
 *   logical       the layer's weights as stored: bf16 for BF16 and FP8_B128, fp32 for F32
 *                 (scale pointers ignored; shared pointers may be NULL when n_shared == 0)
 *   packed        device buffer of *packed_bytes bytes owned by the caller (FP8_B128 only)
 *   prepared      out: the moe_weights to pass to moe_forward / moe_backward
 * With prepared == NULL the call only writes to *packed_bytes the size `packed` needs (0 for BF16
 * and F32) and touches nothing else.  BF16 and F32: the kernels read the weights as stored, so
 * `prepared` receives the logical pointers and nothing is launched.  FP8_B128 (核心概念, FP8 item:
 * E4M3 weights with one fp32 scale per 128x128 block): every stack is quantised as by
 * moe_quantize_weights into `packed` (the six code stacks, then the six scale stacks, each
 * 256-byte aligned), and `prepared` points into it.  `packed` must stay allocated while
 * `prepared` is in use and may not overlap the logical weights.
 * Errors: check_shape's; MOE_ERR_INVALID_ARG for a null logical, packed_bytes, needed weight
 * pointer or (FP8_B128) packed; MOE_ERR_WORKSPACE if *packed_bytes is too small.  Nothing is
 * launched on an error. */
moe_status moe_prepare_weights(const moe_shape* shape, const moe_weights* logical, void* packed,
                               size_t* packed_bytes, moe_weights* prepared, hipStream_t stream);

/* FP8 weight preparation (核心概念, FP8 item: 128x128 block scaling): quantises a stack of
 * n_mats bf16 matrices [rows, cols] into E4M3FN codes [n_mats, rows, cols] and fp32 scales
 * [n_mats, ceil(rows/128), ceil(cols/128)]: scale = amax/448 (1 for an all-zero block), code =
 * round-to-nearest-even E4M3FN of fp32(x / scale), saturating at 448.
 * rows and cols must be multiples of 16; the last blocks may be smaller than 128 (moe_matmul_fp8
 * takes them, the layer needs whole ones). */
moe_status moe_quantize_weights(int32_t n_mats, int32_t rows, int32_t cols, const void* w_bf16,
                                uint8_t* codes, float* scales, hipStream_t stream);

/* FP8 activation quantisation (核心概念, FP8 item: 1x128 tile scaling), the step moe_forward
 * runs on u for FP8_B128: x [rows, cols] bf16 -> codes [rows, cols] E4M3FN and scales
 * [rows, cols/128] fp32, same rounding rule as moe_quantize_weights.  cols % 128 == 0. */
moe_status moe_quantize_act(int32_t rows, int32_t cols, const void* x_bf16, uint8_t* codes,
                            float* scales, hipStream_t stream);

/* ---- Routing from given logits -------------------------------------------------------------
 * For callers whose router is not the sigmoid of u^T e_i above (a softmax router, a learned or
 * quantised product): the selection and its gradient, on logits the caller computed. */
typedef enum moe_score {
  MOE_SCORE_SIGMOID = 0,    /* s_i = 1 / (1 + exp(-l_i)) */
  MOE_SCORE_SOFTMAX = 1     /* s_i = exp(l_i) / sum_j exp(l_j) */
} moe_score;

typedef enum moe_group_score {
  MOE_GROUP_MAX = 0,        /* a group's score: its largest s+b */
  MOE_GROUP_TOP2 = 1        /* the sum of its two largest s+b (of its only one, if it has one) */
} moe_group_score;

/* Limits: tokens >= 0; 1 <= n_routed <= 512; 1 <= top_k <= min(n_routed, 32);
 * 1 <= topk_groups <= n_groups <= 64, n_routed % n_groups == 0 and
 * topk_groups * n_routed / n_groups >= top_k; tokens * top_k < 2^31; scale finite. */
typedef struct moe_gate_config {
  int32_t tokens;        /* T */
  int32_t n_routed;      /* N */
  int32_t top_k;         /* K */
  int32_t logits_dtype;  /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 (logits and their gradient) */
  int32_t score;         /* moe_score */
  int32_t n_groups;      /* equal groups of neighbouring experts; 1: no limit */
  int32_t topk_groups;   /* groups that stay eligible for a token */
  int32_t group_score;   /* moe_group_score */
  int32_t renormalize;   /* non-zero: gates divided by the sum of the selected s */
  float scale;           /* factor of every gate */
  int64_t logits_ld;     /* elements between rows of logits; 0: n_routed */
} moe_gate_config;

/* Bytes of device workspace that moe_gate needs for `config` (0 without expert_load).  For these tokens: fewer may need more. */
moe_status moe_gate_workspace_size(const moe_gate_config* config, size_t* bytes);

/* Selection and gates.
 *   logits      [T, N]  fp32 or bf16, rows logits_ld apart
 *   bias        [N]     fp32, or NULL; only ranks experts
 *   topk_idx    [T, K]  int32 out: experts by s+b descending, ties to the lower index; -1 where no
 *                       eligible expert is left (moe_forward skips such entries)
 *   topk_gate   [T, K]  fp32 out: scale * s (over the sum of the selected s if renormalize); 0 for -1
 *   expert_load [N]     int32 out, or NULL: picks of each expert
 * An expert whose logit or bias is -inf is not eligible; a token whose logits are all -inf (a
 * padding row) picks nothing.  A NaN score ranks below every number, and its gates are NaN.  Scores,
 * sums and gates are fp32, scores and gates below 2^-126 may be 0.  Only a softmax without a bias (or
 * with entries +0 and -inf alone) ranks experts and groups by the logits, so that scores too small for
 * fp32 keep their order; other keys that are equal in fp32 count as ties.  T == 0 writes
 * expert_load = 0.
 * Errors: MOE_ERR_INVALID_ARG outside the limits (n_routed > 512, top_k > 32 or tokens * top_k >= 2^31:
 * MOE_ERR_UNSUPPORTED) or for a null pointer; MOE_ERR_WORKSPACE if workspace_bytes is too small. */
moe_status moe_gate(const moe_gate_config* config, const void* logits, const float* bias, int32_t* topk_idx,
                    float* topk_gate, int32_t* expert_load, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* Gradient of moe_gate's gates with the selection held fixed.
 *   logits, topk_idx   as given to and written by moe_gate (entries outside [0, N) are skipped; the
 *                      others of a row are distinct)
 *   d_gate   [T, K]    fp32 dL/dgate
 *   d_logits [T, N]    out, every element written: fp32 or bf16 (rounded once), rows d_logits_ld apart
 *                      (0: n_routed); may not alias logits
 * The bias gets no gradient.  Errors as moe_gate. */
moe_status moe_gate_backward(const moe_gate_config* config, const void* logits, const int32_t* topk_idx,
                             const float* d_gate, void* d_logits, int64_t d_logits_ld, hipStream_t stream);

/* ---- FP8 products ---------------------------------------------------------------------------
 * The dense layers beside the experts (a dense FFN, a projection), in the experts' FP8 scheme: E4M3
 * codes with one fp32 scale per 1x128 run or 128x128 block, accumulated in fp32 (bf16 outputs: by
 * the FP8 matrix instruction, whose sums of eight products keep 13 bits below the largest; fp32
 * outputs: on the codes widened to f16, exact products in fp32). */
typedef enum moe_fp8_form {
  MOE_FP8_FORWARD = 0,      /* out = a b^T: a [m, k] in 1x128 runs, b [n, k] in 128x128 blocks */
  MOE_FP8_INPUT_GRAD = 1,   /* out = a b:   a [m, k] in 1x128 runs, b [k, n] in 128x128 blocks */
  MOE_FP8_WEIGHT_GRAD = 2   /* out = a b^T: a [m, k] and b [n, k], both in 1x128 runs */
} moe_fp8_form;

/* Limits: m, n, k >= 0, n a multiple of 16, k a multiple of 128; leading dimensions at least the row
 * length, lda and ldb multiples of 16 below 2^24, ldo a multiple of 4. */
typedef struct moe_matmul_shape {
  int32_t m, n, k;
  int32_t form;         /* moe_fp8_form */
  int32_t out_dtype;    /* MOE_DTYPE_BF16 or MOE_DTYPE_F32 */
  int32_t accumulate;   /* non-zero: out += the product (gradients of several micro-batches) */
  int64_t lda, ldb;     /* elements between rows of a and b; 0: dense */
  int64_t ldo;          /* elements between rows of out; 0: n */
} moe_matmul_shape;

/* Bytes of device workspace that moe_matmul_fp8 needs for `shape`.  For this one: a smaller one may need more. */
moe_status moe_matmul_fp8_workspace_size(const moe_matmul_shape* shape, size_t* bytes);

/* out = the product of `shape`'s form.
 *   a, b      E4M3FN codes (16-byte aligned)
 *   a_scale   fp32 [m, k/128] (moe_quantize_act, moe_quantize_act_t)
 *   b_scale   fp32 [ceil(n/128), k/128] forward, [k/128, ceil(n/128)] input gradient (both as
 *             moe_quantize_weights writes them for the stored matrix), [n, k/128] weight gradient
 *   out       [m, n] bf16 or fp32 (16-byte aligned); aliases no input
 * k == 0 gives zeros.  Errors: MOE_ERR_INVALID_ARG (unknown form or type, a negative size, a leading
 * dimension below the row length, a null or misaligned pointer, out aliasing an operand),
 * MOE_ERR_UNSUPPORTED (other limits), MOE_ERR_WORKSPACE. */
moe_status moe_matmul_fp8(const moe_matmul_shape* shape, const uint8_t* a, const float* a_scale, const uint8_t* b,
                          const float* b_scale, void* out, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* The operands of a weight gradient: x [rows, cols] bf16 transposed and quantised in runs of 128 rows:
 *   codes  [cols, R]      E4M3FN, R = rows rounded up to 128, rows past the last as zeros
 *   scales [cols, R/128]  fp32
 * scale = amax * fp32(1/448) (1 for a run of zeros), code = round-to-nearest-even E4M3FN of
 * fp32(x / scale), saturating at 448.  moe_quantize_act's scale is the quotient amax/448: for the
 * transposed matrix its scales are up to one unit in the last place apart, and where they are a value
 * near a rounding tie may have the neighbouring code.  cols must be a multiple of 8 (MOE_ERR_UNSUPPORTED), x and codes
 * 16-byte aligned (MOE_ERR_INVALID_ARG). */
moe_status moe_quantize_act_t(int32_t rows, int32_t cols, const void* x_bf16, uint8_t* codes, float* scales,
                              hipStream_t stream);

/* ---- SwiGLU with its inputs kept in 8 bits --------------------------------------------------
 * moe_forward_train keeps a and b in bf16; here a run of 128 values keeps one fp32 scale
 * amax * fp32(1/127) (1 for a run of zeros) and 8-bit integers round(x / scale), half the memory.  A run that holds an
 * infinity or NaN keeps the scale NaN.
 *   ab       [rows, 2I]      bf16: a then b
 *   h        [rows, I]       bf16 out: a sigmoid(a) b; may be NULL
 *   saved    [rows, 2I]      int8 out
 *   scales   [rows, 2I/128]  fp32 out
 * inter (I) must be a multiple of 128 (MOE_ERR_UNSUPPORTED); ab, h and saved 16-byte aligned, none in
 * place of another (MOE_ERR_INVALID_ARG), here and below. */
moe_status moe_swiglu_forward8(int32_t rows, int32_t inter, const void* ab, void* h, int8_t* saved, float* scales,
                               hipStream_t stream);

/* The backward pass from what moe_swiglu_forward8 kept: with a~, b~ = saved * scale and sg = sigmoid(a~),
 *   d_ab [rows, 2I] bf16 out: dh b~ sg (1 + a~ (1 - sg)), then dh a~ sg
 *   h    [rows, I]  bf16 out: a~ sg b~ (the operand of the next layer's weight gradient); may be NULL
 * for dh [rows, I] bf16. */
moe_status moe_swiglu_backward8(int32_t rows, int32_t inter, const void* dh, const int8_t* saved, const float* scales,
                                void* d_ab, void* h, hipStream_t stream);

/* ---- The layer under a router of the caller's own, with its SwiGLU inputs kept in 8 bits ------
 * moe_gate picks and weighs, moe_forward_train8 runs the experts, moe_backward_gates returns the
 * gates' gradients for moe_gate_backward.  BF16 and FP8_B128, shapes as moe_backward.
 *
 * moe_saved8_size: bytes of the buffer that moe_forward_train8 writes (about half of
 * moe_saved_inputs_size: int8 codes and a scale per 128 values of every row's a and b, as
 * moe_swiglu_forward8 keeps them).  moe_train8_workspace_size: bytes of its workspace.  The gate/up
 * products leave a and b in bf16 there, and a second pass packs them: where 2 * inter > hidden they
 * do not fit into the place of the down products, and the workspace is larger than
 * moe_workspace_size by moe_saved_inputs_size. */
moe_status moe_saved8_size(const moe_shape* shape, size_t* bytes);
moe_status moe_train8_workspace_size(const moe_shape* shape, size_t* bytes);

/* moe_forward_train (same output, to the bit) that keeps a and b in 8 bits in `saved8`, for
 * moe_backward_gates with the same topk_idx.  Errors as moe_forward_train. */
moe_status moe_forward_train8(const moe_shape* shape, const void* u, const moe_weights* weights,
                              const int32_t* topk_idx, const float* topk_gate, void* out, void* saved8,
                              size_t saved8_bytes, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* moe_backward without its router: the gates are inputs, and their gradients come back.
 *   saved8   from moe_forward_train8, or NULL (a and b are computed again, as in moe_backward)
 *   du       [T, d]   bf16 out: the residual and the experts' input gradients; the router's term
 *                     (d_logits times the caller's router weights) is the caller's to add
 *   d_gate   [T, K_r] fp32 out: <dout, FFN_k(u)>, 0 where topk_idx is outside [0, N_r)
 *   dw       as in moe_backward
 * Workspace: moe_backward_workspace_size.  Errors as moe_backward; MOE_ERR_INVALID_ARG for a null
 * d_gate (T > 0); MOE_ERR_WORKSPACE if saved8_bytes < moe_saved8_size. */
moe_status moe_backward_gates(const moe_shape* shape, const void* u, const moe_weights* weights,
                              const int32_t* topk_idx, const float* topk_gate, const void* saved8,
                              size_t saved8_bytes, const void* dout, void* du, float* d_gate,
                              const moe_weight_grads* dw, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* ---- The residual's addition and the norm before a layer -------------------------------------
 * h = x + residual, and its root-mean-square norm y = h / sqrt(mean(h^2) + eps) * weight, as bf16 or
 * fp32 and as the E4M3 codes that moe_matmul_fp8 takes. */
typedef struct moe_norm_shape {
  int32_t rows, cols;   /* rows >= 0; cols >= 8, a multiple of 8 (of 128 with codes), at most 32768 */
  int32_t dtype;        /* MOE_DTYPE_F32 or MOE_DTYPE_BF16: x, residual, sum, y and their gradients */
  float eps;            /* >= 0, finite */
  int64_t x_ld;         /* elements between rows of x, residual, sum, h, d_sum and d_x; 0: cols */
  int64_t y_ld;         /* elements between rows of y and d_y; 0: cols (both multiples of 8) */
} moe_norm_shape;

/* Bytes of device workspace that moe_norm_backward needs for `shape` with d_weight (0 for few rows; moe_norm_forward needs
 * none), or for one that differs from it in having fewer rows. */
moe_status moe_norm_workspace_size(const moe_norm_shape* shape, size_t* bytes);

/*   x         [rows, cols]
 *   residual  [rows, cols], or NULL (h = x)
 *   weight    [cols]  fp32
 *   sum       [rows, cols] out: h, rounded to the type, which is what the norm is taken of; may be x or
 *             residual itself; NULL: not kept.  NULL without a residual
 *   y         [rows, cols] out, or NULL
 *   codes     [rows, cols] out: E4M3FN, and scales [rows, cols/128] fp32: scale = amax/448 of the run
 *             of 128 (1 where that is 0), code = round-to-nearest-even E4M3FN of fp32(y / scale), from
 *             y before its rounding to the type; both or neither NULL.  y or codes is needed
 *   rstd      [rows] fp32 out: 1 / sqrt(mean(h^2) + eps), for moe_norm_backward; may be NULL
 * Squares and sums are fp32: a row whose sum of squares passes 3.4e38 has rstd 0; under eps = 0 a row of
 * zeros is NaN, and one whose squares are all 0 in fp32 (values below 2.6e-23) infinite.  A row's results do not depend on the other rows.  No buffer is another's, but for sum as above;
 * x_ld and y_ld are multiples of 8, and all pointers multiples of 16 (scales, rstd and d_weight: of 4).
 * Errors: MOE_ERR_INVALID_ARG (null or misaligned pointers, a negative size, ld < cols, buffers in
 * place of one another), MOE_ERR_UNSUPPORTED (other limits). */
moe_status moe_norm_forward(const moe_norm_shape* shape, const void* x, const void* residual, const float* weight,
                            void* sum, void* y, uint8_t* codes, float* scales, float* rstd, hipStream_t stream);

/* The gradient, from h (sum, or x without a residual) and rstd of moe_norm_forward.  With u = h rstd and
 * g = d_y weight,
 *   d_x       [rows, cols] out: rstd (g - u mean(g u)) + d_sum, the gradient of x and of residual alike;
 *             may be d_sum itself
 *   d_weight  [cols] fp32 out: the rows' sum of d_y u; NULL: not computed, and no workspace needed
 *   d_y       [rows, cols]; d_sum [rows, cols]: the gradient that reaches `sum` from behind, or NULL
 * rows == 0 gives d_weight zeros.  Errors as moe_norm_forward, MOE_ERR_WORKSPACE. */
moe_status moe_norm_backward(const moe_norm_shape* shape, const void* d_y, const void* d_sum, const void* h,
                             const float* weight, const float* rstd, void* d_x, float* d_weight, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/* ---- Balance loss of a router --------------------------------------------------------------------
 * For callers who route with moe_gate or by themselves: for each sequence of L tokens,
 *   p_t = softmax(l_t), or s_t / sum s_t with the sigmoid;   n_i = picks of expert i
 *   loss = alpha sum_i (N n_i / (K L)) (sum_t p_{t,i} / L)
 * (moe_route_balance's statistic), and its gradient with the picks held fixed.  A pick is an entry
 * of topk_idx in [0, N); a token without one is padding: it is not in L and has no gradient. */
typedef struct moe_balance_config {
  int32_t tokens;        /* T >= 0 */
  int32_t n_routed;      /* N: 1 to 512 */
  int32_t top_k;         /* K: 1 to min(N, 32); tokens * top_k < 2^31 */
  int32_t logits_dtype;  /* MOE_DTYPE_F32 or MOE_DTYPE_BF16 (logits and their gradient) */
  int32_t score;         /* moe_score */
  int32_t n_seqs;        /* S: 1 to 2^24 */
  float alpha;           /* finite */
  int64_t logits_ld;     /* elements between rows of logits; 0: n_routed */
} moe_balance_config;

/* Bytes of device workspace that moe_balance_loss needs for `config` (0 for few tokens), or for one that differs from it in
 * having fewer tokens or sequences. */
moe_status moe_balance_workspace_size(const moe_balance_config* config, size_t* bytes);

/*   logits      [T, N]  fp32 or bf16 (an expert at -inf has p = 0)
 *   topk_idx    [T, K]  int32
 *   seq_start   [S + 1] int32: sequence s is the tokens [seq_start[s], seq_start[s+1]), ascending, within
 *               [0, T], empty ones allowed; tokens outside belong to no sequence.  NULL: one sequence,
 *               all tokens (n_seqs == 1)
 *   loss        [S]     fp32 out (0 for a sequence without tokens)
 *   counts      [S, N]  int32 out: n_i
 *   seq_tokens  [S]     int32 out: L
 *   prob_sum    [S, N]  fp32 out, or NULL: sum_t p_{t,i}.  With counts, seq_tokens and prob_sum added up
 *               over the ranks of a job, the loss of the whole batch is the formula above, and
 *               moe_balance_backward takes the sums
 * Errors: MOE_ERR_INVALID_ARG outside the limits (n_routed > 512, top_k > 32, n_seqs > 2^24 or tokens * top_k >= 2^31:
 * MOE_ERR_UNSUPPORTED), for a null pointer or an output or the workspace in place of another buffer;
 * MOE_ERR_WORKSPACE. */
moe_status moe_balance_loss(const moe_balance_config* config, const void* logits, const int32_t* topk_idx,
                            const int32_t* seq_start, float* loss, int32_t* counts, int32_t* seq_tokens, float* prob_sum,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The gradient with respect to the logits:
 *   logits, topk_idx, seq_start, counts, seq_tokens   as above
 *   d_loss    [S]    fp32 dL/dloss
 *   d_logits  [T, N] out, rows d_logits_ld apart (0: n_routed): fp32 or bf16 (rounded once).  accumulate
 *             zero: every element written; non-zero: added to what is there (moe_gate_backward's), and rows without a
 *             gradient are left as they are.  In place of no input
 * Errors as moe_balance_loss. */
moe_status moe_balance_backward(const moe_balance_config* config, const void* logits, const int32_t* topk_idx,
                                const int32_t* seq_start, const int32_t* counts, const int32_t* seq_tokens,
                                const float* d_loss, void* d_logits, int64_t d_logits_ld, int32_t accumulate,
                                hipStream_t stream);

/* ---- Low-rank adapters of many requests ------------------------------------------------------------
 * Beside a projection that all requests share (moe_matmul_fp8, or a library's): row t belongs to a
 * request whose adapter is e = row_adapter[t], and
 *   out_t = base_t + scale_e B_e (A_e x_t),
 * the contraction over A_e's first ranks[e] rows.  Rows may come in any order; in large batches those of one adapter
 * side by side (prompts) cost least.  For serving: there is no gradient. */
typedef struct moe_adapter_shape {
  int32_t rows;               /* T: 0 to 2^27 - 1 */
  int32_t in_cols, out_cols;  /* 8 to 2^20, multiples of 8 */
  int32_t n_adapters;         /* n >= 1 */
  int32_t rank;               /* r: rows of each A, columns of each B; 8 to 128, a multiple of 8 */
  int32_t out_dtype;          /* MOE_DTYPE_BF16 or MOE_DTYPE_F32: base and out */
  int64_t x_ld, base_ld, out_ld;   /* elements between rows; 0: dense; multiples of 8, x_ld below 2^24 */
} moe_adapter_shape;

/* Bytes of device workspace that moe_adapters needs for `shape`, or for one that differs from it in having fewer rows: a buffer
 * of the largest batch's size serves every smaller one. */
moe_status moe_adapters_workspace_size(const moe_adapter_shape* shape, size_t* bytes);

/*   x            [T, in]     bf16
 *   row_adapter  [T]         int32; outside [0, n): the row has no adapter and out is base, bit for bit
 *   a            [n, r, in]  bf16;   b [n, out, r] bf16
 *   scale        [n]         fp32
 *   ranks        [n]         int32, 0 to r (others: the nearer of the two), what a and b hold from
 *                            there on is not used; NULL: r for all
 *   base         [T, out]    bf16 or fp32, or NULL (zeros); out may be base itself (equal strides)
 *   out          [T, out]    the same type
 * Sums are fp32 and the low-rank values (times the factor) keep 16 bits of their fp32 sums under a bf16 output, 24 under an
 * fp32 one; what of them lies below 2^-133 is lost.  A row's result is its own alone (an infinity or NaN in another row or
 * adapter does not reach it).
 * Errors: MOE_ERR_INVALID_ARG (null pointers, pointers that are not multiples of 16 (row_adapter, scale and
 * ranks: of 4), strides below the row length, out or the workspace in place of another operand),
 * MOE_ERR_UNSUPPORTED (other limits), MOE_ERR_WORKSPACE. */
moe_status moe_adapters(const moe_adapter_shape* shape, const void* x, const int32_t* row_adapter, const void* a,
                        const void* b, const float* scale, const int32_t* ranks, const void* base, void* out,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Static description of a status code (never NULL). */
const char* moe_status_string(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
