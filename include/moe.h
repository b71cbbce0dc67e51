/*
 * moe.h -- C ABI of the single-GPU Mixture-of-Experts feed-forward layer for
 * NVIDIA B200 (sm_100a).
 *
 * The layer is the moe_ffn pseudocode of "Decoding Trillion-Parameter MoE
 * LLMs: Sparse Architecture and Agentic Intelligence", section "Routing:
 * Top-K Experts Plus a Shared Expert":
 *
 *   logits = x Wr^T                                   router GEMM     [T, E]
 *   idx, w = top-k of the scores, renormalised        moe_route       [T, k]
 *   rows of x grouped by expert (dispatch on 1 GPU)   moe_permute     [T*k, d]
 *   h = silu(x W1^T) * (x W3^T);  y = h W2^T          moe_grouped_ffn per expert
 *   out[t] = sum_j w[t,j] y[row(t,j)] + shared(x[t])   moe_combine     [T, d]
 *
 * moe_layer_forward runs all of it on one stream.  Beside the layer: the norms around a
 * block with its gate and residual scale (moe_block_norm), and the experts' products one at
 * a time with their gradients (moe_grouped_gemm, bf16 or 8-bit with block scales).
 *
 * Conventions (all entry points):
 *  - Every pointer argument is caller-owned DEVICE memory unless stated.  The
 *    library allocates nothing and keeps no state between calls; a caller-
 *    provided workspace holds every intermediate.
 *  - Every call is asynchronous on `stream` (stream-ordered), except
 *    moe_workspace_size, moe_status_string and moe_read_device_status.
 *  - Host-side checks run before any launch; a failed check launches nothing
 *    and returns MOE_ERR_INVALID_ARG (null pointer, non-positive size),
 *    MOE_ERR_UNSUPPORTED (k > E, k > 16, E > 1024, d % 128, I % 128, d > 16384,
 *    I > 16384, T*k >= 2^31, n_shared > 8, unsupported dtype combination) or
 *    MOE_ERR_WORKSPACE (workspace too small).  A launch error returns
 *    MOE_ERR_CUDA.
 *  - Faults the device detects (an expert index outside [0, E) fed to
 *    moe_permute; an FP8 block scale that is not a positive normal power of
 *    two; a bounded wait inside a kernel that ran out) are written to
 *    a status word in the first bytes of the workspace, never trapped; read
 *    it with moe_read_device_status.  The workspace must start zeroed once
 *    (moe_reset_device_status) before its first use.
 *  - Matrices are row-major.  Weight matrices are K-major ("nn.Linear"
 *    layout [out_features, in_features]).
 *  - dtypes: activations MOE_BF16, MOE_E4M3 (with fp32 1x128 scales) or
 *    MOE_F32; weights the same family (bf16 weights with bf16 activations,
 *    e4m3 weights + fp32 128x128 block scales with e4m3 activations, f32 with
 *    f32), or MOE_E2M1 (MXFP4) weights with MOE_E4M3 activations; or MOE_BF16
 *    activations with MOE_E4M3 or MOE_E2M1 weights, quantised to e4m3 in the
 *    permutation (see moe_permute).  f32 inputs are rounded to bf16 (nearest
 *    even) on entry; the tensor cores compute in bf16 (or e4m3 / e2m1 x e4m3)
 *    with fp32 accumulation.  The router weights are bf16 for the bf16, e4m3 and
 *    e2m1 families, f32 for f32; the router takes x as given (bf16, or e4m3
 *    dequantised exactly).
 *    FP8 block scales must be positive normal powers of two (exactly what the
 *    tensor cores' UE8M0 scale factors represent); any other scale sets the
 *    device status MOE_ERR_DEVICE_VALUE.  MXFP4 scale bytes are used as given
 *    (code 0xFF, NaN in E8M0, gives undefined results).
 */
#ifndef MOE_B200_H
#define MOE_B200_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,
  MOE_ERR_UNSUPPORTED = 2,
  MOE_ERR_WORKSPACE = 3,
  MOE_ERR_CUDA = 4,
  MOE_ERR_DEVICE_INDEX = 5,   /* device status: an expert index outside [0, E) */
  MOE_ERR_TIMEOUT = 6,        /* device status: a bounded in-kernel wait ran out */
  MOE_ERR_DEVICE_VALUE = 7    /* device status: an FP8 block scale that is not a positive,
                                 normal power of two (the tensor cores take the scale's
                                 exponent only), or (moe_grouped_gemm) two fp32 scales
                                 whose product overflows; the results of that call are not
                                 valid */
} moe_status;

/* Router score function.
 * SOFTMAX: select the k largest logits; gate_j = exp(l_j - max) / sum over the
 *   selected (the "topk_softmax" of the pseudocode).
 * SIGMOID_BIAS: s = sigmoid(l); select the k largest s + sel_bias[e]; gate_j =
 *   s_j / sum over the selected s (the bias steers selection only) -- the
 *   "auxiliary-loss-free bias routing" named by "Chapter 7: Serving Mega MoE
 *   at scale", roadmap item "Architectural Foundations of Trillion-Parameter
 *   Sparse MoE Models".
 * Both: the k slots of a token are ordered by selection key descending,
 * equal keys by lower expert index. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID_BIAS = 1 } moe_score_fn;

/* MOE_E2M1: FP4 weights in the OCP MXFP4 format -- E2M1 codes packed two per byte (element
 * 2j in the low nibble of byte j), one E8M0 scale byte (2^(code - 127)) per 32 consecutive
 * elements along K -- taken with e4m3 activations ("FP8/FP4 grouped GEMM", GC-MoE title).
 * The scale bytes of a [rows, K] weight matrix are stored as 512-byte atoms, one per 128
 * rows x 128 K-elements, [rows/128][K/128][512]: inside an atom the scale of row r (0..127)
 * and 32-element run q (0..3) sits at byte (r % 32) * 16 + (r / 32) * 4 + q -- the layout
 * the tensor cores' scale-factor copy takes, so the kernels copy atoms without reshuffling. */
/* MOE_E4M3_FP32_SCALE: e4m3 values whose fp32 block scales (1x128 for activations, 128x128
 * for weights, as for MOE_E4M3) may be any positive finite value, not only powers of two.
 * The expert GEMMs then multiply without block scaling and fold each 128-K block's
 * s_weight * s_activation into fp32 accumulators (exact up to fp32 rounding), on 32-token
 * tiles for decode-sized batches and 64-token tiles above: slower than MOE_E4M3, whose
 * power-of-two scales the tensor cores apply directly.
 * Activations and weights both take this dtype.  The router takes x = code x scale as a
 * bf16 part plus its bf16 remainder (two router GEMMs, summed with the split-K partials):
 * x to ~2^-17 relative, where a single bf16 rounding would move the logits by ~2^-9. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2, MOE_E2M1 = 3, MOE_E4M3_FP32_SCALE = 4 } moe_dtype;

/* The layer's sizes: T tokens x d_model activations, E routed experts, top_k,
 * expert intermediate size d_ff (I), n_shared always-on shared experts of
 * intermediate d_ff_shared (must equal d_ff).  `out` is MOE_BF16 or MOE_F32. */
typedef struct {
  int32_t T, d_model, E, top_k, d_ff, n_shared, d_ff_shared;
  moe_score_fn score;
  moe_dtype act, weight, out;
} moe_config;

/* Weights of one layer (device pointers).
 *   wr     [E, d]          router weights (bf16; f32 for the f32 family)
 *   sel_bias [E] fp32      selection bias (SIGMOID_BIAS only; may be NULL = 0)
 *   w13    [E, 2I, d]      per expert: W1 (gate, rows 0..I-1) over W3 (up, rows I..2I-1)
 *   w2     [E, d, I]       per expert down projection
 *   w13_s, w2_s            block scales of the weights:
 *                          e4m3: fp32 [E, 2I/128, d/128] and [E, d/128, I/128];
 *                          e2m1: uint8 E8M0 codes in scale atoms (see MOE_E2M1),
 *                          [E, 2I/128, d/128, 512] and [E, d/128, I/128, 512],
 *                          16-byte aligned (w13 is then [E, 2I, d/2] bytes, w2
 *                          [E, d, I/2], both 32-byte aligned); unused (NULL) otherwise
 *   ws13 [S, 2I, d], ws2 [S, d, I] (+ ws13_s, ws2_s): shared experts (NULL when S = 0) */
typedef struct {
  const void *wr;
  const float *sel_bias;
  const void *w13, *w2;
  const void *w13_s, *w2_s;
  const void *ws13, *ws2;
  const void *ws13_s, *ws2_s;
} moe_weights;

/* Bytes of workspace moe_layer_forward / moe_permute / moe_grouped_ffn need
 * for `cfg` (the largest of the three).  Host only; no CUDA call. */
MOE_API moe_status moe_workspace_size(const moe_config *cfg, size_t *bytes);

/* Router top-k and gates ("topk_softmax" step).
 *   logits   [T, E] fp32   router logits (input)
 *   sel_bias [E] fp32 or NULL (SIGMOID_BIAS only)
 *   topk_idx [T, k] int32  selected experts, slot order as above (output)
 *   topk_w   [T, k] fp32   renormalised gates (output)
 * One warp per token; no workspace. */
MOE_API moe_status moe_route(const moe_config *cfg, const float *logits, const float *sel_bias,
                     int32_t *topk_idx, float *topk_w, cudaStream_t stream);

/* Dispatch on one GPU: a stable permutation of the T*k (token, slot) pairs into
 * per-expert contiguous groups, expert-major, ascending token inside a group
 * (the pseudocode's `dispatch(experts, idx)` without the all-to-all).
 *   topk_idx      [T, k] int32 (input); an entry outside [0, E) sets the device
 *                 status MOE_ERR_DEVICE_INDEX and that pair is dropped
 *   x             [T, d] activations (cfg->act); x_scale [T, d/128] fp32 (e4m3) or NULL
 *   x_perm        [T*k, d] permuted rows (output, same dtype as x);
 *                 x_perm_scale [T*k, d/128] (e4m3) or NULL
 *   perm_token    [T*k] int32  token of each permuted row (output)
 *   inv_perm      [T, k] int32 permuted row of (token, slot) (output)
 *   group_offsets [E+1] int32  exclusive prefix of group sizes (output)
 *   ws, ws_bytes  workspace (>= moe_workspace_size)
 * Quantise-in-permute: with bf16 activations and e4m3 or FP4 expert weights
 * (cfg->act MOE_BF16, cfg->weight MOE_E4M3 / MOE_E2M1) the rows are quantised to
 * e4m3 in the same pass, as the expert GEMMs take them: each token's 128-value
 * block gets the scale 2^e, e the smallest integer with amax <= 448 * 2^e (e = 0
 * for an all-zero block), and each value x becomes e4m3(x / 2^e), round to nearest
 * even.  x_perm [T*k, d] then receives e4m3 codes and x_perm_scale [T*k, d/128]
 * (required) the fp32 scales 2^e; x_scale is unused. */
MOE_API moe_status moe_permute(const moe_config *cfg, const int32_t *topk_idx, const void *x,
                       const float *x_scale, void *x_perm, float *x_perm_scale,
                       int32_t *perm_token, int32_t *inv_perm, int32_t *group_offsets,
                       void *ws, size_t ws_bytes, cudaStream_t stream);

/* moe_permute without a workspace, for callers that cannot allocate device
 * memory to give the library -- for instance a plugin whose host application
 * owns every device allocation through its own pool, or code on a latency path
 * where cudaMalloc (which may synchronise the device) is not allowed.  The pages
 * have no counterpart: it is the same permutation with the same arguments and
 * results as moe_permute, minus ws / ws_bytes.
 * bf16 rows for e4m3 or FP4 experts (the quantising permutation) are not taken
 * here: MOE_ERR_UNSUPPORTED.
 * Its scratch is a fixed array inside the library (about 1 MiB per GPU that
 * loads the library, held until the process exits), so it accepts only
 * ceil(T / 256) * E <= 262144 (for example T <= 65536 with E <= 1024); larger
 * shapes return MOE_ERR_UNSUPPORTED.  It calls no allocator.
 *  - The first call on a device looks up the array's device address (with that
 *    device current); make that first call before any stream capture.
 *  - Every call shares the one array, which keeps the previous call's contents;
 *    the call clears what must start at zero itself.  Calls whose kernels
 *    overlap on the GPU (several streams, or several host threads) race on it:
 *    serialise them.
 *  - Every dtype moe_permute takes: f32, bf16, and e4m3 rows, whose fp32
 *    1x128 scales x_scale [T, d/128] are permuted into x_perm_scale
 *    [T*k, d/128] (both required, non-NULL, when act is e4m3 and T > 0).
 *  - No device status is recorded.  Pairs with an expert index outside [0, E)
 *    are dropped (inv_perm = -1, not counted in group_offsets).  An expert
 *    listed twice in one token's row is not detected: both slots get the same
 *    permuted row, the group counts it once, and a combine over this result
 *    adds that expert's output twice.  moe_permute reports both faults as
 *    MOE_ERR_DEVICE_INDEX; call it where the indices are untrusted. */
MOE_API moe_status moe_permute_noalloc(const moe_config *cfg, const int32_t *topk_idx,
                                       const void *x, const float *x_scale, void *x_perm,
                                       float *x_perm_scale, int32_t *perm_token,
                                       int32_t *inv_perm, int32_t *group_offsets,
                                       cudaStream_t stream);

/* Grouped SwiGLU expert FFN over ragged groups (one expert per group):
 *   y[r] = (silu(a[r] W1_g^T) * (a[r] W3_g^T)) W2_g^T  for rows r of group g.
 *   n_groups        G (<= E + n_shared of cfg, which sizes the workspace); group g
 *                   uses weights w13[g], w2[g]
 *   group_offsets   [G+1] int32 DEVICE array of row offsets into a / y
 *                   (non-decreasing; read on the device, never copied to the host).
 *                   Offsets that decrease or pass n_rows set the device status
 *                   MOE_ERR_DEVICE_INDEX and the layer computes nothing.
 *   n_rows          rows allocated in a and y (>= offsets[G], <= T*k + n_shared*T,
 *                   the most the workspace holds); nothing past row n_rows is
 *                   read or written
 *   a               [offsets[G], d] rows in the token dtype of the expert GEMMs:
 *                   cfg->act, except e4m3 whenever the weights are e4m3 or FP4
 *                   (as moe_permute returns them); a_scale [rows, d/128] fp32 for
 *                   e4m3 rows, else NULL.  For the f32 family a, w13 and w2 are
 *                   rounded to bf16 into the workspace first.
 *   w13, w2         [G, 2I, d], [G, d, I] (+ block scales for e4m3 and e2m1 weights,
 *                   laid out as in moe_weights)
 *   y               [offsets[G], d] bf16 output
 * The shared expert is this call with n_groups = 1, offsets {0, T}, a = x.
 * The intermediate h lives in the workspace.  A persistent tcgen05/TMA kernel
 * walks the groups with a device-side tile scheduler (no host sync). */
MOE_API moe_status moe_grouped_ffn(const moe_config *cfg, int32_t n_groups, const int32_t *group_offsets,
                           int32_t n_rows, const void *a, const float *a_scale, const void *w13,
                           const void *w13_s, const void *w2, const void *w2_s, void *y,
                           void *ws, size_t ws_bytes, cudaStream_t stream);

/* Weighted un-permute (the pseudocode's `out += weights[..., k] * e(x)` and
 * `out += s(x)`): out[t] = sum_j topk_w[t,j] * y_perm[inv_perm[t,j]]
 * + sum_s y_shared[s, t], summed in slot order, then shared expert order, in
 * fp32 registers (no atomics), rounded once and written as cfg->out.
 *   y_perm [T*k, d] bf16; inv_perm [T, k] int32 (entries outside [0, T*k) add 0);
 *   topk_w [T, k] fp32;
 *   y_shared [cfg->n_shared, T, d] bf16: the shared experts' outputs stacked, or
 *            NULL (nothing added; also when cfg->n_shared = 0 any pointer is ignored);
 *   y [T, d] (output). */
MOE_API moe_status moe_combine(const moe_config *cfg, const void *y_perm, const int32_t *inv_perm,
                       const float *topk_w, const void *y_shared, void *y, cudaStream_t stream);

/* The whole layer: router GEMM, route, permute, grouped routed + shared expert
 * FFN, combine.  x [T, d] (+ x_scale for e4m3); y [T, d] (cfg->out).
 * topk_idx_out [T, k] / topk_w_out [T, k] receive the routing when non-NULL. */
MOE_API moe_status moe_layer_forward(const moe_config *cfg, const moe_weights *weights, const void *x,
                             const float *x_scale, void *y, int32_t *topk_idx_out,
                             float *topk_w_out, void *ws, size_t ws_bytes, cudaStream_t stream);

/* moe_layer_forward that also records stage_events[0..7] (host array of 8
 * caller-created CUDA events) on `stream`: before the router GEMM and after
 * each of router GEMM, route, permute, tile plan, FFN1 (gate/up GEMM +
 * SwiGLU), FFN2 (down GEMM), combine -- so a caller can time every kernel of
 * the layer in place with cudaEventElapsedTime.  Same results as
 * moe_layer_forward; any null event -> MOE_ERR_INVALID_ARG. */
MOE_API moe_status moe_layer_forward_staged(const moe_config *cfg, const moe_weights *weights,
                                            const void *x, const float *x_scale, void *y,
                                            int32_t *topk_idx_out, float *topk_w_out, void *ws,
                                            size_t ws_bytes, cudaStream_t stream,
                                            cudaEvent_t *stage_events);

/* The whole layer recorded once into a CUDA graph and replayed: every kernel of
 * moe_layer_forward (8 to 14 launches) goes to the GPU as one graph launch, which
 * removes the per-launch host cost and the gaps between the layer's kernels on a
 * decode step ("Fused single-kernel decode layer ... or a CUDA-graph capture"; the
 * 3-node CUDA graph of the GC-MoE key changes).
 *  moe_layer_graph_create  checks its arguments as moe_layer_forward does, then
 *      records the layer for exactly these pointers and sizes on an internal stream
 *      (no kernel runs) and instantiates the graph into *graph_out.  The graph reads x
 *      (and x_scale) and writes y, the routing outputs and ws at the addresses given
 *      here: to run the layer on new activations, write them into x and launch again.
 *      It allocates host memory for the handle and the graph; no device memory.
 *  moe_layer_graph_launch  enqueues one layer call on `stream` (stream-ordered, like
 *      moe_layer_forward).  Launches of one graph must not overlap on the GPU: they
 *      share the workspace.
 *  moe_layer_graph_destroy frees the handle (after its launches have completed). */
typedef struct moe_layer_graph_t *moe_layer_graph;
MOE_API moe_status moe_layer_graph_create(const moe_config *cfg, const moe_weights *weights,
                                          const void *x, const float *x_scale, void *y,
                                          int32_t *topk_idx_out, float *topk_w_out, void *ws,
                                          size_t ws_bytes, moe_layer_graph *graph_out);
MOE_API moe_status moe_layer_graph_launch(moe_layer_graph graph, cudaStream_t stream);
MOE_API moe_status moe_layer_graph_destroy(moe_layer_graph graph);

/* ------------------------------------------------------------------------------------
 * Norms around a block, fused with its gate and residual scale
 * ------------------------------------------------------------------------------------
 * How a block's gate multiplies its branch: not at all, one value per channel [d], one
 * per token [T], or one per element [T, d]. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2, MOE_GATE_FULL = 3 } moe_gate;

/* Sizes and types of a block norm over T tokens (at most 2^30) x d_model channels (a
 * multiple of 8, at most 16384).
 *   res     r, r_out, dr_out, dr (the residual stream)    MOE_BF16 or MOE_F32
 *   act     y, dy, dh and a MOE_GATE_FULL gate / dgate    MOE_BF16 or MOE_F32
 *   weight  w_post, w_pre, a channel or token gate        MOE_BF16 or MOE_F32
 *   out     h: MOE_BF16, MOE_F32, or MOE_E4M3 (d_model % 128 == 0): codes with one
 *           power-of-two fp32 scale per 128 channels, by the rule of moe_permute -- the form
 *           moe_layer_forward takes as MOE_E4M3 activations and moe_grouped_gemm as rows
 *   eps > 0; res_scale and branch_scale finite; w_offset is added to both norm weights (1 for
 *   weights stored as differences from one, else 0) */
typedef struct {
  int32_t T, d_model;
  moe_gate gate;
  moe_dtype res, act, weight, out;
  float eps, res_scale, branch_scale, w_offset;
} moe_norm_config;

/* Bytes of workspace moe_block_norm_backward needs.  Host only; no CUDA call. */
MOE_API moe_status moe_norm_workspace_size(const moe_norm_config *cfg, size_t *bytes);

/* The end of one block and the start of the next:
 *   u     = norm(y; w_post)                      (u = y when w_post is NULL)
 *   r_out = res_scale * r + branch_scale * gate * u
 *   h     = norm(r_out; w_pre)
 *   norm(x; w) = x / sqrt(mean(x^2) + eps) * (w + w_offset)   per token
 * in fp32 registers, each output rounded once (h from the unrounded r_out).  The sum of a row's
 * squares is fp32 as well: it has to stay below 3.4e38.
 *   y      NULL: no branch (r_out = res_scale * r; gate and w_post NULL, gate kind NONE)
 *   w_pre  NULL: no second norm (h NULL)
 *   r_out  NULL: not stored
 *   h_scale [T, d/128] fp32 when cfg->out is MOE_E4M3, else NULL
 * r_out may be r itself; h may be y or r itself where the types have one size.  Tensors
 * 16-byte aligned (a token gate and h_scale: by their element).  T = 0 does nothing.  Neither
 * call records a device status. */
MOE_API moe_status moe_block_norm(const moe_norm_config *cfg, const void *r, const void *y,
                                  const void *w_post, const void *gate, const void *w_pre, void *r_out,
                                  void *h, float *h_scale, cudaStream_t stream);

/* Gradients of moe_block_norm.  r_out, y, w_post, gate, w_pre as in the forward call (the
 * norms' statistics are recomputed from r_out and y); dh [T, d] (cfg->act; required with
 * w_pre) and dr_out [T, d] (cfg->res; NULL = 0) are the gradients of h and r_out.  With
 *   G    = dr_out + dnorm(r_out; w_pre)^T dh
 *   dr   = res_scale * G                              [T, d] cfg->res
 *   dy   = dnorm(y; w_post)^T (branch_scale gate G)   [T, d] cfg->act (required with y)
 *   dgate = branch_scale G u, summed to the gate's shape: fp32 [d] or [T], or cfg->act [T, d]
 *   dw_post, dw_pre [d] fp32
 * dgate, dw_post and dw_pre may be NULL (not computed).  Sums over tokens run in a fixed
 * order (bit-identical reruns); T = 0 writes zeros to the [d] gradients.  cfg->out is not
 * used.  dr may be dr_out and dy may be dh or y where the types match.  Of the workspace
 * only what lies behind its first 256 bytes is used; it need not be zeroed. */
MOE_API moe_status moe_block_norm_backward(const moe_norm_config *cfg, const void *r_out, const void *y,
                                           const void *w_post, const void *gate, const void *w_pre,
                                           const void *dh, const void *dr_out, void *dr, void *dy,
                                           void *dgate, float *dw_post, float *dw_pre, void *ws,
                                           size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------
 * Products grouped by expert, one at a time
 * ------------------------------------------------------------------------------------
 * n_groups weight matrices [n, k] and up to n_rows rows sorted into groups (as moe_permute
 * leaves them): group g holds rows group_offsets[g] .. group_offsets[g + 1] - 1.
 *   in   MOE_BF16 (n and k multiples of 8) or MOE_E4M3_FP32_SCALE (n % 8 == 0, k % 16 == 0;
 *        moe_grouped_gemm only)
 *   out  MOE_BF16 or MOE_F32
 * 1 <= n_groups <= 1024; n, k <= 65536; n_rows <= 2^24.
 * n_rows may be more than the groups hold, but it is also what the kernel is chosen by (at most 8
 * rows per group on average, or 32 in all, 64 in e4m3: tiles of few rows): a call for a few rows
 * at the head of a large buffer is faster with their number, or a bound near it, as n_rows.
 * Products of bf16 are summed 512 at a time on the tensor cores, and those sums in fp32.
 * Calls that share a workspace must not overlap on the GPU.  Tiles that several CTAs sum up
 * are joined in a fixed order: reruns are bit-identical.  After MOE_ERR_TIMEOUT the header must
 * be reset (moe_reset_device_status) before the workspace is used again. */
typedef struct {
  int32_t n_groups, n_rows, n, k;
  moe_dtype in, out;
} moe_product_config;

/* Bytes of workspace the grouped products need.  Host only; no CUDA call. */
MOE_API moe_status moe_product_workspace_size(const moe_product_config *cfg, size_t *bytes);

/* y[r] = a[r] W_g^T for the rows r of group g.
 *   group_offsets [n_groups + 1] int32 DEVICE, non-decreasing, <= n_rows; NULL with one group:
 *                 all n_rows rows.  Offsets that decrease, are negative or pass n_rows set the
 *                 device status MOE_ERR_DEVICE_INDEX and nothing is computed.
 *   a [n_rows, k], w [n_groups, n, k], y [n_rows, n] (cfg->out); rows outside the groups are
 *                 neither used nor written
 *   a_scale, w_scale  MOE_E4M3_FP32_SCALE: fp32 [n_rows, ceil(k/128)] and
 *                 [n_groups, ceil(n/128), ceil(k/128)], one scale per 128 codes of a row and per
 *                 128 x 128 codes of a weight, of any finite value; else NULL.  The product of
 *                 each 128-k block is summed on the tensor cores and multiplied by the product
 *                 of its two scales in fp32.  Where that overflows, the device status becomes
 *                 MOE_ERR_DEVICE_VALUE and the outputs concerned are infinite or NaN; where it
 *                 is below 2^-126 it rounds as a subnormal number, which moves the block's
 *                 share by 2^-125 at most.
 * A dense 8-bit product is this call with one group.  a, w, y 16-byte aligned, scales and
 * group_offsets by their elements.  The first 256
 * bytes of the workspace hold the device status (moe_reset_device_status once before use). */
MOE_API moe_status moe_grouped_gemm(const moe_product_config *cfg, const int32_t *group_offsets,
                                    const void *a, const float *a_scale, const void *w,
                                    const float *w_scale, void *y, void *ws, size_t ws_bytes,
                                    cudaStream_t stream);

/* The gradient of the rows, da[r] = dy[r] W_g: dy [n_rows, n] bf16, w [n_groups, n, k] bf16,
 * da [n_rows, k] (cfg->out).  Offsets, rows outside the groups and workspace as above. */
MOE_API moe_status moe_grouped_gemm_dgrad(const moe_product_config *cfg, const int32_t *group_offsets,
                                          const void *dy, const void *w, void *da, void *ws,
                                          size_t ws_bytes, cudaStream_t stream);

/* The gradient of the weights, dw_g = sum over rows r of group g of dy[r]^T a[r]: dy
 * [n_rows, n] bf16, a [n_rows, k] bf16, dw [n_groups, n, k] (cfg->out), zeros for a group
 * without rows.  Rows outside a group never enter its sum, whatever they hold. */
MOE_API moe_status moe_grouped_gemm_wgrad(const moe_product_config *cfg, const int32_t *group_offsets,
                                          const void *dy, const void *a, void *dw, void *ws,
                                          size_t ws_bytes, cudaStream_t stream);

/* Self-test of the device-side failure path (no counterpart on the pages): a
 * tiny kernel waits on a barrier that nothing completes, gives up after
 * `budget_cycles` SM clock cycles (1 .. 2^33), writes MOE_ERR_TIMEOUT into the
 * status word of workspace `ws` and returns -- the bounded-wait path every
 * tcgen05 kernel of the library takes instead of hanging.  Asynchronous; read
 * the result with moe_read_device_status. */
MOE_API moe_status moe_selftest_bounded_wait(void *ws, long long budget_cycles, cudaStream_t stream);

/* Synchronises `stream`, then reads the device status word of workspace `ws`
 * into *out (MOE_OK when no device fault was recorded).  Does not clear it. */
MOE_API moe_status moe_read_device_status(const void *ws, cudaStream_t stream, moe_status *out);

/* Zeroes the device status word (and the workspace header) of `ws`, on `stream`. */
MOE_API moe_status moe_reset_device_status(void *ws, cudaStream_t stream);

/* Static text for a status code. */
MOE_API const char *moe_status_string(moe_status status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_B200_H */
