/*
 * moe.h — C ABI of libmoe.so: one top-k Mixture-of-Experts layer on one GB300
 * (sm_103a).
 *
 * The layer. Every decoder layer of Muse Spark is a Mixture-of-Experts layer
 * in which each token picks 8 of 256 experts ("How SGLang-TorchTPU
 * accelerated an 816B-parameter MoE on TPU v7", section "Introduction");
 * per-expert outputs are combined after the experts run ("TensorSharp Muse
 * Spark benchmark", section "Performance"); partial sums of expert outputs
 * are kept in fp32 because bf16 partial sums cost quality (same page, section
 * "Answer quality"). The pages leave the gate and FFN open; this library
 * computes, per token t with bf16 input x[t, 0:d]:
 *
 *   logit[e] = sum_c x[c] * Wr[e, c]  (fp32 accumulate) + bias[e]
 *   p        = softmax(logit) over all E experts (fp32)
 *   ids[0:k] = the k largest p, ties to the lower expert id, by descending p
 *   w[j]     = p[ids[j]] / sum_j' p[ids[j']]
 *   h_j      = silu(Wg[ids[j]] x) * (Wu[ids[j]] x)
 *   y        = sum_j w[j] * (Wd[ids[j]] h_j)   (fp32, j ascending) -> bf16
 *
 * Conventions for every call:
 *  - Pointers named *_host are host memory; every other pointer is device
 *    memory owned by the caller, 16-byte aligned, and must stay valid for as
 *    long as the layer or the enqueued work uses it. The library allocates no
 *    device memory: scratch lives in the caller's workspace.
 *  - `stream` is a cudaStream_t passed as void* (NULL: the legacy default
 *    stream). All device work is enqueued on it, in order; calls return
 *    without waiting for the GPU unless stated otherwise.
 *  - bf16 tensors are raw bf16 bits, row-major, innermost index last.
 *  - Argument errors are detected on the host before any work is enqueued
 *    (MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED); launch failures return
 *    MOE_ERR_CUDA; conditions detected by a kernel (a bounded wait that ran
 *    out, an index out of range) set an error word in the workspace that
 *    moe_get_device_status() reports.
 *  - A layer object is not thread-safe; distinct layers may be used from
 *    distinct threads. Two calls on one layer must not overlap on the GPU
 *    (they share the workspace): issue them on one stream.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* null pointer, misaligned pointer, T out of range */
    MOE_ERR_UNSUPPORTED = 2,  /* shape or format this library does not implement */
    MOE_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
    MOE_ERR_DEVICE = 4,       /* a kernel flagged an out-of-range index */
    MOE_ERR_TIMEOUT = 5       /* a kernel's bounded wait ran out */
} moe_status;

/* Expert weight format. NVFP4 ("How SGLang-TorchTPU accelerated an
 * 816B-parameter MoE on TPU v7", section "Results and interpretation", runs
 * experts as NVFP4 weights): 16-element blocks along the contraction index,
 * each element an E2M1 code, each block one E4M3 scale, each tensor (one
 * matrix of one expert) one fp32 scale: w = e2m1 * e4m3 * s_tensor. */
typedef enum { MOE_W_BF16 = 0, MOE_W_NVFP4 = 1 } moe_wfmt;

typedef struct moe_layer moe_layer;

/* Layer description. Shapes: E experts, hidden size d, expert width I, k
 * experts per token, at most max_tokens tokens per call.
 * Supported: 1 <= k <= 8, k <= E <= 256, d and I multiples of 64, d <= 8192,
 * I <= 4096, 1 <= max_tokens <= 65536. */
typedef struct {
    int d, E, top_k, I, max_tokens;
    moe_wfmt fmt;
    const void *w_router;     /* [E, d] bf16 */
    const float *router_bias; /* [E] fp32, or NULL for no bias */
    /* MOE_W_BF16 experts (NULL otherwise) */
    const void *w_gate;       /* [E, I, d] bf16 */
    const void *w_up;         /* [E, I, d] bf16 */
    const void *w_down;       /* [E, d, I] bf16 */
    /* MOE_W_NVFP4 experts (NULL otherwise). Two E2M1 codes per byte, the low
     * nibble holding the lower contraction index; E4M3 scales one per 16. */
    const uint8_t *q_gate, *q_up; /* [E, I, d/2] */
    const uint8_t *q_down;        /* [E, d, I/2] */
    const uint8_t *s_gate, *s_up; /* [E, I, d/16] */
    const uint8_t *s_down;        /* [E, d, I/16] */
    const float *g_gate, *g_up, *g_down; /* [E] per-tensor fp32 scales */
    /* 0: the plain weighted sum. 1: each expert's output is RMS-normalised
     * (Y / sqrt(mean(Y^2) + 1e-6), no learned scale) before the weighted sum,
     * a reading of "Muse Spark normalises each expert's output, then combines"
     * ("TensorSharp Muse Spark benchmark", section "Performance"). */
    int expert_out_norm;
    /* bf16 experts only. 0: w_gate and w_up are separate [E, I, d] tensors.
     * 1: w_gate points to one [E, I, 2, d] tensor holding gate row i then up
     * row i of each expert (the fused gate/up projection, interleaved by row)
     * and w_up is ignored; the small-batch kernels then fetch a row pair as one
     * contiguous copy. */
    int gate_up_interleaved;
} moe_layer_desc;

/* Bytes of device workspace the layer needs (for max_tokens). No GPU work. */
moe_status moe_workspace_size(const moe_layer_desc *desc, size_t *bytes);

/* Create a layer over caller-owned weights and workspace (ws_bytes at least
 * moe_workspace_size; 256-byte aligned). Zeroes the workspace's control words
 * with a synchronous cudaMemset on the current device; *out receives a
 * host-side handle freed by moe_layer_destroy. */
moe_status moe_layer_create(const moe_layer_desc *desc, void *workspace, size_t ws_bytes,
                            moe_layer **out);

/* Routing and token permutation only (router, softmax, top-k, renormalise,
 * then the permutation). x [T, d] bf16. Outputs (device):
 *   ids [T, k] int32 (descending weight), w [T, k] fp32 (sums to 1 per token),
 *   counts [E] int32, offsets [E+1] int32 (exclusive prefix sum of counts),
 *   perm [T*k] int32: perm[offsets[e] + r] = the r-th smallest token id routed
 *   to expert e, pos [T, k] int32: the row of (t, j) in that order.
 * Any output pointer may be NULL to skip it. 1 <= T <= max_tokens. */
moe_status moe_route(moe_layer *layer, const void *x, int T, int32_t *ids, float *w,
                     int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *pos,
                     void *stream);

/* Layer forward: out [T, d] bf16 = MoE(x). out must not alias x. */
moe_status moe_forward(moe_layer *layer, const void *x, void *out, int T, void *stream);

/* out = bf16(res + MoE(x)) with the residual added in fp32. out may alias res
 * but not x. Used between stacked layers (pre-norm residual block). */
moe_status moe_forward_residual(moe_layer *layer, const void *x, const void *res, void *out,
                                int T, void *stream);

/* End-to-end forward from host memory: copies x_host [T, d] bf16 into the
 * workspace, runs moe_forward, copies the result to out_host [T, d] bf16 and
 * waits for the stream. Page-locked host buffers give asynchronous copies. */
moe_status moe_forward_host(moe_layer *layer, const void *x_host, void *out_host, int T,
                            void *stream);

/* Expert outputs of the last forward on this layer, before the weighted sum:
 * Y [T*k, d] fp32, row pos[t, j] holding expert ids[t, j] applied to token t
 * (pos from moe_route on the same x). For parity checks of every slot. After
 * a large-batch forward the outputs were kept in bf16 (the grouped GEMMs'
 * output precision) and are widened to fp32 here. */
moe_status moe_debug_expert_outputs(moe_layer *layer, float *Y, int T, void *stream);

/* Small-batch (T <= 16) kernel choice. Both compute the same layer in one
 * persistent launch; they differ in where the expert FFNs run:
 *   MOE_DECODE_CUDA_CORES: each weight row is multiplied by the tokens on the
 *     CUDA cores as it streams in (suits one token with bf16 weights, where
 *     the stream alone sets the pace);
 *   MOE_DECODE_TENSOR_CORES: 128 weight rows at a time are the M operand of
 *     tcgen05.mma and the tokens the N = 16 operand, NVFP4 codes widened into
 *     tensor memory on the way (suits several tokens or NVFP4 weights);
 *   MOE_DECODE_AUTO (default): the tensor cores for bf16 experts and 8 or
 *     more tokens, else the CUDA cores.
 * The tensor-core kernel needs d % 128 == 0 and no expert_out_norm; where a
 * layer does not meet that, the CUDA-core kernel runs whatever the choice.
 * Stacks follow the choice of their first layer. */
enum { MOE_DECODE_AUTO = 0, MOE_DECODE_CUDA_CORES = 1, MOE_DECODE_TENSOR_CORES = 2 };
moe_status moe_set_decode_path(moe_layer *layer, int path);

/* Routing records of the last forward or route on this layer, as the
 * kernels left them in the workspace (no recomputation): the fields of
 * moe_route, same layouts; any output pointer may be NULL. A forward of
 * T <= 16 tokens leaves the records its single decode launch computed and
 * published; a larger forward leaves those of the large-batch routing
 * kernels, or, where it runs in chunks of 16 tokens, those of its last
 * chunk. T must be the last call's token count. For parity checks of the
 * routing each forward path uses. */
moe_status moe_debug_route_records(moe_layer *layer, int T, int32_t *ids, float *w, int32_t *counts,
                                   int32_t *offsets, int32_t *perm, int32_t *pos, void *stream);

/* Test hook for the device-side failure detection. While hold != 0, every
 * cross-CTA wait of this layer's single-launch decode kernels (T <= 16, and
 * moe_stack_forward on a stack whose first layer is this one) waits for
 * something that never comes: a grid barrier for one arrival more than the
 * grid provides, the hand-off of the router's logits for a tag no CTA
 * writes. Its bounded wait (1.5 s) runs out:
 * the launch unwinds without computing the experts, leaves `out` undefined
 * and sets the timeout bit that moe_get_device_status() reports as
 * MOE_ERR_TIMEOUT. hold = 0 restores normal operation; the next call runs
 * normally (the launch that gave up resets its counters on exit). Enqueued on
 * `stream` (one 4-byte host-to-device copy). */
moe_status moe_debug_hold_grid_barrier(moe_layer *layer, int hold, void *stream);

/* Row-wise RMSNorm without a learned scale: out = x / sqrt(mean(x^2) + eps),
 * x and out [T, d] bf16 (out may alias x), fp32 arithmetic. */
moe_status moe_rmsnorm(const void *x, void *out, int T, int d, float eps, void *stream);

/* NVFP4 quantiser for n tensors of shape [rows, K] (bf16, contiguous):
 *   s_t = amax|W| / (6*448) (1 for an all-zero tensor),
 *   block scale = E4M3((amax_block / 6) / s_t), code = E2M1(w / (scale * s_t)),
 * round-to-nearest-even, saturating. Outputs q [n, rows, K/2], s [n, rows, K/16],
 * g [n] fp32 (g is also used as the amax accumulator). K multiple of 32. */
moe_status moe_quantize_nvfp4(const void *W, int n, int rows, int K, uint8_t *q, uint8_t *s,
                              float *g, void *stream);

/* Waits for `stream`, then reads and clears the layer's device error word:
 * MOE_OK, MOE_ERR_DEVICE or MOE_ERR_TIMEOUT. */
moe_status moe_get_device_status(moe_layer *layer, void *stream);

/* Number of kernel launches the last forward/route on this layer enqueued. */
int moe_last_launch_count(const moe_layer *layer);

/* Per-kernel timing for measurement. After moe_profile_begin(layer, n), each
 * of the next n forwards on the layer also records a CUDA event on its stream
 * before each of its kernels and one after the last (host-side event objects;
 * no device memory). moe_profile_end waits for those events and writes
 * ms[f * max_kernels + i] = duration of kernel i of recorded forward f, and
 * the counts, then stops recording. The launches of a routing, or of the
 * grouped GEMMs, count as one kernel; so does a forward that runs in chunks. */
moe_status moe_profile_begin(moe_layer *layer, int max_forwards);
moe_status moe_profile_end(moe_layer *layer, float *ms_host, int max_kernels, int *n_forwards,
                           int *n_kernels);

/* The pages have no counterpart to this call; it serves callers that cannot
 * allocate device memory (a plugin inside an inference server or engine that
 * owns all device memory and hands it only input and output buffers, or a
 * real-time loop that forbids allocation after start-up).
 *
 * Same result as moe_forward on the CUDA-core small-batch kernel
 * (MOE_DECODE_CUDA_CORES) for 1 <= T <= 16 tokens, with no layer object
 * and no workspace: the scratch lives in one static device array of
 * MOE_STATIC_SCRATCH_BYTES that every GPU which loads libmoe.so holds until
 * the process exits. The call allocates nothing (no cudaMalloc, no
 * allocating library routine). desc is read on the host during the call only;
 * its max_tokens is ignored (the shape is checked as if it were T). x [T, d]
 * and out [T, d] are bf16 device buffers of the caller.
 * - Every call, with the caller's device and context current, looks up the
 *   array's device address in that context (cudaGetSymbolAddress; nothing is
 *   cached, so a new context after cudaDeviceReset, or a context of the
 *   caller's own on the same device, gets its own copy of the array). The
 *   first call in a process may load the library's device code: make it
 *   before any stream capture.
 * - Every call shares the one array and clears its control words at the start
 *   (an async memset on `stream`): calls that overlap on the GPU race, so
 *   issue them on one stream or otherwise order them.
 * - Shapes whose scratch exceeds MOE_STATIC_SCRATCH_BYTES, or whose tokens do
 *   not fit in shared memory beside the weight ring, return
 *   MOE_ERR_UNSUPPORTED; T outside [1, 16] returns MOE_ERR_INVALID_ARG; both
 *   before any GPU work.
 * - Device-side error bits (a bounded wait that ran out) are not reported:
 *   the next call clears them. After such an event `out` is undefined; a
 *   caller that needs the check uses moe_forward and moe_get_device_status. */
#define MOE_STATIC_SCRATCH_BYTES (8u << 20)
moe_status moe_forward_static_scratch(const moe_layer_desc *desc, const void *x, void *out, int T,
                                      void *stream);

/* Stacked layers in one launch (the persistent multi-layer decode kernel
 * the pages' megakernel idea suggests, "How SGLang-TorchTPU accelerated an
 * 816B-parameter MoE on TPU v7", section "Key optimisations"). For
 * l = 0 .. n_layers-1:
 *     x_{l+1} = x_l + MoE_l(RMSNorm(x_l)),   x_0 = x,   out = x_n,
 * RMSNorm without a gain, eps as given, its output rounded to bf16 (the
 * arithmetic of moe_rmsnorm), the sum rounded to bf16 (moe_forward_residual).
 * - moe_stack_create: 1 <= n_layers <= 64 layers of equal d, E, top_k, I and
 *   weight format, without expert_out_norm, whose max_tokens >= 1. It writes
 *   the layers' weight pointers (not the weights) into layers[0]'s workspace
 *   once (a synchronous copy); the stack then runs on that workspace, so the
 *   stack and layers[0] must not run at the same time. The layers must
 *   outlive the stack.
 * - moe_stack_forward: T in [1, 8] and <= layers[0]'s max_tokens; x, out bf16
 *   [T, d] device buffers (out may alias x). layer_out, if not NULL, receives
 *   every layer's output, [n_layers, T, d] bf16. One launch, no host sync.
 *   Errors as for moe_forward. */
typedef struct moe_stack moe_stack;
moe_status moe_stack_create(moe_layer *const *layers, int n_layers, moe_stack **out);
moe_status moe_stack_forward(moe_stack *stack, const void *x, void *out, int T, float eps, void *layer_out,
                             void *stream);
/* End-to-end stack forward from host memory: copies x_host [T, d] bf16 into
 * layers[0]'s workspace, runs moe_stack_forward, copies the result to
 * out_host [T, d] bf16 and waits for the stream. Page-locked host buffers
 * give asynchronous copies. */
moe_status moe_stack_forward_host(moe_stack *stack, const void *x_host, void *out_host, int T, float eps,
                                  void *stream);
moe_status moe_stack_destroy(moe_stack *stack);

/* ---------------------------------------------------------------------------
 * Operators around the layer: routing from logits, the residual addition and
 * norm in front of it, products with 4-bit weights, 4-bit floats and their
 * products, and products grouped by expert. They keep no state:
 * calls on different streams may overlap as long as their buffers (and, for
 * moe_route_logits, their workspaces) differ, and all of them can be captured
 * into a graph. Strides count elements, and rows may lie further apart than
 * their length. Unless stated otherwise a pointer has the alignment of its
 * elements only. Buffers belong to the current device.
 * ------------------------------------------------------------------------- */
typedef enum { MOE_T_BF16 = 0, MOE_T_F16 = 1, MOE_T_F32 = 2, MOE_T_E4M3 = 3 } moe_dtype;

/* Routing. With l the logits of a token,
 *   p = softmax(l) or 1 / (1 + exp(-l)),   c = p + bias (bias NULL: c = p)
 *   group score (n_groups > 1): the best c of the group, or the sum of its two
 *     best (of the one, where only one is left); the topk_groups best are kept
 *   ids = the top_k best c within the kept groups, by descending c
 *   w[j] = scale * p[ids[j]], divided by the sum of the chosen p if renormalise
 * Ties go to the lower index, group or expert. The choice is that of scores
 * in 64-bit arithmetic, without a bias that of the logits (which order the
 * scores; sums of two best always are of scores). An expert whose logit is NaN or -inf takes no part in
 * the softmax and is never chosen; nor is one whose bias is; +inf counts as
 * the largest finite float. Where fewer than top_k experts are left the
 * remaining slots hold id -1, weight 0 and pos -1.
 * Limits: E <= 512, top_k <= 16, n_groups <= 32 and dividing E, the kept
 * groups holding at least top_k experts, T <= 262144. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_rule;
typedef struct {
    int E, top_k;
    moe_score score;
    const float *bias;           /* [E] fp32 (device) or NULL; steers the choice, not the weights */
    int n_groups, topk_groups;   /* 1, 1: no groups */
    moe_group_rule group_rule;
    int renormalise;
    float scale;
} moe_route_desc;

/* Bytes of device workspace moe_route_logits needs for T tokens (0 for few). No GPU work. */
moe_status moe_route_logits_workspace_size(const moe_route_desc *desc, int T, size_t *bytes);

/* logits [T, E] in bf16, f16 or fp32, row_stride elements from row to row.
 * ids [T, top_k] and w [T, top_k] are required; counts [E], offsets [E+1],
 * perm [T*top_k] and pos [T, top_k] as in moe_route, each optional (NULL).
 * Entries of perm past offsets[E] are set to -1. The workspace (16-byte
 * aligned) may be NULL when none of the four is asked for; it needs no
 * initialisation and carries nothing from one call to the next; up to 256
 * tokens need none. The outputs overlap neither each other nor the inputs. T = 0
 * only zeroes counts and offsets. */
moe_status moe_route_logits(const moe_route_desc *desc, const void *logits, moe_dtype type, int64_t row_stride, int T,
                            int32_t *ids, float *w, int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *pos,
                            void *workspace, size_t ws_bytes, void *stream);

/* Makes moe_route and moe_forward* on this layer choose experts as `desc`
 * says, from the layer's own router logits (router_bias included); NULL
 * restores the softmax top-k. E and top_k must be the layer's. desc is copied;
 * its bias is read by every later call and must stay valid until they are done,
 * and as long as a graph that captured one is replayed. Such a forward runs
 * the router, the choice and the expert kernels as separate launches, up to 16
 * tokens those of the split decode whatever moe_set_decode_path says (slower
 * than the single launch, the more so the more tokens). A token left with fewer
 * than top_k experts sets the error word that moe_get_device_status() reports
 * as MOE_ERR_DEVICE, and its output is undefined. Stacks of layers run the
 * softmax top-k only: moe_stack_create and moe_stack_forward return
 * MOE_ERR_UNSUPPORTED while one of their layers has a router set. */
moe_status moe_layer_set_router(moe_layer *layer, const moe_route_desc *desc);

/* Residual addition and RMSNorm:
 *   s = round(x + res)   (to `type`; s = x without res)
 *   y = s / sqrt(mean(s^2) + eps) * gain
 * out_type = type: out = round(y). out_type = MOE_T_E4M3: for every `group`
 * columns (0: the whole row) scale = max|y| / 448 (1 where that is no normal
 * float: a group of zeros) and out = E4M3(y / scale). fp32 arithmetic, roots and
 * quotients within a few 2^-24: where y / scale is the middle between two codes
 * (bf16 and f16 inputs meet it exactly), either may be stored. The norm is of
 * the rounded sum, as moe_rmsnorm after moe_forward_residual. A row of
 * zeros gives zeros (eps = 0 included); a row with an infinity or NaN gives what
 * the formula does, zeros and NaN, and no other row is touched. sum, or out of
 * the inputs' type, may be the same buffer as x or res, with the same stride;
 * any other overlap is not allowed. d <= 16384, group dividing d, at most 4096
 * groups. */
typedef struct {
    const void *x;       /* [T, d] bf16, f16 or fp32 */
    const void *res;     /* [T, d] of the same type, or NULL */
    const void *gain;    /* [d] of the same type, or NULL */
    void *sum;           /* [T, d] of the same type: s, or NULL */
    void *out;           /* [T, d] */
    float *scales;       /* [T, d / group] for E4M3 output, else NULL */
    int64_t x_stride, res_stride, sum_stride, out_stride, scales_stride;
    int T, d, group;
    moe_dtype type, out_type;
    float eps;
} moe_norm_args;
moe_status moe_add_rmsnorm(const moe_norm_args *args, void *stream);

/* y = x W^T + bias for M <= 64 tokens and 4-bit weights W [N, K], two codes
 * per byte, the low nibble holding the lower contraction index:
 *   MOE_W4_NVFP4: w = e2m1 * e4m3 * g, as moe_quantize_nvfp4 writes them
 *     (group 16, s [N, K/16], g one fp32);
 *   MOE_W4_INT4: w = (code - z) * s, codes 0..15, group 32, 64 or 128,
 *     s [N, K/group] bf16 or f16, z [N, K/group] bytes, NULL: 8 everywhere.
 * x [M, K] is bf16, f16, or E4M3 with scales x_scales [M, K/x_group], x_group
 * a multiple of 128 or 0 (one scale per token), as moe_add_rmsnorm writes
 * them. y [M, N] is bf16, f16 or fp32. Weights enter the products exactly, as do
 * f16 and E4M3 x; bf16 x is held relative to the largest finite element of each
 * 128 columns, to 2^-39 of it (exactly down to 2^-29). Products and sums are
 * fp32, NVFP4's in units of g; more than 32 tokens read the weights twice. K a
 * multiple of 32 and of the group, K <= 32768, N <= 2^30; q 16-byte aligned, s
 * 2-byte aligned; y overlaps no input. */
typedef enum { MOE_W4_NVFP4 = 0, MOE_W4_INT4 = 1 } moe_w4_fmt;
typedef struct {
    moe_w4_fmt fmt;
    int M, N, K, group;
    const uint8_t *q;    /* [N, K/2] */
    const void *s;
    moe_dtype s_type;    /* INT4 */
    const float *g;      /* NVFP4: [1] */
    const uint8_t *z;    /* INT4 */
    const void *x;
    moe_dtype x_type;
    int64_t x_stride;
    const float *x_scales;
    int64_t x_scales_stride;
    int x_group;
    const float *bias;   /* [N] fp32 or NULL */
    void *y;
    moe_dtype y_type;
    int64_t y_stride;
} moe_w4_args;
moe_status moe_linear_w4(const moe_w4_args *args, void *stream);

/* A product's waits for its weights are bounded (1.5 s). Where one runs out the
 * call leaves NaN in the rows concerned and sets a bit that belongs to the
 * device, not to the call. moe_linear_w4_status waits for `stream`, then reads
 * and clears the current device's: MOE_OK or MOE_ERR_TIMEOUT. A bit that is set
 * meanwhile by work on another stream is kept for the next call. Not while the
 * stream is being captured. */
moe_status moe_linear_w4_status(void *stream);

/* Test hook: the products launched while hold != 0 copy no weights, so that
 * their waits run out. No GPU work. */
moe_status moe_debug_hold_linear_w4(int hold);

/* Microscaled 4-bit floats: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a
 * sign), two to a byte, the low nibble holding the lower index, and scales:
 *   MOE_FP4_NVFP4: an E4M3 byte s (not negative) per 16 columns and an fp32 g
 *     per row (or matrix); a code stands for e2m1 * s * g;
 *   MOE_FP4_MXFP4: a byte s per 32 columns, the power of two 2^(s - 127), 255
 *     NaN; a code stands for e2m1 * 2^(s - 127).
 * moe_quantize_nvfp4 writes the first, g one per matrix. */
typedef enum { MOE_FP4_NVFP4 = 0, MOE_FP4_MXFP4 = 1 } moe_fp4_fmt;

/* Rows to 4-bit floats. v = x, or silu(x) * up in fp32 with up; rows given:
 * row r of the result is that of x (and up) at rows[r], and stays as it is
 * where rows[r] lies outside [0, T), as perm of the routing does past its end.
 *   NVFP4: g = the smallest power of two >= max|v of the row| / 2688, at least
 *     2^-100, 1 for a row of zeros; s = E4M3(max|v of the block| / 6 / g);
 *     codes E2M1(v / (s g)), 0 where s is 0.
 *   MXFP4: s = floor(log2 max|v of the block|) - 2, clamped to [-127, 127], as
 *     s + 127, 0 for a block of zeros; codes E2M1(v / 2^s), saturating.
 * Nearest, ties to even, of exact quotients (with up: of the fp32 v, which
 * is within (5 + 1.2 |x|) 2^-23 of itself for x > -87.3; below, silu(x) is 0).
 * A row (NVFP4) or block (MXFP4) that holds an infinity or NaN gets codes 0 and
 * NaN as g (255 as s): everything computed from it is NaN. K a multiple of 64,
 * K <= 32768; q 16-byte, s 4-byte aligned, both without gaps between rows. No
 * output overlaps an input. */
typedef struct {
    moe_fp4_fmt fmt;
    moe_dtype type;      /* of x and up: bf16 or f16 */
    const void *x;       /* [T, K] */
    const void *up;      /* [T, K] or NULL */
    int64_t x_stride, up_stride;
    const int32_t *rows; /* [R], or NULL: R = T, in order */
    int T, R, K;
    uint8_t *q;          /* [R, K/2] */
    uint8_t *s;          /* [R, K/16] or [R, K/32] */
    float *g;            /* NVFP4: [R] */
    void *workspace;     /* 16-byte aligned, or NULL */
    size_t ws_bytes;
} moe_quantize_fp4_args;
moe_status moe_quantize_fp4(const moe_quantize_fp4_args *args, void *stream);

/* Bytes of device workspace with which moe_quantize_fp4 is faster, 0 where it
 * uses none: gathered rows that are many times the tokens take every token's
 * codes from there. The results are the same without, it needs no
 * initialisation and carries nothing from one call to the next. Looks at fmt, T,
 * R, K and whether there are rows and up. No GPU work. */
moe_status moe_quantize_fp4_workspace_size(const moe_quantize_fp4_args *args, size_t *bytes);

/* What codes and scales stand for, in fp32 and rounded once to bf16, f16 or
 * fp32. g (NVFP4): [R], or one for all rows, or NULL (1). Alignment and limits
 * as above. */
typedef struct {
    moe_fp4_fmt fmt;
    moe_dtype type;      /* of out */
    const uint8_t *q, *s;
    const float *g;
    int g_rows;          /* nonzero: g holds one scale a row */
    int R, K;
    void *out;           /* [R, K] */
    int64_t out_stride;
} moe_dequantize_fp4_args;
moe_status moe_dequantize_fp4(const moe_dequantize_fp4_args *args, void *stream);

/* Products of rows grouped by expert, y[r] = W[e] x[r] + bias[e] for the rows
 * offsets[e] <= r < offsets[e+1] (device, int32, ascending, as the routing
 * writes them); rows before offsets[0] and from offsets[groups] on are left as
 * they are, and no offset leads outside [0, M) (where offsets run backwards, what
 * rows hold is undefined). offsets NULL (groups = 1): one
 * matrix for all M rows. Products are exact and sums fp32, as the tensor cores add: cut
 * toward zero, not rounded (off by 5e-6 of the result at K = 4096 of random operands, less
 * in proportion for smaller K; rounded sums are off by 1e-7 to 7e-7 there). No row of x reaches another row's
 * result: an infinity or NaN stays in its row. y is bf16, f16 or fp32 and
 * overlaps no input. groups <= 512, M, N and K <= 2^24, groups * N < 2^31.
 *
 * moe_grouped_linear: x and W of one type, bf16 or f16; K a multiple of 8, x
 * 16-byte aligned with a stride that is a multiple of 8, W [groups, N, K]
 * 16-byte aligned.
 * moe_linear_fp4: x and W in 4-bit floats of one format, as above, K as there;
 * block products and their scales are exact, and the product of x's
 * and W's g, formed in fp32, multiplies their sums. With x the rows are first quantised
 * as moe_quantize_fp4 does. */
typedef struct {
    moe_dtype type;
    int groups, M, N, K;
    const int32_t *offsets;
    const void *x;       /* [M, K] */
    int64_t x_stride;
    const void *w;       /* [groups, N, K] */
    const float *bias;   /* [groups, N] fp32 or NULL */
    void *y;             /* [M, N] */
    moe_dtype y_type;
    int64_t y_stride;
} moe_grouped_linear_args;
moe_status moe_grouped_linear(const moe_grouped_linear_args *args, void *stream);

typedef struct {
    moe_fp4_fmt fmt;
    int groups, M, N, K;
    const int32_t *offsets;
    const void *x;           /* NULL, or [M, K] to be quantised first, into xq, xs and xg */
    int64_t x_stride;
    moe_dtype x_type;        /* bf16 or f16 */
    uint8_t *xq, *xs;        /* [M, K/2], [M, K/16 or K/32] */
    float *xg;               /* NVFP4: [M] or, without x, NULL (1) */
    const uint8_t *wq, *ws;  /* [groups, N, K/2], [groups, N, K/16 or K/32] */
    const float *wg;         /* NVFP4: [groups], with wg_cols [groups, N], or NULL (1) */
    int wg_cols;
    const float *bias;       /* [groups, N] fp32 or NULL */
    void *y;                 /* [M, N] */
    moe_dtype y_type;
    int64_t y_stride;
} moe_linear_fp4_args;
moe_status moe_linear_fp4(const moe_linear_fp4_args *args, void *stream);

/* The waits inside these products are bounded (1.5 s). Where one runs out the
 * call leaves NaN in the rows concerned and sets a bit that belongs to the
 * device, not to the call. moe_products_status waits for `stream`, then reads
 * and clears the current device's: MOE_OK or MOE_ERR_TIMEOUT. A bit that is set
 * meanwhile by work on another stream is kept for the next call. Not while the
 * stream is being captured. */
moe_status moe_products_status(void *stream);

/* Test hook: the products launched while hold is 1 copy no operands, so that
 * their waits run out; while it is 2, every second CTA copies none. No GPU work. */
moe_status moe_debug_hold_products(int hold);

moe_status moe_layer_destroy(moe_layer *layer);

const char *moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
