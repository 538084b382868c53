/*
 * moe.h -- C ABI of the MI355X (gfx950) local MoE expert layer.
 *
 * One expert-parallel rank's local expert compute, taken from the DeepEP-style
 * non-expand layout that GitHub issue #68 on Dao-AILab/sonic-moe ("End-to-end
 * DeepEP v2 non-expand + SonicMoE integration") describes:
 *   x [N,H], topk_idx [N,K] (local expert id, -1 = invalid slot),
 *   topk_weights [N,K]  ->  local_out [N,H],
 * with the routing metadata built directly from [N,K] on the device (no host
 * sync, no materialised [P] pair list), a gathered grouped up-projection GEMM
 * with fused SwiGLU, a grouped down-projection GEMM, a deterministic
 * router-weighted combine, and the backward pass including the router-weight
 * gradient in [N,K] layout (question 4 of that issue).
 *
 * Memory and ownership
 *  - Every tensor pointer is a DEVICE pointer; the caller allocates and owns all
 *    memory (inputs, outputs, metadata arrays, workspace). No call allocates,
 *    frees, synchronises, or reads device memory on the host.
 *  - Every call only enqueues kernels on `stream` (a hipStream_t; NULL is the
 *    null stream) and returns; results are ready when the stream reaches them.
 *  - Tensors are dense and row-major. Index arrays are int32.
 *
 * Errors
 *  - Argument errors (null required pointer, bad sizes, short workspace,
 *    unsupported shape or dtype) are returned synchronously, before anything is
 *    enqueued. A launch failure returns MOE_EHIP.
 *  - Data errors never abort: they set bits in meta->status on the device
 *    (MOE_DEV_*), which the caller reads whenever it next synchronises.
 *    An expert id outside [-1,E) is treated as -1. If the pair count P exceeds
 *    meta->capacity, metadata entries at positions >= capacity are dropped and
 *    forward/backward write zeros to out, dx, dw_up, dw_down, d_topk_weights.
 *
 * Concurrency: calls that share a workspace or metadata object must be ordered
 * on one stream.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_EINVAL = 1,       /* bad argument */
  MOE_ENOSPC = 2,       /* workspace smaller than the matching *_workspace() query */
  MOE_EUNSUPPORTED = 3, /* shape/dtype/layout this library does not implement */
  MOE_EHIP = 4          /* a HIP launch failed */
} moe_status;

/* Element type of x, weights, saved activations, outputs and gradients.
 * topk_weights, router_scores and d_topk_weights are always fp32. */
typedef enum {
  MOE_BF16 = 0, /* bf16 storage, fp32 accumulation (matrix cores) */
  MOE_FP32 = 1  /* fp32 storage and arithmetic: the checking mode */
} moe_dtype;

/* Column order of W_up [E,H,2I] (and of dW_up):
 *  INTERLEAVED: column 2j = gate_j, 2j+1 = up_j (the Hysen Labs page on SonicMoE: the
 *               interleaved format is the default);
 *  CONCAT:      columns [0,I) = gates, [I,2I) = ups (the concatenated gate/up format of
 *               HF-style checkpoints that page contrasts it with).
 * The saved activation h_save is always stored interleaved: it is written by the
 * forward and read only by the backward of this library. */
typedef enum { MOE_GATEUP_INTERLEAVED = 0, MOE_GATEUP_CONCAT = 1 } moe_gateup_layout;

/* Device status bits, OR-ed into *meta->status (zeroed by moe_build_metadata). */
enum { MOE_DEV_BAD_EXPERT = 1u, MOE_DEV_OVER_CAPACITY = 2u };

/* Limits of this library (checked synchronously). */
enum { MOE_MAX_EXPERTS = 1024, MOE_MAX_TOPK = 64 };

/* Routing metadata (GitHub issue #68, the list of arrays SonicMoE's grouped GEMM
 * needs). A host struct holding device pointers, all caller-owned.
 * Pairs are the valid slots of topk_idx taken token-major, ascending slot k
 * within a token; q in [0,P) is that pair index. Sorted position s in [0,P)
 * orders pairs by expert, stably (ascending q within an expert). */
typedef struct {
  int32_t N, K, E;  /* rows, slots per row, local experts */
  int32_t capacity; /* length of the [capacity] arrays (pointers may be NULL when
                       0); P <= capacity <= N*K (pass DeepEP's total_pairs) */
  int32_t *expert_frequency;        /* [E]   pairs per expert */
  int32_t *expert_frequency_offset; /* [E+1] exclusive scan; [E] = P */
  int32_t *x_gather_idx;            /* [capacity] s -> token row of x */
  int32_t *s_scatter_idx;           /* [capacity] s -> pair q */
  int32_t *s_reverse_scatter_idx;   /* [capacity] q -> s */
  int32_t *num_activated_expert_per_token_offset; /* [N+1] exclusive scan of
                                                     valid slots per row; [N] = P */
  float *router_scores;             /* [capacity] q -> topk_weights[t,k] */
  uint32_t *status;                 /* [1] MOE_DEV_* bits */
} moe_metadata;

/* Workspace byte counts. Zero means no workspace is needed. */
size_t moe_build_metadata_workspace(int32_t N, int32_t K, int32_t E);
size_t moe_route_workspace(int32_t N, int32_t K, int32_t E);
size_t moe_expert_forward_workspace(const moe_metadata *meta, int32_t H, int32_t I,
                                    moe_dtype dt);
size_t moe_expert_backward_workspace(const moe_metadata *meta, int32_t H, int32_t I,
                                     moe_dtype dt);

/* Builds every array of *meta from topk_idx [N,K] (int32) and topk_weights [N,K]
 * (fp32), and zeroes-then-sets meta->status. The pair count P stays on the
 * device (expert_frequency_offset[E] and num_activated_expert_per_token_offset[N]).
 * Steps: per-block expert histograms (LDS counters), a cross-block scan, then a
 * stable counting-sort scatter ranked inside wavefronts (Qwen3.6 serving-script notes,
 * "Optimization (CCCL segmented-sort pattern)", steps 1-3).
 * Requires 1 <= K <= MOE_MAX_TOPK, 1 <= E <= MOE_MAX_EXPERTS, N >= 0,
 * N*K < 2^31, 0 <= capacity. */
moe_status moe_build_metadata(const int32_t *topk_idx, const float *topk_weights,
                              const moe_metadata *meta, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Allocation-free variant of moe_build_metadata, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc). Same arguments without the workspace, same kernels and the same
 * results: the workspace is a library-owned static device array of
 * MOE_NOALLOC_SCRATCH_BYTES on each GPU (held until the process ends), on the GPU
 * current for the calling thread (the stream must belong to it). A build whose
 * workspace would exceed that (moe_build_metadata_workspace(N, K, E) >
 * MOE_NOALLOC_SCRATCH_BYTES) returns MOE_ENOSPC before anything is enqueued; argument
 * errors as for moe_build_metadata; MOE_EHIP if the array's address cannot be found.
 * Allocates and frees nothing. Every call on one GPU shares that GPU's array, which
 * keeps the last call's contents (no part of it needs to start zeroed): calls that
 * overlap on one GPU (other streams, or unordered host threads) race on it and must
 * not be issued; calls ordered on one stream are safe. */
enum { MOE_NOALLOC_SCRATCH_BYTES = 4 << 20 };
moe_status moe_build_metadata_noalloc(const int32_t *topk_idx, const float *topk_weights,
                                      const moe_metadata *meta, void *stream);

/* Router top-K from logits, fused with the metadata build (the Hysen Labs page on
 * Dao-AILab/sonic-moe, section "Three routing strategies, selected on the command
 * line": softmax over the top-K logits, or top-K over the softmax of all experts with
 * optional renormalisation; the layer also returns an auxiliary load-balancing loss).
 *  logits        [N,E] bf16 or fp32 (logits_dtype), N, K, E taken from *meta; K <= E.
 *  topk_idx      [N,K] int32 out: per token the K experts with the largest logits,
 *                largest first; equal logits go to the lower expert id.
 *  topk_weights  [N,K] fp32 out: MOE_ROUTE_SOFTMAX_TOPK: exp(l_k) / sum over the K;
 *                MOE_ROUTE_TOPK_SOFTMAX: exp(l_k) / sum over all E, divided by the
 *                sum of the K when renormalize != 0.
 *  aux_loss      [1] fp32 out or NULL: E * sum_e f_e * P_e, f_e = share of the N*K
 *                slots routed to e, P_e = mean over tokens of the softmax over all E
 *                at e (0 when N = 0).
 *  meta          filled exactly as moe_build_metadata(topk_idx, topk_weights) would.
 * Device pointers, caller-owned; workspace >= moe_route_workspace(N, K, E). Errors as
 * for moe_build_metadata (MOE_EINVAL also when K > E); only enqueues on stream. */
typedef enum { MOE_ROUTE_SOFTMAX_TOPK = 0, MOE_ROUTE_TOPK_SOFTMAX = 1 } moe_route_mode;
moe_status moe_route(const void *logits, moe_dtype logits_dtype, moe_route_mode mode,
                     int32_t renormalize, int32_t *topk_idx, float *topk_weights,
                     float *aux_loss, const moe_metadata *meta, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Forward (issue #68 dataflow: native non-expand metadata + local expert
 * compute -> local_out [N_recv,H]). For sorted position s of expert e, token t:
 *   h[s,:]  = x[t,:] W_up[e]                     (W_up [E,H,2I], interleaved)
 *   a[s,j]  = silu(h[s,2j]) * h[s,2j+1]          (SwiGLU, no bias)
 *   y[s,:]  = a[s,:] W_down[e]                   (W_down [E,I,H])
 *   out[t,:] = sum over the token's pairs q, ascending, of
 *              router_scores[q] * y[s_reverse_scatter_idx[q],:]   (fp32 sum)
 * Rows with no valid slot are 0. h_save [capacity,2I] (same dtype) receives h
 * for the backward; pass NULL for inference. out is [N,H].
 * H and I must be positive multiples of 8 (whole 16-byte bf16 chunks), at most
 * 2^20; other sizes return MOE_EUNSUPPORTED. Sizes that are not multiples of the
 * 128-wide tiles run with partial edge tiles. */
moe_status moe_expert_forward(const moe_metadata *meta, const void *x, const void *w_up,
                              const void *w_down, int32_t H, int32_t I, moe_dtype dt,
                              moe_gateup_layout layout, void *h_save, void *out,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Backward of moe_expert_forward for upstream gradient dout [N,H]:
 *   dx [N,H], dw_up [E,H,2I], dw_down [E,I,H] (same dtype as x; fully
 *   overwritten, exact zeros for experts with no rows), and
 *   d_topk_weights [N,K] fp32 = <dout[t], y[s]> at every valid slot, 0 at
 *   invalid slots (issue #68, question 4: gradients for routing scores returned
 *   in [N_recv,K] layout).
 * h_saved is the h_save written by the forward with the same metadata.
 * topk_idx is the [N,K] array the metadata was built from. H and I as for the
 * forward. */
moe_status moe_expert_backward(const moe_metadata *meta, const int32_t *topk_idx,
                               const void *x, const void *w_up, const void *w_down,
                               const void *h_saved, const void *dout, int32_t H, int32_t I,
                               moe_dtype dt, moe_gateup_layout layout, void *dx, void *dw_up,
                               void *dw_down, float *d_topk_weights, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ---- 8-bit operands with a scale for each block of 128 --------------------------
 * The expert layer on e4m3 operands (the OCP 8-bit format with 4 exponent and 3
 * mantissa bits, largest value 448, no infinities), with what a program needs ahead of
 * it: an RMS norm that hands its output on in 8 bits, and the quantisation of rows and
 * of weights.
 *
 * Blocks and scales. Rows of activations have one scale per MOE_QBLOCK consecutive
 * values (the last block of a row may be shorter); weights one per block of
 * MOE_QBLOCK x MOE_QBLOCK. A value stands for e4m3 * scale. Scale tensors are dense:
 * [rows, ceil(L/128)] and [E, ceil(out/128), ceil(in/128)].
 *  MOE_SCALE_FP32: fp32 scales. The products take any positive finite ones (those of a
 *                  checkpoint, or of a dispatch); scale products are formed in fp32, so
 *                  the product of a row's and a weight's scale has to be a normal number.
 *  MOE_SCALE_E8M0: one byte b for the power of two 2^(b-127), 0 <= b <= 254 (255 is NaN).
 * The scales this library writes are powers of two in either form: the least s with
 * max|v| <= 448 s over the block's finite values, at least 2^-126. Quotients v/s are
 * then exact, and each value is rounded once: to nearest, ties to even. A value that is
 * not finite becomes NaN (and nothing else in its block changes).
 * e4m3 rows and weights need lengths that are multiples of 16 in the products.
 *
 * Addresses. Tensors and workspaces of these calls start at multiples of 16 bytes (what
 * moe_quantize_rows and the norm write as q: of 8), fp32 scales and rstd of 4, e8m0 scales
 * anywhere; MOE_EINVAL otherwise. Sizes. MOE_EUNSUPPORTED where one launch does not hold
 * the work: N ceil(H/128) from 2^28 on in moe_quantize_rows, E ceil(K/128) ceil(C/128) from
 * 2^24 on in moe_quantize_weights, 2^23 tiles in the products. Apart from the outputs that are said to be allowed in the
 * place of an input, outputs and inputs do not overlap. */
typedef enum { MOE_SCALE_FP32 = 0, MOE_SCALE_E8M0 = 1 } moe_scale_type;
enum { MOE_QBLOCK = 128 };

/* Rows in 8 bits: x [N,H] (dt) -> q [N,H] e4m3, scale [N, ceil(H/128)]. H a positive
 * multiple of 8 up to 2^20. */
moe_status moe_quantize_rows(const void *x, int32_t N, int32_t H, moe_dtype dt, void *q,
                             void *scale, moe_scale_type scale_type, void *stream);

/* Weights in 8 bits, transposed for the products: w [E,K,C] (dt, as moe_expert_forward
 * takes W_up and W_down: K in, C out) -> q [E,C,K] e4m3, scale [E, ceil(C/128),
 * ceil(K/128)]. K and C positive multiples of 16 up to 2^20 (C: 2^21). */
moe_status moe_quantize_weights(const void *w, int32_t E, int32_t K, int32_t C, moe_dtype dt,
                                void *q, void *scale, moe_scale_type scale_type,
                                void *stream);

/* RMS norm with the residual's addition:
 *   r = x + residual, rounded to dt (r = x when residual is NULL);
 *   rstd = 1 / sqrt(mean(r^2) + eps);  y = r * rstd * weight.
 * x, residual, residual_out [N,H], weight [H] in dt. residual_out receives r (required
 * with a residual, NULL without; it may be x or residual itself). y [N,H] (dt), or NULL;
 * q [N,H] e4m3 with scale [N, ceil(H/128)], or NULL; one of the two at least. Both are
 * rounded from the unrounded fp32 y. rstd [N] fp32, or NULL (the backward takes it).
 * H a positive multiple of 8 up to 2^20; eps >= 0. Squares and sums are fp32, in a fixed
 * order (|r| from 2^63 on overflows them: y is 0 there). */
moe_status moe_rmsnorm_forward(const void *x, const void *residual, const void *weight,
                               float eps, int32_t N, int32_t H, moe_dtype dt,
                               void *residual_out, void *y, void *q, void *scale,
                               moe_scale_type scale_type, float *rstd, void *stream);

/* Backward of moe_rmsnorm_forward for dy [N,H], the gradient of y (and, with the rounding
 * to 8 bits taken as the identity, of the values q stands for), and dresidual [N,H], that
 * of residual_out from its other readers (NULL: none). r is residual_out (x without a
 * residual), rstd as written by the forward:
 *   g = dy * weight;  dx = rstd * (g - r * rstd^2 * mean(g * r)) + dresidual;
 *   dweight = sum over the rows of dy * r * rstd.
 * dx [N,H] is the gradient of x and of residual alike (it may be dresidual or dy itself);
 * dweight [H]; both in dt, fully overwritten (dweight zeros when N = 0). Sums are fp32 in
 * a fixed order. workspace >= moe_rmsnorm_backward_workspace(N, H). */
size_t moe_rmsnorm_backward_workspace(int32_t N, int32_t H);
moe_status moe_rmsnorm_backward(const void *dy, const void *r, const void *weight,
                                const float *rstd, const void *dresidual, int32_t N, int32_t H,
                                moe_dtype dt, void *dx, void *dweight, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Matrix products grouped by expert on e4m3 operands: for the sorted positions s of
 * expert e (expert_frequency_offset[e] <= s < expert_frequency_offset[e+1])
 *   out[s,:] = a[row(s),:] W_e^T,   row(s) = x_gather_idx[s] if gather, else s.
 * a [N,K] (gather) or [capacity,K] e4m3, a_scale [rows, ceil(K/128)]; w [E,C,K] e4m3,
 * w_scale [E, ceil(C/128), ceil(K/128)]; out [capacity,C] bf16. Sums are fp32, but for
 * what the matrix cores do with 8-bit operands: of eight products next to each other along
 * K, each is cut off 2^13 below the largest one's power of two before they are added (with
 * operands rounded from normal values about 1.6e-5 of the result, 1/100 of the rounding to
 * bf16; nothing where the values of a block of 8 span at most four powers of two). Rows of
 * out at positions >= P are left as they were; if P > capacity nothing is written. K and C
 * positive multiples of 16 up to 2^20 (C: 2^21). */
moe_status moe_grouped_gemm_fp8(const moe_metadata *meta, const void *a, const void *a_scale,
                                moe_scale_type a_scale_type, const void *w,
                                const void *w_scale, moe_scale_type w_scale_type, int32_t K,
                                int32_t C, int32_t gather, void *out, void *stream);

/* moe_expert_forward on e4m3 operands: x [N,H] with x_scale [N, ceil(H/128)]; w_up
 * [E,2I,H] (rows in the order `layout` gives W_up's columns) and w_down [E,H,I], each
 * row a column of moe_expert_forward's, with their block scales (both of w_scale_type).
 *   h = x W_up_e^T;  a = silu(gate) * up, in e4m3 with a power-of-two scale per 128
 *   values of a row;  y = a W_down_e^T;  out = sum of router_scores * y  (bf16).
 * Sums as in moe_grouped_gemm_fp8; the 8-bit a is rounded from unrounded h; y is kept in
 * fp16 with a power of two per row and 64 columns (few rows: fp32). What the cut-off moves of
 * h moves some a past a tie of its 8 bits: 0.1 to 0.3% of out altogether (few rows: none, their
 * products are not cut off). h_save
 * [capacity,2I] bf16, interleaved, or NULL: moe_expert_backward takes it, with the bf16
 * x and weights that the 8-bit ones stand for (the rounding to 8 bits taken as the
 * identity). out is [N,H] bf16, 0 in rows with no valid slot, all 0 if P > capacity.
 * H and I: positive multiples of 16, at most 2^20. */
size_t moe_expert_forward_fp8_workspace(const moe_metadata *meta, int32_t H, int32_t I);
moe_status moe_expert_forward_fp8(const moe_metadata *meta, const void *x, const void *x_scale,
                                  moe_scale_type x_scale_type, const void *w_up,
                                  const void *w_up_scale, const void *w_down,
                                  const void *w_down_scale, moe_scale_type w_scale_type,
                                  int32_t H, int32_t I, moe_gateup_layout layout,
                                  void *h_save, void *out, void *workspace,
                                  size_t workspace_bytes, void *stream);

const char *moe_status_string(moe_status s);

/* ---- Diagnostics: per-kernel timing with caller-created events ---------------
 * The kernels the calls enqueue, in launch order. */
typedef enum {
  MOE_KERNEL_META_HIST = 0,    /* moe_build_metadata: per-chunk expert histograms
                                  (above 2048 slots) */
  MOE_KERNEL_META_SCAN = 1,    /* moe_build_metadata: prefixes over chunks, totals
                                  (above 256 chunks of 512 slots or 34 experts) */
  MOE_KERNEL_META_SCATTER = 2, /* moe_build_metadata: offsets + stable scatter (up to
                                  2048 slots: the whole build, counts included) */
  MOE_KERNEL_UP_SWIGLU = 3,    /* forward: gathered up-projection + SwiGLU */
  MOE_KERNEL_DOWN = 4,         /* forward: down projection */
  MOE_KERNEL_COMBINE = 5,      /* forward: weighted combine to [N,H] */
  MOE_KERNEL_DOWN_BWD = 6,     /* backward: dout_g W_down^T + dSwiGLU + dscore partials */
  MOE_KERNEL_WGRAD_DOWN = 7,   /* backward: dW_down */
  MOE_KERNEL_UP_BWD = 8,       /* backward: dh W_up^T */
  MOE_KERNEL_WGRAD_UP = 9,     /* backward: dW_up */
  MOE_KERNEL_COMBINE_DX = 10,  /* backward: dx = sum over the token's rows, and
                                  d_topk_weights in [N,K] */
  MOE_KERNEL_ROUTE = 11,       /* moe_route: top-K, weights, histograms, P sums
                                  (then META_SCAN and META_SCATTER, which also form the
                                  load-balancing loss) */
  MOE_KERNEL_QUANT_ROWS = 12,    /* moe_quantize_rows; moe_expert_forward_fp8 with few rows
                                    per expert */
  MOE_KERNEL_QUANT_WEIGHTS = 13, /* moe_quantize_weights */
  MOE_KERNEL_RMSNORM = 14,       /* moe_rmsnorm_forward */
  MOE_KERNEL_RMSNORM_BWD = 15,   /* moe_rmsnorm_backward: dx and partial sums of dweight */
  MOE_KERNEL_RMSNORM_DW = 16,    /* moe_rmsnorm_backward: dweight */
  MOE_KERNEL_GROUPED_FP8 = 17,   /* moe_grouped_gemm_fp8 */
  MOE_KERNEL_UP_SWIGLU_FP8 = 18, /* moe_expert_forward_fp8: up-projection + SwiGLU, in 8 bits */
  MOE_KERNEL_DOWN_FP8 = 19,      /* moe_expert_forward_fp8: down projection (then COMBINE) */
  MOE_KERNEL_COUNT = 20
} moe_kernel_id;

/* After this call, the i-th launch of `kernel` (i < n_launches, counted from this
 * call) made by the calling host thread is bracketed by hipEventRecord(events[2i])
 * just before it and hipEventRecord(events[2i+1]) just after it, on the launch's
 * stream. events holds 2*n_launches hipEvent_t created by the caller (none NULL,
 * else MOE_EINVAL); events == NULL stops recording. The hook is per host thread:
 * launches made by other threads are never bracketed and never touch it. For
 * benchmarks only. Returns the number of launches bracketed since the previous call
 * (from this thread) through *n_recorded (may be NULL). */
moe_status moe_time_kernel(moe_kernel_id kernel, void *const *events, int32_t n_launches,
                           int32_t *n_recorded);
const char *moe_kernel_name(moe_kernel_id kernel);

#ifdef __cplusplus
}
#endif
#endif
