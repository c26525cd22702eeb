/*
 * moe.h -- C ABI of the MI355X (gfx950) DeepSeekMoE layer forward with
 * auxiliary-loss-free (bias) routing.
 *
 * The layer, as the pages state it:
 *   - DeepSeek V3 From Scratch, "The idea": 256 routed experts plus one shared
 *     expert that every token uses; each token goes to its top 8 routed
 *     experts; a per-expert bias, added to the router affinity, steers which
 *     experts are chosen, while the combine weights come from the unbiased
 *     affinities; the bias is a control loop, not a loss term.
 *   - DeepSeek V3 From Scratch, "Worked example" (routing, concretely) and
 *     "In code" (route, update_bias): sigmoid affinities, top-k of affinity
 *     plus bias, the chosen k unbiased affinities renormalised to sum to 1,
 *     and bias <- bias + step * sign(target - load).
 *   - kbwen.com DeepSeek feed, "A bias term for each expert": the bias moves
 *     once per step, from the load over the whole batch, by the same fixed
 *     amount (0.001) up or down; no token is dropped.
 *   - Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture,
 *     "Implementation: A Modular Look": the output is the shared expert's
 *     output plus, for each routed expert, its output on the tokens that
 *     chose it scaled by their weight.
 *   - crackai.dev DeepSeek-V3 summary, "How It Works": the routed work is
 *     split into a dispatch and a combine around the expert computation; FP8
 *     expert matmuls with a scale per tile and FP32 accumulation.
 * Our readings where the pages are silent: each expert is a bias-free SwiGLU
 * FFN y = W_down (silu(W_gate a) * (W_up a)); equal biased scores go to the
 * lower expert id; the k chosen ids are reported in ascending order.
 *
 * Conventions for every call:
 *   - Tensors are row-major and contiguous, in device memory owned by the
 *     caller.  The library never allocates, frees or synchronises, and never
 *     reads device memory on the host.  Work is enqueued on `stream` (a
 *     hipStream_t; NULL is the default stream) and the call returns.
 *   - Arguments are validated on the host before anything is launched:
 *     MOE_EINVAL for a null required pointer, non-positive sizes, k > E, or
 *     d / I not multiples of 128 with e4m3; MOE_ENOTSUP for shapes the library
 *     does not cover (E != 256, k != 8, d or I not a multiple of 64, d not a
 *     multiple of 128 with bf16 weights, T * k >= 2^31 routed rows (their
 *     indices are int32), an unsupported dtype pair); MOE_EWORKSPACE when
 *     ws_bytes is below
 *     moe_workspace_bytes(); MOE_ESCRATCH when moe_dispatch_noalloc gets
 *     more tokens than its static scratch holds; MOE_EHIP when a launch
 *     reports an error.
 *     Device faults surface at the caller's next synchronisation.
 *   - No C++ exception crosses the ABI; the library never aborts.
 *   - Calls are stateless and re-entrant (moe_dispatch_noalloc aside: its
 *     calls share one static scratch per GPU); calls on different streams
 *     that share output buffers race, as with any kernel launch.
 *
 * Storage types (moe_dtype_t): fp32; bf16 as 16-bit patterns (upper half of
 * binary32); e4m3 as OCP FP8 E4M3FN bytes, each 1x128 activation tile and
 * 128x128 weight block with one scale stored as an OCP MX E8M0 byte: byte e
 * stands for 2^(e-127) (e = 0 .. 254), so a scale is a power of two by
 * construction; 255 is the format's NaN, and every output that a tile or
 * block with that byte feeds comes out NaN.  The block-scaled MFMA of gfx950
 * takes these bytes as they are.  Supported
 * (act, wt) pairs: (F32, F32), (BF16, BF16), (BF16, E4M3).  The router is
 * always fp32.
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
    MOE_EINVAL = 1,
    MOE_ENOTSUP = 2,
    MOE_EWORKSPACE = 3,
    MOE_EHIP = 4,
    MOE_ESCRATCH = 5  /* moe_dispatch_noalloc: more tokens than its static scratch holds */
} moe_status_t;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2 } moe_dtype_t;

/* Shape of one layer call.  T tokens, model width d, E routed experts, top-k,
 * expert intermediate width I.  act: storage type of x.  wt: storage type of
 * the expert weights, which is also the type the expert GEMMs read their
 * activations in (x_perm and the intermediate h). */
typedef struct {
    int32_t T, d, E, k, I;
    int32_t act;
    int32_t wt;
} moe_desc_t;

/* Weights of a stack of G SwiGLU experts (G = E routed, or G = 1 shared):
 * gate, up: [G, I, d]; down: [G, d, I] (each row contiguous along the reduced
 * dimension).  For e4m3 the scales hold one E8M0 byte per 128x128 block:
 * s_gate, s_up: [G, I/128, d/128]; s_down: [G, d/128, I/128]; the value of an
 * element is code * 2^(s - 127).  Scales are NULL for fp32 and bf16. */
typedef struct {
    const void *gate, *up, *down;
    const uint8_t *s_gate, *s_up, *s_down;
} moe_ffn_weights_t;

/* Workspace stages for moe_workspace_bytes. */
enum {
    MOE_WS_DISPATCH = 0, MOE_WS_FFN = 1, MOE_WS_COMBINE = 2, MOE_WS_ROUTE = 3, MOE_WS_BACKWARD = 4,
    MOE_WS_ROUTER_LOGITS = 5, MOE_WS_ROUTER_GRAD = 6, MOE_WS_BACKWARD_SAVED = 7
};

/*
 * Router, biased top-k choice and combine weights (DeepSeek V3 From Scratch,
 * "In code": route; "Worked example").
 *   x        [T, d]  act type
 *   w_router [E, d]  fp32; logit of expert e = x_t . w_router[e]
 *   bias     [E]     fp32 balancing bias (read only)
 *   idx      [T, k]  int32 out: the k experts with the largest
 *                    fl32(sigmoid(logit)) + bias, ascending id order; equal
 *                    scores go to the lower id
 *   weights  [T, k]  fp32 out: sigmoid(logit) of each chosen expert divided by
 *                    the sum over the k chosen (bias not included)
 *   gap      [T]     fp32 out or NULL: k-th minus (k+1)-th largest biased
 *                    score, as the kernel computed it
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_ROUTE) bytes of device memory
 *                    (0 for fp32 activations; NULL allowed then)
 * All scores are computed in fp32: the logit is an fp32 accumulation of
 * exact products (bf16 x times the fp32 router split exactly into three bf16
 * terms, or fp32 x times fp32 w).
 */
moe_status_t moe_route(const moe_desc_t *desc, const void *x, const float *w_router,
                       const float *bias, int32_t *idx, float *weights, float *gap,
                       void *workspace, size_t ws_bytes, void *stream);

/*
 * Dispatch: per-expert load, its prefix sum and a stable grouping of the T*k
 * (token, slot) assignments by expert, with the token rows gathered into that
 * order (crackai.dev DeepSeek-V3 summary, "How It Works": dispatch; Scaling
 * Efficiency ..., "Implementation: A Modular Look": each expert sees the
 * tokens that chose it).  Every assignment is kept: no capacity, no drops
 * (kbwen.com DeepSeek feed, "A bias term for each expert").
 *   idx          [T, k]   int32 from moe_route (ids in [0, E), distinct per token; an id
 *                         outside [0, E) is not dispatched: it takes no row, its row_of
 *                         entry is -1 and offsets[E] falls short of T*k by the number
 *                         of such ids; the later calls need a complete dispatch)
 *   x            [T, d]   act type
 *   counts       [E]      int32 out: assignments per expert (the load)
 *   offsets      [E+1]    int32 out: exclusive prefix sum of counts; offsets[E] = T*k
 *   row_src      [T*k]    int32 out: flat assignment id t*k + j of permuted row r;
 *                         within an expert rows are in ascending t*k + j order
 *   row_of       [T*k]    int32 out: the inverse, permuted row of assignment t*k + j
 *   x_perm       [T*k, d] out, in the expert GEMM input type: row r = x[row_src[r] / k];
 *                         for e4m3 the row is quantised per 1x128 tile:
 *   x_perm_scale [T*k, d/128] E8M0 bytes out (e4m3 only, else NULL): scale = the
 *                         smallest power of two at or above amax/448 (the fp32
 *                         quotient; 1 for an all-zero tile), code =
 *                         e4m3_rne_sat(v / scale)
 *   workspace    >= moe_workspace_bytes(desc, MOE_WS_DISPATCH) bytes of device memory
 * x_perm may be NULL: then only counts, offsets, row_src and row_of are
 * written (x and x_perm_scale are not read), for moe_expert_gate_up_rows,
 * which gathers the rows itself.
 * Integer outputs are bit-exact and deterministic (no atomics decide order).
 */
moe_status_t moe_dispatch(const moe_desc_t *desc, const int32_t *idx, const void *x,
                          int32_t *counts, int32_t *offsets, int32_t *row_src, int32_t *row_of,
                          void *x_perm, uint8_t *x_perm_scale, void *workspace, size_t ws_bytes,
                          void *stream);

/*
 * moe_dispatch for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments (minus the workspace) and the same outputs, bit for bit;
 * the per-block count table lives in a static device array of the library
 * instead (4 MiB on each GPU the library runs on, held until the process
 * ends), so T is limited to 1048576 tokens: MOE_ESCRATCH above that, checked
 * before anything is launched.  The array's device address is looked up on
 * the first call on each device (MOE_EHIP if that fails).  No allocation or
 * free happens in any call.  Every call on one GPU uses the same array:
 * calls that overlap in time on one GPU (several streams or host threads)
 * race and must be serialised by the caller.  Each call overwrites every
 * entry it reads, so nothing carries over from an earlier call.
 */
moe_status_t moe_dispatch_noalloc(const moe_desc_t *desc, const int32_t *idx, const void *x,
                                  int32_t *counts, int32_t *offsets, int32_t *row_src, int32_t *row_of,
                                  void *x_perm, uint8_t *x_perm_scale, void *stream);

/*
 * Routed expert FFNs, grouped: rows [offsets[e], offsets[e+1]) of x_perm go
 * through expert e (DeepSeek V3 From Scratch, "The idea": fine-grained routed
 * experts; crackai.dev DeepSeek-V3 summary, "How It Works": FP8 matmuls with
 * per-tile scales and FP32 accumulation).
 *   h = silu(x_perm W_gate[e]^T) * (x_perm W_up[e]^T), fp32 accumulation,
 *       rounded to the wt type (bf16; or e4m3 per 1x128 tile with an E8M0
 *       scale, as in moe_dispatch; or fp32), kept in the workspace;
 *   y_perm = h W_down[e]^T, fp32 accumulation, stored as fp32 (wt = F32) or
 *       bf16 (otherwise).
 *   x_perm, x_perm_scale, offsets: from moe_dispatch; offsets are read on the
 *       device only (no host synchronisation).
 *   experts   E routed experts (see moe_ffn_weights_t)
 *   y_perm    [T*k, d] out
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_FFN) bytes of device memory
 */
moe_status_t moe_expert_ffn(const moe_desc_t *desc, const void *x_perm, const uint8_t *x_perm_scale,
                            const int32_t *offsets, const moe_ffn_weights_t *experts,
                            void *y_perm, void *workspace, size_t ws_bytes, void *stream);

/*
 * The two halves of moe_expert_ffn, for callers that schedule or time them
 * separately.  moe_expert_gate_up computes h (kept in `workspace`);
 * moe_expert_down reads h from the same workspace and writes y_perm.  Called
 * in that order on one stream with one workspace they are exactly
 * moe_expert_ffn.  Arguments as for moe_expert_ffn.
 */
moe_status_t moe_expert_gate_up(const moe_desc_t *desc, const void *x_perm, const uint8_t *x_perm_scale,
                                const int32_t *offsets, const moe_ffn_weights_t *experts,
                                void *workspace, size_t ws_bytes, void *stream);
moe_status_t moe_expert_down(const moe_desc_t *desc, const int32_t *offsets,
                             const moe_ffn_weights_t *experts, void *y_perm, void *workspace,
                             size_t ws_bytes, void *stream);

/*
 * moe_expert_gate_up with the dispatch gather folded into the GEMM: row r of
 * the grouped GEMM's input is token row_src[r] / k of x, read in place, so no
 * x_perm is materialised (the same rows in the same order as moe_dispatch's
 * x_perm, hence the same h bit for bit).  With wt = e4m3, x is first
 * quantised once per token (T rows, 1x128 tiles, as in moe_dispatch) into the
 * workspace.
 *   x         [T, d] act type (the layer input given to moe_dispatch)
 *   row_src   [T*k]  int32 from moe_dispatch (flat assignment ids t*k + j;
 *             row r of the GEMM reads token row_src[r] / k)
 *   offsets, experts, workspace: as for moe_expert_gate_up
 * Then moe_expert_down as usual.
 */
moe_status_t moe_expert_gate_up_rows(const moe_desc_t *desc, const void *x, const int32_t *row_src,
                                     const int32_t *offsets, const moe_ffn_weights_t *experts,
                                     void *workspace, size_t ws_bytes, void *stream);

/*
 * Shared expert plus weighted combine (Scaling Efficiency ..., "Implementation:
 * A Modular Look": shared output plus the routed outputs scaled by their
 * weights; DeepSeek V3 From Scratch, "The idea": one shared expert for every
 * token).
 *   y[t] = shared(x[t]) + sum_{j<k} weights[t, j] * y_perm[row_of[t*k + j]]
 * with the j-sum in ascending expert-id order, in fp32; the shared expert's
 * fp32 accumulator is not rounded before the sum (at small T with bf16
 * weights its K range is split over workgroups and the fp32 partial sums are
 * added in a fixed order, so the result is still deterministic).  The shared expert has the
 * SwiGLU form of the routed ones; with wt = e4m3 its input is x quantised per
 * 1x128 tile (as in moe_dispatch) inside the workspace.
 *   x        [T, d] act type
 *   shared   one expert (G = 1)
 *   y_perm, row_of, weights: from moe_expert_ffn, moe_dispatch, moe_route
 *   y        [T, d] fp32 out
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_COMBINE) bytes of device memory
 */
moe_status_t moe_combine(const moe_desc_t *desc, const void *x, const moe_ffn_weights_t *shared,
                         const void *y_perm, const int32_t *row_of, const float *weights,
                         float *y, void *workspace, size_t ws_bytes, void *stream);

/*
 * Sign-step bias update, once per step after the forward (DeepSeek V3 From
 * Scratch, "In code": update_bias; kbwen.com DeepSeek feed, "A bias term for
 * each expert"):  with load_e = counts[e] / T and target = k / E,
 *   bias[e] <- fl32(bias[e] + gamma * sign(target - load_e)),
 * sign(0) = 0.  The sign is evaluated exactly as sign(k*T - E*counts[e]).
 *   counts [E] int32 (from moe_dispatch); bias [E] fp32, updated in place.
 */
moe_status_t moe_bias_update(const moe_desc_t *desc, const int32_t *counts, float gamma,
                             float *bias, void *stream);

/* Device workspace, in bytes, that a call of the given stage needs for this
 * shape (0 when the shape is invalid). */
size_t moe_workspace_bytes(const moe_desc_t *desc, int32_t stage);

/*
 * Backward of the layer: the gradients of the layer output y for the
 * routing the forward chose, given dy = dL/dy (act = bf16 with wt = bf16 or
 * e4m3; other types give MOE_ENOTSUP).  What is differentiated is the forward above
 * (DeepSeek V3 From Scratch, "The idea", "In code"; Scaling Efficiency ...,
 * "Implementation: A Modular Look"):
 *   y = shared(x) + sum_j g_j * y_perm_j,  g_j = s_j / sum_i s_i over the
 *   chosen experts,  s_e = sigmoid(x . w_router[e]).
 * The choice is piecewise constant and carries no gradient; the bias is used
 * only for the choice and gets no gradient (kbwen.com DeepSeek feed, "A bias
 * term for each expert").  Inside: the routed and shared output gradients
 * (g_j dy and dy) and the SwiGLU input gradients are rounded to bf16 as GEMM
 * inputs, like h in the forward; the expert pre-activations are recomputed;
 * accumulation is fp32.  Deterministic (no atomics).
 * With e4m3 weights (crackai.dev DeepSeek-V3 summary, "How It Works": FP8
 * in the backward pass too, a scale per tile) every backward GEMM takes e4m3
 * operands quantised per 1x128 tile along its reduction: row tiles for the
 * data gradients (against the weight blocks, transposed as blocks); for the
 * weight gradients, each column of a group of 128 of an expert's rows
 * (dispatch order; the shared expert: 128 consecutive tokens) is one tile,
 * quantised from the fp32 values and the bf16 x.
 *   x          [T, d] bf16, the forward's input
 *   w_router   [E, d] fp32
 *   idx, weights [T, k]: from moe_route
 *   offsets, row_src, row_of: from moe_dispatch
 *   experts, shared: as for the forward (bf16, or e4m3 with block scales)
 *   y_perm     [T*k, d] bf16: the forward's routed outputs (moe_expert_ffn)
 *   dy         [T, d] fp32
 * Outputs (fp32, written, not accumulated):
 *   dx [T, d]; dw_router [E, d]; dw_gate, dw_up [E, I, d]; dw_down [E, d, I];
 *   ds_gate, ds_up [I, d]; ds_down [d, I] (the shared expert);
 *   dg [T, k] the combine-weight gradients dy . y_perm_j (NULL: not returned).
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_BACKWARD) bytes of device
 *   memory: about (T*k + T)(6d + 18I) for the per-row intermediates, plus
 *   (T*k + 64E + T)(4d + 6I) for their K-contiguous transposes, 64*E*d
 *   for the router partials, and, only where the data-gradient products
 *   cannot read the weights as stored (fewer than 128 rows per expert on
 *   average, or d or I not a multiple of 256), 6(E + 1)*I*d for transposed
 *   weights
 *   (about 17 GiB at T=16384, d=7168, I=2048, E=256, k=8; with e4m3 weights,
 *   which are always transposed as blocks, about 31 GiB).
 * Requires d % 128 == 0 and I % 128 == 0.
 */
moe_status_t moe_backward(const moe_desc_t *desc, const void *x, const float *w_router, const int32_t *idx,
                          const float *weights, const int32_t *offsets, const int32_t *row_src,
                          const int32_t *row_of, const moe_ffn_weights_t *experts,
                          const moe_ffn_weights_t *shared, const void *y_perm, const float *dy, float *dx,
                          float *dw_router, float *dw_gate, float *dw_up, float *dw_down, float *ds_gate,
                          float *ds_up, float *ds_down, float *dg, void *workspace, size_t ws_bytes,
                          void *stream);

/* ------------------------------------------------------------------------
 * Routing from logits: the router's product on its own, the choice of experts
 * by other rules than moe_route's, the loss that balances each sequence, and
 * their gradients.
 * ------------------------------------------------------------------------ */

/*
 * The router's logits alone: logits[t, e] = x_t . w_router[e], fp32, by the
 * arithmetic of moe_route.
 *   x        [T, d]  act type
 *   w_router [E, d]  fp32
 *   logits   [T, E]  fp32 out
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_ROUTER_LOGITS) bytes of
 *            device memory (0 for fp32 activations; NULL allowed then)
 * x and logits are 16-byte aligned, d is below 2^23.
 */
moe_status_t moe_router_logits(const moe_desc_t *desc, const void *x, const float *w_router, float *logits,
                               void *workspace, size_t ws_bytes, void *stream);

/*
 * Its gradient: dx = dx_in + dlogits . w_router, dw_router = dlogits^T . x.
 *   dlogits   [T, E] fp32 (moe_select_backward)
 *   dx_in     [T, d] fp32 or NULL (zero): the other gradients of x, for instance
 *             moe_backward_saved's dx; may be dx itself
 *   dx        [T, d] fp32 out
 *   dw_router [E, d] fp32 out (written, not accumulated)
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_ROUTER_GRAD) bytes
 * x, dlogits, dw_router and the workspace are 16-byte aligned.  fp32's accuracy,
 * relative to the largest of a row of dlogits and of a column of w_router for dx,
 * to the terms themselves for dw_router; a sum that an infinity or a NaN enters is
 * NaN.  Deterministic.
 */
moe_status_t moe_router_logits_backward(const moe_desc_t *desc, const void *x, const float *w_router,
                                        const float *dlogits, const float *dx_in, float *dx, float *dw_router,
                                        void *workspace, size_t ws_bytes, void *stream);

typedef enum { MOE_SIGMOID = 0, MOE_SOFTMAX = 1 } moe_score_t;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP_TWO = 1 } moe_group_score_t;

/* The rule by which k of E experts are chosen for each of T tokens.
 *   score        moe_score_t: s = sigmoid(logit), or softmax over the E logits
 *   n_group      the experts are n_group runs of E / n_group (1: no groups)
 *   topk_group   only the experts of the topk_group best groups can be chosen;
 *                topk_group * (E / n_group) >= k
 *   group_score  moe_group_score_t: a group's score is the largest of its
 *                experts' biased scores, or the sum of the two largest
 *   renorm       1: the weights are divided by their sum over the chosen
 *   scale        factor on the weights
 *   logits       moe_dtype_t of the logits: MOE_F32 or MOE_BF16
 * Any E up to 1024, k up to 64, T below 2^28 and T * k below 2^31. */
typedef struct {
    int32_t T, E, k;
    int32_t score;
    int32_t n_group, topk_group, group_score;
    int32_t renorm;
    float scale;
    int32_t logits;
} moe_select_t;

/*
 * The choice and its combine weights, in one launch (past 2^25 tokens in several,
 * for rules that a wave per token takes).
 *   logits  [T, E], row t at logits + t * ld (ld >= E, in elements)
 *   bias    [E] fp32 or NULL: added to the scores for the choice only
 *   idx     [T, k] int32 out: ids ascending; the k largest s + bias among the
 *           open groups; equal scores, of experts or groups, go to the lower id
 *   weights [T, k] fp32 out: scale * s of each chosen expert, over the sum of
 *           the chosen s with renorm (0 where that sum is 0)
 * The choice is made by the scores in 64 bits (without a bias by the logits
 * themselves, whose order is theirs), the weights are computed in fp32.  A
 * logit of -inf has the score 0; a NaN score ranks behind every number, and
 * a group with fewer than two numbers behind every group with two
 * (MOE_GROUP_TOP_TWO, groups of more than one).  idx always holds k distinct
 * ids in [0, E).
 * With E = 256, k = 8 idx and weights go straight into moe_dispatch and
 * moe_combine.
 */
moe_status_t moe_select(const moe_select_t *sel, const void *logits, int64_t ld, const float *bias, int32_t *idx,
                        float *weights, void *stream);

/*
 * Gradient with respect to the logits, dlogits [T, E] fp32 (written): through
 * the weights, where dweights [T, k] is given, and through the balance loss,
 * where seq_offsets is; at least one of the two.  The choice carries no
 * gradient.
 *   idx          [T, k] from moe_select (distinct in a row; an id outside [0, E)
 *                is skipped); needed with dweights
 *   seq_offsets  [n_seq + 1], load [n_seq, E]: from moe_balance_loss
 *   dloss        [n_seq] fp32: gradient of each sequence's loss
 *   alpha        as for moe_balance_loss
 * Rows outside every sequence get no balance gradient.  Where a formula's gradient is
 * zero whatever the logits, so is dlogits, exactly: one renormalised choice (its weight
 * is the scale), and the loss where k = E (every load is 1, the loss alpha).
 */
moe_status_t moe_select_backward(const moe_select_t *sel, const void *logits, int64_t ld, const int32_t *idx,
                                 const float *dweights, const int32_t *seq_offsets, int32_t n_seq, const float *load,
                                 const float *dloss, float alpha, float *dlogits, void *stream);

/*
 * Sequence-wise balance loss.  Tokens seq_offsets[q] .. seq_offsets[q+1]-1 are
 * sequence q, of n tokens; p_{t,e} = s_{t,e} / sum_i s_{t,i};
 *   load_{q,e} = E / (k n) * (choices of e in q),  P_{q,e} = mean of p_{t,e},
 *   loss_q = alpha * sum_e load_{q,e} P_{q,e}.
 * A balanced sequence has the loss alpha.  load carries no gradient.
 *   idx         [T, k] the choices that are counted (moe_select's, or others)
 *   seq_offsets [n_seq + 1] int32 on the device, ascending, in [0, T]; empty
 *               sequences are allowed (loss 0, load 0); n_seq below 2^22
 *   loss [n_seq], load [n_seq, E] fp32 out
 *   workspace >= moe_balance_workspace_bytes(sel, n_seq) bytes, 16-byte aligned
 * Of the rule T, E, k, score and logits are read.  Deterministic.
 */
moe_status_t moe_balance_loss(const moe_select_t *sel, const void *logits, int64_t ld, const int32_t *idx,
                              const int32_t *seq_offsets, int32_t n_seq, float alpha, float *loss, float *load,
                              void *workspace, size_t ws_bytes, void *stream);
size_t moe_balance_workspace_bytes(const moe_select_t *sel, int32_t n_seq);

/* ------------------------------------------------------------------------
 * Activation checkpoints in 8 bits: what the backward needs of the forward
 * (x, and y_perm with its T*k rows) kept in half the memory of bf16.
 * ------------------------------------------------------------------------ */

/* Formats of a saved activation [rows, cols].  The 8-bit ones hold one code per
 * value and one E8M0 scale byte per 1x128 tile of a row (the last tile of a row
 * may be shorter), scales [rows, ceil(cols/128)]: byte b stands for 2^(b-127),
 * the smallest power of two at or above the tile's largest magnitude / 448
 * (e4m3) or / 127 (int8), at least 2^-126, and 1 for an all-zero tile; the code
 * is the value over the scale, rounded to nearest even.  e4m3 keeps small values
 * of a tile to 3 bits, int8 keeps all of them to the same step.  A tile with an
 * infinity or a NaN gets the byte 255 and reads back as NaN; a finite value
 * whose rounded one is past fp32's largest reads back as infinity. */
typedef enum { MOE_SAVED_BF16 = 0, MOE_SAVED_E4M3 = 1, MOE_SAVED_I8 = 2 } moe_saved_format_t;
typedef struct {
    const void *data;       /* bf16 values, or 8-bit codes [rows, cols] */
    const uint8_t *scales;  /* the 8-bit formats only, else NULL */
    int32_t format;         /* moe_saved_format_t */
} moe_saved_t;

/*
 * Values to codes and back, rows and columns of any number.
 *   type     MOE_F32 or MOE_BF16: of src and dst
 *   src, dst [rows, cols], row r at + r * ld (ld >= cols, in elements); what
 *            lies between the rows is neither read nor written
 *   format   MOE_SAVED_E4M3 or MOE_SAVED_I8
 *   codes    [rows, cols] bytes, scales [rows, ceil(cols/128)] bytes
 */
moe_status_t moe_checkpoint_pack(int64_t rows, int32_t cols, int32_t type, const void *src, int64_t ld, int32_t format,
                                 uint8_t *codes, uint8_t *scales, void *stream);
moe_status_t moe_checkpoint_unpack(int64_t rows, int32_t cols, int32_t type, const uint8_t *codes,
                                   const uint8_t *scales, int32_t format, void *dst, int64_t ld, void *stream);

/*
 * Gradient of the weighted combine with respect to the routed outputs and the
 * weights, from saved routed outputs:
 *   dg[t, j] = dy[t] . y_perm[row_of[t*k + j]],  dy_perm[row_of[t*k + j]] = weights[t, j] dy[t]
 *   dy      [T, d] fp32
 *   y_perm  saved [T*k, d]
 *   row_of, weights: as for moe_combine; an entry of row_of outside [0, T*k)
 *           (a choice that was not dispatched) has no row: its dg is 0
 *   dy_perm [T*k, d] bf16 out; rows that no entry names are left as they were
 *   dg      [T, k] fp32 out
 * dy, y_perm's data and dy_perm are 16-byte aligned.  d is a multiple of 64,
 * below 2^30, with bf16 weights too, T below 2^26, from d = 2048 on below 2^24.
 * Deterministic.
 */
moe_status_t moe_combine_backward(const moe_desc_t *desc, const float *dy, const moe_saved_t *y_perm,
                                  const int32_t *row_of, const float *weights, void *dy_perm, float *dg, void *stream);

/*
 * moe_backward from saved activations, and with any router.
 *   x       saved [T, d]; y_perm saved [T*k, d]
 *   w_router, dw_router: NULL together where the choice did not come from
 *           moe_route: dx then holds the experts' share alone, idx is not read
 *           (NULL allowed), and dg (required) goes to moe_select_backward as
 *           dweights and on to moe_router_logits_backward
 * All else as for moe_backward; with both activations in bf16 and a w_router
 * it is moe_backward, bit for bit.
 *   workspace >= moe_workspace_bytes(desc, MOE_WS_BACKWARD_SAVED) bytes:
 *   moe_backward's and one bf16 [T, d].
 * The saved data, dy and the workspace are 16-byte aligned.
 */
moe_status_t moe_backward_saved(const moe_desc_t *desc, const moe_saved_t *x, const float *w_router,
                                const int32_t *idx, const float *weights, const int32_t *offsets,
                                const int32_t *row_src, const int32_t *row_of, const moe_ffn_weights_t *experts,
                                const moe_ffn_weights_t *shared, const moe_saved_t *y_perm, const float *dy, float *dx,
                                float *dw_router, float *dw_gate, float *dw_up, float *dw_down, float *ds_gate,
                                float *ds_up, float *ds_down, float *dg, void *workspace, size_t ws_bytes,
                                void *stream);

/* ------------------------------------------------------------------------
 * Microscaled operands, and the experts' products on weights in four bits.
 * ------------------------------------------------------------------------ */

/* Formats of a microscaled (OCP MX) matrix [rows, cols].  Each block of 32
 * columns of a row has one E8M0 scale byte (byte b stands for 2^(b-127)), each
 * value a code: an element is code * 2^(b-127).  e4m3 codes are bytes [rows,
 * cols]; e2m1 codes (1 sign, 2 exponent and 1 mantissa bits: 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives) are two to a byte, [rows, ceil(cols/2)], the even
 * column in the low half.  The scale bytes are [ceil(cols/128), rows, 4]: the
 * four blocks of a 128-column panel of a row are one 32-bit word, and a panel's
 * words lie row behind row, so that a tile's scales of one step of a product are
 * one run of memory. */
typedef enum { MOE_MX_E4M3 = 0, MOE_MX_E2M1 = 1 } moe_mx_format_t;
typedef struct {
    const void *codes;
    const uint8_t *scales;
    int32_t format; /* moe_mx_format_t */
} moe_mx_t;

/*
 * Values to microscaled codes and back, one row and column or more.
 *   type     MOE_F32 or MOE_BF16: of src and dst
 *   src, dst [rows, cols], row r at + r * ld (ld >= cols, in elements); what
 *            lies between the rows is neither read nor written
 *   codes, scales: as above.  Packing writes the scale of a block as the
 *            smallest power of two at or above its largest magnitude / 6 (e2m1)
 *            or / 448 (e4m3), at least 2^-126, and 1 for an all-zero block and
 *            for what a panel has past the columns; the code is the value over
 *            the scale, rounded to nearest even (nothing saturates), the upper
 *            half of an odd row's last byte 0.  A block with an infinity or a
 *            NaN gets the byte 255 and reads back as NaN; a finite value whose
 *            rounded one is past the type's largest reads back as infinity.
 * Scales are 4-byte aligned.
 */
moe_status_t moe_mx_pack(int64_t rows, int32_t cols, int32_t type, const void *src, int64_t ld, int32_t format,
                         uint8_t *codes, uint8_t *scales, void *stream);
moe_status_t moe_mx_unpack(int64_t rows, int32_t cols, int32_t type, const uint8_t *codes, const uint8_t *scales,
                           int32_t format, void *dst, int64_t ld, void *stream);

/* Rows in G groups of any sizes, each with a matrix of its own.
 *   M      rows of the output, from 1 on (a call of none is left out)
 *   x_rows rows of x, from 1 on
 *   k      row r of the product reads row row_src[r] / k of x (with row_src;
 *          without, k = 1, x_rows = M and row r reads row r) */
typedef struct {
    int32_t G, M, N, K;
    int32_t x_rows, k;
} moe_mx_groups_t;

/*
 * Product grouped by expert: out[r, n] = sum_i x[src(r), i] w[g, n, i] for the
 * rows offsets[g] <= r < offsets[g+1] of each group g, summed in fp32 (but for what the
 * matrix unit drops of e4m3 x, below) and rounded once.
 *   x       [x_rows, K] e4m3 or e2m1
 *   row_src [M] int32 or NULL (moe_dispatch's); an entry whose row lies outside
 *           x reads a row of zeros
 *   offsets [G+1] int32 on the device, ascending, in [0, M]; groups may be empty;
 *           rows outside every group are left as they were
 *   w       [G, N, K] e2m1 (its scales [ceil(K/128), G*N, 4])
 *   out     [M, N] of type out_type, MOE_F32 or MOE_BF16
 *   workspace >= moe_mx_product_workspace_bytes(groups, out_type) bytes (0 where
 *           the groups are small: NULL is allowed then)
 * K is a multiple of 32 and below 2^23, G at most 1024, N below 2^21, M and x_rows
 * below 2^29, x's codes with row_src below 2^32 - 2^20 bytes, (M / 32 + G) (N / 128
 * + 1) below 2^31; codes and the workspace are 16-byte aligned, scales 4, out as its
 * type.  What an infinity or a NaN (a scale byte of 255, an e4m3 code
 * 0x7f or 0xff) enters comes out NaN.  Deterministic.
 * The matrix unit sums the products of eight neighbouring columns before they join
 * the fp32 sum, aligned to the largest of them, and drops what lies below 2^-13 of
 * that one: nothing of e2m1 x; of e4m3 x up to 2^-10 of the largest of each eight
 * (about 4e-6 of the result for normally distributed values).
 */
moe_status_t moe_mx_product(const moe_mx_groups_t *groups, const moe_mx_t *x, const int32_t *row_src,
                            const int32_t *offsets, const moe_mx_t *w, int32_t out_type, void *out, void *workspace,
                            size_t ws_bytes, void *stream);
size_t moe_mx_product_workspace_bytes(const moe_mx_groups_t *groups, int32_t out_type);

/*
 * The routed experts' FFN on weights in four bits, with the rows of groups:
 *   h = silu(x W_gate[g]^T) * (x W_up[g]^T) in fp32, packed in x's format (as by
 *       moe_mx_pack), y = h W_down[g]^T in bf16; the sums as moe_mx_product's (what
 *       is dropped of e4m3 x moves some of h's codes to their neighbours).
 *   groups  N = I (the width of h), K = d
 *   gate, up [G, I, d], down [G, d, I] e2m1
 *   y       [M, d] bf16; rows outside every group are left as they were
 *   workspace >= moe_mx_ffn_workspace_bytes(groups, x->format) bytes
 * d and I are multiples of 32, both below 2^21; all else as for moe_mx_product.
 * With E groups and moe_dispatch's offsets and row_src y is moe_expert_ffn's
 * y_perm, for moe_combine.
 */
moe_status_t moe_mx_expert_ffn(const moe_mx_groups_t *groups, const moe_mx_t *x, const int32_t *row_src,
                               const int32_t *offsets, const moe_mx_t *gate, const moe_mx_t *up, const moe_mx_t *down,
                               void *y, void *workspace, size_t ws_bytes, void *stream);
size_t moe_mx_ffn_workspace_bytes(const moe_mx_groups_t *groups, int32_t format);

/* ------------------------------------------------------------------------
 * The optimizer's step over many tensors at once.
 * ------------------------------------------------------------------------ */

/* One tensor of n elements.
 *   w        weights, w_type MOE_F32 or MOE_BF16, updated
 *   g        gradient, g_type MOE_F32 or MOE_BF16
 *   states   32: m and v are fp32 [n].  8: they are e4m3 codes [n], in tiles of
 *            128 elements with an E8M0 scale byte each, m_scales and v_scales
 *            [ceil(n/128)] (the e4m3 checkpoint format of one row); v's codes
 *            stand for its root.  A state that holds nothing yet is zeros (in 8
 *            bits: codes of 0, any scale but 255).
 *   master   fp32 [n] or NULL: the weights that the step works on; w (bf16) is
 *            then their rounding */
typedef struct {
    void *w;
    const void *g;
    void *m, *v;
    uint8_t *m_scales, *v_scales;
    float *master;
    int64_t n;
    int32_t w_type, g_type, states;
} moe_adamw_tensor_t;

/* The step: with g' = g * grad_scale (1 without),
 *   m <- beta1 m + (1 - beta1) g',  v <- beta2 v + (1 - beta2) g'^2,
 *   w <- w - lr weight_decay w - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, by the m and v of this step before any rounding.  What is kept in
 * fewer bits and read again by the next step is rounded stochastically, up with
 * the probability of what lies above the value below: 8-bit states (rounded to
 * nearest a second moment would stand still, since a step moves it by far less
 * than half a step of its codes) and bf16 weights without a master.  The random
 * numbers: for element i of tensor t of the call, h = mix(lo(i) ^ mix(hi(i) +
 * key)), key = mix(lo(seed) ^ mix(hi(seed) ^ mix(lo(step) ^ mix(t)))), lo and hi
 * the 32-bit halves, sums modulo 2^32; m takes h's low 16 bits, v's root its high
 * 16, the weight the high 16 bits of h * 0x9E3779B1 modulo 2^32.  mix(x): x ^= x >> 16, x *= 0x7feb352d, x ^= x
 * >> 15, x *= 0x846ca68b, x ^= x >> 16.  A root above 0 never gets the code of 0
 * (it gets the code behind it), so that no step divides by a root that was lost.
 * The price of a second moment in 8 bits: the roots keep their mean, but many steps'
 * roundings spread them, by a deviation of 11 to 18 % whatever beta2, and the mean
 * square lies above the average that it stands for by that squared (with normal
 * gradients and beta2 = 0.999, 14 % and 3 % after 600 steps, 15 % and 5 % after 6000).
 * A gradient that is not finite leaves fp32 states so at its element, 8-bit ones in its
 * whole tile of 128, for good; grad_scale is there to leave such a step out.
 *   step       from 1 on
 *   grad_scale one fp32 on the device or NULL; where it holds an infinity or a
 *              NaN, the call changes nothing
 *   step_ptr, lr_ptr: on the device, in place of step and lr (NULL: not), so
 *              that a captured step can be replayed with others
 * lr and weight_decay are not negative, eps is 0 or from 2^-126 to 2^126, the
 * betas lie in [0, 1). */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    uint64_t seed;
    const float *grad_scale;
    const int64_t *step_ptr;
    const float *lr_ptr;
} moe_adamw_t;

/*
 * The step of `count` tensors (read on the host before the call returns), in one
 * launch for every 59 of the same types or more.  Tensors of no elements are allowed;
 * pointers are aligned as their type; n below 2^35.  What a call writes overlaps with
 * nothing else of it (the workgroups would race; the binding refuses it): a weight that
 * is used twice is one tensor.  Deterministic.
 */
moe_status_t moe_adamw(const moe_adamw_t *rule, const moe_adamw_tensor_t *tensors, int32_t count, void *stream);

/* Static, human-readable name of a status code. */
const char *moe_status_str(moe_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
