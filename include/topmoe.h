/*
 * topmoe.h — C ABI of the MI355X (gfx950) MiniMind FFN / top-k MoE forward,
 * its backward, and the operators of the block around it.
 *
 * Operations (definitions from the MiniMind course, lesson 13 "FFN and MoE",
 * sections 0, 1.2, 1.5, 1.6 and source walkthrough steps 3-6; minimind3
 * chapter 4 "MLP & MoE", sections 4.2-4.4):
 *
 *   dense FFN      y = W_down( SiLU(W_gate x) * W_up x ),  SiLU(z) = z * sigmoid(z)
 *   MoE router     p = softmax(W_router x);  S = TopK(p, k);
 *                  alpha_e = p_e / (sum_{j in S} p_j + 1e-20)
 *   MoE output     y = sum_{e in S} alpha_e * Expert_e(x), each expert a dense FFN
 *   aux loss       aux = E * coef * sum_e load_e * prob_e,
 *                  load_e = (tokens that selected e) / N,  prob_e = mean_t p_{t,e}
 *   z-loss         z_coef * mean_t logsumexp_e(r_te)^2 (router logits r = W_router x)
 *   capacity       each expert takes at most C = ceil(capacity_factor * N * k / E)
 *                  tokens: the first C of its tokens in ascending token order
 *                  (the dispatch order); the others' (token, expert) pairs are
 *                  dropped and add nothing to y
 *                  (the MiniMind study notes' section 10 table names router
 *                  z-loss and expert capacity without defining them; these are
 *                  the standard forms)
 *   backward       the gradients of these with respect to x and every weight:
 *                  the top-k choice and the counts load_e are discrete and
 *                  carry no gradient; the softmax probabilities carry it back
 *                  through alpha and prob_e (minimind3 chapter 4, section
 *                  4.4; MiniMind study notes, section 7 on router training)
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees or retains them.
 *   - Row-major layouts.  Weights use the nn.Linear [out, in] layout.
 *   - Calls are asynchronous: they validate synchronously on the host, then
 *     enqueue kernels on `stream` (a hipStream_t; NULL = the null stream) and
 *     return.  No host synchronisation, no device-to-host copy.
 *   - On any error nothing is launched and no output is touched.  Errors are
 *     negative status codes (topmoe_strerror gives text).  A HIP launch error
 *     is reported as TOPMOE_ERR_HIP (outputs may then be partly written).
 *   - Results are deterministic: the same inputs give bitwise identical
 *     outputs (no floating-point atomics anywhere).
 *   - `stage_events`, when not NULL, is an array of 2 * stages hipEvent_t
 *     handles (see topmoe_events_create); events 2i and 2i+1 are stamped by
 *     the dispatch of stage i's kernel at its start and end (AMD's
 *     hipExtLaunchKernel start / stop events), so they bracket exactly that
 *     kernel's execution; a stage that launches no kernel records both back
 *     to back.  Pass NULL in production.  Stage counts: TOPMOE_FFN_STAGES,
 *     TOPMOE_MOE_STAGES.
 *
 * dtype
 *   TOPMOE_DTYPE_FP32: x, W_gate, W_up, W_down, y float32; all arithmetic fp32.
 *   TOPMOE_DTYPE_BF16: x, W_gate, W_up, W_down, y bfloat16; fp32 accumulation;
 *                      the SiLU(g)*u intermediate is rounded to bf16; y is
 *                      rounded once (round-to-nearest-even).
 *   The router weight W_router is float32 in both, and routing is fp32.
 *
 * Shape limits: N >= 0 (N == 0 is a no-op apart from zeroed offsets and aux;
 * then x, y, topk_idx, alpha and sorted_token_ids may be NULL),
 * H and I positive multiples of 64, 1 <= E <= 64, 1 <= k <= E,
 * N * max(k, 1) < 2^31, and every GEMM operand below 4 GiB: x (N * H), the
 * intermediate (N * k * I) and one expert's W_gate / W_up / W_down (I * H),
 * counted in bytes of the dtype.
 */
#ifndef TOPMOE_H
#define TOPMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
#define TOPMOE_OK                        0
#define TOPMOE_ERR_NULL_ARG             -1  /* a required pointer is NULL            */
#define TOPMOE_ERR_BAD_SHAPE            -2  /* N, H, I, E or k outside the limits     */
#define TOPMOE_ERR_UNSUPPORTED_DTYPE    -3  /* dtype not FP32 / BF16                  */
#define TOPMOE_ERR_WORKSPACE_TOO_SMALL  -4  /* workspace_bytes < *_workspace_bytes()  */
#define TOPMOE_ERR_HIP                  -5  /* a HIP runtime call or launch failed    */
#define TOPMOE_ERR_BAD_ARG              -6  /* aux_coef, z_coef or capacity_factor negative or not
                                               finite; a negative capacity; aux_grad, z_grad
                                               or residual_scale not finite; eps not positive
                                               and finite; unknown flag bits or gate mode;
                                               misaligned pointer; a launch-shape override
                                               that is not instantiated */
#define TOPMOE_ERR_SCRATCH_TOO_SMALL    -7  /* moe_ffn_fwd_noalloc: the problem's workspace
                                               exceeds the fixed scratch */

/* ---- dtypes ------------------------------------------------------------ */
#define TOPMOE_DTYPE_FP32 0
#define TOPMOE_DTYPE_BF16 1

/* ---- stages (for stage_events) ------------------------------------------ */
#define TOPMOE_FFN_STAGES 2  /* 0 gate/up GEMM + SiLU*up, 1 down GEMM                   */
#define TOPMOE_MOE_STAGES 5  /* 0 router, 1 expert offsets + aux + token scatter,
                                2 grouped gate/up GEMM + SiLU*up, 3 grouped down GEMM
                                + alpha, 4 combine of the k slots (k == 1: empty, or
                                under a capacity the rows of the dropped tokens).
                                Decode-sized inference calls do stage 1 (and, with
                                E <= 16, stage 0) inside the GEMM launches: such a
                                stage launches no kernel                                */
#define TOPMOE_FFN_BWD_STAGES 7  /* 0 weight transposes, 1 x / dy transposes,
                                    2 g, u GEMM (recomputed), 3 dh GEMM + dg, du,
                                    4 dx GEMM, 5 dWg + dWu GEMM, 6 dWd GEMM             */
#define TOPMOE_MOE_BWD_STAGES 12 /* 0 router, 1 offsets + scatter (the forward's routing),
                                    2 weight transposes, 3 grouped x / alpha*dy
                                    transposes, 4 grouped g, u GEMM (recomputed),
                                    5 grouped dh GEMM + dg, du, d alpha, 6 grouped dx GEMM,
                                    7 router backward, 8 dx combine, 9 dW_router,
                                    10 grouped dWg + dWu, 11 grouped dWd               */

/* ---- moe_ffn_fwd flags -------------------------------------------------- */
/* The config's norm_topk_prob = False (lesson 13, walkthrough steps 1 and 5;
 * minimind3 chapter 4, section 4.3 step 2): alpha is the selected
 * probabilities as they are, without renormalisation to sum 1. */
#define TOPMOE_MOE_RAW_TOPK_WEIGHTS 1
/* moe_ffn_bwd only: the workspace already holds the routing, the pairs
 * (g, u) and h^T that moe_ffn_fwd_train wrote into it for the same inputs
 * and arguments, so the router, the permutation and the grouped g, u GEMM
 * (stages 0, 1 and 4) are skipped. */
#define TOPMOE_MOE_BWD_SAVED 2
/* The module outside training (lesson 13, walkthrough step 6: the aux loss
 * is computed only while training; otherwise it is a zero scalar): aux_loss
 * and z_loss are 0 whatever aux_coef and z_coef say, and moe_ffn_bwd passes
 * no gradient through them.  Everything else is unchanged. */
#define TOPMOE_MOE_EVAL 4

/* Workspace needed by ffn_swiglu_fwd: the SiLU(g)*u intermediate [N, I]
 * (dtype-sized elements), 256-byte aligned.  Returns 0 for invalid shapes. */
size_t ffn_workspace_bytes(int64_t N, int64_t H, int64_t I, int dtype);

/* Dense SwiGLU FFN forward (lesson 13, sections 0 and 1.2; walkthrough step 3;
 * minimind3 chapter 4, section 4.2).
 *   x   [N, H]   input tokens (B*S flattened; the caller reshapes)
 *   Wg  [I, H]   gate_proj.weight      Wu [I, H] up_proj.weight
 *   Wd  [H, I]   down_proj.weight
 *   residual [N, H]  optional (NULL = none), same dtype: the block's residual
 *                stream; y = residual + FFN(x) (lesson 13, sections 1.3-1.4:
 *                hidden_states + mlp(...)), summed in fp32 and rounded once.
 *                May alias y (each element is read before it is written).
 *   y   [N, H]   output, same dtype as x; must not alias x or the weights
 *   workspace    device scratch of at least ffn_workspace_bytes(N, H, I, dtype)
 *                bytes, 256-byte aligned; contents on entry are ignored.
 * All tensor pointers must be 16-byte aligned. */
int ffn_swiglu_fwd(const void* x, const void* Wg, const void* Wu, const void* Wd,
                   const void* residual, void* y, int64_t N, int64_t H, int64_t I, int dtype,
                   void* workspace, size_t workspace_bytes,
                   void* stream, void* const* stage_events);

/* Workspace needed by moe_ffn_fwd (routing partials, permutation, the
 * SiLU(g)*u intermediate [N*k, I] and, for k >= 2, the k-slots [N*k, H] of
 * alpha-scaled expert outputs in the dtype).
 * Returns 0 for invalid shapes. */
size_t moe_workspace_bytes(int64_t N, int64_t H, int64_t I, int E, int k, int dtype);

/* Top-k MoE FFN forward (lesson 13, sections 0, 1.5, 1.6 and walkthrough
 * steps 4-6; minimind3 chapter 4, sections 4.3 and 4.4).
 *   x        [N, H]      input tokens (dtype)
 *   Wr       [E, H]      router (gate) weight, float32
 *   Wg, Wu   [E, I, H]   experts' gate_proj / up_proj weights, stacked (dtype)
 *   Wd       [E, H, I]   experts' down_proj weights, stacked (dtype)
 *   residual [N, H]      optional (NULL = none), dtype: y starts from it
 *                        instead of zeros (y = residual + MoE(x), lesson 13,
 *                        sections 1.3-1.4).  May alias y.
 *   aux_coef             router_aux_loss_coef (>= 0); 0 gives aux = 0 exactly,
 *                        which is also the module's value outside training
 *   z_coef               router z-loss coefficient (>= 0); 0 gives z_loss = 0
 *   capacity_factor      expert capacity factor (>= 0), of which the float's own
 *                        value counts (the float nearest 1.2 lies above it); 0 =
 *                        no capacity (dropless, the pages' module); a capacity of
 *                        N or more drops nothing
 *   flags                0, or TOPMOE_MOE_RAW_TOPK_WEIGHTS and / or TOPMOE_MOE_EVAL
 *   y        [N, H]      output (dtype): y_t = residual_t (or 0) + the sum over
 *                        the selected (and kept) experts in ascending expert id
 *                        of alpha * Expert_e(x_t); with k >= 2 (or a capacity)
 *                        each expert term is first rounded to the dtype (the
 *                        terms the pages' index_add_ adds); the sum is taken in
 *                        fp32 and rounded once
 *   topk_idx [N, k]      int32 selected experts, slot order = probability
 *                        descending, equal probabilities by ascending id
 *                        (dropped pairs included: the router's choice)
 *   alpha    [N, k]      float32 weights in the same slot order: renormalised
 *                        to sum 1 (default) or the raw probabilities (flag);
 *                        not renormalised after drops
 *   aux_loss [1]         float32 load-balancing loss (training-mode value; counts
 *                        every selection, kept or dropped)
 *   z_loss   [1]         optional (NULL = not returned) float32 router z-loss
 *   expert_offsets [E+1] optional (NULL = not returned) int32 exclusive prefix
 *                        sum of per-expert token counts (of the kept tokens)
 *   sorted_token_ids [N*k] optional int32: tokens grouped by expert, ascending
 *                        expert id, ascending token id within an expert (kept
 *                        tokens; the remaining positions hold -1)
 *   workspace            at least moe_workspace_bytes(N, H, I, E, k, dtype)
 *                        bytes, 256-byte aligned; contents on entry ignored.
 * Outputs must not alias inputs or each other.  Tensor pointers must be
 * 16-byte aligned (int32/float32 outputs: 4-byte aligned). */
int moe_ffn_fwd(const void* x, const float* Wr, const void* Wg, const void* Wu,
                const void* Wd, const void* residual, int64_t N, int64_t H, int64_t I,
                int E, int k, float aux_coef, float z_coef, float capacity_factor, int flags,
                int dtype, void* y, int32_t* topk_idx, float* alpha, float* aux_loss,
                float* z_loss, int32_t* expert_offsets, int32_t* sorted_token_ids,
                void* workspace, size_t workspace_bytes,
                void* stream, void* const* stage_events);

/* ---- no allocation ------------------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the MoE
 * forward with its workspace in a fixed scratch array that the library holds
 * in device memory, one per GPU it runs on, from the first use until the
 * process ends (TOPMOE_NOALLOC_SCRATCH_BYTES: 64 MiB).  Arguments,
 * outputs, errors and results are those of moe_ffn_fwd (the same bits)
 * without the workspace pair; a problem whose moe_workspace_bytes() exceeds
 * the scratch returns TOPMOE_ERR_SCRATCH_TOO_SMALL before anything else
 * happens.  The call allocates nothing: the scratch's device address is
 * looked up once per device (the device current at the call must be the
 * stream's).  All calls on one GPU share its scratch, so calls that overlap
 * on one GPU (other streams, other host threads) race: serialise them.  The
 * scratch keeps the last call's contents; nothing in it needs clearing. */
#define TOPMOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int moe_ffn_fwd_noalloc(const void* x, const float* Wr, const void* Wg, const void* Wu,
                        const void* Wd, const void* residual, int64_t N, int64_t H, int64_t I,
                        int E, int k, float aux_coef, float z_coef, float capacity_factor,
                        int flags, int dtype, void* y, int32_t* topk_idx, float* alpha,
                        float* aux_loss, float* z_loss, int32_t* expert_offsets,
                        int32_t* sorted_token_ids, void* stream, void* const* stage_events);

/* ---- backward ------------------------------------------------------------
 * Gradients of the forward above (same shapes, dtypes and flags).  The
 * forward's intermediate activations are not needed: the backward recomputes
 * them (and, for the MoE, the routing: same kernels, same choices).
 * Gradient outputs are overwritten, not accumulated; weight gradients have
 * the weights' dtype and layout, dW_router is float32.  The gradient with
 * respect to the residual stream of the forward is dy itself (nothing to
 * compute).  In bf16, the recomputed g and u, [dg | du], dg, du, h and
 * alpha*dy are rounded to bf16 before the arithmetic or GEMMs that consume
 * them; all accumulation is fp32. */

/* Workspace needed by ffn_swiglu_bwd: transposed weights [H, 2I] and [I, H],
 * transposed x and dy [H, round64(N)], the pairs (g, u) [N, I], [dg | du]
 * [N, 2I] and dg^T, du^T, h^T [I, round64(N)] (dtype-sized elements).
 * Returns 0 for invalid shapes. */
size_t ffn_bwd_workspace_bytes(int64_t N, int64_t H, int64_t I, int dtype);

/* Dense SwiGLU FFN backward.  With g = x Wg^T, u = x Wu^T, h = SiLU(g) * u,
 * y = h Wd^T and the upstream gradient dy [N, H]:
 *   dWd = dy^T h,  dh = dy Wd,  dg = dh * u * SiLU'(g),  du = dh * SiLU(g),
 *   dWg = dg^T x,  dWu = du^T x,  dx = dg Wg + du Wu,
 *   SiLU'(z) = sigmoid(z) * (1 + z * (1 - sigmoid(z))).
 *   x, Wg, Wu, Wd   as for ffn_swiglu_fwd;  dy [N, H] (dtype)
 *   dx [N, H], dWg [I, H], dWu [I, H], dWd [H, I]   outputs (dtype); N == 0
 *                   gives zero weight gradients (x, dy, dx may then be NULL)
 *   workspace       at least ffn_bwd_workspace_bytes(N, H, I, dtype) bytes,
 *                   256-byte aligned; contents on entry ignored.
 * Outputs must not alias inputs or each other; tensor pointers 16-byte
 * aligned.  Shape limits as for the forward, plus [N, 2I], [H, 2I] and
 * [I, round64(N)] operands below 4 GiB each. */
int ffn_swiglu_bwd(const void* x, const void* Wg, const void* Wu, const void* Wd,
                   const void* dy, void* dx, void* dWg, void* dWu, void* dWd,
                   int64_t N, int64_t H, int64_t I, int dtype,
                   void* workspace, size_t workspace_bytes,
                   void* stream, void* const* stage_events);

/* ---- training: keep g, u for the backward ----------------------------- */
/* The backward recomputes g = x Wg^T and u = x Wu^T (its stage "g, u GEMM")
 * unless the forward kept them.  These forwards compute exactly what
 * ffn_swiglu_fwd / moe_ffn_fwd compute (the same bits in every output) and
 * in the same gate/up GEMM also write the pairs (g, u) and h^T into `saved`,
 * a backward workspace (the MoE forward keeps its routing there as well:
 * selections, probabilities, offsets and the expert-grouped entry lists): at least ffn_bwd_workspace_bytes(N, H, I, dtype) /
 * moe_bwd_workspace_bytes(N, H, I, E, k, dtype) bytes, 256-byte aligned.
 * Pass that same buffer, untouched in between, as the workspace of
 * ffn_swiglu_bwd_saved / moe_ffn_bwd with TOPMOE_MOE_BWD_SAVED for the same
 * inputs and arguments.  Costs the forward the pair and h^T stores (three
 * times h's bytes), saves the backward its largest GEMM but one (and, for
 * the MoE, its routing kernels).  The other
 * arguments, errors and stage events are those of the plain forwards; a
 * NULL `saved` is TOPMOE_ERR_NULL_ARG. */
int ffn_swiglu_fwd_train(const void* x, const void* Wg, const void* Wu, const void* Wd,
                         const void* residual, void* y, int64_t N, int64_t H, int64_t I,
                         int dtype, void* workspace, size_t workspace_bytes,
                         void* saved, size_t saved_bytes,
                         void* stream, void* const* stage_events);
int moe_ffn_fwd_train(const void* x, const float* Wr, const void* Wg, const void* Wu,
                      const void* Wd, const void* residual, int64_t N, int64_t H, int64_t I,
                      int E, int k, float aux_coef, float z_coef, float capacity_factor,
                      int flags, int dtype, void* y, int32_t* topk_idx, float* alpha,
                      float* aux_loss, float* z_loss, int32_t* expert_offsets,
                      int32_t* sorted_token_ids, void* workspace, size_t workspace_bytes,
                      void* saved, size_t saved_bytes,
                      void* stream, void* const* stage_events);
/* ffn_swiglu_bwd on a workspace that ffn_swiglu_fwd_train filled (stage 2
 * skipped, its events zero-length). */
int ffn_swiglu_bwd_saved(const void* x, const void* Wg, const void* Wu, const void* Wd,
                         const void* dy, void* dx, void* dWg, void* dWu, void* dWd,
                         int64_t N, int64_t H, int64_t I, int dtype,
                         void* workspace, size_t workspace_bytes,
                         void* stream, void* const* stage_events);

/* Workspace needed by moe_ffn_bwd: the routing buffers, transposed expert
 * weights [E, H, 2I] and [E, I, H], the per-entry intermediates and
 * gradients, and float32 router buffers.  Returns 0 for invalid shapes. */
size_t moe_bwd_workspace_bytes(int64_t N, int64_t H, int64_t I, int E, int k, int dtype);

/* Top-k MoE FFN backward.  The routing of moe_ffn_fwd(x, Wr, ..., k,
 * aux_coef, flags) is recomputed; for each token t and selected expert e
 * (weight alpha_{t,e}, expert output o = Expert_e(x_t)):
 *   the expert's own backward (as ffn_swiglu_bwd) with upstream alpha * dy_t;
 *   d alpha_{t,e} = dy_t . o;
 *   then dp through alpha = p_S / (sum p_S + 1e-20) (or alpha = p_S with
 *   TOPMOE_MOE_RAW_TOPK_WEIGHTS), plus aux_grad * aux_coef * E * c_e / N^2 on
 *   every p_{t,e} (c_e = tokens routed to e); dr = p * (dp - sum(p * dp))
 *   + z_grad * z_coef * 2 * logsumexp(r_t) * p / N; dW_router = dr^T x and
 *   dx_t += W_router^T dr_t.  A pair dropped by the capacity contributes
 *   neither an expert gradient nor d alpha.
 *   x, Wr, Wg, Wu, Wd, N, H, I, E, k, aux_coef, z_coef, capacity_factor,
 *   flags, dtype    as for moe_ffn_fwd; flags may add TOPMOE_MOE_BWD_SAVED
 *                   (TOPMOE_MOE_EVAL: no gradient through aux_loss, z_loss)
 *   dy [N, H]       upstream gradient of y (dtype)
 *   aux_grad        upstream gradient of aux_loss (1 when it is added to the
 *                   loss as is); finite
 *   z_grad          upstream gradient of z_loss; finite
 *   aux_grad_scale, z_grad_scale
 *                   optional (NULL = 1) float32 device scalars multiplying
 *                   aux_grad / z_grad: an upstream gradient that is still on
 *                   the device (autograd's) is read by the kernel, with no
 *                   host synchronisation.  Their value is not validated.
 *   dx [N, H] (dtype), dWr [E, H] (float32), dWg, dWu [E, I, H], dWd [E, H, I]
 *                   (dtype) outputs; experts no token selected get zero
 *                   gradients.  N == 0 gives all-zero weight gradients.
 *   workspace       at least moe_bwd_workspace_bytes(N, H, I, E, k, dtype)
 *                   bytes, 256-byte aligned; contents on entry ignored.
 * Outputs must not alias inputs or each other; tensor pointers 16-byte
 * aligned. */
int moe_ffn_bwd(const void* x, const float* Wr, const void* Wg, const void* Wu,
                const void* Wd, const void* dy, float aux_grad, float z_grad,
                const float* aux_grad_scale, const float* z_grad_scale,
                int64_t N, int64_t H, int64_t I, int E, int k, float aux_coef, float z_coef,
                float capacity_factor, int flags, int dtype,
                void* dx, float* dWr, void* dWg, void* dWu, void* dWd,
                void* workspace, size_t workspace_bytes,
                void* stream, void* const* stage_events);

/* ---- rows by expert and back -------------------------------------------
 * The dispatch and combine of a top-k MoE whose experts are the caller's own
 * (the token loop of lesson 13, walkthrough step 5, without the SwiGLU
 * experts): tokens' rows sorted by expert, and the experts' rows back to
 * tokens with their weights; with their gradients.
 *
 * Entry i = t * k + j is slot j of token t.  Its rank is the number of earlier
 * entries of the same expert (a token may name an expert twice: two entries).
 * An expert keeps its first C entries (all of them without a capacity); an
 * entry whose topk_idx is outside [0, E) -- a padding token's -1 -- is kept by
 * none.  Kept entries take the rows
 * [0, expert_offsets[E]), grouped by ascending expert and in rank order; the
 * others take the rows behind them, by (expert, rank), those without an expert
 * last, and their rows hold zeros.  Every row of the [N * k, H] outputs is
 * written.
 *
 * H is a positive multiple of 8 up to 2^20, 1 <= k <= E <= 256, N * k < 2^31;
 * tensor pointers 16-byte aligned, int32 / float32 arrays 4-byte aligned.
 * Outputs must not alias inputs or each other, except where said.  With
 * N == 0 only expert_offsets is written, and every other tensor may be NULL. */
#define TOPMOE_DISPATCH_STAGES 2  /* 0 rows of the entries (empty in the one-launch
                                     dispatch), 1 copy                             */
#define TOPMOE_DISPATCH_MAX_EXPERTS 256
/* The one-launch dispatch, which needs no workspace: at most TOPMOE_DISPATCH_ONE
 * entries (N * k), and x and xs together below TOPMOE_DISPATCH_ONE_BYTES. */
#define TOPMOE_DISPATCH_ONE 32768
#define TOPMOE_DISPATCH_ONE_BYTES ((int64_t)128 << 20)

/* Workspace needed by moe_dispatch_fwd: counts per chunk of entries.  Returns
 * 0 for invalid sizes (and at least 256 for valid ones). */
size_t moe_dispatch_workspace_bytes(int64_t N, int E, int k);

/* xs[row(i)] = x[t].
 *   x        [N, H]     tokens (dtype)
 *   topk_idx [N, k]     int32 experts
 *   capacity_factor     C = ceil(capacity_factor * N * k / E) of the float's own
 *                       value, in double; 0 = no capacity.  The float nearest
 *                       1.2 lies above it: where such a product should be a
 *                       whole number, give C itself (moe_dispatch_fwd_capacity)
 *   xs       [N*k, H]   output (dtype): the rows by expert, zeros behind them
 *   expert_offsets [E+1] int32 output: first row of each expert; [E]: kept rows
 *   row_entry [N*k]     int32 output: the entry of each kept row, then -1
 *   entry_row [N, k]    int32 output: the entry's row, or -1 - row if not kept
 *   workspace           at least moe_dispatch_workspace_bytes(N, E, k) bytes,
 *                       256-byte aligned; contents on entry ignored.  Not used,
 *                       and may be NULL, in the one-launch dispatch. */
int moe_dispatch_fwd(const void* x, const int32_t* topk_idx, int64_t N, int64_t H, int E, int k,
                     float capacity_factor, int dtype, void* xs, int32_t* expert_offsets,
                     int32_t* row_entry, int32_t* entry_row, void* workspace,
                     size_t workspace_bytes, void* stream, void* const* stage_events);
/* The same with C itself: capacity >= 0 entries an expert, 0 = no capacity. */
int moe_dispatch_fwd_capacity(const void* x, const int32_t* topk_idx, int64_t N, int64_t H, int E,
                              int k, int64_t capacity, int dtype, void* xs,
                              int32_t* expert_offsets, int32_t* row_entry, int32_t* entry_row,
                              void* workspace, size_t workspace_bytes, void* stream,
                              void* const* stage_events);
/* dx[t] = the sum over t's kept entries, in slot order, of dxs[entry_row]
 * (fp32, rounded once).  dxs [N*k, H], entry_row [N, k] as the dispatch wrote
 * it, dx [N, H].  One stage. */
int moe_dispatch_bwd(const void* dxs, const int32_t* entry_row, int64_t N, int64_t H, int k,
                     int dtype, void* dx, void* stream, void* const* stage_events);
/* y[t] = residual[t] (or 0) + the sum over t's kept entries, in slot order, of
 * alpha * ys[entry_row] (fp32, rounded once).  A row that no kept entry names
 * is not read, nor is the alpha of an entry that is not kept.
 *   ys [N*k, H] (dtype), alpha [N, k] float32, residual [N, H] optional (may
 *   alias y), y [N, H] (dtype).  One stage. */
int moe_combine_fwd(const void* ys, const int32_t* entry_row, const float* alpha,
                    const void* residual, int64_t N, int64_t H, int k, int dtype, void* y,
                    void* stream, void* const* stage_events);
/* dys[entry_row] = alpha * dy[t] for kept entries, zeros in the others' rows;
 * dalpha = dy[t] . ys[entry_row] (fp32), 0 for entries that are not kept.
 * entry_row must name each row once, as the dispatch's does.  The gradient of
 * the residual is dy itself.  One stage. */
int moe_combine_bwd(const void* dy, const void* ys, const int32_t* entry_row, const float* alpha,
                    int64_t N, int64_t H, int k, int dtype, void* dys, float* dalpha,
                    void* stream, void* const* stage_events);

/* ---- norms around a block -----------------------------------------------
 * The RMS norm before a block (the block's post_attention_layernorm of lesson
 * 13, sections 1.3-1.4) and, after it, an optional RMS norm of its output, a
 * gate, the residual stream with its scale, and the next block's norm, in one
 * pass.  Per token, in fp32:
 *   yh = y / sqrt(mean(y^2) + eps) with a post norm, y without (w NULL)
 *   r  = residual_scale * residual + gate * w * yh,    out = r rounded once
 *   n  = next_w * r / sqrt(mean(r^2) + eps), of the unrounded r, rounded once
 * The sum of the squares is fp32 too: a row whose sum passes its range (one
 * element beyond about 1.8e19 does) has rstd 0, as one with an infinity has.
 * H is a multiple of 8 with 8 <= H <= 16384; N < 2^31; eps positive and finite;
 * weights and gates have x's dtype; tensor pointers are 16-byte aligned (a
 * token gate and its gradient: their element's size; float32 arrays: 4-byte).
 * Outputs must not alias inputs or each other, except where said.  With N == 0
 * tensors of that size may be NULL; weight gradients are then zero. */
#define TOPMOE_NORM_BWD_STAGES 2  /* 0 rows, 1 sums over the tokens (forwards: one stage) */
/* gate_mode: none (1); a value per channel, in gate_rows rows [gate_rows, H]
 * of which row t / (N / gate_rows) belongs to token t (gate_rows divides N: 1
 * shares one row, the batch size gives each sequence its own); a value per
 * token [N]. */
#define TOPMOE_GATE_NONE 0
#define TOPMOE_GATE_CHANNEL 1
#define TOPMOE_GATE_TOKEN 2

/* n = w * x * rstd, rstd = 1 / sqrt(mean(x^2) + eps).  x, n [N, H], w [H],
 * rstd [N] float32 output (for the backward). */
int block_prenorm_fwd(const void* x, const void* w, int64_t N, int64_t H, float eps, int dtype,
                      void* n, float* rstd, void* stream, void* const* stage_events);
/* Workspace of either backward: float32 partial sums.  Returns 0 for invalid
 * sizes.  gate_rows: of a channel gate, otherwise 1. */
size_t block_norm_bwd_workspace_bytes(int64_t N, int64_t H, int64_t gate_rows);
/* dx = dresidual (or 0) + rstd * (a - xh * mean(a * xh)), a = dn * w,
 * xh = x * rstd; dw = sum over tokens of dn * xh.
 *   dresidual [N, H] optional: the gradient that reaches x beside the norm,
 *   along the residual stream (may alias dx).  dx [N, H], dw [H] outputs. */
int block_prenorm_bwd(const void* dn, const void* x, const void* w, const float* rstd,
                      const void* dresidual, int64_t N, int64_t H, int dtype, void* dx, void* dw,
                      void* workspace, size_t workspace_bytes, void* stream,
                      void* const* stage_events);
/*   y, residual [N, H]; w [H] or NULL (no post norm); gate by gate_mode (NULL
 *   for none); next_w [H] or NULL (no next norm)
 *   out [N, H] (may alias residual); rstd [N] float32, needed with w; n [N, H]
 *   and next_rstd [N] float32, needed with next_w */
int block_postnorm_fwd(const void* y, const void* residual, const void* w, const void* gate,
                       const void* next_w, int64_t N, int64_t H, int gate_mode,
                       int64_t gate_rows, float residual_scale, float eps, int dtype, void* out,
                       float* rstd, void* n, float* next_rstd, void* stream,
                       void* const* stage_events);
/* With dr = dout plus the next norm's gradient of out (as block_prenorm_bwd's)
 * and b = dr * gate * w:
 *   dresidual = residual_scale * dr;  dy = rstd * (b - yh * mean(b * yh)), or b
 *   without a post norm;  dw = sum over tokens of gate * dr * yh;  dgate = the
 *   sum of w * dr * yh over what shares the gate value;  dnext_w.
 *   dout [N, H], may be NULL (0) with next_w; dn, out, next_rstd needed with
 *   next_w; rstd, dw with w; dgate with a gate, in the gate's shape and dtype.
 *   dresidual may alias dout. */
int block_postnorm_bwd(const void* dout, const void* dn, const void* y, const void* out,
                       const void* w, const void* gate, const void* next_w, const float* rstd,
                       const float* next_rstd, int64_t N, int64_t H, int gate_mode,
                       int64_t gate_rows, float residual_scale, int dtype, void* dy,
                       void* dresidual, void* dw, void* dgate, void* dnext_w, void* workspace,
                       size_t workspace_bytes, void* stream, void* const* stage_events);

/* ---- activations in 8 bits ----------------------------------------------
 * A [R, C] activation kept for the backward pass as OCP e4m3 values q [R, C]
 * and one scale byte per 32 consecutive channels of a row, scale [R,
 * ceil(C / 32)] (a row's last group may be shorter): value = q * 2^(byte -
 * 127).  The exponent is the smallest of at least -127 for which the group's
 * largest finite magnitude is at most 448 * 2^e (no element saturates; zeros
 * have byte 0), and q is rounded to nearest even: a finite x is kept within
 * max(2^-4 |x|, 2^-10 * 2^e), the second where it lies below e4m3's normal
 * numbers, 2^-6 * 2^e; one up to 2^-10 * 2^e, some 2^-18 of its group's largest,
 * is kept as 0.  An element that is not finite is kept as NaN and takes no part
 * in the scale.  (A value next to the dtype's largest may round up past it, and
 * then unpacks to infinity.)
 * C is a positive multiple of 8 below 2^31, R < 2^31; row pitches (ld*, in
 * elements) are multiples of 8, at least C; q and scale are dense.  Tensor
 * pointers 16-byte aligned, q 8-byte.  Outputs must not alias inputs or each
 * other.  R == 0 is a no-op (pointers may be NULL).  One stage each. */
#define TOPMOE_ACT8_GROUP 32
int act8_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
              uint8_t* scale, void* stream, void* const* stage_events);
int act8_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C, int dtype, void* x,
                int64_t ldx, void* stream, void* const* stage_events);
/* h = SiLU(g) * u [R, C] (dense, rounded once), and g, u kept.  g and u may be
 * the halves of one [R, 2C] projection (pitch 2C). */
int swiglu_act8_fwd(const void* g, int64_t ldg, const void* u, int64_t ldu, int64_t R, int64_t C,
                    int dtype, void* h, uint8_t* gq, uint8_t* gscale, uint8_t* uq,
                    uint8_t* uscale, void* stream, void* const* stage_events);
/* From the kept g, u and dh [R, C] (dense): dg = dh * u * SiLU'(g),
 * du = dh * SiLU(g) (pitches lddg, lddu) and, when h is not NULL, h = SiLU(g) * u
 * again (dense). */
int swiglu_act8_bwd(const uint8_t* gq, const uint8_t* gscale, const uint8_t* uq,
                    const uint8_t* uscale, const void* dh, int64_t R, int64_t C, int dtype,
                    void* dg, int64_t lddg, void* du, int64_t lddu, void* h, void* stream,
                    void* const* stage_events);

/* The (g, u) that ffn_swiglu_fwd_train / moe_ffn_fwd_train left in `saved`, kept
 * in 8 bits instead: keep8 copies them (and the MoE's routing) into `kept`,
 * after which `saved` may be reused, and restore8 puts them, and h^T computed
 * from them, into a backward workspace, from which ffn_swiglu_bwd_saved /
 * moe_ffn_bwd with TOPMOE_MOE_BWD_SAVED run as after the training forward.
 * Between the passes a layer then holds about 2 N k I bytes (2 + 1/16 an
 * element pair) instead of its backward workspace.  The backward then computes
 * from the 8-bit g and u, each as near its value as act8_pack's; y and the
 * routing are as without it.
 *   saved, workspace   *_bwd_workspace_bytes(), kept  *_keep8_bytes(): 256-byte
 *   aligned.  kept holds, each part 256-byte aligned: the MoE's routing, g's
 *   q [rows, I] (rows = N, or N * k in the experts' row order), u's q, g's
 *   scale bytes [rows, I / 32], u's.
 * Shape limits and statuses as for the backward; *_keep8_bytes return 0 for
 * invalid shapes.  Stages: keep8 one, restore8 TOPMOE_RESTORE8_STAGES. */
#define TOPMOE_RESTORE8_STAGES 2  /* 0 routing (dense: empty), 1 g, u and h^T */
size_t ffn_keep8_bytes(int64_t N, int64_t H, int64_t I, int dtype);
int ffn_swiglu_keep8(const void* saved, size_t saved_bytes, int64_t N, int64_t H, int64_t I,
                     int dtype, void* kept, size_t kept_bytes, void* stream,
                     void* const* stage_events);
int ffn_swiglu_restore8(const void* kept, size_t kept_bytes, int64_t N, int64_t H, int64_t I,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream,
                        void* const* stage_events);
size_t moe_keep8_bytes(int64_t N, int64_t H, int64_t I, int E, int k, int dtype);
int moe_ffn_keep8(const void* saved, size_t saved_bytes, int64_t N, int64_t H, int64_t I, int E,
                  int k, int dtype, void* kept, size_t kept_bytes, void* stream,
                  void* const* stage_events);
int moe_ffn_restore8(const void* kept, size_t kept_bytes, int64_t N, int64_t H, int64_t I, int E,
                     int k, int dtype, void* workspace, size_t workspace_bytes, void* stream,
                     void* const* stage_events);

/* Human-readable text for a status code (static storage). */
const char* topmoe_strerror(int status);

/* Library ABI version (major * 100 + minor). */
int topmoe_version(void);

/* ---- instrumentation helpers (not on the hot path) ---------------------- */
/* Launch-shape override of one GEMM of the path, for tuning sweeps and tests.
 *   gemm   TOPMOE_TILE_GATEUP (forward gate/up), TOPMOE_TILE_DOWN (forward down
 *          and the backward's dx), TOPMOE_TILE_BWD_GU, TOPMOE_TILE_BWD_DH,
 *          TOPMOE_TILE_WGRAD_GU (dW_g + dW_u), TOPMOE_TILE_WGRAD_D (dW_d)
 *   shape  int[6] {block rows, block columns, wavefront rows, wavefront
 *          columns, LDS row bytes, ring depth}, or NULL to clear the override
 * Returns TOPMOE_ERR_BAD_ARG, changing nothing, if the library does not
 * instantiate that shape for that GEMM.  Initial overrides come from the
 * environment variables TOPMOE_GATEUP_TILE, TOPMOE_DOWN_TILE,
 * TOPMOE_BWDGU_TILE, TOPMOE_BWDDH_TILE, TOPMOE_WGU_TILE, TOPMOE_WD_TILE
 * ("BMxBNxWMxWNxRBxS"), read once, by the first call that plans a launch;
 * while one of them names a shape that is not instantiated, the calls that
 * would use it return TOPMOE_ERR_BAD_ARG before launching anything.  An
 * override applies to every dtype for which the shape is instantiated. */
#define TOPMOE_TILE_GATEUP 0
#define TOPMOE_TILE_DOWN 1
#define TOPMOE_TILE_BWD_GU 2
#define TOPMOE_TILE_BWD_DH 3
#define TOPMOE_TILE_WGRAD_GU 4
#define TOPMOE_TILE_WGRAD_D 5
int topmoe_set_tile_override(int gemm, const int* shape);

/* The launch plan moe_ffn_fwd (inference, flags without effect on it) follows
 * for a problem, computed on the host without touching a GPU: info[i] for
 * i < n receives field i below (-1 past the last).  Returns TOPMOE_OK, or the
 * status moe_ffn_fwd would return for the sizes, dtype or capacity factor
 * (NULL info with n > 0: TOPMOE_ERR_NULL_ARG). */
#define TOPMOE_PATH_ROUTER_LAYOUT 0  /* 0: W_router in LDS, 16 tokens per pass;
                                        1: one token at a time, H split over
                                        four wavefronts; 2: as 0, 16 lanes per token */
#define TOPMOE_PATH_ROUTER_TOKENS 1  /* tokens per router block                  */
#define TOPMOE_PATH_ROUTER_BLOCKS 2  /* router blocks                            */
#define TOPMOE_PATH_UP_BM 3          /* gate/up tile rows, columns, ring depth   */
#define TOPMOE_PATH_UP_BN 4
#define TOPMOE_PATH_UP_RING 5
#define TOPMOE_PATH_DOWN_BM 6        /* down tile rows, columns, ring depth      */
#define TOPMOE_PATH_DOWN_BN 7
#define TOPMOE_PATH_DOWN_RING 8
#define TOPMOE_PATH_DOWN_KSPLIT 9    /* K chunks of the down projection (1: none) */
#define TOPMOE_PATH_INBLOCK 10       /* 1: the GEMMs group the entries themselves
                                        (no permutation launch)                  */
#define TOPMOE_PATH_ROUTER_IN_UP 11  /* 1: the router runs as blocks of the gate/up
                                        launch, which takes every token against
                                        every expert (no router launch)          */
#define TOPMOE_PATH_FIELDS 12
int moe_ffn_fwd_path(int64_t N, int64_t H, int64_t I, int E, int k, float capacity_factor,
                     int dtype, int32_t* info, int n);

/* Create / destroy n timing-enabled hipEvent_t handles. */
int topmoe_events_create(int n, void** events);
int topmoe_events_destroy(int n, void** events);
/* Wait for `stop` and return the elapsed milliseconds between two events. */
int topmoe_event_elapsed_ms(void* start, void* stop, float* ms);

#ifdef __cplusplus
}
#endif
#endif /* TOPMOE_H */
