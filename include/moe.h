/*
 * moe.h -- C ABI of libmoe, the MI355X (gfx950) MoE expert block.
 *
 * The block, as the pages state the problem: a flat batch of token hidden
 * states goes through an fp32 router and a per-token top-k; the selected
 * (token, expert) rows are sorted by expert; each expert runs its SwiGLU FFN as
 * one grouped matmul over its contiguous rows; the rows come back to their
 * token in the same order, weighted by the top-k probabilities, and are summed
 * ("Halo's 2.8x over TRL is not a kernel, and its own benchmark proves it",
 * section "Where the gap actually is", EP token-routing figure and the EP
 * forward path described under it).  The backward computes the matching
 * activation, expert-weight and router gradients, with the routing adjoint
 * written as gathers, free of atomic adds ("Halo: Frontier-Lab Training for
 * Everyone", section "Some of the hard problems along the way").
 *
 * Conventions for every entry point:
 *  - Status: returns MOE_OK (0) or a negative MOE_ERR_*.  Arguments are
 *    validated on the host before anything is launched; an invalid call
 *    launches nothing and writes nothing.  moe_last_error() gives a message
 *    for the calling thread's last failure.
 *  - Memory: every tensor argument is a caller-owned DEVICE pointer (current
 *    HIP device), row-major and contiguous, 16-byte aligned.  The library
 *    never allocates device memory in these calls; scratch comes from the
 *    caller through a workspace pointer sized by the matching *_workspace_size
 *    query.
 *  - Streams: `stream` is a hipStream_t (NULL = the null stream).  Every call
 *    is asynchronous on that stream and makes no device-to-host copy; per
 *    expert counts and offsets stay on the device.
 *  - dtype: MOE_BF16 or MOE_F32 selects the storage type of activations and
 *    expert weights (x, w_r, w_gu, w_down, x_perm, gu, h, y_perm, y, dy, ...).
 *    Routing tensors are always fp32 / int32; weight and router gradients are
 *    always fp32.  MOE_F32 covers the forward path and the copy-type backward
 *    steps; moe_grouped_ffn_bwd and moe_router_logits_bwd need MOE_BF16.
 *  - Shapes: T >= 0 tokens, d = d_model, f = d_ff, E experts, k = top-k;
 *    1 <= k <= E <= 1024, k <= 32; d and f positive multiples of 8;
 *    R = T*k routed rows, R < 2^31.  Element offsets are computed in 64 bits.
 *  - Determinism: no floating-point atomics anywhere; repeated calls on the
 *    same inputs give bitwise identical results.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK               0
#define MOE_ERR_INVALID_ARG (-1)   /* null pointer, bad size, misalignment */
#define MOE_ERR_UNSUPPORTED (-2)   /* dtype / shape outside the supported set */
#define MOE_ERR_WORKSPACE   (-3)   /* workspace missing or too small */
#define MOE_ERR_HIP         (-4)   /* HIP launch or runtime error */

#define MOE_F32  0
#define MOE_BF16 1

/* Library version (major*10000 + minor*100 + patch). */
int moe_version(void);
/* Static description of a status code. */
const char *moe_strerror(int status);
/* Message for the calling thread's last failed call ("" if none). */
const char *moe_last_error(void);

/* ---------------------------------------------------------------- router */

/*
 * Router logits in fp32.  The pages fix the precision ("fp32 router logits" in
 * the EP forward path, section "Where the gap actually is"; `fp32_router:
 * true` in the recipe of section "The small-hardware end").  The summation
 * order is fixed as part of the definition so that top-k decisions are
 * reproducible bit for bit:
 *   logits[t,e] = ((fma chain over c = 0..d-1 of x[t,c]*w_r[e,c], from +0)
 *                  + bias[e]) + logit_add[t,e]
 * x: [T,d] (dtype), w_r: [E,d] (dtype), bias: [E] fp32 or NULL,
 * logit_add: [T,E] fp32 or NULL (additive noise), logits: [T,E] fp32 (out).
 */
int moe_router_logits(const void *x, const void *w_r, const float *bias,
                      const float *logit_add, int dtype, int64_t T, int d, int E,
                      float *logits, void *stream);

/*
 * Per-token top-k and the combine weights (the "per-token top-k router" and
 * "weighted by the top-k probabilities" of the EP token-routing figure).
 * topk_idx[t,0..k-1]: the k largest logits of token t, by value descending;
 * equal values go to the lower expert id (-0 equals +0); a NaN ranks below
 * every number (NaNs among themselves by lower id) and +-inf order as numbers,
 * so the selection is always defined.  topk_w[t,j] = softmax over the k
 * selected logits (NaN for every j when the selection holds a NaN or its
 * largest logit is +inf; finite logits are the intended use).
 * logits: [T,E] fp32; topk_idx: [T,k] int32 (out); topk_w: [T,k] fp32 (out).
 */
int moe_route(const float *logits, int64_t T, int E, int k,
              int32_t *topk_idx, float *topk_w, void *stream);

/* ---------------------------------------------------------------- permute */

size_t moe_permute_workspace_size(int64_t T, int E, int k);

/*
 * Sorts the selected (token, expert) slots by expert -- the single-GPU core of
 * the EP dispatch, which hands each expert its tokens "sorted by expert" (EP
 * token-routing figure).  Slot s = t*k + j.  Rows are expert-major; inside an
 * expert, slots keep ascending order.  Outputs:
 *   counts[E], offsets[E+1] (offsets[0]=0, offsets[E]=R), slot_to_row[R],
 *   row_to_slot[R] (int32);
 *   x_perm[r] = x[row_to_slot[r] / k]   (exact copy; x may be NULL to skip),
 *   w_perm[r] = topk_w[row_to_slot[r]]  (topk_w and w_perm may be NULL).
 * topk_idx entries must lie in [0,E) and a token's k entries must be distinct.
 * ws: device workspace of at least moe_permute_workspace_size(T,E,k) bytes.
 */
int moe_permute(const void *x, const int32_t *topk_idx, const float *topk_w, int dtype,
                int64_t T, int d, int E, int k,
                int32_t *counts, int32_t *offsets, int32_t *slot_to_row, int32_t *row_to_slot,
                void *x_perm, float *w_perm, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- experts */

size_t moe_grouped_ffn_workspace_size(int64_t R, int E, int d, int f, int dtype);

/*
 * Grouped SwiGLU expert FFN over rows sorted by expert ("grouped GEMM and
 * fused SwiGLU", "Halo: Frontier-Lab Training for Everyone", section "Novel
 * model integration example"; experts stored as single 3-D weight tensors,
 * section "One trainer architecture, one parallelism stack").  For each
 * expert e and each of its rows r in [offsets[e], offsets[e+1]):
 *   [g | u] = x_perm[r] . w_gu[e]^T        (gate rows 0..f-1, up rows f..2f-1)
 *   gu[r]   = store([g | u])                (store = dtype rounding)
 *   h[r]    = store(silu(gu_g) * gu_u),  silu(v) = v / (1 + exp(-v))
 *   y_perm[r] = store(row_scale[r] * (h[r] . w_down[e]^T))   (row_scale NULL = 1)
 * fp32 accumulation.  Experts with no rows are skipped.
 * x_perm: [R,d]; w_gu: [E,2f,d]; w_down: [E,d,f]; row_scale: [R] fp32 or NULL;
 * gu: [R,2f] (out, or NULL if not needed for a backward); h: [R,f] (out);
 * y_perm: [R,d] (out).  offsets: [E+1] int32 on the device, offsets[E] = R.
 */
int moe_grouped_ffn_fwd(const void *x_perm, const int32_t *offsets, int E, int64_t R,
                        int d, int f, const void *w_gu, const void *w_down,
                        const float *row_scale, int dtype, void *gu, void *h, void *y_perm,
                        void *ws, size_t ws_bytes, void *stream);

/*
 * moe_grouped_ffn_fwd without a workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Same arguments, results (bit for bit), errors and
 * conventions as moe_grouped_ffn_fwd minus ws / ws_bytes.  Its scratch -- the
 * forward's two tile-start tables with their tile counters -- lives in a
 * static device array of 8704 bytes (enough for E <= 1024; a larger need
 * returns MOE_ERR_UNSUPPORTED), one copy per device, held until the process
 * ends; its address is taken once per device on that device's first call.
 * The call allocates nothing and clears what it needs itself, in stream
 * order.  Every call on one device shares that array: calls that may run
 * concurrently on one device (different streams, or threads) race and must
 * be serialised by the caller.
 */
int moe_grouped_ffn_fwd_noalloc(const void *x_perm, const int32_t *offsets, int E, int64_t R,
                                int d, int f, const void *w_gu, const void *w_down,
                                const float *row_scale, int dtype, void *gu, void *h,
                                void *y_perm, void *stream);

/*
 * Backward of moe_grouped_ffn_fwd (expert weights receive gradients: the
 * "expert gradient all-to-all" that LoRA skips, section "One trainer
 * architecture, one parallelism stack", is the exchange of these).  Per row r
 * of expert e, with w = row_scale[r] (1 if NULL):
 *   Gd          = dy_perm[r] . w_down[e]                      (fp32)
 *   d_row_scale[r] = sum_c h[r,c] * Gd[c]                      (fp32)
 *   dH = w*Gd;  s = sigmoid(g);  dg = dH*u*s*(1 + g*(1-s));  du = dH*g*s
 *   dgu[r]      = store([dg | du])
 *   dx_perm[r]  = store(dgu[r] . w_gu[e])
 *   dw_down[e]  = sum_r store(w*dy_perm[r])^T (x) h[r]          (fp32, [E,d,f])
 *   dw_gu[e]    = sum_r dgu[r]^T (x) x_perm[r]                  (fp32, [E,2f,d])
 * (g, u = the stored gu; experts with no rows get exactly zero dw.)
 * Inputs: x_perm [R,d], gu [R,2f], h [R,f] (saved by the forward), dy_perm [R,d].
 * Outputs: dgu [R,2f], dx_perm [R,d], dw_gu, dw_down, d_row_scale [R] (or NULL).
 * dtype must be MOE_BF16.
 */
int moe_grouped_ffn_bwd(const void *x_perm, const void *gu, const void *h,
                        const int32_t *offsets, int E, int64_t R, int d, int f,
                        const void *w_gu, const void *w_down, const float *row_scale,
                        const void *dy_perm, int dtype, void *dgu, void *dx_perm,
                        float *dw_gu, float *dw_down, float *d_row_scale,
                        void *ws, size_t ws_bytes, void *stream);

/*
 * The grouped FFN with the row permutation folded into the GEMM operand
 * loads: the tokens go to their experts as one grouped matmul over the rows
 * sorted by expert ("Halo's 2.8x over TRL is not a kernel, and its own
 * benchmark proves it", section "Where the gap actually is"), and the sorted
 * rows are read from the token-major tensors where the GEMMs load them, so
 * x_perm and dy_perm are never stored.  Row r of the expert-sorted order is
 * token row_to_slot[r] / k (row_to_slot from moe_permute, which then needs no
 * x / x_perm).
 *
 * moe_grouped_ffn_fwd_gather: the results of moe_grouped_ffn_fwd with
 *   x_perm[r] = x[row_to_slot[r] / k]; x: [T,d] bf16, R = T*k.
 * moe_grouped_ffn_bwd_gather: the results of moe_grouped_ffn_bwd with that
 *   x_perm and dy_perm[r] = dy[row_to_slot[r] / k]; dy: [T,d] bf16;
 *   slot_to_row: [R], the inverse of row_to_slot (moe_permute writes both;
 *   S = w * dY_perm is formed from dY in token order through it).  x_perm:
 *   [R,d] or NULL; when given (the forward's permuted rows), the dW_gu GEMM
 *   reads it instead of gathering X, and x may be NULL.
 * Every other argument, output and the workspace
 * (moe_grouped_ffn_workspace_size(T*k, E, d, f, MOE_BF16)) are those of the
 * plain calls; bf16 only.  Limits (else MOE_ERR_UNSUPPORTED): k <= 32,
 * T*d < 2^30, T*k*k < 2^32.  row_to_slot must hold a permutation of
 * 0..T*k-1 and slot_to_row its inverse (as moe_permute writes them); other
 * values are not checked and index outside x, dy and the outputs.
 */
int moe_grouped_ffn_fwd_gather(const void *x, int64_t T, const int32_t *row_to_slot, int k,
                               const int32_t *offsets, int E, int d, int f,
                               const void *w_gu, const void *w_down, const float *row_scale,
                               void *gu, void *h, void *y_perm,
                               void *ws, size_t ws_bytes, void *stream);
int moe_grouped_ffn_bwd_gather(const void *x, const void *x_perm, const void *dy, int64_t T,
                               const int32_t *row_to_slot, const int32_t *slot_to_row, int k,
                               const void *gu, const void *h,
                               const int32_t *offsets, int E, int d, int f,
                               const void *w_gu, const void *w_down, const float *row_scale,
                               void *dgu, void *dx_perm, float *dw_gu, float *dw_down,
                               float *d_row_scale, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- combine */

/*
 * Returns each row to its token and sums ("the same rows in the same order",
 * EP token-routing figure; the weights were applied by the down projection):
 *   y[t] = store(sum over j = 0..k-1, ascending, of y_perm[slot_to_row[t*k+j]])
 * with an fp32 running sum.  y_perm: [R,d]; slot_to_row: [R]; y: [T,d] (out).
 */
int moe_combine(const void *y_perm, const int32_t *slot_to_row, int dtype,
                int64_t T, int d, int k, void *y, void *stream);

/*
 * Adjoint of moe_combine: a copy of each token's gradient to its k rows,
 *   dy_perm[slot_to_row[t*k+j]] = dy[t].
 * The combine returns each expert output row to its token ("Halo's 2.8x over
 * TRL is not a kernel, and its own benchmark proves it", section "Where the
 * gap actually is", EP token-routing figure); its adjoint is written as this
 * copy through the forward's own map, a gather with no atomic adds ("Halo:
 * Frontier-Lab Training for Everyone", section "Some of the hard problems
 * along the way", on the atomic-free routing backward).  dy: [T,d] (dtype);
 * slot_to_row: [T*k] int32 from moe_permute; dy_perm: [T*k,d] (out, every row
 * written once).  Errors as moe_combine.
 */
int moe_combine_bwd(const void *dy, const int32_t *slot_to_row, int dtype,
                    int64_t T, int d, int k, void *dy_perm, void *stream);

/*
 * Adjoint of the row permutation, as a gather (no atomic adds; "Halo:
 * Frontier-Lab Training for Everyone", section "Some of the hard problems
 * along the way"):
 *   dx[t] = store(sum over j ascending of dx_perm[slot_to_row[t*k+j]] + dx_add[t])
 * with an fp32 running sum; dx_add: [T,d] fp32 or NULL (the router's share).
 */
int moe_permute_bwd(const void *dx_perm, const int32_t *slot_to_row, const float *dx_add,
                    int dtype, int64_t T, int d, int k, void *dx, void *stream);

/* ---------------------------------------------------------------- grouped LoRA */

/*
 * LoRA on the fused expert weights with the experts frozen ("Halo:
 * Frontier-Lab Training for Everyone", section "One trainer architecture, one
 * parallelism stack": a grouped LoRA that adapts the 3-D expert tensors
 * directly, so the frozen experts need no gradients).  Per expert e, rank r,
 * scale s: W_gu[e] + s B_gu[e] A_gu[e] and W_down[e] + s B_dn[e] A_dn[e] with
 * a_gu [E,r,d], b_gu [E,2f,r] (gate rows then up rows), a_dn [E,r,f],
 * b_dn [E,d,r], all bf16, caller-owned device memory.  r is a multiple of 16,
 * 16 <= r <= 64; dtype must be MOE_BF16; other shapes, errors and conventions
 * as moe_grouped_ffn_fwd / _bwd.  Stored intermediates (bf16, [R,r]):
 *   z_gu = store(s X_perm A_gu^T),  z_dn = store(s H A_dn^T)      (forward outputs)
 * forward:  GU = store(X_perm W_gu^T + z_gu B_gu^T) (one fp32 accumulation:
 *           the rank-r product is one more K stage of the grouped GEMM),
 *           H = store(silu(g) u),  Y_perm = store(w (H W_down^T + z_dn B_dn^T)).
 * backward: u_dn = store(s dY_perm B_dn);  Gd = dY_perm W_down + u_dn A_dn
 *           feeds the dSwiGLU epilogue and d_row_scale as in moe_grouped_ffn_bwd;
 *           u_gu = store(s dGU B_gu);  dX_perm = store(dGU W_gu + u_gu A_gu);
 *           dB_gu = dGU^T z_gu [E,2f,r], dA_gu = u_gu^T X_perm [E,r,d],
 *           dB_dn = S^T z_dn [E,d,r] (S = store(w dY_perm)),
 *           dA_dn = store(w u_dn)^T H [E,r,f]; fp32, fully written (zeros for
 *           empty experts).  No expert weight gradients are formed.
 * ws: moe_grouped_ffn_lora_workspace_size(R,E,d,f,r) bytes for either call.
 */
size_t moe_grouped_ffn_lora_workspace_size(int64_t R, int E, int d, int f, int r);
int moe_grouped_ffn_fwd_lora(const void *x_perm, const int32_t *offsets, int E, int64_t R, int d,
                             int f, const void *w_gu, const void *w_down, const float *row_scale,
                             const void *a_gu, const void *b_gu, const void *a_dn,
                             const void *b_dn, int r, float scale, int dtype, void *z_gu,
                             void *z_dn, void *gu, void *h, void *y_perm, void *ws,
                             size_t ws_bytes, void *stream);
int moe_grouped_ffn_bwd_lora(const void *x_perm, const void *gu, const void *h,
                             const int32_t *offsets, int E, int64_t R, int d, int f,
                             const void *w_gu, const void *w_down, const float *row_scale,
                             const void *dy_perm, const void *a_gu, const void *b_gu,
                             const void *a_dn, const void *b_dn, int r, float scale,
                             const void *z_gu, const void *z_dn, int dtype, void *dgu,
                             void *dx_perm, float *d_row_scale, float *da_gu, float *db_gu,
                             float *da_dn, float *db_dn, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * Where moe_grouped_ffn_bwd_lora leaves its stored rank-r rows in the
 * workspace `ws` it was given (same R, E, d, f, r): u_dn = store(s dY_perm
 * B_dn), uw_dn = store(w u_dn) (written only when row_scale was given) and
 * u_gu = store(s dGU B_gu), each [R,r] bf16 row-major.  The values are those
 * of the last backward call on that workspace, in stream order.  For
 * inspection and tests; the pointers alias ws and are not to be freed.
 * Errors: NULL pointers or r not in {16,32,48,64}: MOE_ERR_INVALID_ARG;
 * ws_bytes below moe_grouped_ffn_lora_workspace_size: MOE_ERR_WORKSPACE.
 */
int moe_grouped_ffn_lora_bwd_saved(const void *ws, size_t ws_bytes, int64_t R, int E, int d,
                                   int f, int r, const void **u_dn, const void **uw_dn,
                                   const void **u_gu);

/*
 * moe_permute_bwd with the router's share of the token gradient formed in the
 * same pass instead of read from memory:
 *   dx[t] = store(sum_{j asc} fp32(dx_perm[slot_to_row[t*k+j]]) + r[t]),
 *   r[t,:] = d_logits[t,:] . w_r  (fp32 fma chain over e ascending from +0,
 *            entries with d_logits == 0 skipped),
 * bit for bit what moe_router_logits_bwd's dx_router followed by
 * moe_permute_bwd gives, without storing dx_router ([T,d] fp32).  Same
 * pass as B6 of the backward; the router term is B8's dX (the router linear
 * map's adjoint, "fp32 router logits" in "Halo's 2.8x over TRL is not a
 * kernel, and its own benchmark proves it", section "Where the gap actually
 * is").  d_logits: [T,E] fp32; w_r: [E,d] (dtype); 1 <= E <= 1024; other
 * arguments and errors as moe_permute_bwd.
 */
int moe_permute_bwd_router(const void *dx_perm, const int32_t *slot_to_row, const float *d_logits,
                           const void *w_r, int dtype, int64_t T, int d, int E, int k, void *dx,
                           void *stream);

/* ---------------------------------------------------------------- router bwd */

/*
 * Adjoint of the softmax over the selected logits.  The routers are trained:
 * they receive the gradient of the loss through the combine weights (the
 * TorchTurbo page, "inclusionAI open-sources TorchTurbo, a SuperNode-native
 * post-training engine", section "Adapter": the routers apply the gradient of
 * the auxiliary loss, so they carry gradients), and the combine weights are
 * the top-k probabilities of the fp32 router ("Halo's 2.8x over TRL is not a
 * kernel, and its own benchmark proves it", section "Where the gap actually
 * is", EP token-routing figure).  With g_j =
 * d_row_scale[slot_to_row[t*k+j]] (the gradient of the loss with respect to
 * topk_w[t,j]):
 *   d_topk_w[t,j] = g_j                         (d_topk_w may be NULL)
 *   d_logits[t,topk_idx[t,j]] = w_j * (g_j - sum_i w_i g_i), 0 elsewhere.
 * All fp32; d_logits: [T,E] (out, fully written).  topk_idx / topk_w: [T,k]
 * from moe_route; d_row_scale: [T*k] from moe_grouped_ffn_bwd; slot_to_row:
 * [T*k] from moe_permute.  Invalid sizes or NULL required pointers:
 * MOE_ERR_INVALID_ARG, nothing launched.
 */
int moe_route_bwd(const int32_t *topk_idx, const float *topk_w, const float *d_row_scale,
                  const int32_t *slot_to_row, int64_t T, int E, int k,
                  float *d_topk_w, float *d_logits, void *stream);

size_t moe_router_logits_bwd_workspace_size(int64_t T, int d, int E);

/*
 * Adjoint of the router linear map that forms the fp32 router logits ("fp32
 * router logits" in the EP forward path, "Halo's 2.8x over TRL is not a
 * kernel, and its own benchmark proves it", section "Where the gap actually
 * is"; the routers are trained, the TorchTurbo page, section "Adapter").  Bias
 * and added noise carry no gradient:
 *   dx_router = d_logits . w_r    ([T,d] fp32, or NULL to skip)
 *   dw_r      = d_logits^T . x    ([E,d] fp32, or NULL to skip)
 * fp32 accumulation in a fixed order: dx_router as an fma chain over e
 * ascending (zero entries skipped), dw_r as per-chunk partials over 256-token
 * chunks summed in chunk order.  x: [T,d], w_r: [E,d] (dtype); d_logits:
 * [T,E] fp32.  dtype must be MOE_BF16.  ws:
 * moe_router_logits_bwd_workspace_size(T,d,E) bytes (MOE_ERR_WORKSPACE if
 * smaller).
 */
int moe_router_logits_bwd(const void *x, const void *w_r, const float *d_logits, int dtype,
                          int64_t T, int d, int E, float *dx_router, float *dw_r,
                          void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- router variants */

/*
 * The pages name three router features without giving formulas: balancing
 * through a bias on expert selection for a model family without a router
 * auxiliary loss ("Halo's 2.8x over TRL is not a kernel, and its own benchmark
 * proves it", section "The small-hardware end": the LFM2 config,
 * `moe_balancing: bias_update`, and the paragraph after it); a router
 * load-balancing auxiliary loss with a per-run coefficient whose gradient the
 * routers apply and whose unscaled and scaled values they report (the
 * TorchTurbo page, "inclusionAI open-sources TorchTurbo, a SuperNode-native
 * post-training engine", section "Adapter", ms-swift DPO); and MoE statistics
 * that ignore the right-padded tail of a batch, the valid prefix being n_valid
 * tokens (same TorchTurbo page, section "Model", sequence-parallel input
 * contract).  The formulas below are the plainest readings.
 */

/*
 * Top-k on the selection score fp32(logits[t,e] + sel_bias[e]) (by value
 * descending, equal scores to the lower expert id, as moe_route); topk_w[t,j]
 * is the softmax over the k selected logits WITHOUT the bias, so the bias only
 * steers which experts are chosen.  sel_bias: [E] fp32, not NULL (moe_route
 * is the unbiased call).  Other arguments and errors as moe_route; moe_route_bwd
 * is the adjoint with respect to the logits (the bias gets no gradient).
 */
int moe_route_biased(const float *logits, const float *sel_bias, int64_t T, int E, int k,
                     int32_t *topk_idx, float *topk_w, void *stream);

size_t moe_expert_load_workspace_size(int64_t T, int E, int k);

/*
 * Expert load over the valid prefix: load[e] = number of slots (t, j) with
 * t < n_valid and topk_idx[t,j] = e (ids outside [0,E) are not counted).
 * 0 <= n_valid <= T, else MOE_ERR_INVALID_ARG.  topk_idx: [T,k] int32;
 * load: [E] int32 (out, fully written; all zero when n_valid = 0).  Exact and
 * deterministic (per-block integer histograms summed in block order).
 * ws: moe_expert_load_workspace_size(T,E,k) bytes.
 */
int moe_expert_load(const int32_t *topk_idx, int64_t T, int64_t n_valid, int E, int k,
                    int32_t *load, void *ws, size_t ws_bytes, void *stream);

/*
 * Selection-bias balancing step, in place:
 *   sel_bias[e] += rate * sign(n_valid*k/E - load[e])
 * (under-loaded experts are raised, over-loaded lowered, an expert exactly at
 * the mean load is unchanged; the sign is decided exactly in integers; one fp32
 * add per expert).  load from moe_expert_load with the same n_valid.  rate must
 * be finite and >= 0.  load: [E] int32; sel_bias: [E] fp32 (in/out).
 */
int moe_bias_update(const int32_t *load, int64_t n_valid, int E, int k, float rate,
                    float *sel_bias, void *stream);

size_t moe_aux_loss_workspace_size(int64_t T, int E);

/*
 * Load-balancing auxiliary loss over the valid prefix (n = n_valid):
 *   p[t,:] = softmax(logits[t,:]) over all E experts (fp32),
 *   P_e = (1/n) sum_{t<n} p[t,e],  f_e = load[e] / (n k),
 *   aux = E * sum_e f_e P_e  (= 1 for balanced load and uniform p),
 *   aux_out[0] = aux, aux_out[1] = coeff * aux.
 * If d_logits is not NULL the gradient of coeff*aux with respect to the logits
 * is ADDED to it (the load is a count and carries none):
 *   d_logits[t,e] += p[t,e] (g_e - sum_e' p[t,e'] g_e'),  g_e = coeff E load[e] / (n^2 k),
 * for t < n; rows t >= n are not touched.  n = 0 writes aux_out = {0, 0} and
 * touches nothing else.  logits: [T,E] fp32; load: [E] int32 from moe_expert_load
 * with the same n_valid; aux_out: [2] fp32 (out); d_logits: [T,E] fp32 (in/out)
 * or NULL; coeff must be finite.  Deterministic: per-block partial sums
 * combined in a fixed order.  ws: moe_aux_loss_workspace_size(T,E) bytes.
 * (Beside moe_route_scored with sigmoid scores this is not the loss of the
 * router's own scores.)
 */
int moe_aux_loss(const float *logits, const int32_t *load, int64_t T, int64_t n_valid, int E,
                 int k, float coeff, float *aux_out, float *d_logits, void *ws, size_t ws_bytes,
                 void *stream);

/*
 * Routing by scores over all E experts.  The other form of a router beside
 * moe_route's softmax over the k selected logits: every expert has a score,
 *   score MOE_SCORE_SOFTMAX: s_e = exp(x_e) / sum_i exp(x_i)
 *         MOE_SCORE_SIGMOID: s_e = 1 / (1 + exp(-x_e)),      x = logits[t,:],
 * the experts compete by c_e = s_e + sel_bias[e] (sel_bias NULL: by x_e
 * itself, which orders them as s_e does), and the weights are those of the
 * selected scores without the bias:
 *   topk_w[t,j] = scale * s_j / sum_i s_i  (renorm != 0; i over the k selected)
 *                 scale * s_j              (renorm == 0).
 * Groups: the experts form n_group groups of E / n_group consecutive ids; a
 * group's value is its largest c_e (group_top 1) or the sum of its two
 * largest (group_top 2; s_e in place of c_e without a bias), and only experts
 * of the topk_group groups of largest value can be selected.  n_group 1, or
 * topk_group = n_group: no restriction.
 * Every comparison decides as arithmetic in 64 bits on the fp32 logits and
 * bias does; equal values go to the lower id (group or expert), a NaN ranks
 * below every number (in a group's value it counts as -inf).  topk_idx is in
 * descending order of c_e.  Logits of -inf (masked experts) have score 0;
 * with renorm, a selection of scores that are all 0 gets weights 0 (scores
 * too small for fp32 still share the weight in proportion).  A NaN logit makes
 * its own sigmoid score, or all softmax scores of its row, NaN, and +inf the
 * softmax scores of its row; with renorm only what is selected matters.  sel_bias must be finite.
 * 1 <= n_group <= 32 and a divisor of E; group_top 2 needs groups of two
 * experts or more; k <= topk_group * E / n_group; scale positive and finite;
 * T < 2^26; logits 16-byte aligned.  Outputs as moe_route's.
 */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
int moe_route_scored(const float *logits, const float *sel_bias, int64_t T, int E, int k,
                     int score, int n_group, int topk_group, int group_top, int renorm,
                     float scale, int32_t *topk_idx, float *topk_w, void *stream);

/*
 * Adjoint of moe_route_scored's weights with respect to the logits (the
 * selection and the bias carry no gradient).  With g_j = d_row_scale[
 * slot_to_row[t*k+j]] (0 for a negative row; slot_to_row NULL: g_j =
 * d_row_scale[t*k+j]), w_j = topk_w[t,j], p_j = w_j / scale, m = sum_i p_i g_i:
 *   d_topk_w[t,j] = g_j                                  (d_topk_w may be NULL)
 *   d_logits[t,e] = 0 but, for e = topk_idx[t,j],
 *     sigmoid, renorm:  w_j (1 - s_j) (g_j - m)     plain:  w_j (1 - s_j) g_j
 *     softmax, renorm:  w_j (g_j - m)
 *   softmax, plain (every e): -scale s_e m, and w_j g_j added at the selected.
 * d_logits: [T,E] (out, fully written); it can be given to
 * moe_router_logits_bwd and moe_permute_bwd_router.  score, renorm and scale
 * as in the forward call; topk_idx distinct within a token (an id outside
 * [0,E) gets nothing); logits, d_logits 16-byte aligned; the two must not
 * overlap.  A row whose weights are all 0 gets zeros.
 */
int moe_route_scored_bwd(const float *logits, const int32_t *topk_idx, const float *topk_w,
                         const float *d_row_scale, const int32_t *slot_to_row, int64_t T, int E,
                         int k, int score, int renorm, float scale, float *d_topk_w,
                         float *d_logits, void *stream);

/* ---------------------------------------------------------------- 8-bit experts */

/*
 * Expert products in 8-bit floating point with a scale for each block of 128.
 * Values are e4m3 (OCP: largest 448, no infinity, NaN 0x7f / 0xff), one byte
 * each.  A block's scale is a power of two 2^s, stored as the byte s + 127:
 * s is the smallest integer >= -127 with (largest finite |x| of the block)
 * <= 448 * 2^s, and 0 for a block without a finite nonzero value; the stored
 * value is x * 2^-s rounded to e4m3 (nearest even).  NaN and infinities
 * become NaN, so that they reach the result.
 *  - Rows (activations) [R,K]: a scale per 128 consecutive k of a row,
 *    [R, moe_fp8_scale_cols(K)] bytes.
 *  - Weights [E,N,K]: a scale per 128 (n) x 128 (k),
 *    [E, ceil(N/128), moe_fp8_scale_cols(K)] bytes.
 * moe_fp8_scale_cols(K) = ceil(K/128) rounded up to a multiple of 4; the
 * padding bytes hold 127 and no value depends on them.  All sizes are
 * multiples of 16 from 16 to 65536; 1 <= E <= 1024; R < 2^31; pointers
 * 16-byte aligned.  Products accumulate in fp32, after the matrix
 * instruction has added each 8 consecutive k with at least 13 bits below the
 * largest of their products (the gate/up product of few rows per expert adds
 * them whole).  R, E and the sizes decide which kernel forms a product, and with
 * it the order of these sums: a row's result depends on its own values and on
 * those sizes, and on no other row.  Launches of another R or E, an expert
 * split among several included, may differ in it by the sums' errors, and where
 * such a sum is rounded to 8 bits (h) by a step of e4m3.  Rows at or past
 * offsets[E] are not read and not written.  Offsets that are no ascending
 * sequence in [0,R] are clamped to it and give unspecified rows.
 */
int moe_fp8_scale_cols(int K);

/* Rows x [R,K] (dtype MOE_BF16 or MOE_F32) to q [R,K] and scale. */
int moe_quant_rows_fp8(const void *x, int dtype, int64_t R, int K, uint8_t *q, uint8_t *scale,
                       void *stream);

/*
 * Expert weights w [E,N,K] (dtype MOE_BF16 or MOE_F32) to q [E,N,K] and scale.
 * With qt and scale_t (both or neither NULL) also the transposed weights
 * qt [E,K,N], scale_t [E, ceil(K/128), moe_fp8_scale_cols(N)]: the same
 * values (a square block keeps its scale), laid out for the product that
 * forms the gradient of the rows.
 */
int moe_quant_weights_fp8(const void *w, int dtype, int E, int N, int K, uint8_t *q,
                          uint8_t *scale, uint8_t *qt, uint8_t *scale_t, void *stream);

/*
 * Grouped product over rows sorted by expert: for each expert e and each of
 * its rows r in [offsets[e], offsets[e+1]), with A and B the values that
 * bytes and scales stand for,
 *   c[r,n] = bf16(row_scale[r] * sum_k A[r,k] B[e,n,k])   (row_scale NULL = 1).
 * a [R,K], a_scale; or, with row_to_slot (as moe_permute writes it) and k,
 * unpermuted token rows a [R/k, K]: row r reads token row_to_slot[r] / k
 * (R a multiple of k, k <= 32, (R/k) * K < 2^31, R * k < 2^32; entries
 * outside [0,R) read zeros).  row_to_slot NULL: k is ignored.  b [E,N,K],
 * b_scale; c: [R,N] bf16 (out).  With the transposed weights of
 * moe_quant_weights_fp8 and the quantised output gradient as a, c is the
 * gradient of the rows.
 */
int moe_grouped_gemm_fp8(const uint8_t *a, const uint8_t *a_scale, const int32_t *row_to_slot,
                         int k, const int32_t *offsets, int E, int64_t R, int N, int K,
                         const uint8_t *b, const uint8_t *b_scale, const float *row_scale,
                         void *c, void *stream);

/*
 * moe_grouped_ffn_fwd with 8-bit weights and activations (frozen experts:
 * rollouts, serving).  Per row r of expert e:
 *   [g | u] = X[r] . W_gu[e]^T      (fp32; gate rows 0..f-1, up rows f..2f-1)
 *   h[r]    = 8 bits of silu(g) * u, as moe_quant_rows_fp8 (h, h_scale: out)
 *   y_perm[r] = bf16(row_scale[r] * (H[r] . W_down[e]^T))
 * x, x_scale: rows [R,d], or token rows with row_to_slot and k as above;
 * w_gu [E,2f,d], w_gu_scale [E, ceil(2f/128), moe_fp8_scale_cols(d)];
 * w_down [E,d,f], w_down_scale [E, ceil(d/128), moe_fp8_scale_cols(f)];
 * h [R,f], h_scale [R, moe_fp8_scale_cols(f)]; y_perm [R,d] bf16.
 */
int moe_grouped_ffn_fwd_fp8(const uint8_t *x, const uint8_t *x_scale, const int32_t *row_to_slot,
                            int k, const int32_t *offsets, int E, int64_t R, int d, int f,
                            const uint8_t *w_gu, const uint8_t *w_gu_scale,
                            const uint8_t *w_down, const uint8_t *w_down_scale,
                            const float *row_scale, uint8_t *h, uint8_t *h_scale, void *y_perm,
                            void *stream);

/* ---------------------------------------------------------------- around the block */

/*
 * The residual stream around a block: the norm of the block's output, its
 * gate, the scaled residual, and the norm before the next block, in one pass.
 * With r(v) = (mean over the row of v^2 + eps)^-1/2, over each row t:
 *   p      = y r(y) w_post                         (y where w_post is NULL)
 *   out    = store(res_scale x + gate p)           (x NULL: gate p)
 *   n      = store(out r(out) w_pre)               (w_pre NULL: not formed)
 * in fp32; the second norm is of the stored out, which is all that a backward
 * has.  y NULL: n = store(x r(x) w_pre) alone, and out, w_post and gate are
 * NULL, res_scale 1.
 * x, y, out, n: [T,d] (dtype); w_post, w_pre: [d] (dtype); gate by gate_kind:
 * MOE_GATE_NONE NULL, _CHANNEL [d] (dtype), _TOKEN [T] fp32, _ELEMENT [T,d]
 * (dtype).  rstd_post, rstd_pre: [T] fp32, r(y) and r(out) (out, or NULL).
 * out may be x, n may be y; else no two tensors may overlap.  d a multiple of
 * 8, at most 16384; T at most 2^26 - 4 (the gradient: 2^26 - 1), and T times the
 * row's waves (up to 16) below 2^26 too (MOE_ERR_UNSUPPORTED).  Null or
 * misaligned pointers, a norm's rstd or n without its weight, a gate that does
 * not go with gate_kind (a channel's also where T = 0), eps <= 0:
 * MOE_ERR_INVALID_ARG, nothing launched.  The sum of a row's squares is formed
 * in another order where T is below 2048 (rows of 1 to 8 KB): its last bits
 * depend on that, and on no other row.
 */
#define MOE_GATE_NONE    0
#define MOE_GATE_CHANNEL 1
#define MOE_GATE_TOKEN   2
#define MOE_GATE_ELEMENT 3
int moe_residual_norm(const void *x, const void *y, const void *gate, int gate_kind,
                      const void *w_post, const void *w_pre, float res_scale, float eps, int dtype,
                      int64_t T, int d, void *out, void *n, float *rstd_post, float *rstd_pre,
                      void *stream);

/*
 * Gradient of moe_residual_norm.  d_out: [T,d], the gradient that reaches out
 * by the stream (NULL: none); d_n: [T,d], that of n (NULL exactly where w_pre
 * is); out, y, gate, w_post, w_pre, rstd_post, rstd_pre, res_scale as the
 * forward had or gave them (out is read for w_pre only, y for w_post or
 * d_gate only).  With D the whole gradient of out:
 *   D   = d_out + rn (q - out rn^2 mean(q out)),  q = d_n w_pre, rn = rstd_pre
 *   d_x = store(res_scale D),   P = gate D
 *   d_y = store(rp (P w_post - y rp^2 mean(P w_post y))), rp = rstd_post (P without w_post)
 *   d_w_pre = sum_t d_n out rn,  d_w_post = sum_t P y rp,      [d] fp32
 *   d_gate  = D p, summed over what the gate is shared by: [d] fp32, [T] fp32
 *             or [T,d] (dtype)
 * Each output may be NULL.  After moe_residual_norm with y NULL: out is its x,
 * y, gate and w_post are NULL and d_x is the gradient.  d_x may be d_out; else
 * no output may overlap another tensor.  Sums over t are formed in a fixed
 * order.  T = 0 gives zero weight gradients.  ws:
 * moe_residual_norm_bwd_workspace_size(T,d) bytes, needed for d_w_pre,
 * d_w_post and a channel gate's gradient (MOE_ERR_WORKSPACE if smaller); calls
 * that may overlap, also in captured graphs, need one each.
 */
size_t moe_residual_norm_bwd_workspace_size(int64_t T, int d);
int moe_residual_norm_bwd(const void *d_out, const void *d_n, const void *out, const void *y,
                          const void *gate, int gate_kind, const void *w_post, const void *w_pre,
                          const float *rstd_post, const float *rstd_pre, float res_scale, int dtype,
                          int64_t T, int d, void *d_x, void *d_y, float *d_w_post, float *d_w_pre,
                          void *d_gate, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_combine with the weights applied where the rows come back ("weighted by
 * the top-k probabilities", EP token-routing figure), for expert rows that do
 * not carry them yet (row_scale NULL in the expert calls):
 *   y[t] = store(sum over j ascending, an fp32 fma chain from +0, of
 *                weights[t*k+j] y_perm[slot_to_row[t*k+j]])
 * y_perm: [R,d].  A slot_to_row entry outside [0,R) has no row and adds
 * nothing; what y_perm holds for rows that no slot names is not read.
 * weights: [T,k] fp32, by slot.  d a multiple of 8, a row below 2^31 bytes; T*k
 * below 2^31, T times a row's pieces of 2 KB at most 2^26 - 4.  Sizes outside of
 * what a call takes: MOE_ERR_UNSUPPORTED; null or misaligned pointers, T or R
 * below 0: MOE_ERR_INVALID_ARG; nothing is launched then.
 */
int moe_combine_weighted(const void *y_perm, int64_t R, const int32_t *slot_to_row,
                         const float *weights, int dtype, int64_t T, int d, int k, void *y,
                         void *stream);

/*
 * Gradient of moe_combine_weighted: for every slot s = t*k+j that has a row r,
 *   dy_perm[r] = store(weights[s] dy[t]),   d_row_scale[r] = <dy[t], y_perm[r]>
 * by row, as moe_route_bwd and moe_route_scored_bwd read it; y_perm, dy_perm
 * [R,d], d_row_scale [R].  Rows that no
 * slot names are left as they were.  dy_perm or d_row_scale may be NULL, y_perm too
 * where d_row_scale is; dy_perm may not overlap y_perm.  No two slots may
 * name the same row.  T*k at most 2^26 - 4.
 */
int moe_combine_weighted_bwd(const void *dy, const void *y_perm, int64_t R,
                             const int32_t *slot_to_row, const float *weights, int dtype, int64_t T,
                             int d, int k, void *dy_perm, float *d_row_scale, void *stream);

/*
 * moe_combine_weighted (weights NULL: moe_combine) and moe_residual_norm on
 * its rows in one pass, bit for bit what the two calls give: y, the combined
 * rows [T,d], is stored for a backward, or NULL; y may not overlap another
 * tensor.  Arguments, limits and errors as moe_residual_norm's; R below 0, k
 * outside of 1 to 32 or T*k of 2^31 and more: MOE_ERR_INVALID_ARG.
 */
int moe_combine_residual_norm(const void *y_perm, int64_t R, const int32_t *slot_to_row,
                              const float *weights, int k, const void *x, const void *gate,
                              int gate_kind, const void *w_post, const void *w_pre, float res_scale,
                              float eps, int dtype, int64_t T, int d, void *y, void *out, void *n,
                              float *rstd_post, float *rstd_pre, void *stream);

/* ---------------------------------------------------------------- optimizer */

/*
 * One AdamW step over n tensors (the pages' trainer keeps bf16 weights with
 * stochastic rounding and identically seeded random numbers: "Halo:
 * Frontier-Lab Training for Everyone").  For each element, in fp32, each
 * operation rounded by itself, g = grad * grad_scale[0] (1 if NULL):
 *   m = beta1 m + (1-beta1) g,   v = beta2 v + ((1-beta2) g) g
 *   p = p (1 - lr weight_decay) - lr/(1-beta1^step) m / (sqrt(v)/sqrt(1-beta2^step) + eps)
 * (root and reciprocal to 1 ulp).  param: param_dtype; grad: grad_dtype, fp32
 * or, for bf16 parameters, bf16.  A bf16 parameter has a 32-bit copy `master`,
 * which is what is stepped and then rounded to nearest, or (all tensors of a
 * call alike) none; then p is rounded at random between its two bf16
 * neighbours, the upper with the probability of p's place between them.
 * State: state_bits 32: m, v [numel] fp32.  8: m [numel] e4m3, v [numel] e5m2,
 * and a power of two 2^s for each 128 elements, m_scale and v_scale
 * [ceil(numel/128)], the byte s + 127: s >= -126 the smallest with the block's
 * largest finite magnitude <= 448 2^s (m) or 57344 2^s (v).  Both are rounded
 * at random like p, with 16 random bits; a v that is not zero is at least the
 * smallest code, since its root divides.  NaN and infinities become 0x7f.
 * Zero bytes with scale bytes of 127 are the state before the first step.
 * Random bits: with mix(a): a ^= a >> 16, a *= 0x971cbef1, a ^= a >> 15,
 * a *= 0x6a695495, a ^= a >> 16 (32 bits),
 *   key = mix(mix(mix(mix(seed & 0xffffffff) ^ seed >> 32) ^ step) ^ i) ^ (e >> 32)
 *   r   = mix(key ^ (e & 0xffffffff)) for element e of tensors[i];
 * p takes r's low half, m its high half, v the high half of r * 0x30e9132d.
 * 0 <= beta < 1, eps in [1e-30, 1e30), lr and weight_decay finite.
 * step: 1, 2, ... below 2^32.  lr_dev (fp32) and step_dev (int64), both or
 * neither: the learning rate and the step count are read from the device, for
 * a captured step; lr and step are not used, and 1-beta^step is formed in fp32.
 * tensors: a HOST array, read before the call returns.  Tensors with numel 0
 * are skipped; a param, master, m or v that is listed twice is refused, and no
 * two may overlap.  param, grad, master, m, v 16-byte aligned.
 */
typedef struct moe_adamw_tensor {
  void *param;
  const void *grad;
  float *master;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  int64_t numel;
  double weight_decay;
} moe_adamw_tensor;
int moe_adamw_step(const moe_adamw_tensor *tensors, int n, int param_dtype, int grad_dtype,
                   int state_bits, double lr, double beta1, double beta2, double eps, int64_t step,
                   uint64_t seed, const float *grad_scale, const float *lr_dev,
                   const int64_t *step_dev, void *stream);

/* ---------------------------------------------------------------- timing */

/*
 * Per-kernel timing for measurement.  While enabled, every kernel launch is
 * bracketed by a pair of HIP events on its own stream.  moe_timing_query
 * waits for the recorded events and returns, for launches recorded under
 * `name` (NULL = all), the summed duration in milliseconds and the launch
 * count.  moe_timing_reset drops all records.  Off by default.  Launch names:
 * router_logits, route_topk, permute_hist, permute_scan, permute_place,
 * permute_rows, tile_prefix, gg_fwd_gate_up_swiglu, gg_fwd_down_scale,
 * combine, combine_bwd, gg_bwd_dh_dswiglu, drs_reduce, gg_bwd_dx,
 * gg_bwd_dw_down, gg_bwd_dw_gate_up, route_bwd, router_dx, router_dw_partial,
 * router_dw_reduce, router_dw_zero, permute_bwd, ffn_gu_f32, ffn_down_f32,
 * route_topk_biased, expert_load, expert_load_reduce, bias_update, aux_loss,
 * aux_loss_final, lora_proj, lora_transpose, lora_grad,
 * gg_fwd_gate_up_swiglu_gather, gg_bwd_dh_dswiglu_gather, row_scale,
 * gg_bwd_dw_gate_up_gather, route_scored, route_scored_bwd, quant_rows_fp8,
 * quant_weights_fp8, gg_fp8, gg_fp8_gate_up, gg_fp8_down, residual_norm,
 * combine_residual_norm, residual_norm_bwd, norm_weights, combine_weighted,
 * combine_weighted_bwd, adamw.
 */
int moe_timing_enable(int on);
int moe_timing_reset(void);
int moe_timing_query(const char *name, double *total_ms, int64_t *launches);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
