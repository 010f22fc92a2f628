/*
 * moe.h -- C ABI of the routed Mixture-of-Experts feed-forward layer for AMD Instinct MI355X
 * (gfx950).  Four calls make one layer: moe_route -> moe_bucket -> moe_expert_ffn -> moe_combine.  In front of it
 * stand moe_linear, moe_add_rms_norm and moe_route_grouped, and the attention: moe_rope_cache -> moe_attention_prompt or
 * moe_attention_decode.
 *
 * Sources (cited by page title and section; the pages print no code):
 *  [NV]  same post and section: NVFP4 also stores E2M1 values, with an E4M3 scale per 16 values
 *        and a second, tensor-wide scale.
 *  [MX]  "DeepSeek-V4-Flash on a four-GPU Ampere workstation" (FreeToken blog post), section
 *        "MXFP4 is not NVFP4, and the difference matters on Ampere": packed E2M1 codes with one
 *        unsigned E8M0 scale per 32 values, decoded weight v(c) * 2^(e-127), 4.25 bits/weight,
 *        decode inside the reduction with FP32 accumulation, row-major banks read with no repack.
 *  [BP]  same post, section "Why it would not run": a partition that cuts an FP4 32-value block
 *        is rejected instead of producing garbage; weights and scale grids are sliced together.
 *  [C31] "Cascadia: Resident 975B MoE Inference on Eleven AI PCs", Sec. 3.1: expert weights are
 *        stored expert by expert; each selected expert is a SwiGLU block (two input projections,
 *        the gated activation, one output projection) whose outputs are summed with the routing
 *        coefficients; the router hands the expert path ids plus coefficients, and shared experts
 *        are selections every row carries after its routed ones.
 *  [C32] Cascadia Sec. 3.2: a layer call supplies rows, expert ids and routing weights; the
 *        expert path returns FP32 output (Fig. 2).
 *  [C33] Cascadia Sec. 3.3, Eq. 1: range management across the FP16/FP32 boundary -- a per-layer
 *        power-of-two attenuation of the up projection and a per-row power-of-two factor on the
 *        routing weights, both undone in FP32.
 *  [C34] Cascadia Sec. 3.4, Eq. 2: a dense FFN is the sum of its all-active, unit-weight slices,
 *        cut at quantisation-group boundaries.
 *
 * Conventions for every call:
 *  - Pointers are DEVICE pointers of the current HIP device unless a comment says "host".
 *    The caller owns and allocates every buffer; the library never allocates, frees or keeps
 *    device memory, and keeps no state between calls.
 *  - Calls only validate arguments on the host and enqueue work on `stream` (a hipStream_t, or
 *    NULL for the default stream); they never synchronise and never read device memory on the
 *    host.  Results are ready when the stream has reached that point.
 *  - Validation happens before anything is enqueued; on any error nothing is launched and the
 *    status says why.  T == 0 returns MOE_OK without touching any pointer.
 *  - Inputs are read-only; outputs are overwritten (never accumulated into); buffers must not
 *    alias each other (but moe_add_rms_norm's residual_out may be its residual, moe_rope_cache's outputs its
 *    inputs).  Calls that share no output buffer and no workspace may run concurrently on different streams.
 *  - Results are deterministic: the same inputs give bit-identical outputs on every run (no
 *    floating-point atomics anywhere).
 */
#ifndef MOE_H
#define MOE_H
#include <stddef.h>
#include <stdint.h>
#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 2
#define MOE_MAX_EXPERTS 1024  /* routed experts E, and buckets / experts E' of the later calls */
#define MOE_MAX_SLOTS_PER_TOKEN 256  /* top_k + n_shared */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,      /* a required pointer is NULL */
  MOE_ERR_SHAPE = 2,     /* a size is negative, zero where it must not be, or beyond a limit */
  MOE_ERR_BLOCK = 3,     /* an MXFP4 dimension, slice base or stride cuts a 32-value block [BP] */
  MOE_ERR_ALIGN = 4,     /* a pointer or byte stride is not aligned (activations, outputs, FP16) */
  MOE_ERR_DTYPE = 5,     /* an unknown enum value, or an activation dtype the format cannot take */
  MOE_ERR_TOPK = 6,      /* top_k < 1 or top_k > E */
  MOE_ERR_WORKSPACE = 7, /* workspace NULL or smaller than the size query returns */
  MOE_ERR_HIP = 8        /* a kernel launch failed (the HIP error is lost; nothing else ran) */
} moe_status;

typedef enum { MOE_ACT_BF16 = 0, MOE_ACT_FP16 = 1 } moe_act_dtype;
/* Storage types of moe_add_rms_norm, moe_select_experts, moe_linear and the attention (the first two as above). */
typedef enum { MOE_DT_BF16 = 0, MOE_DT_FP16 = 1, MOE_DT_FP32 = 2 } moe_dtype;
typedef enum { MOE_W_MXFP4 = 0, MOE_W_FP16 = 1, MOE_W_INT4_G32 = 2, MOE_W_NVFP4 = 3 } moe_w_format;

/* One projection of every expert: logical [n_experts][N][K], K contiguous within a row [MX].
 *  MXFP4: `w` holds two E2M1 codes per byte, element k of a row in byte k/2 with even k in the
 *         low nibble (bits 3..0) and odd k in the high nibble; bit 3 of a code is its sign.
 *         `scales` holds one E8M0 byte per 32 elements: scale of element k at byte k/32 of the
 *         row.  Decoded weight = v(code) * 2^(scale - 127) [MX].  Scale codes 0..252 are
 *         supported (every decoded value is then finite in fp32 and bf16); at 253 and 254 the
 *         largest magnitudes overflow bf16, and 255 is outside the contract.
 *  FP16:  `w` holds IEEE binary16 values; `scales` must be NULL.
 *  INT4_G32 [C31] (Cascadia Sec. 3.1 and 3.5): `w` holds unsigned 4-bit codes packed as for
 *         MXFP4; group g = k/32 of a row has a binary16 scale (little-endian bytes 2g, 2g+1 of the
 *         scale row) and an unsigned 4-bit zero point (zero row byte g/2, even g in the low
 *         nibble); decoded weight = (code - zero) * scale (4.625 bits per weight).
 *  NVFP4 [NV] (FreeToken post, "MXFP4 is not NVFP4"): `w` holds E2M1 codes packed as for MXFP4;
 *         block b = k/16 has an E4M3 scale byte (byte b of the scale row; the two NaN codes are
 *         outside the contract) and every expert one fp32 tensor scale; decoded weight =
 *         v(code) * e4m3(scale) * tensor_scale[e] (4.5 bits per weight plus the tensor scale).
 *  INT4_G32 and NVFP4 run on the K-split kernels with bf16 activations; their weights are exact
 *  MFMA operands (INT4 as a bf16 high + low pair, NVFP4 in one bf16), the NVFP4 tensor scale
 *  multiplies the fp32 sums.
 *  Strides are in bytes between consecutive experts / rows, so a projection may be a slice of a
 *  larger matrix [C34] -- e.g. columns [j*I, (j+1)*I) of a dense [H][8*I] down projection have
 *  w = base + j*I*(bytes per element), w_expert_stride = I*(bytes per element),
 *  w_row_stride = 8*I*(bytes per element).  w, w_expert_stride and w_row_stride must be
 *  multiples of 16 bytes: for MXFP4 that is exactly one 32-code block, so a base or stride off
 *  that grid would start inside a block and is refused with MOE_ERR_BLOCK [BP]; for FP16 it is
 *  the 128-bit load alignment (MOE_ERR_ALIGN).  Scale pointers and strides have no alignment rule. */
typedef struct {
  const void *w;
  const uint8_t *scales;
  int64_t w_expert_stride, w_row_stride;
  int64_t s_expert_stride, s_row_stride;
  const uint8_t *zeros;        /* INT4_G32 zero points (NULL for the other formats) */
  int64_t z_expert_stride, z_row_stride;
  const float *tensor_scale;   /* NVFP4: [n_experts] fp32 (NULL for the other formats) */
} moe_proj;

/* All expert weights of a layer [C31].  gate and up: N = inter, K = hidden; down: N = hidden,
 * K = inter.  n_experts = E' = routed + shared experts (one bucket each).  hidden and inter must
 * be positive multiples of 32.  The struct itself is a HOST struct holding device pointers. */
typedef struct {
  moe_w_format fmt;
  int n_experts;
  int hidden;
  int inter;
  moe_proj gate, up, down;
} moe_expert_weights;

/* ---------------------------------------------------------------------------------------------
 * moe_route -- router logits, softmax, top-k, renormalised weights, shared slots.
 *
 * Per token t (reading of [C31]; the pages print no softmax router, the order below is the
 * method's statement): L[t,e] = sum_h x[t,h] * w_router[e,h] + logit_bias[e] (fp32 accumulation),
 * p = softmax(L[t,:]); the top_k experts by (L descending, index ascending) -- i.e. by p with the
 * lowest index winning exact ties -- fill slots j = 0..top_k-1 in that order with
 * weights[t,j] = p_j / sum_{j'<top_k} p_j'; slots top_k .. top_k+n_shared-1 get the shared
 * experts E .. E+n_shared-1 with weight 1.0.
 *   x          [T][H] bf16 or fp16 (x_dtype), rows contiguous, 16-byte aligned
 *   w_router   [E][H] fp32 (4-byte aligned, like every int32/fp32 array below)
 *   logit_bias [E] fp32 added to the logits before the softmax, or NULL
 *   ids        [T][top_k+n_shared] int32 out;  weights [T][top_k+n_shared] fp32 out
 *   probs      [T][E] fp32 out (the full softmax), or NULL
 *   workspace  moe_route_workspace_bytes(T, H, E) bytes, 16-byte aligned (NULL if that is 0)
 * Errors: NULL, SHAPE (T<0, H<1, E<1, E>MOE_MAX_EXPERTS, n_shared<0), TOPK (also
 * top_k+n_shared > MOE_MAX_SLOTS_PER_TOKEN), DTYPE, ALIGN, WORKSPACE, HIP. */
size_t moe_route_workspace_bytes(int T, int H, int E);
moe_status moe_route(const void *x, moe_act_dtype x_dtype, int T, int H, const float *w_router,
                     const float *logit_bias, int E, int top_k, int n_shared, int32_t *ids,
                     float *weights, float *probs, void *workspace, size_t workspace_bytes,
                     void *stream);

/* moe_route_sigmoid -- the sigmoid router of [C31] (Cascadia Sec. 3.1: sigmoid scores, a
 * bias-adjusted top-k selection, normalisation of the selected weights and a model scale factor;
 * the page names these steps without formulas, and the plainest forms are taken):
 *   L[t,e] = sum_h x[t,h] * w_router[e,h] (fp32 accumulation), s[t,e] = 1 / (1 + e^-L[t,e]);
 *   the top_k experts by (s[t,e] + selection_bias[e] descending, index ascending) fill slots
 *   j = 0..top_k-1 in that order with weights[t,j] = routed_scale * s_j / sum_{j'<top_k} s_j'
 *   (the bias moves the selection only, never a weight); slots top_k .. top_k+n_shared-1 hold
 *   the shared experts E .. E+n_shared-1 with weight shared_weight (Cascadia's rows carry six
 *   routed and two shared selections, ids 256 and 257).
 *   scores [T][E] fp32 out (the sigmoid scores s), or NULL; other arguments as for moe_route,
 *   with the same workspace size.
 * Errors: as moe_route, and SHAPE for a non-finite routed_scale or shared_weight. */
moe_status moe_route_sigmoid(const void *x, moe_act_dtype x_dtype, int T, int H, const float *w_router,
                             const float *selection_bias, int E, int top_k, int n_shared,
                             float routed_scale, float shared_weight, int32_t *ids, float *weights,
                             float *scores, void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Routing by a rule: scores, a balance bias, groups of experts, top-k (group-limited routing; not on
 * the pages).  Per token with logits L[e], e < E, and b = selection_bias (0 without one):
 *   scores    s[e] = 1 / (1 + e^-L[e]) (SIGMOID), or softmax(L) over the experts with finite L (SOFTMAX);
 *   keys      s[e] + b[e]: the bias moves the choice only, never a weight;
 *   available an expert with a finite logit and a finite bias.  A logit of -inf masks an expert for a
 *             token, a bias of -inf for all tokens (NaN and +inf mask too);
 *   groups    group g holds experts g * E/n_groups .. (g+1) * E/n_groups - 1.  Its rank is the sum of its
 *             two largest available keys (TOP2; the one key where it has only one) or the largest (MAX).
 *             The topk_groups groups of the largest ranks stay, the lowest index first on ties;
 *   slots     j = 0 .. top_k-1 hold the available experts of those groups by (key descending, index
 *             ascending), weights[t,j] = routed_scale * s_j, divided by the sum of the selected s if
 *             renormalise.  Where fewer than top_k are left, the other slots get id -1 and weight 0 (as
 *             moe_pad_rows marks them: moe_bucket drops them, moe_combine leaves them out).  A sum of scores that underflows fp32 gives
 *             weights of 0;
 *   shared    slots top_k .. top_k+n_shared-1 hold experts E .. E+n_shared-1 with weight shared_weight.
 * The choice is that of the keys in 64 bits, also where two keys or ranks are closer than fp32 can
 * tell.  Without a bias the logits stand for the keys (in a group's MAX rank too): the scores rise with
 * them, also where 64 bits cannot tell the scores apart (SIGMOID of logits beyond 37, SOFTMAX 745 below
 * the largest).  With a bias, a bias of zeros among them, such keys tie and the lowest index comes
 * first; so do TOP2 ranks, which are sums of scores.  The choice is a function of the logits; ids of
 * moe_route_grouped also depend on the logits' own fp32 rounding, as moe_route's do.
 * The struct is a HOST struct; selection_bias is a device pointer to [E] fp32, or NULL. */
#define MOE_MAX_GROUPS 64
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef enum { MOE_GROUP_TOP2 = 0, MOE_GROUP_MAX = 1 } moe_group_score;
typedef struct {
  moe_score score;
  int top_k, n_shared;
  int n_groups, topk_groups;   /* 1 and 1: no groups */
  moe_group_score group_score;
  int renormalise;
  float routed_scale, shared_weight;
  const float *selection_bias;
} moe_route_rule;

/* moe_select_experts -- the rule on given logits.
 *   logits  [T] rows of E values (bf16, fp16 or fp32), row_stride values apart (>= E), aligned to a value
 *   ids     [T][top_k+n_shared] int32 out;  weights [T][top_k+n_shared] fp32 out
 *   scores  [T][E] fp32 out (s; 0 for an expert whose logit is not finite), or NULL
 * One launch, no workspace.
 * Errors: NULL, SHAPE (T<0, T>2^25, E<1, E>MOE_MAX_EXPERTS, n_shared<0, row_stride<E, n_groups outside
 * [1, MOE_MAX_GROUPS] or not a divisor of E, topk_groups outside [1, n_groups], a routed_scale or
 * shared_weight that is not finite), TOPK (top_k < 1 or beyond topk_groups * E/n_groups, or
 * top_k+n_shared > MOE_MAX_SLOTS_PER_TOKEN), DTYPE, ALIGN, HIP. */
moe_status moe_select_experts(const void *logits, moe_dtype logits_dtype, int64_t row_stride, int T, int E,
                              const moe_route_rule *rule, int32_t *ids, float *weights, float *scores,
                              void *stream);
/* moe_route_grouped -- the rule on L = x w_router^T (fp32, as moe_route computes it).  x, w_router, workspace
 * (moe_route_workspace_bytes(T, H, E) bytes) as for moe_route, the rest as above.
 * Errors: as both calls. */
moe_status moe_route_grouped(const void *x, moe_act_dtype x_dtype, int T, int H, const float *w_router, int E,
                             const moe_route_rule *rule, int32_t *ids, float *weights, float *scores,
                             void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Fixed row shapes [C32] (Cascadia Sec. 3.2: a call's rows are run at one of the row shapes the
 * compiled layer supports, the extra rows padded with zero routing weights, and only the real
 * rows are handed back).  Here a row shape is a T for which the caller has buffers (and, say, a
 * captured HIP graph of the layer's calls); the real row count n lives in device memory, so one
 * graph serves every n up to its shape:
 *   moe_route(..., T_shape, ...) -> moe_pad_rows(n_rows, T_shape, ...) -> moe_bucket ->
 *   moe_expert_ffn -> moe_combine, then read rows [0, n) of y.
 *
 * moe_row_shape (host): the smallest entry of shapes[0 .. n_shapes) that is >= T (entries <= 0
 * are ignored; the array need not be sorted); -1 when none is, or for T < 0, shapes NULL or
 * n_shapes < 1. */
int moe_row_shape(int T, const int *shapes, int n_shapes);
/* moe_pad_rows: with n = *n_rows (a device int32, clamped to [0, T_shape]), every slot of rows
 * t >= n gets weights[t,j] = 0 and ids[t,j] = -1 -- the invalid id makes moe_bucket drop it, so no
 * expert runs on padding.  Rows < n are untouched.  Padding changes no real row's result: every
 * kernel computes each token from its own x row and weights only (the rows past n of y_slots and
 * y are left unspecified).  ids, weights [T_shape][k_total] in/out.
 * Errors: NULL, SHAPE (T_shape < 0, k_total outside [1, MOE_MAX_SLOTS_PER_TOKEN]), ALIGN, HIP. */
moe_status moe_pad_rows(const int32_t *n_rows, int T_shape, int k_total, int32_t *ids, float *weights,
                        void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_route_bucket -- moe_route, then moe_bucket of its ids over n_buckets = E + n_shared, then
 * (W non-NULL) moe_expert_ffn_plan into ffn_workspace, with the same results bit for bit: for
 * T <= 8 in two launches instead of four (one workgroup selects, buckets and writes the tile
 * table), up to 2048 slots in three (the bucketing workgroup also writes the tile table), beyond
 * that as the separate kernels.  Arguments as for those calls; W->n_experts must
 * equal E + n_shared; ffn_workspace then is the workspace that the following
 * moe_expert_ffn_gateup / moe_expert_ffn_down calls use.  workspace:
 * moe_route_bucket_workspace_bytes(T, H, E, top_k, n_shared) bytes, 16-byte aligned (it holds
 * the router's partial sums and the bucketing's scratch).
 * Errors: as for the three calls. */
size_t moe_route_bucket_workspace_bytes(int T, int H, int E, int top_k, int n_shared);
moe_status moe_route_bucket(const void *x, moe_act_dtype x_dtype, int T, int H, const float *w_router,
                            const float *logit_bias, int E, int top_k, int n_shared, int32_t *ids,
                            float *weights, float *probs, int32_t *counts, int32_t *offsets,
                            int32_t *sorted_slot, int32_t *slot_pos, const moe_expert_weights *W,
                            void *ffn_workspace, size_t ffn_workspace_bytes, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_bucket -- group slots by expert (the fused path runs only the selected experts' work
 * [C31]).  Slot s = t*k_total + j.
 *   counts[b]      number of slots with ids[s] == b                         ([n_buckets])
 *   offsets[b]     exclusive prefix sum of counts; offsets[n_buckets] = number of valid slots
 *   sorted_slot[r] slot indices bucket by bucket, ascending slot index within a bucket (stable)
 *   slot_pos[s]    inverse permutation: sorted_slot[slot_pos[s]] == s           (or NULL)
 * A slot whose id is outside [0, n_buckets) is dropped: slot_pos = -1 and it is not counted;
 * entries of sorted_slot past offsets[n_buckets] are -1.  (Ids live on the device, so this is
 * the only possible check; the expert FFN then leaves that slot's y_slots row unwritten.)
 *   workspace  moe_bucket_workspace_bytes(n_slots, n_buckets) bytes (NULL if that is 0)
 * Errors: NULL, SHAPE (n_slots<0, n_buckets<1 or >MOE_MAX_EXPERTS), ALIGN, WORKSPACE, HIP. */
size_t moe_bucket_workspace_bytes(int n_slots, int n_buckets);
moe_status moe_bucket(const int32_t *ids, int n_slots, int n_buckets, int32_t *counts,
                      int32_t *offsets, int32_t *sorted_slot, int32_t *slot_pos, void *workspace,
                      size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_expert_ffn -- grouped SwiGLU experts over the buckets [C31], decode inside the reduction
 * with FP32 accumulation [MX].
 * For every expert e and sorted row r in [offsets[e], offsets[e+1]) with slot s = sorted_slot[r]
 * and token t = s / k_total:
 *   g = W_gate[e] x_t,  u = W_up[e] x_t  (fp32 accumulation of exact products),
 *   h = SiLU(g) * u     (fp32; fed to the down projection as a high + low pair: bf16 for MXFP4
 *                        weights, about 16 significant bits over the whole fp32 range; binary16
 *                        for FP16 weights, which holds only |h| <= 65504 -- larger h overflows
 *                        to infinity, see moe_expert_ffn_f16 [C33] -- and keeps about 22 bits
 *                        for |h| >= 2^-3, below which the low part is subnormal and the pair's
 *                        error stays under 2^-25 absolute),
 *   y_slots[s,:] = W_down[e] h   (fp32).
 *   x        [T][hidden] activations; MXFP4 weights need MOE_ACT_BF16, FP16 weights MOE_ACT_FP16
 *   W        host pointer to the weight description (device pointers inside)
 *   offsets  [W->n_experts + 1], sorted_slot [T*k_total] as written by moe_bucket
 *   y_slots  [T*k_total][hidden] fp32 out; rows of dropped slots are left unwritten
 *   workspace moe_expert_ffn_workspace_bytes(T, k_total, W) bytes, 16-byte aligned
 * Sorted rows whose slot lies outside [0, T*k_total) are skipped, so corrupt device-side indices
 * cannot cause out-of-bounds accesses.
 * Errors: NULL, SHAPE, BLOCK (MXFP4 hidden or inter not a multiple of 32, or a weight base or
 * stride that cuts a 32-value block), ALIGN, DTYPE, WORKSPACE, HIP. */
size_t moe_expert_ffn_workspace_bytes(int T, int k_total, const moe_expert_weights *W);
moe_status moe_expert_ffn(const void *x, moe_act_dtype x_dtype, int T, int k_total,
                          const moe_expert_weights *W, const int32_t *offsets,
                          const int32_t *sorted_slot, float *y_slots, void *workspace,
                          size_t workspace_bytes, void *stream);

/* moe_expert_ffn_static -- moe_expert_ffn for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc): the same kernels
 * and the same results, bit for bit, with the workspace taken from a fixed array of
 * MOE_FFN_STATIC_SCRATCH_BYTES bytes inside the library's device code (one per GPU, held until the
 * process ends) instead of a caller buffer.  The call allocates nothing.  Limit: calls whose
 * moe_expert_ffn_workspace_bytes(T, k_total, W) exceeds MOE_FFN_STATIC_SCRATCH_BYTES are refused
 * with MOE_ERR_WORKSPACE (with inter 2048 and top-8 that is T = 256 and above).  Every call on
 * a GPU shares that GPU's array: calls that overlap in time on one GPU (different streams, or
 * several host threads) race and give wrong results; calls ordered on one stream are safe.
 * Arguments and other errors as for moe_expert_ffn; HIP also when the array's device address
 * cannot be looked up. */
#define MOE_FFN_STATIC_SCRATCH_BYTES ((size_t)16 << 20)
moe_status moe_expert_ffn_static(const void *x, moe_act_dtype x_dtype, int T, int k_total,
                                 const moe_expert_weights *W, const int32_t *offsets,
                                 const int32_t *sorted_slot, float *y_slots, void *stream);

/* The three steps of moe_expert_ffn as separate calls, for callers that time or overlap them.
 * moe_expert_ffn_plan writes the tile schedule (which expert and sorted rows each 16-row tile
 * covers, from offsets) into the workspace; moe_expert_ffn_gateup computes
 * h = SiLU(W_gate x) * (W_up x) for every sorted row into the workspace; moe_expert_ffn_down
 * turns the workspace's h into y_slots.  Both phases read the schedule, so the plan must run first
 * on the same workspace with the same T, k_total, W->n_experts and offsets contents; a schedule
 * left from other arguments gives wrong rows, but the kernels check every schedule entry against
 * the call's bounds and never access memory outside the buffers described.  Calling plan, gateup
 * and down on one stream with the same arguments gives exactly moe_expert_ffn's result (it
 * launches the same kernels).  x_dtype of the plan and down calls only selects the format check
 * (it must match W->fmt as in moe_expert_ffn); the plan reads only W's sizes.  Errors as for
 * moe_expert_ffn. */
moe_status moe_expert_ffn_plan(moe_act_dtype x_dtype, int T, int k_total,
                               const moe_expert_weights *W, const int32_t *offsets, void *workspace,
                               size_t workspace_bytes, void *stream);
moe_status moe_expert_ffn_gateup(const void *x, moe_act_dtype x_dtype, int T, int k_total,
                                 const moe_expert_weights *W, const int32_t *offsets,
                                 const int32_t *sorted_slot, void *workspace,
                                 size_t workspace_bytes, void *stream);
moe_status moe_expert_ffn_down(moe_act_dtype x_dtype, int T, int k_total,
                               const moe_expert_weights *W, const int32_t *offsets,
                               const int32_t *sorted_slot, float *y_slots, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Range-managed FP16 path [C33] (Cascadia Sec. 3.3, Eq. 1).  For a layer with attenuation
 * A = 2^attenuation_log2 applied to its up projection, the expert path works on E(x) / A and
 * crosses the FP16 boundary in binary16; every row i is combined with its weights divided by
 * F_i = 2^ceil(log2 max(1, sum_j |w_ij|)) and restored as y_i = A F_i y~_i in FP32.  In real
 * arithmetic the result is the plain layer's; the attenuation keeps h, the expert outputs and
 * the combination inside the binary16 range (the configuration recorded for layer 8 uses A = 16),
 * and the factors, being powers of two, are applied and removed exactly.
 *
 * moe_expert_ffn_f16: for every sorted row as in moe_expert_ffn,
 *   u~ = (W_up[e] x_t) / A,  h~ = binary16(SiLU(W_gate[e] x_t) * u~)   (fp32, then rounded),
 *   y_slots[s,:] = binary16(W_down[e] h~)                              (fp32 accumulation)
 * i.e. binary16 expert outputs E(x) / A (IEEE half bits; values past 65504 become infinite, which
 * is what the attenuation is for).  Weights MXFP4 (bf16 x) or FP16 (fp16 x), as for
 * moe_expert_ffn; runs the K-split kernels.  y_slots [T*k_total][hidden] binary16, 2-byte aligned;
 * dropped slots' rows are left unwritten.  workspace: moe_expert_ffn_f16_workspace_bytes bytes,
 * 16-byte aligned.  Errors as for moe_expert_ffn, plus SHAPE for attenuation_log2 outside
 * [0, MOE_MAX_ATTENUATION_LOG2]. */
#define MOE_MAX_ATTENUATION_LOG2 30
size_t moe_expert_ffn_f16_workspace_bytes(int T, int k_total, const moe_expert_weights *W);
moe_status moe_expert_ffn_f16(const void *x, moe_act_dtype x_dtype, int T, int k_total,
                              const moe_expert_weights *W, int attenuation_log2,
                              const int32_t *offsets, const int32_t *sorted_slot, uint16_t *y_slots,
                              void *workspace, size_t workspace_bytes, void *stream);
/* moe_combine_restore: per token t with F_t = 2^ceil(log2 max(1, sum_j |weights[t,j]|)) (fp32 sum
 * in ascending j),
 *   y~[t,:] = binary16(sum_{j ascending} (weights[t,j] / F_t) * y_slots[t*k_total+j,:])  (fp32 sum)
 *   y[t,:]  = A * F_t * y~[t,:]                                                      (fp32, exact)
 * A slot of weight 0 adds nothing, whatever its row holds.
 * y_slots [T*k_total][H] binary16 (8-byte aligned), weights [T][k_total] fp32, y [T][H] fp32 out
 * (16-byte aligned), H % 4 == 0.  Errors: NULL, SHAPE (also attenuation_log2 out of range), ALIGN,
 * HIP. */
moe_status moe_combine_restore(const uint16_t *y_slots, const float *weights, int T, int k_total, int H,
                               int attenuation_log2, float *y, void *stream);

/* ---------------------------------------------------------------------------------------------
 * MX mode (prefill).  Not on the pages, which define only the MXFP4 weight block [MX]: the
 * activations are quantised to an OCP Microscaling element format, one E8M0 scale per 32
 * consecutive values along K, so that the expert FFN can run the FP4 weights on the matrix
 * cores' scaled FP4 x FP8/FP6/FP4 instructions.  The result is NOT the exact layer: it differs
 * from moe_expert_ffn by the quantisation of x and h (use moe_expert_ffn for exact results).
 *
 * Element formats (sign | exponent | fraction, subnormals at exponent field 0):
 *   MOE_MX_FP8_E4M3  8-bit, bias 7, largest 448 (S.1111.111 is NaN and never produced)
 *   MOE_MX_FP4_E2M1  4-bit, bias 1, largest 6 (the weights' E2M1 codes)
 *   MOE_MX_FP6_E2M3  6-bit, bias 1, largest 7.5
 * Quantisation of a block of 32 values v_i with amax = max |v_i|: scale code
 * c = clamp(floor(log2 amax) - emax + 127, 0, 254) (emax = 8, 2, 2; c = 0 for an all-zero block),
 * X = 2^(c - 127), and code_i = the element value nearest to v_i / X, ties to the even code,
 * saturating at the largest value, with the sign of v_i (so -0 and tiny negative values give the
 * negative-zero code).
 * Packed codes: a block takes 4 * bits bytes -- FP8 one code per byte; FP4 two per byte, element
 * 2j in the low nibble of byte j; FP6 element j in bits 6j .. 6j+5 of the block's little-endian
 * 192-bit string.  A row of K values is K/32 consecutive blocks, rows are consecutive. */
typedef enum { MOE_MX_FP8_E4M3 = 1, MOE_MX_FP4_E2M1 = 2, MOE_MX_FP6_E2M3 = 3 } moe_mx_format;

/* Bytes of one packed row of K values (K/32 * 4 * bits); 0 for an unknown format or K % 32 != 0. */
size_t moe_mx_row_bytes(moe_mx_format fmt, int K);

/* moe_mx_quantize -- the activation quantiser of the MX mode on its own:
 *   x [n_rows][K] bf16 or fp16 (contiguous, 16-byte aligned), codes [n_rows][row bytes] out
 *   (16-byte aligned), scales [n_rows][K/32] E8M0 out.
 * Errors: NULL, SHAPE (n_rows < 0, K < 1), BLOCK (K % 32), DTYPE (format or x dtype), ALIGN, HIP. */
moe_status moe_mx_quantize(const void *x, moe_act_dtype x_dtype, int n_rows, int K, moe_mx_format fmt,
                           uint8_t *codes, uint8_t *scales, void *stream);

/* moe_expert_ffn_mx -- moe_expert_ffn with MX activations: for every sorted row r of expert e
 * with slot s and token t = s / k_total,
 *   xq = dequant(quant(x[t,:])),  g = W_gate[e] xq,  u = W_up[e] xq  (fp32 accumulation),
 *   h = SiLU(g) * u (fp32),  hq = dequant(quant(h)),  y_slots[s,:] = W_down[e] hq  (fp32),
 * quant/dequant being the block quantisation above along hidden (x) and inter (h).  Weights must
 * be MXFP4 and x bf16.  hidden and inter must be multiples of 256; scale pointers and strides
 * multiples of 8 bytes.  Arguments otherwise as for moe_expert_ffn, with the workspace from
 * moe_expert_ffn_mx_workspace_bytes (it holds the x and h codes and the tile table).
 * Errors: NULL, SHAPE (also hidden or inter not a multiple of 256, or buffers past 2^31 bytes),
 * BLOCK, ALIGN, DTYPE (weights not MXFP4, x not bf16, unknown format), WORKSPACE, HIP. */
size_t moe_expert_ffn_mx_workspace_bytes(int T, int k_total, const moe_expert_weights *W,
                                         moe_mx_format fmt);
moe_status moe_expert_ffn_mx(const void *x, moe_act_dtype x_dtype, int T, int k_total,
                             const moe_expert_weights *W, moe_mx_format fmt, const int32_t *offsets,
                             const int32_t *sorted_slot, float *y_slots, void *workspace,
                             size_t workspace_bytes, void *stream);
/* Where moe_expert_ffn_mx leaves its quantised activations in the workspace, for inspection:
 * offsets[0] x codes ([T] packed rows of `hidden` values), offsets[1] x scales ([T][hidden/32]),
 * offsets[2] h codes ([T*k_total] packed rows of `inter` values, row r belonging to sorted row r,
 * i.e. slot sorted_slot[r]; rows of empty slots are unspecified), offsets[3] h scales
 * ([T*k_total][inter/32]).  offsets is a host array of 4.  Errors: NULL, SHAPE, DTYPE. */
moe_status moe_expert_ffn_mx_workspace_layout(int T, int k_total, const moe_expert_weights *W,
                                              moe_mx_format fmt, size_t *offsets);

/* moe_expert_ffn_mx_codes -- moe_expert_ffn_mx on an x that is quantised already (by moe_mx_quantize, or by
 * moe_add_rms_norm): x_codes [T] packed rows of `hidden` values (16-byte aligned), x_scales [T][hidden/32]
 * E8M0 (4-byte aligned).  The same results, bit for bit, as moe_expert_ffn_mx on the x they came from, without
 * its quantisation launch.  workspace: moe_expert_ffn_mx_workspace_bytes (its x part stays unused).
 * Errors: as moe_expert_ffn_mx. */
moe_status moe_expert_ffn_mx_codes(const uint8_t *x_codes, const uint8_t *x_scales, int T, int k_total,
                                   const moe_expert_weights *W, moe_mx_format fmt, const int32_t *offsets,
                                   const int32_t *sorted_slot, float *y_slots, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_add_rms_norm -- the residual addition and root-mean-square norm in front of a layer (not on the pages).
 * Per row t, in fp32 with one rounding at each output:
 *   s = x[t,:] + residual[t,:]   (s = x[t,:] without a residual)
 *   residual_out[t,:] = s
 *   y[t,h] = s[h] * weight[h] / sqrt(sum_h s[h]^2 / hidden + eps)
 *   codes[t], scales[t] = the MX block quantisation (see MX mode) of the fp32 y before it is rounded to y_dtype;
 *   fmt MOE_MX_FP8_E4M3 is the 8-bit output, in the layout of moe_expert_ffn_mx_codes.  y must be finite there (the
 *   codes hold no NaN: one becomes a finite value).
 * A NaN in s makes its row's y NaN, an infinity NaN where it stands and 0 elsewhere, as does a sum of squares past
 * fp32 (0 everywhere); other rows are untouched.
 * Types: x, residual (and residual_out), weight and y each bf16, fp16 or fp32.  x may be moe_combine's or
 * moe_linear's fp32 output, y is what moe_route, moe_linear and moe_expert_ffn read.
 *   x, residual, residual_out  [T] rows of `hidden` values, *_row_stride values apart (>= hidden), aligned to a
 *       value.  residual may be NULL (then residual_out must be too); residual_out may be NULL, and may be
 *       residual itself (same pointer and stride: the sum replaces it in place; another stride there is a SHAPE
 *       error, any other overlap an error that is not checked)
 *   y       [T][hidden], aligned to a value, or NULL
 *   codes   [T] packed rows (moe_mx_row_bytes), 16-byte aligned; scales [T][hidden/32]; fmt 0: both NULL
 * Rows of 8 to 32768 values take the fast kernels.
 * Errors: NULL (also neither y nor codes wanted, residual_out without residual), SHAPE (T<0, hidden<1, a stride
 * below hidden, eps negative or not finite), BLOCK (codes with hidden % 32), DTYPE, ALIGN, HIP. */
typedef struct {
  const void *weight;  /* [hidden], aligned to a value */
  moe_dtype weight_dtype;
  int hidden;
  float eps;
} moe_norm;
moe_status moe_add_rms_norm(const moe_norm *norm, const void *x, moe_dtype x_dtype, int64_t x_row_stride,
                            const void *residual, moe_dtype residual_dtype, int64_t residual_row_stride, int T,
                            void *residual_out, int64_t residual_out_row_stride, void *y, moe_dtype y_dtype,
                            int fmt, uint8_t *codes, uint8_t *scales, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_linear -- a product with 4-bit weights (an attention projection, a dense FFN's matrix, an output head):
 *   y[t,n] = sum_k x[t,k] * W[n,k] + bias[n]   (exact decoded weights and products, fp32 sums, one rounding)
 * W: one matrix [n_out][k_in] in MXFP4, INT4_G32 or NVFP4 (moe_proj; its expert strides are not used, an NVFP4
 * tensor_scale is one value).  k_in a positive multiple of 32, n_out any.  x bf16, as for every 4-bit format.
 *   x    [T] rows of k_in values, x_row_stride values apart (>= k_in, a multiple of 8), 16-byte aligned
 *   bias [n_out] fp32, or NULL
 *   y    [T] rows of n_out values (bf16, fp16 or fp32), y_row_stride values apart (>= n_out), aligned to a value
 *   workspace moe_linear_workspace_bytes(T, W) bytes, 16-byte aligned (NULL if that is 0)
 * Up to four tokens sum a block's products before its scale is applied, which stays inside fp32 while |x| <
 * 2^119.  A NaN or infinity in x makes that token's outputs NaN or infinite and no other token's (INT4 weights may
 * make an infinity NaN: they multiply in two parts).
 * Errors: NULL, SHAPE (also a weight, scale or zero-point row stride of 2^24 bytes or more, an x row stride of
 * 2^23 values or more, T > 2^30, or n_out > 2^26), BLOCK, ALIGN, DTYPE (FP16 weights, x not bf16), WORKSPACE, HIP. */
typedef struct {
  moe_w_format fmt;
  int n_out, k_in;
  moe_proj w;
} moe_linear_weights;
size_t moe_linear_workspace_bytes(int T, const moe_linear_weights *W);
moe_status moe_linear(const void *x, moe_act_dtype x_dtype, int64_t x_row_stride, int T,
                      const moe_linear_weights *W, const float *bias, void *y, moe_dtype y_dtype,
                      int64_t y_row_stride, void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Attention: the other half of the block (not on the pages).  The projected q, k and v turn by their positions and go
 * into a paged cache (moe_rope_cache); a prompt attends over its own rows (moe_attention_prompt), a new token over the
 * cache (moe_attention_decode).  Query heads h = 0 .. n_q_heads-1 share key-value heads in groups of
 * G = n_q_heads / n_kv_heads: h reads key-value head h / G.
 *
 * moe_heads: [tokens][heads][head_dim] values; a head's values are contiguous, tokens and heads are token_stride and
 * head_stride values apart (both >= 0), so that q, k and v may be parts of one product's output, or 0 apart (broadcast).
 * Rows that are written share no memory: in order of their strides, each stride of more than one step is at least the
 * values that the smaller ones reach over, head_dim first (else MOE_ERR_SHAPE; so it is for a cache that is written and its
 * scales).  They lie over no input but where a call says so.  A HOST struct. */
#define MOE_MAX_HEADS 1024
#define MOE_MAX_HEAD_DIM 256   /* a multiple of 8 */
typedef struct {
  void *p;                     /* inputs are read only */
  moe_dtype dtype;
  int64_t token_stride, head_stride;
} moe_heads;

/* A key-value cache of n_pages pages of page_size tokens each: value d of token i of page p and key-value head h is
 * value p * page_stride + h * head_stride + i * token_stride + d of k or v (any order of the three; 64-bit offsets).
 * Formats: MOE_KV_BF16 and MOE_KV_FP16 hold the values; MOE_KV_MXFP8 holds MOE_MX_FP8_E4M3 codes (one byte each) with an
 * E8M0 scale byte per 32 values along head_dim at s_page_stride, s_head_stride, s_token_stride (scales NULL otherwise;
 * head_dim % 32 == 0, else MOE_ERR_BLOCK).  k, v: 16-byte aligned, strides multiples of 16 bytes.
 * n_pages * page_size < 2^31.  A HOST struct. */
typedef enum { MOE_KV_BF16 = 0, MOE_KV_FP16 = 1, MOE_KV_MXFP8 = 2 } moe_kv_format;
typedef struct {
  moe_kv_format fmt;
  int n_pages, page_size, n_kv_heads, head_dim;
  void *k, *v;
  int64_t page_stride, head_stride, token_stride;
  uint8_t *k_scales, *v_scales;
  int64_t s_page_stride, s_head_stride, s_token_stride;
} moe_kv_cache;

/* Angles of the positions: cos and sin [n_positions][rotary_dim / 2] fp32.  Of a head's first rotary_dim values (even,
 * at most head_dim) pair i is (i, i + rotary_dim/2) (HALVES) or (2i, 2i + 1) (NEIGHBOURS); the others stay. */
typedef enum { MOE_ROPE_HALVES = 0, MOE_ROPE_NEIGHBOURS = 1 } moe_rope_pairs;
typedef struct {
  const float *cos, *sin;
  int n_positions, rotary_dim;
  moe_rope_pairs pairs;
} moe_rope;

/* moe_rope_cache -- per token t, in fp32 with one rounding at each output: pairs (a, b) of q's and k's heads become
 * (a cos - b sin, b cos + a sin) at position positions[t]; q_out, k_out and v_out (bf16, fp16 or fp32) get the turned q
 * and k, and v; slot slots[t] = page * page_size + token of the cache gets the turned k, and v (MXFP8: codes of the fp32
 * values, which must be finite).
 *   rope, positions  [T] int32, or both NULL (nothing turns).  A token whose position is outside [0, n_positions) is
 *                    padding: none of its outputs is written
 *   q, k, v          bf16, fp16 or fp32, the same for all, aligned to a value.  n_q_heads or n_kv_heads may be 0 (then
 *                    those pointers are not used); v may be NULL where neither v_out nor cache is given
 *   q_out            may be q itself (same pointer, type and strides: it turns in place); so may k_out and v_out
 *   k_out, v_out     or NULL
 *   cache, slots     [T] int32, or both NULL.  A slot outside the cache is not written.  Slots that two tokens of a call
 *                    share hold a mixture of both
 * Errors: NULL (also key-value heads without any output), SHAPE (T<0, T * (n_q_heads + 2 n_kv_heads) > 2^27, heads,
 * head_dim, strides, rotary_dim, a cache of other heads, in place with other strides), BLOCK, DTYPE, ALIGN, HIP. */
moe_status moe_rope_cache(const moe_rope *rope, const int32_t *positions, int T, int n_q_heads, int n_kv_heads,
                          int head_dim, const moe_heads *q, const moe_heads *k, const moe_heads *v,
                          const moe_heads *q_out, const moe_heads *k_out, const moe_heads *v_out,
                          const moe_kv_cache *cache, const int32_t *slots, void *stream);

/* moe_attention_prompt -- n_seqs sequences packed one after another: sequence b has queries cu_q[b] .. cu_q[b+1]-1 and
 * keys cu_k[b] .. cu_k[b+1]-1 (device int32 [n_seqs+1], ascending; clamped to [0, Tq] and [0, Tk]).  With nq queries and
 * nk keys, query i stands at key position p = i + nk - nq and sees keys j with j <= p (causal) and j > p - window
 * (window > 0; causal only):
 *   y[i,h] = sum_j softmax_j(scale * q[i,h] . k[j,h/G]) v[j,h/G],  lse[i,h] = ln sum_j exp(scale * q[i,h] . k[j,h/G])
 * (fp32 sums; the exponentials are rounded to the 16-bit type before their product with v, not in their sum, which moves y by
 * up to half a step of the mean magnitude of v; one rounding of y).  In fp16 a weight below 2^-14 of the largest of its 64 keys
 * is off by up to 2^-25 of that one (among the keys of the row's largest: below 2^-21, by up to 2^-32).  A row that sees no
 * key, or only keys of score -inf, gets y = 0 and lse = -inf.  A NaN or infinity in a key or value reaches the rows that see
 * it and no other.  Rows of y outside the sequences are not touched.
 *   q, y  [Tq][n_q_heads][head_dim], k, v [Tk][n_kv_heads][head_dim]: one type, bf16 or fp16; 16-byte aligned, strides
 *         multiples of 8 values
 *   lse   [Tq][n_q_heads] fp32, or NULL
 *   workspace moe_attention_prompt_workspace_bytes(...) bytes, 16-byte aligned (NULL if that is 0)
 * Errors: NULL, SHAPE (Tq<0, Tk<0, n_seqs<0 or >2^20, heads, head_dim, Tq * n_q_heads from 2^31 on, Tq + Tk > 2^30, more than
 * 2^23 workgroups, a scale that is not positive and finite, window<0 or without causal), DTYPE, ALIGN, WORKSPACE, HIP. */
size_t moe_attention_prompt_workspace_bytes(int Tq, int Tk, int n_seqs, int n_q_heads, int n_kv_heads, int head_dim);
moe_status moe_attention_prompt(const moe_heads *q, const moe_heads *k, const moe_heads *v, const int32_t *cu_q,
                                const int32_t *cu_k, int n_seqs, int Tq, int Tk, int n_q_heads, int n_kv_heads,
                                int head_dim, float scale, int causal, int window, const moe_heads *y, float *lse,
                                void *workspace, size_t workspace_bytes, void *stream);

/* moe_attention_decode -- row b is the newest token of a sequence with n = lens[b] cached tokens (its own among them;
 * clamped to [0, max_len]), token j on page page_table[b][j / page_size] at j % page_size.  It sees the last `window` of
 * them, or all (window 0):
 *   y[b,h], lse[b,h] as for moe_attention_prompt (fp32 sums; the exponentials are two 16-bit parts, so an infinite
 *   value that is seen may give NaN; one rounding of y).  In fp16 the low part of a weight is off by up to 2^-25 of the
 *   largest weight of its 32 keys (2^-32 among the keys of the row's largest).  MXFP8 values are taken as bf16 ones: exact
 *   above 2^-126, multiples of 2^-133 below, infinities from 2^128 on.
 * No keys: y = 0, lse = -inf.  Tokens on a page number outside [0, n_pages) are left out.  Rows may share pages and table
 * rows (several newest tokens of one sequence: one row each, with rising lens).
 *   q, y        [B][n_q_heads][head_dim] bf16 (MOE_KV_BF16, MOE_KV_MXFP8) or fp16 (MOE_KV_FP16), 16-byte aligned, strides
 *               multiples of 8 values
 *   page_table  [B] rows of table_width int32, table_stride apart;  lens [B] int32
 *   max_len     at most table_width * page_size and 2^30; the work is shared out by it, so it should be near the longest row
 *   lse         [B][n_q_heads] fp32, or NULL
 *   workspace   moe_attention_decode_workspace_bytes(...) bytes, 16-byte aligned (NULL if that is 0)
 * Errors: NULL, SHAPE (B<0, B * n_q_heads > 2^23, heads, head_dim, strides, max_len, scale, window<0), BLOCK, DTYPE,
 * ALIGN, WORKSPACE, HIP. */
size_t moe_attention_decode_workspace_bytes(int B, int n_q_heads, int n_kv_heads, int head_dim, int max_len);
moe_status moe_attention_decode(const moe_heads *q, int B, int n_q_heads, const moe_kv_cache *cache,
                                const int32_t *page_table, int64_t table_stride, int table_width, const int32_t *lens,
                                int max_len, float scale, int window, const moe_heads *y, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_combine -- weighted reduction [C31] with FP32 output [C32]:
 *   y[t,:] = sum_{j = 0 .. k_total-1, in ascending j} weights[t,j] * y_slots[t*k_total+j,:]
 * Every output element has exactly one owner (no atomics).  A slot of weight 0 adds nothing, whatever
 * its row holds: rows of dropped slots are not written by the expert FFN.
 *   y_slots [T*k_total][H] fp32, weights [T][k_total] fp32, y [T][H] fp32 out; H % 4 == 0,
 *   y_slots and y 16-byte aligned.
 * Errors: NULL, SHAPE, ALIGN, HIP. */
moe_status moe_combine(const float *y_slots, const float *weights, int T, int k_total, int H,
                       float *y, void *stream);

/* ---------------------------------------------------------------------------------------------
 * moe_mxfp4_dequant -- the device decode primitive of the expert FFN, exposed on its own: writes
 * out[n][k] = bf16(v(code) * 2^(scale-127)) for an [n_rows][K] MXFP4 matrix [MX].  The value is
 * exact in bf16 whenever it is finite (all scale codes 0..252; larger codes can overflow).
 *   codes [n_rows] rows of K/2 bytes at code_row_stride; scales [n_rows] rows of K/32 bytes at
 *   scale_row_stride; out [n_rows][K] bf16 (uint16 bits), 16-byte aligned.
 * Errors: NULL, SHAPE, BLOCK (K % 32, or codes / code_row_stride off the 16-byte block grid),
 * ALIGN (out), HIP. */
moe_status moe_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, int n_rows, int K,
                             int64_t code_row_stride, int64_t scale_row_stride, uint16_t *out,
                             void *stream);

/* moe_stream_read -- a measurement utility, not a step of the layer: reads `bytes` of device memory
 * at `buf` once, with 16-byte nontemporal loads in which consecutive lanes take consecutive 16-byte
 * pieces (every wave load covers whole 128-byte lines, the shape in which the streaming FFN
 * kernels read their weights), and folds them into a checksum.  Timed over a buffer much larger
 * than the caches, it gives the practical HBM read rate that those kernels are compared with.
 *   buf device memory, 16-byte aligned, read only; bytes a multiple of 16 (0 is a no-op);
 *   sink one device uint32, written only when the checksum takes one fixed value, so its
 *   contents are meaningless (it exists so that the loads cannot be removed).
 * Errors: NULL, ALIGN (buf or bytes), HIP. */
moe_status moe_stream_read(const void *buf, size_t bytes, uint32_t *sink, void *stream);

/* Short text for a status code (host, static storage). */
const char *moe_status_str(moe_status status);
/* MOE_ABI_VERSION of the built library. */
int moe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
