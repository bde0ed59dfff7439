/*
 * moe.h -- C ABI of a sparse top-k Mixture-of-Experts feed-forward layer
 * (Mixtral 8x7B style top-2, and the fine-grained many-expert form with a
 * shared expert) implemented with hand-written HIP kernels for AMD Instinct
 * MI355X (gfx950).
 *
 * The layer (pages: "Mixtral and Mixture-of-Experts, Explained", section
 * "How it works"; "Mixtral" study notes, section "MoE Layer"):
 *   logits  = x . W_g^T (+ b)                 router, one logit per expert
 *   G(x)    = Softmax(TopK(logits)), k = 2     non-selected logits at -inf
 *   y       = sum_i G(x)_i * Expert_i(x)
 *   Expert  = w2( silu(x w1^T) * (x w3^T) )    SwiGLU, no biases
 * General form ("Mixtral 8x7B" interview page, section on how MoE design
 * changed since Mixtral: DeepSeek-V3 routes each token to 8 of 256 experts
 * and sends every token through one shared expert as well):
 *   top_k = k in 1..8 of up to 256 routed experts, G = softmax over the k
 *   kept logits, and with n_shared = 1
 *   y      += Expert_E(x)                      shared expert, weight 1
 *   (weights of the shared expert are stored as expert index E, after the
 *   routed ones; it takes every token and no capacity limit applies to it).
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensor arguments are DEVICE pointers to row-major arrays owned by
 *   the caller, each 16-byte aligned (as allocator-returned memory is; a
 *   misaligned one returns MOE_ERR_INVALID_ARG): the kernels' vector loads
 *   and stores stay aligned from there under the shape limits below.  The
 *   library allocates no memory, keeps no mutable global state and is
 *   re-entrant; calls on different streams may overlap.  The one
 *   exception is moe_forward_noalloc (below), which uses a device array of the
 *   library's own and remembers its address per device.
 * - `stream` is a hipStream_t passed as an opaque pointer (NULL = the null
 *   stream).  Every call only enqueues work on it and returns without
 *   waiting for the device; no call reads device memory on the host.
 * - Host-side validation happens before anything is enqueued.  On any
 *   error nothing is enqueued and a status other than MOE_OK is returned;
 *   MOE_ERR_HIP means a launch failed (its HIP error is consumed).
 * - Device contents are not validated.  Preconditions: x, W_g, weights and
 *   scales finite; ids written by moe_route_topk (or equivalent) in [0, E).
 * - T = 0 is legal: every call returns MOE_OK and enqueues nothing.
 * - Expert ids count from 0.  A token's slots follow its logits in
 *   descending order (slot 0 the largest); equal logits go to the lower
 *   expert index.
 * - Assignment ("slot") (t, s) of token t has index t*k + s, s < k.  With a
 *   shared expert the T extra assignments (t, shared) have indices
 *   T*k + t.  S = n_shared, R = T*(k + S) is the number of slots.
 * - Rows of the permuted buffers are grouped by expert (routed experts
 *   0..E-1, then the shared expert E); inside an expert they follow
 *   ascending token index (a token has at most one row per expert).
 *   Buffers indexed by row are sized for R rows, the most any call can
 *   produce, so one set of buffers serves dropless and capacity modes.
 *
 * dtypes (moe_shape_t.act_dtype / w_dtype):
 *   act F32  + w F32       : x, W_g, y fp32; x_perm fp32; h fp32.
 *   act BF16 + w BF16      : x, W_g, y bf16; x_perm bf16; h bf16; fp32 accumulate.
 *   act BF16 + w FP8_E4M3  : x, W_g, y bf16; expert weights are OCP e4m3 codes
 *                            with one fp32 scale per output channel (row of the
 *                            [out, in] weight).  Activations are quantised for
 *                            the fp8 matrix cores: x_perm and h are e4m3 codes
 *                            with one power-of-two scale per row and per block
 *                            of 32 consecutive elements, stored as an E8M0
 *                            byte (scale = 2^(byte - 127)); the block exponent
 *                            is ceil(log2(fp32(amax / 448))), 127 for a zero
 *                            block.  fp32 accumulate.
 *   act BF16 + w MXFP4     : x, W_g, y bf16; x_perm bf16; h bf16.  Expert weights
 *                            are OCP Microscaling FP4: E2M1 codes, two per byte
 *                            (even element in the low nibble), [E+S, F, d/2] /
 *                            [E+S, d, F/2] bytes, with one E8M0 scale byte
 *                            (2^(byte - 127)) per row and block of 32
 *                            consecutive input elements, [E+S, F, d/32] /
 *                            [E+S, d, F/32] bytes.  The matrix cores see the
 *                            exact dequantised weights in bf16; fp32
 *                            accumulate.  A weight-streaming (decode) format:
 *                            at most 64 rows per expert (T <= 64, or capacity
 *                            <= 64 without a shared expert), d_model and d_ff
 *                            multiples of 256.
 *   Other combinations return MOE_ERR_UNSUPPORTED.
 *
 * Shape limits: 1 <= top_k <= 8 (top_k <= n_experts); 2 <= n_experts <= 256
 * (fp32 activations: <= 64); n_shared 0 or 1; d_model and d_ff multiples
 * of 64; 1 <= T <= 2^24 (or 0); capacity == MOE_DROPLESS or >= 0;
 * MOE_OVERFLOW_NEXT_BEST with a capacity needs top_k == 2.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* NULL required pointer, pointer not 16-byte aligned, bad shape value */
  MOE_ERR_UNSUPPORTED = 2,   /* legal but not implemented: shape limit, dtype combo */
  MOE_ERR_WORKSPACE = 3,     /* workspace NULL or smaller than moe_workspace_bytes() */
  MOE_ERR_HIP = 4            /* a kernel launch failed */
} moe_status_t;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_FP8_E4M3 = 2, MOE_MXFP4 = 3 } moe_dtype_t;

#define MOE_DROPLESS (-1)

/* What happens to an assignment the capacity limit drops (moe_shape_t.overflow).
 * Pages: "How Mixtral 8x7B uses mixture of experts", section "Routing without
 * auxiliary loss": tokens over an expert's capacity are dropped there and
 * handed to a fallback, most often the token's next-best expert.
 *   MOE_OVERFLOW_DROP       it contributes nothing.
 *   MOE_OVERFLOW_NEXT_BEST  one fallback round: a dropped slot is offered to the
 *     token's best expert outside its top-2 (3rd-ranked by logit; when both
 *     slots of the token were dropped, slot 0 to the 3rd- and slot 1 to the
 *     4th-ranked), keeping its gate weight.  Each expert takes the offers into
 *     the slots the capacity round left free (capacity minus what it kept),
 *     ranked like the capacity round (gate weight descending, then token
 *     ascending); the other offers stay dropped.  The ranking ties to the
 *     lower expert index, like the top-2.  Defined for top_k == 2 only. */
#define MOE_OVERFLOW_DROP 0
#define MOE_OVERFLOW_NEXT_BEST 1

typedef struct {
  int32_t T;          /* tokens (batch * seq_len, flattened) */
  int32_t d_model;    /* hidden size d */
  int32_t d_ff;       /* expert FFN width F */
  int32_t n_experts;  /* E routed experts */
  int32_t top_k;      /* k, 1..8 */
  int32_t capacity;   /* MOE_DROPLESS, or slots per expert (0 drops every assignment) */
  int32_t act_dtype;  /* moe_dtype_t of x, W_g, y */
  int32_t w_dtype;    /* moe_dtype_t of w1, w3, w2 */
  int32_t overflow;   /* MOE_OVERFLOW_DROP or MOE_OVERFLOW_NEXT_BEST (ignored when dropless) */
  int32_t n_shared;   /* S: 0, or 1 shared expert (weights at expert index E) */
} moe_shape_t;

/* Which call a workspace is sized for. */
typedef enum { MOE_CALL_PERMUTE = 0, MOE_CALL_GATE_UP = 1, MOE_CALL_DOWN = 2,
               MOE_CALL_FORWARD = 3, MOE_CALL_ROUTE = 4,
               /* of moe_linear_workspace_bytes only */
               MOE_CALL_LINEAR = 5, MOE_CALL_LINEAR_BACKWARD = 6,
               /* of moe_ffn_workspace_bytes only */
               MOE_CALL_FFN_GATE_UP = 7, MOE_CALL_FFN_BACKWARD = 8 } moe_call_t;

/* Human-readable name of a status.  Never NULL. */
const char* moe_status_string(moe_status_t status);

/* Library version string, e.g. "moe-mi355x 0.1 gfx950". */
const char* moe_version(void);

/* Bytes of device workspace `call` needs for `shape` (0 is possible; a
 * NULL workspace is accepted then).  Host-only.  Workspace contents need
 * not be initialised and are garbage after the call.  Errors: NULL
 * argument or invalid shape. */
moe_status_t moe_workspace_bytes(const moe_shape_t* shape, moe_call_t call, size_t* bytes);

/* Router + top-k + gate weights.
 * Pages: "Mixtral" study notes, MixtralMoE.forward (gate, topk, softmax over
 * the kept logits); "Mixtral and Mixture-of-Experts, Explained", gate
 * equation G(x) = Softmax(TopK(x . W_g)).
 *   x            [T, d]   act dtype
 *   w_gate       [E, d]   act dtype (nn.Linear [out, in] layout)
 *   router_bias  [E] fp32 or NULL, added to the fp32 logits after the dot product
 *   topk_ids     [T, k] int32 out: the k largest logits in descending order,
 *                ties -> lower index
 *   topk_weights [T, k] fp32 out.  k == 2: w0 = 1/(1+exp(l1-l0)), w1 = 1-w0
 *                (w0+w1 == 1 exactly).  Otherwise w_j = exp(l_j - l_0) / sum_i
 *                exp(l_i - l_0) over the kept logits (k == 1: w0 = 1).
 *   logits       [T, E] fp32 out, or NULL
 *   next_ids     [T, 2] int32 out, or NULL: the experts ranked k+1 and k+2 of
 *                each token (same order: logit descending, ties -> lower index),
 *                -1 where n_experts is too small.  moe_permute needs them for
 *                MOE_OVERFLOW_NEXT_BEST.
 * Logits accumulate in fp32.
 * Workspace: moe_workspace_bytes(MOE_CALL_ROUTE) bytes, 16-byte aligned: T*E*4
 * (an fp32 logit buffer) for bf16 shapes with more than 64 experts, whose
 * router runs as a logits kernel over a token x expert grid followed by a
 * selection kernel; 0 otherwise.  When `logits` is given it serves as that
 * buffer and the workspace may be NULL.  Too small or NULL when needed ->
 * MOE_ERR_WORKSPACE. */
moe_status_t moe_route_topk(const moe_shape_t* shape, const void* x, const void* w_gate,
                            const float* router_bias, int32_t* topk_ids, float* topk_weights,
                            float* logits, int32_t* next_ids, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Capacity selection (when shape->capacity >= 0) and grouping of tokens by expert.
 * Pages: "How Mixtral 8x7B uses mixture of experts", sections "Routing without
 * auxiliary loss" (capacity-limited dispatch, excess dropped) and the
 * bincount of the top-2 ids (expert activation listing); the simplified
 * forward pass, which batches each expert's tokens and writes results back in
 * token order.
 *   topk_ids, topk_weights [T, k] from moe_route_topk
 *   next_ids       [T, 2] from moe_route_topk; required with a capacity and
 *                  MOE_OVERFLOW_NEXT_BEST, else ignored (may be NULL)
 *   x              [T, d] act dtype
 *   expert_counts  [E+S] int32 out: kept assignments per expert (shared: T)
 *   expert_offsets [E+S+1] int32 out: exclusive prefix sum of counts
 *   perm_src       [R] int32 out: rows 0..offsets[E+S]-1 hold the slot index
 *                  (t*k+s, or T*k+t for the shared expert) of each row
 *   slot_to_row    [R] int32 out: row of each slot, -1 if dropped
 *   drop_mask      [T*k] uint8 out or NULL: 0 = kept by its top-k expert,
 *                  1 = dropped, 2 = kept by its fallback expert (NEXT_BEST)
 *   x_perm         [R, d] out: x_perm[row] = x[token of perm_src[row]]; fp8 configs:
 *                  e4m3 codes [R, d] plus x_perm_scale [R, d/32] E8M0 bytes
 *   x_perm_scale   fp8 configs only (else ignored; may be NULL)
 * Capacity rule: per expert, assignments ranked by gate weight (descending,
 * compared as fp32), ties to the lower token index; the first `capacity`
 * are kept.  A dropped assignment contributes nothing and the token's other
 * slots are not renormalised; with MOE_OVERFLOW_NEXT_BEST the fallback round
 * above runs next and the rows of each expert include the slots it took
 * (still one row per token and expert, in ascending token order).
 * Workspace: moe_workspace_bytes(MOE_CALL_PERMUTE). */
moe_status_t moe_permute(const moe_shape_t* shape, const int32_t* topk_ids,
                         const float* topk_weights, const int32_t* next_ids, const void* x,
                         int32_t* expert_counts,
                         int32_t* expert_offsets, int32_t* perm_src, int32_t* slot_to_row,
                         uint8_t* drop_mask, void* x_perm, uint8_t* x_perm_scale,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Grouped expert gate/up projection with the SwiGLU product fused in:
 * h[row] = silu(x_perm[row] . w1[e]^T) * (x_perm[row] . w3[e]^T) for every row of
 * expert e (rows offsets[e] .. offsets[e+1]-1).
 * Pages: "Mixtral" study notes, MixtralExpert.forward and "SwiGLU Experts".
 *   x_perm, x_perm_scale as written by moe_permute
 *   expert_offsets [E+S+1] int32 (device)
 *   w1, w3         [E+S, F, d] weight dtype (MXFP4: [E+S, F, d/2] bytes); w1_scale,
 *                  w3_scale: fp8 [E+S, F] fp32, MXFP4 [E+S, F, d/32] E8M0 bytes, else unused
 *   h              [R, F] out (bf16 / fp32 / e4m3 codes); h_scale [R, F/32] E8M0 (fp8 only)
 * Workspace: moe_workspace_bytes(MOE_CALL_GATE_UP). */
moe_status_t moe_expert_gemm_gate_up(const moe_shape_t* shape, const void* x_perm,
                                     const uint8_t* x_perm_scale, const int32_t* expert_offsets,
                                     const void* w1, const void* w3, const void* w1_scale,
                                     const void* w3_scale, void* h, uint8_t* h_scale,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* Grouped expert down projection: y_perm[row] = h[row] . w2[e]^T (fp32 out).
 * Pages: "Mixtral" study notes, MixtralExpert.forward (self.w2).
 *   h, h_scale     as written by moe_expert_gemm_gate_up
 *   expert_offsets [E+S+1] int32
 *   w2             [E+S, d, F] weight dtype (MXFP4: [E+S, d, F/2] bytes); w2_scale: fp8
 *                  [E+S, d] fp32, MXFP4 [E+S, d, F/32] E8M0 bytes, else unused
 *   y_perm         [R, d] fp32 out
 * Workspace: moe_workspace_bytes(MOE_CALL_DOWN) bytes, 16-byte aligned, device
 * memory owned by the caller (0 for shapes that need none; then it may be
 * NULL).  bf16 shapes with more than 64 rows per expert use it for fp32
 * partial tiles: the tiles left over after the last full round of the
 * persistent launch are split along K across workgroups and summed by a
 * second kernel in K order, so results do not depend on timing.  Its
 * contents need no initialisation and are garbage afterwards.  Too small or
 * NULL when needed -> MOE_ERR_WORKSPACE.  Two calls that share a workspace
 * must not run concurrently. */
moe_status_t moe_expert_gemm_down(const moe_shape_t* shape, const void* h, const uint8_t* h_scale,
                                  const int32_t* expert_offsets, const void* w2,
                                  const void* w2_scale, float* y_perm, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Gate-weighted combine back to token order:
 * y[t] = sum over kept slots s of topk_weights[t, s] * y_perm[slot_to_row[t*k+s]]
 *        (+ y_perm[slot_to_row[T*k+t]] with a shared expert),
 * 0 when every slot is dropped and there is no shared expert; accumulated in
 * fp32 in slot order (shared last), cast to the act dtype (round to nearest even).
 * Pages: "Mixtral and Mixture-of-Experts, Explained", y = sum_i G(x)_i Expert_i(x);
 * study notes, an all-zero output of x's shape, then weighted accumulation.
 *   y_perm [R, d] fp32; slot_to_row [R] int32; topk_weights [T, k] fp32
 *   y      [T, d] act dtype out.  No workspace. */
moe_status_t moe_combine(const moe_shape_t* shape, const float* y_perm, const int32_t* slot_to_row,
                         const float* topk_weights, void* y, void* stream);

/* The whole layer on one stream, with no host synchronisation:
 * route -> (capacity) -> permute -> gate/up -> down -> combine.
 *   x [T, d], w_gate [E, d] act dtype; router_bias [E] fp32 or NULL
 *   w1, w3 [E+S, F, d], w2 [E+S, d, F] weight dtype; w*_scale as for the two GEMM calls
 *   (fp8: fp32 per output channel; MXFP4: E8M0 bytes per 32-element block)
 *   y [T, d] act dtype out
 *   optional outputs (NULL to skip): topk_ids_out [T, k] int32, topk_weights_out [T, k]
 *   fp32, expert_counts_out [E+S] int32, drop_mask_out [T*k] uint8 (0 / 1 / 2 as in
 *   moe_permute), logits_out [T, E] fp32
 * topk_ids_out are the router's choices; with MOE_OVERFLOW_NEXT_BEST a slot
 * whose drop mask is 2 was processed by its fallback expert instead.
 * Results equal the five calls above made in order, bit for bit.  Fewer
 * kernels run where they can: with bf16 activations and bf16 or MXFP4 experts,
 * gate/up reads the token rows of x through perm_src instead of a permuted
 * copy when at most 64 rows reach any expert, and (bf16 experts) when the
 * routed experts average at most 320 rows; for decode batches (T <= 16,
 * E <= 16, top-2, dropless, no shared expert) the router's product runs on
 * eight workgroups and a ninth selects and also groups the tokens, and with
 * bf16 experts the down projection and the combine are one kernel (no
 * y_perm).
 * Workspace: moe_workspace_bytes(MOE_CALL_FORWARD) holds every intermediate. */
moe_status_t moe_forward(const moe_shape_t* shape, const void* x, const void* w_gate,
                         const float* router_bias, const void* w1, const void* w3, const void* w2,
                         const void* w1_scale, const void* w3_scale, const void* w2_scale,
                         void* y, int32_t* topk_ids_out, float* topk_weights_out,
                         int32_t* expert_counts_out, uint8_t* drop_mask_out, float* logits_out,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the device scratch array behind moe_forward_noalloc (64 MiB per GPU). */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* moe_forward for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, results (bit for bit) and errors as moe_forward, without the
 * workspace: the intermediates live in a file-scope device array of
 * MOE_NOALLOC_SCRATCH_BYTES bytes that the library holds on every GPU it runs
 * on until the process ends.  This call allocates nothing and calls no
 * allocating routine.
 *   Limit: a shape whose moe_workspace_bytes(shape, MOE_CALL_FORWARD) exceeds
 *   MOE_NOALLOC_SCRATCH_BYTES returns MOE_ERR_WORKSPACE with nothing enqueued.
 *   That admits the weight-streaming (decode) shapes: at d_model 4096, d_ff
 *   14336, top-2 bf16 a token needs about 106 KiB (T <= 64 there: larger
 *   batches take the tiled path, whose split-tail buffer alone is larger).
 *   Device: `stream` must belong to the current device (else
 *   MOE_ERR_INVALID_ARG); the first call on a device looks up that device's
 *   address of the array (MOE_ERR_HIP if that fails; at most 64 devices).
 *   Concurrency: all calls on one GPU share its array, which keeps the last
 *   call's contents; calls that overlap on one GPU (other streams or threads)
 *   race on it and must be serialised by the caller.  No kernel of the layer
 *   reads scratch it has not written in the same call, so nothing needs
 *   clearing between calls. */
moe_status_t moe_forward_noalloc(const moe_shape_t* shape, const void* x, const void* w_gate,
                                 const float* router_bias, const void* w1, const void* w3,
                                 const void* w2, const void* w1_scale, const void* w3_scale,
                                 const void* w2_scale, void* y, int32_t* topk_ids_out,
                                 float* topk_weights_out, int32_t* expert_counts_out,
                                 uint8_t* drop_mask_out, float* logits_out, void* stream);

/* ---- scored routing ----
 * The general router of fine-grained layers, on given logits: moe_route_topk's
 * place is taken by a product for the logits (moe_linear with fp32 output) and
 * moe_route_scored; its ids, weights and next_ids go to moe_permute, moe_combine
 * and moe_forward_routed like moe_route_topk's. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;

typedef struct {
  int32_t score;        /* moe_score_t: s = softmax(logits) over all E experts, or sigmoid(logits) */
  int32_t n_groups;     /* groups of n_experts / n_groups consecutive experts, 1..64 (1: no groups) */
  int32_t topk_groups;  /* groups a token may choose from, 1..n_groups */
  int32_t group_top;    /* a group's score is the sum of its 1 or 2 largest choices */
  int32_t renormalize;  /* 1: weights divided by the sum of the chosen scores; 0: not */
  float scale;          /* weights are multiplied by this (finite) */
} moe_router_t;

/* Scored top-k selection.  Uses T, n_experts (to 256, whatever the types) and top_k
 * of the shape; its other fields are not looked at.
 * Pages: "How Mixtral 8x7B uses mixture of experts", the simplified forward pass
 * (softmax over all experts, top-k, renormalise); "Mixtral 8x7B" interview page,
 * section on how MoE design changed since Mixtral.
 *   logits       [T, E] fp32
 *   balance_bias [E] fp32 or NULL: added to the scores for the choice only,
 *                c = s + balance_bias
 *   topk_ids     [T, k] int32 out: the k largest c among the experts of the
 *                topk_groups best groups, in descending order, ties -> lower
 *                index (groups likewise)
 *   topk_weights [T, k] fp32 out: scale * s_j, divided by the sum of the k
 *                chosen s with renormalize
 *   scores       [T, E] fp32 out or NULL: s
 *   next_ids     [T, 2] int32 out or NULL: the experts ranked k+1 and k+2 among
 *                the same groups' experts, -1 where there are no more
 * The order is that of the scores of the given logits as fp64 arithmetic has
 * them (without a balance bias: that of the logits), whatever fp32 rounding would
 * make of them, so it depends on nothing but the row.
 * Logits may be -inf (a masked expert: score 0, so c = balance_bias; a row of
 * nothing else gets zero weights) and balance_bias -inf (never chosen while
 * another candidate is left).  A NaN logit counts as -inf, in rank, score, weight
 * and gradient; +inf counts as the largest finite value; a NaN balance_bias ranks as
 * -inf.  The ids of a row are distinct and in [0, E) whatever the contents.
 * Errors: MOE_ERR_INVALID_ARG for a router value outside its range, n_groups
 * that does not divide n_experts, group_top above the group's size, or fewer
 * than top_k experts in topk_groups groups; MOE_ERR_UNSUPPORTED above 64 groups.
 * No workspace. */
moe_status_t moe_route_scored(const moe_shape_t* shape, const moe_router_t* router, const float* logits,
                              const float* balance_bias, int32_t* topk_ids, float* topk_weights,
                              float* scores, int32_t* next_ids, void* stream);

/* Gradient of moe_route_scored at the logits (the choice itself has none).
 *   logits, topk_ids  as given to / written by moe_route_scored (an id outside
 *                [0, E) adds nothing; an expert named twice gets both gradients)
 *   dweights     [T, k] fp32: gradient at topk_weights
 *   dscores      [T, E] fp32 or NULL: gradient that arrives at the scores from
 *                elsewhere (a balance loss)
 *   dlogits      [T, E] fp32 out
 * No workspace. */
moe_status_t moe_route_scored_backward(const moe_shape_t* shape, const moe_router_t* router,
                                       const float* logits, const int32_t* topk_ids,
                                       const float* dweights, const float* dscores, float* dlogits,
                                       void* stream);

/* Gradient of moe_combine.
 *   dy           [T, d] act dtype: gradient at y
 *   y_perm, slot_to_row, topk_weights as given to moe_combine (y_perm may be NULL
 *                when dweights is)
 *   dy_perm      [R, d] act dtype out, or NULL: gradient at y_perm, w[t, s] * dy[t]
 *                (shared expert: dy[t]) in row slot_to_row of each kept slot; rows
 *                no slot points to are left as they were
 *   dweights     [T, k] fp32 out, or NULL: <dy[t], y_perm[row]>, summed in fp64; 0
 *                for a dropped slot
 * At least one output must be given where T > 0.  No workspace. */
moe_status_t moe_combine_backward(const moe_shape_t* shape, const void* dy, const float* y_perm,
                                  const int32_t* slot_to_row, const float* topk_weights, void* dy_perm,
                                  float* dweights, void* stream);

/* moe_forward from a given routing (moe_route_scored's, or any other) instead of
 * its own router: permute -> gate/up -> down -> combine, bit for bit the staged
 * calls on the same ids and weights.
 *   topk_ids [T, k], topk_weights [T, k]; next_ids [T, 2], required with a
 *   capacity and MOE_OVERFLOW_NEXT_BEST, else ignored (may be NULL); the ids of a
 *   token distinct, in [0, E)
 *   other arguments as for moe_forward
 * Workspace: moe_workspace_bytes(MOE_CALL_FORWARD). */
moe_status_t moe_forward_routed(const moe_shape_t* shape, const void* x, const int32_t* topk_ids,
                                const float* topk_weights, const int32_t* next_ids, const void* w1,
                                const void* w3, const void* w2, const void* w1_scale,
                                const void* w3_scale, const void* w2_scale, void* y,
                                int32_t* expert_counts_out, uint8_t* drop_mask_out, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---- dense product ----
 *   y = act(x . w^T + bias) + residual
 * The router's product (fp32 logits) and the dense projections around the
 * experts (Pages: "Mixtral" study notes, nn.Linear of MixtralMoE and
 * MixtralBlock). */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2,
               MOE_ACT_GELU = 3,        /* p Phi(p), with erf */
               MOE_ACT_GELU_TANH = 4    /* its tanh form, sqrt(2/pi) (p + 0.044715 p^3) */
} moe_act_t;

typedef struct {
  int32_t M;        /* rows (tokens), 0..2^24 */
  int32_t N;        /* output channels: a multiple of 8, at most 2^18 */
  int32_t K;        /* input channels: a multiple of 8, at most 2^18 */
  int32_t dtype;    /* x, w, pre, dx, dw: MOE_BF16 or MOE_F32 */
  int32_t y_dtype;  /* y, residual, dy: MOE_BF16 or MOE_F32 (MOE_F32 with MOE_F32 operands) */
  int32_t act;      /* moe_act_t */
} moe_linear_t;

/* Bytes of device workspace moe_linear (MOE_CALL_LINEAR) or moe_linear_backward
 * (MOE_CALL_LINEAR_BACKWARD) needs; 0 is possible (a NULL workspace is accepted
 * then).  Two calls that share a workspace must not run concurrently. */
moe_status_t moe_linear_workspace_bytes(const moe_linear_t* linear, moe_call_t call, size_t* bytes);

/*   x        [M, K] dtype;  w [N, K] dtype (nn.Linear [out, in] layout)
 *   bias     [N] fp32 or NULL;  residual [M, N] y_dtype or NULL
 *   y        [M, N] y_dtype out; may be the residual's memory, else overlaps no input
 *   pre      [M, N] dtype out, or NULL: x . w^T + bias, kept for the backward pass
 * fp32 accumulation; bias, activation and residual in fp32, one rounding to
 * y_dtype (the activation sees the unrounded pre).  The order of an element's sum
 * depends on M, N, K, the element's row and channel and the device's number of CUs,
 * and is the same from call to call; equal rows of x may differ in their last bits,
 * within one call and between calls of other M. */
moe_status_t moe_linear(const moe_linear_t* linear, const void* x, const void* w, const float* bias,
                        const void* residual, void* y, void* pre, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Gradients of moe_linear.  With dpre = dy * act'(pre):
 *   dx       [M, K] dtype out or NULL:  dpre . w        (needs w)
 *   dw       [N, K] dtype out or NULL:  dpre^T . x      (needs x)
 *   dbias    [N] fp32 out or NULL:      column sums of dpre, from its fp32 values
 *   dy       [M, N] y_dtype;  pre [M, N] dtype as written by moe_linear, required
 *            unless act is MOE_ACT_NONE (then ignored); the residual's gradient
 *            is dy itself
 * dpre is rounded to dtype for the two products, their matrix-core operand (an fp32 dy
 * of bf16 operands too; MOE_F32 operands keep it whole).  They accumulate in fp32, in
 * an order that depends on the sizes, the element's place, the device's number of CUs
 * and which outputs are asked for, and is the same from call to call.  relu'(0) = 0.
 * Outputs overlap no input and are fully written, with M = 0 too (dw and dbias are
 * then zero).  At least one output must be given where M > 0. */
moe_status_t moe_linear_backward(const moe_linear_t* linear, const void* dy, const void* pre,
                                 const void* x, const void* w, void* dx, void* dw, float* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- gated feed-forward block, dense or grouped by expert, and its gradients ----
 *   g = x . w1[e]^T,  u = x . w3[e]^T,  h = act(g) * u,  y = h . w2[e]^T
 * for the rows of group e.  Pages: "Mixtral" study notes, MixtralExpert.forward and
 * "SwiGLU Experts".  The training form of moe_expert_gemm_gate_up (which keeps nothing
 * and has silu only) and the gated block of a dense layer or shared expert. */
typedef struct {
  int32_t M;        /* rows of the row buffers, 0..2^24 */
  int32_t d_model;  /* channels of x, y: a multiple of 8, at most 2^18 */
  int32_t d_ff;     /* channels of g, u, h: a multiple of 8, at most 2^18 */
  int32_t groups;   /* experts, the shared one included: 1..257 */
  int32_t dtype;    /* every tensor: MOE_BF16 or MOE_F32 */
  int32_t act;      /* moe_act_t */
} moe_ffn_t;
/* No buffer has more than 2^36 elements (M d_model, M d_ff, groups d_model d_ff;
 * MOE_ERR_UNSUPPORTED).
 *
 * offsets [groups + 1] int32 (device), as expert_offsets of moe_permute: group e has the
 * rows offsets[e] .. offsets[e + 1] - 1.  NULL with one group: all M rows.  Groups may be
 * empty.  Rows of no group are not read, and left as they were in every output.
 * (Offsets below 0, above M or descending are read as the nearest that are not.) */

/* Bytes of device workspace moe_ffn_gate_up (MOE_CALL_FFN_GATE_UP) or moe_ffn_backward
 * (MOE_CALL_FFN_BACKWARD) needs; 0 is possible (a NULL workspace is accepted then).  Two
 * calls that share a workspace must not run concurrently. */
moe_status_t moe_ffn_workspace_bytes(const moe_ffn_t* ffn, moe_call_t call, size_t* bytes);

/*   x        [M, d_model];  w1, w3 [groups, d_ff, d_model]
 *   h        [M, d_ff] out
 *   pre1, pre3 [M, d_ff] out, both or neither NULL: g and u, kept for the backward pass
 * fp32 accumulation; h from the unrounded g and u, one rounding.  Outputs overlap no
 * input.  The order of an element's sum depends on M, the widths, the offsets, the element's place
 * and the device's number of CUs, and is the same from call to call. */
moe_status_t moe_ffn_gate_up(const moe_ffn_t* ffn, const void* x, const int32_t* offsets, const void* w1,
                             const void* w3, void* h, void* pre1, void* pre3, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Gradients of y = h . w2[e]^T, h = moe_ffn_gate_up(x).  With dh = dy . w2[e] (fp32),
 * dg = dh * u * act'(g), du = dh * act(g), g and u as kept:
 *   dx       [M, d_model] out or NULL:  dg . w1[e] + du . w3[e]  (needs w1, w3)
 *   dw1, dw3 [groups, d_ff, d_model] out, both or neither NULL:  dg^T . x, du^T . x over the
 *            group's rows  (needs x)
 *   dw2      [groups, d_model, d_ff] out or NULL:  dy^T . h  (needs h)
 *   dy       [M, d_model]
 *   pre1, pre3 [M, d_ff] as written by moe_ffn_gate_up, w2 [groups, d_model, d_ff]:
 *            required for dx, dw1 and dw3
 * dg and du are rounded to dtype for the products, their matrix-core operands (MOE_F32:
 * kept whole); sums in fp32, in an order that is the same from call to call (MOE_F32: dx
 * and weight gradients in parts of 2^15 terms at most).  relu'(0) = 0.  Weight gradients
 * are fully written, zero for a group without rows (M = 0 too).
 * Outputs overlap no input.  At least one output must be given where M > 0. */
moe_status_t moe_ffn_backward(const moe_ffn_t* ffn, const void* dy, const int32_t* offsets, const void* x,
                              const void* pre1, const void* pre3, const void* h, const void* w1,
                              const void* w3, const void* w2, void* dx, void* dw1, void* dw3, void* dw2,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of moe_permute's x_perm at x.  Uses T, d_model, top_k, n_shared and act_dtype
 * of the (valid) shape.
 *   dx_perm      [R, d] act dtype: gradient at x_perm
 *   slot_to_row  [R] as written by moe_permute
 *   addend       [T, d] act dtype or NULL: gradient that reaches x elsewhere (the router's)
 *   dx           [T, d] act dtype out: addend[t] + the sum over kept slots of
 *                dx_perm[slot_to_row[t*k+s]] (+ dx_perm[slot_to_row[T*k+t]] with a shared
 *                expert), in fp32 in that order, rounded once; may be the addend's memory,
 *                else overlaps no input
 * No workspace. */
moe_status_t moe_permute_backward(const moe_shape_t* shape, const void* dx_perm, const int32_t* slot_to_row,
                                  const void* addend, void* dx, void* stream);

/* ---- norm of a list of gradients, and clipping ---- */
typedef struct {
  void* data;       /* device; aligned to its elements (no more), NULL with n = 0 */
  int64_t n;        /* elements, 0..2^40 */
  int32_t dtype;    /* MOE_BF16 or MOE_F32 */
} moe_tensor_t;

/* Bytes of device workspace moe_grad_norm needs for the list. */
moe_status_t moe_grad_norm_workspace_bytes(const moe_tensor_t* tensors, int32_t count, size_t* bytes);

/*   tensors      host array of `count` (0..2^16) tensors; read before the call returns
 *   sum_squares  [1] fp64 out: the sum of the squares of all elements, in fp64, in an
 *                order that depends on the list's sizes and alignments alone.  (Ranks that
 *                hold parts of a model add theirs before moe_grad_clip.)
 *   norm         [1] fp32 out or NULL: its square root (infinite above FLT_MAX)
 * An infinite or NaN element makes both so. */
moe_status_t moe_grad_norm(const moe_tensor_t* tensors, int32_t count, double* sum_squares, float* norm,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Scales the list to a norm of at most max_norm: out = in * min(1, max_norm / sqrt(*sum_squares)),
 * one rounding.  A norm that is not finite in fp32, as moe_grad_norm stores it (the sum may be:
 * a norm above FLT_MAX), scales nothing: the caller sees it there.
 *   tensors, outs  host arrays of `count` tensors each; outs[i] has tensors[i]'s n and dtype
 *                and may be its memory.  outs NULL: in place.  Nothing else may overlap an
 *                output (MOE_ERR_INVALID_ARG).
 *   sum_squares  [1] fp64 (device), read by the kernels, in no output's memory;  max_norm >= 0 */
moe_status_t moe_grad_clip(const moe_tensor_t* tensors, const moe_tensor_t* outs, int32_t count,
                           const double* sum_squares, float max_norm, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
