/*
 * tpmlp_block.h -- C ABI of what a training or serving step does around the
 * products of tpmlp.h, in the same library (libtpmlp.so):
 *
 *   tp_block_norm_fwd / _bwd    the seam between two blocks: the norm after
 *                               a block, its gate and residual scale, the
 *                               residual sum and the next block's norm
 *   tp_moe_route_fwd / _bwd     router scores -> the top-k experts and
 *                               their weights, and the logits' gradient
 *   tp_moe_route_tables         the dispatch tables and expert offsets that
 *                               tp_moe_permute / _combine / _combine_bwd
 *                               and tp_grouped_expert_*_devoff read
 *   tp_adamw_step               one AdamW step over many tensors, states in
 *                               32 or in 8 bits
 *
 * The conventions of tpmlp.h hold: layouts, types, ownership (the library
 * never allocates, frees or synchronizes), 16-byte aligned device pointers
 * unless stated, host-side argument checks before anything is enqueued,
 * errors through tp_last_error().  Every call can be captured into a graph.
 * Results do not depend on timing: no floating-point atomics anywhere.
 *
 * Citations: [P3] "Megatron Core 带读" (§03 layer order: norm -> attention /
 * MLP -> residual; §09 MoE router -> top-k -> dispatch -> combine), [P1]
 * "Megatron-LM 源码精读——大模型并行训练全景" (§五 the optimizer and its fp32
 * main parameters).
 */
#ifndef TPMLP_BLOCK_H
#define TPMLP_BLOCK_H

#include "tpmlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Block norms
 * ------------------------------------------------------------------------
 * For every token n, with the block's output O, the residual stream X, a =
 * res_scale, b = branch_scale:
 *
 *   u = norm(O; w_post, b_post)          (O itself where w_post is NULL)
 *   Y = a X + b gate[n mod gate_rows] u  (no gate where gate_rows is 0)
 *   Hn = norm(Y; w_pre, b_pre)           (not made where w_pre is NULL)
 *
 *   TP_NORM_RMS:   norm(t) = t r w + b,        r = (mean t^2 + eps)^(-1/2)
 *   TP_NORM_LAYER: norm(t) = (t - mu) r w + b, r = (mean (t-mu)^2 + eps)^(-1/2)
 *
 * O NULL: there is no block before the norm, Y = X: then w_post, b_post,
 * gate, Y, stat_post are NULL (gate_rows 0) and only Hn = norm(X) is made.
 *
 * gate_rows: 1 a learned gate for each channel; B one gate row for each
 * sequence of an [S,B,H] batch (token n = s*B + b has row n mod B); N one
 * for each token; any number is taken.
 *
 * Everything between loading and storing is fp32; Hn comes from Y before
 * Y's rounding.  Statistics, fp32: stat_* [N] = r (TP_NORM_RMS) or [2N] =
 * r then mu (TP_NORM_LAYER); NULL where no backward follows.
 */
typedef enum tp_norm_kind { TP_NORM_RMS = 0, TP_NORM_LAYER = 1 } tp_norm_kind;

/* N tokens (0 .. 2^30), width H (a positive multiple of 8 for bf16, 4 for
 * fp32, at most 2^21), gate_rows 0 .. 2^30, kind a tp_norm_kind, dtype a
 * tp_dtype (activations, weights and gate alike), eps > 0, eps and scales
 * finite. */
typedef struct tp_norm_desc {
    int64_t N, H, gate_rows;
    int32_t kind, dtype;
    float eps, res_scale, branch_scale;
} tp_norm_desc;

/*
 * tp_block_norm_fwd
 *   X [N,H], O [N,H] or NULL, w_post, b_post, w_pre, b_pre [H] (each bias
 *   may be NULL; a bias needs its weight), gate [gate_rows,H] (NULL if 0)
 *   Y [N,H], Hn [N,H] out; stat_post, stat_pre out (may be NULL)
 * Y may be X itself (the residual stream updated in place); no other
 * overlap is allowed.
 * Errors: TP_ERR_SHAPE, TP_ERR_DTYPE, TP_ERR_NULL, TP_ERR_ALIGN (stat_*:
 * 4-byte), TP_ERR_ALIAS, TP_ERR_DEVICE, TP_ERR_HIP.
 */
int tp_block_norm_fwd(const tp_norm_desc *desc, const void *X, const void *O, const void *w_post,
                      const void *b_post, const void *gate, const void *w_pre, const void *b_pre,
                      void *Y, void *Hn, float *stat_post, float *stat_pre, void *stream);

/*
 * tp_block_norm_bwd -- gradients of the forward above, from its stored Y
 * (X where O is NULL), O and statistics:
 *   dY  [N,H] or NULL   gradient that reaches Y other than through Hn
 *   dHn [N,H]           gradient of Hn (NULL exactly where w_pre is NULL)
 * with D = dY + d norm(Y)^T dHn:
 *   dX = a D   (D where O is NULL)            [N,H]
 *   dO = d norm(O)^T (b gate D)               [N,H]
 *   dgate[g] = b sum over {n mod gate_rows = g} of D u     [gate_rows,H] fp32
 *   dw_post, db_post, dw_pre, db_pre                       [H] fp32
 * accumulate 0: the fp32 gradients are written; 1: added to (as
 * tp_mlp_shard_bwd_accum does).  N = 0 writes zeros (or adds nothing).
 * dw_post / dw_pre are required where the norm is there, db_* where the
 * caller wants them (NULL: not made; they need only the norm), dgate where
 * gate_rows > 0.  b_post is read for dgate only.  Nothing may overlap.
 * Sums over tokens are fp32 in a fixed order: equal calls give equal bits.
 * workspace: tp_block_norm_bwd_workspace(desc) bytes, 16-byte aligned, not
 * shared with a call that may run at the same time (two graphs replayed
 * together, say); its contents do not matter before or after.
 */
size_t tp_block_norm_bwd_workspace(const tp_norm_desc *desc);
int tp_block_norm_bwd(const tp_norm_desc *desc, const void *dY, const void *dHn, const void *Y,
                      const void *O, const void *w_post, const void *b_post, const void *gate,
                      const void *w_pre, const float *stat_post, const float *stat_pre, void *dX,
                      void *dO, float *dw_post, float *db_post, float *dgate, float *dw_pre,
                      float *db_pre, void *workspace, size_t ws_bytes, int32_t accumulate,
                      void *stream);

/* ------------------------------------------------------------------------
 * Routing to experts
 * ------------------------------------------------------------------------
 * For each token, over its E logits l (fp32 or bf16):
 *   s = softmax(l) or sigmoid(l)               scores
 *   c = s + bias  (bias NULL: the order of the logits)     choice
 *   groups > 1: the experts form `groups` equal runs; a run is worth the
 *     sum of its group_best (1 or 2) largest c, and only the experts of the
 *     groups_kept runs worth most stay
 *   the K experts with the largest c, largest first
 *   weight_j = scale s_j                        (renorm 0)
 *   weight_j = scale s_j / (sum_i s_i + 1e-20)  (renorm 1, over the chosen)
 * The bias steers the choice alone (load balance); it is not in the
 * weights.  Equal values go to the lower expert (run).  Choices are decided
 * as by arithmetic in 64 bits, for any finite bias; weights are fp32, from
 * scores off by about 2^-22 relative and by 2^-23 more for each unit of
 * l_max - l (softmax) or |l| (sigmoid): the exponent's rounding.  The gradient
 * has scores of its own, without that growth for a sigmoid.
 * A logit that is NaN, -inf, or at most the lowest finite bf16 (-3.3895e38)
 * takes its expert out of the row: score 0, never chosen.  +inf counts as
 * the largest finite fp32.  Slots left over hold expert -1, weight 0.
 */
typedef enum tp_score { TP_SCORE_SOFTMAX = 0, TP_SCORE_SIGMOID = 1 } tp_score;

/* Limits: E in 1..1024, K in 1..32 (and at most groups_kept * E / groups),
 * groups in 1..64 dividing E, N in 0..2^30 with N*K and N*E below 2^40. */
#define TP_ROUTE_MAX_EXPERTS 1024
#define TP_ROUTE_MAX_K 32
#define TP_ROUTE_MAX_GROUPS 64
typedef struct tp_route_desc {
    int64_t N;
    int32_t E, K;
    int32_t groups, groups_kept, group_best;
    int32_t score, renorm;
    int32_t dtype; /* of the logits and their gradient */
    float scale;   /* finite */
} tp_route_desc;

/*
 * tp_moe_route_fwd
 *   logits [N,E], bias [E] fp32 or NULL (finite)
 *   topk_expert [N,K] int32, topk_weight [N,K] fp32 out
 * Logits (and dlogits) 16-byte aligned, the other pointers 4-byte.
 */
int tp_moe_route_fwd(const tp_route_desc *desc, const void *logits, const float *bias,
                     int32_t *topk_expert, float *topk_weight, void *stream);

/*
 * tp_moe_route_bwd: dlogits [N,E] (the logits' type) from the weights'
 * gradient.  The choice itself has no gradient.
 *   slot_row NULL:  d_weight [N,K], the gradient of topk_weight
 *   slot_row [N,K] (tp_moe_route_tables):  d_weight [R], a gradient for
 *     each row as tp_moe_combine_bwd leaves it; a slot whose row is outside
 *     [0,R) has none
 * A topk_expert outside [0,E) is no choice; one that stands twice in a row
 * counts twice.  Rows without a choice get zeros.  R 0 .. 2^40.
 */
int tp_moe_route_bwd(const tp_route_desc *desc, const void *logits, const int32_t *topk_expert,
                     const float *d_weight, const int32_t *slot_row, int64_t R, void *dlogits,
                     void *stream);

/*
 * tp_moe_route_tables: the dispatch tables of the experts [first_expert,
 * first_expert + n_local), all int32 (row_weight fp32), built on the
 * device.  The (token, slot) pairs whose expert is local become rows,
 * ordered by (expert, token, slot):
 *   offsets    [n_local+1]  the rows of local expert e are offsets[e] ..
 *                           offsets[e+1]-1; offsets[n_local] rows in all
 *   row_token  [R]          the row's token; -1 past the last row
 *   row_weight [R]          its weight; 0 past the last row
 *   tok_ptr    [N+1], tok_rows [R]   each token's rows, ascending (CSR);
 *                           tok_rows -1 past the last
 *   slot_row   [N,K]        the row of (token, slot), -1 if it has none
 * R >= N*K rows (every choice local), below 2^31.  Calls that read the
 * tables may be given any smaller R that offsets[n_local] does not exceed.
 * topk_expert values outside the local range give no row.  n_local in
 * 1..1024 (the grouped calls take 64), first_expert >= 0.  topk_weight and
 * row_weight may both be NULL.  Pointers 4-byte aligned.  workspace:
 * tp_moe_route_tables_workspace(N, K, n_local) bytes (at least 16), 16-byte
 * aligned, not shared with a call that may run at the same time (two graphs
 * replayed together, say); its contents do not matter before or after.
 */
size_t tp_moe_route_tables_workspace(int64_t N, int32_t K, int32_t n_local);
int tp_moe_route_tables(int64_t N, int32_t K, int32_t first_expert, int32_t n_local, int64_t R,
                        const int32_t *topk_expert, const float *topk_weight, int32_t *offsets,
                        int32_t *row_token, float *row_weight, int32_t *tok_ptr,
                        int32_t *tok_rows, int32_t *slot_row, void *workspace, size_t ws_bytes,
                        void *stream);

/* ------------------------------------------------------------------------
 * AdamW
 * ------------------------------------------------------------------------
 * One step over n tensors in few launches.  For each element, with the
 * gradient g = grad * grad_scale, in fp32:
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * param is the fp32 main parameter; param_bf16 (may be NULL) receives its
 * rounding to bf16, the weight that the products read.
 *
 * state_bits 32: m, v fp32 [count]; m_scale, v_scale NULL.
 * state_bits 8: m holds the E4M3 codes of m, v those of r = sqrt(v), one
 *   byte each, with one fp32 scale for each block of TP_ADAMW_BLOCK
 *   elements of a tensor (m_scale, v_scale [ceil(count / 256)]): m = code *
 *   scale, v = (code * scale)^2, scale = max|.| / 448 over the block (0 and
 *   zero values if that maximum is at most 2^-100).  Codes are rounded up
 *   or down by chance such that m and v (not r) are kept on average:
 *   nearest rounding would hold a state still whenever a step changes it by
 *   less than half a code.  The chance comes from a hash of (seed, step,
 *   tensor's place in the list, element), so equal calls give equal bits.
 *   A positive r is never stored as 0, so that a small gradient later does
 *   not meet an empty denominator.
 *   Zeroed codes and scales are the state before the first step.
 *   A NaN or an infinity makes its block's state NaN.
 *
 * step counts from 1.  dev_step (int32), dev_lr (fp32), grad_scale (fp32):
 * device scalars, each may be NULL; dev_step and dev_lr take the place of
 * the descriptor's, so that a captured graph follows them.  If *grad_scale
 * is not finite nothing is changed (an overflowed gradient norm skips the
 * step on the device); if *dev_step < 1, likewise.
 */
#define TP_ADAMW_BLOCK 256
#define TP_ADAMW_MAX_TENSORS 65536
typedef struct tp_adamw_desc {
    double lr, beta1, beta2, eps; /* lr finite in fp32, 0 <= beta < 1, 1e-30 <= eps <= 1e30 */
    int32_t step;                 /* >= 1 (unused with dev_step)       */
    int32_t grad_dtype;           /* a tp_dtype                        */
    int32_t state_bits;           /* 32 or 8                           */
    uint32_t seed;                /* of the 8-bit states' rounding     */
} tp_adamw_desc;

typedef struct tp_adamw_tensor {
    float *param;
    void *param_bf16; /* or NULL */
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale; /* 8-bit states */
    int64_t count;            /* 0 .. 2^40 */
    float weight_decay;       /* finite */
    int32_t reserved;         /* 0 */
} tp_adamw_tensor;

/* tensors: host array of n (it may be freed when the call returns).  No two
 * buffers of the call may overlap.  Pointers 16-byte aligned, scales and
 * device scalars 4-byte. */
int tp_adamw_step(const tp_adamw_desc *desc, int32_t n, const tp_adamw_tensor *tensors,
                  const int32_t *dev_step, const float *dev_lr, const float *grad_scale,
                  void *stream);

#ifdef __cplusplus
}
#endif
#endif /* TPMLP_BLOCK_H */
