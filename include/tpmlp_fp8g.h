/*
 * tpmlp_fp8g.h -- C ABI of FP8 with group scales, in the same library
 * (libtpmlp.so): one scale for each 128 values of a row, or for each 128 x 128
 * square of a weight, where the FP8 calls of tpmlp.h have one for a tensor.
 * A group's scale comes from its own values, so there is no history to keep,
 * and a channel far above the rest costs the others of its group at most
 * their bits, not the tensor's.
 *
 *   tp_fp8g_quantize       values -> codes and scales, along the rows, along
 *                          the columns (of the transpose), or both
 *   tp_fp8g_gemm           the product of two matrices of codes
 *   tp_fp8g_glu_fwd        a gated feed-forward block's two projections, its
 *                          activation and product, and the codes of the
 *                          result: one kernel, or for small sizes two with
 *                          fp32 values between them (in the workspace)
 *   tp_fp8g_glu_bwd        the gradient of both projections' outputs from the
 *                          block's output gradient, and its codes, likewise
 *
 * Codes and scales.  A group of 128 values x with a = max|x| has codes
 * q = round(x / s), E4M3 (448 the largest) or E5M2 (57344), nearest, ties to
 * even, fmax = the largest:
 *   TP_GROUP_F32    s = fp32(a / fmax), codes of fp32(x * fp32(fmax / a))
 *   TP_GROUP_E8M0   s = the least power of two with a / s <= fmax, one byte,
 *                   2^(byte - 127): a quarter of the scales' bytes, and
 *                   nothing is rounded in applying it.  An operand's bytes have
 *                   to be among 12 .. 247 with E4M3 codes, 12 .. 240 with E5M2
 *                   ones, as those made here are, or 255 (NaN)
 * A group with a <= 2^-100 has zero codes and s = 1.  A group that holds a
 * NaN or an infinity has s = NaN (byte 255) and zero codes: what is computed from it
 * is NaN.
 *
 * Layout.  A matrix of R rows and C columns grouped along its rows: codes
 * [R, P(C)] one byte each, P(C) = C rounded up to a multiple of 128, the codes
 * behind C zeros; scales [P(C)/128, R] (the scales of one group of columns,
 * for all rows, lie together).  In squares: the same codes, scales
 * [P(R)/128, P(C)/128].  Every product here runs over groups: it takes
 * two matrices whose rows are grouped along the summed index, C = A B^T.
 *
 * A training step of a gated block, X [N,H], weights Ag, Au [H,F] (gate and
 * up), B [F,H]: quantize X (codes and those of X^T), the weights in squares
 * (codes and those of the transposes), then
 *   glu_fwd   X, Ag^T, Au^T        -> Z, H (along F and along tokens)
 *   gemm      H, B^T               -> Y [N,H]
 *   quantize  dY                   -> along H, along tokens
 *   glu_bwd   dY, B, Z             -> dZ = [dG|dU] (along F and along tokens)
 *   gemm      dZ, [Ag|Au]          -> dX [N,H]     (parts 2)
 *   gemm      H^T, dY^T            -> dB [F,H]
 *   gemm      X^T, dG^T and dU^T   -> dAg, dAu [H,F]
 *
 * The conventions of tpmlp.h hold: layouts, ownership (the library never
 * allocates, frees or synchronizes), 16-byte aligned device pointers (scales
 * 4-byte, E8M0 ones any; those of squares are read in aligned words of 4 bytes, so up
 * to 3 bytes before the first and behind the last are read too, and not
 * used), host-side argument checks before anything is
 * enqueued, errors through tp_last_error().  Every call can be captured into
 * a graph.  Sums are fp32 in an order that goes by the sizes alone, without
 * atomics: equal calls give equal bits.
 *
 * Citations: [P1] "Megatron-LM 源码精读——大模型并行训练全景" (§8.2 FP8), [P3]
 * "Megatron Core 带读" (§10 FP8: quantize by scale/amax -> FP8 kernel ->
 * dequantize).
 */
#ifndef TPMLP_FP8G_H
#define TPMLP_FP8G_H

#include "tpmlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TP_FP8G_GROUP 128
typedef enum tp_group_scale { TP_GROUP_F32 = 0, TP_GROUP_E8M0 = 1 } tp_group_scale;

/* The activation of the gate: H = act(G) U.  SiLU is that of
 * TP_ACT_SWIGLU, GeLU the tanh form. */
typedef enum tp_gate { TP_GATE_SILU = 0, TP_GATE_GELU_TANH = 1 } tp_gate;

/* rows 0 .. 2^30, cols a positive multiple of 8 for bf16, 4 for fp32, at most
 * 2^21; dtype of x (a tp_dtype); fmt TP_FP8_E4M3 or TP_FP8_E5M2; scale a
 * tp_group_scale; square 0: groups of 128 along rows (columns for the
 * transpose), 1: of 128 x 128. */
typedef struct tp_fp8g_quant_desc {
    int64_t rows, cols;
    int32_t dtype, fmt, scale, square;
} tp_fp8g_quant_desc;

/*
 * tp_fp8g_quantize: x [rows,cols] is read once.
 *   q [rows,P(cols)], s            its codes and scales; both NULL: not made
 *   q_t [cols,P(rows)], s_t        those of its transpose; likewise.  In
 *                                  squares q_t is q transposed.
 */
int tp_fp8g_quantize(const tp_fp8g_quant_desc *desc, const void *x, void *q, void *s, void *q_t,
                     void *s_t, void *stream);

/* M 0 .. 2^30; N a positive multiple of 8 for bf16, 4 for fp32, at most 2^21; K a
 * multiple of 128, at most 2^21, for one part (parts 2: 2^20), positive for bf16; of
 * fp32 results K may be 0 (a weight gradient of no tokens: zeros, or C as it was where
 * accumulate is 1; nothing of A, B or the scales is read); parts 1 or 2;
 * fmt_a, fmt_b: both E4M3, or one of them E5M2; scale of A and B alike; square: of B;
 * dtype of C; accumulate 1: added into C (fp32 only). */
typedef struct tp_fp8g_gemm_desc {
    int64_t M, N, K;
    int32_t parts, fmt_a, fmt_b, scale, square, dtype, accumulate;
} tp_fp8g_gemm_desc;

/*
 * tp_fp8g_gemm: C [M,N] = sum over parts p of A_p B_p^T
 *   A [M,parts*K], sA [parts*K/128,M]
 *   B [N,K], sB: part 0;  B2, sB2: part 1 (NULL where parts is 1)
 * Products of codes are exact.  fp32 results, and bf16 ones of at most 64
 * rows or of sizes with few outputs, add them in fp32, group by group
 * (TP_GROUP_F32: a group's sum times fp32(sA sB), which has to be in fp32's
 * range).  The other bf16 results take a group's sum from the FP8 matrix
 * instruction, which keeps 13 bits below the largest of 8 products: it loses
 * 1.5e-5 of a sum of normally distributed codes (root mean square), up to some
 * 3e-4 where a few values are far above the rest; the rounding to bf16 takes
 * 1.7e-3, at most 2^-8.  A result near cancellation, where that loss is large
 * beside it, may so differ between a batch of 64 rows and one of 65.  Groups are
 * added in fp32 (with E8M0 scales by the instruction itself, to 24 bits of the
 * running sum) and C is rounded once.
 */
int tp_fp8g_gemm(const tp_fp8g_gemm_desc *desc, const void *A, const void *sA, const void *B,
                 const void *sB, const void *B2, const void *sB2, void *C, void *stream);

/* N 0 .. 2^30 tokens, H and F positive multiples of 8 (H at most 2^21, F 2^20);
 * gate a tp_gate; scale of every operand and result; fmt: of dY and dZ
 * (glu_bwd; every other code is E4M3, and glu_fwd takes fmt TP_FP8_E4M3 alone). */
typedef struct tp_fp8g_glu_desc {
    int64_t N, H, F;
    int32_t gate, scale, fmt;
} tp_fp8g_glu_desc;

/*
 * tp_fp8g_glu_fwd: G = X Wg^T, U = X Wu^T, H = act(G) U
 *   X [N,P(H)], sX [P(H)/128,N]
 *   Wg, Wu [F,P(H)] in squares (the transposes of A [H,F], A_up)
 *   Z_save [N,2F]  bf16, row n = [G(n,:)|U(n,:)]; NULL where no backward follows
 *   H_act [N,F]    bf16, or NULL
 *   Hq [N,P(F)], sH [P(F)/128,N]        codes of H; both NULL: not made
 *   Hq_t [F,P(N)], sH_t [P(N)/128,F]    codes of H^T; likewise
 * Every output comes from the fp32 H (G, U); at least one of H_act, Hq, Hq_t is there.
 * workspace: tp_fp8g_glu_fwd_workspace(desc) bytes (at least 16), 16-byte
 * aligned, not shared with a call that may run at the same time (two graphs
 * replayed together, say); its contents do not matter before or after.
 */
size_t tp_fp8g_glu_fwd_workspace(const tp_fp8g_glu_desc *desc);
int tp_fp8g_glu_fwd(const tp_fp8g_glu_desc *desc, const void *X, const void *sX, const void *Wg,
                    const void *sWg, const void *Wu, const void *sWu, void *Z_save, void *H_act,
                    void *Hq, void *sH, void *Hq_t, void *sH_t, void *workspace, size_t ws_bytes,
                    void *stream);

/*
 * tp_fp8g_glu_bwd: dH = dY B^T, dG = dH U act'(G), dU = dH act(G)
 *   dY [N,P(H)], sdY [P(H)/128,N]
 *   B [F,P(H)] in squares (the block's down projection [F,H] in its own layout)
 *   Z_save [N,2F] bf16, of the forward
 *   dZ [N,2P(F)], sdZ [2P(F)/128,N]     codes of [dG|dU], each part's
 *       columns padded: parts 2 of tp_fp8g_gemm with K = P(F)
 *   dZ_t [2,F,P(N)], sdZ_t [2,P(N)/128,F]   codes of dG^T, then of dU^T
 * Either pair may be NULL.  workspace as above.
 */
size_t tp_fp8g_glu_bwd_workspace(const tp_fp8g_glu_desc *desc);
int tp_fp8g_glu_bwd(const tp_fp8g_glu_desc *desc, const void *dY, const void *sdY, const void *B,
                    const void *sB, const void *Z_save, void *dZ, void *sdZ, void *dZ_t,
                    void *sdZ_t, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* TPMLP_FP8G_H */
