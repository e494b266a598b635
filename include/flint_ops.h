/*
 * flint_ops.h - C ABI of the standalone operators around the Flint MoE layer (sm_100a): linear products
 * with the layer's two 4-bit weight formats at any width, products grouped by expert with 16-bit weights
 * and ragged sizes, the permutation and the combination around them, and the norms before and after a
 * block fused with its gate and residual scale.
 *
 * The conventions of flint_moe.h hold: device pointers owned by the caller, work enqueued on `stream` and
 * never waited for, nothing allocated, bad arguments refused before anything is launched. Every function
 * is stateless (no handle), so calls on different streams may overlap as long as they share no workspace,
 * and all of them can be captured into CUDA graphs. The current device must be the stream's. Leading dimensions (ld*)
 * count elements between rows. Outputs must not overlap inputs unless a function says so. Sums run in fp32 in a
 * fixed order: the same call gives the same bits. Results are rounded once, to the output's type.
 */
#ifndef FLINT_OPS_H
#define FLINT_OPS_H

#include "flint_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of activations */
#define FLINT_T_BF16 0
#define FLINT_T_F16 1
#define FLINT_T_F32 2 /* flint_block_norm only: the residual and the norm weights */

/* y[t][n] = sum_k W[n][k] x[t][k] for T tokens, W in one of the storage formats that flint_quantize_int4_g128
 * and flint_quantize_nvfp4 write (flint_quant.h):
 *   fmt FLINT_W_INT4_G128_FWHT128: codes u8 [N][K/2], scales bf16 [N][K/128], K a multiple of 128.
 *       rotated = 1: the codes store W blockdiag(Hn), and x is rotated here (Hn per 128-segment);
 *       rotated = 0: the codes store W itself.
 *   fmt FLINT_W_NVFP4: codes u8 [N][K/2], scales E4M3 [N][K/16], K a multiple of 16; rotated = 0.
 * tscale f32 [1] (device) multiplies the sum: required for NVFP4, optional (NULL = 1) for int4.
 * x [T][K] and y [T][N] are of `type` (BF16 or F16). codes and x are 16-byte aligned and ldx is a multiple of
 * 8; y, ldy need no alignment beyond their element's. K, T <= 65536, N <= 2^30, N * K <= 2^37. Made for few tokens
 * (T <= 64): larger T run in chunks that read the weights again. T = 0 is a no-op.
 * Rounding before the sums: rotated activations, per (token, 128-segment), to 16-bit fixed point of the segment's
 * largest value (T <= 8) or, scaled by a power of two, to fp16's 11 bits (T > 8, BF16) or 22 bits (T > 8, F16). Unrotated
 * ones, and the codes times NVFP4's block scales, enter exactly, but for activations below 2^-29 of their segment's largest.
 * A group scale times the segment's largest activation is formed in fp32 at 2^-18 of its size: between 2^-100 and 2^127 that
 * loses nothing.
 * workspace: flint_q4_linear_workspace_size(K, T) bytes of device memory (the activations as the kernel's operand),
 * 256-byte aligned, in use until the call's work is done; may be NULL when that size is 0, as it is for the smallest
 * calls. The size is 0 for invalid arguments too. */
size_t flint_q4_linear_workspace_size(int K, int T);
flint_status flint_q4_linear(int fmt, int N, int K, int rotated, const void* codes, const void* scales,
                             const float* tscale, const void* x, long long ldx, int T, int type, void* y, long long ldy,
                             void* workspace, size_t workspace_bytes, void* stream);

#define FLINT_ACT_NONE 0
#define FLINT_ACT_SWIGLU 1

/* Products grouped by expert, of 16-bit weights: row p of y for p in [offsets[e], offsets[e+1]) is
 *   y[p] = W[e] x[r(p)],  r(p) = row_of ? row_of[p] / row_div : p.
 * w [E][N][K], x [x_rows][K], y [P][N] of `type` (BF16 or F16). act FLINT_ACT_SWIGLU: N is even, rows 0..N/2-1
 * of W[e] are the gate and the rest the up projection, and y [P][N/2] = silu(gate) * up, formed in fp32.
 * offsets int32 [E+1] (device): ascending, offsets[0] = 0, offsets[E] <= P; values outside [0, P] are clamped,
 * a group that ends before it begins is empty. Rows of y at or behind offsets[E] are left as they were.
 * row_of int32 [P] (device) or NULL; with the permutation of flint_expert_permute or flint_moe_routing
 * (perm[p] = token * top_k + slot), row_div = top_k makes r(p) the token. r(p) outside [0, x_rows) is clamped.
 * 1 <= E <= 1024, K a multiple of 8, K <= 65536, E * N < 2^31, (N/64 + 1) E (P/64 + 1) < 2^31; w and x are 16-byte
 * aligned, ldx is a multiple of 8; y needs no alignment beyond its element's. P = 0 is a no-op. */
flint_status flint_grouped_linear(int E, int N, int K, int act, int type, const void* w, const void* x, long long ldx,
                                  int x_rows, const int* row_of, int row_div, const int* offsets, int P, void* y,
                                  long long ldy, void* stream);

/* Expert-major order of T * top_k (token, slot) pairs, as the layer's own permutation but for any E and with
 * dropped slots: ids int32 [T][top_k]; an id outside [0, E) (a padded token, say) belongs to no expert.
 *   offsets int32 [E+1]: exclusive prefix of the pairs per expert; offsets[E] = number of kept pairs
 *   perm int32 [T*top_k]: p in [offsets[e], offsets[e+1]) lists expert e's pairs t*top_k+k, ascending; -1 behind
 *   inv int32 [T][top_k]: the pair's position p, -1 for a dropped one
 * 1 <= E <= 1024, 1 <= top_k <= 64, T * top_k <= 2^22. With T = 0 only offsets is written (zeros). */
flint_status flint_expert_permute(const int* ids, int T, int top_k, int E, int* offsets, int* perm, int* inv,
                                  void* stream);

/* y[t] = scale * sum_k w[t][k] o[inv[t][k]] + addend[t]  (slot order; slots with inv outside [0, P) are skipped,
 * whatever their weight). o [P][H], addend [T][H] (NULL: none) and y [T][H] of `type` (BF16 or F16); inv int32,
 * w f32 [T][top_k]. addend may be y. 1 <= top_k <= 64, 1 <= H <= 2^23. T = 0 is a no-op. */
flint_status flint_expert_combine(const void* o, long long ldo, int P, const int* inv, const float* w, int T, int top_k,
                                  int H, float scale, const void* addend, long long lda, int type, void* y,
                                  long long ldy, void* stream);

#define FLINT_GATE_NONE 0    /* the gate's values as they are */
#define FLINT_GATE_SIGMOID 1 /* their sigmoid */

/* The residual step around a block with its norms: for each of T rows of H columns,
 *   b    = post_norm ? y / sqrt(mean(y^2) + eps) * post_weight : y
 *   x'   = res_scale * x + branch_scale * act(gate) * b           (x' = res_scale * x when y is NULL)
 *   z    = x' / sqrt(mean(x'^2) + eps) * pre_weight
 * (absent weights and gate count as 1; z is formed from x' before its rounding). flint_residual_rmsnorm is
 * this with no weights, gate or scales at H = 2048. */
typedef struct flint_norm_args {
  const void* x;           /* [T][H] of res_type */
  void* x_out;             /* x' [T][H] of res_type; may be x; NULL: x' is not stored */
  const void* y;           /* the branch [T][H] of type, or NULL */
  const void* gate;        /* of type, or NULL; ldg = 0: one row [H] for all tokens */
  const void* post_weight; /* [H] of w_type, or NULL */
  const void* pre_weight;  /* [H] of w_type, or NULL */
  void* z;                 /* [T][H] of type; NULL: not formed */
  long long ldx, ldxo, ldy, ldg, ldz;
  int T, H;                /* 1 <= H <= 32768 */
  int type;                /* FLINT_T_BF16 or FLINT_T_F16 */
  int res_type;            /* FLINT_T_F32 or type */
  int w_type;              /* FLINT_T_F32 or type */
  int post_norm;           /* 0 or 1 (needs y) */
  int gate_act;            /* FLINT_GATE_* */
  float res_scale, branch_scale, eps;
} flint_norm_args;

flint_status flint_block_norm(const flint_norm_args* args, void* stream);

/* Reads and clears the operators' error word of the current device: 0, or the timeout bit (4) when a bounded wait
 * inside a kernel of flint_q4_linear or flint_grouped_linear gave up since the last call (its output is then
 * incomplete). Waits for the device. */
flint_status flint_ops_error_word(unsigned* out);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_OPS_H */
