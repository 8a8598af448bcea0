/*
 * sgemm_layers.h — C ABI of the operators of layers in 16 bits: products of
 * bfloat16 operands with bias, activation and a joined matrix in their
 * epilogue (dense, over groups of rows, over groups' rows as the shared
 * length), the gradient of that epilogue, and the root-mean-square norm with
 * its gradient.
 *
 * Pointers, streams, status codes, asynchrony, ownership and thread safety are
 * those of sgemm.h, types of matrices and the rows form of 8-bit values those
 * of sgemm_experts.h: all pointers are caller-owned device memory, a call
 * returns after enqueueing on `stream`, an error code means that nothing was
 * written, and sgemm_check_status() reports device-side timeouts. Calls may be
 * captured into a CUDA graph once one call has run on the device. No result
 * depends on the order in which threads run: the same inputs give the same
 * bits. sgemm_epilogue_backward() with a bias gradient and
 * sgemm_rms_norm_backward() with a weight gradient take scratch from the
 * library's pool. The first call on a device sets up these kernels and those of
 * sgemm_experts.h.
 *
 * Sizes go up to 2^31 - 1024; larger ones return SGEMM_ERR_OVERFLOW. Outputs
 * overlap neither inputs nor each other, except where a place is named below.
 * Float and bfloat16 matrices have any leading dimension and lie on any
 * multiple of their elements' size, except A and B of the products: these lie
 * on 16-byte boundaries, with leading dimensions (and strides between groups)
 * that are multiples of 8, which is what the product's copies need; values
 * between a row's last and its leading dimension are never read. Matrices
 * whose rows all begin on 16 bytes are fastest.
 */
#ifndef DENSE_FP32_MATRIX_07_GB300_SGEMM_LAYERS_H
#define DENSE_FP32_MATRIX_07_GB300_SGEMM_LAYERS_H

#include "sgemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* relu max(z, 0); gelu z Phi(z); gelu_tanh 0.5 z (1 + tanh(sqrt(2/pi) (z +
 * 0.044715 z^3))); silu z / (1 + exp(-z)). relu of a NaN is that NaN.
 *
 * Evaluated in FP32, from z in FP32, each is within this part of its value, in
 * units of 2^-24 (before it is rounded to its type): silu 8 + 2 |z|, gelu 32 +
 * 2 z^2, gelu_tanh 8 + 12 |z| + 0.5 |z|^3; values below |z| 2^-125 may be 0.
 * Slopes are within 8 more of the sum of their two terms' magnitudes (Phi + z phi;
 * s + z s (1 - s) x' for a sigmoid s of x). */
enum { SGEMM_ACT_NONE = 0, SGEMM_ACT_RELU = 1, SGEMM_ACT_GELU = 2, SGEMM_ACT_GELU_TANH = 3, SGEMM_ACT_SILU = 4 };
enum { SGEMM_JOIN_NONE = 0, SGEMM_JOIN_ADD = 1, SGEMM_JOIN_MUL = 2 };
enum { SGEMM_BF16_DENSE = 0, SGEMM_BF16_GROUPED = 1, SGEMM_BF16_GROUPED_K = 2 };

/*
 * sgemm_bf16 — C = act(op(A) . op(B) + bias), joined with D, on bfloat16 A, B.
 *
 *   op_a, A, lda    op_a = 0: A is M x K; 1: A is stored K x M.
 *   op_b, B, ldb    op_b = 0: B is K x N; 1: B is stored N x K (a layer's
 *                   weights, outputs by inputs).
 *   bias            N values, or NULL.
 *   act             SGEMM_ACT_*, of z = op(A) . op(B) + bias.
 *   pre, ld_pre     NULL, or M x N: z, for sgemm_epilogue_backward().
 *   join, D, ldd    SGEMM_JOIN_NONE (D is not read); _ADD: C = act(z) + D (a
 *                   residual, or C itself: D == C with ldd == ldc adds to C);
 *                   _MUL: C = act(z) * D (the other half of a gated layer).
 *   C, c_type, ldc  M x N of c_type, which is also that of pre and D.
 *
 * Products are summed in FP32 over all of K, the epilogue is FP32, and each
 * stored value is rounded once. The tensor cores cut sums off instead of
 * rounding them; they are added up over 768 of K at a time for a float C (where
 * all terms are positive, 1e-6 of a sum at most is lost at K = 768) and over
 * 8192 for a bfloat16 C (4e-5 on average). K == 0 is the empty sum. With x (M x
 * K) and w (N x K) of a layer: its output is op_a = 0, op_b = 1 of x, w; the
 * gradient of x is op_a = 0, op_b = 0 of dz (M x N), w; that of w is op_a = 1,
 * op_b = 0 of dz, x.
 */
int sgemm_bf16(int op_a, int op_b, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
               const float *bias, int act, void *pre, int64_t ld_pre, int join, const void *D, int64_t ldd,
               void *C, int c_type, int64_t ldc, cudaStream_t stream);

/*
 * sgemm_bf16_grouped — sgemm_bf16() of each group of rows of A (op_a = 0) with
 * its own B and bias.
 *
 *   groups, offsets up to 512 groups; offsets (groups + 1, ascending, in device
 *                   memory) as sgemm_dispatch() writes them: group g has rows
 *                   [offsets[g], offsets[g+1]) of A, C, pre and D. Groups may
 *                   be empty. Rows outside every group are not written.
 *   rows            rows of A and C; offsets are held to [0, rows].
 *   B, stride_b     group g's matrix at B + g * stride_b (elements).
 *   bias,           group g's N values at bias + g * stride_bias, or NULL.
 *   stride_bias
 */
int sgemm_bf16_grouped(int op_b, int64_t groups, const int32_t *offsets, int64_t rows, int64_t N, int64_t K,
                       const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b,
                       const float *bias, int64_t stride_bias, int act, void *pre, int64_t ld_pre,
                       int join, const void *D, int64_t ldd, void *C, int c_type, int64_t ldc, cudaStream_t stream);

/*
 * sgemm_bf16_grouped_k — C_g = A_g^T . B_g over the rows of each group: the
 * weight gradients of the experts (A = dz, rows x M; B = x, rows x N).
 *
 *   accumulate      1: C_g += instead.
 *   C, stride_c     group g's M x N matrix at C + g * stride_c (elements). An
 *                   empty group's is zeros (accumulate: as it was).
 */
int sgemm_bf16_grouped_k(int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N,
                         const void *A, int64_t lda, const void *B, int64_t ldb, int accumulate,
                         void *C, int c_type, int64_t ldc, int64_t stride_c, cudaStream_t stream);

/*
 * sgemm_bf16_plan — host-only view of the kernel that a product takes (needs no
 * GPU): mode SGEMM_BF16_DENSE (groups 1), _GROUPED (M = rows) or _GROUPED_K (K =
 * rows). out_cols: columns of the tile held in tensor memory's columns;
 * out_pair: 1 where two CTAs share a tile of 256 lanes (else 128); out_swap: 1
 * where the lanes hold columns of C; out_split: CTAs that share a tile's K;
 * out_grid: CTAs (0 for an empty C). Each may be NULL.
 */
int sgemm_bf16_plan(int mode, int64_t groups, int64_t M, int64_t N, int64_t K, int num_sms,
                    int *out_cols, int *out_pair, int *out_swap, int *out_split, int64_t *out_grid);

/*
 * sgemm_epilogue_backward — from grad_out, the gradient of C = act(z) (* D):
 *
 *   grad_pre = grad_out * act'(z) (* D)           NULL: not written
 *   grad_D   = grad_out * act(z)                  NULL: not written; SGEMM_JOIN_MUL only
 *   grad_bias[g][n] = sum over group g's rows of grad_pre (before it is rounded), FP32; NULL: not written
 *
 * (SGEMM_JOIN_ADD: the gradient of D is grad_out.) All matrices are rows x
 * cols of `type`. pre may be NULL where act is SGEMM_ACT_NONE and grad_D NULL;
 * D is read for SGEMM_JOIN_MUL only.
 *
 *   groups, offsets NULL offsets (groups = 1): one group of all rows. Else as
 *                   for sgemm_bf16_grouped(); rows outside every group are not
 *                   read or written.
 *   stride_gb       between groups' bias gradients, at least cols.
 *
 * The slope of relu at 0 is 0.
 */
int sgemm_epilogue_backward(int64_t rows, int64_t cols, int type, const void *grad_out, int64_t ld_go,
                            const void *pre, int64_t ld_pre, int act, int join, const void *D, int64_t ldd,
                            int64_t groups, const int32_t *offsets, void *grad_pre, int64_t ld_gp,
                            void *grad_D, int64_t ld_gd, float *grad_bias, int64_t stride_gb, cudaStream_t stream);

/*
 * sgemm_rms_norm — s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight,
 * per row; y also (or only) in 8 bits.
 *
 *   rows, cols      cols <= 16384.
 *   x, residual     rows x cols of `type`; residual may be NULL.
 *   weight          cols values, or NULL (ones).
 *   sum             NULL, or s (what sgemm_rms_norm_backward() takes).
 *   y               NULL, or y. sum or y may be x or residual themselves (the
 *                   same pointer and leading dimension).
 *   q, ldq,         NULL, or y in the rows form of sgemm_experts.h (before it
 *   scales, lds     is rounded to `type`): ldq >= cols, a multiple of 16, on
 *                   16 bytes; ceil(cols/128) x rows scales, lds >= rows.
 *
 * eps >= 0; a row of zeros with eps = 0 is NaN. Squares are summed in FP32: where
 * they pass its range (values of 2^64), y is 0, as beside an infinity.
 */
int sgemm_rms_norm(int64_t rows, int64_t cols, int type, const void *x, int64_t ldx, const void *residual, int64_t ld_res,
                   const float *weight, float eps, void *sum, int64_t ld_sum, void *y, int64_t ldy,
                   uint8_t *q, int64_t ldq, float *scales, int64_t lds, cudaStream_t stream);

/*
 * sgemm_rms_norm_backward — gradients of y with respect to s (= x + residual,
 * both of which have this gradient) and to the weight.
 *
 *   grad_y, s       rows x cols of `type`; s as sgemm_rms_norm() stored it.
 *   grad_sum        NULL, or the gradient that reaches s along the residual
 *                   stream, added to the result.
 *   grad_s          rows x cols; may be grad_y or grad_sum itself.
 *   grad_weight     NULL, or cols values.
 */
int sgemm_rms_norm_backward(int64_t rows, int64_t cols, int type, const void *grad_y, int64_t ld_gy,
                            const void *s, int64_t ld_s, const float *weight, float eps,
                            const void *grad_sum, int64_t ld_gsum, void *grad_s, int64_t ld_gs, float *grad_weight,
                            cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_FP32_MATRIX_07_GB300_SGEMM_LAYERS_H */
