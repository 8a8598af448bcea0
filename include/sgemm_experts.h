/*
 * sgemm_experts.h — C ABI of the operators around products over experts:
 * routing, quantisation to 8 bits, block-scaled 8-bit products (dense and over
 * groups of rows), and the weighted sum of the experts' outputs.
 *
 * Pointers, streams, status codes, asynchrony, ownership and thread safety are
 * those of sgemm.h: all pointers are caller-owned device memory, a call
 * returns after enqueueing on `stream`, an error code means that nothing was
 * written, and sgemm_check_status() reports device-side timeouts. Calls may be
 * captured into a CUDA graph once one call has run on the device. No result
 * depends on the order in which threads run: the same inputs give the same
 * bits. Only sgemm_dispatch() takes scratch (from the library's pool).
 *
 * The first call of these on a device sets their kernels up, also where
 * products of sgemm.h have run; a failure of that fails no product there.
 *
 * Sizes go up to 2^31 - 1024 (sgemm_fp8_quantize_rows() and sgemm_combine():
 * 2^24 - 256 columns); larger ones return SGEMM_ERR_OVERFLOW.
 *
 * Types of matrices: SGEMM_F32 (float), SGEMM_BF16 (bfloat16). Row-major, any
 * leading dimension and any alignment of whole elements (an array that does not
 * lie on a multiple of its elements' size is refused), except the 8-bit ones:
 * q, A and B lie on 16-byte boundaries with leading dimensions (and batch
 * strides) that are multiples of 16, which is what the product's copies need;
 * the bytes between a row's last value and its leading dimension may be written
 * (after the last row's, those to the next multiple of 8, or of 16 in a
 * transposed form: no other matrix of the call may lie there) and are never
 * read as values.
 *
 * 8-bit values are e4m3 (largest 448) and share scales by blocks of 128:
 *   rows form     value (r, c) stands for q[r*ldq + c] * scales[(c/128)*lds + r]
 *                 (block-major, so that a product reads neighbouring rows'
 *                 scales together);
 *   blocks form   q[r*ldq + c] * scales[(r/128)*lds + c/128].
 * Of a block with largest magnitude m, a = max(m, 2^-96): scale = a / 448 and
 * q = e4m3(x * (448 / a)), rounded to nearest even. A block that holds a NaN
 * is NaN throughout; one that holds an infinity is NaN there and has an
 * infinite scale.
 */
#ifndef DENSE_FP32_MATRIX_07_GB300_SGEMM_EXPERTS_H
#define DENSE_FP32_MATRIX_07_GB300_SGEMM_EXPERTS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SGEMM_F32 = 0, SGEMM_BF16 = 1 };
enum { SGEMM_SCALE_BLOCKS = 0, SGEMM_SCALE_ROWS = 1 };
enum { SGEMM_SCORE_SOFTMAX = 0, SGEMM_SCORE_SIGMOID = 1 };
enum { SGEMM_FP8_DENSE = 0, SGEMM_FP8_GROUPED = 1, SGEMM_FP8_GROUPED_K = 2 };

/*
 * sgemm_fp8_quantize_rows — rows form of a rows x cols matrix.
 *
 *   src, type, ld   src_rows rows of cols values.
 *   gather          row r of q is row gather[r] of src; NULL: row r (then
 *                   src_rows >= rows). A row outside [0, src_rows) is zeros.
 *   q, ldq          rows x cols bytes, ldq >= cols.
 *   scales, lds     ceil(cols/128) x rows, lds >= rows.
 */
int sgemm_fp8_quantize_rows(int64_t rows, int64_t cols, const void *src, int type, int64_t ld,
                            const int32_t *gather, int64_t src_rows,
                            uint8_t *q, int64_t ldq, float *scales, int64_t lds, cudaStream_t stream);

/*
 * sgemm_fp8_quantize_cols — the transpose, scaled along the rows of src: what
 * a product that sums over them (a weight gradient) reads.
 *
 * The rows are in `groups` groups, group g holding rows [offsets[g],
 * offsets[g+1]) (device memory, ascending, groups <= 512); NULL offsets: one
 * group of all rows. Blocks do not cross groups: in q_t each group begins on
 * the next multiple of 128 columns, filled up with zeros.
 *
 *   padded          columns of q_t to write, a multiple of 128: groups past it
 *                   are cut off, and columns past the last group are zeros.
 *                   rows + 127 * min(rows, groups), rounded up, always holds
 *                   all; at least `rows` without offsets.
 *   q_t, ldq_t      cols x padded bytes.
 *   scales_t, lds_t padded/128 x cols: column c's block b at [b*lds_t + c].
 */
int sgemm_fp8_quantize_cols(int64_t rows, int64_t cols, const void *src, int type, int64_t ld,
                            const int32_t *gather, int64_t src_rows,
                            int64_t groups, const int32_t *offsets, int64_t padded,
                            uint8_t *q_t, int64_t ldq_t, float *scales_t, int64_t lds_t, cudaStream_t stream);

/*
 * sgemm_fp8_quantize_both — sgemm_fp8_quantize_rows() and _cols() of the same
 * matrix from one read of it. q may be NULL (the column form alone). Rows that
 * no group holds, or that `padded` cuts off, are not written in the row form.
 */
int sgemm_fp8_quantize_both(int64_t rows, int64_t cols, const void *src, int type, int64_t ld,
                            const int32_t *gather, int64_t src_rows,
                            int64_t groups, const int32_t *offsets, int64_t padded,
                            uint8_t *q, int64_t ldq, float *scales, int64_t lds,
                            uint8_t *q_t, int64_t ldq_t, float *scales_t, int64_t lds_t, cudaStream_t stream);

/*
 * sgemm_fp8_quantize_blocks — blocks form of `batch` rows x cols matrices, or
 * of their transposes (transpose = 1: q is cols x rows, scales
 * ceil(cols/128) x ceil(rows/128)), which the gradient of a product's input
 * reads. Strides in elements, ignored for batch == 1; stride_src may be 0.
 */
int sgemm_fp8_quantize_blocks(int64_t rows, int64_t cols, const void *src, int type, int64_t ld, int64_t stride_src,
                              int transpose, uint8_t *q, int64_t ldq, int64_t stride_q,
                              float *scales, int64_t lds, int64_t stride_s, int64_t batch, cudaStream_t stream);

/*
 * sgemm_fp8 — C = A . B^T + beta * C on 8-bit operands, K contiguous in both.
 *
 *   A, sa           M x K in rows form (ld_sa >= M).
 *   B, sb           N x K in b_form: SGEMM_SCALE_BLOCKS (weights; ld_sb >=
 *                   ceil(K/128)) or SGEMM_SCALE_ROWS (ld_sb >= N).
 *                   (ld_sa and ld_sb are ignored for scales of one row.)
 *   C, c_type, ldc  M x N. beta == 0: C is not read.
 *
 * Products within a block of 128 are summed on the tensor cores, the scaled
 * sums of the blocks in FP32. The two scales of a block and its sum are
 * multiplied in either order: where the product of any two of the three leaves
 * FP32's range (values near 2^113 and above, or scales whose product is below
 * 2^-126), the result may be infinite, NaN or short of digits, though the
 * whole product would not be. K == 0 is the empty sum. With x the input
 * (M x K) and w the weights (N x K) of a layer: its output is A = x (rows), B =
 * w (blocks); the gradient of x is A = the output's gradient (rows), B = w
 * transposed (blocks, transpose = 1); the gradient of w is A = the output's
 * gradient and B = x, both by sgemm_fp8_quantize_cols(), SGEMM_SCALE_ROWS.
 */
int sgemm_fp8(int b_form, int64_t M, int64_t N, int64_t K,
              const uint8_t *A, int64_t lda, const float *sa, int64_t ld_sa,
              const uint8_t *B, int64_t ldb, const float *sb, int64_t ld_sb,
              float beta, void *C, int c_type, int64_t ldc, cudaStream_t stream);

/*
 * sgemm_fp8_grouped — sgemm_fp8() of each group of rows of A with its own B:
 * rows [offsets[g], offsets[g+1]) of C = those of A . B_g^T (+ beta * C).
 *
 *   groups, offsets up to 512 groups; offsets (groups + 1, ascending, in device
 *                   memory) as sgemm_dispatch() writes them. Groups may be
 *                   empty. Rows outside every group are not written.
 *   rows            rows of A and C; offsets are held to [0, rows].
 *   B, stride_b     group g's N x K matrix at B + g * stride_b, blocks form,
 *                   its scales at sb + g * stride_sb.
 */
int sgemm_fp8_grouped(int64_t groups, const int32_t *offsets, int64_t rows, int64_t N, int64_t K,
                      const uint8_t *A, int64_t lda, const float *sa, int64_t ld_sa,
                      const uint8_t *B, int64_t ldb, int64_t stride_b,
                      const float *sb, int64_t ld_sb, int64_t stride_sb,
                      float beta, void *C, int c_type, int64_t ldc, cudaStream_t stream);

/*
 * sgemm_fp8_grouped_k — one product per group over that group's rows:
 * C_g = A_g . B_g^T (+ beta * C_g), the weight gradients of the experts.
 *
 *   A, B            M x padded and N x padded, as sgemm_fp8_quantize_cols()
 *                   writes them with the same offsets and padded.
 *   C, stride_c     group g's M x N matrix at C + g * stride_c (elements). An
 *                   empty group's is beta * C_g.
 */
int sgemm_fp8_grouped_k(int64_t groups, const int32_t *offsets, int64_t padded, int64_t M, int64_t N,
                        const uint8_t *A, int64_t lda, const float *sa, int64_t ld_sa,
                        const uint8_t *B, int64_t ldb, const float *sb, int64_t ld_sb,
                        float beta, void *C, int c_type, int64_t ldc, int64_t stride_c, cudaStream_t stream);

/*
 * sgemm_fp8_plan — host-only view of the kernel that a product takes (needs no
 * GPU): mode SGEMM_FP8_DENSE (groups 1), _GROUPED (M = rows) or _GROUPED_K (K =
 * padded). out_cols: columns of the tile held in tensor memory's columns;
 * out_swap: 1 where those are rows of A (its 128 lanes then rows of B), 0 where
 * they are rows of B; out_split: CTAs that share a tile's K blocks; out_grid:
 * CTAs (0 for an empty C). Each may be NULL.
 */
int sgemm_fp8_plan(int mode, int64_t groups, int64_t M, int64_t N, int64_t K, int num_sms,
                   int *out_cols, int *out_swap, int *out_split, int64_t *out_grid);

/*
 * sgemm_route — the experts of each token and their weights.
 *
 *   logits          T x E (E <= 1024). An expert whose logit is -infinity or
 *                   NaN is not chosen.
 *   bias            NULL, or E values added to the scores for the choice only.
 *   score           SGEMM_SCORE_SOFTMAX or SGEMM_SCORE_SIGMOID of the logits.
 *   groups, kept,   the E experts are `groups` (<= 32) runs of equal length, of
 *   two             which `kept` stay: those whose best key (two = 0) or whose
 *                   two best keys' sum (two = 1; a group with fewer eligible
 *                   comes last) is largest. groups = kept = 1: no such step.
 *   k               experts per token, 1 .. min(32, E): the largest keys in
 *                   falling order, ties to the lowest expert.
 *   renorm, scale   weights = scale * score, with renorm = 1 divided by the
 *                   sum of the chosen scores.
 *   weights,        T x k. A slot without an eligible expert: weight 0,
 *   indices         index -1.
 *
 * The key is score + bias where a bias is given or two = 1, else the logit
 * (in both cases the order of the scores).
 */
int sgemm_route(int64_t T, int64_t E, const void *logits, int type, int64_t ld, const float *bias, int score,
                int groups, int kept, int two, int k, int renorm, float scale,
                float *weights, int32_t *indices, cudaStream_t stream);

/*
 * sgemm_route_backward — gradient of sgemm_route()'s weights (grad_w, T x k)
 * with respect to the logits (grad_logits, T x E, of the logits' type, written
 * whole); the choice of experts has none. Slots of index -1 are skipped.
 */
int sgemm_route_backward(int64_t T, int64_t E, const void *logits, int type, int64_t ld, int score, int k,
                         int renorm, float scale, const int32_t *indices, const float *grad_w,
                         void *grad_logits, int64_t ld_g, cudaStream_t stream);

/*
 * sgemm_dispatch — sorts the T * k (token, slot) pairs by expert, pairs of one
 * expert by token and slot.
 *
 *   indices         T x k; outside [0, E): the pair has no row.
 *   offsets         E + 1: expert e has rows [offsets[e], offsets[e+1]).
 *   row_of          T x k: the pair's row, or -1.
 *   token_of        T * k: the token of each row, -1 past offsets[E]. It is
 *                   the `gather` of the quantisers.
 */
int sgemm_dispatch(int64_t T, int k, int64_t E, const int32_t *indices,
                   int32_t *offsets, int32_t *row_of, int32_t *token_of, cudaStream_t stream);

/*
 * sgemm_combine — out[t] = sum_j weights[t, j] * Y[row_of[t, j]], j < k <= 32.
 *
 * Y is rows x cols; a row outside [0, rows) adds nothing. weights NULL: ones
 * (the gradient of gathering by token_of). Sums are in FP32, in slot order.
 */
int sgemm_combine(int64_t T, int k, int64_t cols, int64_t rows, const void *Y, int type, int64_t ldy,
                  const int32_t *row_of, const float *weights, void *out, int64_t ld_out, cudaStream_t stream);

/*
 * sgemm_combine_backward — from grad_out (T x cols):
 * grad_y[row_of[t, j]] = weights[t, j] * grad_out[t] and
 * grad_w[t, j] = <grad_out[t], Y[row_of[t, j]]> (0 without a row).
 *
 * Either of grad_y and grad_w may be NULL; Y is read for grad_w only. No two
 * pairs may name the same row. Rows of grad_y that no pair names are not
 * written.
 */
int sgemm_combine_backward(int64_t T, int k, int64_t cols, int64_t rows, const void *grad_out, int type,
                           int64_t ld_go, const void *Y, int64_t ldy, const int32_t *row_of, const float *weights,
                           void *grad_y, int64_t ld_gy, float *grad_w, cudaStream_t stream);

/*
 * sgemm_test_fail_next_setups — test hook: the next n times that a call above
 * would set its kernels up on a device (the first call there does) count as
 * failed: it returns SGEMM_ERR_CUDA with nothing enqueued, and a later call
 * tries again. The products of sgemm.h do not set these kernels up. n = 0
 * clears a pending count. Returns SGEMM_OK, or SGEMM_ERR_INVALID_VALUE for
 * n < 0. Host only; needs no GPU.
 */
int sgemm_test_fail_next_setups(int n);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_FP32_MATRIX_07_GB300_SGEMM_EXPERTS_H */
