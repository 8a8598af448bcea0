// C entries of include/sgemm_layers.h: argument checks, scratch, dispatch.
#include "../../include/sgemm_layers.h"
#include "checks.cuh"
#include "layers.cuh"

#include <cmath>

using namespace sgemm_gb300;

namespace {

bool bad_act(int act) { return act < SGEMM_ACT_NONE || act > SGEMM_ACT_SILU; }
bool bad_join(int join) { return join < SGEMM_JOIN_NONE || join > SGEMM_JOIN_MUL; }

// The products' operands: 16-byte rows on a 16-byte base.
bool bad_bf16(const void *p, int64_t ld, int64_t cols) { return !p || !aligned(p, 16) || ld < cols || ld % 8 != 0; }

// An input that is the output itself, element for element, is not an overlap.
Region unless_same(const void *in, int64_t ld, const void *out, int64_t ld_out, int64_t bytes, int64_t size)
{
    return Region{in, in == out && ld == ld_out ? 0 : bytes, size};
}

int run_product(Bf16Args &g, cudaStream_t stream)
{
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != SGEMM_OK) return rc;
    g.status = dev.status;
    g.num_sms = dev.num_sms;
    return launched(launch_bf16(g, stream));
}

// A call's scratch, from the library's pool, given back on the stream.
class Scratch {
public:
    Scratch(size_t bytes, const DeviceInfo &dev, cudaStream_t stream) : stream_(stream)
    {
        if (bytes == 0) return;
        if (take_alloc_failure() || cudaMallocFromPoolAsync(&p_, bytes, dev.pool, stream) != cudaSuccess) {
            cudaGetLastError();
            failed_ = true;
        }
    }
    ~Scratch()
    {
        if (p_ && !failed_) cudaFreeAsync(p_, stream_);
    }
    Scratch(const Scratch &) = delete;
    Scratch &operator=(const Scratch &) = delete;
    void *get() const { return p_; }
    bool failed() const { return failed_; }

private:
    void *p_ = nullptr;
    cudaStream_t stream_;
    bool failed_ = false;
};

// Where C, pre and D lie, and what they must not meet.
int check_epilogue(const Bf16Args &g, const Region &a, const Region &b, const Region &offsets)
{
    const int64_t size = g.c_bf16 ? 2 : 4, bytes = span(g.M, g.N, g.ldc, size);
    const bool joins = g.join != SGEMM_JOIN_NONE;
    const Region out[] = {{g.C, bytes, size}, {g.pre, g.pre ? span(g.M, g.N, g.ld_pre, size) : 0, size}};
    const int64_t d_bytes = joins ? span(g.M, g.N, g.ldd, size) : 0;
    const Region in[] = {a,
                         b,
                         offsets,
                         {g.bias, g.bias ? span(g.groups, g.N, g.stride_bias, 4) : 0},
                         unless_same(g.D, g.ldd, g.C, g.ldc, d_bytes, size)};
    const int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    // D in C's place still keeps clear of pre; its own extent is C's.
    if (d_bytes < 0) return SGEMM_ERR_OVERFLOW;
    return SGEMM_OK;
}

bool bad_epilogue(int act, int join, const void *pre, int64_t ld_pre, const void *D, int64_t ldd, const void *C, int64_t ldc,
                  int64_t N)
{
    return bad_act(act) || bad_join(join) || !C || ldc < N || (pre && ld_pre < N) ||
           (join != SGEMM_JOIN_NONE && (!D || ldd < N));
}

}  // namespace

extern "C" {

int sgemm_bf16(int op_a, int op_b, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
               const float *bias, int act, void *pre, int64_t ld_pre, int join, const void *D, int64_t ldd, void *C,
               int c_type, int64_t ldc, cudaStream_t stream)
{
    if (bad_size(M) || bad_size(N) || bad_size(K) || !type_size(c_type)) return SGEMM_ERR_INVALID_VALUE;
    if ((op_a != 0 && op_a != 1) || (op_b != 0 && op_b != 1) || bad_act(act) || bad_join(join))
        return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (bad_epilogue(act, join, pre, ld_pre, D, ldd, C, ldc, N)) return SGEMM_ERR_INVALID_VALUE;
    const int64_t a_rows = op_a ? K : M, a_cols = op_a ? M : K, b_rows = op_b ? N : K, b_cols = op_b ? K : N;
    if (K > 0 && (bad_bf16(A, lda, a_cols) || bad_bf16(B, ldb, b_cols))) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    Bf16Args g{};
    g.mode = kBf16Dense;
    g.op_a = op_a, g.op_b = op_b;
    g.M = M, g.N = N, g.K = K;
    g.A = A, g.lda = lda, g.B = B, g.ldb = ldb;
    g.groups = 1;
    g.bias = bias, g.act = act, g.join = join;
    g.pre = pre, g.ld_pre = ld_pre, g.D = D, g.ldd = ldd;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc;
    const int rc = check_epilogue(g, {A, span(a_rows, a_cols, lda, 2), 2}, {B, span(b_rows, b_cols, ldb, 2), 2},
                                  {nullptr, 0, 4});
    if (rc != SGEMM_OK) return rc;
    return run_product(g, stream);
}

int sgemm_bf16_grouped(int op_b, int64_t groups, const int32_t *offsets, int64_t rows, int64_t N, int64_t K, const void *A,
                       int64_t lda, const void *B, int64_t ldb, int64_t stride_b, const float *bias, int64_t stride_bias,
                       int act, void *pre, int64_t ld_pre, int join, const void *D, int64_t ldd, void *C, int c_type,
                       int64_t ldc, cudaStream_t stream)
{
    if (groups < 0 || groups > kMaxGroups || bad_size(rows) || bad_size(N) || bad_size(K) || !type_size(c_type) ||
        (op_b != 0 && op_b != 1) || bad_act(act) || bad_join(join))
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || rows == 0 || N == 0) return SGEMM_OK;
    if (!offsets || stride_b < 0 || bad_epilogue(act, join, pre, ld_pre, D, ldd, C, ldc, N)) return SGEMM_ERR_INVALID_VALUE;
    if (bias && (stride_bias < 0 || (groups > 1 && stride_bias < N))) return SGEMM_ERR_INVALID_VALUE;
    const int64_t b_rows = op_b ? N : K, b_cols = op_b ? K : N;
    if (K > 0 && (bad_bf16(A, lda, K) || bad_bf16(B, ldb, b_cols))) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    const int64_t b_one = span(b_rows, b_cols, ldb, 2);
    if (b_one < 0) return SGEMM_ERR_OVERFLOW;
    if (K > 0 && groups > 1 && (stride_b < b_one / 2 || stride_b % 8 != 0)) return SGEMM_ERR_INVALID_VALUE;
    Bf16Args g{};
    g.mode = kBf16GroupRows;
    g.op_b = op_b;
    g.M = rows, g.N = N, g.K = K;
    g.A = A, g.lda = lda, g.B = B, g.ldb = ldb, g.stride_b = stride_b;
    g.groups = (int)groups;
    g.offsets = offsets;
    g.bias = bias, g.stride_bias = groups > 1 ? stride_bias : 0, g.act = act, g.join = join;
    g.pre = pre, g.ld_pre = ld_pre, g.D = D, g.ldd = ldd;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc;
    const int rc = check_epilogue(g, {A, span(rows, K, lda, 2), 2}, {B, span(b_rows, b_cols, ldb, 2, groups, stride_b), 2},
                                  {offsets, (groups + 1) * 4, 4});
    if (rc != SGEMM_OK) return rc;
    return run_product(g, stream);
}

int sgemm_bf16_grouped_k(int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, const void *A,
                         int64_t lda, const void *B, int64_t ldb, int accumulate, void *C, int c_type, int64_t ldc,
                         int64_t stride_c, cudaStream_t stream)
{
    if (groups < 0 || groups > kMaxGroups || bad_size(rows) || bad_size(M) || bad_size(N) || !type_size(c_type) ||
        (accumulate != 0 && accumulate != 1) || stride_c < 0)
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || M == 0 || N == 0) return SGEMM_OK;
    if (!offsets || !C || ldc < N) return SGEMM_ERR_INVALID_VALUE;
    if (rows > 0 && (bad_bf16(A, lda, M) || bad_bf16(B, ldb, N))) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(rows)) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(c_type), c_one = span(M, N, ldc, size);
    if (c_one < 0) return SGEMM_ERR_OVERFLOW;
    if (groups > 1 && stride_c < c_one / size) return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{C, span(M, N, ldc, size, groups, stride_c), size}};
    const Region in[] = {{A, span(rows, M, lda, 2), 2}, {B, span(rows, N, ldb, 2), 2}, {offsets, (groups + 1) * 4}};
    const int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    Bf16Args g{};
    g.mode = kBf16GroupK;
    g.op_a = 1, g.op_b = 0;
    g.M = M, g.N = N, g.K = rows;
    g.A = A, g.lda = lda, g.B = B, g.ldb = ldb;
    g.groups = (int)groups;
    g.offsets = offsets;
    g.join = accumulate ? kJoinAdd : kJoinNone;
    g.D = C, g.ldd = ldc;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc, g.stride_c = groups > 1 ? stride_c : 0;
    return run_product(g, stream);
}

int sgemm_bf16_plan(int mode, int64_t groups, int64_t M, int64_t N, int64_t K, int num_sms, int *out_cols, int *out_pair,
                    int *out_swap, int *out_split, int64_t *out_grid)
{
    if (mode < SGEMM_BF16_DENSE || mode > SGEMM_BF16_GROUPED_K || bad_size(M) || bad_size(N) || bad_size(K) ||
        num_sms <= 0 || groups < 1 || groups > kMaxGroups || (mode == SGEMM_BF16_DENSE && groups != 1))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    Bf16Plan p{0, false, false, 0, 0};
    if (M > 0 && N > 0) {
        Bf16Args g{};
        g.mode = mode;
        g.M = M, g.N = N, g.K = K;
        g.groups = (int)groups;
        g.num_sms = num_sms;
        p = plan_bf16(g);
    }
    if (out_cols) *out_cols = p.cols;
    if (out_pair) *out_pair = p.pair ? 1 : 0;
    if (out_swap) *out_swap = p.swap ? 1 : 0;
    if (out_split) *out_split = p.split;
    if (out_grid) *out_grid = p.grid;
    return SGEMM_OK;
}

int sgemm_epilogue_backward(int64_t rows, int64_t cols, int type, const void *grad_out, int64_t ld_go, const void *pre,
                            int64_t ld_pre, int act, int join, const void *D, int64_t ldd, int64_t groups,
                            const int32_t *offsets, void *grad_pre, int64_t ld_gp, void *grad_D, int64_t ld_gd,
                            float *grad_bias, int64_t stride_gb, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || !type_size(type) || bad_act(act) || bad_join(join) || groups < 0 ||
        groups > kMaxGroups || (!offsets && groups != 1) || (grad_D && join != SGEMM_JOIN_MUL))
        return SGEMM_ERR_INVALID_VALUE;
    if (cols == 0 || groups == 0 || (!grad_pre && !grad_D && !grad_bias)) return SGEMM_OK;
    if (rows == 0 && !grad_bias) return SGEMM_OK;
    const bool reads_z = act != SGEMM_ACT_NONE || grad_D, reads_d = join == SGEMM_JOIN_MUL;
    if (rows > 0 && (!grad_out || ld_go < cols || (reads_z && (!pre || ld_pre < cols)) || (reads_d && (!D || ldd < cols)) ||
                     (grad_pre && ld_gp < cols) || (grad_D && ld_gd < cols)))
        return SGEMM_ERR_INVALID_VALUE;
    if (grad_bias && (stride_gb < 0 || (groups > 1 && stride_gb < cols))) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || too_large(cols)) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(type);
    const Region out[] = {{grad_pre, grad_pre ? span(rows, cols, ld_gp, size) : 0, size},
                          {grad_D, grad_D ? span(rows, cols, ld_gd, size) : 0, size},
                          {grad_bias, grad_bias ? span(groups, cols, stride_gb, 4) : 0}};
    const Region in[] = {{grad_out, span(rows, cols, ld_go, size), size},
                         {pre, reads_z ? span(rows, cols, ld_pre, size) : 0, size},
                         {D, reads_d ? span(rows, cols, ldd, size) : 0, size},
                         {offsets, offsets ? (groups + 1) * 4 : 0}};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    EpilogueBackwardArgs g{};
    g.rows = rows, g.cols = cols, g.bf16 = type == SGEMM_BF16;
    g.grad_out = grad_out, g.ld_go = ld_go, g.pre = pre, g.ld_pre = ld_pre;
    g.act = act, g.join = join, g.D = D, g.ldd = ldd;
    g.groups = (int)groups, g.offsets = offsets;
    g.grad_pre = grad_pre, g.ld_gp = ld_gp, g.grad_D = grad_D, g.ld_gd = ld_gd;
    g.grad_bias = grad_bias, g.stride_gb = groups > 1 ? stride_gb : 0;
    g.num_sms = dev.num_sms;
    const Scratch scratch(epilogue_backward_scratch_bytes(g), dev, stream);
    if (scratch.failed()) return SGEMM_ERR_ALLOC;
    return launched(launch_epilogue_backward(g, scratch.get(), stream));
}

int sgemm_rms_norm(int64_t rows, int64_t cols, int type, const void *x, int64_t ldx, const void *residual, int64_t ld_res,
                   const float *weight, float eps, void *sum, int64_t ld_sum, void *y, int64_t ldy, uint8_t *q, int64_t ldq,
                   float *scales, int64_t lds, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || !type_size(type) || !(eps >= 0.0f) || std::isinf(eps)) return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0 || (!sum && !y && !q)) return SGEMM_OK;
    if (!x || ldx < cols || (residual && ld_res < cols) || (sum && ld_sum < cols) || (y && ldy < cols))
        return SGEMM_ERR_INVALID_VALUE;
    if (q && (bad_fp8(q, ldq, cols) || !scales || lds < rows)) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || cols > kMaxNormCols) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(type);
    const Region o_sum{sum, sum ? span(rows, cols, ld_sum, size) : 0, size};
    const Region o_y{y, y ? span(rows, cols, ldy, size) : 0, size};
    const Region i_x{x, span(rows, cols, ldx, size), size};
    const Region i_res{residual, residual ? span(rows, cols, ld_res, size) : 0, size};
    const Region out[] = {o_sum, o_y, {q, q ? span_fp8(rows, cols, ldq, 8) : 0}, {scales, q ? span(ceil_div(cols, kBlock), rows, lds, 4) : 0}};
    const Region w[] = {{weight, weight ? cols * 4 : 0}};
    int rc = check_regions(out, w);
    if (rc != SGEMM_OK) return rc;
    // x and residual against each output that is not in their place.
    const Region sums[] = {o_sum}, ys[] = {o_y}, rest[] = {out[2], out[3]}, both[] = {i_x, i_res};
    const Region for_sum[] = {unless_same(x, ldx, sum, ld_sum, i_x.bytes, size),
                              unless_same(residual, ld_res, sum, ld_sum, i_res.bytes, size)};
    const Region for_y[] = {unless_same(x, ldx, y, ldy, i_x.bytes, size),
                            unless_same(residual, ld_res, y, ldy, i_res.bytes, size)};
    if ((rc = check_regions(sums, for_sum)) != SGEMM_OK || (rc = check_regions(ys, for_y)) != SGEMM_OK ||
        (rc = check_regions(rest, both)) != SGEMM_OK)
        return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    RmsNormArgs g{};
    g.rows = rows, g.cols = cols, g.bf16 = type == SGEMM_BF16;
    g.x = x, g.ldx = ldx, g.residual = residual, g.ld_res = ld_res;
    g.weight = weight, g.eps = eps;
    g.sum = sum, g.ld_sum = ld_sum, g.y = y, g.ldy = ldy;
    g.q = q, g.ldq = ldq, g.scales = scales, g.lds = lds;
    return launched(launch_rms_norm(g, stream));
}

int sgemm_rms_norm_backward(int64_t rows, int64_t cols, int type, const void *grad_y, int64_t ld_gy, const void *s,
                            int64_t ld_s, const float *weight, float eps, const void *grad_sum, int64_t ld_gsum,
                            void *grad_s, int64_t ld_gs, float *grad_weight, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || !type_size(type) || !(eps >= 0.0f) || std::isinf(eps)) return SGEMM_ERR_INVALID_VALUE;
    if (cols == 0 || (rows == 0 && !grad_weight)) return SGEMM_OK;
    if (rows > 0 && (!grad_y || ld_gy < cols || !s || ld_s < cols || !grad_s || ld_gs < cols || (grad_sum && ld_gsum < cols)))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || cols > kMaxNormCols) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(type);
    const Region g_y{grad_y, span(rows, cols, ld_gy, size), size};
    const Region g_sum{grad_sum, grad_sum ? span(rows, cols, ld_gsum, size) : 0, size};
    const Region out[] = {{grad_s, span(rows, cols, ld_gs, size), size}, {grad_weight, grad_weight ? cols * 4 : 0}};
    const Region in[] = {{s, span(rows, cols, ld_s, size), size},
                         {weight, weight ? cols * 4 : 0},
                         unless_same(grad_y, ld_gy, grad_s, ld_gs, g_y.bytes, size),
                         unless_same(grad_sum, ld_gsum, grad_s, ld_gs, g_sum.bytes, size)};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    RmsNormBackwardArgs g{};
    g.rows = rows, g.cols = cols, g.bf16 = type == SGEMM_BF16;
    g.grad_y = grad_y, g.ld_gy = ld_gy, g.x = s, g.ldx = ld_s;
    g.weight = weight, g.eps = eps;
    g.grad_sum = grad_sum, g.ld_gs = ld_gsum;
    g.grad_x = grad_s, g.ld_gx = ld_gs, g.grad_weight = grad_weight;
    g.num_sms = dev.num_sms;
    const Scratch scratch(rms_norm_backward_scratch_bytes(g), dev, stream);
    if (scratch.failed()) return SGEMM_ERR_ALLOC;
    return launched(launch_rms_norm_backward(g, scratch.get(), stream));
}

}  // extern "C"
