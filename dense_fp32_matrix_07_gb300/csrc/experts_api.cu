// C entries of include/sgemm_experts.h: argument checks, scratch, dispatch.
#include "../../include/sgemm_experts.h"
#include "experts.cuh"

#include <climits>

using namespace sgemm_gb300;

namespace {

// Largest row, column or token count: tile arithmetic stays below 2^31.
constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1024;
// Most columns of a row quantised by sgemm_fp8_quantize_rows() or summed by
// sgemm_combine(): a grid has 65535 blocks of 256 along its second dimension.
constexpr int64_t kMaxCols = 65535 * 256;

bool bad_size(int64_t n) { return n < 0; }
bool too_large(int64_t n) { return n > kMaxSize; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t type_size(int type) { return type == SGEMM_F32 ? 4 : type == SGEMM_BF16 ? 2 : 0; }
bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Bytes from the first to past the last element of `batch` matrices, -1 if
// they would not fit 63 bits.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t size, int64_t batch = 1, int64_t stride = 0)
{
    if (rows <= 0 || cols <= 0 || batch <= 0) return 0;
    const __int128 e = ((__int128)(batch - 1) * stride + (__int128)(rows - 1) * ld + cols) * size;
    return e > (__int128)INT64_MAX ? -1 : (int64_t)e;
}

// The same of an 8-bit output: the quantisers store `piece` bytes of a row at a
// time, the last row's padding with its last values (rows start on 16 bytes).
int64_t span_fp8(int64_t rows, int64_t cols, int64_t ld, int64_t piece, int64_t batch = 1, int64_t stride = 0)
{
    return span(rows, ceil_div(cols, piece) * piece, ld, 1, batch, stride);
}

// An array of a call: where it lies, its extent, and the size of its elements.
struct Region {
    const void *p;
    int64_t bytes, size;
    template <class T>
    Region(const T *p, int64_t bytes) : Region(p, bytes, sizeof(T)) {}
    Region(const void *p, int64_t bytes, int64_t size) : p(p), bytes(bytes), size(size) {}
};

bool overlap(const Region &a, const Region &b)
{
    if (a.bytes <= 0 || b.bytes <= 0 || !a.p || !b.p) return false;
    const __int128 a0 = (__int128)reinterpret_cast<uintptr_t>(a.p), b0 = (__int128)reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// SGEMM_OK, or why a call must not run: a region that overflows, elements that
// do not lie on multiples of their size, an output that overlaps an input or
// another output.
template <int NOUT, int NIN>
int check_regions(const Region (&out)[NOUT], const Region (&in)[NIN])
{
    for (const Region &o : out)
        if (o.bytes < 0) return SGEMM_ERR_OVERFLOW;
    for (const Region &i : in)
        if (i.bytes < 0) return SGEMM_ERR_OVERFLOW;
    auto between = [](const Region &r) { return r.bytes > 0 && !aligned(r.p, (uintptr_t)r.size); };
    for (const Region &o : out)
        if (between(o)) return SGEMM_ERR_INVALID_VALUE;
    for (const Region &i : in)
        if (between(i)) return SGEMM_ERR_INVALID_VALUE;
    for (int a = 0; a < NOUT; ++a) {
        for (int b = 0; b < a; ++b)
            if (overlap(out[a], out[b])) return SGEMM_ERR_INVALID_VALUE;
        for (const Region &i : in)
            if (overlap(out[a], i)) return SGEMM_ERR_INVALID_VALUE;
    }
    return SGEMM_OK;
}

// The product's operands in 8 bits: 16-byte rows on a 16-byte base.
bool bad_fp8(const void *p, int64_t ld, int64_t cols) { return !p || !aligned(p, 16) || ld < cols || ld % 16 != 0; }

// The product's scales: the leading dimension of a single row is not used.
bool bad_scales(const float *p, int64_t ld, int64_t rows, int64_t cols) { return !p || (rows > 1 && ld < cols); }

int launched(cudaError_t e)
{
    if (e == cudaSuccess) return SGEMM_OK;
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
}

int run_product(Fp8Args &g, cudaStream_t stream)
{
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != SGEMM_OK) return rc;
    g.status = dev.status;
    g.num_sms = dev.num_sms;
    return launched(launch_fp8(g, stream));
}

}  // namespace

extern "C" {

int sgemm_fp8_quantize_rows(int64_t rows, int64_t cols, const void *src, int type, int64_t ld, const int32_t *gather,
                            int64_t src_rows, uint8_t *q, int64_t ldq, float *scales, int64_t lds, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || bad_size(src_rows) || !type_size(type)) return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) return SGEMM_OK;
    if (ld < cols || lds < rows || !scales || bad_fp8(q, ldq, cols)) return SGEMM_ERR_INVALID_VALUE;
    if (!gather && src_rows < rows) return SGEMM_ERR_INVALID_VALUE;
    if (!src && src_rows > 0) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || cols > kMaxCols || too_large(src_rows)) return SGEMM_ERR_OVERFLOW;
    const Region out[] = {{q, span_fp8(rows, cols, ldq, 8)}, {scales, span(ceil_div(cols, kBlock), rows, lds, 4)}};
    const Region in[] = {{src, span(src_rows, cols, ld, type_size(type)), type_size(type)}, {gather, gather ? rows * 4 : 0}};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    return launched(launch_quantize_rows(rows, cols, src, type == SGEMM_BF16, ld, gather, src_rows, q, ldq, scales, lds,
                                         stream));
}

int sgemm_fp8_quantize_both(int64_t rows, int64_t cols, const void *src, int type, int64_t ld, const int32_t *gather,
                            int64_t src_rows, int64_t groups, const int32_t *offsets, int64_t padded, uint8_t *q,
                            int64_t ldq, float *scales, int64_t lds, uint8_t *q_t, int64_t ldq_t, float *scales_t,
                            int64_t lds_t, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || bad_size(src_rows) || bad_size(padded) || padded % kBlock || !type_size(type))
        return SGEMM_ERR_INVALID_VALUE;
    if (offsets ? (groups < 1 || groups > kMaxGroups) : padded < rows) return SGEMM_ERR_INVALID_VALUE;
    if (cols == 0 || padded == 0) return SGEMM_OK;
    if (bad_fp8(q_t, ldq_t, padded) || !scales_t || lds_t < cols) return SGEMM_ERR_INVALID_VALUE;
    if (q && rows > 0 && (bad_fp8(q, ldq, cols) || !scales || lds < rows)) return SGEMM_ERR_INVALID_VALUE;
    if (ld < cols || (!gather && src_rows < rows) || (!src && src_rows > 0)) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || too_large(cols) || too_large(src_rows) || too_large(padded)) return SGEMM_ERR_OVERFLOW;
    const Region out[] = {{q_t, span(cols, padded, ldq_t, 1)},
                          {scales_t, span(padded / kBlock, cols, lds_t, 4)},
                          {q, q ? span_fp8(rows, cols, ldq, 8) : 0},
                          {scales, q ? span(ceil_div(cols, kBlock), rows, lds, 4) : 0}};
    const Region in[] = {{src, span(src_rows, cols, ld, type_size(type)), type_size(type)},
                         {gather, gather ? rows * 4 : 0},
                         {offsets, offsets ? (groups + 1) * 4 : 0}};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    return launched(launch_quantize_cols(rows, cols, src, type == SGEMM_BF16, ld, gather, src_rows, (int)groups, offsets,
                                         padded, rows > 0 ? q : nullptr, ldq, scales, lds, q_t, ldq_t, scales_t, lds_t,
                                         dev.num_sms, stream));
}

int sgemm_fp8_quantize_cols(int64_t rows, int64_t cols, const void *src, int type, int64_t ld, const int32_t *gather,
                            int64_t src_rows, int64_t groups, const int32_t *offsets, int64_t padded, uint8_t *q_t,
                            int64_t ldq_t, float *scales_t, int64_t lds_t, cudaStream_t stream)
{
    return sgemm_fp8_quantize_both(rows, cols, src, type, ld, gather, src_rows, groups, offsets, padded, nullptr, 0,
                                   nullptr, 0, q_t, ldq_t, scales_t, lds_t, stream);
}

int sgemm_fp8_quantize_blocks(int64_t rows, int64_t cols, const void *src, int type, int64_t ld, int64_t stride_src,
                              int transpose, uint8_t *q, int64_t ldq, int64_t stride_q, float *scales, int64_t lds,
                              int64_t stride_s, int64_t batch, cudaStream_t stream)
{
    if (bad_size(rows) || bad_size(cols) || bad_size(batch) || !type_size(type) || (transpose != 0 && transpose != 1))
        return SGEMM_ERR_INVALID_VALUE;
    if (stride_src < 0 || stride_q < 0 || stride_s < 0) return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0 || batch == 0) return SGEMM_OK;
    const int64_t qr = transpose ? cols : rows, qc = transpose ? rows : cols;
    const int64_t sr = ceil_div(qr, kBlock), sc = ceil_div(qc, kBlock);
    if (!src || ld < cols || bad_fp8(q, ldq, qc) || !scales || lds < sc) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || too_large(cols) || too_large(batch)) return SGEMM_ERR_OVERFLOW;
    const int64_t q_one = span(qr, qc, ldq, 1), s_one = span(sr, sc, lds, 4);
    if (q_one < 0 || s_one < 0) return SGEMM_ERR_OVERFLOW;
    if (batch > 1 && (stride_q < q_one || stride_q % 16 != 0 || stride_s < s_one / 4)) return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{q, span_fp8(qr, qc, ldq, transpose ? 16 : 8, batch, stride_q)},
                          {scales, span(sr, sc, lds, 4, batch, stride_s)}};
    const Region in[] = {{src, span(rows, cols, ld, type_size(type), batch, stride_src), type_size(type)}};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    return launched(launch_quantize_blocks(rows, cols, src, type == SGEMM_BF16, ld, stride_src, transpose == 1, q, ldq,
                                           stride_q, scales, lds, stride_s, batch, dev.num_sms, stream));
}

int sgemm_fp8(int b_form, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const float *sa,
              int64_t ld_sa, const uint8_t *B, int64_t ldb, const float *sb, int64_t ld_sb, float beta, void *C,
              int c_type, int64_t ldc, cudaStream_t stream)
{
    if (bad_size(M) || bad_size(N) || bad_size(K) || !type_size(c_type)) return SGEMM_ERR_INVALID_VALUE;
    if (b_form != SGEMM_SCALE_BLOCKS && b_form != SGEMM_SCALE_ROWS) return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!C || ldc < N) return SGEMM_ERR_INVALID_VALUE;
    const bool rows_form = b_form == SGEMM_SCALE_ROWS;
    const int64_t nk = ceil_div(K, kBlock);
    const int64_t nb = ceil_div(N, kBlock);
    if (K > 0 && (bad_fp8(A, lda, K) || bad_fp8(B, ldb, K) || bad_scales(sa, ld_sa, nk, M) ||
                  bad_scales(sb, ld_sb, rows_form ? nk : nb, rows_form ? N : nk)))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    const Region out[] = {{C, span(M, N, ldc, type_size(c_type)), type_size(c_type)}};
    const Region in[] = {{A, span(M, K, lda, 1)},
                         {B, span(N, K, ldb, 1)},
                         {sa, span(nk, M, ld_sa, 4)},
                         {sb, rows_form ? span(nk, N, ld_sb, 4) : span(nb, nk, ld_sb, 4)}};
    const int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    Fp8Args g{};
    g.mode = kFp8Dense;
    g.rows_form = rows_form;
    g.M = M, g.N = N, g.K = K;
    g.A = A, g.lda = lda, g.sa = sa, g.ld_sa = ld_sa;
    g.B = B, g.ldb = ldb, g.sb = sb, g.ld_sb = ld_sb;
    g.groups = 1;
    g.beta = beta;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc;
    return run_product(g, stream);
}

int sgemm_fp8_grouped(int64_t groups, const int32_t *offsets, int64_t rows, int64_t N, int64_t K, const uint8_t *A,
                      int64_t lda, const float *sa, int64_t ld_sa, const uint8_t *B, int64_t ldb, int64_t stride_b,
                      const float *sb, int64_t ld_sb, int64_t stride_sb, float beta, void *C, int c_type, int64_t ldc,
                      cudaStream_t stream)
{
    if (groups < 0 || groups > kMaxGroups || bad_size(rows) || bad_size(N) || bad_size(K) || !type_size(c_type))
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || rows == 0 || N == 0) return SGEMM_OK;
    if (!offsets || !C || ldc < N || stride_b < 0 || stride_sb < 0) return SGEMM_ERR_INVALID_VALUE;
    const int64_t nk = ceil_div(K, kBlock), nb = ceil_div(N, kBlock);
    if (K > 0 && (bad_fp8(A, lda, K) || bad_fp8(B, ldb, K) || bad_scales(sa, ld_sa, nk, rows) || bad_scales(sb, ld_sb, nb, nk)))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(rows) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    const int64_t b_one = span(N, K, ldb, 1), s_one = span(nb, nk, ld_sb, 4);
    if (b_one < 0 || s_one < 0) return SGEMM_ERR_OVERFLOW;
    if (K > 0 && groups > 1 && (stride_b < b_one || stride_b % 16 != 0 || stride_sb < s_one / 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{C, span(rows, N, ldc, type_size(c_type)), type_size(c_type)}};
    const Region in[] = {{A, span(rows, K, lda, 1)},
                         {B, span(N, K, ldb, 1, groups, stride_b)},
                         {sa, span(nk, rows, ld_sa, 4)},
                         {sb, span(nb, nk, ld_sb, 4, groups, stride_sb)},
                         {offsets, (groups + 1) * 4}};
    const int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    Fp8Args g{};
    g.mode = kFp8GroupRows;
    g.M = rows, g.N = N, g.K = K;
    g.A = A, g.lda = lda, g.sa = sa, g.ld_sa = ld_sa;
    g.B = B, g.ldb = ldb, g.stride_b = stride_b, g.sb = sb, g.ld_sb = ld_sb, g.stride_sb = groups > 1 ? stride_sb : 0;
    g.groups = (int)groups;
    g.offsets = offsets;
    g.beta = beta;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc;
    return run_product(g, stream);
}

int sgemm_fp8_grouped_k(int64_t groups, const int32_t *offsets, int64_t padded, int64_t M, int64_t N, const uint8_t *A,
                        int64_t lda, const float *sa, int64_t ld_sa, const uint8_t *B, int64_t ldb, const float *sb,
                        int64_t ld_sb, float beta, void *C, int c_type, int64_t ldc, int64_t stride_c,
                        cudaStream_t stream)
{
    if (groups < 0 || groups > kMaxGroups || bad_size(padded) || padded % kBlock || bad_size(M) || bad_size(N) ||
        !type_size(c_type) || stride_c < 0)
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || M == 0 || N == 0) return SGEMM_OK;
    if (!offsets || !C || ldc < N) return SGEMM_ERR_INVALID_VALUE;
    const int64_t nk = padded / kBlock;
    if (padded > 0 && (bad_fp8(A, lda, padded) || bad_fp8(B, ldb, padded) || bad_scales(sa, ld_sa, nk, M) ||
                       bad_scales(sb, ld_sb, nk, N)))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(padded)) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(c_type), c_one = span(M, N, ldc, size);
    if (c_one < 0) return SGEMM_ERR_OVERFLOW;
    if (groups > 1 && stride_c < c_one / size) return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{C, span(M, N, ldc, size, groups, stride_c), size}};
    const Region in[] = {{A, span(M, padded, lda, 1)},
                         {B, span(N, padded, ldb, 1)},
                         {sa, span(nk, M, ld_sa, 4)},
                         {sb, span(nk, N, ld_sb, 4)},
                         {offsets, (groups + 1) * 4}};
    const int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    Fp8Args g{};
    g.mode = kFp8GroupK;
    g.rows_form = true;
    g.M = M, g.N = N, g.K = padded;
    g.A = A, g.lda = lda, g.sa = sa, g.ld_sa = ld_sa;
    g.B = B, g.ldb = ldb, g.sb = sb, g.ld_sb = ld_sb;
    g.groups = (int)groups;
    g.offsets = offsets;
    g.beta = beta;
    g.C = C, g.c_bf16 = c_type == SGEMM_BF16, g.ldc = ldc, g.stride_c = groups > 1 ? stride_c : 0;
    return run_product(g, stream);
}

int sgemm_fp8_plan(int mode, int64_t groups, int64_t M, int64_t N, int64_t K, int num_sms, int *out_cols, int *out_swap,
                   int *out_split, int64_t *out_grid)
{
    if (mode < SGEMM_FP8_DENSE || mode > SGEMM_FP8_GROUPED_K || bad_size(M) || bad_size(N) || bad_size(K) || num_sms <= 0 ||
        groups < 1 || groups > kMaxGroups || (mode == SGEMM_FP8_DENSE && groups != 1))
        return SGEMM_ERR_INVALID_VALUE;
    if (too_large(M) || too_large(N) || too_large(K)) return SGEMM_ERR_OVERFLOW;
    Fp8Plan p{0, false, 0, 0};
    if (M > 0 && N > 0) {
        Fp8Args g{};
        g.mode = mode;
        g.M = M, g.N = N, g.K = K;
        g.groups = (int)groups;
        g.num_sms = num_sms;
        p = plan_fp8(g);
    }
    if (out_cols) *out_cols = p.cols;
    if (out_swap) *out_swap = p.swap ? 1 : 0;
    if (out_split) *out_split = p.split;
    if (out_grid) *out_grid = p.grid;
    return SGEMM_OK;
}

static int check_route(int64_t T, int64_t E, int type, int64_t ld, int score, int k, int renorm)
{
    if (bad_size(T) || E < 1 || E > kMaxExperts || !type_size(type) || ld < E) return SGEMM_ERR_INVALID_VALUE;
    if (score != SGEMM_SCORE_SOFTMAX && score != SGEMM_SCORE_SIGMOID) return SGEMM_ERR_INVALID_VALUE;
    if (k < 1 || k > kMaxTop || k > E || (renorm != 0 && renorm != 1)) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(T)) return SGEMM_ERR_OVERFLOW;
    return SGEMM_OK;
}

int sgemm_route(int64_t T, int64_t E, const void *logits, int type, int64_t ld, const float *bias, int score,
                int groups, int kept, int two, int k, int renorm, float scale, float *weights, int32_t *indices,
                cudaStream_t stream)
{
    int rc = check_route(T, E, type, ld, score, k, renorm);
    if (rc != SGEMM_OK) return rc;
    if (groups < 1 || groups > 32 || E % groups || kept < 1 || kept > groups || (two != 0 && two != 1) ||
        (two && E / groups < 2))
        return SGEMM_ERR_INVALID_VALUE;
    if (T == 0) return SGEMM_OK;
    if (!logits || !weights || !indices) return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{weights, span(T, k, k, 4)}, {indices, span(T, k, k, 4)}};
    const Region in[] = {{logits, span(T, E, ld, type_size(type)), type_size(type)}, {bias, bias ? E * 4 : 0}};
    if ((rc = check_regions(out, in)) != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    const RouteArgs r{T, (int)E, logits, type == SGEMM_BF16, ld, bias, score == SGEMM_SCORE_SIGMOID, groups, kept,
                      two == 1, k, renorm == 1, scale};
    return launched(launch_route(r, weights, indices, stream));
}

int sgemm_route_backward(int64_t T, int64_t E, const void *logits, int type, int64_t ld, int score, int k, int renorm,
                         float scale, const int32_t *indices, const float *grad_w, void *grad_logits, int64_t ld_g,
                         cudaStream_t stream)
{
    int rc = check_route(T, E, type, ld, score, k, renorm);
    if (rc != SGEMM_OK) return rc;
    if (ld_g < E) return SGEMM_ERR_INVALID_VALUE;
    if (T == 0) return SGEMM_OK;
    if (!logits || !indices || !grad_w || !grad_logits) return SGEMM_ERR_INVALID_VALUE;
    const Region out[] = {{grad_logits, span(T, E, ld_g, type_size(type)), type_size(type)}};
    const Region in[] = {{logits, span(T, E, ld, type_size(type)), type_size(type)},
                         {indices, span(T, k, k, 4)},
                         {grad_w, span(T, k, k, 4)}};
    if ((rc = check_regions(out, in)) != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    const RouteArgs r{T, (int)E, logits, type == SGEMM_BF16, ld, nullptr, score == SGEMM_SCORE_SIGMOID, 1, 1, false, k,
                      renorm == 1, scale};
    return launched(launch_route_backward(r, indices, grad_w, grad_logits, ld_g, stream));
}

int sgemm_dispatch(int64_t T, int k, int64_t E, const int32_t *indices, int32_t *offsets, int32_t *row_of,
                   int32_t *token_of, cudaStream_t stream)
{
    if (bad_size(T) || k < 1 || E < 1 || E > kMaxExperts || !offsets) return SGEMM_ERR_INVALID_VALUE;
    if (T > 0 && (!indices || !row_of || !token_of)) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(T) || T * k > kMaxSize) return SGEMM_ERR_OVERFLOW;
    const Region out[] = {{offsets, (E + 1) * 4}, {row_of, T * k * 4}, {token_of, T * k * 4}};
    const Region in[] = {{indices, T * k * 4}};
    int rc = check_regions(out, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    void *scratch = nullptr;
    const size_t bytes = dispatch_scratch_bytes(T * k, (int)E);
    if (bytes > 0 && (take_alloc_failure() || cudaMallocFromPoolAsync(&scratch, bytes, dev.pool, stream) != cudaSuccess)) {
        cudaGetLastError();
        return SGEMM_ERR_ALLOC;
    }
    rc = launched(launch_dispatch(T, k, (int)E, indices, offsets, row_of, token_of, scratch, stream));
    if (scratch) cudaFreeAsync(scratch, stream);
    return rc;
}

int sgemm_combine(int64_t T, int k, int64_t cols, int64_t rows, const void *Y, int type, int64_t ldy,
                  const int32_t *row_of, const float *weights, void *out, int64_t ld_out, cudaStream_t stream)
{
    if (bad_size(T) || k < 1 || k > kMaxTop || bad_size(cols) || bad_size(rows) || !type_size(type))
        return SGEMM_ERR_INVALID_VALUE;
    if (T == 0 || cols == 0) return SGEMM_OK;
    if ((!Y && rows > 0) || !row_of || !out || ldy < cols || ld_out < cols) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(T) || cols > kMaxCols || too_large(rows)) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(type);
    const Region o[] = {{out, span(T, cols, ld_out, size), size}};
    const Region in[] = {{Y, span(rows, cols, ldy, size), size},
                         {row_of, span(T, k, k, 4)},
                         {weights, weights ? span(T, k, k, 4) : 0}};
    int rc = check_regions(o, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    return launched(launch_combine(T, k, cols, rows, Y, type == SGEMM_BF16, ldy, row_of, weights, out, ld_out, stream));
}

int sgemm_combine_backward(int64_t T, int k, int64_t cols, int64_t rows, const void *grad_out, int type, int64_t ld_go,
                           const void *Y, int64_t ldy, const int32_t *row_of, const float *weights, void *grad_y,
                           int64_t ld_gy, float *grad_w, cudaStream_t stream)
{
    if (bad_size(T) || k < 1 || k > kMaxTop || bad_size(cols) || bad_size(rows) || !type_size(type))
        return SGEMM_ERR_INVALID_VALUE;
    if (T == 0 || (!grad_y && !grad_w)) return SGEMM_OK;
    if (!row_of || (cols > 0 && !grad_out) || ld_go < cols) return SGEMM_ERR_INVALID_VALUE;
    if (grad_y && ld_gy < cols) return SGEMM_ERR_INVALID_VALUE;
    if (grad_w && ((!Y && rows > 0 && cols > 0) || ldy < cols)) return SGEMM_ERR_INVALID_VALUE;
    if (too_large(T) || too_large(cols) || too_large(rows)) return SGEMM_ERR_OVERFLOW;
    const int64_t size = type_size(type);
    const Region o[] = {{grad_y, grad_y ? span(rows, cols, ld_gy, size) : 0, size},
                        {grad_w, grad_w ? span(T, k, k, 4) : 0}};
    const Region in[] = {{grad_out, span(T, cols, ld_go, size), size},
                         {Y, grad_w ? span(rows, cols, ldy, size) : 0, size},
                         {row_of, span(T, k, k, 4)},
                         {weights, weights ? span(T, k, k, 4) : 0}};
    int rc = check_regions(o, in);
    if (rc != SGEMM_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    return launched(launch_combine_backward(T, k, cols, rows, grad_out, type == SGEMM_BF16, ld_go, Y, ldy, row_of, weights,
                                            grad_y, ld_gy, grad_w, stream));
}

}  // extern "C"
