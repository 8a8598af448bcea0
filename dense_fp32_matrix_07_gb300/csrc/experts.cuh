// Shared definitions of the operators around products over experts: routing,
// 8-bit quantisation, block-scaled 8-bit products and the combining sum
// (declared in include/sgemm_experts.h).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace sgemm_gb300 {

constexpr int kBlock = 128;              // values that share a scale
constexpr int kMaxGroups = 512;          // groups of a grouped product (one table entry each in shared memory)
constexpr int kMaxExperts = 1024;        // experts a router scores (32 per lane of a warp)
constexpr int kMaxTop = 32;              // experts per token (one lane each)

// Largest e4m3 magnitude, and the magnitude a block counts as at least
// (2^-96: 448 / 2^-96 and 2^-96 / 448 are both normal floats, so a block of
// zeros or denormals has a finite scale and a finite reciprocal).
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Least = 0x1p-96f;

// Per-device state of the library (sgemm_api.cu): the error word, the number
// of SMs and the scratch pool. Returns an SGEMM_* code.
struct DeviceInfo {
    unsigned int *status;
    int num_sms;
    cudaMemPool_t pool;
};
int device_info(DeviceInfo *out);
// Whether a pending sgemm_test_fail_next_allocs() failure was taken.
bool take_alloc_failure();

// ------------------------------------------------------------ 8-bit products

enum Fp8Mode : int {
    kFp8Dense = 0,     // C = A . B^T
    kFp8GroupRows = 1, // rows [offsets[g], offsets[g+1]) of A meet B_g
    kFp8GroupK = 2     // C_g = A . B^T over the K blocks of group g
};

struct Fp8Args {
    int mode;
    bool rows_form;            // B's scales per row and K block, else per 128 x 128 block
    int64_t M, N, K;           // rows of A (all groups'), rows of B (one group's), shared length
    const uint8_t *A;
    int64_t lda;
    const float *sa;           // sa[kb * ld_sa + row]
    int64_t ld_sa;
    const uint8_t *B;
    int64_t ldb, stride_b;
    const float *sb;           // blocks: sb[g * stride_sb + nb * ld_sb + kb]; rows: sb[kb * ld_sb + n]
    int64_t ld_sb, stride_sb;
    int groups;
    const int32_t *offsets;
    float beta;
    void *C;
    int c_bf16;
    int64_t ldc, stride_c;
    unsigned int *status;
    int num_sms;
};

// The kernel shape of a product: `cols` columns of tensor memory per tile,
// `swap` = B's rows on the 128 lanes (few tokens), `split` CTAs of a cluster
// sharing each tile's K range.
struct Fp8Plan {
    int cols;
    bool swap;
    int split;
    int64_t grid;
};
Fp8Plan plan_fp8(const Fp8Args &g);
cudaError_t prepare_fp8();
cudaError_t launch_fp8(const Fp8Args &g, cudaStream_t stream);

// -------------------------------------------------------------- quantisation

cudaError_t launch_quantize_rows(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                 const int32_t *gather, int64_t src_rows, uint8_t *q, int64_t ldq, float *scales,
                                 int64_t lds, cudaStream_t stream);
// The transposed column form (qt, scales_t) and, where q is given, the row form from the same read.
cudaError_t launch_quantize_cols(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                 const int32_t *gather, int64_t src_rows, int groups, const int32_t *offsets,
                                 int64_t padded, uint8_t *q, int64_t ldq, float *scales, int64_t lds, uint8_t *qt,
                                 int64_t ldqt, float *scales_t, int64_t ldst, int num_sms, cudaStream_t stream);
cudaError_t launch_quantize_blocks(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                   int64_t stride_src, bool transpose, uint8_t *q, int64_t ldq, int64_t stride_q,
                                   float *scales, int64_t lds, int64_t stride_s, int64_t batch, int num_sms,
                                   cudaStream_t stream);

// ------------------------------------------------------- routing, combination

struct RouteArgs {
    int64_t T;
    int E;
    const void *logits;
    bool bf16;
    int64_t ld;
    const float *bias;
    bool sigmoid;
    int groups, kept;
    bool two;
    int k;
    bool renorm;
    float scale;
};
cudaError_t launch_route(const RouteArgs &r, float *weights, int32_t *indices, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs &r, const int32_t *indices, const float *grad_w, void *grad_logits,
                                  int64_t ld_g, cudaStream_t stream);
// One-time set-up of the device (shared memory above 48 KB).
cudaError_t prepare_route();
// Bytes of scratch launch_dispatch() needs (0: none).
size_t dispatch_scratch_bytes(int64_t n, int E);
cudaError_t launch_dispatch(int64_t T, int k, int E, const int32_t *indices, int32_t *offsets, int32_t *row_of,
                            int32_t *token_of, void *scratch, cudaStream_t stream);
cudaError_t launch_combine(int64_t T, int k, int64_t cols, int64_t rows, const void *Y, bool bf16, int64_t ldy,
                           const int32_t *row_of, const float *weights, void *out, int64_t ld_out, cudaStream_t stream);
cudaError_t launch_combine_backward(int64_t T, int k, int64_t cols, int64_t rows, const void *grad_out, bool bf16,
                                    int64_t ld_go, const void *Y, int64_t ldy, const int32_t *row_of,
                                    const float *weights, void *grad_y, int64_t ld_gy, float *grad_w,
                                    cudaStream_t stream);

// ------------------------------------------------------------ device helpers

// One value of a float or bfloat16 array as float, and back.
__device__ __forceinline__ float load_as_float(const float *p) { return *p; }
__device__ __forceinline__ float load_as_float(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_from_float(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_from_float(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace sgemm_gb300
