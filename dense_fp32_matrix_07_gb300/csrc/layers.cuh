// Shared definitions of the operators of layers in 16 bits: products with an
// epilogue (dense and over experts), the epilogue's gradient, and the
// root-mean-square norm (declared in include/sgemm_layers.h).
#pragma once

#include "experts.cuh"

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <type_traits>

namespace sgemm_gb300 {

enum Activation : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
enum Join : int { kJoinNone = 0, kJoinAdd = 1, kJoinMul = 2 };

// ----------------------------------------------------------- 16-bit products

enum Bf16Mode : int {
    kBf16Dense = 0,      // C = op(A) . op(B)
    kBf16GroupRows = 1,  // rows [offsets[g], offsets[g+1]) of A meet B_g
    kBf16GroupK = 2      // C_g = A^T . B over the rows of group g
};

struct Bf16Args {
    int mode;
    int op_a, op_b;            // as stored: A M x K (0) or K x M (1), B K x N (0) or N x K (1)
    int64_t M, N, K;           // rows and columns of C (one group's under GroupK), shared length
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb, stride_b;
    int groups;
    const int32_t *offsets;
    const float *bias;         // N values (of group g at g * stride_bias), or null
    int64_t stride_bias;
    int act, join;
    void *pre;                 // the sums before the activation, or null
    int64_t ld_pre;
    const void *D;
    int64_t ldd;
    void *C;
    int c_bf16;                // C, pre and D are bfloat16, else float
    int64_t ldc, stride_c;     // GroupK: C (and D) of group g at g * stride_c
    unsigned int *status;
    int num_sms;
};

// The kernel shape of a product: `cols` accumulator columns per tile, `pair` =
// two CTAs on a 256-lane tile, `swap` = the lanes hold columns of C, `split`
// CTAs of a cluster sharing each tile's K blocks.
struct Bf16Plan {
    int cols;
    bool pair, swap;
    int split;
    int64_t grid;
};
Bf16Plan plan_bf16(const Bf16Args &g);
cudaError_t prepare_bf16();
cudaError_t launch_bf16(const Bf16Args &g, cudaStream_t stream);

// ------------------------------------------------------ gradient of the epilogue

struct EpilogueBackwardArgs {
    int64_t rows, cols;
    bool bf16;
    const void *grad_out;
    int64_t ld_go;
    const void *pre;
    int64_t ld_pre;
    int act, join;
    const void *D;
    int64_t ldd;
    int groups;
    const int32_t *offsets;    // null: one group of all rows
    void *grad_pre;
    int64_t ld_gp;
    void *grad_D;
    int64_t ld_gd;
    float *grad_bias;
    int64_t stride_gb;
    int num_sms;
};
size_t epilogue_backward_scratch_bytes(const EpilogueBackwardArgs &g);
cudaError_t launch_epilogue_backward(const EpilogueBackwardArgs &g, void *scratch, cudaStream_t stream);

// --------------------------------------------------------- root-mean-square norm

constexpr int64_t kMaxNormCols = 16384;   // a row is held in registers by its block

struct RmsNormArgs {
    int64_t rows, cols;
    bool bf16;
    const void *x;
    int64_t ldx;
    const void *residual;
    int64_t ld_res;
    const float *weight;
    float eps;
    void *sum;
    int64_t ld_sum;
    void *y;
    int64_t ldy;
    uint8_t *q;
    int64_t ldq;
    float *scales;
    int64_t lds;
};
// One-time set-up of the device (shared memory above 48 KB).
cudaError_t prepare_rms_norm();
cudaError_t launch_rms_norm(const RmsNormArgs &g, cudaStream_t stream);

struct RmsNormBackwardArgs {
    int64_t rows, cols;
    bool bf16;
    const void *grad_y;
    int64_t ld_gy;
    const void *x;
    int64_t ldx;
    const float *weight;
    float eps;
    const void *grad_sum;
    int64_t ld_gs;
    void *grad_x;
    int64_t ld_gx;
    float *grad_weight;
    int num_sms;
};
size_t rms_norm_backward_scratch_bytes(const RmsNormBackwardArgs &g);
cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs &g, void *scratch, cudaStream_t stream);

// ---------------------------------------------------------------- host helpers

// Whether a matrix's rows (null: none) can be accessed 16 bytes at a time.
inline bool pieces16(const void *p, int64_t ld, int64_t per16)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % per16 == 0);
}

// A launch whose blocks may begin before the stream's last kernel has ended:
// they wait for that themselves (griddepcontrol.wait) before they read it.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, static_cast<Params>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------ device helpers

// N values of T as one access of up to 16 bytes.
template <class T, int N>
struct alignas(sizeof(T) * N) Values {
    T v[N];
};

// Eight neighbouring values of a row as they are stored, by 16-byte accesses.
template <class T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    // Those from lo on, below hi; the others are zeros.
    __device__ __forceinline__ void load_some(const T *p, int lo, int hi)
    {
        uint32_t w[2 * sizeof(T)] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < lo || e >= hi) continue;
            if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(p[e]);
            else w[e / 2] |= (uint32_t) * reinterpret_cast<const uint16_t *>(p + e) << (16 * (e & 1));
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ float get(int e) const
    {
        const uint4 &q = u[sizeof(T) == 4 ? e / 4 : 0];
        const int i = sizeof(T) == 4 ? e % 4 : e / 2;
        const uint32_t x = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
        if constexpr (sizeof(T) == 4) return __uint_as_float(x);
        else return __uint_as_float((e & 1) ? x & 0xffff0000u : x << 16);
    }
};

__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// exp(x) by one multiplication and the hardware's 2^x: 2^-22 relative, and
// 1.5 |x| 2^-24 from the rounded argument and its constant. 0 below 2^-126.
__device__ __forceinline__ float fast_exp(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504088896341f));
    return y;
}

// 1 / x by the hardware's reciprocal (1 ulp), for x >= 1; 0 past 2^126.
__device__ __forceinline__ float fast_reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + exp(-x)); 0 where exp(-x) passes 2^126 (1e-38 at most is lost).
__device__ __forceinline__ float sigmoid(float x) { return fast_reciprocal(1.0f + fast_exp(-x)); }

// The normal distribution's integral at z, and exp(-z^2 / 2) on the way, without
// branches: for z >= 0 the integral at -z is exp(-z^2 / 2) t P(t), t = 1 / (1 +
// 0.3 z). P is of degree 7, fitted in 64 bits for z up to 14 (least squares of
// the relative error, weights raised where it is largest) to 1.7e-7 of the
// integral itself: a formula of absolute error (1.5e-7 of erf) was off by 4.7e-4
// of gelu at -4 and 1e-2 at -8. With roundings, (32 + 2 z^2) 2^-24 relative.
__device__ __forceinline__ float normal_integral(float z, float &e)
{
    const float t = fast_reciprocal(fmaf(0.3f, fabsf(z), 1.0f));
    e = fast_exp(-0.5f * z * z);
    float q = fmaf(0.0356747786f, t, -0.157203101f);
    q = fmaf(q, t, 0.206353537f);
    q = fmaf(q, t, -0.0536836714f);
    q = fmaf(q, t, 0.12856164f);
    q = fmaf(q, t, 0.0999134882f);
    q = fmaf(q, t, 0.120753957f);
    q = fmaf(q, t, 0.119629299f);
    q *= t * e;
    return z < 0.0f ? q : 1.0f - q;
}

// 2 sqrt(2/pi) (z + 0.044715 z^3): gelu_tanh is z times the sigmoid of it, as
// 1 + tanh(u) is twice the sigmoid of 2 u.
__device__ __forceinline__ float tanh_argument(float z)
{
    return 1.59576912160573071f * fmaf(0.044715f * z * z, z, z);
}

// The activations, in FP32 (a NaN stays one).
template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    float e;
    if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;
    else if constexpr (ACT == kActGelu) return z * normal_integral(z, e);
    else if constexpr (ACT == kActGeluTanh) return z * sigmoid(tanh_argument(z));
    else if constexpr (ACT == kActSilu) return z * sigmoid(z);
    else return z;
}

// f(integral_constant) of the activation that the host gave as a number.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f)
{
    switch (act) {
    case kActRelu: return f(std::integral_constant<int, kActRelu>{});
    case kActGelu: return f(std::integral_constant<int, kActGelu>{});
    case kActGeluTanh: return f(std::integral_constant<int, kActGeluTanh>{});
    case kActSilu: return f(std::integral_constant<int, kActSilu>{});
    default: return f(std::integral_constant<int, kActNone>{});
    }
}

}  // namespace sgemm_gb300
