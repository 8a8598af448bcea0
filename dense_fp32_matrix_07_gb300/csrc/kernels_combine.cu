// The experts' outputs summed per token, and the gradients of that sum:
//
//   out[t] = sum_j w[t, j] Y[row_of[t, j]]
//   dY[row_of[t, j]] = w[t, j] dout[t],   dw[t, j] = <dout[t], Y[row_of[t, j]]>
//
// Without weights (w = 1) the sum is also the gradient of gathering rows for
// their experts. A slot whose row is outside [0, rows) adds nothing. Sums are
// in FP32, in slot order. Bound by memory: Y, out and dout once. Measured on
// one GB300, 8191 tokens of 6 rows of 2048 bfloat16: the sum 42.5 us (5.5
// TB/s), its gradients 78 us (5.6 TB/s). Requesting four or eight rows before
// the first is added took 72 us and more; two rows at a time in the gradients
// changed nothing. Columns or strides that are no multiples of 16 bytes go one
// value at a time: 2047 columns 3.7 times the sum's time, 1.7 times that of the
// gradients.
#include "experts.cuh"

namespace sgemm_gb300 {

namespace {

// N values of T as one access of up to 16 bytes.
template <class T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// One thread per N columns of a token: blockDim.x columns' threads, blockDim.y
// tokens (16 tokens of a decode step: 6 us, launch and one chain of loads).
template <class T, int N>
__global__ void __launch_bounds__(256)
combine_kernel(int64_t tokens, int k, int64_t cols, int64_t rows, const T *__restrict__ Y, int64_t ldy,
               const int32_t *__restrict__ row_of, const float *__restrict__ weights, T *__restrict__ out,
               int64_t ld_out)
{
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (t >= tokens || c >= cols) return;
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
#pragma unroll 8
    for (int j = 0; j < k; ++j) {
        const int64_t r = row_of[t * k + j];
        if (r < 0 || r >= rows) continue;
        const float w = weights ? weights[t * k + j] : 1.0f;
        const Pack<T, N> y = *reinterpret_cast<const Pack<T, N> *>(Y + r * ldy + c);
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w, load_as_float(&y.v[i]), sum[i]);
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) store_from_float(&o.v[i], sum[i]);
    *reinterpret_cast<Pack<T, N> *>(out + t * ld_out + c) = o;
}

// One warp per token; each lane holds STEPS packs of the token's gradient at a
// time and meets every slot's row with them.
template <class T, int N, int STEPS>
__global__ void __launch_bounds__(256)
combine_backward_kernel(int64_t tokens, int k, int64_t cols, int64_t rows, const T *__restrict__ grad_out,
                        int64_t ld_go, const T *__restrict__ Y, int64_t ldy, const int32_t *__restrict__ row_of,
                        const float *__restrict__ weights, T *__restrict__ grad_y, int64_t ld_gy,
                        float *__restrict__ grad_w)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= tokens) return;
    const int my_row = lane < k ? row_of[t * k + lane] : -1;
    const float my_w = lane < k ? (weights ? weights[t * k + lane] : 1.0f) : 0.0f;
    float dw = 0.0f;                                  // lane j: slot j
    for (int64_t c0 = 0; c0 < cols; c0 += 32 * N * STEPS) {
        Pack<T, N> g[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int64_t c = c0 + (32 * s + lane) * N;
            if (c < cols) g[s] = *reinterpret_cast<const Pack<T, N> *>(grad_out + t * ld_go + c);
        }
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(0xffffffffu, my_row, j);
            const float w = __shfl_sync(0xffffffffu, my_w, j);
            if (r < 0 || r >= rows) continue;
            float dot = 0.0f;
            Pack<T, N> y[STEPS];
            if (grad_w) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int64_t c = c0 + (32 * s + lane) * N;
                    if (c < cols) y[s] = *reinterpret_cast<const Pack<T, N> *>(Y + r * ldy + c);
                }
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int64_t c = c0 + (32 * s + lane) * N;
                if (c < cols) {
                    Pack<T, N> o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float x = load_as_float(&g[s].v[i]);
                        if (grad_w) dot = fmaf(x, load_as_float(&y[s].v[i]), dot);
                        store_from_float(&o.v[i], w * x);
                    }
                    if (grad_y) *reinterpret_cast<Pack<T, N> *>(grad_y + r * ld_gy + c) = o;
                }
            }
            if (grad_w) {
#pragma unroll
                for (int d = 16; d; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (lane == j) dw += dot;
            }
        }
    }
    if (grad_w && lane < k) grad_w[t * k + lane] = dw;
}

bool aligned16(const void *p, int64_t ld, int64_t per16)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % per16 == 0;
}

template <class T, int N>
cudaError_t combine_of(int64_t T_, int k, int64_t cols, int64_t rows, const T *Y, int64_t ldy, const int32_t *row_of,
                       const float *weights, T *out, int64_t ld_out, cudaStream_t stream)
{
    const int64_t packs = (cols + N - 1) / N;
    unsigned x = 32;
    while (x < 256 && (int64_t)x < packs) x *= 2;
    const unsigned y = 256 / x;
    const dim3 grid((unsigned)((T_ + y - 1) / y), (unsigned)((packs + x - 1) / x));
    combine_kernel<T, N><<<grid, dim3(x, y), 0, stream>>>(T_, k, cols, rows, Y, ldy, row_of, weights, out, ld_out);
    return cudaGetLastError();
}

template <class T, int N, int STEPS>
cudaError_t combine_backward_of(int64_t T_, int k, int64_t cols, int64_t rows, const T *go, int64_t ld_go, const T *Y,
                                int64_t ldy, const int32_t *row_of, const float *weights, T *gy, int64_t ld_gy,
                                float *gw, cudaStream_t stream)
{
    combine_backward_kernel<T, N, STEPS><<<(unsigned)((T_ + 7) / 8), 256, 0, stream>>>(
        T_, k, cols, rows, go, ld_go, Y, ldy, row_of, weights, gy, ld_gy, gw);
    return cudaGetLastError();
}

template <class T>
cudaError_t combine_t(int64_t T_, int k, int64_t cols, int64_t rows, const void *Y, int64_t ldy, const int32_t *row_of,
                      const float *weights, void *out, int64_t ld_out, cudaStream_t stream)
{
    constexpr int per16 = 16 / (int)sizeof(T);
    const T *y = static_cast<const T *>(Y);
    T *o = static_cast<T *>(out);
    if (cols % per16 == 0 && aligned16(Y, ldy, per16) && aligned16(out, ld_out, per16))
        return combine_of<T, per16>(T_, k, cols, rows, y, ldy, row_of, weights, o, ld_out, stream);
    return combine_of<T, 1>(T_, k, cols, rows, y, ldy, row_of, weights, o, ld_out, stream);
}

template <class T>
cudaError_t combine_backward_t(int64_t T_, int k, int64_t cols, int64_t rows, const void *go, int64_t ld_go,
                               const void *Y, int64_t ldy, const int32_t *row_of, const float *weights, void *gy,
                               int64_t ld_gy, float *gw, cudaStream_t stream)
{
    constexpr int per16 = 16 / (int)sizeof(T);
    const T *g = static_cast<const T *>(go), *y = static_cast<const T *>(Y);
    T *o = static_cast<T *>(gy);
    const bool vec = cols % per16 == 0 && aligned16(go, ld_go, per16) && (!gw || aligned16(Y, ldy, per16)) &&
                     (!gy || aligned16(gy, ld_gy, per16));
    if (vec)
        return combine_backward_of<T, per16, 4>(T_, k, cols, rows, g, ld_go, y, ldy, row_of, weights, o, ld_gy, gw, stream);
    return combine_backward_of<T, 1, 8>(T_, k, cols, rows, g, ld_go, y, ldy, row_of, weights, o, ld_gy, gw, stream);
}

}  // namespace

cudaError_t launch_combine(int64_t T, int k, int64_t cols, int64_t rows, const void *Y, bool bf16, int64_t ldy,
                           const int32_t *row_of, const float *weights, void *out, int64_t ld_out, cudaStream_t stream)
{
    return bf16 ? combine_t<__nv_bfloat16>(T, k, cols, rows, Y, ldy, row_of, weights, out, ld_out, stream)
                : combine_t<float>(T, k, cols, rows, Y, ldy, row_of, weights, out, ld_out, stream);
}

cudaError_t launch_combine_backward(int64_t T, int k, int64_t cols, int64_t rows, const void *grad_out, bool bf16,
                                    int64_t ld_go, const void *Y, int64_t ldy, const int32_t *row_of,
                                    const float *weights, void *grad_y, int64_t ld_gy, float *grad_w,
                                    cudaStream_t stream)
{
    return bf16 ? combine_backward_t<__nv_bfloat16>(T, k, cols, rows, grad_out, ld_go, Y, ldy, row_of, weights, grad_y,
                                                    ld_gy, grad_w, stream)
                : combine_backward_t<float>(T, k, cols, rows, grad_out, ld_go, Y, ldy, row_of, weights, grad_y, ld_gy,
                                            grad_w, stream);
}

}  // namespace sgemm_gb300
