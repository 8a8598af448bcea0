// Quantisation to e4m3 with one scale per block of 128 values (along a row,
// along a column within a group of rows, or 128 x 128):
//
//   a = max(max |x| over the block, 2^-96),  scale = a / 448,
//   q = e4m3(x * (448 / a))   (round to nearest even, saturating)
//
// A block with a NaN gets a NaN scale and NaN values; one with an infinity an
// infinite scale, zeros for its finite values and NaN for the infinity.
// All forms are bound by memory: each value is read once and written as one
// byte per form.
#include "experts.cuh"

#include <cuda_fp8.h>

namespace sgemm_gb300 {

namespace {

// Magnitudes as unsigned integers: they order like the floats, with NaN above
// infinity, so that a NaN in a block wins the maximum.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

struct Scale {
    float inv, scale;
};

__device__ __forceinline__ Scale scale_of(uint32_t amax)
{
    float a = __uint_as_float(amax);
    if (a < kFp8Least) a = kFp8Least;   // false for NaN
    return Scale{__fdiv_rn(kFp8Max, a), __fdiv_rn(a, kFp8Max)};
}

// Four values to four bytes (cvt.rn.satfinite.e4m3x2.f32 keeps NaN).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// N consecutive values from p (N * sizeof(T) a multiple of 16, p 16-byte aligned).
template <int N>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + j);
        v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
    }
}

template <int N>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&v)[N])
{
    static_assert(N % 8 == 0, "16-byte pieces");
#pragma unroll
    for (int j = 0; j < N; j += 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p + j);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[j + 2 * i] = __uint_as_float(w[i] << 16);
            v[j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// Values c .. c + N - 1 of a row of `cols`, zeros past its end.
template <int N, class T>
__device__ __forceinline__ void load_row(const T *row, int64_t c, int64_t cols, bool vec, float (&v)[N])
{
    if (vec && c + N <= cols) {
        load_vec<N>(row + c, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c + j < cols ? load_as_float(row + c + j) : 0.0f;
}

// ---------------------------------------------------------------------------
// Rows: 16 lanes per block of 128 (8 values each), so a warp quantises two
// blocks at a time and every lane's load and store is 16 (32 for float) and 8
// bytes wide. A CTA covers 16 rows x 4 blocks; the scales, [block][row], leave
// through shared memory as runs of 16 rows.
constexpr int kRowsPerCta = 16, kBlocksPerCta = 4;

template <class T>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(int64_t rows, int64_t cols, const T *__restrict__ src, int64_t ld,
                     const int32_t *__restrict__ gather, int64_t src_rows, uint8_t *__restrict__ q, int64_t ldq,
                     float *__restrict__ scales, int64_t lds, int vec)
{
    __shared__ float tile[kBlocksPerCta][kRowsPerCta];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int64_t nb = (cols + kBlock - 1) / kBlock;
    const int64_t b0 = (int64_t)blockIdx.y * kBlocksPerCta;
    const int64_t r0 = (int64_t)blockIdx.x * kRowsPerCta;
    // Warp w: rows 2w and 2w + 1, each half of the warp blocks half and half + 2.
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 2 * warp + (i >> 1), b = b0 + half + 2 * (i & 1);
        int64_t from = -1;
        if (r < rows) from = gather ? (int64_t)gather[r] : r;
        if (from >= 0 && from < src_rows && b < nb) {
            load_row<8>(src + from * ld, b * kBlock + 8 * l, cols, vec != 0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 2 * warp + (i >> 1), b = b0 + half + 2 * (i & 1);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, magnitude(v[i][j]));
#pragma unroll
        for (int d = 8; d; d /= 2) m = umax(m, __shfl_xor_sync(0xffffffffu, m, d));
        const Scale s = scale_of(m);
        const int64_t c = b * kBlock + 8 * l;
        if (r < rows && c < cols) {
            uint2 o;
            o.x = to_e4m3x4(v[i][0] * s.inv, v[i][1] * s.inv, v[i][2] * s.inv, v[i][3] * s.inv);
            o.y = to_e4m3x4(v[i][4] * s.inv, v[i][5] * s.inv, v[i][6] * s.inv, v[i][7] * s.inv);
            *reinterpret_cast<uint2 *>(q + r * ldq + c) = o;
        }
        if (l == 0) tile[half + 2 * (i & 1)][2 * warp + (i >> 1)] = s.scale;
    }
    __syncthreads();
    if (threadIdx.x < kBlocksPerCta * kRowsPerCta) {
        const int64_t b = b0 + threadIdx.x / kRowsPerCta, r = r0 + threadIdx.x % kRowsPerCta;
        if (b < nb && r < rows) scales[b * lds + r] = tile[threadIdx.x / kRowsPerCta][threadIdx.x % kRowsPerCta];
    }
}

// ---------------------------------------------------------------------------
// Tiles of 128 x 128: thread (x, y) of 16 x 16 holds rows 8y .. 8y+7 of
// columns 8x .. 8x+7 in registers, so that one read of the tile serves the
// row form (8 bytes of each of its rows), the column form and the block form.
// Transposed output goes through shared memory: column c's 128 bytes are one
// row there, its 8-byte pieces permuted by XOR with c / 8 against bank
// conflicts.
struct TileArgs {
    int64_t rows, cols;
    const void *src;
    int64_t ld, stride_src;
    const int32_t *gather;
    int64_t src_rows;
    int groups;                    // column form: groups of rows, or 0 for one group of all rows
    const int32_t *offsets;
    int64_t row_blocks, col_blocks, batch;
    uint8_t *q;                    // row form or block form, or null
    int64_t ldq, stride_q;
    float *scales;
    int64_t lds, stride_s;
    uint8_t *qt;                   // column form or transposed block form, or null
    int64_t ldqt, stride_qt;
    float *scales_t;
    int64_t ldst, stride_st;
    int vec;
};

template <class T, bool BLOCKS>
__global__ void __launch_bounds__(256)
quantize_tiles_kernel(const TileArgs a)
{
    __shared__ uint32_t red[8][128];
    __shared__ uint4 turned[128 * 8];
    __shared__ int table[kMaxGroups + 2];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!BLOCKS && a.groups > 0) {
        // table[g] = blocks of the groups before g.
        for (int g = threadIdx.x; g < a.groups; g += 256) {
            int64_t lo = a.offsets[g], hi = a.offsets[g + 1];
            lo = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
            hi = hi < lo ? lo : hi > a.rows ? a.rows : hi;
            table[g] = (int)((hi - lo + kBlock - 1) / kBlock);
        }
        __syncthreads();
        if (warp == 0) {
            int64_t carry = 0;
            for (int g0 = 0; g0 < a.groups; g0 += 32) {
                const int g = g0 + lane;
                const int64_t mine = g < a.groups ? table[g] : 0;
                int64_t sum = mine;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += up;
                }
                const int64_t before = carry + sum - mine;
                if (g < a.groups) table[g] = (int)(before < a.row_blocks ? before : a.row_blocks);
                carry += __shfl_sync(0xffffffffu, sum, 31);
                if (g0 + 32 >= a.groups && lane == 0) table[a.groups] = (int)(carry < a.row_blocks ? carry : a.row_blocks);
            }
        }
        __syncthreads();
    }
    const int64_t per = a.row_blocks * a.col_blocks;
    for (int64_t t = blockIdx.x; t < per * a.batch; t += gridDim.x) {
        const int64_t e = t / per, rb = (t % per) / a.col_blocks, cb = (t % per) % a.col_blocks;
        // Rows [r0, r1) of this tile.
        int64_t r0 = rb * kBlock, r1 = r0 + kBlock < a.rows ? r0 + kBlock : a.rows;
        if (!BLOCKS && a.groups > 0) {
            if (rb >= table[a.groups]) {
                r0 = r1 = 0;                         // past the last group: zeros
            } else {
                int lo = 0, hi = a.groups - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (table[mid] <= rb)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                int64_t g0 = a.offsets[lo], g1 = a.offsets[lo + 1];
                g0 = g0 < 0 ? 0 : g0 > a.rows ? a.rows : g0;
                g1 = g1 < g0 ? g0 : g1 > a.rows ? a.rows : g1;
                r0 = g0 + (rb - table[lo]) * kBlock;
                r1 = r0 + kBlock < g1 ? r0 + kBlock : g1;
            }
        }
        const T *src = static_cast<const T *>(a.src) + e * a.stride_src;
        const int64_t c = cb * kBlock + 8 * x;
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 8 * y + i;
            int64_t from = -1;
            if (r < r1) from = a.gather ? (int64_t)a.gather[r] : r;
            if (from >= 0 && from < a.src_rows) {
                load_row<8>(src + from * a.ld, c, a.cols, a.vec != 0, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
        }
        if (!BLOCKS && a.q) {
            // Row form: a row's 128 columns are the 16 lanes of a half warp.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = umax(m, magnitude(v[i][j]));
#pragma unroll
                for (int d = 8; d; d /= 2) m = umax(m, __shfl_xor_sync(0xffffffffu, m, d));
                const Scale s = scale_of(m);
                const int64_t r = r0 + 8 * y + i;
                if (r < r1) {
                    if (c < a.cols) {
                        uint2 o;
                        o.x = to_e4m3x4(v[i][0] * s.inv, v[i][1] * s.inv, v[i][2] * s.inv, v[i][3] * s.inv);
                        o.y = to_e4m3x4(v[i][4] * s.inv, v[i][5] * s.inv, v[i][6] * s.inv, v[i][7] * s.inv);
                        *reinterpret_cast<uint2 *>(a.q + r * a.ldq + c) = o;
                    }
                    if (x == 0) a.scales[cb * a.lds + r] = s.scale;
                }
            }
        }
        // Columns' (or the block's) largest magnitudes.
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = umax(m[j], magnitude(v[i][j]));
            m[j] = umax(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        }
        Scale s[8];
        if (BLOCKS) {
            uint32_t all = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) all = umax(all, m[j]);
            all = __reduce_max_sync(0xffffffffu, all);
            __syncthreads();
            if (lane == 0) red[warp][0] = all;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 8; ++w) all = umax(all, red[w][0]);
            s[0] = scale_of(all);
#pragma unroll
            for (int j = 1; j < 8; ++j) s[j] = s[0];
            if (threadIdx.x == 0) {
                if (a.q)
                    a.scales[e * a.stride_s + rb * a.lds + cb] = s[0].scale;
                else
                    a.scales_t[e * a.stride_st + cb * a.ldst + rb] = s[0].scale;
            }
            if (a.q) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t r = r0 + 8 * y + i;
                    if (r < r1 && c < a.cols) {
                        uint2 o;
                        o.x = to_e4m3x4(v[i][0] * s[0].inv, v[i][1] * s[0].inv, v[i][2] * s[0].inv, v[i][3] * s[0].inv);
                        o.y = to_e4m3x4(v[i][4] * s[0].inv, v[i][5] * s[0].inv, v[i][6] * s[0].inv, v[i][7] * s[0].inv);
                        *reinterpret_cast<uint2 *>(a.q + e * a.stride_q + r * a.ldq + c) = o;
                    }
                }
                continue;
            }
        } else {
            __syncthreads();
            if (lane < 16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) red[warp][8 * x + j] = m[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int w = 0; w < 8; ++w) m[j] = umax(m[j], red[w][8 * x + j]);
                s[j] = scale_of(m[j]);
            }
            if (y == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < a.cols) a.scales_t[rb * a.ldst + c + j] = s[j].scale;
            }
        }
        // Turn the tile: 8 bytes of each of this thread's columns.
        uint2 *const pieces = reinterpret_cast<uint2 *>(turned);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint2 o;
            o.x = to_e4m3x4(v[0][j] * s[j].inv, v[1][j] * s[j].inv, v[2][j] * s[j].inv, v[3][j] * s[j].inv);
            o.y = to_e4m3x4(v[4][j] * s[j].inv, v[5][j] * s[j].inv, v[6][j] * s[j].inv, v[7][j] * s[j].inv);
            pieces[(8 * x + j) * 16 + (y ^ x)] = o;
        }
        __syncthreads();
        const int64_t end = BLOCKS ? a.rows : a.row_blocks * kBlock;   // length of a transposed row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = threadIdx.x + 256 * i, col = n >> 3, piece = n & 7, cx = col >> 3;
            // Pieces 2p and 2p + 1 of the column lie side by side, swapped for odd cx.
            uint4 o = turned[col * 8 + (piece ^ (cx >> 1))];
            if (cx & 1) o = make_uint4(o.z, o.w, o.x, o.y);
            const int64_t cc = cb * kBlock + col, r = rb * kBlock + 16 * piece;
            if (cc < a.cols && r < end) *reinterpret_cast<uint4 *>(a.qt + e * a.stride_qt + cc * a.ldqt + r) = o;
        }
        __syncthreads();
    }
}

template <class T>
int vec_ok(const T *src, int64_t ld, int64_t stride)
{
    const int64_t per16 = 16 / (int64_t)sizeof(T);
    return ((reinterpret_cast<uintptr_t>(src) & 15) == 0 && ld % per16 == 0 && stride % per16 == 0) ? 1 : 0;
}

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

template <class T, bool BLOCKS>
cudaError_t launch_tiles(TileArgs &a, int num_sms, cudaStream_t stream)
{
    a.vec = vec_ok(static_cast<const T *>(a.src), a.ld, a.batch > 1 ? a.stride_src : 0);
    const int64_t tiles = a.row_blocks * a.col_blocks * a.batch, most = (int64_t)num_sms * 2;
    quantize_tiles_kernel<T, BLOCKS><<<(unsigned)(tiles < most ? tiles : most), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                 const int32_t *gather, int64_t src_rows, uint8_t *q, int64_t ldq, float *scales,
                                 int64_t lds, int, cudaStream_t stream)
{
    const dim3 grid((unsigned)((rows + kRowsPerCta - 1) / kRowsPerCta),
                    (unsigned)((blocks_of(cols) + kBlocksPerCta - 1) / kBlocksPerCta));
    if (bf16) {
        const __nv_bfloat16 *s = static_cast<const __nv_bfloat16 *>(src);
        quantize_rows_kernel<<<grid, 256, 0, stream>>>(rows, cols, s, ld, gather, src_rows, q, ldq, scales, lds, vec_ok(s, ld, 0));
    } else {
        const float *s = static_cast<const float *>(src);
        quantize_rows_kernel<<<grid, 256, 0, stream>>>(rows, cols, s, ld, gather, src_rows, q, ldq, scales, lds, vec_ok(s, ld, 0));
    }
    return cudaGetLastError();
}

cudaError_t launch_quantize_cols(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                 const int32_t *gather, int64_t src_rows, int groups, const int32_t *offsets,
                                 int64_t padded, uint8_t *q, int64_t ldq, float *scales, int64_t lds, uint8_t *qt,
                                 int64_t ldqt, float *scales_t, int64_t ldst, int num_sms, cudaStream_t stream)
{
    TileArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.src = src;
    a.ld = ld;
    a.gather = gather;
    a.src_rows = src_rows;
    a.groups = offsets ? groups : 0;
    a.offsets = offsets;
    a.row_blocks = padded / kBlock;
    a.col_blocks = blocks_of(cols);
    a.batch = 1;
    a.q = q;
    a.ldq = ldq;
    a.scales = scales;
    a.lds = lds;
    a.qt = qt;
    a.ldqt = ldqt;
    a.scales_t = scales_t;
    a.ldst = ldst;
    return bf16 ? launch_tiles<__nv_bfloat16, false>(a, num_sms, stream) : launch_tiles<float, false>(a, num_sms, stream);
}

cudaError_t launch_quantize_blocks(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                   int64_t stride_src, bool transpose, uint8_t *q, int64_t ldq, int64_t stride_q,
                                   float *scales, int64_t lds, int64_t stride_s, int64_t batch, int num_sms,
                                   cudaStream_t stream)
{
    TileArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.src = src;
    a.ld = ld;
    a.stride_src = stride_src;
    a.src_rows = rows;
    a.row_blocks = blocks_of(rows);
    a.col_blocks = blocks_of(cols);
    a.batch = batch;
    if (transpose) {
        a.qt = q;
        a.ldqt = ldq;
        a.stride_qt = stride_q;
        a.scales_t = scales;
        a.ldst = lds;
        a.stride_st = stride_s;
    } else {
        a.q = q;
        a.ldq = ldq;
        a.stride_q = stride_q;
        a.scales = scales;
        a.lds = lds;
        a.stride_s = stride_s;
    }
    return bf16 ? launch_tiles<__nv_bfloat16, true>(a, num_sms, stream) : launch_tiles<float, true>(a, num_sms, stream);
}

}  // namespace sgemm_gb300
