// Quantisation to e4m3 with one scale per block of 128 values (along a row,
// along a column within a group of rows, or 128 x 128):
//
//   a = max(max |x| over the block, 2^-96),  scale = a / 448,
//   q = e4m3(x * (448 / a))   (round to nearest even, saturating)
//
// A block with a NaN gets a NaN scale and NaN values; one with an infinity an
// infinite scale, zeros for its finite values and NaN for the infinity.
// Each value is read once and written as one byte per form. Measured on one
// GB300: 16383 x 4096 bfloat16 values along rows 36.4 us (5.5 TB/s: memory);
// along rows and, transposed, along 16 groups of rows 55 us (5.0 TB/s),
// bound by instructions as much as by memory (about 700 per warp and tile:
// conversions, and two products, two maxima per value); 8192 x 4096 in 128 x
// 128 blocks and their transposes 40 us for the two calls.
#include "experts.cuh"
#include "fp8_values.cuh"

namespace sgemm_gb300 {

namespace {

// Eight consecutive values of a row as they are stored: pairs of bfloat16 in
// four registers, or eight floats.
template <class T>
struct Eight;

template <>
struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const float *p)
    {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(int j, const float *p) { v[j] = *p; }
    __device__ __forceinline__ float2 pair(int j) const { return make_float2(v[2 * j], v[2 * j + 1]); }
    // Magnitude bits of pair j, as one or two numbers packed for max_of().
    __device__ __forceinline__ uint2 mags(int j) const { return make_uint2(magnitude(v[2 * j]), magnitude(v[2 * j + 1])); }
    static __device__ __forceinline__ uint2 max_of(uint2 a, uint2 b, uint2 c)
    {
        return make_uint2(__vimax3_u32(a.x, b.x, c.x), __vimax3_u32(a.y, b.y, c.y));
    }
    static __device__ __forceinline__ uint32_t first(uint2 m) { return m.x; }
    static __device__ __forceinline__ uint32_t second(uint2 m) { return m.y; }
};

template <>
struct Eight<__nv_bfloat16> {
    uint32_t v[4];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = 0;
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    }
    __device__ __forceinline__ void set(int j, const __nv_bfloat16 *p)
    {
        const uint32_t x = *reinterpret_cast<const uint16_t *>(p);
        v[j / 2] |= (j & 1) ? x << 16 : x;
    }
    __device__ __forceinline__ float2 pair(int j) const
    {
        return make_float2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xffff0000u));
    }
    __device__ __forceinline__ uint32_t mags(int j) const { return v[j] & 0x7fff7fffu; }
    static __device__ __forceinline__ uint32_t max_of(uint32_t a, uint32_t b, uint32_t c) { return __vimax3_u16x2(a, b, c); }
    static __device__ __forceinline__ uint32_t first(uint32_t m) { return m << 16; }
    static __device__ __forceinline__ uint32_t second(uint32_t m) { return m & 0xffff0000u; }
};

// Values c .. c + 7 of a row of `cols`, zeros past its end.
template <class T>
__device__ __forceinline__ void load_row(const T *row, int64_t c, int64_t cols, bool vec, Eight<T> &x)
{
    if (vec && c + 8 <= cols) {
        x.load(row + c);
        return;
    }
    x.zero();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < cols) x.set(j, row + c + j);
}

// Largest magnitude of the eight.
template <class T>
__device__ __forceinline__ uint32_t max_of_eight(const Eight<T> &x)
{
    const auto last = x.mags(3), m = Eight<T>::max_of(Eight<T>::max_of(x.mags(0), x.mags(1), x.mags(2)), last, last);
    return umax(Eight<T>::first(m), Eight<T>::second(m));
}

// The eight times inv, as eight bytes.
template <class T>
__device__ __forceinline__ uint2 eight_bytes(const Eight<T> &x, float inv)
{
    const float2 f = make_float2(inv, inv);
    const float2 a = __fmul2_rn(x.pair(0), f), b = __fmul2_rn(x.pair(1), f), c = __fmul2_rn(x.pair(2), f),
                 d = __fmul2_rn(x.pair(3), f);
    return make_uint2(to_e4m3x4(a.x, a.y, b.x, b.y), to_e4m3x4(c.x, c.y, d.x, d.y));
}

// Maxima over the 16 lanes of a half warp of N values each (N = 8 or 4), one
// of them per lane in the end: halves of the values are traded with the lanes
// 8, 4, ... away, so that this takes N shuffles instead of 4 N, and the two
// divisions of a scale are done once per value instead of by all 16 lanes.
// Lane l of the half holds value l / (16 / N).
template <int N>
__device__ __forceinline__ uint32_t max_over_half(uint32_t (&m)[N], int lane)
{
    int d = 8;
#pragma unroll
    for (int n = N; n > 1; n /= 2, d /= 2) {
        const bool upper = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const uint32_t keep = upper ? m[i + n / 2] : m[i], give = upper ? m[i] : m[i + n / 2];
            m[i] = umax(keep, __shfl_xor_sync(0xffffffffu, give, d));
        }
    }
#pragma unroll
    for (; d > 0; d /= 2) m[0] = umax(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
    return m[0];
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
    Eight<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 2 * warp + (i >> 1), b = b0 + half + 2 * (i & 1);
        int64_t from = -1;
        if (r < rows) from = gather ? (int64_t)gather[r] : r;
        if (from >= 0 && from < src_rows && b < nb)
            load_row<T>(src + from * ld, b * kBlock + 8 * l, cols, vec != 0, v[i]);
        else
            v[i].zero();
    }
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max_of_eight(v[i]);
    const Scale s = scale_of(max_over_half<4>(m, lane));       // of block l / 4
    if ((l & 3) == 0) tile[half + 2 * ((l >> 2) & 1)][2 * warp + (l >> 3)] = s.scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 2 * warp + (i >> 1), c = (b0 + half + 2 * (i & 1)) * kBlock + 8 * l;
        const float inv = __shfl_sync(0xffffffffu, s.inv, (lane & 16) | (4 * i));
        if (r < rows && c < cols) *reinterpret_cast<uint2 *>(q + r * ldq + c) = eight_bytes(v[i], inv);
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
// conflicts. Each scale's divisions are done by one thread.
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
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
quantize_tiles_kernel(const TileArgs a)
{
    __shared__ uint32_t red[8][128];
    __shared__ float4 inv_of[32];                     // 448 / a of the 128 columns
    __shared__ uint4 turned[128 * 8];
    __shared__ int table[BLOCKS ? 1 : kMaxGroups + 2], begins[BLOCKS ? 1 : kMaxGroups], ends[BLOCKS ? 1 : kMaxGroups];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!BLOCKS && a.groups > 0) {
        // table[g] = blocks of the groups before g; group g's rows are
        // [begins[g], ends[g]), held to the rows there are.
        const int rows = (int)a.rows;
        for (int g = threadIdx.x; g < a.groups; g += 256) {
            const int o0 = a.offsets[g], o1 = a.offsets[g + 1];
            const int lo = o0 < 0 ? 0 : o0 > rows ? rows : o0;
            const int hi = o1 < lo ? lo : o1 > rows ? rows : o1;
            begins[g] = lo;
            ends[g] = hi;
            table[g] = (hi - lo + kBlock - 1) / kBlock;
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
    const uint32_t col_blocks = (uint32_t)a.col_blocks, per = (uint32_t)a.row_blocks * col_blocks;
    const uint32_t tiles = per * (uint32_t)a.batch;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const uint32_t in = BLOCKS ? t % per : t, row_block = in / col_blocks;
        const int64_t e = BLOCKS ? t / per : 0, rb = row_block, cb = in - row_block * col_blocks;
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
                r0 = begins[lo] + (rb - table[lo]) * kBlock;
                r1 = r0 + kBlock < ends[lo] ? r0 + kBlock : ends[lo];
            }
        }
        const T *src = static_cast<const T *>(a.src) + e * a.stride_src;
        const int64_t c = cb * kBlock + 8 * x;
        const int64_t ry = r0 + 8 * y;               // this thread's first row
        const int n = (int)(r1 - ry);                // its rows: those below n
        Eight<T> v[8];
        if (!a.gather && a.vec && c + 8 <= a.cols) {
            const T *p = src + ry * a.ld + c;
#pragma unroll
            for (int i = 0; i < 8; ++i, p += a.ld) {
                if (i < n)
                    v[i].load(p);
                else
                    v[i].zero();
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int64_t from = -1;
                if (i < n) from = a.gather ? (int64_t)a.gather[ry + i] : ry + i;
                if (from >= 0 && from < a.src_rows)
                    load_row<T>(src + from * a.ld, c, a.cols, a.vec != 0, v[i]);
                else
                    v[i].zero();
            }
        }
        if (!BLOCKS && a.q) {
            // Row form: a row's 128 columns are the 16 lanes of a half warp.
            uint32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = max_of_eight(v[i]);
            const Scale s = scale_of(max_over_half<8>(m, lane));   // of row x / 2
            if ((x & 1) == 0 && (x >> 1) < n) a.scales[cb * a.lds + ry + (x >> 1)] = s.scale;
            uint8_t *q = a.q + ry * a.ldq + c;
            const int nq = c < a.cols ? n : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i, q += a.ldq) {
                const float inv = __shfl_sync(0xffffffffu, s.inv, (lane & 16) | (2 * i));
                if (i < nq) *reinterpret_cast<uint2 *>(q) = eight_bytes(v[i], inv);
            }
        }
        // Columns' (or the block's) largest magnitudes.
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            auto p = Eight<T>::max_of(v[0].mags(j), v[1].mags(j), v[2].mags(j));
            p = Eight<T>::max_of(p, v[3].mags(j), v[4].mags(j));
            p = Eight<T>::max_of(p, v[5].mags(j), v[6].mags(j));
            const auto last = v[7].mags(j);
            p = Eight<T>::max_of(p, last, last);
            m[2 * j] = Eight<T>::first(p);
            m[2 * j + 1] = Eight<T>::second(p);
        }
        float inv[8];
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
            const Scale s = scale_of(all);
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = s.inv;
            if (threadIdx.x == 0) {
                if (a.q)
                    a.scales[e * a.stride_s + rb * a.lds + cb] = s.scale;
                else
                    a.scales_t[e * a.stride_st + cb * a.ldst + rb] = s.scale;
            }
            if (a.q) {
                uint8_t *q = a.q + e * a.stride_q + ry * a.ldq + c;
                const int nq = c < a.cols ? n : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i, q += a.ldq)
                    if (i < nq) *reinterpret_cast<uint2 *>(q) = eight_bytes(v[i], s.inv);
                continue;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = umax(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
            // The last tile's reads of `red` and `turned` are behind the barriers that ended it.
            if (lane < 16) {
                *reinterpret_cast<uint4 *>(&red[warp][8 * x]) = make_uint4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<uint4 *>(&red[warp][8 * x + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
            }
            __syncthreads();
            if (threadIdx.x < 128) {
                uint32_t all = 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) all = umax(all, red[w][threadIdx.x]);
                const Scale s = scale_of(all);
                reinterpret_cast<float *>(inv_of)[threadIdx.x] = s.inv;
                const int64_t col = cb * kBlock + threadIdx.x;
                if (col < a.cols) a.scales_t[rb * a.ldst + col] = s.scale;
            }
            __syncthreads();
            const float4 lo = inv_of[2 * x], hi = inv_of[2 * x + 1];
            inv[0] = lo.x, inv[1] = lo.y, inv[2] = lo.z, inv[3] = lo.w;
            inv[4] = hi.x, inv[5] = hi.y, inv[6] = hi.z, inv[7] = hi.w;
        }
        // Turn the tile: 8 bytes of each of this thread's columns.
        uint2 *const pieces = reinterpret_cast<uint2 *>(turned);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = make_float2(inv[2 * j], inv[2 * j + 1]);
            float2 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = __fmul2_rn(v[i].pair(j), f);
            pieces[(8 * x + 2 * j) * 16 + (y ^ x)] =
                make_uint2(to_e4m3x4(p[0].x, p[1].x, p[2].x, p[3].x), to_e4m3x4(p[4].x, p[5].x, p[6].x, p[7].x));
            pieces[(8 * x + 2 * j + 1) * 16 + (y ^ x)] =
                make_uint2(to_e4m3x4(p[0].y, p[1].y, p[2].y, p[3].y), to_e4m3x4(p[4].y, p[5].y, p[6].y, p[7].y));
        }
        __syncthreads();
        const int64_t end = BLOCKS ? a.rows : a.row_blocks * kBlock;   // length of a transposed row
        {
            // This thread: piece threadIdx.x % 8 of columns threadIdx.x / 8 + 32 i.
            const int piece = threadIdx.x & 7, col0 = threadIdx.x >> 3;
            const int64_t r = rb * kBlock + 16 * piece;
            const int left = r < end ? (int)(a.cols - cb * kBlock < kBlock ? a.cols - cb * kBlock : kBlock) - col0 : 0;
            uint8_t *q = a.qt + e * a.stride_qt + (cb * kBlock + col0) * a.ldqt + r;
#pragma unroll
            for (int i = 0; i < 4; ++i, q += 32 * a.ldqt) {
                const int col = col0 + 32 * i, cx = col >> 3;
                // Pieces 2p and 2p + 1 of the column lie side by side, swapped for odd cx.
                uint4 o = turned[col * 8 + (piece ^ (cx >> 1))];
                if (cx & 1) o = make_uint4(o.z, o.w, o.x, o.y);
                if (32 * i < left) *reinterpret_cast<uint4 *>(q) = o;
            }
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
    // Tiles are counted in 32 bits (2^31 of them would be 2^45 values).
    if ((__int128)a.row_blocks * a.col_blocks * a.batch > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t tiles = a.row_blocks * a.col_blocks * a.batch, most = (int64_t)num_sms * (sizeof(T) == 2 ? 4 : 2);
    quantize_tiles_kernel<T, BLOCKS><<<(unsigned)(tiles < most ? tiles : most), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t rows, int64_t cols, const void *src, bool bf16, int64_t ld,
                                 const int32_t *gather, int64_t src_rows, uint8_t *q, int64_t ldq, float *scales,
                                 int64_t lds, cudaStream_t stream)
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
