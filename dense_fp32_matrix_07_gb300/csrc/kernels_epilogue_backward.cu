// Gradient of the 16-bit products' epilogue, C = act(z) [* D], z = A.B + bias:
//
//   dz = g act'(z) [* D],   dD = g act(z),   db[n] = sum over a group's rows of dz[., n]
//
// g, z and D are read once, dz and dD written once. A block takes 32 to 256
// rows of one group by 256 columns at a time, a warp every eighth of the rows,
// a lane eight columns, whose sums it keeps; the block's sums go to scratch,
// and a second launch adds each group's in order (no atomics: the result does
// not depend on timing). db sums the unrounded dz, in FP32. Measured on one
// GB300 in a row of calls, bfloat16: 8191 x 4096 with gelu and the bias gradient
// 48 us (4.2 TB/s; DRAM 51 % busy, issue slots 66 %), with silu and a factor 54
// (6.2 TB/s), 60 with the bias gradient; 16 groups of 16383 x 2048 with those 57
// and 65. Rows off 16 bytes go a value at a time: 8191 x 4095 105 and 156; FP32
// takes 39 and 54 for half of the rows, 40 and 124 of 4095 columns.
#include "layers.cuh"
#include "ptx.cuh"
#include "tc_roles.cuh"

namespace sgemm_gb300 {

namespace {

constexpr int kCols = 256;    // columns of a block's unit: 32 lanes, 8 each

template <class T>
struct Params {
    int64_t rows, cols;
    const T *g, *z, *D;
    int64_t ld_g, ld_z, ldd;
    int groups;
    const int32_t *offsets;
    T *dz, *dD;
    int64_t ld_dz, ld_dD;
    float *parts;             // sums of each unit of rows, or null
    int unit_rows;            // rows of a block's unit
    int units;                // units of rows, at most
    int strips;               // of kCols columns
};

__device__ __forceinline__ void group_rows(const int32_t *offsets, int64_t rows, int g, int64_t &lo, int64_t &hi)
{
    if (!offsets) {
        lo = 0, hi = rows;
        return;
    }
    int first, end;
    group_range(offsets, g, (int)rows, first, end);
    lo = first, hi = end;
}

__device__ __forceinline__ int group_units(const int32_t *offsets, int groups, int64_t rows, int unit_rows, int g)
{
    if (g >= groups) return 0;
    int64_t lo, hi;
    group_rows(offsets, rows, g, lo, hi);
    return (int)((hi - lo + unit_rows - 1) / unit_rows);
}

// table[g] = units of the groups before g, held to `units` (offsets that are
// not a partition may sum to anything). By one block of 256 threads, two
// groups each.
static_assert(kMaxGroups <= 512, "two groups per thread");

__device__ void fill_table(int *table, const int32_t *offsets, int groups, int64_t rows, int unit_rows, int units)
{
    __shared__ int64_t ends[8];
    const int g = 2 * threadIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int first = group_units(offsets, groups, rows, unit_rows, g);
    const int64_t mine = (int64_t)first + group_units(offsets, groups, rows, unit_rows, g + 1);
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
    }
    if (lane == 31) ends[warp] = sum;
    __syncthreads();
    int64_t before = sum - mine;
#pragma unroll
    for (int w = 0; w < 8; ++w)
        if (w < warp) before += ends[w];
    auto held = [&](int64_t n) { return (int)(n < units ? n : units); };
    if (g <= groups) table[g] = held(before);
    if (g + 1 <= groups) table[g + 1] = held(before + first);
    if (threadIdx.x == 255 && groups == 512) table[512] = held(before + mine);
    __syncthreads();
}

// act(z) and its slope. (Where gelu_tanh's sigmoid is 0 or 1 the polynomial
// beside it may be infinite.)
template <int ACT>
__device__ __forceinline__ float2 act_and_slope(float z)
{
    if constexpr (ACT == kActRelu) {
        return make_float2(z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z);
    } else if constexpr (ACT == kActGelu) {
        float e;
        const float phi = normal_integral(z, e);
        return make_float2(z * phi, fmaf(0.39894228040143268f * z, e, phi));
    } else if constexpr (ACT == kActGeluTanh) {
        const float s = sigmoid(tanh_argument(z)), edge = s * (1.0f - s);
        const float rise = 1.59576912160573071f * fmaf(0.134145f * z, z, 1.0f);
        return make_float2(z * s, edge > 0.0f ? fmaf(z * edge, rise, s) : s + edge);
    } else if constexpr (ACT == kActSilu) {
        const float s = sigmoid(z);
        return make_float2(z * s, s * fmaf(z, 1.0f - s, 1.0f));
    } else {
        return make_float2(z, 1.0f);
    }
}

// Columns of a lane: eight neighbours, by 16-byte accesses (VEC), or eight that
// are 32 apart, one at a time.
template <bool VEC>
__device__ __forceinline__ int column(int lane, int e) { return VEC ? 8 * lane + e : lane + 32 * e; }

// The lane's eight values of a row as they are stored, and back.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T *row, int lane, int cols, Raw8<T> &v)
{
    if constexpr (VEC) {
        v.load(row + 8 * lane);
    } else {
        T x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            store_from_float(&x[e], lane + 32 * e < cols ? load_as_float(row + lane + 32 * e) : 0.0f);
        v.load_some(x, 0, 8);
    }
}

template <class T, bool VEC>
__device__ __forceinline__ void put8(T *row, int lane, int cols, const float (&v)[8])
{
    if constexpr (VEC) {
        store8(row + 8 * lane, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < cols) store_from_float(row + lane + 32 * e, v[e]);
    }
}

// A warp's rows r, r + 8, .. below hi of a unit's columns from c0 on, and their sums.
template <class T, bool VEC, int ACT, bool MUL>
__device__ __forceinline__ void run_rows(const Params<T> &p, int64_t r, int64_t hi, int64_t c0, int cols, int lane,
                                         float (&sum)[8])
{
    if (VEC && 8 * lane >= cols) return;
    // Rows requested together: of one at a time, most of the time is a wait
    // for memory (8191 x 4096 bfloat16, gelu: 89 us).
    constexpr int BATCH = VEC && sizeof(T) == 2 ? 4 : 2;
    const T *g_at = p.g + r * p.ld_g + c0, *z_at = p.z ? p.z + r * p.ld_z + c0 : nullptr,
            *d_at = MUL ? p.D + r * p.ldd + c0 : nullptr;
    T *dz_at = p.dz ? p.dz + r * p.ld_dz + c0 : nullptr, *dD_at = p.dD ? p.dD + r * p.ld_dD + c0 : nullptr;
#pragma unroll 1
    for (; r < hi; r += 8 * BATCH) {
        Raw8<T> g[BATCH], z[BATCH], d[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (r + 8 * i >= hi) continue;
            load8<T, VEC>(g_at + 8 * i * p.ld_g, lane, cols, g[i]);
            if (z_at) load8<T, VEC>(z_at + 8 * i * p.ld_z, lane, cols, z[i]);
            else z[i].zero();
            if (MUL) load8<T, VEC>(d_at + 8 * i * p.ldd, lane, cols, d[i]);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (r + 8 * i >= hi) continue;
            float o[8], v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float up = g[i].get(e);
                const float2 a = act_and_slope<ACT>(z[i].get(e));
                o[e] = MUL ? up * a.x : 0.0f;
                v[e] = ACT != kActNone ? up * a.y : up;
                if (MUL) v[e] *= d[i].get(e);
                sum[e] += v[e];
            }
            if (dz_at) put8<T, VEC>(dz_at + 8 * i * p.ld_dz, lane, cols, v);
            if (MUL && dD_at) put8<T, VEC>(dD_at + 8 * i * p.ld_dD, lane, cols, o);
        }
        g_at += 8 * BATCH * p.ld_g;
        if (z_at) z_at += 8 * BATCH * p.ld_z;
        if (MUL) d_at += 8 * BATCH * p.ldd;
        if (dz_at) dz_at += 8 * BATCH * p.ld_dz;
        if (dD_at) dD_at += 8 * BATCH * p.ld_dD;
    }
}

// vec: rows are in whole 16-byte pieces, which holds for a unit whose columns
// are a multiple of eight.
template <class T, int ACT, bool MUL>
__global__ void __launch_bounds__(256, 2)
epilogue_backward_kernel(const __grid_constant__ Params<T> p, const bool vec)
{
    __shared__ int table[kMaxGroups + 1];
    __shared__ float sums[8][kCols];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (p.offsets) fill_table(table, p.offsets, p.groups, p.rows, p.unit_rows, p.units);
    const int units = p.offsets ? table[p.groups] : p.units;
    const int64_t all = (int64_t)units * p.strips;
    for (int64_t t = blockIdx.x; t < all; t += gridDim.x) {
        const int unit = (int)(t / p.strips), strip = (int)(t % p.strips);
        int64_t lo = 0, hi = p.rows;
        int first = unit;
        if (p.offsets) {
            int a = 0, b = p.groups - 1;
            while (a < b) {
                const int mid = (a + b + 1) / 2;
                if (table[mid] <= unit) a = mid;
                else b = mid - 1;
            }
            first = unit - table[a];
            group_rows(p.offsets, p.rows, a, lo, hi);
        }
        lo += (int64_t)first * p.unit_rows;
        hi = lo + p.unit_rows < hi ? lo + p.unit_rows : hi;
        const int64_t c0 = (int64_t)strip * kCols;
        const int cols = (int)(p.cols - c0 < kCols ? p.cols - c0 : kCols);
        float sum[8] = {};
        const bool whole = vec && cols % 8 == 0;
        if (whole) run_rows<T, true, ACT, MUL>(p, lo + warp, hi, c0, cols, lane, sum);
        else run_rows<T, false, ACT, MUL>(p, lo + warp, hi, c0, cols, lane, sum);
        if (p.parts) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[warp][whole ? column<true>(lane, e) : column<false>(lane, e)] = sum[e];
            __syncthreads();
            if ((int)threadIdx.x < cols) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
                p.parts[(int64_t)unit * p.cols + c0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// db[g][c] = sum of the parts of group g's units, in order within interleaved
// runs, a warp each (32 at most; a choice by the sizes alone). Its launch
// overlaps the end of the kernel before, for whose end it waits.
__global__ void __launch_bounds__(1024)
add_units_kernel(const float *parts, int64_t rows, int64_t cols, int groups, const int32_t *offsets, int unit_rows, int units,
                 float *grad_bias, int64_t stride)
{
    __shared__ int64_t counts[32];
    __shared__ float sums[32][33];
    const int lane = threadIdx.x % 32, run = threadIdx.x / 32, g = blockIdx.y, runs = blockDim.x / 32;
    ptx::grid_dependency_wait();
    int u0 = 0, u1 = units;
    if (offsets) {
        // The units of the groups before.
        int64_t n = 0;
        for (int i = threadIdx.x; i < g; i += blockDim.x) n += group_units(offsets, groups, rows, unit_rows, i);
#pragma unroll
        for (int d = 16; d; d /= 2) n += __shfl_xor_sync(0xffffffffu, n, d);
        if (lane == 0) counts[run] = n;
        __syncthreads();
        n = lane < runs ? counts[lane] : 0;
#pragma unroll
        for (int d = 16; d; d /= 2) n += __shfl_xor_sync(0xffffffffu, n, d);
        u0 = (int)(n < units ? n : units);
        n += group_units(offsets, groups, rows, unit_rows, g);
        u1 = (int)(n < units ? n : units);
    }
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int u = u0 + run; u < u1; u += runs) s += parts[(int64_t)u * cols + c];
    }
    sums[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < cols) {
        for (int i = 1; i < runs; ++i) s += sums[i][lane];
        grad_bias[g * stride + c] = s;
    }
}

// Rows of a unit: many, for few sums to be stored and added, where there are
// units for six turns of all SMs, two blocks in each; with fewer the last turn
// counts (8191 x 4096 gelu: 64 rows 48 us, 128 rows 50).
int unit_rows_of(const EpilogueBackwardArgs &g)
{
    const int64_t strips = (g.cols + kCols - 1) / kCols, enough = 12 * (int64_t)g.num_sms;
    int n = 256;
    while (n > 32 && g.rows / n * strips < enough) n /= 2;
    return n;
}

// Units of rows at most: each group's last may be short.
int64_t most_units(const EpilogueBackwardArgs &g)
{
    const int n = unit_rows_of(g);
    if (!g.offsets) return (g.rows + n - 1) / n;
    return g.rows / n + (g.groups < g.rows ? g.groups : g.rows);
}

template <class T>
cudaError_t backward_of(const EpilogueBackwardArgs &g, void *scratch, cudaStream_t stream)
{
    constexpr int64_t per16 = 16 / (int64_t)sizeof(T);
    Params<T> p{};
    p.rows = g.rows, p.cols = g.cols;
    p.g = static_cast<const T *>(g.grad_out), p.ld_g = g.ld_go;
    const bool uses_z = g.act != kActNone || g.grad_D;
    p.z = uses_z ? static_cast<const T *>(g.pre) : nullptr, p.ld_z = g.ld_pre;
    p.D = static_cast<const T *>(g.D), p.ldd = g.ldd;
    p.groups = g.groups, p.offsets = g.offsets;
    p.dz = static_cast<T *>(g.grad_pre), p.ld_dz = g.ld_gp;
    p.dD = static_cast<T *>(g.grad_D), p.ld_dD = g.ld_gd;
    p.parts = g.grad_bias ? static_cast<float *>(scratch) : nullptr;
    p.unit_rows = unit_rows_of(g);
    p.units = (int)most_units(g);
    p.strips = (int)((g.cols + kCols - 1) / kCols);
    const bool vec = pieces16(p.g, p.ld_g, per16) && pieces16(p.z, p.ld_z, per16) && pieces16(p.dz, p.ld_dz, per16) &&
                     pieces16(p.dD, p.ld_dD, per16) && (g.join != kJoinMul || pieces16(p.D, p.ldd, per16));
    if (p.units > 0) {
        const int64_t all = (int64_t)p.units * p.strips, most = (int64_t)g.num_sms * 8;
        const unsigned grid = (unsigned)(all < most ? all : most);
        auto launch = [&](auto a) {
            if (g.join == kJoinMul) epilogue_backward_kernel<T, decltype(a)::value, true><<<grid, 256, 0, stream>>>(p, vec);
            else epilogue_backward_kernel<T, decltype(a)::value, false><<<grid, 256, 0, stream>>>(p, vec);
        };
        using std::integral_constant;
        switch (g.act) {
        case kActRelu: launch(integral_constant<int, kActRelu>{}); break;
        case kActGelu: launch(integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: launch(integral_constant<int, kActGeluTanh>{}); break;
        case kActSilu: launch(integral_constant<int, kActSilu>{}); break;
        default: launch(integral_constant<int, kActNone>{});
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (g.grad_bias) {
        const dim3 grid((unsigned)((g.cols + 31) / 32), (unsigned)g.groups);
        const int64_t each = p.units / g.groups;
        const unsigned runs = each > 64 ? 32 : each > 16 ? 8 : 4;
        return launch_after(add_units_kernel, grid, dim3(32 * runs), stream, (const float *)p.parts, g.rows, g.cols, g.groups,
                            g.offsets, p.unit_rows, p.units, g.grad_bias, g.stride_gb);
    }
    return cudaSuccess;
}

}  // namespace

size_t epilogue_backward_scratch_bytes(const EpilogueBackwardArgs &g)
{
    return g.grad_bias ? (size_t)most_units(g) * (size_t)g.cols * 4 : 0;
}

cudaError_t launch_epilogue_backward(const EpilogueBackwardArgs &g, void *scratch, cudaStream_t stream)
{
    return g.bf16 ? backward_of<__nv_bfloat16>(g, scratch, stream) : backward_of<float>(g, scratch, stream);
}

}  // namespace sgemm_gb300
