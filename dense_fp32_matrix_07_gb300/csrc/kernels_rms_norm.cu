// Root-mean-square norm of rows, with the residual's addition before it and
// 8-bit values after it, and its gradient:
//
//   s = x + residual,  i = 1 / sqrt(mean(s^2) + eps),  y = s i w
//   q, scales: y in the rows form (a scale per row and 128 columns)
//
//   h = s i,  ds = i (g w - h mean(g w h)) + gs,  dw = sum over rows of g h
//
// A row is held in registers by one warp (short rows) or one block, eight
// neighbouring columns to a thread, so that everything is read once and
// written once. Sums are in FP32; y and q come from the unrounded s, and each
// stored value is rounded once. The gradient takes s as it was stored and
// finds i again from it. Bound by memory; measured on one GB300 (in a row of
// calls): 8191 x 4096 bfloat16 with the residual, y and q 47 us (6.45 TB/s);
// the gradient of 16383 x 2048 with one along the residual 45.5 us (5.9 TB/s,
// issue slots 62 % busy), with the weights' 51: their sums per block go to
// scratch and a second, overlapped launch adds them in order. Above 4096 columns
// the gradient's rows do not fit the registers of their 1024 threads: 4095 x
// 8192 67 us (4.0 TB/s), 2047 x 16384 101 (2.7).
//
// Rows that do not begin on 16 bytes (an odd number of columns): where all
// matrices' rows lie alike, the threads' eights are shifted so that they begin
// on 16 bytes, and only the row's ends are single values (4097 x 3001 floats
// 32.6 -> 20.5 us). Else, and for 8-bit values, whose blocks of 128 columns are
// 16 lanes', rows pass through shared memory.
#include "fp8_values.cuh"
#include "layers.cuh"
#include "ptx.cuh"

#include <type_traits>

namespace sgemm_gb300 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// The threads that share a row: a warp each (WARPS = 1, eight rows a block) or
// the whole block.
template <int WARPS>
struct Team {
    static constexpr int SIZE = 32 * WARPS;
    static constexpr int ROWS = WARPS == 1 ? 8 : 1;
    static constexpr int THREADS = SIZE * ROWS;
    static __device__ __forceinline__ int rank() { return (int)threadIdx.x % SIZE; }
    static __device__ __forceinline__ int row() { return (int)threadIdx.x / SIZE; }
    static __device__ __forceinline__ void sync()
    {
        if constexpr (WARPS == 1) __syncwarp();
        else __syncthreads();
    }
    // The sums of a and of b over the team, in a fixed order; `turn` alternates
    // between calls, so that one barrier is enough.
    static __device__ __forceinline__ float2 sum(float2 v, int turn)
    {
#pragma unroll
        for (int d = 16; d; d /= 2) {
            v.x += __shfl_xor_sync(kAll, v.x, d);
            v.y += __shfl_xor_sync(kAll, v.y, d);
        }
        if constexpr (WARPS > 1) {
            __shared__ float2 part[2][WARPS];
            if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = v;
            __syncthreads();
            v = part[turn][threadIdx.x % WARPS];
#pragma unroll
            for (int d = WARPS / 2; d; d /= 2) {
                v.x += __shfl_xor_sync(kAll, v.x, d);
                v.y += __shfl_xor_sync(kAll, v.y, d);
            }
        }
        return v;
    }
};

// How a row's eights lie: kWhole on 16 bytes, kShifted on 16 bytes from a
// column before the first on, kStaged through shared memory.
enum Layout : int { kStaged = 0, kShifted = 1, kWhole = 2 };

// Columns of a thread's pack k: 8 from here on, `shift` before where they
// would begin.
template <int WARPS>
__device__ __forceinline__ int column(int k, int shift)
{
    return 8 * (Team<WARPS>::rank() + k * Team<WARPS>::SIZE) - shift;
}

// Values of a row before its first that lies on 16 bytes, taken from the 16
// bytes before.
template <class T, int LAYOUT>
__device__ __forceinline__ int shift_of(const T *row)
{
    return LAYOUT == kShifted ? (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)) : 0;
}

template <class T>
struct NormParams {
    int64_t rows;
    int cols;
    const T *x, *residual;
    const float *weight;
    float eps;
    T *sum, *y;
    uint8_t *q;
    float *scales;
    int64_t ldx, ld_res, ld_sum, ldy, ldq, lds;
    int weight16;      // the weights lie on 16 bytes
};

// Eight weights from column c on, zeros outside the row. (Where c is a
// multiple of 8 the compiler is told so: choosing among twelve for any c costs
// 24 instructions.)
template <int LAYOUT>
__device__ __forceinline__ void load_weight(const float *w, int c, int cols, bool whole16, float (&v)[8])
{
    const int off = LAYOUT == kShifted ? c & 3 : 0;
    if (whole16 && c >= 0 && c + (off ? 12 - off : 8) <= cols) {
        const float4 *at = reinterpret_cast<const float4 *>(w + (c - off));
        const float4 a = __ldg(at), b = __ldg(at + 1);
        float f[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (off) {
            const float4 d = __ldg(at + 2);
            f[8] = d.x, f[9] = d.y, f[10] = d.z, f[11] = d.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = off == 0 ? f[e] : off == 1 ? f[e + 1] : off == 2 ? f[e + 2] : f[e + 3 < 12 ? e + 3 : 0];
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e >= 0 && c + e < cols ? __ldg(w + c + e) : 0.0f;
}

// A thread's eights of a row, zeros outside it; kStaged: through `line`.
template <class T, int WARPS, int PACKS, int LAYOUT>
__device__ __forceinline__ void load_row(const T *row, int cols, int shift, T *line, Raw8<T> (&v)[PACKS])
{
    using Tm = Team<WARPS>;
    if constexpr (LAYOUT == kStaged) {
        Tm::sync();
#pragma unroll 4
        for (int c = Tm::rank(); c < (cols + 7) / 8 * 8; c += Tm::SIZE) store_from_float(line + c, c < cols ? load_as_float(row + c) : 0.0f);
        Tm::sync();
    }
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
        const int c = column<WARPS>(k, shift);
        if constexpr (LAYOUT != kStaged) {
            if (c >= 0 && c + 8 <= cols) v[k].load(row + c);
            else v[k].load_some(row + c, -c, cols - c);
        } else {
            if (c < cols) v[k].load(line + c);
            else v[k].zero();
        }
    }
}

// A thread's eight from column c on to a row (kStaged: to `line`).
template <class T, int LAYOUT>
__device__ __forceinline__ void store_pack(T *row, T *line, int c, int cols, const float (&v)[8])
{
    if constexpr (LAYOUT == kStaged) {
        if (c < cols) store8(line + c, v);
    } else if (c >= 0 && c + 8 <= cols) {
        store8(row + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e >= 0 && c + e < cols) store_from_float(row + c + e, v[e]);
    }
}

// kStaged: `line`, as the team has stored it, to a row.
template <class T, int WARPS>
__device__ __forceinline__ void store_line(T *row, const T *line, int cols)
{
    using Tm = Team<WARPS>;
    Tm::sync();
#pragma unroll 4
    for (int c = Tm::rank(); c < cols; c += Tm::SIZE) row[c] = line[c];
}

template <class T, int WARPS, int PACKS, int LAYOUT>
__global__ void __launch_bounds__(Team<WARPS>::THREADS)
rms_norm_kernel(const __grid_constant__ NormParams<T> p)
{
    using Tm = Team<WARPS>;
    extern __shared__ uint4 staging[];
    const int64_t r = (int64_t)blockIdx.x * Tm::ROWS + Tm::row();
    if (r >= p.rows) return;          // whole teams
    const int cols = p.cols, shift = shift_of<T, LAYOUT>(p.x + r * p.ldx);
    T *const line = reinterpret_cast<T *>(staging) + Tm::row() * ((cols + 7) / 8 * 8);
    float v[PACKS][8];
    {
        Raw8<T> x[PACKS], a[PACKS];
        load_row<T, WARPS, PACKS, LAYOUT>(p.x + r * p.ldx, cols, shift, line, x);
        if (p.residual) load_row<T, WARPS, PACKS, LAYOUT>(p.residual + r * p.ld_res, cols, shift, line, a);
#pragma unroll
        for (int k = 0; k < PACKS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = p.residual ? x[k].get(e) + a[k].get(e) : x[k].get(e);
    }
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < PACKS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss.x = fmaf(v[k][e], v[k][e], ss.x);
    // Every value of the row has been read: the sum may go where x or the residual was.
    const float inv = rsqrtf(Tm::sum(ss, 0).x / (float)cols + p.eps);

    if (p.sum) {
        T *const to = p.sum + r * p.ld_sum;
        if constexpr (LAYOUT == kStaged) Tm::sync();
#pragma unroll
        for (int k = 0; k < PACKS; ++k) store_pack<T, LAYOUT>(to, line, column<WARPS>(k, shift), cols, v[k]);
        if constexpr (LAYOUT == kStaged) {
            store_line<T, WARPS>(to, line, cols);
            Tm::sync();
        }
    }
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
        const int c = column<WARPS>(k, shift);
        if (p.weight) {
            float w[8];
            load_weight<LAYOUT>(p.weight, c, cols, p.weight16, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * inv * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= inv;
        }
        if (p.y) store_pack<T, LAYOUT>(p.y + r * p.ldy, line, c, cols, v[k]);
        if (LAYOUT != kShifted && p.q) {
            // A block of 128 columns lies in 16 neighbouring lanes.
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) most = umax(most, c + e < cols ? magnitude(v[k][e]) : 0u);
#pragma unroll
            for (int d = 8; d; d /= 2) most = umax(most, __shfl_xor_sync(kAll, most, d));
            if (c < cols) {
                const Scale s = scale_of(most);
                const uint2 b = make_uint2(
                    to_e4m3x4(v[k][0] * s.inv, v[k][1] * s.inv, v[k][2] * s.inv, v[k][3] * s.inv),
                    to_e4m3x4(v[k][4] * s.inv, v[k][5] * s.inv, v[k][6] * s.inv, v[k][7] * s.inv));
                *reinterpret_cast<uint2 *>(p.q + r * p.ldq + c) = b;
                if (c % kBlock == 0) p.scales[(int64_t)(c / kBlock) * p.lds + r] = s.scale;
            }
        }
    }
    if constexpr (LAYOUT == kStaged) {
        if (p.y) store_line<T, WARPS>(p.y + r * p.ldy, line, cols);
    }
}

template <class T>
struct NormBackwardParams {
    int64_t rows;
    int cols;
    const T *g, *x, *gs;
    const float *weight;
    float eps;
    T *dx;
    float *parts;      // one row of partial weight gradients per block, or null
    int64_t ld_g, ldx, ld_gs, ld_dx;
    int weight16;
};

// Blocks of the gradient's kernel in an SM: what their rows need in registers.
template <class T>
constexpr int backward_resident(int threads)
{
    const int all = sizeof(T) == 2 ? 768 : 512;
    return threads < all ? all / threads : 1;
}

template <class T, int WARPS, int PACKS, int LAYOUT>
__global__ void __launch_bounds__(Team<WARPS>::THREADS, backward_resident<T>(Team<WARPS>::THREADS))
rms_norm_backward_kernel(const __grid_constant__ NormBackwardParams<T> p)
{
    using Tm = Team<WARPS>;
    extern __shared__ uint4 staging[];
    const int cols = p.cols, padded = (cols + 7) / 8 * 8;
    T *const line = reinterpret_cast<T *>(staging) + Tm::row() * padded;
    // Shifted eights are other columns in every row: their weight gradients
    // are summed in shared memory, a row of them per team, column by column.
    float *const columns = reinterpret_cast<float *>(staging) + Tm::row() * padded;
    float dw[PACKS][8];
#pragma unroll
    for (int k = 0; k < PACKS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[k][e] = 0.0f;
    if (LAYOUT == kShifted && p.parts) {
        for (int c = Tm::rank(); c < padded; c += Tm::SIZE) columns[c] = 0.0f;
        Tm::sync();
    }
    // The weights of columns that stay the same stay in registers.
    constexpr bool KEEP = PACKS == 1 && LAYOUT != kShifted;
    float kept[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) kept[e] = 1.0f;
    if (KEEP && p.weight) load_weight<LAYOUT>(p.weight, column<WARPS>(0, 0), cols, p.weight16, kept);
    auto weights = [&](int c, float (&w)[8]) {
        if constexpr (!KEEP) {
            if (p.weight) {
                load_weight<LAYOUT>(p.weight, c, cols, p.weight16, w);
                return;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = kept[e];
    };
    int turn = 0;
    // Rows are requested one ahead (63 -> 57 us for 16383 x 2048 bfloat16 with
    // a gradient along the residual). A ring of rows in shared memory,
    // filled by asynchronous copies, took 56 for 49: the instructions per row
    // count, not the loads.
    constexpr bool AHEAD = LAYOUT != kStaged;
    const int64_t step = (int64_t)gridDim.x * Tm::ROWS;
    int64_t r = (int64_t)blockIdx.x * Tm::ROWS + Tm::row();
    Raw8<T> x[PACKS], g[PACKS], gs[PACKS];
    auto load = [&](int64_t r) {
        const int shift = shift_of<T, LAYOUT>(p.x + r * p.ldx);
        load_row<T, WARPS, PACKS, LAYOUT>(p.x + r * p.ldx, cols, shift, line, x);
        load_row<T, WARPS, PACKS, LAYOUT>(p.g + r * p.ld_g, cols, shift, line, g);
        if (p.gs) load_row<T, WARPS, PACKS, LAYOUT>(p.gs + r * p.ld_gs, cols, shift, line, gs);
    };
    if (AHEAD && r < p.rows) load(r);
    for (; r < p.rows; r += step, turn ^= 1) {
        if (!AHEAD) load(r);
        const int shift = shift_of<T, LAYOUT>(p.x + r * p.ldx);
        float2 s = make_float2(0.0f, 0.0f);
        Raw8<T> x0[PACKS], g0[PACKS], gs0[PACKS];
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            float w[8];
            weights(column<WARPS>(k, shift), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s.x = fmaf(x[k].get(e), x[k].get(e), s.x);
                s.y = fmaf(g[k].get(e) * w[e], x[k].get(e), s.y);
            }
            x0[k] = x[k], g0[k] = g[k];
            if (p.gs) gs0[k] = gs[k];
        }
        if (AHEAD && r + step < p.rows) load(r + step);
        s = Tm::sum(s, turn);
        const float inv = rsqrtf(s.x / (float)cols + p.eps);
        const float mean = s.y * inv / (float)cols;     // of g w h
        T *const to = p.dx + r * p.ld_dx;
        if constexpr (LAYOUT == kStaged) Tm::sync();
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = column<WARPS>(k, shift);
            float w[8], d[8];
            weights(c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = x0[k].get(e) * inv, gw = g0[k].get(e) * w[e];
                if constexpr (LAYOUT == kShifted) dw[k][e] = g0[k].get(e) * h;
                else dw[k][e] = fmaf(g0[k].get(e), h, dw[k][e]);
                d[e] = inv * (gw - h * mean);
                if (p.gs) d[e] += gs0[k].get(e);
            }
            store_pack<T, LAYOUT>(to, line, c, cols, d);
            if (LAYOUT == kShifted && p.parts) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e >= 0 && c + e < cols) columns[c + e] += dw[k][e];
            }
        }
        // The next row's sums are behind a barrier of the team's (in sum()).
        if constexpr (LAYOUT == kStaged) store_line<T, WARPS>(to, line, cols);
        if (LAYOUT == kShifted && WARPS == 1) __syncwarp();
    }
    if (!p.parts) return;
    float *const to = p.parts + (int64_t)blockIdx.x * cols;
    if constexpr (WARPS == 1) {
        // The eight rows' warps, in order.
        float *const all = reinterpret_cast<float *>(staging);
        __syncthreads();
        if constexpr (LAYOUT != kShifted) {
#pragma unroll
            for (int k = 0; k < PACKS; ++k) {
                const int c = column<WARPS>(k, 0);
                if (c < cols) store8(all + Tm::row() * padded + c, dw[k]);
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < cols; c += Tm::THREADS) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < Tm::ROWS; ++i) s += all[i * padded + c];
            to[c] = s;
        }
    } else if constexpr (LAYOUT == kShifted) {
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += Tm::THREADS) to[c] = columns[c];
    } else {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = column<WARPS>(k, 0);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) to[c + e] = dw[k][e];
        }
    }
}

// out[c] = sum of parts[.][c], in order within 32 interleaved runs. Its launch
// overlaps the end of the kernel before, for whose end it waits.
__global__ void __launch_bounds__(1024) add_parts_kernel(const float *parts, int count, int cols, float *out)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x % 32, run = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    ptx::grid_dependency_wait();
    if (c < cols) {
#pragma unroll 8
        for (int i = run; i < count; i += 32) s += parts[(int64_t)i * cols + c];
    }
    sums[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sums[i][lane];
        out[c] = s;
    }
}

struct Rows {
    const void *p;
    int64_t ld;
};

// How the rows of these matrices (null: none) can be accessed together.
template <class T, int N>
Layout layout_of(const Rows (&all)[N], bool shiftable)
{
    constexpr uint64_t per16 = 16 / sizeof(T);
    uint64_t phase = 0, ld = 0;
    bool first = true, alike = true;
    for (const Rows &m : all) {
        if (!m.p) continue;
        const uint64_t at = reinterpret_cast<uintptr_t>(m.p) / sizeof(T) % per16, step = (uint64_t)m.ld % per16;
        if (first) phase = at, ld = step;
        alike = alike && at == phase && step == ld;
        first = false;
    }
    return !alike ? kStaged : phase == 0 && ld == 0 ? kWhole : shiftable ? kShifted : kStaged;
}

// Calls f(Warps, Packs) with the shape of `cols` columns: forward few threads,
// so that several rows' loads are under way in an SM; the gradient, which
// holds several matrices' rows, one eight per thread.
template <bool FORWARD, class F>
cudaError_t with_shape(int64_t cols, F f)
{
    using std::integral_constant;
    auto call = [&](auto w, auto k) { return f(w, k); };
    if (cols <= 256) return call(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if constexpr (FORWARD) {
        if (cols <= 1024) return call(integral_constant<int, 1>{}, integral_constant<int, 4>{});
        if (cols <= 2048) return call(integral_constant<int, 4>{}, integral_constant<int, 2>{});
        if (cols <= 4096) return call(integral_constant<int, 8>{}, integral_constant<int, 2>{});
        if (cols <= 8192) return call(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    } else {
        if (cols <= 1024) return call(integral_constant<int, 4>{}, integral_constant<int, 1>{});
        if (cols <= 2048) return call(integral_constant<int, 8>{}, integral_constant<int, 1>{});
        if (cols <= 4096) return call(integral_constant<int, 16>{}, integral_constant<int, 1>{});
        if (cols <= 8192) return call(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    }
    return call(integral_constant<int, 32>{}, integral_constant<int, 2>{});
}

// Shared memory of a block whose rows pass through it. Up to 32 KB, except for
// rows of more than 8192 columns (32 warps, two eights each): these kernels are
// allowed their most once, by prepare_rms_norm(), as what a call set for
// itself another thread's call could undo before the launch.
constexpr int staging_bytes(int64_t cols, int rows) { return (int)((cols + 7) / 8 * 32 * rows); }

template <class T>
cudaError_t prepare_widest()
{
    constexpr int most = staging_bytes(kMaxNormCols, 1);
    cudaError_t e = cudaFuncSetAttribute(rms_norm_kernel<T, 32, 2, kStaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(rms_norm_backward_kernel<T, 32, 2, kStaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(rms_norm_backward_kernel<T, 32, 2, kShifted>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e;
}

template <class K>
cudaError_t launch(K kernel, unsigned grid, int threads, int bytes, const void *params, cudaStream_t stream)
{
    void *args[] = {const_cast<void *>(params)};
    const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(threads), args,
                                           (size_t)bytes, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <class T>
cudaError_t norm_of(const RmsNormArgs &g, cudaStream_t stream)
{
    NormParams<T> p{};
    p.rows = g.rows, p.cols = (int)g.cols;
    p.x = static_cast<const T *>(g.x), p.ldx = g.ldx;
    p.residual = static_cast<const T *>(g.residual), p.ld_res = g.ld_res;
    p.weight = g.weight, p.eps = g.eps;
    p.weight16 = (reinterpret_cast<uintptr_t>(g.weight) & 15u) == 0;
    p.sum = static_cast<T *>(g.sum), p.ld_sum = g.ld_sum;
    p.y = static_cast<T *>(g.y), p.ldy = g.ldy;
    p.q = g.q, p.ldq = g.ldq, p.scales = g.scales, p.lds = g.lds;
    const Rows all[] = {{g.x, g.ldx}, {g.residual, g.ld_res}, {g.sum, g.ld_sum}, {g.y, g.ldy}};
    const Layout layout = layout_of<T>(all, !g.q && g.cols + 7 <= kMaxNormCols);
    return with_shape<true>(layout == kShifted ? g.cols + 7 : g.cols, [&](auto w, auto k) {
        constexpr int W = decltype(w)::value, P = decltype(k)::value;
        const unsigned grid = (unsigned)((g.rows + Team<W>::ROWS - 1) / Team<W>::ROWS);
        if (layout == kWhole) return launch(rms_norm_kernel<T, W, P, kWhole>, grid, Team<W>::THREADS, 0, &p, stream);
        if (layout == kShifted) return launch(rms_norm_kernel<T, W, P, kShifted>, grid, Team<W>::THREADS, 0, &p, stream);
        return launch(rms_norm_kernel<T, W, P, kStaged>, grid, Team<W>::THREADS, staging_bytes(g.cols, Team<W>::ROWS), &p,
                      stream);
    });
}

// Blocks of the gradient's kernel: each holds a row of weight gradients.
template <class T, int W>
unsigned backward_blocks(const RmsNormBackwardArgs &g)
{
    const int64_t all = (g.rows + Team<W>::ROWS - 1) / Team<W>::ROWS;
    const int64_t most = (int64_t)g.num_sms * backward_resident<T>(Team<W>::THREADS);
    return (unsigned)(all < most ? all : most);
}

template <class T>
Layout backward_layout(const RmsNormBackwardArgs &g)
{
    const Rows all[] = {{g.grad_y, g.ld_gy}, {g.x, g.ldx}, {g.grad_sum, g.ld_gs}, {g.grad_x, g.ld_gx}};
    return layout_of<T>(all, g.cols + 7 <= kMaxNormCols);
}

// The columns that a row's eights reach over.
template <class T>
int64_t backward_cols(const RmsNormBackwardArgs &g)
{
    return backward_layout<T>(g) == kShifted ? g.cols + 7 : g.cols;
}

template <class T>
cudaError_t norm_backward_of(const RmsNormBackwardArgs &g, void *scratch, cudaStream_t stream)
{
    NormBackwardParams<T> p{};
    p.rows = g.rows, p.cols = (int)g.cols;
    p.g = static_cast<const T *>(g.grad_y), p.ld_g = g.ld_gy;
    p.x = static_cast<const T *>(g.x), p.ldx = g.ldx;
    p.gs = static_cast<const T *>(g.grad_sum), p.ld_gs = g.ld_gs;
    p.weight = g.weight, p.eps = g.eps;
    p.weight16 = (reinterpret_cast<uintptr_t>(g.weight) & 15u) == 0;
    p.dx = static_cast<T *>(g.grad_x), p.ld_dx = g.ld_gx;
    p.parts = g.grad_weight ? static_cast<float *>(scratch) : nullptr;
    const Layout layout = backward_layout<T>(g);
    return with_shape<false>(backward_cols<T>(g), [&](auto w, auto k) {
        constexpr int W = decltype(w)::value, P = decltype(k)::value;
        const unsigned grid = backward_blocks<T, W>(g);
        // Warps add their weight gradients up in shared memory, shifted rows theirs.
        const bool adds = p.parts && (W == 1 || layout == kShifted);
        const int bytes = layout == kStaged || adds ? staging_bytes(g.cols, Team<W>::ROWS) : 0;
        cudaError_t e = cudaSuccess;
        if (grid > 0)
            e = layout == kWhole ? launch(rms_norm_backward_kernel<T, W, P, kWhole>, grid, Team<W>::THREADS, bytes, &p, stream)
                : layout == kShifted
                    ? launch(rms_norm_backward_kernel<T, W, P, kShifted>, grid, Team<W>::THREADS, bytes, &p, stream)
                    : launch(rms_norm_backward_kernel<T, W, P, kStaged>, grid, Team<W>::THREADS, bytes, &p, stream);
        if (e != cudaSuccess || !g.grad_weight) return e;
        return launch_after(add_parts_kernel, dim3((unsigned)((g.cols + 31) / 32)), dim3(1024), stream, (const float *)p.parts,
                            (int)grid, (int)g.cols, g.grad_weight);
    });
}

}  // namespace

cudaError_t prepare_rms_norm()
{
    const cudaError_t e = prepare_widest<float>();
    return e != cudaSuccess ? e : prepare_widest<__nv_bfloat16>();
}

cudaError_t launch_rms_norm(const RmsNormArgs &g, cudaStream_t stream)
{
    return g.bf16 ? norm_of<__nv_bfloat16>(g, stream) : norm_of<float>(g, stream);
}

size_t rms_norm_backward_scratch_bytes(const RmsNormBackwardArgs &g)
{
    if (!g.grad_weight) return 0;
    size_t bytes = 0;
    with_shape<false>(g.bf16 ? backward_cols<__nv_bfloat16>(g) : backward_cols<float>(g), [&](auto w, auto) {
        constexpr int W = decltype(w)::value;
        const unsigned blocks = g.bf16 ? backward_blocks<__nv_bfloat16, W>(g) : backward_blocks<float, W>(g);
        bytes = (size_t)blocks * (size_t)g.cols * 4;
        return cudaSuccess;
    });
    return bytes;
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs &g, void *scratch, cudaStream_t stream)
{
    return g.bf16 ? norm_backward_of<__nv_bfloat16>(g, scratch, stream) : norm_backward_of<float>(g, scratch, stream);
}

}  // namespace sgemm_gb300
