// Routing of tokens to experts: scores and top-k with their gradient, and the
// stable counting sort of (token, slot) pairs by expert.
//
// Scores of a token's logits l: softmax e_i / sum e, e_i = exp(l_i - max l),
// or sigmoid 1 / (1 + exp(-l_i)). The key that orders experts is score + bias
// where there is a bias or groups rank by the sum of their two best, and the
// logit itself otherwise (softmax and sigmoid keep its order, and comparing
// logits cannot be upset by rounding). Keys are compared as integers that
// order like the floats; 0 stands for "not eligible" (a logit or key that is
// -infinity or NaN).
#include "experts.cuh"

namespace sgemm_gb300 {

namespace {

// Floats as unsigned integers in the same order; every number above
// -infinity maps above kNoKey.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The key of value x (-0 and +0 are one value), 0 when it is not eligible.
__device__ __forceinline__ uint32_t key_of(float x)
{
    return x > __uint_as_float(0xff800000u) ? ordered(x + 0.0f) : 0u;   // false for NaN
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// exp(l - m); 1 where both are the same infinity.
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

constexpr int kRouteWarps = 8;

// One warp per token; lane j holds experts j, j + 32, ...: NPER of them.
template <class T, int NPER>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_kernel(int64_t tokens, int E, const T *__restrict__ logits, int64_t ld, const float *__restrict__ bias,
             int use_sigmoid, int groups, int kept, int two, int k, int renorm, float scale,
             float *__restrict__ weights, int32_t *__restrict__ indices)
{
    extern __shared__ uint32_t group_keys[];      // E per warp, where groups are ranked
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= tokens) return;
    const T *row = logits + t * ld;
    float l[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < E ? load_as_float(row + e) : __uint_as_float(0xff800000u);
    }
    // Softmax statistics over the eligible logits.
    float m = 0.0f, sum = 1.0f;
    if (!use_sigmoid) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i) best = max(best, key_of(l[i]));
        best = __reduce_max_sync(0xffffffffu, best);
        if (best) {
            m = unordered(best);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (key_of(l[i])) sum += exp_below(l[i], m);
            sum = warp_sum(sum);
        }
    }
    auto score = [&](float x) { return use_sigmoid ? sigmoid(x) : __fdiv_rn(exp_below(x, m), sum); };
    const bool by_score = bias != nullptr || two;
    uint32_t key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        key[i] = key_of(l[i]);
        if (by_score && key[i]) {
            float x = score(l[i]);
            if (bias) x += bias[lane + 32 * i];
            key[i] = key_of(x);
        }
    }
    if (kept < groups) {
        const int size = E / groups;
        uint32_t *const mine = group_keys + warp * E;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < E) mine[lane + 32 * i] = key[i];
        __syncwarp();
        // `per` lanes (a power of two) scan each group.
        int per = 1;
        while (2 * per * groups <= 32) per *= 2;
        const int g = lane / per, sub = lane % per;
        uint32_t b1 = 0, b2 = 0;
        if (g < groups)
            for (int j = sub; j < size; j += per) {
                const uint32_t x = mine[g * size + j];
                b2 = max(b2, min(b1, x));
                b1 = max(b1, x);
            }
        for (int d = 1; d < per; d *= 2) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, d), o2 = __shfl_xor_sync(0xffffffffu, b2, d);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        // A group's rank; with `two` a group of fewer than two eligible
        // experts comes last.
        uint32_t rank = b1;
        if (two) rank = b2 ? key_of(unordered(b1) + unordered(b2)) : 0u;
        int before = 0;
        for (int o = 0; o < groups; ++o) {
            const uint32_t other = __shfl_sync(0xffffffffu, rank, o * per);
            before += (other > rank || (other == rank && o < g)) ? 1 : 0;
        }
        const uint32_t ballot = __ballot_sync(0xffffffffu, g < groups && before < kept);
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            const int e = lane + 32 * i;
            if (e < E && !((ballot >> ((e / size) * per)) & 1u)) key[i] = 0;
        }
    }
    // k times the largest key, the lowest expert first among equals.
    int chosen = -1;                              // lane j: the expert of slot j
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = NPER - 1; i >= 0; --i)
            if (key[i] >= best) best = key[i], at = i;
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0) break;
        const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(lane + 32 * at) : 0xffffffffu);
        if (lane == j) chosen = e;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i == e) key[i] = 0;
    }
    float w = chosen >= 0 ? score(load_as_float(row + chosen)) : 0.0f;
    if (renorm) {
        const float total = warp_sum(w);
        w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
    }
    if (lane < k) {
        weights[t * k + lane] = w * scale;
        indices[t * k + lane] = chosen;
    }
}

// Gradient of the weights with respect to the logits. With S the chosen
// experts, g_j the gradient of slot j and c the scale:
//   softmax, renormalised: dl_j = w_j (g_j - sum_S w_i g_i / c), w_j = c e_j / sum_S e   (j in S)
//   softmax:               dl_i = c p_i (g_i [i in S] - sum_S p_j g_j)                   (every i)
//   sigmoid, renormalised: dl_j = c / D (g_j - sum_S g_i s_i / D) s_j (1 - s_j), D = sum_S s
//   sigmoid:               dl_j = c g_j s_j (1 - s_j)
// with 1 - s taken as sigmoid(-l), which keeps its digits where s is near 1.
// Only the second needs the whole row of logits; the others read the chosen
// ones and write a row of zeros with k values in it.
template <class T>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_backward_kernel(int64_t tokens, int E, const T *__restrict__ logits, int64_t ld, int use_sigmoid, int k,
                      int renorm, float scale, const int32_t *__restrict__ indices,
                      const float *__restrict__ grad_w, T *__restrict__ grad, int64_t ld_g)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= tokens) return;
    const T *row = logits + t * ld;
    T *out = grad + t * ld_g;
    int e = -1;
    float g = 0.0f, l = 0.0f;
    if (lane < k) {
        e = indices[t * k + lane];
        if (e < 0 || e >= E) e = -1;
        if (e >= 0) {
            g = grad_w[t * k + lane];
            l = load_as_float(row + e);
        }
    }
    float d = 0.0f;
    if (use_sigmoid) {
        if (e >= 0) {
            const float s = sigmoid(l), slope = s * sigmoid(-l);
            d = scale * g * slope;
        }
        if (renorm) {
            const float s = e >= 0 ? sigmoid(l) : 0.0f;
            const float D = warp_sum(s), mean = warp_sum(s * g);
            d = 0.0f;
            if (e >= 0 && D > 0.0f) d = scale / D * (g - mean / D) * (s * sigmoid(-l));
        }
        for (int i = lane; i < E; i += 32) store_from_float(out + i, 0.0f);
    } else if (renorm) {
        float m = e >= 0 ? l : __uint_as_float(0xff800000u);
#pragma unroll
        for (int o = 16; o; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float x = e >= 0 ? exp_below(l, m) : 0.0f;
        const float total = warp_sum(x);
        const float w = total > 0.0f ? x / total : 0.0f;
        const float mean = warp_sum(w * g);
        d = scale * w * (g - mean);
        for (int i = lane; i < E; i += 32) store_from_float(out + i, 0.0f);
    } else {
        uint32_t best = 0;
        for (int i = lane; i < E; i += 32) best = max(best, key_of(load_as_float(row + i)));
        best = __reduce_max_sync(0xffffffffu, best);
        const float m = best ? unordered(best) : 0.0f;
        float sum = 0.0f;
        for (int i = lane; i < E; i += 32) {
            const float x = load_as_float(row + i);
            if (key_of(x)) sum += exp_below(x, m);
        }
        sum = warp_sum(sum);
        const float p = e >= 0 && sum > 0.0f ? exp_below(l, m) / sum : 0.0f;
        const float mean = warp_sum(p * g);
        d = scale * p * (g - mean);
        for (int i = lane; i < E; i += 32) {
            const float x = load_as_float(row + i);
            const float q = key_of(x) ? exp_below(x, m) / sum : 0.0f;
            store_from_float(out + i, -scale * q * mean);
        }
    }
    __syncwarp();   // the chosen entries after the rest of the row
    if (e >= 0) store_from_float(out + e, d);
}

// ---------------------------------------------------------------------------
// Dispatch: the (token, slot) pairs sorted by expert, pairs of one expert in
// their own order. Blocks take equal runs of the n pairs and the 32 warps of
// a block equal parts of its run; each warp counts its experts in shared
// memory, the counts become starting rows (experts before, blocks before,
// warps before), and each warp walks its part again, 32 pairs at a time,
// ranking equal experts within the 32 by their lane. Nothing depends on the
// order in which threads run.
constexpr int kDispatchThreads = 1024, kDispatchWarps = 32;

struct DispatchArgs {
    int64_t n, run;                 // pairs, and pairs per block (a multiple of 1024)
    int k, E;
    const int32_t *indices;
    int32_t *offsets, *row_of, *token_of;
    int32_t *counts;                // [block][E], with more than one block
    int blocks;
};

// Lanes whose expert equals this lane's, among the lanes of the warp.
__device__ __forceinline__ uint32_t same_expert(int e, int bits)
{
    uint32_t same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xffffffffu, (e >> b) & 1);
        same &= ((e >> b) & 1) ? set : ~set;
    }
    return same;
}

__device__ __forceinline__ int valid_expert(const DispatchArgs &a, int64_t i)
{
    if (i >= a.n) return -1;
    const int e = a.indices[i];
    return e >= 0 && e < a.E ? e : -1;
}

__global__ void __launch_bounds__(kDispatchThreads)
dispatch_count_kernel(const DispatchArgs a)
{
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < a.E; e += kDispatchThreads) hist[e] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * a.run, i1 = i0 + a.run < a.n ? i0 + a.run : a.n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kDispatchThreads) {
        const int e = valid_expert(a, i);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kDispatchThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

__global__ void __launch_bounds__(kDispatchThreads)
dispatch_place_kernel(const DispatchArgs a)
{
    extern __shared__ int next[];                 // [warp][E]: counts, then the next row of each expert
    __shared__ int sums[kDispatchWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kDispatchWarps * a.E; i += kDispatchThreads) next[i] = 0;
    __syncthreads();
    const int64_t part = a.run / kDispatchWarps;
    const int64_t i0 = (int64_t)blockIdx.x * a.run + warp * part;
    int *const mine = next + warp * a.E;
    for (int64_t i = i0 + lane; i < i0 + part && i < a.n; i += 32) {
        const int e = valid_expert(a, i);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // Thread e: expert e (E <= 1024).
    const int e = threadIdx.x;
    int total = 0, before = 0;
    if (e < a.E) {
        if (a.blocks > 1) {
            for (int b = 0; b < a.blocks; ++b) {
                const int c = a.counts[(int64_t)b * a.E + e];
                total += c;
                before += b < (int)blockIdx.x ? c : 0;
            }
        } else {
            for (int w = 0; w < kDispatchWarps; ++w) total += next[w * a.E + e];
        }
    }
    // Exclusive prefix sum of `total` over the experts.
    int sum = total;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += sums[w];
    const int first = base + sum - total;
    if (e < a.E) {
        int at = first + before;
        for (int w = 0; w < kDispatchWarps; ++w) {
            const int c = next[w * a.E + e];
            next[w * a.E + e] = at;
            at += c;
        }
        if (blockIdx.x == 0) a.offsets[e] = first;
    }
    int all = 0;
    for (int w = 0; w < kDispatchWarps; ++w) all += sums[w];
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
    __syncthreads();
    const int bits = 32 - __clz(a.E);             // E itself marks "no expert"
    for (int64_t b = i0; b < i0 + part && b < a.n; b += 32) {
        const int64_t i = b + lane;
        const int x = valid_expert(a, i), as = x < 0 ? a.E : x;
        const uint32_t same = same_expert(as, bits);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int at = -1;
        if (x >= 0) at = mine[x] + rank;
        __syncwarp();
        if (x >= 0 && rank == 0) mine[x] += __popc(same);
        __syncwarp();
        if (i < a.n) a.row_of[i] = at;
        if (at >= 0) a.token_of[at] = (int32_t)(i / a.k);
    }
    // Rows that no pair has.
    for (int64_t r = all + (int64_t)blockIdx.x * kDispatchThreads + threadIdx.x; r < a.n;
         r += (int64_t)gridDim.x * kDispatchThreads)
        a.token_of[r] = -1;
}

// Blocks of a dispatch: one up to 16384 pairs (512 per warp), at most 128.
int64_t dispatch_run(int64_t n)
{
    if (n <= 16384) return n > 0 ? (n + 1023) / 1024 * 1024 : 1024;
    int64_t run = (n + 127) / 128;
    run = (run + 1023) / 1024 * 1024;
    return run < 4096 ? 4096 : run;
}

template <class T>
cudaError_t route_of(const RouteArgs &r, float *weights, int32_t *indices, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((r.T + kRouteWarps - 1) / kRouteWarps);
    const size_t smem = r.kept < r.groups ? (size_t)kRouteWarps * r.E * 4 : 0;
    const T *l = static_cast<const T *>(r.logits);
    auto go = [&](auto kernel) {
        kernel<<<grid, kRouteWarps * 32, smem, stream>>>(r.T, r.E, l, r.ld, r.bias, r.sigmoid, r.groups, r.kept, r.two,
                                                         r.k, r.renorm, r.scale, weights, indices);
        return cudaGetLastError();
    };
    const int per = (r.E + 31) / 32;
    if (per <= 1) return go(route_kernel<T, 1>);
    if (per <= 2) return go(route_kernel<T, 2>);
    if (per <= 4) return go(route_kernel<T, 4>);
    if (per <= 8) return go(route_kernel<T, 8>);
    if (per <= 16) return go(route_kernel<T, 16>);
    return go(route_kernel<T, 32>);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &r, float *weights, int32_t *indices, int, cudaStream_t stream)
{
    return r.bf16 ? route_of<__nv_bfloat16>(r, weights, indices, stream) : route_of<float>(r, weights, indices, stream);
}

cudaError_t launch_route_backward(const RouteArgs &r, const int32_t *indices, const float *grad_w, void *grad_logits,
                                  int64_t ld_g, int, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((r.T + kRouteWarps - 1) / kRouteWarps);
    if (r.bf16)
        route_backward_kernel<<<grid, kRouteWarps * 32, 0, stream>>>(
            r.T, r.E, static_cast<const __nv_bfloat16 *>(r.logits), r.ld, r.sigmoid, r.k, r.renorm, r.scale, indices,
            grad_w, static_cast<__nv_bfloat16 *>(grad_logits), ld_g);
    else
        route_backward_kernel<<<grid, kRouteWarps * 32, 0, stream>>>(
            r.T, r.E, static_cast<const float *>(r.logits), r.ld, r.sigmoid, r.k, r.renorm, r.scale, indices, grad_w,
            static_cast<float *>(grad_logits), ld_g);
    return cudaGetLastError();
}

size_t dispatch_scratch_bytes(int64_t n, int E)
{
    const int64_t run = dispatch_run(n), blocks = (n + run - 1) / run;
    return blocks > 1 ? (size_t)(blocks * E) * 4 : 0;
}

cudaError_t prepare_route()
{
    return cudaFuncSetAttribute(dispatch_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kDispatchWarps * kMaxExperts * 4);
}

cudaError_t launch_dispatch(int64_t T, int k, int E, const int32_t *indices, int32_t *offsets, int32_t *row_of,
                            int32_t *token_of, void *scratch, cudaStream_t stream)
{
    DispatchArgs a{};
    a.n = T * k;
    a.run = dispatch_run(a.n);
    a.k = k;
    a.E = E;
    a.indices = indices;
    a.offsets = offsets;
    a.row_of = row_of;
    a.token_of = token_of;
    a.counts = static_cast<int32_t *>(scratch);
    a.blocks = (int)((a.n + a.run - 1) / a.run);
    if (a.blocks < 1) a.blocks = 1;
    if (a.blocks > 1) {
        dispatch_count_kernel<<<a.blocks, kDispatchThreads, (size_t)E * 4, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    dispatch_place_kernel<<<a.blocks, kDispatchThreads, (size_t)kDispatchWarps * E * 4, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace sgemm_gb300
