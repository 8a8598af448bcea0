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
#include "ptx.cuh"

#include <atomic>

namespace sgemm_gb300 {

namespace {

// Floats as unsigned integers in the same order; every number maps above 0.
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

// Sum and maximum over groups of L neighbouring lanes.
template <int L>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int d = L / 2; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <int L>
__device__ __forceinline__ float lanes_max(float x)
{
#pragma unroll
    for (int d = L / 2; d; d /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// exp(l - m); 1 where both are the same infinity.
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// The score of logit l over exp(min(m, 0)) (sigmoid) or, but for the sum over
// the row, over exp(m) (softmax): between 1/2 and 1 for l = m, so that the
// ratios of chosen scores keep range and digits where the scores themselves
// are below 2^-126. For m >= 0 the sigmoid is the score itself.
__device__ __forceinline__ float relative_score(float l, float m, int use_sigmoid)
{
    if (!use_sigmoid) return exp_below(l, m);
    return __fdiv_rn(exp_below(fminf(l, 0.0f), fminf(m, 0.0f)), 1.0f + expf(-fabsf(l)));
}

// Four neighbouring values.
__device__ __forceinline__ void load4(const float *p, float *v)
{
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}

__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *v)
{
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
}

constexpr int kRouteWarps = 8;

// L lanes per token, each with NPER logits: runs of four, 4 L apart. Bound by
// instructions (about 450 per warp of 128 experts and 8 rounds), not by the
// logits' bytes. Fewer lanes with more logits each need fewer instructions a
// token, but a longer chain of them: 8 lanes of 16 took 12.0 us for 16383
// tokens and 11.8 us for 8 of them, 32 lanes of 4 take 11.0 us and 5.9 us.
template <class T, int L, int NPER>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_kernel(int64_t tokens, int E, const T *__restrict__ logits, int64_t ld, int vec, const float *__restrict__ bias,
             int use_sigmoid, int groups, int kept, int two, int k, int renorm, float scale,
             float *__restrict__ weights, int32_t *__restrict__ indices)
{
    constexpr int TOKENS = kRouteWarps * 32 / L;  // of this CTA
    extern __shared__ uint32_t group_keys[];      // E per token, where groups are ranked
    __shared__ uint32_t ranks[TOKENS][32];
    __shared__ int chosen[TOKENS][kMaxTop];
    const int slot = threadIdx.x / L, sub = threadIdx.x % L;
    const int64_t t0 = (int64_t)blockIdx.x * TOKENS + slot;
    const bool there = t0 < tokens;
    const int64_t t = there ? t0 : tokens - 1;    // lanes without a token go along and store nothing
    const T *row = logits + t * ld;
    float l[NPER];
#pragma unroll
    for (int i = 0; i < NPER; i += 4) {
        const int e = (i / 4) * (4 * L) + 4 * sub;
        if (vec && e + 4 <= E) {
            load4(row + e, l + i);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) l[i + j] = e + j < E ? load_as_float(row + e + j) : __uint_as_float(0xff800000u);
        }
    }
    auto expert = [&](int i) { return (i / 4) * (4 * L) + 4 * sub + (i & 3); };
    // Softmax statistics over the eligible logits, for keys and weights that
    // are scores. Renormalised weights need none: the row's sum cancels.
    const bool by_score = bias != nullptr || two;
    float m = 0.0f, sum = 1.0f;
    if (!use_sigmoid && (by_score || !renorm)) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i) best = max(best, key_of(l[i]));
#pragma unroll
        for (int d = L / 2; d; d /= 2) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
        m = best ? unordered(best) : 0.0f;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (key_of(l[i])) sum += exp_below(l[i], m);
        sum = lanes_sum<L>(sum);
        if (!best) sum = 1.0f;
    }
    auto score = [&](float x) { return use_sigmoid ? sigmoid(x) : __fdiv_rn(exp_below(x, m), sum); };
    uint32_t key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        key[i] = key_of(l[i]);
        if (by_score && key[i]) {
            float x = score(l[i]);
            if (bias) x += bias[expert(i)];
            key[i] = key_of(x);
        }
    }
    if (kept < groups) {
        const int size = E / groups;
        uint32_t *const mine = group_keys + slot * E;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (expert(i) < E) mine[expert(i)] = key[i];
        __syncwarp();
        // `per` lanes (a power of two) scan each group, L / per groups at a time.
        int per = 1;
        while (2 * per * groups <= L) per *= 2;
        for (int g0 = 0; g0 < groups; g0 += L / per) {
            const int g = g0 + sub / per;
            uint32_t b1 = 0, b2 = 0;
            if (g < groups)
                for (int j = sub % per; j < size; j += per) {
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
            if (g < groups && sub % per == 0)
                ranks[slot][g] = !two ? b1 : b2 ? key_of(unordered(b1) + unordered(b2)) : 0u;
        }
        __syncwarp();
        uint32_t keep = 0;
        for (int g = sub; g < groups; g += L) {
            const uint32_t rank = ranks[slot][g];
            int before = 0;
            for (int o = 0; o < groups; ++o) {
                const uint32_t other = ranks[slot][o];
                before += (other > rank || (other == rank && o < g)) ? 1 : 0;
            }
            if (before < kept) keep |= 1u << g;
        }
#pragma unroll
        for (int d = L / 2; d; d /= 2) keep |= __shfl_xor_sync(0xffffffffu, keep, d);
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (expert(i) < E && !((keep >> (expert(i) / size)) & 1u)) key[i] = 0;
    }
    // k times the largest key, the lowest expert first among equals.
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[NPER - 1];
        int at = NPER - 1;
#pragma unroll
        for (int i = NPER - 2; i >= 0; --i)
            if (key[i] >= best) best = key[i], at = i;
        int e = expert(at);
        if constexpr (L == 32) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)e : 0xffffffffu);
            best = top;
        } else {
#pragma unroll
            for (int d = L / 2; d; d /= 2) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, best, d);
                const int oe = __shfl_xor_sync(0xffffffffu, e, d);
                if (other > best || (other == best && oe < e)) best = other, e = oe;
            }
        }
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (expert(i) == e) key[i] = 0;
        if (sub == 0) chosen[slot][j] = best ? e : -1;
    }
    __syncwarp();
    constexpr int HELD = kMaxTop / L;             // slots per lane
    int e[HELD];
    float x[HELD], w[HELD], total = 0.0f;
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int j = sub + h * L;
        e[h] = j < k ? chosen[slot][j] : -1;
        x[h] = e[h] >= 0 ? load_as_float(row + e[h]) : __uint_as_float(0xff800000u);
    }
    // Renormalised weights are ratios of the chosen scores: taken relative to
    // the largest of these, which a bias may put far below the row's and a row
    // of very negative logits below what 32 bits hold.
    if (renorm) {
        m = x[0];
#pragma unroll
        for (int h = 1; h < HELD; ++h) m = fmaxf(m, x[h]);
        m = lanes_max<L>(m);
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        w[h] = e[h] < 0 ? 0.0f : renorm ? relative_score(x[h], m, use_sigmoid) : score(x[h]);
        total += w[h];
    }
    if (renorm) total = lanes_sum<L>(total);
    if (!there) return;
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int j = sub + h * L;
        if (j < k) {
            if (renorm) w[h] = total > 0.0f ? __fdiv_rn(w[h], total) : 0.0f;
            weights[t * k + j] = w[h] * scale;
            indices[t * k + j] = e[h];
        }
    }
}

// Gradient of the weights with respect to the logits. With S the chosen
// experts, g_j the gradient of slot j and c the scale:
//   softmax, renormalised: dl_j = w_j (g_j - sum_S w_i g_i / c), w_j = c e_j / sum_S e   (j in S)
//   softmax:               dl_i = c p_i (g_i [i in S] - sum_S p_j g_j)                   (every i)
//   sigmoid, renormalised: dl_j = w_j (g_j - sum_S w_i g_i / c) (1 - s_j), w_j = c s_j / sum_S s
//   sigmoid:               dl_j = c g_j s_j (1 - s_j)
// with 1 - s taken as sigmoid(-l), which keeps its digits where s is near 1,
// and the weights from scores relative to the largest chosen one.
// Only the second needs the whole row of logits; the others read the chosen
// ones and write a row of zeros with k values in it. One warp per token;
// bound by instructions and the latency of its three dependent loads (16383
// tokens of 128 experts: 7.0 us, 1.2 us of bytes).
template <class T>
__device__ __forceinline__ void zero_row(T *out, int E, int vec, int lane)
{
    constexpr int N = 16 / (int)sizeof(T);
    if (vec) {
        for (int i = lane * N; i < E; i += 32 * N) *reinterpret_cast<uint4 *>(out + i) = make_uint4(0, 0, 0, 0);
    } else {
        for (int i = lane; i < E; i += 32) store_from_float(out + i, 0.0f);
    }
}

template <class T>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_backward_kernel(int64_t tokens, int E, const T *__restrict__ logits, int64_t ld, int use_sigmoid, int k,
                      int renorm, float scale, const int32_t *__restrict__ indices,
                      const float *__restrict__ grad_w, T *__restrict__ grad, int64_t ld_g, int vec)
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
    if (renorm) {
        const float least = __uint_as_float(0xff800000u);
        float m = e >= 0 ? l : least;
        m = lanes_max<32>(m);
        const float x = e >= 0 && l != least ? relative_score(l, m, use_sigmoid) : 0.0f;
        const float total = warp_sum(x);
        const float w = total > 0.0f ? x / total : 0.0f;
        const float mean = warp_sum(w * g);
        d = scale * w * (g - mean);
        if (use_sigmoid) d *= sigmoid(-l);
        zero_row(out, E, vec, lane);
    } else if (use_sigmoid) {
        if (e >= 0) d = scale * g * (sigmoid(l) * sigmoid(-l));
        zero_row(out, E, vec, lane);
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
//
// Up to 131072 pairs (where the device takes clusters of 16; else 65536) the
// blocks are one cluster, which reads its neighbours' counts from their shared
// memory: one launch, no scratch. Beyond that 128 blocks run behind a launch
// that leaves every block's counts in scratch: what bounds large sorts is the
// scattered writes of token_of, about one a cycle and SM. Measured: 48 pairs
// 5.4 us; 131064 pairs of 128 experts 12.6 us (128 blocks behind a counting
// launch: 12.4 us in two launches and an allocation, which cost the host more
// than the first; 8 blocks: 18 us).
constexpr int kDispatchThreads = 1024, kDispatchWarps = 32, kDispatchHeld = 8, kDispatchCluster = 16;
constexpr int64_t kDispatchRun = 32 * kDispatchWarps * kDispatchHeld;   // pairs a block can hold in registers

struct DispatchArgs {
    int64_t n, run;                 // pairs, and pairs per block (a multiple of 1024)
    int k, E;
    const int32_t *indices;
    int32_t *offsets, *row_of, *token_of;
    int32_t *counts;                // [block][E], with blocks that are no cluster
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

// The expert of pair i, E where it has none.
__device__ __forceinline__ int valid_expert(const DispatchArgs &a, int64_t i)
{
    if (i >= a.n) return a.E;
    const int e = a.indices[i];
    return e >= 0 && e < a.E ? e : a.E;
}

__global__ void __launch_bounds__(kDispatchThreads)
dispatch_count_kernel(const DispatchArgs a)
{
    extern __shared__ int hist[];
    ptx::grid_launch_dependents();                // the placing kernel's blocks read their pairs meanwhile
    for (int e = threadIdx.x; e < a.E; e += kDispatchThreads) hist[e] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * a.run, i1 = i0 + a.run < a.n ? i0 + a.run : a.n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kDispatchThreads) {
        const int e = valid_expert(a, i);
        if (e < a.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kDispatchThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// HELD: the warp's part of the run stays in registers between the two walks.
template <bool HELD>
__global__ void __launch_bounds__(kDispatchThreads)
dispatch_place_kernel(const DispatchArgs a)
{
    extern __shared__ int next[];                 // [warp][E]: counts, then the next row of each expert
    __shared__ int sums[kDispatchWarps];
    __shared__ int totals[kMaxExperts], earlier[kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t part = a.run / kDispatchWarps, i0 = (int64_t)blockIdx.x * a.run + warp * part;
    const int steps = (int)(part / 32);
    int held[HELD ? kDispatchHeld : 1];
    if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < kDispatchHeld; ++j) held[j] = j < steps ? valid_expert(a, i0 + 32 * j + lane) : a.E;
    }
    for (int i = threadIdx.x; i < kDispatchWarps * a.E; i += kDispatchThreads) next[i] = 0;
    __syncthreads();
    int *const mine = next + warp * a.E;
    if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < kDispatchHeld; ++j)
            if (held[j] < a.E) atomicAdd(&mine[held[j]], 1);
    } else {
        for (int j = 0; j < steps; ++j) {
            const int e = valid_expert(a, i0 + 32 * j + lane);
            if (e < a.E) atomicAdd(&mine[e], 1);
        }
    }
    __syncthreads();
    // Thread e: expert e (E <= 1024).
    const int e = threadIdx.x;
    int total = 0, before = 0, of_warp[kDispatchWarps];
    if (e < a.E) {
#pragma unroll
        for (int w = 0; w < kDispatchWarps; ++w) of_warp[w] = next[w * a.E + e];
#pragma unroll
        for (int w = 0; w < kDispatchWarps; ++w) total += of_warp[w];
    }
    if (a.counts) {
        // Sums over the blocks: 1024 / (E rounded up to a power of two) threads
        // share an expert.
        ptx::grid_dependency_wait();
        int width = 32;
        while (width < a.E) width *= 2;
        const int x = threadIdx.x % width, share = threadIdx.x / width, shares = kDispatchThreads / width;
        const int b0 = a.blocks * share / shares, b1 = a.blocks * (share + 1) / shares;
        int all_of = 0, before_of = 0;
        if (x < a.E) {
#pragma unroll 16
            for (int b = b0; b < b1; ++b) {
                const int c = __ldcg(a.counts + (int64_t)b * a.E + x);
                all_of += c;
                before_of += b < (int)blockIdx.x ? c : 0;
            }
        }
        totals[threadIdx.x] = all_of;
        earlier[threadIdx.x] = before_of;
        __syncthreads();
        total = 0;
        if (e < a.E)
            for (int s = 0; s < shares; ++s) {
                total += totals[s * width + e];
                before += earlier[s * width + e];
            }
    } else if (a.blocks > 1) {
        // The blocks of the cluster trade their counts.
        if (e < a.E) totals[e] = total;
        ptx::cluster_sync_all();
        if (e < a.E) {
            total = 0;
#pragma unroll 8
            for (int b = 0; b < a.blocks; ++b) {
                int of_block;
                asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\t"
                             "ld.shared::cluster.s32 %0, [ra];\n\t}"
                             : "=r"(of_block)
                             : "r"(ptx::smem_addr(&totals[e])), "r"(b)
                             : "memory");
                total += of_block;
                before += b < (int)blockIdx.x ? of_block : 0;
            }
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
    const int others = sums[lane];
    const int base = __reduce_add_sync(0xffffffffu, lane < warp ? others : 0);
    const int all = __reduce_add_sync(0xffffffffu, others);
    const int first = base + sum - total;
    if (e < a.E) {
        int at = first + before;
#pragma unroll
        for (int w = 0; w < kDispatchWarps; ++w) {
            next[w * a.E + e] = at;
            at += of_warp[w];
        }
        if (blockIdx.x == 0) a.offsets[e] = first;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
    __syncthreads();
    const int bits = 32 - __clz(a.E);             // E itself marks "no expert"
    auto place = [&](int64_t i, int x) {
        const uint32_t same = same_expert(x, bits);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int at = -1;
        if (x < a.E) at = mine[x] + rank;
        __syncwarp();
        if (x < a.E && rank == 0) mine[x] += __popc(same);
        __syncwarp();
        if (i < a.n) a.row_of[i] = at;
        if (at >= 0) a.token_of[at] = (int32_t)(i / a.k);
    };
    if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < kDispatchHeld; ++j)
            if (j < steps) place(i0 + 32 * j + lane, held[j]);
    } else {
        for (int j = 0; j < steps; ++j) place(i0 + 32 * j + lane, valid_expert(a, i0 + 32 * j + lane));
    }
    // Rows that no pair has.
    for (int64_t r = all + (int64_t)blockIdx.x * kDispatchThreads + threadIdx.x; r < a.n;
         r += (int64_t)gridDim.x * kDispatchThreads)
        a.token_of[r] = -1;
    // No block leaves while another may read its counts.
    if (!a.counts && a.blocks > 1) ptx::cluster_sync_all();
}

// Largest cluster that every device of this process so far takes.
std::atomic<int> g_dispatch_cluster{kDispatchCluster};

// One block up to 4096 pairs (128 per warp), then a cluster of 8, then the
// largest cluster (the last blocks of either may have nothing), then 128.
int64_t dispatch_blocks(int64_t n)
{
    const int most = g_dispatch_cluster.load();
    return n <= 4096 ? 1 : n <= 16384 ? 8 : n <= most * kDispatchRun ? most : 128;
}

bool dispatch_clustered(int64_t n) { return n <= g_dispatch_cluster.load() * kDispatchRun; }

int64_t dispatch_run(int64_t n)
{
    const int64_t blocks = dispatch_blocks(n), run = (n + blocks - 1) / blocks;
    return run > 0 ? (run + 1023) / 1024 * 1024 : 1024;
}

template <class T>
cudaError_t route_of(const RouteArgs &r, float *weights, int32_t *indices, cudaStream_t stream)
{
    const T *l = static_cast<const T *>(r.logits);
    // Runs of four logits in one load.
    const int vec = (reinterpret_cast<uintptr_t>(l) % (4 * sizeof(T)) == 0 && r.ld % 4 == 0) ? 1 : 0;
    auto go = [&](auto kernel, int lanes) {
        const int per_cta = kRouteWarps * 32 / lanes;
        const size_t smem = r.kept < r.groups ? (size_t)per_cta * r.E * 4 : 0;
        kernel<<<(unsigned)((r.T + per_cta - 1) / per_cta), kRouteWarps * 32, smem, stream>>>(
            r.T, r.E, l, r.ld, vec, r.bias, r.sigmoid, r.groups, r.kept, r.two, r.k, r.renorm, r.scale, weights, indices);
        return cudaGetLastError();
    };
    if (r.E <= 32) return go(route_kernel<T, 8, 4>, 8);
    if (r.E <= 64) return go(route_kernel<T, 16, 4>, 16);
    if (r.E <= 128) return go(route_kernel<T, 32, 4>, 32);
    if (r.E <= 256) return go(route_kernel<T, 32, 8>, 32);
    if (r.E <= 512) return go(route_kernel<T, 32, 16>, 32);
    return go(route_kernel<T, 32, 32>, 32);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &r, float *weights, int32_t *indices, cudaStream_t stream)
{
    return r.bf16 ? route_of<__nv_bfloat16>(r, weights, indices, stream) : route_of<float>(r, weights, indices, stream);
}

cudaError_t launch_route_backward(const RouteArgs &r, const int32_t *indices, const float *grad_w, void *grad_logits,
                                  int64_t ld_g, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((r.T + kRouteWarps - 1) / kRouteWarps);
    const int64_t per16 = r.bf16 ? 8 : 4;
    const int vec = (reinterpret_cast<uintptr_t>(grad_logits) % 16 == 0 && ld_g % per16 == 0 && r.E % per16 == 0) ? 1 : 0;
    if (r.bf16)
        route_backward_kernel<<<grid, kRouteWarps * 32, 0, stream>>>(
            r.T, r.E, static_cast<const __nv_bfloat16 *>(r.logits), r.ld, r.sigmoid, r.k, r.renorm, r.scale, indices,
            grad_w, static_cast<__nv_bfloat16 *>(grad_logits), ld_g, vec);
    else
        route_backward_kernel<<<grid, kRouteWarps * 32, 0, stream>>>(
            r.T, r.E, static_cast<const float *>(r.logits), r.ld, r.sigmoid, r.k, r.renorm, r.scale, indices, grad_w,
            static_cast<float *>(grad_logits), ld_g, vec);
    return cudaGetLastError();
}

size_t dispatch_scratch_bytes(int64_t n, int E)
{
    return dispatch_clustered(n) ? 0 : (size_t)(dispatch_blocks(n) * E) * 4;
}

cudaError_t prepare_route()
{
    const int smem = kDispatchWarps * kMaxExperts * 4;
    cudaError_t e = cudaFuncSetAttribute(dispatch_place_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(dispatch_place_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(dispatch_place_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    // Clusters of 16 where the device can hold one at the largest size.
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kDispatchCluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    lc.gridDim = dim3(kDispatchCluster);
    lc.blockDim = dim3(kDispatchThreads);
    lc.dynamicSmemBytes = smem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, dispatch_place_kernel<true>, &lc) != cudaSuccess || clusters < 1) {
        cudaGetLastError();
        g_dispatch_cluster.store(8);
    }
    return cudaSuccess;
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
    a.blocks = (int)dispatch_blocks(a.n);
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    if (scratch) {
        dispatch_count_kernel<<<a.blocks, kDispatchThreads, (size_t)E * 4, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        lc.numAttrs = 1;
    } else {
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)a.blocks;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        lc.numAttrs = a.blocks > 1 ? 1 : 0;
    }
    lc.attrs = &attr;
    lc.gridDim = dim3((unsigned)a.blocks);
    lc.blockDim = dim3(kDispatchThreads);
    lc.dynamicSmemBytes = (size_t)kDispatchWarps * E * 4;
    lc.stream = stream;
    const cudaError_t e = a.run <= kDispatchRun ? cudaLaunchKernelEx(&lc, dispatch_place_kernel<true>, a)
                                                : cudaLaunchKernelEx(&lc, dispatch_place_kernel<false>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sgemm_gb300
