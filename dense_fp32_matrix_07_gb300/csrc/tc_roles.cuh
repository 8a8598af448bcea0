// What the kernels with warps in roles (TMA producer, MMA issuer, tile finder,
// epilogue) share: predicated copies, MMAs' commits and arrivals, looks at
// barriers, tensor memory loads, the groups of a product over experts, and the
// host's tensor map encoder.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

namespace sgemm_gb300 {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Division by a number the host knows, n / d for n < 2^31, by the multiplier
// and shift of Granlund and Montgomery ("Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
    uint32_t d, mul, shift;   // n / d = (umulhi(n, mul) + n) >> shift, in 33 bits
};

inline FastDiv fast_div(uint32_t d)
{
    FastDiv f{d, 0, 0};
    while ((uint64_t(1) << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
    return f;
}

__device__ __forceinline__ uint32_t div(uint32_t n, const FastDiv &f)
{
    // umulhi(n, mul) <= n < 2^31: the sum fits 32 bits.
    return (__umulhi(n, f.mul) + n) >> f.shift;
}

__device__ __forceinline__ int clamp_to(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Rows [lo, hi) of group g, forced into [0, rows] whatever the offsets hold.
__device__ __forceinline__ void group_range(const int32_t *offsets, int g, int rows, int &lo, int &hi)
{
    lo = clamp_to(offsets[g], 0, rows);
    hi = clamp_to(offsets[g + 1], lo, rows);
}

// The group that owns entry x of the prefix table: table[g] <= x < table[g+1].
__device__ __forceinline__ int find_group(const int *table, int groups, int x)
{
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Nonzero in one lane of a converged warp, always the same one.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

__device__ __forceinline__ void mbar_arrive_if(uint32_t on, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(on)
                 : "memory");
}

__device__ __forceinline__ void mbar_expect_if(uint32_t on, uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
                 "@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes), "r"(on)
                 : "memory");
}

__device__ __forceinline__ void tma_load_if(uint32_t on, uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z, uint64_t policy)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %7, 0;\n\t"
                 "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy), "r"(on)
                 : "memory");
}

__device__ __forceinline__ void mma_commit_if(uint32_t on, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                 "r"(on)
                 : "memory");
}

// Whether phase `parity` of the barrier is complete, without waiting. A wait
// costs over a hundred cycles even when there is nothing to wait for, so the
// loops below look at the next block's barriers while they work on this one,
// and wait only where that look came too early.
__device__ __forceinline__ uint32_t mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done;
}

// ptx::wait_phase_warp(), off the straight line: `early` is mbar_test()'s look.
#define TC_WAIT(early, bar, parity) \
    (__builtin_expect(__all_sync(0xffffffffu, (early)) != 0, 1) || ptx::wait_phase_warp(bar, parity))

// CHUNK consecutive columns of this warp's 32 lanes, and the wait for them.
// Tensor memory is not memory to the compiler: both are ordered among the
// volatile instructions (barriers, each other) and leave plain loads free to
// move; the wait is tied to the loaded registers, so that no use of them can
// be scheduled before it.
template <int CHUNK>
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, uint32_t (&v)[CHUNK])
{
    if constexpr (CHUNK == 32) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                     "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                       "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
                       "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
                       "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
                       "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                     : "r"(taddr));
    } else {
        static_assert(CHUNK == 16, "tensor memory chunk");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                     "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                       "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
                       "=r"(v[14]), "=r"(v[15])
                     : "r"(taddr));
    }
}

template <int CHUNK>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[CHUNK])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;");
#pragma unroll
    for (int j = 0; j < CHUNK; j += 8)
        asm volatile("" : "+r"(v[j]), "+r"(v[j + 1]), "+r"(v[j + 2]), "+r"(v[j + 3]), "+r"(v[j + 4]), "+r"(v[j + 5]),
                     "+r"(v[j + 6]), "+r"(v[j + 7]));
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t rank, float v)
{
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "st.shared::cluster.f32 [ra], %2;\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v)
                 : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_u32x4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_u32x4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fnp = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fnp, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fnp = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fnp);
    }();
    return encode;
}

}  // namespace sgemm_gb300
