// Block-scaled 8-bit products on the 5th-generation tensor cores:
//
//   C[m, n] = sum_kb sa[kb, m] * sb[kb, n] * (sum_{k in block kb} A[m, k] * B[n, k])  + beta * C[m, n]
//
// with A and B in e4m3, K contiguous, one scale for each 128 values along K
// (and, for weights, for 128 rows at once). The inner sums are
// tcgen05.mma .kind::f8f6f4 into tensor memory, one K block at a time; the
// outer, scaled sum is kept in FP32 registers, because the scales are FP32
// numbers that change with the block: each finished block is read back with
// tcgen05.ld and added with one FMA per element (two where both operands are
// scaled per row).
//
// Roles of a CTA:
//   warp 0      TMA producer: one 128-byte-wide slab of each operand per K
//               block (128-byte swizzle), full/empty barrier per stage;
//   warp 1      TMEM owner and MMA issuer: 4 MMAs (K 32 each) per block into
//               one of NBUF accumulators, then a commit that frees the stage
//               and hands the accumulator on;
//   warps 2, 3  warp 2 finds the CTA's tiles, up to four ahead, for all (found
//               by each role, a tile cost the adding warps 2000 cycles); both
//               copy the scales of the accumulator's columns, where each has
//               its own: asynchronous 4-byte copies into a ring, since rows of
//               scales start at any address;
//   warps 4..   promotion and epilogue: warp 4 + i reads lanes 32 (i % 4) ..
//               of accumulator columns (i / 4) * CW ..; its lanes' scales (and
//               the one that its columns share) it fetches itself, two K
//               blocks ahead (through the ring they cost 165 cycles a block).
//
// The 128 lanes of tensor memory hold rows of A and the columns rows of B
// ("wide"), or, where there are few rows of A, the other way round ("swap"):
// the tile then spends MMA columns, registers and promotion only on the rows
// of A there are, and reads each weight once.
//
// Work is a list of (token tile, weight tile) pairs, walked by a persistent
// grid. Grouped products find their groups from the offsets in device memory:
// every CTA builds the prefix sum of its groups' tiles (or K blocks) in
// shared memory first. A tile may read rows past its group's end: they are
// the next group's, or zero fill, and are never stored.
//
// Few tiles: `split` CTAs of a cluster share a tile's K blocks. Each sends its
// partial sums of column j to the shared memory of CTA j % split, and after a
// cluster barrier that CTA adds the parts in rank order: the result does not
// depend on timing.
//
// Every wait is bounded; a role that gives up sets the device error word and
// goes to the teardown, which drains copies and MMAs.
//
// What bounds it, and what it measured (one GB300):
//   16384 x 4096 x 4096, blocks form: 217 us, 2.53 PFLOP/s, 1.33 times the
//   measured bf16 rate. MMAs alone would take 512 cycles a K block (N = 256);
//   it takes 830, the rest being the accumulator's round through commit,
//   barrier, read, add and release, with two accumulators to overlap it.
//   Counters at 4096^3 (69 us): tensor pipe 52 % active; shared memory gives
//   384 accesses of 128 bytes a block to the MMAs and 36 to the warps, and its
//   clients collide in under 1 % of the cycles.
//   4096 x 4096 x 4096 with scales per row of both operands: 97 us, 1190
//   cycles a block. There the warps read the columns' scales too: 384 + 620
//   accesses of shared memory a block are its bound (and an element takes two
//   operations).
//   16 x 4096 x 4096: 10.1 us, most of it launch, set-up and the two
//   barriers of a split tile; 48 experts of 2048 x 2048 on 2 rows each:
//   38.8 us, 5.2 TB/s of weights.
// Not taken: pairs of CTAs on 256 x 256 tiles (cta_group::2; 433 us: the
// round goes through two SMs), two accumulators of 128 columns with barriers
// of their own (285 us), C stored from the registers (225 us; gradients of
// 16 experts' 2048 x 2048 weights from 16383 rows 132 us for 124: the warps
// that add held a tile 1100 cycles a piece), waits that poll without a pause
// (241 to 304 us: they take issue slots from the warps that add).
#include "common.cuh"
#include "experts.cuh"
#include "ptx.cuh"
#include "tc_roles.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <type_traits>

namespace sgemm_gb300 {

namespace {

constexpr int kScaleBatch = 2;   // K blocks whose scales are handed over together
constexpr int kItems = 4;        // tiles found ahead of their sums
constexpr int kItemBytes = 32;
constexpr int kStaging = 4096;   // a piece of a tile on its way to C: 128 bytes of each of a warp's 32 rows

template <int BN_, bool SWAP_>
struct Fp8Cfg {
    static constexpr int BN = BN_;
    static constexpr bool SWAP = SWAP_;
    static constexpr int ROW_BYTES = kBlock;                 // one K block per slab row
    static constexpr int P_TILE = 128 * ROW_BYTES;           // lanes' operand
    static constexpr int Q_TILE = BN * ROW_BYTES;            // columns' operand
    static constexpr int STAGE_BYTES = P_TILE + Q_TILE;
    static constexpr int STAGES = BN == 256 ? 3 : BN == 128 ? 4 : 7;   // more of 48 or 32 KB: the same time
    static constexpr int NBUF = BN == 256 ? 2 : 4;           // accumulators in tensor memory
    static constexpr int TMEM_COLS = NBUF * BN < 32 ? 32 : NBUF * BN;
    static constexpr int EPI_WARPS = BN >= 128 ? 8 : 4;
    static constexpr int CW = BN / (EPI_WARPS / 4);          // columns per epilogue warp
    // Columns per tcgen05.ld, of which two are in flight: 32 of them beside
    // 128 sums spill (302 us against 240 for 16 at 16384 x 4096 x 4096).
    static constexpr int CHUNK = CW < 32 || BN == 256 ? 16 : 32;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    // Registers move from the first four warps to the eight that hold up to
    // 128 sums per thread: 168 * 384 at launch, 72 * 128 + 216 * 256 (or
    // 88 * 128 + 208 * 256) after: the splits with the fewest spills.
    static constexpr int EPI_REGS = BN == 256 ? 216 : BN == 128 ? 208 : 0;
    static constexpr int SDEPTH = BN == 256 ? 4 : 6;         // ring of scales
    static constexpr int SLOT = kScaleBatch * BN;            // floats of one slot
    static constexpr bool CAN_SPLIT = SWAP;
    static constexpr int STAGING = SWAP ? 0 : EPI_WARPS * 2 * kStaging;
    static constexpr int PARTIAL = CAN_SPLIT ? BN * 128 * 4 : 0;
    static constexpr int NUM_BARS = 2 * STAGES + NBUF + 2 * SDEPTH + 2 * kItems + 1;
    static constexpr int OFF_STAGING = STAGES * STAGE_BYTES;
    static constexpr int OFF_PARTIAL = OFF_STAGING + STAGING;
    static constexpr int OFF_SCALES = OFF_PARTIAL + PARTIAL;
    static constexpr int OFF_ITEMS = OFF_SCALES + SDEPTH * SLOT * 4;
    static constexpr int OFF_TABLE = OFF_ITEMS + kItems * kItemBytes;
    static constexpr int OFF_BARS = OFF_TABLE + (kMaxGroups + 2) * 4;
    static constexpr int SMEM_BYTES = 1024 + OFF_BARS + NUM_BARS * 8 + 16;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tensor memory columns");
    static_assert(OFF_BARS % 8 == 0, "barrier alignment");
};

struct Fp8Params {
    int mode;
    int M, N;                    // rows of A, rows of B
    int nk;                      // K blocks in all
    const float *sa, *sb;
    int64_t ld_sa, ld_sb, stride_sb;
    int groups;
    const int32_t *offsets;
    int token_tiles;             // dense and grouped-K products; grouped rows: from the table
    int weight_tiles;
    FastDiv by_weights, by_group;   // weight_tiles; tiles of one group (grouped-K products)
    int split;
    float beta;
    void *C;
    int64_t ldc, stride_c;
    int c_bf16;
    int tma_c;                   // mapC holds C (whole 16-byte pieces, beta 0)
    unsigned int *status;
};

// One tile: its group, first row of A and of B, the end of its rows of A,
// its K blocks, and whether the CTA has another after it.
struct Fp8Item {
    int group, a_row, a_end, b_row, kb0, kb1, more;
};

// An item on its way through shared memory.
__device__ __forceinline__ void store_item(uint32_t at, const Fp8Item &w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w.group), "r"(w.a_row), "r"(w.a_end), "r"(w.b_row)
                 : "memory");
    asm volatile("st.shared.v4.u32 [%0+16], {%1,%2,%3,%3};" ::"r"(at), "r"(w.kb0), "r"(w.kb1), "r"(w.more) : "memory");
}

__device__ __forceinline__ Fp8Item load_item(uint32_t at)
{
    Fp8Item w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.group), "=r"(w.a_row), "=r"(w.a_end), "=r"(w.b_row)
                 : "r"(at)
                 : "memory");
    asm volatile("{\n\t.reg .u32 x;\n\tld.shared.v4.u32 {%0,%1,%2,x}, [%3+16];\n\t}"
                 : "=r"(w.kb0), "=r"(w.kb1), "=r"(w.more)
                 : "r"(at)
                 : "memory");
    return w;
}

constexpr int kRaster = 16;   // token tiles walked together, so that a wave of CTAs shares both operands in L2

template <class Cfg>
__device__ __forceinline__ Fp8Item fp8_item(const Fp8Params &p, const int *table, uint32_t t, int rank)
{
    constexpr int TT = Cfg::SWAP ? Cfg::BN : 128;    // rows of A per tile
    constexpr int WT = Cfg::SWAP ? 128 : Cfg::BN;    // rows of B per tile
    Fp8Item it;
    it.group = it.more = 0;
    int tokens = p.token_tiles;
    if (p.mode == kFp8GroupRows) tokens = table[p.groups];
    if (p.mode == kFp8GroupK) {
        it.group = (int)div(t, p.by_group);
        t -= it.group * p.by_group.d;
    }
    // Bands of kRaster token tiles, the token tile fastest.
    static_assert((kRaster & (kRaster - 1)) == 0, "a power of two");
    const uint32_t band = div(t / kRaster, p.by_weights), first = band * kRaster;
    const uint32_t r = t - first * p.weight_tiles;
    const uint32_t high = tokens - first;
    uint32_t wt, tt;
    if (high >= kRaster) {
        wt = r / kRaster;
        tt = first + r % kRaster;
    } else {
        wt = r / high;
        tt = first + r - wt * high;
    }
    it.b_row = (int)wt * WT;
    if (p.mode == kFp8GroupRows) {
        it.group = find_group(table, p.groups, (int)tt);
        int lo, hi;
        group_range(p.offsets, it.group, p.M, lo, hi);
        it.a_row = lo + ((int)tt - table[it.group]) * TT;
        it.a_end = hi;
    } else {
        it.a_row = (int)tt * TT;
        it.a_end = p.M;
    }
    int k0 = 0, k1 = p.nk;
    if (p.mode == kFp8GroupK) {
        k0 = table[it.group];
        k1 = table[it.group + 1];
    }
    it.kb0 = k0;
    it.kb1 = k1;
    if constexpr (Cfg::CAN_SPLIT) {
        if (p.split > 1) {
            it.kb0 = k0 + (int)((int64_t)(k1 - k0) * rank / p.split);
            it.kb1 = k0 + (int)((int64_t)(k1 - k0) * (rank + 1) / p.split);
        }
    }
    return it;
}

// One element of C, and old values where beta asks for them.
__device__ __forceinline__ void store_c(const Fp8Params &p, int64_t at, float v)
{
    if (p.c_bf16) {
        __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(p.C) + at;
        if (p.beta != 0.0f) v = fmaf(p.beta, __bfloat162float(*c), v);
        *c = __float2bfloat16_rn(v);
    } else {
        float *c = static_cast<float *>(p.C) + at;
        if (p.beta != 0.0f) v = fmaf(p.beta, *c, v);
        *c = v;
    }
}

// The loops of the roles are straight lines: a taken branch costs an
// instruction fetch of 50 to 100 cycles here, where twelve warps run five
// different pieces of code, and these loops have about 500 cycles per K block.
// So copies, MMAs and arrivals are predicated instructions (`on` nonzero in
// the one lane that issues them) instead of branches of one lane, loops run
// over whole batches of K blocks, and waits branch away only to wait.

// D (+)= P . Q^T on e4m3 operands.
__device__ __forceinline__ void mma_f8_if(uint32_t on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}

// Instruction descriptor of .kind::f8f6f4, both operands e4m3 (format 0) and
// K-major, FP32 accumulation.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const float *src, bool there)
{
    const int bytes = there ? 4 : 0;   // 0: writes a zero without reading
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// This thread's arrival on `bar` once its cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A box in shared memory (128-byte swizzle) to its place in C, asynchronously,
// as part of the thread's next bulk group.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}

// ROWS_FORM: B's scales are per row. COLS_SCALED: every column of the
// accumulator has a scale of its own, else the CW columns of a warp share one.
template <class Cfg, bool ROWS_FORM>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
fp8_product_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                   const __grid_constant__ CUtensorMap mapC, const __grid_constant__ Fp8Params p)
{
    constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES, NBUF = Cfg::NBUF, SD = Cfg::SDEPTH, CW = Cfg::CW;
    constexpr int CHUNK = Cfg::CHUNK;
    constexpr bool SWAP = Cfg::SWAP;
    constexpr bool COLS_SCALED = ROWS_FORM || SWAP;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    int *const table = reinterpret_cast<int *>(smem_raw + (base - raw) + Cfg::OFF_TABLE);
    const uint32_t bars = base + Cfg::OFF_BARS;
    auto stage_p = [&](int s) { return base + s * Cfg::STAGE_BYTES; };
    auto stage_q = [&](int s) { return base + s * Cfg::STAGE_BYTES + Cfg::P_TILE; };
    auto full_bar = [&](int s) { return bars + 8u * s; };
    // MMAs of a stage done: the stage is free and its accumulator is complete.
    auto done_bar = [&](int s) { return bars + 8u * (STAGES + s); };
    auto acce_bar = [&](int b) { return bars + 8u * (2 * STAGES + b); };
    auto sfull_bar = [&](int s) { return bars + 8u * (2 * STAGES + NBUF + s); };
    auto sempty_bar = [&](int s) { return bars + 8u * (2 * STAGES + NBUF + SD + s); };
    auto ifull_bar = [&](uint32_t i) { return bars + 8u * (2 * STAGES + NBUF + 2 * SD + i); };
    auto iempty_bar = [&](uint32_t i) { return bars + 8u * (2 * STAGES + NBUF + 2 * SD + kItems + i); };
    const uint32_t drain_bar = bars + 8u * (2 * STAGES + NBUF + 2 * SD + 2 * kItems);
    const uint32_t tmem_slot = bars + 8u * Cfg::NUM_BARS;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = Cfg::CAN_SPLIT ? p.split : 1;
    const int rank = split > 1 ? (int)ptx::cluster_ctarank() : 0;
    if (split > 1 && ptx::cluster_nctarank() != (uint32_t)split) {
        // Launched without its cluster, it would read peers that do not exist.
        if (threadIdx.x == 0) atomicOr(p.status, kStatusLaunchConfig);
        return;
    }

    if (warp == 2 && lane == 0) {
        ptx::prefetch_tensormap(&mapP);
        ptx::prefetch_tensormap(&mapQ);
        if (!SWAP && p.tma_c) ptx::prefetch_tensormap(&mapC);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(done_bar(s), 1);
        }
        for (int b = 0; b < NBUF; ++b) ptx::mbar_init(acce_bar(b), Cfg::EPI_WARPS);
        for (int s = 0; s < SD; ++s) {
            ptx::mbar_init(sfull_bar(s), 64);
            ptx::mbar_init(sempty_bar(s), Cfg::EPI_WARPS);
        }
        for (int i = 0; i < kItems; ++i) {
            // Read by the producer, the MMA issuer, the warps that store and,
            // where columns have scales, warp 3.
            ptx::mbar_init(ifull_bar(i), 1);
            ptx::mbar_init(iempty_bar(i), Cfg::EPI_WARPS + (COLS_SCALED ? 3 : 2));
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::mbar_init_fence();
    }
    if (warp == 1) ptx::tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    if (p.mode != kFp8Dense) {
        // table[g] = tiles (or K blocks) of the groups before g.
        const int unit = p.mode == kFp8GroupK ? kBlock : SWAP ? BN : 128;
        const int rows = p.mode == kFp8GroupK ? INT32_MAX : p.M;
        for (int g = threadIdx.x; g < p.groups; g += Cfg::THREADS) {
            int lo, hi;
            group_range(p.offsets, g, rows, lo, hi);
            table[g] = (int)(((uint32_t)(hi - lo) + (uint32_t)unit - 1) / (uint32_t)unit);
        }
        __syncthreads();
        if (warp == 0) {
            // Offsets that are not a partition may sum to anything: no entry
            // passes what the kernel can walk. (A group has at most 2^27
            // tiles, so 32 of them and a carry held to 2^27 stay below 2^32.)
            const uint32_t most = p.mode == kFp8GroupK ? (uint32_t)p.nk
                                                       : (uint32_t)(INT32_MAX / p.weight_tiles - 2 * kRaster);
            const uint32_t held = most < (1u << 27) ? most : 1u << 27;
            uint32_t carry = 0;
            for (int g0 = 0; g0 < p.groups; g0 += 32) {
                const int g = g0 + lane;
                const uint32_t mine = g < p.groups ? table[g] : 0;
                uint32_t sum = mine < held ? mine : held;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum = sum + up < held ? sum + up : held;
                }
                const uint32_t end = carry + sum < held ? carry + sum : held;
                const uint32_t before = __shfl_up_sync(0xffffffffu, end, 1);
                if (g < p.groups) table[g] = (int)(lane == 0 ? carry : before);
                carry = __shfl_sync(0xffffffffu, end, 31);
                if (g0 + 32 >= p.groups && lane == 0) table[p.groups] = (int)carry;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // The CTAs of a split tile write into each other's shared memory in the
    // end: each says that it has begun, and waits for the others before that.
    if (Cfg::CAN_SPLIT && split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const uint32_t taddr = *reinterpret_cast<uint32_t *>(smem_raw + (tmem_slot - raw));

    const uint32_t t_first = blockIdx.x / split, t_step = gridDim.x / split;
    uint32_t tiles = (uint32_t)p.weight_tiles * (uint32_t)(p.mode == kFp8Dense       ? p.token_tiles
                                                           : p.mode == kFp8GroupRows ? table[p.groups]
                                                                                     : p.token_tiles * p.groups);
    if (split > 1 && tiles > t_step) tiles = t_step;   // a split grid has one tile per cluster

    // The CTA's nth tile, once warp 2 has found it; not to be read after done_with().
    auto item_at = [&](uint32_t n) { return base + Cfg::OFF_ITEMS + (n % kItems) * kItemBytes; };
    auto item_there = [&](uint32_t n) {
        const uint32_t bar = ifull_bar(n % kItems), phase = (n / kItems) & 1;
        return TC_WAIT(mbar_test(bar, phase), bar, phase);
    };
    auto done_with = [&](uint32_t n) {
        __syncwarp();
        mbar_arrive_if(lane == 0, iempty_bar(n % kItems));
    };

    if constexpr (Cfg::EPI_REGS > 0) {
        if (warp < 4) ptx::setmaxnreg_dec<BN == 256 ? 72 : 88>();
    }
    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        const uint32_t on = elect_one();
        const uint64_t policy = ptx::policy_evict_last();
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (uint32_t t = t_first; ok && t < tiles; t += t_step, ++n) {
            if (!item_there(n)) {
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
                break;
            }
            const Fp8Item w = load_item(item_at(n));
            done_with(n);
            const int z = p.mode == kFp8GroupRows ? w.group : 0;
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const int s = (int)(it % STAGES);
                const uint32_t phase = ((it / STAGES) & 1) ^ 1;
                if (!TC_WAIT(mbar_test(done_bar(s), phase), done_bar(s), phase)) {
                    if (lane == 0) atomicOr(p.status, kStatusTimeout);
                    ok = false;
                    break;
                }
                mbar_expect_if(on, full_bar(s), Cfg::STAGE_BYTES);
                tma_load_if(on, stage_p(s), &mapP, full_bar(s), kb * kBlock, SWAP ? w.b_row : w.a_row, SWAP ? z : 0,
                            policy);
                tma_load_if(on, stage_q(s), &mapQ, full_bar(s), kb * kBlock, SWAP ? w.a_row : w.b_row, SWAP ? 0 : z,
                            policy);
            }
        }
        // Every byte bound for this CTA lands before it leaves.
        for (uint32_t back = 0; back < STAGES && back < it; ++back) {
            const uint32_t i = it - 1 - back;
            if (!ptx::wait_phase_warp(full_bar((int)(i % STAGES)), (i / STAGES) & 1) && lane == 0)
                atomicOr(p.status, kStatusTimeout);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        constexpr uint32_t idesc = idesc_e4m3(128, BN);
        const uint64_t desc_p = ptx::sdesc_kmajor(stage_p(0), Cfg::ROW_BYTES);
        const uint64_t desc_q = ptx::sdesc_kmajor(stage_q(0), Cfg::ROW_BYTES);
        const uint32_t on = elect_one();
        uint32_t it = 0, early = 0, n = 0;
        bool ok = true;
        for (uint32_t t = t_first; ok && t < tiles; t += t_step, ++n) {
            if (!item_there(n)) {
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
                break;
            }
            const Fp8Item w = load_item(item_at(n));
            done_with(n);
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const int s = (int)(it % STAGES), b = (int)(it % NBUF);
                const uint32_t full = (it / STAGES) & 1, free = ((it / NBUF) & 1) ^ 1, next = it + 1;
                if (!TC_WAIT(mbar_test(full_bar(s), full), full_bar(s), full) || !TC_WAIT(early, acce_bar(b), free)) {
                    if (lane == 0) atomicOr(p.status, kStatusTimeout);
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                // Addresses in the descriptors count 16 bytes.
                const uint32_t d = taddr + (uint32_t)(b * BN);
                const uint64_t off = (uint64_t)(s * (Cfg::STAGE_BYTES / 16));
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f8_if(on, d, desc_p + off + 2 * ks, desc_q + off + 2 * ks, idesc, ks != 0 ? 1u : 0u);
                mma_commit_if(on, done_bar(s));
                early = mbar_test(acce_bar((int)(next % NBUF)), ((next / NBUF) & 1) ^ 1);
            }
        }
        // Everything issued finishes before TMEM is released.
        mma_commit_if(on, drain_bar);
        if (!ptx::wait_phase_warp(drain_bar, 0) && lane == 0) atomicOr(p.status, kStatusTimeout);
    } else if (warp < 4) {
        // -------------------------- tiles and scales --------------------------
        // Warp 2 finds the tiles, ahead of the others. A slot of the scales
        // holds BN of them for each of up to kScaleBatch K blocks of a tile.
        const int th = threadIdx.x - 64;
        uint32_t it = 0, n = 0;
        bool ok = COLS_SCALED || warp == 2;
        for (uint32_t t = t_first; ok && t < tiles; t += t_step, ++n) {
            Fp8Item w;
            if (warp == 2) {
                w = fp8_item<Cfg>(p, table, t, rank);
                w.more = t + t_step < tiles;
                // The place is free when the tile kItems before is stored; a
                // wait's limit is far above the time of 2^16 K blocks.
                const uint32_t bar = iempty_bar(n % kItems), phase = ((n / kItems) & 1) ^ 1;
                ok = ptx::wait_phase_warp(bar, phase);
                for (int k = p.nk >> 16; !ok && k > 0; --k) ok = ptx::wait_phase_warp(bar, phase);
                if (ok && lane == 0) store_item(item_at(n), w);
                mbar_arrive_if(ok && lane == 0, ifull_bar(n % kItems));
            } else {
                ok = item_there(n);
                if (ok) {
                    w = load_item(item_at(n));
                    done_with(n);
                }
            }
            if (!ok) {
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
                break;
            }
            if (!COLS_SCALED) continue;
            const float *src = SWAP ? p.sa : p.sb;
            const int64_t ld = SWAP ? p.ld_sa : p.ld_sb;
            const int first = SWAP ? w.a_row : w.b_row, end = SWAP ? w.a_end : p.N;
            for (int k0 = w.kb0; k0 < w.kb1; k0 += kScaleBatch, ++it) {
                const int s = (int)(it % SD);
                if (!ptx::wait_phase_warp(sempty_bar(s), ((it / SD) & 1) ^ 1)) {
                    if (lane == 0) atomicOr(p.status, kStatusTimeout);
                    ok = false;
                    break;
                }
                const uint32_t slot = base + Cfg::OFF_SCALES + s * (Cfg::SLOT * 4);
#pragma unroll
                for (int j = 0; j < kScaleBatch; ++j) {
                    if (k0 + j >= w.kb1) break;
                    const float *sk = src + (int64_t)(k0 + j) * ld;
#pragma unroll
                    for (int i = th; i < BN; i += 64) {
                        const bool there = first + i < end;
                        cp_async_4(slot + 4 * (BN * j + i), there ? sk + first + i : src, there);
                    }
                }
                cp_async_arrive(sfull_bar(s));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------ promotion and epilogue ------------------------
        const int ew = warp - 4, q = ew & 3, half = ew >> 2;
        const int row = 32 * q + lane;                    // lane of tensor memory
        const uint32_t lanes = taddr + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * CW);
        const float *const slots = reinterpret_cast<const float *>(smem_raw + (base - raw) + Cfg::OFF_SCALES);
        if (Cfg::CAN_SPLIT && split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if constexpr (Cfg::EPI_REGS > 0) ptx::setmaxnreg_inc<Cfg::EPI_REGS>();
        uint32_t it = 0, batch = 0, n = 0;
        bool ok = true;
        // Where the next K block's scales are: this lane's, and the one that
        // this warp's columns share. Past a tile's last block the place stays,
        // and rows that are not stored read the last one's: loads without
        // conditions, hence without branches.
        const float *lane_at = p.sa, *cols_at = p.sb;
        float lane_next[kScaleBatch], cols_next[kScaleBatch];
        const int64_t lane_step = !SWAP ? p.ld_sa : ROWS_FORM ? p.ld_sb : 1;
        auto fetch = [&](int kb, int kb1) {
#pragma unroll
            for (int j = 0; j < kScaleBatch; ++j) {
                lane_next[j] = __ldg(lane_at);
                if constexpr (!COLS_SCALED) cols_next[j] = __ldg(cols_at);
                const bool last = kb + j + 1 >= kb1;
                lane_at += last ? 0 : lane_step;
                if constexpr (!COLS_SCALED) cols_at += last ? 0 : 1;
            }
        };
        auto start = [&](const Fp8Item &w) {
            if (w.kb0 >= w.kb1) return;
            const float *sbg = p.sb + (p.mode == kFp8GroupRows ? w.group * p.stride_sb : 0);
            if constexpr (!SWAP) {
                lane_at = p.sa + (int64_t)w.kb0 * p.ld_sa + (w.a_row + row < w.a_end ? w.a_row + row : w.a_end - 1);
            } else if constexpr (ROWS_FORM) {
                lane_at = p.sb + (int64_t)w.kb0 * p.ld_sb + (w.b_row + row < p.N ? w.b_row + row : p.N - 1);
            } else {
                lane_at = sbg + (int64_t)(w.b_row / 128) * p.ld_sb + w.kb0;
            }
            if constexpr (!COLS_SCALED) {
                const int col = w.b_row + half * CW;
                cols_at = sbg + (int64_t)((col < p.N ? col : p.N - 1) / 128) * p.ld_sb + w.kb0;
            }
            fetch(w.kb0, w.kb1);
        };
        // Of a tile the sums' loop keeps its K blocks alone: the store reads
        // it again. (Registers: what the store needs, kept through the loop,
        // spills there and costs a quarter of its speed.)
        int kb0 = 0, kb1 = 0;
        auto enter = [&](uint32_t i) {
            if (!item_there(i)) {
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
                ok = false;
                return;
            }
            const Fp8Item w = load_item(item_at(i));
            start(w);
            kb0 = w.kb0;
            kb1 = w.kb1;
        };
        bool more = t_first < tiles;
        if (more) enter(0);
        for (; ok && more; ++n) {
            float2 acc[CW / 2];
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            // The loads run one chunk ahead of the sums, across K blocks too:
            // the next block's first chunk is requested before this block's
            // last one is added.
            uint32_t v[2][CHUNK];
            float fl[kScaleBatch] = {};
            const float *cols = nullptr;                  // the batch's slot, this warp's columns
            // Waits for block i's sums and requests their first chunk.
            auto begin = [&](uint32_t i, uint32_t early, uint32_t (&dst)[CHUNK]) {
                ok = ok && TC_WAIT(early, done_bar((int)(i % STAGES)), (i / STAGES) & 1);
                ptx::tc_fence_after();
                tmem_ld_chunk<CHUNK>(lanes + (uint32_t)((int)(i % NBUF) * BN), dst);
            };
            auto add = [&](int j0, int c0, const uint32_t (&x)[CHUNK]) {
                const float2 f2 = make_float2(fl[j0], fl[j0]);
#pragma unroll
                for (int j = 0; j < CHUNK; j += 4) {
                    const float2 v0 = make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                    const float2 v1 = make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
                    float2 &a0 = acc[(c0 + j) / 2], &a1 = acc[(c0 + j) / 2 + 1];
                    if constexpr (COLS_SCALED) {
                        const float4 sc = *reinterpret_cast<const float4 *>(cols + BN * j0 + c0 + j);
                        a0 = __ffma2_rn(__fmul2_rn(v0, f2), make_float2(sc.x, sc.y), a0);
                        a1 = __ffma2_rn(__fmul2_rn(v1, f2), make_float2(sc.z, sc.w), a1);
                    } else {
                        a0 = __ffma2_rn(v0, f2, a0);
                        a1 = __ffma2_rn(v1, f2, a1);
                    }
                }
            };
            constexpr int NCH = CW / CHUNK;
            // Block j of a batch, whose first chunk has been requested: adds it,
            // and requests the first chunk of the block after it, if any.
            auto block = [&](auto J, bool more) {
                constexpr int j = decltype(J)::value;
                const int b = (int)(it % NBUF);
                const uint32_t next = it + 1;
                uint32_t early = 0;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int at = NCH == 1 ? j & 1 : c & 1;
                    tmem_ld_wait_for<CHUNK>(v[at]);
                    if (c + 1 < NCH) tmem_ld_chunk<CHUNK>(lanes + (uint32_t)(b * BN + (c + 1) * CHUNK), v[at ^ 1]);
                    if (c == 0) early = mbar_test(done_bar((int)(next % STAGES)), (next / STAGES) & 1);
                    if (c + 1 == NCH) {
                        // The accumulator is read: the MMA warp may reuse it.
                        ptx::tc_fence_before();
                        mbar_arrive_if(lane == 0, acce_bar(b));
                        if (more) begin(next, early, v[at ^ 1]);
                    }
                    add(j, c * CHUNK, v[at]);
                }
                ++it;
            };
            static_assert((NCH == 1 || NCH % 2 == 0) && kScaleBatch == 2, "chunks alternate between two buffers");
            using std::integral_constant;
            if (kb0 < kb1) begin(it, mbar_test(done_bar((int)(it % STAGES)), (it / STAGES) & 1), v[0]);
            for (int kb = kb0; ok && kb < kb1; kb += kScaleBatch) {
                const int left = kb1 - kb;
#pragma unroll
                for (int j = 0; j < kScaleBatch; ++j) fl[j] = COLS_SCALED ? lane_next[j] : lane_next[j] * cols_next[j];
                fetch(kb + kScaleBatch, kb1);
                if constexpr (COLS_SCALED) {
                    const int s = (int)(batch % SD);
                    const uint32_t phase = (batch / SD) & 1;
                    ok = ok && TC_WAIT(mbar_test(sfull_bar(s), phase), sfull_bar(s), phase);
                    cols = slots + s * Cfg::SLOT + half * CW;
                }
                if (left >= kScaleBatch) {
                    block(integral_constant<int, 0>{}, true);
                    block(integral_constant<int, 1>{}, left > kScaleBatch);
                } else {
                    block(integral_constant<int, 0>{}, false);
                }
                if constexpr (COLS_SCALED) {
                    __syncwarp();
                    mbar_arrive_if(lane == 0, sempty_bar((int)(batch % SD)));
                    ++batch;
                }
            }
            if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
            if (!ok && split == 1) break;
            // The next tile's first scales are on their way while this one is stored.
            more = ld_shared_u32(item_at(n) + 24) != 0;
            if (more) enter(n + 1);
            const Fp8Item w = load_item(item_at(n));
            done_with(n);
            const int64_t c_base = p.mode == kFp8GroupK ? w.group * p.stride_c : 0;
            if constexpr (SWAP) {
                // Lane = row of B (column of C), column = row of A.
                if (split == 1) {
                    const int n = w.b_row + row, m0 = w.a_row + half * CW;
                    const int rows = n < p.N ? w.a_end - m0 : 0;
                    const int64_t at = c_base + (int64_t)m0 * p.ldc + n;
                    if (p.c_bf16 && p.beta == 0.0f) {
                        __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(p.C) + at;
#pragma unroll
                        for (int j = 0; j < CW; ++j, c += p.ldc)
                            if (j < rows) *c = __float2bfloat16_rn((j & 1) ? acc[j / 2].y : acc[j / 2].x);
                    } else if (p.beta == 0.0f) {
                        float *c = static_cast<float *>(p.C) + at;
#pragma unroll
                        for (int j = 0; j < CW; ++j, c += p.ldc)
                            if (j < rows) *c = (j & 1) ? acc[j / 2].y : acc[j / 2].x;
                    } else {
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            if (j < rows) store_c(p, at + j * p.ldc, (j & 1) ? acc[j / 2].y : acc[j / 2].x);
                    }
                } else {
                    // To the CTA that adds column j over the cluster: j % split.
                    const int per = BN / split, shift = __ffs(split) - 1;
                    const uint32_t mine = base + Cfg::OFF_PARTIAL + 4 * (rank * per * 128 + row);
#pragma unroll
                    for (int j = 0; j < CW; ++j) {
                        const int col = half * CW + j;
                        st_cluster_f32(mine + 4 * 128 * (col >> shift), (uint32_t)(col & (split - 1)),
                                       (j & 1) ? acc[j / 2].y : acc[j / 2].x);
                    }
                }
            } else {
                // Lane = row of A; 128 bytes of each of 32 rows at a time go
                // through shared memory and leave by TMA, while the next piece
                // is written beside them and the next tile begun. Rows that
                // end inside the 32 at the next group's first, columns that
                // end inside the 128 bytes (TMA stores whole 16 bytes), and C
                // that TMA cannot address or that is read, are stored by the
                // lanes. (Read, beta != 0: one element after the other; 16
                // experts' 2048 x 2048 FP32 gradients 937 us, 115 with beta 0.)
                const int row0 = w.a_row + 32 * q;
                const bool whole_rows = p.mode != kFp8GroupRows || row0 + 32 <= w.a_end;
                // Writes 128 bytes of the warp's columns from h on: 32 floats, or 64 bfloat16.
                auto flush = [&](const uint32_t (&u)[32], int cols, int h) {
                    const int col0 = w.b_row + half * CW + h, place = (h / cols) & 1;
                    const uint32_t st = base + Cfg::OFF_STAGING + (2 * ew + place) * kStaging;
                    const bool pieces = p.tma_c && col0 + cols <= p.N, whole = pieces && whole_rows;
                    // The piece that was last here has left: the one before the
                    // last, or the last where a tile has only one.
                    if (lane == 0) {
                        if (cols < CW) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        st_shared_u32x4(st + 128 * lane + 16 * (c ^ (lane & 7)),
                                        make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]));
                    if (whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (whole && row0 < w.a_end)
                            tma_store(&mapC, st, col0, row0, p.mode == kFp8GroupK ? w.group : 0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // one group per piece, if empty
                    }
                    if (whole) return;
                    if (pieces) {
                        // 16 bytes per lane, of four rows at a time.
                        const int size = 128 / cols;
                        uint8_t *dst = static_cast<uint8_t *>(p.C) +
                                       (c_base + (int64_t)(row0 + (lane >> 3)) * p.ldc + col0) * size + 16 * (lane & 7);
#pragma unroll 4
                        for (int i = 0; i < 8; ++i) {
                            const int r = 4 * i + (lane >> 3), c = lane & 7;
                            if (row0 + r < w.a_end)
                                *reinterpret_cast<uint4 *>(dst) = ld_shared_u32x4(st + 128 * r + 16 * (c ^ (r & 7)));
                            dst += 4 * p.ldc * size;
                        }
                        return;
                    }
                    // Lane by lane, eight rows read before the first is stored.
                    const int64_t at = c_base + (int64_t)row0 * p.ldc + col0;
                    const int rows = w.a_end - row0;
#pragma unroll 1
                    for (int r0 = 0; r0 < 32; r0 += 8) {
                        uint32_t x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            x[i] = ld_shared_u32(st + 128 * (r0 + i) + 16 * ((lane >> 2) ^ i) + 4 * (lane & 3));
                        if (cols == 32) {
                            // Lane: column.
                            if (p.beta == 0.0f) {
                                float *c = static_cast<float *>(p.C) + at + r0 * p.ldc + lane;
#pragma unroll
                                for (int i = 0; i < 8; ++i, c += p.ldc)
                                    if (r0 + i < rows && col0 + lane < p.N) *c = __uint_as_float(x[i]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (r0 + i < rows && col0 + lane < p.N)
                                        store_c(p, at + (r0 + i) * p.ldc + lane, __uint_as_float(x[i]));
                            }
                        } else {
                            // Lane: columns 2 lane and 2 lane + 1.
                            uint16_t *c = static_cast<uint16_t *>(p.C) + at + r0 * p.ldc + 2 * lane;
#pragma unroll
                            for (int i = 0; i < 8; ++i, c += p.ldc)
                                if (r0 + i < rows) {
                                    if (col0 + 2 * lane < p.N) c[0] = (uint16_t)x[i];
                                    if (col0 + 2 * lane + 1 < p.N) c[1] = (uint16_t)(x[i] >> 16);
                                }
                        }
                    }
                };
                uint32_t u[32];
                if (p.c_bf16 && p.beta == 0.0f) {
#pragma unroll
                    for (int h = 0; h < CW; h += 64) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) u[j] = pack_bf16(acc[h / 2 + j].x, acc[h / 2 + j].y);
                        flush(u, 64, h);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < CW; h += 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            u[j] = __float_as_uint((j & 1) ? acc[h / 2 + j / 2].y : acc[h / 2 + j / 2].x);
                        flush(u, 32, h);
                    }
                }
            }
        }
        if (!SWAP && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
        ptx::tc_fence_before();
    }

    // ------------------------------ teardown ------------------------------
    if constexpr (Cfg::CAN_SPLIT) {
        if (split > 1) {
            __syncwarp();
            if (warp < 4) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            // One tile per cluster. Its columns' parts are here, one set per
            // CTA of the cluster; this CTA adds columns rank, rank + split, ..
            // in rank order. Nothing reaches into another CTA after this
            // barrier.
            ptx::cluster_sync_all();
            if (t_first < tiles) {
                const Fp8Item w = fp8_item<Cfg>(p, table, t_first, rank);
                const int64_t c_base = p.mode == kFp8GroupK ? w.group * p.stride_c : 0;
                const uint32_t part = base + Cfg::OFF_PARTIAL;
                const int per = BN / split;
                for (int i = threadIdx.x; i < per * 128; i += Cfg::THREADS) {
                    const int m = w.a_row + (i >> 7) * split + rank, n = w.b_row + (i & 127);
                    if (m < w.a_end && n < p.N) {
                        float v = 0.0f;
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            if (r < split) v += ld_shared_f32(part + 4 * (r * per * 128 + i));
                        store_c(p, c_base + (int64_t)m * p.ldc + n, v);
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(taddr, Cfg::TMEM_COLS);
    }
}

// Tensor map of an 8-bit operand: `rows` rows of K bytes, `groups` of them
// `stride` bytes apart, in boxes of one K block by box_rows rows.
cudaError_t encode_fp8(CUtensorMap *map, const uint8_t *ptr, int64_t rows, int64_t k, int64_t ld, int64_t groups,
                       int64_t stride, int box_rows)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)stride};
    const cuuint32_t box[3] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows, 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(ptr), dims, strides, box,
                              elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tensor map of C (of all groups' under grouped K), in boxes of 128 bytes by
// the 32 rows of an epilogue warp.
cudaError_t encode_c(CUtensorMap *map, const Fp8Args &g)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const int64_t size = g.c_bf16 ? 2 : 4, many = g.mode == kFp8GroupK ? g.groups : 1;
    const cuuint64_t dims[3] = {(cuuint64_t)g.N, (cuuint64_t)g.M, (cuuint64_t)many};
    const cuuint64_t strides[2] = {(cuuint64_t)(g.ldc * size), (cuuint64_t)((many > 1 ? g.stride_c : g.M * g.ldc) * size)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), 32, 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = encode(map, g.c_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, g.C,
                              dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

using Wide256 = Fp8Cfg<256, false>;
using Wide128 = Fp8Cfg<128, false>;
using Swap64 = Fp8Cfg<64, true>;
using Swap32 = Fp8Cfg<32, true>;
using Swap16 = Fp8Cfg<16, true>;

template <class Cfg>
cudaError_t prepare_cfg()
{
    cudaError_t e = cudaFuncSetAttribute(fp8_product_kernel<Cfg, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fp8_product_kernel<Cfg, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg::SMEM_BYTES);
}

template <class Cfg>
cudaError_t launch_cfg(const Fp8Args &g, const Fp8Plan &plan, cudaStream_t stream)
{
    constexpr int tt = Cfg::SWAP ? Cfg::BN : 128, wt = Cfg::SWAP ? 128 : Cfg::BN;
    CUtensorMap map_a, map_b;
    const int64_t bg = g.mode == kFp8GroupRows ? g.groups : 1;
    const int64_t sb = bg > 1 ? g.stride_b : (g.N * g.ldb);
    cudaError_t e;
    if (g.K > 0) {
        e = encode_fp8(&map_a, g.A, g.M, g.K, g.lda, 1, g.M * g.lda, tt);
        if (e == cudaSuccess) e = encode_fp8(&map_b, g.B, g.N, g.K, g.ldb, bg, sb, wt);
    } else {
        // The empty sum: no copy is ever issued, the maps only have to be valid.
        const uint8_t *any = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(g.C) & ~uintptr_t(15));
        e = encode_fp8(&map_a, any, 1, 1, 16, 1, 16, tt);
        if (e == cudaSuccess) e = encode_fp8(&map_b, any, 1, 1, 16, 1, 16, wt);
    }
    if (e != cudaSuccess) return e;
    Fp8Params p{};
    p.mode = g.mode;
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.nk = (int)ceil_div(g.K, kBlock);
    p.sa = g.sa;
    p.sb = g.sb;
    p.ld_sa = g.ld_sa;
    p.ld_sb = g.ld_sb;
    p.stride_sb = g.stride_sb;
    p.groups = g.groups;
    p.offsets = g.offsets;
    p.token_tiles = (int)ceil_div(g.M, tt);
    p.weight_tiles = (int)ceil_div(g.N, wt);
    // Tiles are counted in 32 bits (2^31 of them would be a C of 2^42 elements).
    const int64_t groups_hit = g.groups < g.M ? g.groups : g.M;
    const int64_t tokens = g.mode == kFp8Dense ? p.token_tiles
                           : g.mode == kFp8GroupRows ? g.M / tt + groups_hit : (int64_t)p.token_tiles * g.groups;
    if (tokens + 2 * kRaster > INT32_MAX / p.weight_tiles - 2 * kRaster) return cudaErrorInvalidValue;
    p.by_weights = fast_div((uint32_t)p.weight_tiles);
    p.by_group = fast_div((uint32_t)((int64_t)p.token_tiles * p.weight_tiles));
    p.split = plan.split;
    p.beta = g.beta;
    p.C = g.C;
    p.ldc = g.ldc;
    p.stride_c = g.stride_c;
    p.c_bf16 = g.c_bf16;
    p.status = g.status;
    CUtensorMap &mp = Cfg::SWAP ? map_b : map_a, &mq = Cfg::SWAP ? map_a : map_b;
    CUtensorMap map_c = map_a;                        // any valid one where C goes without
    const int64_t per16 = g.c_bf16 ? 8 : 4;
    if (!Cfg::SWAP && g.beta == 0.0f && (reinterpret_cast<uintptr_t>(g.C) & 15u) == 0 && g.ldc % per16 == 0 &&
        (g.mode != kFp8GroupK || g.stride_c % per16 == 0))
        p.tma_c = encode_c(&map_c, g) == cudaSuccess ? 1 : 0;
    void *args[] = {&mp, &mq, &map_c, &p};
    const void *fn = g.rows_form ? reinterpret_cast<const void *>(fp8_product_kernel<Cfg, true>)
                                 : reinterpret_cast<const void *>(fp8_product_kernel<Cfg, false>);
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attrs[1];
    if (plan.split > 1) {
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = (unsigned)plan.split;
        attrs[0].val.clusterDim.y = 1;
        attrs[0].val.clusterDim.z = 1;
        lc.attrs = attrs;
        lc.numAttrs = 1;
    }
    lc.gridDim = dim3((unsigned)plan.grid);
    lc.blockDim = dim3(Cfg::THREADS);
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = stream;
    e = cudaLaunchKernelExC(&lc, fn, args);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Which kernel, by sizes (152 SMs, N = K = 4096 or 64 experts of 2048 x 2048;
// us):
//   rows of A per group up to 16, 32, 64: as many columns, B on the lanes. 16
//   rows 10.1; 64 rows 12.5, on 128 x 128 tiles 17.6.
//   65 to 128 rows: 128 x 128 tiles with A on the lanes where they fill half
//   the SMs (128 x 16384: 22.1 against 26.5; 8000 rows over the experts 75.6
//   against 97.2), else 64 columns with split tiles (128 x 4096: 14.6 against
//   17.6).
//   More: 128 x 256 or 128 x 128 tiles, by their waves of CTAs, a wave of the
//   latter counted as 3/4 of one of the former (N = K = 4096: 512 rows, one
//   wave of either, 23.2 and 17.0; 1024 rows, one and two, 23.2 and 27.3; 1280
//   rows, two and three, 37.5 and 35.5, where the rule takes the former; 2048
//   rows, two and four, 39.6 and 45.7).
// Groups go by their average: how many rows each has only the device knows.
// 2048 rows over 64 experts are given 32 columns a tile, and where all are in
// two of them these read their weights 32 times (38.5; as two groups 17.0).
Fp8Plan plan_fp8(const Fp8Args &g)
{
    const int64_t nk = ceil_div(g.K, kBlock), sms = g.num_sms;
    const int64_t per = g.mode == kFp8GroupRows ? ceil_div(g.M, g.groups) : g.M;
    // Tiles of tt rows of A by wt of B; for groups of rows, at most.
    auto tiles_of = [&](int64_t tt, int64_t wt) {
        const int64_t hit = g.groups < g.M ? g.groups : g.M;
        const int64_t tokens = g.mode == kFp8GroupRows ? g.M / tt + hit : ceil_div(g.M, tt);
        return tokens * ceil_div(g.N, wt) * (g.mode == kFp8GroupK ? g.groups : 1);
    };
    Fp8Plan p{256, false, 1, 0};
    if (g.mode != kFp8GroupK && per <= 64) {
        p.swap = true;
        p.cols = per <= 16 ? 16 : per <= 32 ? 32 : 64;
    } else if (g.mode != kFp8GroupK && per <= 128) {
        p.swap = 2 * tiles_of(128, 128) < sms;
        p.cols = p.swap ? 64 : 128;
    } else if (4 * ceil_div(tiles_of(128, 256), sms) > 3 * ceil_div(tiles_of(128, 128), sms)) {
        p.cols = 128;
    }
    const int64_t tiles = p.swap ? tiles_of(p.cols, 128) : tiles_of(128, p.cols);
    // Few tiles: clusters of 2, 4 or 8 CTAs share each tile's K blocks.
    if (p.swap)
        while (p.split < 8 && tiles * p.split * 2 <= sms && nk >= p.split * 4) p.split *= 2;
    const int64_t most = sms / p.split * p.split;
    p.grid = tiles * p.split < most ? tiles * p.split : most;
    return p;
}

cudaError_t prepare_fp8()
{
    cudaError_t e = prepare_cfg<Wide256>();
    if (e == cudaSuccess) e = prepare_cfg<Wide128>();
    if (e == cudaSuccess) e = prepare_cfg<Swap64>();
    if (e == cudaSuccess) e = prepare_cfg<Swap32>();
    if (e == cudaSuccess) e = prepare_cfg<Swap16>();
    return e;
}

cudaError_t launch_fp8(const Fp8Args &g, cudaStream_t stream)
{
    const Fp8Plan p = plan_fp8(g);
    if (!p.swap) return p.cols == 256 ? launch_cfg<Wide256>(g, p, stream) : launch_cfg<Wide128>(g, p, stream);
    return p.cols == 16   ? launch_cfg<Swap16>(g, p, stream)
           : p.cols == 32 ? launch_cfg<Swap32>(g, p, stream)
                          : launch_cfg<Swap64>(g, p, stream);
}

}  // namespace sgemm_gb300
