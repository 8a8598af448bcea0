// Products of bfloat16 operands on the 5th-generation tensor cores, with an
// epilogue:
//
//   z[m, n] = sum_k op(A)[m, k] op(B)[k, n] + bias[n]     (pre = z on request)
//   C[m, n] = act(z[m, n])  [+ D[m, n]  or  * D[m, n]]
//
// dense, over groups of rows of A with a B (and bias) each, or over each
// group's rows as K (tcgen05.mma .kind::f16, FP32 sums in tensor memory). The
// epilogue is FP32, with one rounding as C and pre are stored. The tensor
// cores cut the sums off with each 16 of K instead of rounding them, which
// adds up along K: measured, sums of random sign are off by 1.7e-6 at K = 2049
// and 4.4e-6 at 4096, and sums of positive values, where each cut is a loss,
// lose 6e-9 K of their size on average (1.6e-3 at 2^18, 6.6e-3 at 2^20). So an
// FP32 C is summed in tensor memory over 768 of K at a time, and these sums in
// FP32 registers; a bfloat16 C, whose rounding takes up to 3.9e-3, over 8192 of
// K at a time (a loss of 4e-5).
//
// A tile has 128 (or, by a pair of CTAs, 256) lanes of tensor memory, which
// hold rows of C, and BN columns, which hold columns of C; with `swap` it is
// the other way round, so that few rows of A cost few columns and each value
// of B is read once. Operands come by TMA in slabs of 64 along K with the
// 128-byte swizzle: one box where K is contiguous, boxes of 64 x 64 where the
// rows (or columns) of C are; the MMA reads either from its descriptor.
//
// Roles of a CTA:
//   warp 0      TMA producer, full/done barrier per stage;
//   warp 1      TMEM owner and MMA issuer, two accumulators;
//   warp 2      finds the CTA's tiles, up to four ahead, for all;
//   warp 3      over groups' rows as K: zeroes the rows of a group's last slab
//               that are the next group's (infinities and NaN there must not
//               meet this group's), as far as an MMA of 16 reads them;
//   warps 4..   epilogue: warp 4 + i reads lanes 32 (i % 4) .. of columns
//               (i / 4) * CW .., 32 columns at a time, which turn in shared
//               memory so that D, pre and C are accessed along rows.
//
// Pairs (cta_group::2): each CTA loads its 128 rows of the lanes' operand and
// half of the columns' operand, and the first CTA's MMA warp issues for both.
// Few tiles: `split` CTAs of a cluster share a tile's K slabs; each sends its
// partial sums of column j to the CTA j % split, which adds them in rank order
// after a cluster barrier: the result does not depend on timing.
//
// Every wait is bounded; a role that gives up sets the device error word and
// goes to the teardown, which drains copies and MMAs.
//
// What bounds it, and what it measured (one GB300, in a row of calls):
//   16384 x 4096 x 4096, bfloat16: 284 to 326 us, 1.9 to 1.7 PFLOP/s, bound by
//   the tensor cores and, in a long row of calls, the power cap on the clock (the
//   library's product in the same run: 282 to 316); with bias, gelu_tanh and pre
//   293 to 342 (tensor pipe 90 % active). MMAs and copies want their operands in
//   registers that a warp shares: without uniform() it took 306 for 286. A CTA
//   per tile of 128 x 128 instead of pairs took 457 for 286.
//   4097 x 3001 x 2049 into FP32 with bias, gelu and D: 89 us (tensor pipe
//   25 % active, issue slots 32 %). Cold 95; with rows on 16 bytes 72, without
//   D 70, without bias and gelu 87: a D off 16 bytes arrives a chunk at a time.
//   16384 rows over 60 experts of 2048 x 2048 with silu and a factor: 147 us;
//   741 MB (operands, D and C are 705), DRAM 62 % busy, tensor pipe 43 %.
//   16 x 4096 x 4096: 17 us with cold caches (the weights alone 5; DRAM 24 %
//   busy), 11 where a part of the weights is still in L2.
//   96 rows over 48 experts: 68 to 70 us, the weights at 5.8 TB/s.
// Not taken: FP32 D held in registers for a whole chunk (100 us for 89, it
// spills); groups of rows cut into pieces for their last wave (no change).
#include "common.cuh"
#include "layers.cuh"
#include "ptx.cuh"
#include "row_pieces.cuh"
#include "tc_roles.cuh"

namespace sgemm_gb300 {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSlab = 64;        // K values per stage: 128 bytes of a row
constexpr int kPart = 12 * kSlab;          // K that an FP32 C (and a split tile) is summed over in tensor memory
constexpr int kPartBf16 = 128 * kSlab;     // the same of a bfloat16 C
constexpr int kItems = 4;        // tiles found ahead of their sums
constexpr int kItemBytes = 32;
constexpr int kStaging = 4096;   // 32 x 32 floats on their way to C
constexpr int kRaster = 16;      // row tiles walked together, so that a wave of CTAs shares both operands in L2

// JOINS: D comes ahead of the sums, by TMA or asynchronous copies. With 32 KB
// of operands per 512 cycles and several stages of them on their way, a load of
// D's by the warps that use it waits 2500 cycles in the queue (16384 rows over
// 60 experts of 2048 x 2048 with silu and a factor 165 us, with D ahead 152).
template <int BN_, bool PAIR_, bool JOINS_ = false>
struct Bf16Cfg {
    static constexpr int BN = BN_;
    static constexpr bool PAIR = PAIR_, JOINS = JOINS_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int LANES = 128 * CTAS;
    static constexpr int QR = BN / CTAS;                           // rows of the columns' operand a CTA loads
    static constexpr int P_TILE = 128 * 128;
    static constexpr int Q_TILE = (QR < 64 ? 64 : QR) * 128;       // a box of 64 x 64 at least
    static constexpr int STAGE_BYTES = P_TILE + Q_TILE;
    static constexpr int STAGES = PAIR ? (BN == 256 ? 6 : 8) - (JOINS ? BN == 256 ? 2 : 3 : 0) : BN == 128 ? 5 : 8;
    static constexpr int NBUF = 2;
    static constexpr int TMEM_COLS = NBUF * BN < 32 ? 32 : NBUF * BN;
    static constexpr int EPI_WARPS = BN >= 128 ? 8 : 4;
    static constexpr int CW = BN / (EPI_WARPS / 4);                // columns per epilogue warp
    static constexpr int CHUNK = CW < 32 ? 16 : 32;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    // Registers move from the first four warps to the eight of the epilogue:
    // 168 * 384 at launch, 72 * 128 + 216 * 256 after.
    static constexpr bool MOVE_REGS = EPI_WARPS == 8;
    static constexpr bool CAN_SPLIT = !PAIR;
    // Partial sums of a split tile lie where whole tiles are staged.
    static constexpr int PARTIAL = CAN_SPLIT ? BN * 128 * 4 : 0;
    static constexpr int EXTRA = PARTIAL > EPI_WARPS * kStaging ? PARTIAL : EPI_WARPS * kStaging;
    // Each epilogue warp's chunks of D: four of bfloat16 or two of floats.
    static constexpr int D_BYTES = JOINS ? 4 * 32 * 32 * 2 : 0;
    static constexpr int D_BARS = JOINS ? 4 * EPI_WARPS : 0;
    static constexpr int NUM_BARS = 3 * STAGES + 2 * NBUF + 2 * kItems + 1 + D_BARS;
    static constexpr int OFF_EXTRA = STAGES * STAGE_BYTES;
    static constexpr int OFF_D = OFF_EXTRA + EXTRA;
    static constexpr int OFF_ITEMS = OFF_D + EPI_WARPS * D_BYTES;
    static constexpr int OFF_TABLE = OFF_ITEMS + kItems * kItemBytes;
    static constexpr int OFF_BARS = OFF_TABLE + (kMaxGroups + 2) * 4;
    static constexpr int SMEM_BYTES = OFF_BARS + NUM_BARS * 8 + 16;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tensor memory columns");
    static_assert(OFF_BARS % 8 == 0 && STAGE_BYTES % 1024 == 0, "alignment");
};

struct Bf16Params {
    int mode, swap;
    int M, N, K;                 // GroupK: K = rows of both operands
    int p_mn, q_mn;              // the operand's rows (not K) are contiguous
    int groups;
    const int32_t *offsets;
    int tm, tn;                  // rows and columns of C per tile
    int row_tiles, col_tiles;    // (grouped rows: row tiles by group)
    FastDiv by_cols;             // col_tiles
    int split;
    int even;                    // GroupK: extra tiles go to the CTAs with the least work so far
    const float *bias;
    int64_t stride_bias;
    int act, join;
    void *pre;
    int64_t ld_pre;
    const void *D;
    int64_t ldd;
    void *C;
    int64_t ldc, stride_c;
    int c_bf16;
    int vec;                     // C, pre and D in whole 16-byte pieces
    unsigned int *status;
};

// The same value in all lanes, known to the compiler as such (what an MMA or a
// copy takes lies in registers that the warp shares: 75 cycles per MMA to
// bring it there where the compiler cannot tell).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kAll, x, 0); }

// One tile: its group, rows [m, m_end) and first column of C, its range of K,
// and the accumulator's columns that it needs (0: no tile, all are done).
struct Item {
    int group, m, m_end, n, k0, k1, cols;
};

__device__ __forceinline__ void store_item(uint32_t at, const Item &w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w.group), "r"(w.m), "r"(w.m_end), "r"(w.n)
                 : "memory");
    asm volatile("st.shared.v4.u32 [%0+16], {%1,%2,%3,%3};" ::"r"(at), "r"(w.k0), "r"(w.k1), "r"(w.cols) : "memory");
}

__device__ __forceinline__ Item load_item(uint32_t at)
{
    Item w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.group), "=r"(w.m), "=r"(w.m_end), "=r"(w.n)
                 : "r"(at)
                 : "memory");
    asm volatile("{\n\t.reg .u32 x;\n\tld.shared.v4.u32 {%0,%1,%2,x}, [%3+16];\n\t}"
                 : "=r"(w.k0), "=r"(w.k1), "=r"(w.cols)
                 : "r"(at)
                 : "memory");
    w.group = uniform(w.group), w.m = uniform(w.m), w.m_end = uniform(w.m_end), w.n = uniform(w.n);
    w.k0 = uniform(w.k0), w.k1 = uniform(w.k1), w.cols = uniform(w.cols);
    return w;
}

__device__ __forceinline__ int slabs(int k0, int k1) { return (int)(((uint32_t)(k1 - k0) + kSlab - 1) / kSlab); }

// An MMA's columns come in 16s, in 32s by a pair.
template <class Cfg>
__device__ __forceinline__ int whole_columns(int n)
{
    constexpr int unit = Cfg::PAIR ? 32 : 16;
    const int up = (n + unit - 1) / unit * unit;
    return up < unit ? unit : up < Cfg::BN ? up : Cfg::BN;
}

// How a grid of `units` pairs walks `tiles`: where the last wave would leave
// half of them (or three quarters) idle, its tiles are cut into two (four)
// pieces along the accumulator's columns (80 tiles for 76 pairs, 2560 x 2048 x
// 2048: 23.3 us for 29.6; 8191 x 2048 x 4096 87.0 for 89.9; 16384 x 4096 x 4096
// 327 for 331, in turn).
struct Walk {
    uint32_t whole, pieces, steps;   // tiles that are not cut, pieces of the others, all in all
    __device__ __forceinline__ Walk(uint32_t tiles, uint32_t units, bool cut)
    {
        const uint32_t last = tiles % units;
        pieces = !cut || last == 0 || 2 * last > units ? 1 : 4 * last > units ? 2 : 4;
        whole = tiles - last;
        steps = whole + last * pieces;
    }
};

// Row tile and column tile t of `rows` by col_tiles: bands of kRaster row
// tiles, the row tile fastest.
__device__ __forceinline__ int2 raster(const Bf16Params &p, int rows, uint32_t t)
{
    const uint32_t band = div(t / kRaster, p.by_cols), first = band * kRaster;
    const uint32_t r = t - first * p.col_tiles;
    const uint32_t high = rows - first < (uint32_t)kRaster ? rows - first : kRaster;
    const uint32_t ct = high == kRaster ? r / kRaster : r / high;
    return make_int2((int)(first + r - ct * high), (int)ct);
}

// The CTA's part of K, where a cluster shares a tile.
__device__ __forceinline__ void split_range(const Bf16Params &p, int rank, Item &it)
{
    if (p.split == 1) return;
    const int n = slabs(0, p.K);
    const int64_t k1 = (int64_t)((int64_t)n * (rank + 1) / p.split) * kSlab;
    it.k0 = (int)((int64_t)n * rank / p.split) * kSlab;
    it.k1 = k1 < p.K ? (int)k1 : p.K;
}

template <class Cfg>
__device__ __forceinline__ Item dense_item(const Bf16Params &p, const Walk &walk, uint32_t t, int rank)
{
    int piece = 0;
    const bool cut = Cfg::PAIR && t >= walk.whole && walk.pieces > 1;
    if (cut) {
        const uint32_t over = t - walk.whole, shift = walk.pieces >> 1;   // of 2 or 4
        piece = (int)(over & (walk.pieces - 1));
        t = walk.whole + (over >> shift);
    }
    const int2 at = raster(p, p.row_tiles, t);
    Item it;
    it.group = 0;
    it.m = at.x * p.tm;
    it.m_end = p.M - it.m < p.tm ? p.M : it.m + p.tm;
    it.n = at.y * p.tn;
    it.k0 = 0;
    it.k1 = p.K;
    it.cols = whole_columns<Cfg>(p.swap ? it.m_end - it.m : p.N - it.n);
    if (cut) {
        const int wide = whole_columns<Cfg>((it.cols + (int)walk.pieces - 1) / (int)walk.pieces);
        it.cols = wide;
        it.n += piece * wide;      // past C's columns: this piece has none
    }
    split_range(p, rank, it);
    return it;
}

// A group's rows of C, and how many of them a tile takes.
struct Group {
    int lo, hi, tiles, tall;
};

template <class Cfg>
__device__ __forceinline__ Group group_of(const Bf16Params &p, int g)
{
    Group o;
    group_range(p.offsets, g, p.M, o.lo, o.hi);
    o.tiles = (int)(((uint32_t)(o.hi - o.lo) + (uint32_t)p.tm - 1) / (uint32_t)p.tm);
    // Evenly over the tiles, whose columns they are: of 273, 160 and 113 take
    // less than 256 and 17.
    const int each = o.tiles > 1 ? (o.hi - o.lo + o.tiles - 1) / o.tiles : o.hi - o.lo;
    o.tall = whole_columns<Cfg>(each);
    return o;
}

// Tile t of the groups' rows, which lie on the columns (swap): table[g] row
// tiles are in the groups before g.
template <class Cfg>
__device__ __forceinline__ Item rows_item(const Bf16Params &p, const int *table, uint32_t t, int rank)
{
    const int2 at = raster(p, table[p.groups], t);
    Item it;
    it.group = find_group(table, p.groups, at.x);
    const Group o = group_of<Cfg>(p, it.group);
    it.m = o.lo + (at.x - table[it.group]) * o.tall;
    it.m = it.m < o.hi ? it.m : o.hi;
    it.m_end = o.hi - it.m < o.tall ? o.hi : it.m + o.tall;
    it.n = at.y * p.tn;
    it.k0 = 0;
    it.k1 = p.K;
    it.cols = whole_columns<Cfg>(it.m_end - it.m);
    split_range(p, rank, it);
    return it;
}

// Tile t of group g's product over its rows.
template <class Cfg>
__device__ __forceinline__ Item k_item(const Bf16Params &p, int g, uint32_t t)
{
    const int2 at = raster(p, p.row_tiles, t);
    Item it;
    it.group = g;
    it.m = at.x * p.tm;
    it.m_end = p.M - it.m < p.tm ? p.M : it.m + p.tm;
    it.n = at.y * p.tn;
    group_range(p.offsets, g, p.K, it.k0, it.k1);
    it.cols = whole_columns<Cfg>(p.swap ? it.m_end - it.m : p.N - it.n);
    // Nothing is added: C stays as it is.
    if (it.k0 >= it.k1 && p.join == kJoinAdd) it.m_end = it.m;
    return it;
}

// What the CTAs (pairs) have been given, for groups of uneven length: the
// tiles of a group that are left over after each has had the same number go to
// those that have the least so far. (Every units-th tile instead leaves 16
// groups' weight gradients of 2048 x 2048 from 16383 rows at 119 us for 111,
// with even groups 95; shares of neighbouring tiles, even in their work, at 158:
// CTAs that are at different groups share no operands in L2.) A warp's lanes
// hold the work of walkers lane, lane + 32, ..; all warps find the same.
constexpr int kWalkers = 5;    // per lane: up to 160

struct Shares {
    uint32_t work[kWalkers] = {};

    // Gives a group's tiles, `cost` each: `rounds` to all of the `units`
    // walkers and `extra` (below units) to those with the least work, by their
    // numbers where that is equal. Which of the extra ones walker `unit` gets
    // (`extra`: none).
    __device__ __forceinline__ uint32_t give(uint32_t units, uint32_t unit, uint32_t rounds, uint32_t extra, uint32_t cost, int lane)
    {
        // The least limit that `extra` walkers are within, by bisection.
        uint32_t low = ~0u, high = 0;
#pragma unroll
        for (int i = 0; i < kWalkers; ++i) {
            if ((uint32_t)(lane + 32 * i) >= units) continue;
            low = work[i] < low ? work[i] : low;
            high = work[i] > high ? work[i] : high;
        }
        low = __reduce_min_sync(kAll, low);
        high = __reduce_max_sync(kAll, high);
        while (low < high) {
            const uint32_t mid = low + (high - low) / 2;
            uint32_t within = 0;
#pragma unroll
            for (int i = 0; i < kWalkers; ++i)
                within += __popc(__ballot_sync(kAll, (uint32_t)(lane + 32 * i) < units && work[i] <= mid));
            if (within >= extra) high = mid;
            else low = mid + 1;
        }
        uint32_t left = extra;          // for those at the limit
#pragma unroll
        for (int i = 0; i < kWalkers; ++i)
            left -= __popc(__ballot_sync(kAll, (uint32_t)(lane + 32 * i) < units && work[i] < low));
        const uint32_t below = (1u << lane) - 1;
        uint32_t mine = extra, given = 0, at_limit = 0;
#pragma unroll
        for (int i = 0; i < kWalkers; ++i) {
            const bool there = (uint32_t)(lane + 32 * i) < units, equal = there && work[i] == low;
            const uint32_t equals = __ballot_sync(kAll, equal);
            const bool gets = there && (work[i] < low || (equal && at_limit + __popc(equals & below) < left));
            at_limit += __popc(equals);
            const uint32_t all = __ballot_sync(kAll, gets);
            if (unit / 32 == (uint32_t)i && ((all >> (unit % 32)) & 1)) mine = given + __popc(all & ((1u << (unit % 32)) - 1));
            given += __popc(all);
            work[i] += (rounds + (gets ? 1u : 0u)) * cost;
        }
        return mine;
    }
};

// The address of `addr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// As tma_load_if() and mbar_expect_if(), for a pair: the barrier may be the
// other CTA's (an address of shared::cluster).
__device__ __forceinline__ void tma_load_pair_if(uint32_t on, uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %7, 0;\n\t"
                 "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                 ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy), "r"(on)
                 : "memory");
}

__device__ __forceinline__ void mbar_expect_cluster_if(uint32_t on, uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
                 "@q mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes), "r"(on)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster_if(uint32_t on, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(on)
                 : "memory");
}

// Takes over what came before the arrivals, from the pair's other CTA too, at
// a phase that is known to be complete. (A fence instead costs 1000 cycles.)
__device__ __forceinline__ void mbar_seen_cluster(uint32_t bar, uint32_t parity)
{
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(parity)
                 : "memory");
}

// The commit's arrival at the barrier of both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair_if(uint32_t on, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::
                     "r"(bar),
                 "r"(on)
                 : "memory");
}

// Waits for phase `parity` of the barrier, unless it was `early` seen to be
// complete; false after about ptx::kWaitLimitNs. The clock is read after 64
// probes only: reading it costs more than the usual wait.
__device__ __forceinline__ bool wait_bar(uint32_t early, uint32_t bar, uint32_t parity)
{
    if (__builtin_expect(__all_sync(kAll, early) != 0, 1)) return true;
    bool ok = false;
    uint64_t t0 = 0;
    for (uint32_t n = 0; !ok && n < kSpinLimit; ++n) {
#pragma unroll 1
        for (int r = 0; !ok && r < 64; ++r) ok = ptx::mbar_try_wait(bar, parity);
        if (ok) break;
        const uint64_t t = ptx::global_timer_ns();
        if (n == 0) t0 = t;
        else if (t - t0 > ptx::kWaitLimitNs) break;
    }
    return __all_sync(kAll, ok) != 0;
}

// A wait for what may take as long as a tile of nk slabs.
__device__ __forceinline__ bool wait_tile(uint32_t bar, uint32_t parity, int nk)
{
    if (wait_bar(mbar_test(bar, parity), bar, parity)) return true;
    for (int k = nk >> 16; k > 0; --k)
        if (wait_bar(0, bar, parity)) return true;
    return false;
}

// D (+)= P . Q^T on bfloat16 operands, given the descriptors' lower words (the
// upper ones are the same for both).
template <bool PAIR>
__device__ __forceinline__ void mma_bf16_if(uint32_t on, uint32_t d_tmem, uint32_t p_desc, uint32_t q_desc, uint32_t upper,
                                            uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
            "r"(p_desc), "r"(q_desc), "r"(upper), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
            "r"(p_desc), "r"(q_desc), "r"(upper), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
}

// Instruction descriptor of .kind::f16: FP32 accumulation (bits 4-5 = 1), both
// operands bfloat16 (bits 7-9 and 10-12 = 1), K or the rows contiguous (bits
// 15 and 16), N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_bf16(int m, int n, int p_mn, int q_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)p_mn << 15) | ((uint32_t)q_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory descriptor of an operand in boxes of 64 (contiguous rows) by
// 64 (along K), 128-byte swizzle: 8192 bytes from one 64 rows to the next
// (leading offset), 1024 from 8 values of K to the next (stride).
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        ptx::tmem_alloc(slot, cols);
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
    else
        ptx::tmem_dealloc(taddr, cols);
}

// ------------------------------------------------------------------- epilogue

// Where the rows of a tile lie in C, pre and D, and its group's bias.
template <class T>
struct Place {
    T *C, *pre;
    const T *D;
    const float *bias;
};

template <class T>
__device__ __forceinline__ Place<T> place_of(const Bf16Params &p, int group)
{
    const int64_t base = p.mode == kBf16GroupK ? group * p.stride_c : 0;
    Place<T> q;
    q.C = static_cast<T *>(p.C) + base;
    q.pre = p.pre ? static_cast<T *>(p.pre) : nullptr;
    q.D = p.join != kJoinNone ? static_cast<const T *>(p.D) + base : nullptr;
    q.bias = p.bias ? p.bias + (p.mode == kBf16GroupRows ? group * p.stride_bias : 0) : nullptr;
    return q;
}

__device__ __forceinline__ float joined(float y, float d, int join)
{
    return join == kJoinAdd ? y + d : join == kJoinMul ? y * d : y;
}

// One element (m, n) of C from its sum.
template <class T>
__device__ __forceinline__ void store_one(const Bf16Params &p, const Place<T> &q, int64_t m, int n, float z)
{
    if (q.bias) z += __ldg(q.bias + n);
    if (q.pre) store_from_float(q.pre + m * p.ld_pre + n, z);
    float y = z;
    with_activation(p.act, [&](auto a) { y = activate<decltype(a)::value>(z); });
    if (q.D) y = joined(y, load_as_float(q.D + m * p.ldd + n), p.join);
    store_from_float(q.C + m * p.ldc + n, y);
}

// Staging of a chunk of C's sums: rows of 32 floats, their 16-byte pieces
// exchanged by row: element (r, c).
__device__ __forceinline__ uint32_t staged(uint32_t st, int r, int c)
{
    return st + 128 * r + 16 * ((c >> 2) ^ (r & 7)) + 4 * (c & 3);
}

// A chunk of the warp's accumulators, v[j] column j of this lane, to staging:
// the lane is a row of C, or (swap) the column is.
template <int CHUNK>
__device__ __forceinline__ void stage(uint32_t st, int lane, bool swap, const float *v)
{
    if (swap) {
#pragma unroll
        for (int j = 0; j < CHUNK; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(staged(st, j, lane)), "f"(v[j]) : "memory");
    } else {
#pragma unroll
        for (int j = 0; j < CHUNK; j += 4)
            st_shared_u32x4(staged(st, lane, j), make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]),
                                                            __float_as_uint(v[j + 2]), __float_as_uint(v[j + 3])));
    }
}

// Staged sums to R rows of C from m on, 32 columns from n on (`rows` and
// `cols` of them exist), V values of a row per access; put() stages them.
// What of D a lane needs is requested before that, unless it comes by TMA:
// then `dbuf` is where, in rows of 32 values, once there() returns.
// HELD: the warp's sums are in registers meanwhile.
template <class T, int R, int V, bool TMA_D, bool HELD, class Put, class There>
__device__ __forceinline__ void store_chunk(const Bf16Params &p, const Place<T> &q, uint32_t st, int lane, Put put, int64_t m,
                                            int rows, int n, int cols, uint32_t dbuf, There there)
{
    constexpr int PER_ROW = 32 / V, PER_PASS = 32 / PER_ROW, PASSES = R / PER_PASS;
    // Rows whose sums are in registers together: of one, each activation would
    // wait for the one before (600 cycles a row where C goes by single values).
    constexpr int MOST = V == 1 ? 8 : V == 4 ? 2 : HELD ? 1 : 4, AHEAD = PASSES < MOST ? PASSES : MOST;
    const int r0 = lane / PER_ROW, c0 = (lane % PER_ROW) * V;
    const bool whole = V == 1 ? c0 < cols : c0 + V <= cols;
    Values<T, V> d[AHEAD];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = r0 + (i0 + i) * PER_PASS;
            if (whole && r < rows) d[i] = *reinterpret_cast<const Values<T, V> *>(q.D + (m + r) * p.ldd + n + c0);
        }
    };
    if (!TMA_D && q.D) fetch(0);
    float b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = 0.0f;
    if (q.bias) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c0 + e < cols) b[e] = __ldg(q.bias + n + c0 + e);
    }
    put();
    if constexpr (TMA_D) there();
    __syncwarp();
    if (!whole) {
        // The columns where C ends inside an access.
#pragma unroll 1
        for (int i = 0; i < PASSES * (V > 1 ? cols - c0 : 0); ++i) {
            const int r = r0 + i % PASSES * PER_PASS, c = c0 + i / PASSES;
            if (r < rows) store_one(p, q, m + r, n + c, ld_shared_f32(staged(st, r, c)));
        }
    } else {
        with_activation(p.act, [&](auto a) {
#pragma unroll 1
            for (int i0 = 0; i0 < PASSES; i0 += AHEAD) {
                if (!TMA_D && i0 > 0 && q.D) fetch(i0);
                float z[AHEAD][V];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int r = r0 + (i0 + i) * PER_PASS;
                    if constexpr (V == 1) {
                        z[i][0] = ld_shared_f32(staged(st, r, c0));
                    } else {
#pragma unroll
                        for (int e = 0; e < V; e += 4) {
                            const uint4 u = ld_shared_u32x4(staged(st, r, c0 + e));
                            z[i][e] = __uint_as_float(u.x), z[i][e + 1] = __uint_as_float(u.y);
                            z[i][e + 2] = __uint_as_float(u.z), z[i][e + 3] = __uint_as_float(u.w);
                        }
                    }
                }
                auto store = [&](T *to, int64_t ld) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        const int r = r0 + (i0 + i) * PER_PASS;
                        Values<T, V> o;
#pragma unroll
                        for (int e = 0; e < V; ++e) store_from_float(&o.v[e], z[i][e]);
                        if (r < rows) *reinterpret_cast<Values<T, V> *>(to + (m + r) * ld + n + c0) = o;
                    }
                };
                if (q.bias) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                        for (int e = 0; e < V; ++e) z[i][e] += b[e];
                }
                if (q.pre) store(q.pre, p.ld_pre);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) z[i][e] = activate<decltype(a)::value>(z[i][e]);
                if constexpr (TMA_D) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        const int r = r0 + (i0 + i) * PER_PASS;
                        if constexpr (V == 1) {
                            // Rows of pieces, each from its 16-byte boundary on.
                            const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(q.D + (m + r) * p.ldd + n) & 15u;
                            const uint32_t from = dbuf + r * (sizeof(T) == 4 ? 144 : 80) + shift + (uint32_t)sizeof(T) * c0;
                            if constexpr (sizeof(T) == 4) {
                                d[i].v[0] = ld_shared_f32(from);
                            } else {
                                uint16_t u;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(from) : "memory");
                                d[i].v[0] = *reinterpret_cast<const T *>(&u);
                            }
                        } else {
                            const uint4 u = ld_shared_u32x4(dbuf + (uint32_t)sizeof(T) * (32 * r + c0));
                            d[i] = *reinterpret_cast<const Values<T, V> *>(&u);
                        }
                    }
                }
                if (q.D) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                        for (int e = 0; e < V; ++e) z[i][e] = joined(z[i][e], load_as_float(&d[i].v[e]), p.join);
                }
                store(q.C, p.ldc);
            }
        });
    }
    __syncwarp();
}

// Where chunk c of a warp's part of a tile lies in C, and how much of it exists.
struct Chunk {
    int m, n, rows, cols;
    __device__ __forceinline__ Chunk(const Bf16Params &p, const Item &w, int lane0, int col)
        : m(w.m + (p.swap ? col : lane0)), n(w.n + (p.swap ? lane0 : col)), rows(w.m_end - m), cols(p.N - n)
    {
        if (!p.swap && cols > w.cols - col) cols = w.cols - col;
    }
    __device__ __forceinline__ bool some() const { return rows > 0 && cols > 0; }
};

// A warp's chunks of D on their way to shared memory: those of one tile, in
// order, as many as its buffers hold. By TMA; where TMA cannot address D, in
// the 16-byte pieces that a row's 32 values lie in, wherever they begin.
template <class Cfg>
struct Arrivals {
    uint32_t buffers, bars;
    int next;                      // column of the tile to ask for next
    uint32_t asked = 0, taken = 0;
    bool ok = true;

    static __device__ __forceinline__ int pieces(const Bf16Params &p) { return p.c_bf16 ? 5 : 9; }
    static __device__ __forceinline__ uint32_t log_depth(const Bf16Params &p) { return (p.c_bf16 ? 2 : 1) - (p.vec ? 0 : 1); }
    static __device__ __forceinline__ uint32_t bytes(const Bf16Params &p)
    {
        return Cfg::CHUNK * (p.vec ? 32 * (p.c_bf16 ? 2 : 4) : 16 * pieces(p));
    }
    __device__ __forceinline__ uint32_t slot(const Bf16Params &p, uint32_t i) const { return i & ((1u << log_depth(p)) - 1); }
    __device__ __forceinline__ uint32_t buffer(const Bf16Params &p, uint32_t i) const { return buffers + bytes(p) * slot(p, i); }

    // Copies of a chunk's pieces. What lies between D's rows is not read: it may
    // be anyone's. Only chunks at the ends of rows (of D, where nothing lies
    // between its rows) look at what each piece may hold; done for all, 4097 x
    // 3001 x 2049 with everything took 103 us for 88.
    template <class T, int PIECES>
    static __device__ __forceinline__ void copy(const Bf16Params &p, const Item &w, const Chunk &c, uint32_t to, int lane)
    {
        constexpr int PER16 = 16 / (int)sizeof(T);
        const T *const all = static_cast<const T *>(p.D) + (p.mode == kBf16GroupK ? w.group * p.stride_c : 0);
        const T *const first = all + c.m * p.ldd + c.n;
        const int bytes = (int)sizeof(T) * (c.cols < 32 ? c.cols : 32);
        const bool close = p.ldd == p.N && p.N >= PER16;
        const bool inside = (c.n > 0 || (close && c.m > 0)) && (p.N - c.n >= 32 + PER16 || (close && p.M - c.m > Cfg::CHUNK));
        if (inside) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int at = 32 * i + lane, r = at / PIECES, q = at % PIECES;
                const uintptr_t row = reinterpret_cast<uintptr_t>(first + r * p.ldd), from = (row & ~uintptr_t(15)) + 16 * q;
                if (r < c.rows && from < row + bytes)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * (r * PIECES + q)), "l"(from) : "memory");
            }
        } else {
#pragma unroll 1
            for (int at = lane; at < 32 * PIECES; at += 32) {
                const int r = at / PIECES, q = at % PIECES;
                if (r >= c.rows) continue;
                const T *const row = first + r * p.ldd - c.n, *const begin = close ? all : row;
                const T *const end = close ? all + p.M * p.ldd : row + p.N;
                const RowPiece piece = row_piece(reinterpret_cast<uintptr_t>(begin), reinterpret_cast<uintptr_t>(end),
                                                 reinterpret_cast<uintptr_t>(row + c.n), bytes, q);
                const uint32_t dst = to + 16 * (r * PIECES + q);
                if (piece.some() && piece.whole()) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(piece.from) : "memory");
                    continue;
                }
                for (int e = piece.lo; e < piece.hi; e += (int)sizeof(T)) {
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + e), "f"(*reinterpret_cast<const float *>(piece.from + e)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + e), "h"(*reinterpret_cast<const uint16_t *>(piece.from + e)) : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    __device__ __forceinline__ void ask(const Bf16Params &p, const CUtensorMap *map, const Item &w, int lane, int lane0, int col0)
    {
        while (next < Cfg::CW && asked - taken < (1u << log_depth(p))) {
            const Chunk c(p, w, lane0, col0 + next);
            next += Cfg::CHUNK;
            if (!c.some()) continue;
            if (p.vec) {
                const uint32_t on = lane == 0, bar = bars + 8 * slot(p, asked);
                mbar_expect_if(on, bar, bytes(p));
                tma_load_if(on, buffer(p, asked), map, bar, c.n, c.m, p.mode == kBf16GroupK ? w.group : 0,
                            ptx::policy_evict_last());
            } else if (p.c_bf16) {
                copy<__nv_bfloat16, 5>(p, w, c, buffer(p, asked), lane);
            } else {
                copy<float, 9>(p, w, c, buffer(p, asked), lane);
            }
            ++asked;
        }
    }
    // Waits for the oldest chunk (copies: this lane's; a __syncwarp() makes it all).
    __device__ __forceinline__ void wait(const Bf16Params &p)
    {
        if (!p.vec) {
            if (asked - taken > 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            return;
        }
        const uint32_t b = bars + 8 * slot(p, taken), phase = (taken >> log_depth(p)) & 1;
        ok = wait_bar(mbar_test(b, phase), b, phase) && ok;
    }
};

// A warp's part of a tile: CW columns from the tile's column col0 on; put(c)
// stages the chunk from its column c on.
template <class T, class Cfg, bool HELD, class Put>
__device__ __forceinline__ void store_part(const Bf16Params &p, const Item &w, uint32_t st, int lane, int lane0, int col0,
                                           Put put, const CUtensorMap *map, Arrivals<Cfg> &d)
{
    constexpr int CHUNK = Cfg::CHUNK, V = 16 / (int)sizeof(T);
    Place<T> q = place_of<T>(p, w.group);
    if constexpr (Cfg::PAIR && !Cfg::JOINS) q.D = nullptr;     // as the host chose this kernel
#pragma unroll 1
    for (int c = 0; c < Cfg::CW; c += CHUNK) {
        const Chunk at(p, w, lane0, col0 + c);
        if (!at.some()) continue;
        auto chunk = [&]() { put(c); };
        if constexpr (Cfg::JOINS) {
            const uint32_t from = d.buffer(p, d.taken);
            auto there = [&]() { d.wait(p); };
            if (p.vec)
                store_chunk<T, CHUNK, V, true, HELD>(p, q, st, lane, chunk, at.m, at.rows, at.n, at.cols, from, there);
            else
                store_chunk<T, CHUNK, 1, true, HELD>(p, q, st, lane, chunk, at.m, at.rows, at.n, at.cols, from, there);
            ++d.taken;
            d.ask(p, map, w, lane, lane0, col0);
        } else if (p.vec) {
            store_chunk<T, CHUNK, V, false, HELD>(p, q, st, lane, chunk, at.m, at.rows, at.n, at.cols, 0, [] {});
        } else {
            store_chunk<T, CHUNK, 1, false, HELD>(p, q, st, lane, chunk, at.m, at.rows, at.n, at.cols, 0, [] {});
        }
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
bf16_product_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                    const __grid_constant__ CUtensorMap mapD, const __grid_constant__ Bf16Params p)
{
    constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES, NBUF = Cfg::NBUF, CW = Cfg::CW, QR = Cfg::QR;
    constexpr bool PAIR = Cfg::PAIR;
    // The swizzle goes by the address: stages begin on 1024 bytes.
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = ptx::smem_addr(smem);
    int *const table = reinterpret_cast<int *>(smem + Cfg::OFF_TABLE);
    const uint32_t bars = base + Cfg::OFF_BARS;
    auto stage_p = [&](int s) { return base + s * Cfg::STAGE_BYTES; };
    auto stage_q = [&](int s) { return base + s * Cfg::STAGE_BYTES + Cfg::P_TILE; };
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto done_bar = [&](int s) { return bars + 8u * (STAGES + s); };
    auto accf_bar = [&](int b) { return bars + 8u * (2 * STAGES + b); };
    auto acce_bar = [&](int b) { return bars + 8u * (2 * STAGES + NBUF + b); };
    auto ifull_bar = [&](uint32_t i) { return bars + 8u * (2 * STAGES + 2 * NBUF + i); };
    auto iempty_bar = [&](uint32_t i) { return bars + 8u * (2 * STAGES + 2 * NBUF + kItems + i); };
    auto tail_bar = [&](int s) { return bars + 8u * (2 * STAGES + 2 * NBUF + 2 * kItems + s); };
    const uint32_t drain_bar = bars + 8u * (3 * STAGES + 2 * NBUF + 2 * kItems);
    const uint32_t d_bars = drain_bar + 8;
    const uint32_t tmem_slot = bars + 8u * Cfg::NUM_BARS;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int split = Cfg::CAN_SPLIT ? p.split : 1;
    const int cluster = PAIR ? 2 : split;
    const int rank = cluster > 1 ? (int)ptx::cluster_ctarank() : 0;
    if ((base & 1023u) != 0 || (cluster > 1 && ptx::cluster_nctarank() != (uint32_t)cluster)) {
        // Launched without its cluster, it would reach for peers that do not exist.
        if (threadIdx.x == 0) atomicOr(p.status, kStatusLaunchConfig);
        return;
    }
    const bool group_k = p.mode == kBf16GroupK;

    if (warp == 2 && lane == 0) {
        ptx::prefetch_tensormap(&mapP);
        ptx::prefetch_tensormap(&mapQ);
        if (Cfg::JOINS) ptx::prefetch_tensormap(&mapD);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), Cfg::CTAS);   // the producer (or the last slab's warp 3) of each CTA
            ptx::mbar_init(done_bar(s), 1);
            ptx::mbar_init(tail_bar(s), 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            ptx::mbar_init(accf_bar(b), 1);
            ptx::mbar_init(acce_bar(b), Cfg::CTAS * Cfg::EPI_WARPS);
        }
        for (int i = 0; i < kItems; ++i) {
            // Read by the producer, the MMA issuer, the epilogue and, over groups' K, warp 3.
            ptx::mbar_init(ifull_bar(i), 1);
            ptx::mbar_init(iempty_bar(i), Cfg::EPI_WARPS + (group_k ? 3 : 2));
        }
        ptx::mbar_init(drain_bar, 1);
        for (int i = 0; i < Cfg::D_BARS; ++i) ptx::mbar_init(d_bars + 8 * i, 1);
        ptx::mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<PAIR>(tmem_slot, Cfg::TMEM_COLS);
    if (p.mode == kBf16GroupRows) {
        // table[g] = row tiles of the groups before g.
        for (int g = threadIdx.x; g < p.groups; g += Cfg::THREADS) table[g] = group_of<Cfg>(p, g).tiles;
        __syncthreads();
        if (warp == 0) {
            // Offsets that are not a partition may sum to anything: no entry
            // passes what the kernel can walk.
            const uint32_t most = (uint32_t)(INT32_MAX / p.col_tiles - 2 * kRaster);
            const uint32_t held = most < (1u << 26) ? most : 1u << 26;
            uint32_t carry = 0;
            for (int g0 = 0; g0 < p.groups; g0 += 32) {
                const int g = g0 + lane;
                const uint32_t mine = g < p.groups ? table[g] : 0;
                uint32_t sum = mine < held ? mine : held;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const uint32_t up = __shfl_up_sync(kAll, sum, d);
                    if (lane >= d) sum = sum + up < held ? sum + up : held;
                }
                const uint32_t end = carry + sum < held ? carry + sum : held;
                const uint32_t before = __shfl_up_sync(kAll, end, 1);
                if (g < p.groups) table[g] = (int)(lane == 0 ? carry : before);
                carry = __shfl_sync(kAll, end, 31);
                if (g0 + 32 >= p.groups && lane == 0) table[p.groups] = (int)carry;
            }
        }
    }
    ptx::tc_fence_before();
    // A pair's barriers and tensor memory are there in both CTAs before either goes on.
    if constexpr (PAIR) ptx::cluster_sync_all();
    else __syncthreads();
    ptx::tc_fence_after();
    // The CTAs of a split tile write into each other's shared memory in the
    // end: each says that it has begun, and waits for the others before that.
    if (Cfg::CAN_SPLIT && split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const uint32_t taddr = *reinterpret_cast<uint32_t *>(smem + (tmem_slot - base));

    const uint32_t unit = blockIdx.x / cluster, units = gridDim.x / cluster;

    // The CTA's nth tile, once warp 2 has found it; not to be read after done_with().
    const int longest = slabs(0, p.K);
    auto item_at = [&](uint32_t n) { return base + Cfg::OFF_ITEMS + (n % kItems) * kItemBytes; };
    auto item_there = [&](uint32_t n) {
        const uint32_t bar = ifull_bar(n % kItems), phase = (n / kItems) & 1;
        return wait_tile(bar, phase, longest);
    };
    auto done_with = [&](uint32_t n) {
        __syncwarp();
        mbar_arrive_if(lane == 0, iempty_bar(n % kItems));
    };
    auto gave_up = [&]() {
        if (lane == 0) atomicOr(p.status, kStatusTimeout);
    };
    // K that an accumulator takes before it is handed on.
    const int part = p.c_bf16 && split == 1 ? kPartBf16 : kPart;
    // Where this CTA's lanes and its rows of the columns' operand begin.
    const int pair_rank = PAIR ? rank : 0;

    if constexpr (Cfg::MOVE_REGS) {
        if (warp < 4) ptx::setmaxnreg_dec<72>();
    }
    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        const uint32_t on = elect_one();
        const uint64_t policy = ptx::policy_evict_last();
        // Boxes of 64 along K by 64 rows (or columns of C), of the columns'
        // operand, where its K is contiguous, 32 rows: as many as the tile
        // needs, without branches.
        constexpr int Q_BOXES = QR > 32 ? QR / 32 : 1;
        const int q_rows = p.q_mn ? 64 : QR < 32 ? QR : 32, q_bytes = 128 * q_rows;
        const bool p_mn = p.p_mn, q_mn = p.q_mn;
        auto load = [&](uint32_t yes, uint32_t dst, const CUtensorMap *map, uint32_t bar, bool mn, int row, int k, int z) {
            const int x = mn ? row : k, y = mn ? k : row;
            if constexpr (PAIR) tma_load_pair_if(on & yes, dst, map, bar, x, y, z, policy);
            else tma_load_if(on & yes, dst, map, bar, x, y, z, policy);
        };
        uint32_t it = 0, n = 0, early = 1;
        bool ok = true;
        for (; ok; ++n) {
            if (!item_there(n)) {
                gave_up();
                break;
            }
            const Item w = load_item(item_at(n));
            done_with(n);
            if (w.cols == 0) break;
            const int z = p.mode == kBf16GroupRows ? w.group : 0;
            const int pz = p.swap ? z : 0, qz = p.swap ? 0 : z;
            const int need = PAIR ? w.cols / 2 : w.cols;     // rows of the columns' operand here
            const int p_row = (p.swap ? w.n : w.m) + 128 * pair_rank, q_row = (p.swap ? w.m : w.n) + need * pair_rank;
            const uint32_t bytes = Cfg::P_TILE + (need + q_rows - 1) / q_rows * q_bytes;
            for (int k = w.k0; k < w.k1; k += kSlab, ++it) {
                const int s = (int)(it % STAGES);
                if (!wait_bar(early, done_bar(s), ((it / STAGES) & 1) ^ 1)) {
                    gave_up();
                    ok = false;
                    break;
                }
                // A group's last rows go to warp 3 first, unless they are whole 16s.
                const bool tail = group_k && w.k1 - k < kSlab && (w.k1 - k) % 16 != 0;
                uint32_t bar = tail ? tail_bar(s) : full_bar(s);
                if constexpr (PAIR) {
                    bar = map_shared(bar, tail ? rank : 0);
                    mbar_expect_cluster_if(on, bar, bytes);
                } else {
                    mbar_expect_if(on, bar, bytes);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) load(1, stage_p(s) + 8192 * c, &mapP, bar, p_mn, p_row + 64 * c, k, pz);
#pragma unroll
                for (int c = 0; c < Q_BOXES; ++c)
                    load(c * q_rows < need, stage_q(s) + q_bytes * c, &mapQ, bar, q_mn, q_row + q_rows * c, k, qz);
                const uint32_t next = it + 1;
                early = mbar_test(done_bar((int)(next % STAGES)), ((next / STAGES) & 1) ^ 1);
            }
        }
        // Every byte bound for this CTA lands before it leaves: its MMAs wait
        // for all of them, and the last of each stage are done with.
        for (uint32_t back = 0; back < STAGES && back < it; ++back) {
            const uint32_t i = it - 1 - back;
            if (!wait_bar(0, done_bar((int)(i % STAGES)), (i / STAGES) & 1)) gave_up();
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        const uint64_t desc_p = p.p_mn ? sdesc_rows(stage_p(0)) : ptx::sdesc_kmajor(stage_p(0), 128);
        const uint64_t desc_q = p.q_mn ? sdesc_rows(stage_q(0)) : ptx::sdesc_kmajor(stage_q(0), 128);
        const uint32_t upper = (uint32_t)(desc_p >> 32);   // stride, version, swizzle: 1024 bytes either way
        const uint32_t first_p = (uint32_t)desc_p, first_q = (uint32_t)desc_q;
        // 16 values of K further, in 16 bytes: along a row, or 16 rows down.
        const uint32_t step_p = p.p_mn ? 128 : 2, step_q = p.q_mn ? 128 : 2;
        const bool leader = rank == 0 || !PAIR;
        const uint32_t on = elect_one();
        uint32_t it = 0, n = 0, acc = 0, early = 0;
        bool ok = true;
        for (; ok; ++n) {
            if (!item_there(n)) {
                gave_up();
                break;
            }
            const Item w = load_item(item_at(n));
            done_with(n);
            if (w.cols == 0) break;
            if (!leader) continue;
            const uint32_t idesc = idesc_bf16(Cfg::LANES, w.cols, p.p_mn, p.q_mn);
            int k = w.k0;
            do {
                const int b = (int)(acc % NBUF), first = k, end = w.k1 - k > part ? k + part : w.k1;
                if (!wait_tile(acce_bar(b), ((acc / NBUF) & 1) ^ 1, longest)) {
                    gave_up();
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = taddr + (uint32_t)(b * BN);
                for (; k < end; k += kSlab, ++it) {
                    const int s = (int)(it % STAGES);
                    if (!wait_bar(early, full_bar(s), (it / STAGES) & 1)) {
                        gave_up();
                        ok = false;
                        break;
                    }
                    // What warp 3 of the other CTA zeroed there is seen here too.
                    if (PAIR && group_k && w.k1 - k < kSlab) mbar_seen_cluster(full_bar(s), (it / STAGES) & 1);
                    ptx::tc_fence_after();
                    const uint32_t off = (uint32_t)(s * (Cfg::STAGE_BYTES / 16));
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_if<PAIR>(on & (uint32_t)(16 * ks < w.k1 - k), d, first_p + off + ks * step_p,
                                          first_q + off + ks * step_q, upper, idesc, ks != 0 || k != first ? 1u : 0u);
                    if constexpr (PAIR) mma_commit_pair_if(on, done_bar(s));
                    else mma_commit_if(on, done_bar(s));
                    const uint32_t next = it + 1;
                    early = mbar_test(full_bar((int)(next % STAGES)), (next / STAGES) & 1);
                }
                if constexpr (PAIR) mma_commit_pair_if(on & (uint32_t)ok, accf_bar(b));
                else mma_commit_if(on & (uint32_t)ok, accf_bar(b));
                ++acc;
            } while (ok && k < w.k1);
        }
        // Everything issued finishes before TMEM is released.
        if (leader) {
            if constexpr (PAIR)
                asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                             "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                                 drain_bar),
                             "r"(on)
                             : "memory");
            else mma_commit_if(on, drain_bar);
            if (!wait_bar(0, drain_bar, 0)) gave_up();
        }
    } else if (warp == 2) {
        // ------------------------------ tiles ------------------------------
        uint32_t n = 0;
        // The place is free when the tile kItems before is stored.
        auto give = [&](const Item &w) {
            if (!wait_tile(iempty_bar(n % kItems), ((n / kItems) & 1) ^ 1, longest)) {
                gave_up();
                return false;
            }
            if (lane == 0) store_item(item_at(n), w);
            __syncwarp();
            mbar_arrive_if(lane == 0, ifull_bar(n % kItems));
            ++n;
            return true;
        };
        bool ok = true;
        if (p.mode == kBf16Dense) {
            const Walk walk((uint32_t)p.col_tiles * (uint32_t)p.row_tiles, units, PAIR);
            for (uint32_t t = unit; ok && t < walk.steps; t += units) ok = give(dense_item<Cfg>(p, walk, t, rank));
        } else if (p.mode == kBf16GroupRows) {
            const uint32_t tiles = (uint32_t)p.col_tiles * (uint32_t)table[p.groups];
            for (uint32_t t = unit; ok && t < tiles; t += units) {
                ok = give(rows_item<Cfg>(p, table, t, rank));
                if (split > 1) break;      // one tile per cluster
            }
        } else if (p.even) {
            const uint32_t tiles = (uint32_t)p.col_tiles * (uint32_t)p.row_tiles, rounds = tiles / units;
            Shares shares;
            for (int g = 0; ok && g < p.groups; ++g) {
                for (uint32_t i = 0; ok && i < rounds; ++i) ok = give(k_item<Cfg>(p, g, i * units + unit));
                int lo, hi;
                group_range(p.offsets, g, p.K, lo, hi);
                // A tile's work: its slabs, and what it takes besides.
                const uint32_t extra = tiles - rounds * units;
                const uint32_t place = shares.give(units, unit, rounds, extra, (uint32_t)slabs(lo, hi) + 4, lane);
                if (ok && place < extra) ok = give(k_item<Cfg>(p, g, rounds * units + place));
            }
        } else {
            const uint32_t tiles = (uint32_t)p.col_tiles * (uint32_t)p.row_tiles;
            int g = 0;
            for (uint32_t t = unit; ok; t += units) {
                for (; g < p.groups && t >= tiles; ++g) t -= tiles;
                if (g >= p.groups) break;
                ok = give(k_item<Cfg>(p, g, t));
            }
        }
        if (ok) give(Item{});
    } else if (warp == 3) {
        // --------------------- the ends of groups along K ---------------------
        // Both operands have K along the rows of their boxes here.
        // A stage's next such slab comes after this one's MMAs: one phase each.
        uint32_t it = 0, n = 0, phases = 0;
        for (; group_k; ++n) {
            if (!item_there(n)) {
                gave_up();
                break;
            }
            const Item w = load_item(item_at(n));
            done_with(n);
            if (w.cols == 0) break;
            const int nk = slabs(w.k0, w.k1), valid = (w.k1 - w.k0) % kSlab;
            it += nk;
            if (valid % 16 == 0) continue;
            const int s = (int)((it - 1) % STAGES);
            if (!wait_tile(tail_bar(s), (phases >> s) & 1, longest)) {
                gave_up();
                break;
            }
            phases ^= 1u << s;
            const int end = (valid + 15) / 16 * 16;
            constexpr int boxes = 2 + (QR + 63) / 64;
            // Four rows of 128 bytes at a time.
            for (int r = valid + lane / 8; r < end; r += 4) {
#pragma unroll
                for (int box = 0; box < boxes; ++box)
                    st_shared_u32x4(stage_p(s) + 8192 * box + 128 * r + 16 * (lane % 8), make_uint4(0, 0, 0, 0));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if constexpr (PAIR) mbar_arrive_cluster_if(lane == 0, map_shared(full_bar(s), 0));
            else mbar_arrive_if(lane == 0, full_bar(s));
        }
    } else {
        // ------------------------------ epilogue ------------------------------
        const int ew = warp - 4, quarter = ew & 3, col0 = (ew >> 2) * CW;
        const int lane0 = 32 * quarter + 128 * pair_rank;
        const uint32_t lanes = taddr + ((uint32_t)(32 * quarter) << 16) + (uint32_t)col0;
        const uint32_t st = base + Cfg::OFF_EXTRA + ew * kStaging;
        if (Cfg::CAN_SPLIT && split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if constexpr (Cfg::MOVE_REGS) ptx::setmaxnreg_inc<216>();
        constexpr int CHUNK = Cfg::CHUNK;
        Arrivals<Cfg> d{base + Cfg::OFF_D + ew * Cfg::D_BYTES, d_bars + 32u * ew, 0};
        uint32_t n = 0, acc = 0;
        // The next accumulator, once complete, and its way back to the MMA warp.
        auto take = [&](uint32_t &from) {
            const int b = (int)(acc % NBUF);
            from = lanes + (uint32_t)(b * BN);
            const bool there = wait_tile(accf_bar(b), (acc / NBUF) & 1, longest);
            ptx::tc_fence_after();
            if (!there) gave_up();
            return there;
        };
        auto give_back = [&]() {
            const int b = (int)(acc % NBUF);
            ptx::tc_fence_before();
            __syncwarp();
            if constexpr (PAIR) mbar_arrive_cluster_if(lane == 0, map_shared(acce_bar(b), 0));
            else mbar_arrive_if(lane == 0, acce_bar(b));
            ++acc;
        };
        for (;; ++n) {
            if (!item_there(n)) {
                gave_up();
                break;
            }
            const Item w = load_item(item_at(n));
            if (w.cols == 0) break;
            if constexpr (Cfg::JOINS) {
                d.next = 0;
                d.ask(p, &mapD, w, lane, lane0, col0);
            }
            uint32_t from;
            if (part == kPartBf16 && w.k1 - w.k0 <= kPartBf16) {
                // bfloat16 C, its sums whole: from tensor memory.
                if (!take(from)) break;
                store_part<__nv_bfloat16, Cfg, false>(p, w, st, lane, lane0, col0, [&](int c) {
                    uint32_t v[CHUNK];
                    float z[CHUNK];
                    tmem_ld_chunk<CHUNK>(from + c, v);
                    tmem_ld_wait_for<CHUNK>(v);
#pragma unroll
                    for (int j = 0; j < CHUNK; ++j) z[j] = w.k0 < w.k1 ? __uint_as_float(v[j]) : 0.0f;
                    stage<CHUNK>(st, lane, p.swap, z);
                }, &mapD, d);
                give_back();
                done_with(n);
                continue;
            }
            float sum[CW];
#pragma unroll
            for (int j = 0; j < CW; ++j) sum[j] = 0.0f;
            bool ok = true;
            int k = w.k0;
            do {
                if (!(ok = take(from))) break;
                if (k < w.k1) {
                    // One load ahead of the additions.
                    uint32_t v[2][16];
                    tmem_ld_chunk<16>(from, v[0]);
#pragma unroll
                    for (int c = 0; c < CW; c += 16) {
                        const int at = c / 16 % 2;
                        tmem_ld_wait_for<16>(v[at]);
                        if (c + 16 < CW) tmem_ld_chunk<16>(from + c + 16, v[at ^ 1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(v[at][j]);
                    }
                }
                give_back();
                k = w.k1 - k > part ? k + part : w.k1;
            } while (k < w.k1);
            if (!ok) break;
            if (split == 1) {
                auto put = [&](int c) {
#pragma unroll
                    for (int i = 0; i < CW; i += CHUNK)
                        if (c == i) stage<CHUNK>(st, lane, p.swap, sum + i);
                };
                if (p.c_bf16) store_part<__nv_bfloat16, Cfg, true>(p, w, st, lane, lane0, col0, put, &mapD, d);
                else store_part<float, Cfg, true>(p, w, st, lane, lane0, col0, put, &mapD, d);
            } else if constexpr (Cfg::CAN_SPLIT) {
                // To the CTA that adds column j over the cluster: j % split.
                const int per = BN / split, shift = __ffs(split) - 1;
                const uint32_t mine = base + Cfg::OFF_EXTRA + 4 * (rank * per * 128 + 32 * quarter + lane);
#pragma unroll
                for (int j = 0; j < CW; ++j) {
                    const int col = col0 + j;
                    st_cluster_f32(mine + 4 * 128 * (col >> shift), (uint32_t)(col & (split - 1)), sum[j]);
                }
            }
            done_with(n);
        }
        // What a role that gave up has asked for lands before the CTA leaves.
        for (; d.asked != d.taken; ++d.taken) d.wait(p);
        if (!d.ok) gave_up();
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
            // in rank order (of lanes that hold columns of C: a split tile is
            // swapped). Nothing reaches into another CTA after this barrier.
            ptx::cluster_sync_all();
            Item w{};
            if (p.mode == kBf16Dense) {
                const Walk walk((uint32_t)p.col_tiles * (uint32_t)p.row_tiles, units, false);
                if (unit < walk.steps) w = dense_item<Cfg>(p, walk, unit, rank);
            } else if (unit < (uint32_t)p.col_tiles * (uint32_t)table[p.groups]) {
                w = rows_item<Cfg>(p, table, unit, rank);
            }
            if (w.cols > 0) {
                const uint32_t part = base + Cfg::OFF_EXTRA;
                const int per = BN / split;
                auto add = [&](auto q) {
                    using T = std::remove_reference_t<decltype(*q.C)>;
                    constexpr int V = 16 / (int)sizeof(T), PER_COL = 128 / V;
                    for (int i = threadIdx.x; i < per * PER_COL; i += Cfg::THREADS) {
                        const int col = i / PER_COL, at = i % PER_COL * V;
                        const int m = w.m + col * split + rank, n = w.n + at;
                        if (m >= w.m_end || n >= p.N) continue;
                        const bool whole = p.vec && n + V <= p.N;
                        Values<T, V> d;
                        if (whole && q.D) d = *reinterpret_cast<const Values<T, V> *>(q.D + m * p.ldd + n);
                        float z[V] = {};
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            if (r >= split) continue;
#pragma unroll
                            for (int e = 0; e < V; e += 4) {
                                const uint4 u = ld_shared_u32x4(part + 4 * ((r * per + col) * 128 + at + e));
                                z[e] += __uint_as_float(u.x), z[e + 1] += __uint_as_float(u.y);
                                z[e + 2] += __uint_as_float(u.z), z[e + 3] += __uint_as_float(u.w);
                            }
                        }
                        if (!whole) {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                if (n + e < p.N) store_one(p, q, m, n + e, z[e]);
                            continue;
                        }
                        if (q.bias) {
#pragma unroll
                            for (int e = 0; e < V; ++e) z[e] += __ldg(q.bias + n + e);
                        }
                        Values<T, V> o;
                        if (q.pre) {
#pragma unroll
                            for (int e = 0; e < V; ++e) store_from_float(&o.v[e], z[e]);
                            *reinterpret_cast<Values<T, V> *>(q.pre + m * p.ld_pre + n) = o;
                        }
                        with_activation(p.act, [&](auto a) {
#pragma unroll
                            for (int e = 0; e < V; ++e) z[e] = activate<decltype(a)::value>(z[e]);
                        });
                        if (q.D) {
#pragma unroll
                            for (int e = 0; e < V; ++e) z[e] = joined(z[e], load_as_float(&d.v[e]), p.join);
                        }
#pragma unroll
                        for (int e = 0; e < V; ++e) store_from_float(&o.v[e], z[e]);
                        *reinterpret_cast<Values<T, V> *>(q.C + m * p.ldc + n) = o;
                    }
                };
                if (p.c_bf16) add(place_of<__nv_bfloat16>(p, w.group));
                else add(place_of<float>(p, w.group));
            }
        }
    }
    // Neither CTA of a pair leaves while the other's MMAs or arrivals reach it.
    if constexpr (PAIR) {
        __syncwarp();
        ptx::cluster_sync_all();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        tmem_dealloc<PAIR>(taddr, Cfg::TMEM_COLS);
    }
}

// Tensor map of an operand: `outer` rows of `inner` values, `groups` of them
// `stride` values apart, in boxes of 64 values by box_rows rows.
cudaError_t encode_bf16(CUtensorMap *map, const void *ptr, int64_t inner, int64_t outer, int64_t ld, int64_t groups,
                        int64_t stride, int box_rows)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)groups};
    // (The stride of a single row or matrix is not used, whatever it is.)
    const int64_t row = outer > 1 ? ld : (inner + 7) / 8 * 8;
    const cuuint64_t strides[2] = {(cuuint64_t)(2 * row), (cuuint64_t)(2 * (groups > 1 ? stride : row * outer))};
    const cuuint32_t box[3] = {(cuuint32_t)kSlab, (cuuint32_t)box_rows, 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tensor map of D (of all groups' under GroupK), in boxes of a chunk.
cudaError_t encode_d(CUtensorMap *map, const Bf16Args &g, int box_rows)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const int64_t size = g.c_bf16 ? 2 : 4, many = g.mode == kBf16GroupK ? g.groups : 1;
    const cuuint64_t dims[3] = {(cuuint64_t)g.N, (cuuint64_t)g.M, (cuuint64_t)many};
    const int64_t row = g.M > 1 ? g.ldd : (g.N + 7) / 8 * 8;
    const cuuint64_t strides[2] = {(cuuint64_t)(row * size), (cuuint64_t)((many > 1 ? g.stride_c : g.M * row) * size)};
    const cuuint32_t box[3] = {32, (cuuint32_t)box_rows, 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = encode(map, g.c_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                              const_cast<void *>(g.D), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class Cfg>
cudaError_t prepare_cfg()
{
    return cudaFuncSetAttribute(bf16_product_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
}

// Whether C, pre and D can be accessed 16 bytes at a time.
bool in_pieces(const Bf16Args &g)
{
    const int64_t per16 = g.c_bf16 ? 8 : 4;
    return pieces16(g.C, g.ldc, per16) && pieces16(g.pre, g.ld_pre, per16) &&
           (g.join == kJoinNone || pieces16(g.D, g.ldd, per16)) && (g.mode != kBf16GroupK || g.stride_c % per16 == 0);
}

template <class Cfg>
cudaError_t launch_cfg(const Bf16Args &g, const Bf16Plan &plan, cudaStream_t stream)
{
    Bf16Params p{};
    p.mode = g.mode;
    p.swap = plan.swap;
    p.M = (int)g.M, p.N = (int)g.N, p.K = (int)g.K;
    p.tm = plan.swap ? Cfg::BN : Cfg::LANES;
    p.tn = plan.swap ? Cfg::LANES : Cfg::BN;
    // A stored K x M and B stored K x N have their rows (M, N) contiguous.
    const bool a_mn = g.op_a == 1, b_mn = g.op_b == 0;
    p.p_mn = plan.swap ? b_mn : a_mn;
    p.q_mn = plan.swap ? a_mn : b_mn;
    CUtensorMap map_a, map_b;
    const int64_t bg = g.mode == kBf16GroupRows ? g.groups : 1;
    const int q_rows = Cfg::QR < 32 ? Cfg::QR : 32, a_rows = plan.swap ? q_rows : 64, b_rows = plan.swap ? 64 : q_rows;
    cudaError_t e;
    if (g.K > 0) {
        const int64_t a_outer = a_mn ? g.K : g.M, b_outer = b_mn ? g.K : g.N;
        e = encode_bf16(&map_a, g.A, a_mn ? g.M : g.K, a_outer, g.lda, 1, a_outer * g.lda, a_mn ? kSlab : a_rows);
        if (e == cudaSuccess)
            e = encode_bf16(&map_b, g.B, b_mn ? g.N : g.K, b_outer, g.ldb, bg, bg > 1 ? g.stride_b : b_outer * g.ldb,
                            b_mn ? kSlab : b_rows);
    } else {
        // The empty sum: no copy is ever issued, the maps only have to be valid.
        const void *any = reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(g.C) & ~uintptr_t(15));
        e = encode_bf16(&map_a, any, 8, 1, 8, 1, 8, 8);
        map_b = map_a;
    }
    if (e != cudaSuccess) return e;
    p.groups = g.groups;
    p.offsets = g.offsets;
    p.row_tiles = (int)ceil_div(g.M, p.tm);
    p.col_tiles = (int)ceil_div(g.N, p.tn);
    // Tiles are counted in 32 bits.
    const int64_t hit = g.groups < g.M ? g.groups : g.M;
    const int64_t rows = g.mode == kBf16Dense       ? p.row_tiles
                         : g.mode == kBf16GroupRows ? g.M / p.tm + hit
                                                    : (int64_t)p.row_tiles * g.groups;
    if (rows + 2 * kRaster > INT32_MAX / p.col_tiles - 2 * kRaster) return cudaErrorInvalidValue;
    p.by_cols = fast_div((uint32_t)p.col_tiles);
    // Worth it where a group's tiles are about a wave of CTAs (16 uneven groups
    // of 2048 x 2048, 64 tiles for 76 pairs: 119 -> 111 us): with many more the
    // rest matters little, with few and many groups the finding costs more.
    const int64_t units = plan.grid / (Cfg::PAIR ? 2 : 1), each = (int64_t)p.row_tiles * p.col_tiles;
    p.even = g.mode == kBf16GroupK && g.groups > 1 && g.groups <= 128 && units <= 32 * kWalkers && 4 * each >= units &&
             each <= 16 * units && each % units != 0;
    p.split = plan.split;
    p.bias = g.bias;
    p.stride_bias = g.stride_bias;
    p.act = g.act;
    p.join = g.join;
    p.pre = g.pre;
    p.ld_pre = g.ld_pre;
    p.D = g.D;
    p.ldd = g.ldd;
    p.C = g.C;
    p.ldc = g.ldc;
    p.stride_c = g.stride_c;
    p.c_bf16 = g.c_bf16;
    p.vec = in_pieces(g);
    p.status = g.status;
    CUtensorMap &mp = plan.swap ? map_b : map_a, &mq = plan.swap ? map_a : map_b;
    CUtensorMap map_d = map_a;                        // any valid one where D does not come by it
    if (Cfg::JOINS && p.vec && (e = encode_d(&map_d, g, Cfg::CHUNK)) != cudaSuccess) return e;
    void *args[] = {&mp, &mq, &map_d, &p};
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attrs[1];
    const unsigned cluster = Cfg::PAIR ? 2u : (unsigned)plan.split;
    if (cluster > 1) {
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = cluster;
        attrs[0].val.clusterDim.y = 1;
        attrs[0].val.clusterDim.z = 1;
        lc.attrs = attrs;
        lc.numAttrs = 1;
    }
    lc.gridDim = dim3((unsigned)plan.grid);
    lc.blockDim = dim3(Cfg::THREADS);
    lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
    lc.stream = stream;
    e = cudaLaunchKernelExC(&lc, reinterpret_cast<const void *>(bf16_product_kernel<Cfg>), args);
    return e != cudaSuccess ? e : cudaGetLastError();
}

using Pair256 = Bf16Cfg<256, true>;
using Pair128 = Bf16Cfg<128, true>;
using Pair256Joins = Bf16Cfg<256, true, true>;
using Pair128Joins = Bf16Cfg<128, true, true>;
using One128 = Bf16Cfg<128, false>;
using One64 = Bf16Cfg<64, false>;
using One32 = Bf16Cfg<32, false>;
using One16 = Bf16Cfg<16, false>;

}  // namespace

Bf16Plan plan_bf16(const Bf16Args &g)
{
    const int64_t sms = g.num_sms;
    const int64_t hit = g.groups < g.M ? g.groups : g.M;
    auto tiles_of = [&](int64_t tm, int64_t tn) {
        const int64_t rows = g.mode == kBf16GroupRows ? g.M / tm + hit : ceil_div(g.M, tm);
        return rows * ceil_div(g.N, tn) * (g.mode == kBf16GroupK ? g.groups : 1);
    };
    const int64_t nk = ceil_div(g.mode == kBf16GroupK ? ceil_div(g.K, g.groups) : g.K, kSlab);
    const int64_t per = g.mode == kBf16GroupRows ? ceil_div(g.M, g.groups) : g.M;
    Bf16Plan best{256, true, false, 1, 0};
    double least = 0.0;
    auto consider = [&](int cols, bool pair, bool swap, int split) {
        const int lanes = pair ? 256 : 128;
        const int64_t tm = swap ? cols : lanes, tn = swap ? lanes : cols;
        // Row tiles of groups by their average, as the device finds them.
        const int64_t rows = g.mode == kBf16GroupRows ? hit * ceil_div(per, tm) : ceil_div(g.M, tm);
        const int64_t tiles = rows * ceil_div(g.N, tn) * (g.mode == kBf16GroupK ? g.groups : 1);
        const int64_t at_once = sms / ((pair ? 2 : 1) * split), units = at_once > 0 ? at_once : 1;
        const int64_t last = tiles % units;
        // A dense product's last wave is cut into pieces of a half or a quarter,
        // which take more than that of the time: the lanes' operand is as wide.
        const bool cut = pair && g.mode == kBf16Dense;
        const double half = cols == 256 ? 0.58 : 0.84, quarter = cols == 256 ? 0.49 : 0.76;
        const double waves = (double)(tiles / units) + (last == 0 ? 0.0 : !cut || 2 * last > units ? 1.0 : 4 * last > units ? half : quarter);
        const double slab = pair ? 80.0 + 1.75 * cols : 220.0 + 1.4 * cols;
        const double time = waves * ((double)ceil_div(nk, split) * slab + 600.0 + 8.0 * cols) + (split > 1 ? 1500.0 : 0.0);
        if (least == 0.0 || time < least) {
            least = time;
            best = Bf16Plan{cols, pair, swap, split, 0};
        }
    };
    for (int cols = 16; cols <= 128; cols *= 2) {
        consider(cols, false, true, 1);
        // 16 columns are for few rows: their chunks have 16 rows of C.
        if (g.mode == kBf16Dense && cols > 16) consider(cols, false, false, 1);
        if (g.mode != kBf16GroupK)
            for (int split = 2; split <= 8; split *= 2)
                // Clusters of 8 do not fill the SMs: 16 of them take two turns
                // (256 x 256 x 16384 in 32 columns 29 us, 8 in 64 columns 17).
                if (nk >= 4 * split && tiles_of(cols, 128) * split <= (split == 8 ? sms * 3 / 4 : sms)) consider(cols, false, true, split);
    }
    for (int cols = 128; sms >= 2 && cols <= 256; cols *= 2) consider(cols, true, g.mode == kBf16GroupRows, 1);
    const int64_t lanes = best.pair ? 256 : 128;
    const int64_t tiles = best.swap ? tiles_of(best.cols, lanes) : tiles_of(lanes, best.cols);
    const int64_t cluster = best.pair ? 2 : best.split;
    const int64_t most = sms / cluster * cluster;
    // A single wave that leaves half of the SMs idle, in its pieces.
    const int64_t pieces = !best.pair || g.mode != kBf16Dense || 2 * tiles * cluster > most ? 1 : 4 * tiles * cluster > most ? 2 : 4;
    best.grid = tiles * cluster * pieces < most ? tiles * cluster * pieces : most;
    return best;
}

cudaError_t prepare_bf16()
{
    cudaError_t e = prepare_cfg<Pair256>();
    if (e == cudaSuccess) e = prepare_cfg<Pair128>();
    if (e == cudaSuccess) e = prepare_cfg<Pair256Joins>();
    if (e == cudaSuccess) e = prepare_cfg<Pair128Joins>();
    if (e == cudaSuccess) e = prepare_cfg<One128>();
    if (e == cudaSuccess) e = prepare_cfg<One64>();
    if (e == cudaSuccess) e = prepare_cfg<One32>();
    if (e == cudaSuccess) e = prepare_cfg<One16>();
    return e;
}

cudaError_t launch_bf16(const Bf16Args &g, cudaStream_t stream)
{
    const Bf16Plan p = plan_bf16(g);
    if (p.grid == 0) return cudaSuccess;
    if (p.pair && g.join != kJoinNone)
        return p.cols == 256 ? launch_cfg<Pair256Joins>(g, p, stream) : launch_cfg<Pair128Joins>(g, p, stream);
    if (p.pair) return p.cols == 256 ? launch_cfg<Pair256>(g, p, stream) : launch_cfg<Pair128>(g, p, stream);
    return p.cols == 128  ? launch_cfg<One128>(g, p, stream)
           : p.cols == 64 ? launch_cfg<One64>(g, p, stream)
           : p.cols == 32 ? launch_cfg<One32>(g, p, stream)
                          : launch_cfg<One16>(g, p, stream);
}

}  // namespace sgemm_gb300
