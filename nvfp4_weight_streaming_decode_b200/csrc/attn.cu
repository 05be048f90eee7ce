// attn.cu -- attention of decode rows and drafted trees over the paged cache,
// on the fifth-generation tensor cores.
//
// A lane's T rows times the G query heads that share a cached head form one
// block of up to N = 16..128 query rows against the same keys and values, so
// those are read once for all of them.  Per tile of 128 slots
//     S^T [128 slots][N] = K Q^T        (A = K as it lies in the cache, B = Q)
//     P^T = exp2(S^T c - m),            l += column sums (per thread, joined at the end)
//     O^T [D][N] += V^T P^T             (A = V as it lies, read transposed, B = P)
// with S^T and O^T in tensor memory.  Slots are the 128 rows of the first
// product and head values those of the second, so few query rows cost few
// columns instead of a padded tile of rows: one row and eight drafts run the
// same code at the same memory rate.
//
// The reference m of a column is 24 above the maximum of a segment's first tile
// (or of the first to show it a slot), in log2, not above the running maximum: FP32
// and bf16 hold a weight as exactly at 2^-24 as at 1.  O^T is rescaled only when a
// weight passes 2^-16 -- rarely, by a vote of the 128 threads that share the columns.
// So no weight is above 2^-16, and 65,536 slots of the largest bf16 value still sum
// to a finite O^T (with weights up to 2^32, as far as they are exact too, values
// from 2^96 on overflowed).  What that costs lies below: weights 2^-102 of the largest are
// zero, and values below 2^-102 lose bits.  The weights' one rounding to bf16 is
// the tensor cores' operand type; their sums are taken before it.
//
// Split: the tiles of all (lane, cached head) pairs form one line that the
// grid's CTAs share evenly (ragged lanes balance by themselves).  A pair cut
// between CTAs leaves partial (m, l, O) in the workspace, and a second kernel
// joins them in CTA order.  Lanes with more than N query rows have
// their blocks on neighbouring CTAs in step, so that the second reader of a
// tile finds it in L2.
//
// A CTA (one per SM): eight softmax warps (two per 32 slots, half the columns
// each), a warp that fetches pages with TMA (128-byte swizzle; K of tile t + 1
// before V of tile t), a thread that issues the products (S of tile t + 1
// before O of tile t, so the tensor cores work while the softmax does).
//
// What a row must not see: the score is replaced, not weighted, so masked keys
// can hold anything; a masked value would still enter as 0 * NaN, so the rows
// of V behind the last slot or of a bad page are zeroed in shared memory, and
// non-finite values of drafted slots are zeroed there and added back at the
// end to the rows that do see them.
//
// Lanes of more than 128 query rows to a cached head have a kernel of their own
// (attn_wide_kernel, heads of 64 and 128), the other way round.
//
// What bounds it: memory, while a block has up to 64 rows or so; then the softmax
// (a tile of 128 x 128 costs some 3,000 cycles, of which the exponentials alone
// take 1,024, and the operands' way through shared memory about as much as the
// products); for short contexts the chain of one tile's steps.  Measured
// (device time of a call, join included; the fraction is of 6,530 GB/s copied):
//   8 lanes x 1 row, 40 / 40 heads of 128, up to 4,000 slots   78 us  5.8 TB/s 0.89
//   8 lanes x 8 rows, 40 / 8 heads of 128, up to 32,768 slots 123 us  6.0 TB/s 0.92
//   5 lanes x 2-8 rows, 24 / 4 heads of 256, up to 20,011      56 us  4.9 TB/s 0.76
//   1 row, 40 / 8 heads, no context                           7.1 us
//   1 lane x 64 rows, 64 / 8 heads of 128, 65,537 slots       135 us  1.02 PFLOP/s (attn_wide_kernel; 161 us and
//                                                             0.86 PFLOP/s in a long run, under the power limit)
//   1 lane x 16 rows, 64 / 8 heads of 64, 65,537 slots         57 us  2.3 TB/s 0.36 (blocks of 128 rows: the softmax)
//
// Every wait is bounded; one that runs out flags the device status, stops the
// CTA, waits (bounded) for copies and products in flight, frees the tensor
// memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "async.cuh"
#include "cache.cuh"
#include "internal.h"

namespace nvfp4 {

__device__ unsigned int g_attn_status;

namespace {

constexpr unsigned kBadPage = 1u, kGaveUp = 4u;
constexpr int kTile = 128;                 // slots per tile
constexpr int kMaxLanes = NVFP4_CACHE_MAX_LANES;
constexpr float kAbove = 24.f;             // a reference lies this far above its score, in log2
constexpr float kUp = 16777216.f;          // 2^kAbove
constexpr float kMostLog = -16.f;          // a score with more than this against its reference raises it
constexpr float kMostWeight = 1.f / 65536;  // 2^kMostLog
constexpr float kMostFloat = 3.402823466e38f;
constexpr float kUnseen = -kMostFloat;     // reference of a column that has seen no slot
constexpr uint32_t kSleepNs = 1000;
constexpr uint32_t kPolls = 1u << 20;      // about a second

// Shared-memory plan of a variant.  The ring's entries are 128 slots x up to
// 128 values of K or V, as atoms of 128 slots x 64 values (128 bytes a slot).
// N = 256: two halves of 128 query rows as the products' rows (attn_wide_kernel).
template <int D, int N>
struct Plan {
    static constexpr bool kWide = N == 256;
    static constexpr int kD = D, kN = N;
    static constexpr int kAtoms = D >= 128 ? 2 : 1;          // atoms per ring entry
    static constexpr int kEntry = kAtoms * kTile * 128;      // bytes
    static constexpr int kPer = D > 128 ? 2 : 1;             // entries per tile of K (or V)
    static constexpr int kPBufs = kWide ? 0 : N == 128 && D == 256 ? 1 : 2;
    static constexpr int kPBytes = kTile * N * 2;
    static constexpr int kQBytes = N * D * 2;
    static constexpr int kBudget = 226 * 1024 - 8192;        // what is left holds barriers and the lane tables
    static constexpr int kFit = (kBudget - kQBytes - kPBufs * kPBytes) / kEntry;
    static constexpr int kRing = kFit > 12 ? 12 : kFit;
    static constexpr int kOffP = kRing * kEntry;
    static constexpr int kOffQ = kOffP + kPBufs * kPBytes;
    static constexpr int kOffMisc = kOffQ + kQBytes;
    // Softmax warps come in two groups of four (32 slots each), half the columns each.
    static constexpr int kCols = N / 2;                      // columns per softmax thread
    static constexpr int kSoftWarps = 8, kSoftThreads = 32 * kSoftWarps;
    static constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
    static constexpr int kThreads = kSoftThreads + 128;      // the last group: pages, products, queries, an idle warp
    // Registers: kThreads x kLaunch at launch = softmax threads x kSoft + 128 x kRest
    // (what one side gains the other gives up, or the gaining side would wait forever).
    static constexpr int kLaunch = 168, kSoft = 208, kRest = 88;
    static_assert(kThreads * kLaunch == kSoftThreads * kSoft + 128 * kRest && kThreads * kLaunch <= 65536, "registers");
    static constexpr int kOBlocks = D > 128 ? 2 : 1;         // 128-row blocks of O^T
    // loads and products take entries in one order, so a tile of V beside one entry of K is enough to go on
    static_assert(kRing > kPer, "V of a tile fits the ring");
    static_assert(kWide ? D <= 128 : 2 * N + kOBlocks * N <= 512, "tensor memory");
};

// What the schedule goes by.
struct Lanes {
    int tiles[kMaxLanes], lo[kMaxLanes], nodes[kMaxLanes], len[kMaxLanes], end[kMaxLanes];
    int base[kMaxLanes + 1];  // first unit of each lane
    int width;                // CTAs that share a (lane, head), one per block of query rows
    int groups;               // of `width` CTAs, that share the units
    int whole;                // a (lane, cached head) pair is one unit: none is cut
};

constexpr int kCleaned = 8;  // more than the tiles of V a ring holds

struct Shared {  // at kOffMisc
    uint64_t full[12], empty[12];
    uint64_t sfull[4], pfull[4], pfree[2];
    uint64_t qfull, qempty, ofull, drain;
    uint64_t cleaned[kCleaned], odone[2], left[2];  // of attn_wide_kernel
    uint32_t tmem;
    int abort;
    unsigned long long bad_v;          // drafted slots with non-finite values, this segment
    Lanes lanes;
    uint64_t vis[128];                 // drafted slots each column sees
    alignas(16) float neg_m[128];      // each column's reference, negated
    uint8_t raw[128];                  // whether it is a raw score
    float inv[128];                    // 1 / sum; before, while references rise, the factor of what was weighed so far
    int64_t off[128];                  // where each column's output row starts
    int lse[128];
    float red[4][128];
};
static_assert(sizeof(Shared) <= 8192, "what the plans leave for it");

struct AttnParams {
    nvfp4_cache c;
    nvfp4_attn_args a;
    float* part_o;       // [ctas][2][N][D]
    float2* part_ml;     // [ctas][2][N]: reference and sum, negative where the reference is a raw score
    int ctas;            // of the attention kernel
    int per_block;       // rows of a lane per block: as many whole rows (of G columns) as fit N
    int q_box;           // rows a copy of Q brings (at most per_block)
};

// -------------------------------------------------------------- tensor cores

// K-major operand, 128-byte swizzle: 8-row groups of 128-byte rows, 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major operand, 128-byte swizzle: rows of k, 64 values of mn each; the next
// 64 values `mn_step` bytes on, the next 8 rows of k 1024 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t mn_step)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(mn_step >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major operand without swizzle: 8 x 16-byte core matrices (8 rows of k, 8
// values of mn), the next 8 rows of k 128 bytes on, the next 8 values of mn
// 128 slots x 16 bytes on.
__device__ __forceinline__ uint64_t desc_p(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(kTile * 16 >> 4) << 32) |
           ((uint64_t)1 << 46);
}

// The whole warp runs the code around these, and its leader (one lane, always
// the same) issues: operands then stay in uniform registers.  Under a branch of
// one lane each product took 105 cycles to issue, so 32 of work.
__device__ __forceinline__ void mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%6, %6, %6, %6}, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader), "r"(0u)
        : "memory");
}
// The same with A in tensor memory: a row's values in pairs, 16 of them in 8 columns.
__device__ __forceinline__ void mma_tm(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%6, %6, %6, %6}, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader), "r"(0u)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ uint32_t elect()
{
    uint32_t r;
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 8 columns of this warp's 32 lanes.
__device__ __forceinline__ void tm_ld8(uint32_t t, float* v)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t t, float* v)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t t, const float* v)
{
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// After tm_wait_ld: what was loaded is not used before this.
template <int C>
__device__ __forceinline__ void settled(float (&v)[C])
{
#pragma unroll
    for (int i = 0; i < C; ++i) asm volatile("" : "+f"(v[i]));
}

template <int C>
__device__ __forceinline__ void tm_ld(uint32_t t, float (&v)[C])
{
    if constexpr (C == 8) {
        tm_ld8(t, v);
    } else {
#pragma unroll
        for (int i = 0; i < C; i += 16) tm_ld16(t + i, v + i);
    }
    tm_wait_ld();
    settled(v);
}

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page,
                                         uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(head), "r"(row), "r"(bar)
        : "memory");
}

// ----------------------------------------------------------- bounded waits

// A plain test first: a try_wait costs hundreds of cycles even when the phase is complete.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// A whole warp.
__device__ __forceinline__ bool waitw(uint32_t bar, uint32_t parity, volatile int* abort)
{
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    for (uint32_t it = 0; it < kPolls; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, kSleepNs))) return true;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
    }
    return false;
}
__device__ __forceinline__ void give_up(volatile int* abort)
{
    if (!*abort) {
        *abort = 1;
        atomicOr(&g_attn_status, kGaveUp);
    }
}

// Barrier over `n` threads that tells each whether any of them said yes.
__device__ __forceinline__ bool any_of(int id, int n, bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
        " selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of FP32 in one instruction: half the issue slots of the softmax.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// ------------------------------------------------------------- the schedule

// Units are (lane, cached head, tile), lane by lane; a group of `width` CTAs
// (one per block of query rows) takes a contiguous range of them.  Each pair
// begins with kStart units without a tile, about what starting and ending a
// pair costs a CTA (with 0 the CTAs that got a border ran 10 % longer).
constexpr int kStart = 4;

struct Segment {
    int b, h;         // lane and cached head
    int t0, t1;       // tiles
    int first;        // the pair's first unit
    int next;         // the unit after the segment
};

// (In 32 bits where the product fits: a 64-bit division takes some 500 cycles,
// and the first page is fetched only after it.)
constexpr int kSmallUnits = 1 << 23;  // times at most 512 groups
__device__ __forceinline__ int range_begin(int units, int groups, int g)
{
    return units < kSmallUnits ? (int)((uint32_t)units * (uint32_t)g / (uint32_t)groups)
                               : (int)((int64_t)units * g / groups);
}
__device__ __forceinline__ int range_owner(int units, int groups, int u)
{
    return units < kSmallUnits ? (int)((((uint32_t)u + 1) * (uint32_t)groups - 1) / (uint32_t)units)
                               : (int)((((int64_t)u + 1) * groups - 1) / units);
}

// Units of a pair of n tiles.
__device__ __forceinline__ int units_of(const Lanes& s, int n) { return n == 0 ? 0 : s.whole ? 1 : n + kStart; }

// Cutting pairs and joining their parts costs a call about what kCut tiles do
// (8 lanes x 8 heads, 8 rows each: 17.8 us cut and 16.0 whole at 800 slots, 19.0
// and 19.1 at 1,200, 22.1 and 25.1 at 2,000).  So pairs stay whole where the CTAs that get the
// most of them need no more tiles for it than an even share and kCut.
constexpr int kCut = 8;
__host__ __device__ __forceinline__ int turns(int pairs, int width, int ctas) { return (pairs * width + ctas - 1) / ctas; }

// The lanes' rows, lengths and tiles, and the groups, for a whole CTA (two
// barriers inside; the caller's own follows).
__device__ __forceinline__ void plan_lanes(const AttnParams& p, Lanes& s, int tid, bool tell)
{
    const nvfp4_cache& c = p.c;
    if (tid < kMaxLanes) {
        int lo = 0, hi = 0, len = 0, end = 0, tiles = 0;
        if (tid < c.lanes) {
            lane_rows(p.a.row_start, tid, p.a.rows, lo, hi);
            const int64_t cap = (int64_t)c.max_pages * c.page_size;
            const int64_t n = max(c.len[tid], 0);
            len = (int)(n < cap ? n : cap);
            const int64_t e = n + (hi - lo);
            end = (int)(e < cap ? e : cap);
            if (hi > lo) {
                tiles = (end + kTile - 1) / kTile;
                if (e > cap && tell) atomicOr(&g_attn_status, kBadPage);
            }
        }
        s.lo[tid] = lo;
        s.nodes[tid] = hi - lo;
        s.len[tid] = len;
        s.end[tid] = end;
        s.tiles[tid] = tiles;
    }
    __syncthreads();
    if (tid < 32) {
        // prefix sums of units and the widest lane, two lanes per thread
        const int lane = tid;
        const int n0 = s.tiles[2 * lane], n1 = s.tiles[2 * lane + 1];
        const int most = __reduce_max_sync(0xffffffffu, max(s.nodes[2 * lane], s.nodes[2 * lane + 1]));
        const int longest = __reduce_max_sync(0xffffffffu, max(n0, n1));
        const int pairs = __reduce_add_sync(0xffffffffu, (n0 > 0) + (n1 > 0)) * c.kv_heads;
        const int64_t tiles = (int64_t)__reduce_add_sync(0xffffffffu, n0 + n1) * c.kv_heads;
        const int width = max(1, (most + p.per_block - 1) / p.per_block);
        const bool whole = (int64_t)turns(pairs, width, p.ctas) * longest <= tiles * width / p.ctas + kCut;
        const int add = whole ? 0 : kStart;
        const int x0 = n0 == 0 ? 0 : (whole ? 1 : n0 + add) * c.kv_heads, x1 = n1 == 0 ? 0 : (whole ? 1 : n1 + add) * c.kv_heads;
        int incl = x0 + x1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        s.base[2 * lane] = incl - x0 - x1;
        s.base[2 * lane + 1] = incl - x1;
        if (lane == 31) {
            s.base[kMaxLanes] = incl;
            s.width = width;
            s.whole = whole;
            s.groups = min(p.ctas / width, incl);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ Segment segment_at(const Lanes& s, int lanes, int u, int u1)
{
    Segment g;
    int b = 0;
    while (b + 1 < lanes && s.base[b + 1] <= u) ++b;
    const int r = u - s.base[b], n = units_of(s, s.tiles[b]);
    g.b = b;
    g.h = r / n;
    g.first = s.base[b] + g.h * n;
    g.next = min(g.first + n, u1);
    if (s.whole) {
        g.t0 = 0;
        g.t1 = s.tiles[b];
        return g;
    }
    g.t0 = max(u - g.first - kStart, 0);
    g.t1 = g.next - g.first - kStart;  // <= t0: nothing but (a part of) the start
    return g;
}

// Position in the order of loads of a segment of n tiles: K0, K1, V0, K2, V1, ...
__device__ __forceinline__ int pos_k(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int pos_v(int t, int n) { return t + 1 < n ? 2 * t + 2 : 2 * n - 1; }

// A log2 weight is s sl - m, one rounding; but m is a rounded score, so the largest
// weight may be off 2^-kAbove by that.  From kRaw on, long before that would show,
// a reference is a raw score r (before the scale) instead: the weight is
// (s - r) sl - kAbove, and s - r is exact for the scores that count.
constexpr float kRaw = 4096.f;
__device__ __forceinline__ bool is_raw(float top) { return fabsf(top) >= kRaw && fabsf(top) <= kMostFloat; }
__device__ __forceinline__ float raw_weight(float s, float neg_r, float sl) { return (s + neg_r) * sl - kAbove; }

// A column's reference: -m, or -r where raw.
struct Reference {
    float neg;
    bool raw;
};

// The reference `was` raised to the score whose u = s sign(sl) is `top`, where that lies
// higher; down: the log2 factor of what has been weighed so far.
__device__ __forceinline__ Reference raised(Reference was, float top, float sl, float& down)
{
    const float mag = fabsf(sl), u = sl < 0.f ? was.neg : -was.neg;  // (of a raw one)
    const float at = top * mag;
    down = 0.f;
    if (was.raw ? !(top > u) : !(at + kAbove > -was.neg)) return was;
    const Reference now = is_raw(at) ? Reference{sl < 0.f ? top : -top, true} : Reference{-(at + kAbove), false};
    if (was.raw)
        down = now.raw ? (u - top) * mag : fmaf(u, mag, now.neg) + kAbove;
    else
        down = now.raw ? -(fmaf(top, mag, was.neg) + kAbove) : now.neg - was.neg;
    return now;
}

// Log-sum-exp of weights that sum to `sum` against a reference.
__device__ __forceinline__ float log_sum(float sum, Reference m, float sl)
{
    if (sum == 0.f) return -INFINITY;
    return (log2f(sum * kUp) + (m.raw ? -m.neg * sl : -m.neg - kAbove)) * 0.6931471805599453f;
}

// C scores of this thread's slot from tensor memory, as log2 weights against the
// references: x = s scale log2(e) - m.  Masked ones are -inf, whatever the
// scale's sign.  `plain`: the whole warp's slots are seen by every row; `all`:
// this slot is.  `some_raw`: a column's reference is a raw score.
template <int C>
__device__ __forceinline__ void read_scores(uint32_t at, float (&x)[C], bool plain, bool all, uint64_t bit, float sl,
                                            const uint64_t* vis, const float* neg_m, bool some_raw, const uint8_t* raw)
{
    tm_ld<C>(at, x);
    const f32x2 f = pair(sl, sl);
#pragma unroll
    for (int i = 0; i < C; i += 4) {
        const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(neg_m + i);
        unpair(fma2(pair(x[i], x[i + 1]), f, m.x), x[i], x[i + 1]);
        unpair(fma2(pair(x[i + 2], x[i + 3]), f, m.y), x[i + 2], x[i + 3]);
    }
    if (some_raw) {  // (reads again what it needs: kept apart, so that the common path has its registers)
#pragma unroll
        for (int i = 0; i < C; i += 8) {
            float y[8];
            tm_ld(at + i, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (raw[i + j]) x[i + j] = raw_weight(y[j], neg_m[i + j], sl);
        }
    }
    if (!plain) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (!all && !(vis[i] & bit)) x[i] = -INFINITY;
    }
}

// C log2 scores become weights, which also go to this slot's row of P, rounded
// to bf16; returns the largest score.
template <int C>
__device__ __forceinline__ float weigh(float (&x)[C], uint8_t* prow)
{
    float over = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 0; i < C; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            over = max3(over, x[i + j], x[i + j + 1]);
            x[i + j] = fast_exp2(x[i + j]);
            x[i + j + 1] = fast_exp2(x[i + j + 1]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[i + j], x[i + j + 1]);
            w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(prow + (i >> 3) * (kTile * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return over;
}

// Zero for the NaN and infinities of 64 bf16 values; whether there were any.
__device__ __forceinline__ bool drop_non_finite(uint4* v4)
{
    // an exponent of all ones carries into the sign's place
    uint32_t ones = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint4 v = v4[k];
        ones |= ((v.x & 0x7F807F80u) + 0x00800080u) | ((v.y & 0x7F807F80u) + 0x00800080u) |
                ((v.z & 0x7F807F80u) + 0x00800080u) | ((v.w & 0x7F807F80u) + 0x00800080u);
    }
    if (!(ones & 0x80008000u)) return false;
    uint16_t* h = reinterpret_cast<uint16_t*>(v4);
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
        if ((h[k] & 0x7F80) == 0x7F80) h[k] = 0;
    return true;
}

// ------------------------------------------------------------ references

// C columns of a warp's 32 slots joined by op, to out[column].  Halving: each
// step a lane keeps half of its columns and takes the other lane's of them, C - 1
// exchanges in all where one column after the other would take 5 C.
template <int C, class Op>
__device__ __forceinline__ void join_columns(const float (&x)[C], int lane, float* out, Op op)
{
    constexpr int W = C < 32 ? C : 32;
#pragma unroll
    for (int g = 0; g < C; g += W) {
        float y[W / 2];
#pragma unroll
        for (int w = W / 2; w > 0; w >>= 1) {
            const bool upper = lane & w;
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float a = w == W / 2 ? x[g + i] : y[i], b = w == W / 2 ? x[g + i + w] : y[i + w];
                y[i] = op(upper ? b : a, __shfl_xor_sync(0xffffffffu, upper ? a : b, w));
            }
        }
#pragma unroll
        for (int w = W; w < 32; w <<= 1) y[0] = op(y[0], __shfl_xor_sync(0xffffffffu, y[0], w));
        if (lane < W) out[g + lane] = y[0];
    }
}

// The first tile of a segment: its columns' maxima (of scores read with references of
// 0) become the references.  A column that sees nothing yet stays unseen, and so
// does one whose reference has to be a raw score: its weights then show as too
// large, and rise() sees to it.
template <int C>
__device__ __forceinline__ void first_references(Shared& s, const float (&x)[C], int c0, int quad, int lane, int bar)
{
    join_columns<C>(x, lane, s.red[quad] + c0, [](float a, float b) { return fmaxf(a, b); });
    any_of(bar, 128, false);
    if (quad * 32 + lane < C) {
        const int col = c0 + quad * 32 + lane;
        const float top = fmaxf(fmaxf(s.red[0][col], s.red[1][col]), fmaxf(s.red[2][col], s.red[3][col]));
        s.neg_m[col] = -(is_raw(top) ? kUnseen : fmaxf(top + kAbove, kUnseen));
    }
    any_of(bar, 128, false);
}

// This group of four warps raises the references of the columns with a weight above
// 2^kMostLog in this tile, those alone (a row's result does not depend on the others'),
// to the maxima of the tile's scores, and scales its sums and O^T so far.  Returns
// whether a reference is a raw score.
template <int D, int N>
__device__ __forceinline__ bool rise(Shared& s, uint32_t at_s, uint32_t at_o, bool plain, bool all, uint64_t bit, float sl,
                                     int c0, int quad, int lane, int bar, bool started, f32x2 (&l)[N / 4],
                                     uint32_t pfree, uint32_t parity, volatile int* abort, bool& fail)
{
    using L = Plan<D, N>;
    constexpr int C = L::kCols;
    const float sign = sl < 0.f ? -1.f : 1.f;
#pragma unroll 1
    for (int i0 = 0; i0 < C; i0 += 8) {
        float x[8];
        tm_ld(at_s + i0, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = plain || all || (s.vis[c0 + i0 + i] & bit) ? x[i] * sign : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            if (lane == 0) s.red[quad][c0 + i0 + i] = v;
        }
    }
    any_of(bar, 128, false);
    bool raw = false;
    if (quad * 32 + lane < C) {
        const int col = c0 + quad * 32 + lane;
        const float top = fmaxf(fmaxf(s.red[0][col], s.red[1][col]), fmaxf(s.red[2][col], s.red[3][col]));
        float down = 0.f;
        Reference now = {s.neg_m[col], s.raw[col] != 0};
        // the largest weight, as read_scores has it
        if ((now.raw ? raw_weight(top * sign, now.neg, sl) : fmaf(top * sign, sl, now.neg)) > kMostLog)
            now = raised(now, top, sl, down);
        s.inv[col] = down == 0.f ? 1.f : fast_exp2(down);
        s.neg_m[col] = now.neg;
        s.raw[col] = raw = now.raw;
    }
    raw = any_of(bar, 128, raw);
    // O^T so far, once every product before this tile is done
    if (started) {
        fail = fail || !waitw(pfree, parity, abort);
        fence_after();
    }
#pragma unroll
    for (int i0 = 0; i0 < C; i0 += 8) {
        float down[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) down[j] = s.inv[c0 + i0 + j];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float v, w;
            unpair(l[(i0 + j) / 2], v, w);
            l[(i0 + j) / 2] = pair(v * down[j], w * down[j + 1]);
        }
        if (started) {
#pragma unroll
            for (int blkd = 0; blkd < L::kOBlocks; ++blkd) {
                float o[8];
                const uint32_t at = at_o + blkd * N + i0;
                tm_ld(at, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] *= down[j];
                tm_st8(at, o);
                tm_wait_st();
            }
        }
    }
    fence_before();
    return raw;
}

// ------------------------------------------------- what both kernels share

// Barriers, tensor memory, the schedule (for a whole CTA; ends with a barrier).
template <class L>
__device__ __forceinline__ void start_cta(const AttnParams& p, Shared& s, uint8_t* sm, const CUtensorMap& map_k,
                                          const CUtensorMap& map_v, const CUtensorMap& map_q)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < 12; ++i) {
            mbar_init(smem_addr(&s.full[i]), 1);
            mbar_init(smem_addr(&s.empty[i]), 1);
        }
        for (int i = 0; i < (L::kWide ? 4 : 2); ++i) {
            mbar_init(smem_addr(&s.sfull[i]), 1);
            mbar_init(smem_addr(&s.pfull[i]), L::kWide ? 4 : L::kSoftWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s.pfree[i]), 1);
        }
        mbar_init(smem_addr(&s.qfull), 1);
        mbar_init(smem_addr(&s.qempty), 1);
        mbar_init(smem_addr(&s.ofull), 1);
        mbar_init(smem_addr(&s.drain), 1);
        if (L::kWide) {
            for (int i = 0; i < kCleaned; ++i) mbar_init(smem_addr(&s.cleaned[i]), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_addr(&s.odone[i]), 1);
                mbar_init(smem_addr(&s.left[i]), 4);
            }
        }
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == L::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    if (warp == L::kLoadWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
    }
    // columns of Q that no copy writes stay zero
    for (int i = tid; i < L::kQBytes / 16; i += L::kThreads)
        *reinterpret_cast<uint4*>(sm + L::kOffQ + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async();
    // The join may start once what came before this kernel is complete: it then
    // reads row ranges and lengths while this one runs out.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    plan_lanes(p, s.lanes, tid, blockIdx.x == 0);
    fence_after();
    __syncthreads();
}

// A warp: pages -> ring, in the order K0, K1, V0, K2, V1, ...
template <class L>
__device__ __forceinline__ void load_pages(const AttnParams& p, Shared& s, uint32_t ring, const CUtensorMap& map_k,
                                           const CUtensorMap& map_v, int u0, int u1, int blk, int lane)
{
    const nvfp4_cache& c = p.c;
    const int shift = __ffs(c.page_size) - 1;
    volatile int* abort = &s.abort;
    int idx = 0;  // entries issued so far
    int done = 0;
    bool ok = true;
    const int box = min(c.page_size, kTile);         // slots per copy
    const int pieces = kTile / box;                  // copies per atom of a tile
    for (int u = u0; ok && u < u1;) {
        const Segment g = segment_at(s.lanes, c.lanes, u, u1);
        u = g.next;
        if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
        const int n = g.t1 - g.t0;
        const int32_t* row = c.table + (int64_t)g.b * c.max_pages;
        const int end = s.lanes.end[g.b];
        // lane i < pieces holds the page of piece i; one tile ahead for K
        auto page_of = [&](int t) {
            const int slot = (g.t0 + t) * kTile + lane * box;
            return lane < pieces && slot < end ? row[slot >> shift] : -1;
        };
        auto fetch = [&](const CUtensorMap* map, int pg, int t, int pos) {
            const bool good = pg >= 0 && pg < c.pages;
            const unsigned have = __ballot_sync(0xffffffffu, good);
            const int off = ((g.t0 + t) * kTile + lane * box) & (c.page_size - 1);
            for (int e = 0; e < L::kPer; ++e) {
                const int q = idx + pos * L::kPer + e, slot = q % L::kRing;
                if (q >= L::kRing && !waitw(smem_addr(&s.empty[slot]), ((q / L::kRing) - 1) & 1, abort)) return false;
                const uint32_t bar = smem_addr(&s.full[slot]);
                if (lane == 0) mbar_expect_tx(bar, (uint32_t)(__popc(have) * L::kAtoms * box * 128));
                __syncwarp();
                if (good) {
                    const uint32_t dst = ring + slot * L::kEntry + lane * box * 128;
#pragma unroll
                    for (int x = 0; x < L::kAtoms; ++x)
                        tma_page(dst + x * kTile * 128, map, e * 128 + x * 64, off, g.h, pg, bar);
                }
                done = q + 1;
            }
            return true;
        };
        int prev = page_of(0), next = n > 1 ? page_of(1) : -1;
        ok = fetch(&map_k, prev, 0, 0);
        for (int t = 1; ok && t < n; ++t) {
            const int cur = next;
            if (t + 1 < n) next = page_of(t + 1);
            ok = fetch(&map_k, cur, t, pos_k(t)) && fetch(&map_v, prev, t - 1, pos_v(t - 1, n));
            prev = cur;
        }
        ok = ok && fetch(&map_v, prev, n - 1, pos_v(n - 1, n));
        idx += 2 * n * L::kPer;
    }
    if (!ok && lane == 0) give_up(abort);
    // nothing in flight when the CTA ends: the last ring's worth of entries
    for (int q = max(0, done - L::kRing); q < done; ++q)
        warp_wait(smem_addr(&s.full[q % L::kRing]), (q / L::kRing) & 1);
}

// A warp: the block's rows x the pair's G heads, as the columns' order wants them.
template <class L>
__device__ __forceinline__ void load_queries(const AttnParams& p, Shared& s, uint32_t qbuf, const CUtensorMap& map_q,
                                             int u0, int u1, int blk, int lane)
{
    const nvfp4_cache& c = p.c;
    const int G = p.a.q_heads / c.kv_heads;
    volatile int* abort = &s.abort;
    int seg = 0;
    bool ok = true;
    for (int u = u0; ok && u < u1;) {
        const Segment g = segment_at(s.lanes, c.lanes, u, u1);
        u = g.next;
        if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
        if (seg > 0) ok = waitw(smem_addr(&s.qempty), (seg - 1) & 1, abort);
        if (ok && lane == 0) {
            const uint32_t bar = smem_addr(&s.qfull);
            mbar_expect_tx(bar, (uint32_t)(p.q_box * G * L::kD * 2));
            for (int x = 0; x < L::kD / 64; ++x)
                tma_rows(qbuf + x * L::kN * 128, &map_q, x * 64, g.h * G, s.lanes.lo[g.b] + blk * p.per_block, bar);
        }
        __syncwarp();
        ++seg;
    }
    if (seg > 0) {
        if (!ok && lane == 0) give_up(abort);
        warp_wait(smem_addr(&s.qfull), (seg - (ok ? 1 : 2)) & 1);  // the last copy has landed
    }
}

// ---------------------------------------------------------------- the kernel

template <int D, int N>
__global__ void __launch_bounds__(Plan<D, N>::kThreads, 1)
    attn_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q)
{
    using L = Plan<D, N>;
    // columns of a softmax thread, and those of O it reads at once
    constexpr int C = L::kCols, CE = 8;
    constexpr int kSoftWarps = L::kSoftWarps, kSoftThreads = L::kSoftThreads, kLoadWarp = L::kLoadWarp,
                  kMmaWarp = L::kMmaWarp, kQWarp = L::kMmaWarp + 1;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Shared& s = *reinterpret_cast<Shared*>(sm + L::kOffMisc);
    const uint32_t ring = smem_addr(sm), pbuf = ring + L::kOffP, qbuf = ring + L::kOffQ;
    const nvfp4_cache& c = p.c;
    const nvfp4_attn_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, and known to be
    const int G = a.q_heads / c.kv_heads;
    const int shift = __ffs(c.page_size) - 1;
    volatile int* abort = &s.abort;

    start_cta<L>(p, s, sm, map_k, map_v, map_q);
    const uint32_t tmem = s.tmem;
    const uint32_t tm_s = tmem, tm_o = tmem + 2 * N;
    // this CTA's range and its block of query rows
    const int units = s.lanes.base[kMaxLanes], width = s.lanes.width, groups = s.lanes.groups;
    const int group = blockIdx.x / width, blk = blockIdx.x % width;
    const bool idle = group >= groups;
    const int u0 = idle ? 0 : range_begin(units, groups, group), u1 = idle ? 0 : range_begin(units, groups, group + 1);

    if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRest));
    if (warp == kLoadWarp) {
        load_pages<L>(p, s, ring, map_k, map_v, u0, u1, blk, lane);
    } else if (warp == kQWarp) {
        load_queries<L>(p, s, qbuf, map_q, u0, u1, blk, lane);
    } else if (warp == kMmaWarp) {
        // ---- the products
        const uint32_t lead = elect();
        constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
        constexpr uint32_t kIdS = kBase, kIdO = kBase | (1u << 15) | (1u << 16);
        int idx = 0, seg = 0;
        int done = 0;  // tiles of earlier segments
        bool ok = true;
        for (int u = u0; ok && u < u1;) {
            const Segment g = segment_at(s.lanes, c.lanes, u, u1);
            u = g.next;
            if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
            const int n = g.t1 - g.t0;
            ok = waitw(smem_addr(&s.qfull), seg & 1, abort);
            fence_after();
            for (int t = 0; ok && t <= n; ++t) {
                if (t < n) {  // S of tile t
                    const int T = done + t, sb = T & 1;
                    // its buffer is free: S of tile t - 2 was read before that tile's
                    // weights were announced, and O of tile t - 2 waited for those
                    for (int e = 0; ok && e < L::kPer; ++e) {
                        const int q = idx + pos_k(t) * L::kPer + e, slot = q % L::kRing;
                        ok = waitw(smem_addr(&s.full[slot]), (q / L::kRing) & 1, abort);
                        if (!ok) break;
                        fence_after();
#pragma unroll
                        for (int x = 0; x < L::kAtoms; ++x)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma(lead, tm_s + sb * N, desc_k(ring + slot * L::kEntry + x * kTile * 128 + k * 32),
                                    desc_k(qbuf + (e * L::kAtoms + x) * N * 128 + k * 32), kIdS, (e | x | k) != 0);
                        commit(lead, smem_addr(&s.empty[slot]));
                    }
                    if (ok) {
                        commit(lead, smem_addr(&s.sfull[sb]));
                        if (t == n - 1) commit(lead, smem_addr(&s.qempty));
                    }
                }
                if (ok && t > 0) {  // O of tile t - 1
                    const int T = done + t - 1, pb = T % L::kPBufs;
                    ok = waitw(smem_addr(&s.pfull[pb]), (T / L::kPBufs) & 1, abort);
                    for (int e = 0; ok && e < L::kPer; ++e) {
                        const int q = idx + pos_v(t - 1, n) * L::kPer + e, slot = q % L::kRing;
                        ok = waitw(smem_addr(&s.full[slot]), (q / L::kRing) & 1, abort);
                        if (!ok) break;
                        fence_after();
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            // head_dim 64: both halves of the 128 rows read the one atom
                            mma(lead, tm_o + e * N, desc_mn(ring + slot * L::kEntry + k * 2048, L::kAtoms == 2 ? kTile * 128 : 0),
                                desc_p(pbuf + pb * L::kPBytes + k * 256), kIdO, t > 1 || k != 0);
                        commit(lead, smem_addr(&s.empty[slot]));
                    }
                    if (ok) {
                        commit(lead, smem_addr(&s.pfree[pb]));
                        if (t == n) commit(lead, smem_addr(&s.ofull));
                    }
                }
            }
            idx += 2 * n * L::kPer;
            done += n;
            ++seg;
        }
        if (!ok && lane == 0) give_up(abort);
        commit(lead, smem_addr(&s.drain));  // products in flight (a wait that the abort does not cut short)
        warp_wait(smem_addr(&s.drain), 0);
    } else if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoft));
        // ---- softmax: thread = slot (and value row of O^T), half the columns
        const int wg = warp >> 2, quad = warp & 3, srow = quad * 32 + lane, c0 = wg * C;
        const uint32_t lanebits = (uint32_t)(quad * 32) << 16;
        const float sl = a.scale * 1.4426950408889634f;
        const int bar = 1 + wg;
        constexpr int kAllBar = 5;
        int seg = 0, done = 0, idx = 0;
        bool fail = false;
        for (int u = u0; u < u1;) {
            const Segment g = segment_at(s.lanes, c.lanes, u, u1);
            u = g.next;
            if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
            const int n = g.t1 - g.t0;
            const int len = s.lanes.len[g.b], end = s.lanes.end[g.b], lo = s.lanes.lo[g.b];
            const int rows = min(p.per_block, s.lanes.nodes[g.b] - blk * p.per_block) * G;  // columns in use
            const int32_t* trow = c.table + (int64_t)g.b * c.max_pages;
            int pg = g.t0 * kTile + srow < end ? trow[(g.t0 * kTile + srow) >> shift] : -1;
            // column j of the block is row lo + i, i = blk per_block + j / G, head h G + j % G
            if (tid < N) {
                uint64_t w = 0;
                if (tid < rows) {
                    const int i = blk * p.per_block + tid / G, head = g.h * G + tid % G, T = s.lanes.nodes[g.b];
                    w = a.mask ? a.mask[lo + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
                    if (T < 64) w &= (1ull << T) - 1;
                    s.off[tid] = (int64_t)(lo + i) * a.ldo + (int64_t)head * D;
                    s.lse[tid] = (lo + i) * a.q_heads + head;
                }
                s.vis[tid] = w;
                s.neg_m[tid] = 0.f;
                s.raw[tid] = 0;
                if (tid == 0) s.bad_v = 0;
            }
            any_of(kAllBar, kSoftThreads, false);

            f32x2 l[C / 2];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) l[i] = 0;
            bool stop = false, some_raw = false;
            for (int t = 0; t < n; ++t) {
                const int T = done + t, sb = T & 1, pb = T % L::kPBufs;
                const int slot = (g.t0 + t) * kTile + srow;
                const bool valid = slot < end && pg >= 0 && pg < c.pages;
                if (slot < end && !valid) atomicOr(&g_attn_status, kBadPage);
                const bool plain = __all_sync(0xffffffffu, valid && slot < len);
                if (t + 1 < n) pg = slot + kTile < end ? trow[(slot + kTile) >> shift] : -1;
                const bool all = slot < len && valid;
                const uint64_t bit = valid && slot >= len ? 1ull << (slot - len) : 0ull;
                const uint32_t at_s = tm_s + sb * N + c0 + lanebits;
                fail = fail || !waitw(smem_addr(&s.sfull[sb]), (T >> 1) & 1, abort);
                fence_after();
                float x[C];
                // Two buffers of P: S of this tile was issued after O of the tile before the
                // last, so once S is there the weights of that tile are done with.
                if (L::kPBufs == 1 && T > 0) fail = fail || !waitw(smem_addr(&s.pfree[0]), (T - 1) & 1, abort);
                uint8_t* prow = sm + L::kOffP + pb * L::kPBytes + (srow >> 3) * 128 + (srow & 7) * 16;
                // Turn 0: the first tile's references.  The weights are formed before it is
                // known whether the references hold (the maxima hide behind the
                // exponentials); if not, again in turn 2.
#pragma unroll 1
                for (int turn = t == 0 ? 0 : 1;; ++turn) {
                    read_scores<C>(at_s, x, plain, all, bit, sl, s.vis + c0, s.neg_m + c0, some_raw, s.raw + c0);
                    if (turn == 0) {
                        first_references<C>(s, x, c0, quad, lane, bar);
                        continue;
                    }
                    const float over = weigh<C>(x, prow + (c0 >> 3) * (kTile * 16));
                    if (turn == 2 || !any_of(bar, 128, over > kMostLog || fail)) break;
                    if (any_of(bar, 128, fail)) {
                        if (lane == 0) give_up(abort);
                        stop = true;
                        break;
                    }
                    some_raw = rise<D, N>(s, at_s, tm_o + c0 + lanebits, plain, all, bit, sl, c0, quad, lane, bar, t > 0, l,
                               smem_addr(&s.pfree[(T + L::kPBufs - 1) % L::kPBufs]), ((T - 1) / L::kPBufs) & 1, abort, fail);
                }
                if (stop) break;
#pragma unroll
                for (int i = 0; i < C / 2; ++i) l[i] = add2(l[i], pair(x[2 * i], x[2 * i + 1]));
                if (!plain) {
                    // V rows that are nobody's slot: zero; of drafted slots: their non-finite values
                    for (int e = 0; e < L::kPer; ++e) {
                        const int q = idx + pos_v(t, n) * L::kPer + e, ent = q % L::kRing;
                        fail = fail || !waitw(smem_addr(&s.full[ent]), (q / L::kRing) & 1, abort);
                        if (all || wg >= L::kAtoms) continue;  // one group of warps per atom
                        bool bad = false;
                        uint4* v4 = reinterpret_cast<uint4*>(sm + ent * L::kEntry + wg * kTile * 128 + srow * 128);
                        if (!valid) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) v4[k] = make_uint4(0, 0, 0, 0);
                        } else {
                            bad = drop_non_finite(v4);
                        }
                        if (bad) atomicOr(&s.bad_v, 1ull << (slot - len));
                    }
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s.pfull[pb]));
            }
            // the columns' sums
            if (!stop) {
                float sums[C];
#pragma unroll
                for (int i = 0; i < C / 2; ++i) unpair(l[i], sums[2 * i], sums[2 * i + 1]);
                join_columns<C>(sums, lane, s.red[quad] + c0, [](float a, float b) { return a + b; });
                fail = fail || !waitw(smem_addr(&s.ofull), seg & 1, abort);
                fence_after();
            }
            if (any_of(kAllBar, kSoftThreads, fail || stop)) {
                fail = true;
                break;
            }
            const bool whole = g.t0 == 0 && g.t1 == s.lanes.tiles[g.b];
            const int pslot = g.first <= u0 ? 0 : 1;
            const int64_t part = (int64_t)blockIdx.x * 2 + pslot;
            if (tid < N) {
                const float sum = (s.red[0][tid] + s.red[1][tid]) + (s.red[2][tid] + s.red[3][tid]);
                s.inv[tid] = sum == 0.f ? 0.f : 1.f / sum;
                if (tid < rows) {
                    const Reference m = {s.neg_m[tid], s.raw[tid] != 0};
                    if (!whole)
                        p.part_ml[part * N + tid] = make_float2(-m.neg, m.raw ? -sum : sum);
                    else if (a.lse)
                        a.lse[s.lse[tid]] = log_sum(sum, m, sl);
                }
            }
            any_of(kAllBar, kSoftThreads, false);
            // O^T: this thread's value row(s), its share of the columns
            const uint64_t badv = s.bad_v;
#pragma unroll 1
            for (int blkd = 0; blkd < L::kOBlocks; ++blkd) {
                const int d = blkd * 128 + srow;
                float* po = p.part_o + (part * N + c0) * D + d;
                __nv_bfloat16* out = (__nv_bfloat16*)a.out + d;
#pragma unroll 1
                for (int i0 = 0; i0 < C && c0 + i0 < rows; i0 += CE) {
                    float o[CE];
                    tm_ld<CE>(tm_o + blkd * N + c0 + i0 + lanebits, o);
                    if (d >= D) continue;
                    if (badv) {
#pragma unroll 1
                        for (int j = 0; j < CE; ++j) {
                            for (uint64_t w = badv & s.vis[c0 + i0 + j]; w; w &= w - 1) {
                                const int sl2 = len + __ffsll(w) - 1;
                                const int pgv = trow[sl2 >> shift];
                                const float v = __bfloat162float(
                                    ((const __nv_bfloat16*)c.v)[((((int64_t)a.layer * c.pages + pgv) * c.kv_heads + g.h) *
                                                                     c.page_size + (sl2 & (c.page_size - 1))) * D + d]);
#pragma unroll
                                for (int z = 0; z < CE; ++z)
                                    if (z == j && !isfinite(v)) o[z] += v;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < CE; ++j) {
                        const int col = c0 + i0 + j;
                        if (col < rows) {
                            if (whole)
                                out[s.off[col]] = __float2bfloat16(o[j] * s.inv[col]);
                            else
                                po[(i0 + j) * D] = o[j];
                        }
                    }
                }
            }
            fence_before();
            any_of(kAllBar, kSoftThreads, false);  // the tables of this segment are done with
            done += n;
            idx += 2 * n * L::kPer;
            ++seg;
        }
        if (fail && lane == 0) give_up(abort);
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------- many rows to a head

// What is not in `seen` becomes -inf.
__device__ __forceinline__ void unseen_out(float (&x)[32], bool plain, uint32_t seen)
{
    if (!plain) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1)) x[i] = -INFINITY;
    }
}

// 32 of a row's scores as log2 weights, x = s scale log2(e) - m; those not in `seen` -inf.
__device__ __forceinline__ void log2_weights(float (&x)[32], float sl, Reference m, bool some_raw, bool plain, uint32_t seen)
{
    if (some_raw) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = m.raw ? raw_weight(x[i], m.neg, sl) : fmaf(x[i], sl, m.neg);
    } else {
        const f32x2 scale = pair(sl, sl), minus = pair(m.neg, m.neg);
#pragma unroll
        for (int i = 0; i < 32; i += 2) unpair(fma2(pair(x[i], x[i + 1]), scale, minus), x[i], x[i + 1]);
    }
    unseen_out(x, plain, seen);
}

// The largest of a row's 64 scores, times the scale's sign.
__device__ __forceinline__ float row_top(uint32_t at, float sl, bool plain, const uint32_t (&seen)[2])
{
    const float sign = sl < 0.f ? -1.f : 1.f;
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float x[32];
        tm_ld(at + 32 * c, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= sign;
        unseen_out(x, plain, c == 0 ? seen[0] : seen[1]);
#pragma unroll
        for (int i = 0; i < 32; i += 2) top = max3(top, x[i], x[i + 1]);
    }
    return top;
}

// A row's weights as packed bf16 pairs; returns their sum (before the rounding).
__device__ __forceinline__ float weigh_row(uint32_t at, float sl, Reference m, bool some_raw, bool plain,
                                           const uint32_t (&seen)[2], uint32_t (&w)[32])
{
    f32x2 s0 = 0, s1 = 0;
    float buf[2][32];
    tm_ld16(at, buf[0]);
    tm_ld16(at + 16, buf[0] + 16);
#pragma unroll
    for (int z = 0; z < 2; ++z) {  // 32 at a time, the next ones on their way
        float(&x)[32] = buf[z];
        tm_wait_ld();
        settled(x);
        if (z == 0) {
            tm_ld16(at + 32, buf[1]);
            tm_ld16(at + 48, buf[1] + 16);
        }
        log2_weights(x, sl, m, some_raw, plain, seen[z]);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
#pragma unroll
            for (int j = i; j < i + 4; ++j) x[j] = fast_exp2(x[j]);
            s0 = add2(s0, pair(x[i], x[i + 1]));
            s1 = add2(s1, pair(x[i + 2], x[i + 3]));
#pragma unroll
            for (int j = i; j < i + 4; j += 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[j], x[j + 1]);
                w[16 * z + j / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    float a, b, c, d;
    unpair(s0, a, b);
    unpair(s1, c, d);
    return (a + b) + (c + d);
}

// For lanes with more than 128 query rows to a cached head.  The rows are the
// products' rows here,
//     S [128 rows][128 slots] = Q K^T,   O [128 rows][D] += P V
// so a thread owns a row: no maximum or sum crosses threads, and P goes back to
// tensor memory, over the scores it came from, which takes its 32 KB (written
// and read) out of the shared memory's way.  A CTA has two halves of 128 rows,
// four warps each.  Scores come in steps of 64 slots and two buffers, so that a half's warps
// have the next scores while the tensor cores take up the weights of the last.
// V is shared, so one more warp looks after its slots that rows must not see, ahead
// of the products.
//
// Measured against blocks of 128 rows in attn_kernel (64 query heads, 8 cached ones,
// one lane; us here and there):
//              heads of 128                        heads of 64
//   slots      20 rows   32     48      64         20 rows   32     48      64
//    1,000     22  22  20  20  22  26  23  27      20  21  16  18  19  24  19  25
//    4,000     22  21  24  21  27  25  28  27      18  20  19  20  22  24  22  26
//   16,000     35  38  38  39  51  49  50  59      30  36  31  37  42  47  43  57
//   65,537     78  97  81  97 136 140 135 179      68  96  69  97 122 140 120 181
// Heads of 128 with a block and a half lose up to 10 % between 4,000 and 16,000 slots, as
// does a full block at 4,000; everything else gains, up to 30 %.  The lengths are not known
// where the kernel is chosen, so any lane of more than 128 rows to a head comes here.
//
// Bound by the softmax warps' own chain: a step of 64 slots for both halves takes
// 1,860 cycles, of which the exponentials and the products take 1,024 each (52 % of
// either unit's cycles), and leaving out the exponentials changes nothing, the
// products 10 %.  A warp's step is page lookup and ballots, the wait for the scores, their
// loads, packing, the store and its wait, one after the other, and there are two warps to
// a quarter of the SM to hide it.  Runs of some milliseconds meet the power limit (161 us).
// Not kept: a warp of products for each half, waits that poll, other orders of
// the halves (140 to 146 us).
template <int D>
__global__ void __launch_bounds__(Plan<D, 256>::kThreads, 1)
    attn_wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q)
{
    using L = Plan<D, 256>;
    constexpr int kHalf = 128, kStep = kTile / 2, kSoftWarps = L::kSoftWarps, kLoadWarp = L::kLoadWarp, kMmaWarp = L::kMmaWarp,
                  kQWarp = L::kMmaWarp + 1;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Shared& s = *reinterpret_cast<Shared*>(sm + L::kOffMisc);
    const uint32_t ring = smem_addr(sm), qbuf = ring + L::kOffQ;
    const nvfp4_cache& c = p.c;
    const nvfp4_attn_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = a.q_heads / c.kv_heads;
    const int shift = __ffs(c.page_size) - 1;
    volatile int* abort = &s.abort;

    start_cta<L>(p, s, sm, map_k, map_v, map_q);
    const uint32_t tmem = s.tmem;
    const uint32_t tm_s = tmem, tm_o = tmem + 4 * kStep;  // [half][2 steps][64], [half][128]
    const int units = s.lanes.base[kMaxLanes], width = s.lanes.width, groups = s.lanes.groups;
    const int group = blockIdx.x / width, blk = blockIdx.x % width;
    const bool idle = group >= groups;
    const int u0 = idle ? 0 : range_begin(units, groups, group), u1 = idle ? 0 : range_begin(units, groups, group + 1);

    if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRest));
    if (warp == kLoadWarp) {
        load_pages<L>(p, s, ring, map_k, map_v, u0, u1, blk, lane);
    } else if (warp == kQWarp) {
        load_queries<L>(p, s, qbuf, map_q, u0, u1, blk, lane);
    } else if (warp == kMmaWarp) {
        // ---- the products
        const uint32_t lead = elect();
        constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
        constexpr uint32_t kIdS = kBase | ((uint32_t)(kStep >> 3) << 17);
        constexpr uint32_t kIdO = kBase | (1u << 16) | ((uint32_t)(D >> 3) << 17);
        int idx = 0, seg = 0, tiles = 0;
        int did[2] = {0, 0};     // steps of earlier segments, per half
        int issued[2] = {0, 0};  // products P V, per half
        bool ok = true;
        for (int u = u0; ok && u < u1;) {
            const Segment g = segment_at(s.lanes, c.lanes, u, u1);
            u = g.next;
            if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
            const int n = g.t1 - g.t0, steps = 2 * n;
            const int halves = min(p.per_block, s.lanes.nodes[g.b] - blk * p.per_block) * G > kHalf ? 2 : 1;
            ok = waitw(smem_addr(&s.qfull), seg & 1, abort);
            // S of step i (half a tile), where the weights of the step before the last were
            auto scores = [&](int i, int w) {
                if (i >= steps) return true;
                const int t = i / 2, q = idx + pos_k(t), slot = q % L::kRing, S = did[w] + i;
                if (w == 0 && i % 2 == 0 && !waitw(smem_addr(&s.full[slot]), (q / L::kRing) & 1, abort)) return false;
                if (issued[w] > 0 && !waitw(smem_addr(&s.pfree[w]), (issued[w] - 1) & 1, abort)) return false;
                fence_after();
                const uint32_t at = tm_s + (2 * w + S % 2) * kStep, rows = i % 2 * kStep * 128;
#pragma unroll
                for (int x = 0; x < L::kAtoms; ++x)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma(lead, at, desc_k(qbuf + x * 256 * 128 + w * kHalf * 128 + k * 32),
                            desc_k(ring + slot * L::kEntry + x * kTile * 128 + rows + k * 32), kIdS, (x | k) != 0);
                commit(lead, smem_addr(&s.sfull[2 * w + S % 2]));
                if (w == halves - 1 && i % 2) {
                    commit(lead, smem_addr(&s.empty[slot]));
                    if (i == steps - 1) commit(lead, smem_addr(&s.qempty));
                }
                return true;
            };
            // O of step i
            auto values = [&](int i, int w) {
                const int t = i / 2, q = idx + pos_v(t, n), slot = q % L::kRing, S = did[w] + i, V = tiles + t;
                if (w == 0 && i % 2 == 0 &&
                    (!waitw(smem_addr(&s.full[slot]), (q / L::kRing) & 1, abort) ||
                     !waitw(smem_addr(&s.cleaned[V % kCleaned]), (V / kCleaned) & 1, abort)))
                    return false;
                if (!waitw(smem_addr(&s.pfull[2 * w + S % 2]), (S / 2) & 1, abort)) return false;
                fence_after();
                const uint32_t at = tm_s + (2 * w + S % 2) * kStep;
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k)
                    mma_tm(lead, tm_o + w * kHalf, at + 8 * k,
                           desc_mn(ring + slot * L::kEntry + (i % 2 * (kStep / 16) + k) * 2048,
                                   L::kAtoms == 2 ? kTile * 128 : 0),
                           kIdO, i > 0 || k != 0);
                commit(lead, smem_addr(&s.pfree[w]));
                ++issued[w];
                if (w == halves - 1 && i % 2) commit(lead, smem_addr(&s.empty[slot]));
                if (i == steps - 1) commit(lead, smem_addr(&s.odone[w]));
                return true;
            };
            if (halves == 2) {
                // each half's scores follow the other half's values, when its own last values are done
                ok = ok && scores(0, 0) && scores(0, 1) && scores(1, 0);
                for (int i = 0; ok && i < steps; ++i)
                    ok = values(i, 0) && scores(i + 1, 1) && values(i, 1) && scores(i + 2, 0);
            } else {
                ok = ok && scores(0, 0) && scores(1, 0);
                for (int i = 0; ok && i < steps; ++i) ok = values(i, 0) && scores(i + 2, 0);
            }
            idx += 2 * n;
            tiles += n;
            did[0] += steps;
            if (halves == 2) did[1] += steps;
            ++seg;
        }
        if (!ok && lane == 0) give_up(abort);
        commit(lead, smem_addr(&s.drain));
        warp_wait(smem_addr(&s.drain), 0);
    } else if (warp == kQWarp + 1) {
        // ---- V's rows behind the last slot or of a bad page become zero, and the
        // non-finite values of drafted slots too; a lane looks at four slots
        int idx = 0, tiles = 0;
        int segs[2] = {0, 0};  // earlier segments, per half
        bool ok = true;
        for (int u = u0; ok && u < u1;) {
            const Segment g = segment_at(s.lanes, c.lanes, u, u1);
            u = g.next;
            if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
            const int n = g.t1 - g.t0;
            const int len = s.lanes.len[g.b], end = s.lanes.end[g.b];
            const int32_t* trow = c.table + (int64_t)g.b * c.max_pages;
            // the results of the segments before are out: bad_v is free
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if (segs[w] > 0) ok = ok && waitw(smem_addr(&s.left[w]), (segs[w] - 1) & 1, abort);
            if (lane == 0) s.bad_v = 0;
            __syncwarp();
            for (int t = 0; ok && t < n; ++t) {
                const int q = idx + pos_v(t, n), ent = q % L::kRing, V = tiles + t;
                const int slot0 = (g.t0 + t) * kTile + lane;
                unsigned good = 0, all = 0;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int slot = slot0 + 32 * z;
                    const int pg = slot < end ? trow[slot >> shift] : -1;
                    const bool valid = slot < end && pg >= 0 && pg < c.pages;
                    if (slot < end && !valid) atomicOr(&g_attn_status, kBadPage);
                    good |= valid ? 1u << z : 0u;
                    all |= valid && slot < len ? 1u << z : 0u;
                }
                ok = waitw(smem_addr(&s.full[ent]), (q / L::kRing) & 1, abort);
                if (!ok) break;
                if (__any_sync(0xffffffffu, all != 15u)) {
#pragma unroll 1
                    for (int z = 0; z < 4 * L::kAtoms; ++z) {
                        const int zs = z / L::kAtoms, slot = slot0 + 32 * zs;
                        if (all >> zs & 1) continue;
                        uint4* v4 = reinterpret_cast<uint4*>(sm + ent * L::kEntry + z % L::kAtoms * kTile * 128 +
                                                             (lane + 32 * zs) * 128);
                        if (!(good >> zs & 1)) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) v4[k] = make_uint4(0, 0, 0, 0);
                        } else if (drop_non_finite(v4)) {
                            atomicOr(&s.bad_v, 1ull << (slot - len));
                        }
                    }
                    fence_async();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(smem_addr(&s.cleaned[V % kCleaned]));
            }
            idx += 2 * n;
            tiles += n;
            ++segs[0];
            if (min(p.per_block, s.lanes.nodes[g.b] - blk * p.per_block) * G > kHalf) ++segs[1];
        }
        if (!ok && lane == 0) give_up(abort);
    } else if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoft));
        // ---- softmax: thread = row
        const int half = warp >> 2, quad = warp & 3, col = half * kHalf + quad * 32 + lane;
        const uint32_t lanebits = (uint32_t)(quad * 32) << 16;
        const uint32_t at_half = tm_s + 2 * half * kStep + lanebits, at_o = tm_o + half * kHalf + lanebits;
        const float sl = a.scale * 1.4426950408889634f;
        int seg = 0, did = 0, tiles = 0;
        bool ok = true;
        for (int u = u0; ok && u < u1;) {
            const Segment g = segment_at(s.lanes, c.lanes, u, u1);
            u = g.next;
            if (g.t1 <= g.t0 || blk * p.per_block >= s.lanes.nodes[g.b]) continue;
            const int n = g.t1 - g.t0, steps = 2 * n;
            const int len = s.lanes.len[g.b], end = s.lanes.end[g.b], lo = s.lanes.lo[g.b], nodes = s.lanes.nodes[g.b];
            const int rows = min(p.per_block, nodes - blk * p.per_block) * G;
            tiles += n;
            if (half * kHalf >= rows) continue;
            const int32_t* trow = c.table + (int64_t)g.b * c.max_pages;
            // row `col` of the block: node i of the lane, head `head`
            const int i = blk * p.per_block + col / G, head = g.h * G + col % G;
            uint64_t vis = 0;
            if (col < rows) {
                vis = a.mask ? a.mask[lo + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
                if (nodes < 64) vis &= (1ull << nodes) - 1;
            }
            int pg[2];
            auto pages_of = [&](int i) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int slot = g.t0 * kTile + i * kStep + 32 * z + lane;
                    pg[z] = slot < end ? trow[slot >> shift] : -1;
                }
            };
            pages_of(0);
            Reference m = {-kUnseen, false};
            float l = 0.f;
            bool some_raw = false;  // a reference of the warp's is
            for (int st = 0; st < steps; ++st) {
                const int slot0 = g.t0 * kTile + st * kStep, S = did + st;
                const uint32_t at_s = at_half + S % 2 * kStep;
                uint32_t seen[2];
                bool plain = slot0 + kStep <= len;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    // an entry behind the last slot is -1
                    seen[z] = __ballot_sync(0xffffffffu, pg[z] >= 0 && pg[z] < c.pages);
                    plain = plain && seen[z] == 0xffffffffu;
                }
                if (!plain) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int ahead = len - (slot0 + 32 * z);  // context slots from here on
                        const uint32_t context = ahead >= 32 ? 0xffffffffu : ahead > 0 ? (1u << ahead) - 1 : 0u;
                        const uint32_t drafts = ahead >= 32    ? 0u
                                                : ahead >= 0   ? (uint32_t)(vis << ahead)
                                                : ahead > -64 ? (uint32_t)(vis >> -ahead)
                                                              : 0u;
                        seen[z] &= context | drafts;
                    }
                }
                if (st + 1 < steps) pages_of(st + 1);
                ok = waitw(smem_addr(&s.sfull[2 * half + S % 2]), (S / 2) & 1, abort);
                if (!ok) break;
                fence_after();
                uint32_t w[kStep / 2];
                float sum;
                // The references go by the first step's largest scores; later they rise where the
                // weights' sum is above kMostWeight, which costs nothing to see.
                bool rise = st == 0;
#pragma unroll 1
                for (int turn = 0; turn < 2; ++turn) {
                    if (__any_sync(0xffffffffu, rise)) {
                        const float top = row_top(at_s, sl, plain, seen);
                        float down = 0.f;
                        if (rise) m = raised(m, top, sl, down);
                        down = down == 0.f ? 1.f : fast_exp2(down);
                        l *= down;
                        some_raw = __any_sync(0xffffffffu, m.raw);
                        if (st > 0) {
                            // O so far, once the step before is in (S waited for the one before that)
                            ok = ok && waitw(smem_addr(&s.pfree[half]), (S - 1) & 1, abort);
                            fence_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 8) {
                                float o[8];
                                tm_ld(at_o + d, o);
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] *= down;
                                tm_st8(at_o + d, o);
                            }
                        }
                    }
                    sum = weigh_row(at_s, sl, m, some_raw, plain, seen, w);
                    rise = sum > kMostWeight;
                    if (!__any_sync(0xffffffffu, rise)) break;
                }
                if (!ok) break;
                l += sum;
#pragma unroll
                for (int z = 0; z < kStep / 2; z += 16) tm_st16(at_s + z, w + z);
                tm_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s.pfull[2 * half + S % 2]));
            }
            ok = ok && waitw(smem_addr(&s.odone[half]), seg & 1, abort);
            ok = ok && waitw(smem_addr(&s.cleaned[(tiles - 1) % kCleaned]), ((tiles - 1) / kCleaned) & 1, abort);
            if (!ok) break;
            fence_after();
            const bool whole = g.t0 == 0 && g.t1 == s.lanes.tiles[g.b];
            const int64_t part = ((int64_t)blockIdx.x * 2 + (g.first <= u0 ? 0 : 1)) * 256 + col;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (col < rows) {
                if (!whole)
                    p.part_ml[part] = make_float2(-m.neg, m.raw ? -l : l);
                else if (a.lse)
                    a.lse[(lo + i) * a.q_heads + head] = log_sum(l, m, sl);
            }
            const uint64_t badv = s.bad_v & vis;
            uint16_t* out = (uint16_t*)a.out + (int64_t)(lo + i) * a.ldo + (int64_t)head * D;
            float* po = p.part_o + part * D;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                float o[16];
                tm_ld(at_o + d, o);
                for (uint64_t b = badv; b; b &= b - 1) {
                    const int slot = len + __ffsll(b) - 1;
                    const __nv_bfloat16* v = (const __nv_bfloat16*)c.v +
                                             ((((int64_t)a.layer * c.pages + trow[slot >> shift]) * c.kv_heads + g.h) *
                                                  c.page_size + (slot & (c.page_size - 1))) * D + d;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float x = __bfloat162float(v[j]);
                        if (!isfinite(x)) o[j] += x;
                    }
                }
                if (col < rows && whole) {
                    uint32_t h[8];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(o[j] * inv, o[j + 1] * inv);
                        h[j / 2] = *reinterpret_cast<const uint32_t*>(&y);
                    }
                    *reinterpret_cast<uint4*>(out + d) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(out + d + 8) = make_uint4(h[4], h[5], h[6], h[7]);
                } else if (col < rows) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(po + d + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
                __syncwarp();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s.left[half]));
            did += steps;
            ++seg;
        }
        if (!ok && lane == 0) give_up(abort);
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ------------------------------------------------------------------- joins

// The parts of (lane, head) pairs that were cut between CTAs, joined in CTA
// order: a warp per (row, head), all warps of the GPU at once.  (The last CTA
// of a pair joining it in the first kernel took 20 us and more for twelve parts
// of 48 x 256: one SM's loads.)
// The bounds are the registers that eight loads in flight take: at the compiler's own
// choice of 32 to 48 it spills (1 lane x 16 rows, 64 / 8 heads of 64, 65,537 slots 61.3 us,
// at 64 registers 59.3; 32 rows, 16 / 4 heads of 256, 40,000 slots 59.6, at 80 53.9).
template <int D, int N>
__global__ void __launch_bounds__(256, D == 256 ? 3 : 4) attn_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ Lanes s;
    const nvfp4_attn_args& a = p.a;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    plan_lanes(p, s, threadIdx.x, false);
    const int lane = threadIdx.x & 31, id = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = id / a.q_heads, head = id - r * a.q_heads, G = a.q_heads / p.c.kv_heads;
    if (r >= a.rows) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    // the row's lane: the one whose rows hold it (two lanes per thread)
    const int b0 = 2 * lane, b1 = 2 * lane + 1;
    const unsigned h0 = __ballot_sync(0xffffffffu, r >= s.lo[b0] && r < s.lo[b0] + s.nodes[b0]);
    const unsigned h1 = __ballot_sync(0xffffffffu, r >= s.lo[b1] && r < s.lo[b1] + s.nodes[b1]);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
    if (!(h0 | h1)) return;
    const int b = h0 ? 2 * (__ffs(h0) - 1) : 2 * (__ffs(h1) - 1) + 1;
    const int i = r - s.lo[b], blk = i / p.per_block, col = (i - blk * p.per_block) * G + head % G;
    if (s.whole) return;
    const int units = s.base[kMaxLanes], first = s.base[b] + head / G * (kStart + s.tiles[b]);
    const int glo = range_owner(units, s.groups, first + kStart),
              ghi = range_owner(units, s.groups, first + kStart + s.tiles[b] - 1);
    if (glo == ghi) return;  // not cut: written by the attention kernel
    // part q of the pair: CTA (glo + q) width + blk, its last segment for q = 0 (unless that is its only one)
    const int np = ghi - glo + 1, lo_slot = range_begin(units, s.groups, glo) >= first ? 0 : 1;
    const int64_t rest = ((int64_t)(glo * s.width + blk) * 2) * N + col, step = (int64_t)s.width * 2 * N;
    auto at = [&](int q) { return q ? rest + q * step : rest + lo_slot * N; };
    constexpr int kPer = D / 32;  // values per lane
    // The highest reference m, and the highest u = r sign(sl) of the raw ones: those above
    // zero lie above every m, the others below (but above a part that saw nothing).
    const float sl = a.scale * 1.4426950408889634f, mag = fabsf(sl);
    auto u_of = [&](float r) { return sl < 0.f ? -r : r; };
    float top = kUnseen, top_u = -INFINITY;
    bool raws = false;
    for (int q = lane; q < np; q += 32) {
        const float2 ml = __ldcg(&p.part_ml[at(q)]);
        if (signbit(ml.y)) {
            raws = true;
            top_u = fmaxf(top_u, u_of(ml.x));
        } else {
            top = fmaxf(top, ml.x);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    raws = __any_sync(0xffffffffu, raws);
    if (raws) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top_u = fmaxf(top_u, __shfl_xor_sync(0xffffffffu, top_u, o));
    }
    const bool raw = top_u > 0.f || (top == kUnseen && top_u > -INFINITY);
    // log2 factor of a part's weights against the highest reference, as in raised()
    auto factor = [&](float2 ml) {
        if (raws && signbit(ml.y)) {
            const float u = u_of(ml.x);
            return raw ? (u - top_u) * mag : fmaf(u, mag, -top) + kAbove;
        }
        return raw ? -(fmaf(top_u, mag, -ml.x) + kAbove) : ml.x == top ? 0.f : ml.x - top;
    };
    float sum = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    for (int q0 = 0; q0 < np; q0 += 32) {
        float w = 0.f;
        if (q0 + lane < np) {
            const float2 ml = __ldcg(&p.part_ml[at(q0 + lane)]);
            w = fast_exp2(factor(ml));
            sum += fabsf(ml.y) * w;
        }
        const int n = min(32, np - q0);
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const float* src = p.part_o + at(q0 + j) * D;
            if constexpr (kPer == 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                acc[0] += wj * v.x;
                acc[1] += wj * v.y;
            } else {
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + lane + 8 * e);
                    acc[e] += wj * v.x;
                    acc[e + 1] += wj * v.y;
                    acc[e + 2] += wj * v.z;
                    acc[e + 3] += wj * v.w;
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t* out = reinterpret_cast<uint32_t*>((uint16_t*)a.out + (int64_t)r * a.ldo + (int64_t)head * D);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
        // lane's values: 2 from 2 lane on (64), else 4 from 4 lane + 128 (e / 4) on
        const int d = kPer == 2 ? 2 * lane : 4 * lane + 32 * (e & ~3) + (e & 2);
        out[d / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (lane == 0 && a.lse)
        a.lse[(int64_t)r * a.q_heads + head] = log_sum(sum, raw ? Reference{-u_of(top_u), true} : Reference{-top, false}, sl);
}

// ------------------------------------------------------------------- host

// The driver's tensor-map encoder, looked up once (no link against the driver).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
int encoder(EncodeFn* out)
{
    static std::atomic<EncodeFn> known{nullptr};
    EncodeFn f = known.load();
    if (!f) {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        NVFP4_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r));
        if (r != cudaDriverEntryPointSuccess || !q) return fail_cuda(cudaErrorSymbolNotFound);
        f = (EncodeFn)q;
        known.store(f);
    }
    *out = f;
    return NVFP4_OK;
}

// One layer's pool as [pages][kv_heads][page_size][head_dim], fetched 64 values x a page (at most a tile) at a time.
int page_map(EncodeFn encode, const nvfp4_cache& c, void* pool, int layer, CUtensorMap* map)
{
    const cuuint64_t row = (cuuint64_t)c.head_dim * 2, head = row * c.page_size, page = head * c.kv_heads;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {row, head, page};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < kTile ? c.page_size : kTile), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (uint8_t*)pool + (size_t)layer * c.pages * page,
                              dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? NVFP4_OK : fail_cuda(cudaErrorInvalidValue);
}

// The query rows as [rows][q_heads][head_dim], fetched 64 values x g heads x q_box rows at a time.
int query_map(EncodeFn encode, const nvfp4_attn_args& a, int g, int q_box, CUtensorMap* map)
{
    const cuuint64_t dims[3] = {(cuuint64_t)a.cache->head_dim, (cuuint64_t)a.q_heads, (cuuint64_t)a.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.cache->head_dim * 2, (cuuint64_t)a.ldq * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)q_box};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? NVFP4_OK : fail_cuda(cudaErrorInvalidValue);
}

// Query rows per block: what one lane is expected to have.
int block_rows(int max_nodes, int rows, int g, int head_dim)
{
    const int r = (max_nodes < rows ? max_nodes : rows) * g;
    return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : r <= 128 || head_dim > 128 ? 128 : 256;
}

struct Workspace {
    size_t o, bytes;  // (m, l) pairs first
};
Workspace workspace(int head_dim, int sms)
{
    // two parts per CTA at the widest block
    const int rows = block_rows(NVFP4_ATTN_MAX_ROWS, NVFP4_ATTN_MAX_ROWS, 32, head_dim);
    Workspace w;
    w.o = (size_t)sms * 2 * rows * sizeof(float2);
    w.bytes = w.o + (size_t)sms * 2 * rows * head_dim * sizeof(float);
    return w;
}

template <int D, int N>
auto kernel_of()
{
    if constexpr (N == 256)
        return attn_wide_kernel<D>;
    else
        return attn_kernel<D, N>;
}

template <int D, int N>
int launch_variant(const AttnParams& p, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
                   cudaStream_t stream)
{
    using L = Plan<D, N>;
    constexpr int kBytes = L::kOffMisc + (int)sizeof(Shared) + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
    static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
    int dev = 0;
    NVFP4_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64) return NVFP4_ERR_ARG;
    const auto kernel = kernel_of<D, N>();
    if (!(ready.load() >> dev & 1)) {
        NVFP4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes));
        ready.fetch_or(1ull << dev);
    }
    NVFP4_CUDA_TRY(launch_pdl(kernel, dim3((unsigned)p.ctas), dim3(L::kThreads), kBytes, stream, p, mk, mv, mq));
    // where no pair can be cut, whatever the lengths, there is nothing to join
    const int lanes = p.c.lanes < p.a.rows ? p.c.lanes : p.a.rows;
    const int64_t tiles = ((int64_t)p.c.max_pages * p.c.page_size + kTile - 1) / kTile;
    const int most = turns(lanes * p.c.kv_heads, (p.a.rows + p.per_block - 1) / p.per_block, p.ctas);
    if (most * tiles > kCut) {
        const unsigned grid = (unsigned)((p.a.rows * p.a.q_heads + 7) / 8);
        NVFP4_CUDA_TRY(launch_pdl(attn_join_kernel<D, N>, dim3(grid), dim3(256), 0, stream, p));
    }
    return NVFP4_OK;
}

template <int D>
int launch_dim(int n, const AttnParams& p, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
               cudaStream_t stream)
{
    switch (n) {
    case 16: return launch_variant<D, 16>(p, mk, mv, mq, stream);
    case 32: return launch_variant<D, 32>(p, mk, mv, mq, stream);
    case 64: return launch_variant<D, 64>(p, mk, mv, mq, stream);
    case 128: return launch_variant<D, 128>(p, mk, mv, mq, stream);
    }
    if constexpr (D <= 128) return launch_variant<D, 256>(p, mk, mv, mq, stream);
    return NVFP4_ERR_SHAPE;  // not reached: blocks of 256 are for heads of up to 128
}

}  // namespace

int read_and_clear_attn_status(unsigned* status)
{
    unsigned v = 0;
    NVFP4_CUDA_TRY(cudaDeviceSynchronize());
    NVFP4_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_attn_status, sizeof v));
    if (v != 0) {
        const unsigned zero = 0;
        NVFP4_CUDA_TRY(cudaMemcpyToSymbol(g_attn_status, &zero, sizeof zero));
    }
    *status = v;
    return NVFP4_OK;
}

int validate_attn(const nvfp4_attn_args* a)
{
    if (!a) return NVFP4_ERR_ARG;
    const nvfp4_cache* c = a->cache;
    const int st = check_cache(c);
    if (st != NVFP4_OK) return st;
    if (!a->q || !a->out || !a->workspace) return NVFP4_ERR_ARG;
    if (a->rows < 1 || a->rows > NVFP4_ATTN_MAX_ROWS || (!a->row_start && a->rows > c->lanes)) return NVFP4_ERR_M;
    const int64_t width = (int64_t)a->q_heads * c->head_dim;
    if (a->layer < 0 || a->layer >= c->layers || a->q_heads < 1 || a->q_heads % c->kv_heads ||
        a->q_heads > 32 * c->kv_heads || a->max_nodes < 1 || a->ldq < width || a->ldo < width ||
        (int64_t)c->lanes * c->kv_heads * ((int64_t)c->max_pages * c->page_size / kTile + 1 + kStart) >= (1 << 30) ||
        a->ldq > ((int64_t)1 << 38) || a->ldo > ((int64_t)1 << 40))
        return NVFP4_ERR_SHAPE;
    if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->workspace) || (a->ldq & 7) || (a->ldo & 7) ||
        (((uintptr_t)a->row_start | (uintptr_t)a->lse) & 3) || ((uintptr_t)a->mask & 7))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int launch_attn(const nvfp4_attn_args* a, cudaStream_t stream)
{
    AttnParams p;
    p.c = *a->cache;
    p.a = *a;
    int sms = 0;
    int st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    p.ctas = sms;
    const Workspace w = workspace(p.c.head_dim, sms);
    if (a->workspace_bytes < w.bytes) return NVFP4_ERR_SCRATCH;
    uint8_t* base = (uint8_t*)a->workspace;
    p.part_ml = (float2*)base;
    p.part_o = (float*)(base + w.o);
    EncodeFn encode = nullptr;
    st = encoder(&encode);
    CUtensorMap mk, mv;
    if (st == NVFP4_OK) st = page_map(encode, p.c, p.c.k, a->layer, &mk);
    if (st == NVFP4_OK) st = page_map(encode, p.c, p.c.v, a->layer, &mv);
    if (st != NVFP4_OK) return st;
    // at least one whole row per block, so a lane has at most 64 blocks
    const int g = a->q_heads / p.c.kv_heads, n = block_rows(a->max_nodes, a->rows, g, p.c.head_dim);
    p.per_block = n / g;
    p.q_box = p.per_block < a->rows ? p.per_block : a->rows;
    CUtensorMap mq;
    st = query_map(encode, *a, g, p.q_box, &mq);
    if (st != NVFP4_OK) return st;
    if (sms < NVFP4_ATTN_MAX_ROWS) return fail_cuda(cudaErrorInvalidDevice);
    if (p.ctas > 512) p.ctas = 512;  // what the schedule's arithmetic takes
    return p.c.head_dim == 64    ? launch_dim<64>(n, p, mk, mv, mq, stream)
           : p.c.head_dim == 128 ? launch_dim<128>(n, p, mk, mv, mq, stream)
                                 : launch_dim<256>(n, p, mk, mv, mq, stream);
}

}  // namespace nvfp4

extern "C" int nvfp4_attn_tree_workspace(int rows, int q_heads, int kv_heads, int head_dim, int sm_count,
                                         size_t* bytes)
{
    if (!bytes || sm_count < 1) return NVFP4_ERR_ARG;
    if (rows < 1 || rows > NVFP4_ATTN_MAX_ROWS) return NVFP4_ERR_M;
    if (kv_heads < 1 || q_heads < 1 || q_heads % kv_heads || q_heads > 32 * kv_heads || kv_heads > 256 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return NVFP4_ERR_SHAPE;
    *bytes = nvfp4::workspace(head_dim, sm_count).bytes;
    return NVFP4_OK;
}

extern "C" int nvfp4_attn_tree(const nvfp4_attn_args* args, cudaStream_t stream)
{
    const int st = nvfp4::validate_attn(args);
    return st != NVFP4_OK ? st : nvfp4::launch_attn(args, stream);
}
