// cache.cu -- page operations of the paged cache: fork (beams reordered,
// sequences shared, lanes freed), reserve (new pages, copy of shared last
// pages), compact (the accepted drafts of a verified tree moved together) and
// trim.  All state -- page tables, lengths, reference counts -- is device
// memory, so a decode step that forks, reserves and commits needs no host
// round trip and can be captured in a graph.  There is no free list: a page is
// free when its reference count is 0, and the lowest free ids are taken first,
// so the answer does not depend on scheduling.
//
// All four are chains of a few small loads and one atomic, 2.5 to 5 us a call,
// and where slots move, what HBM gives: eight beams' fork and reserve at 64 layers
// with three copies of 47 slots (74 MB read and written) 19 to 20 us; trim,
// reserve and compact of eight lanes x 8 drafts at 64 layers 11.6 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"

namespace nvfp4 {

__device__ unsigned int g_cache_status;

namespace {

constexpr int kMaxLanes = NVFP4_CACHE_MAX_LANES;
constexpr unsigned kRefused = 1u, kNoPages = 2u;

// ---------------------------------------------------------------- fork
// A thread owns (one of 32 columns, every eighth lane); the old column is read
// into shared memory before any entry of it is written.  Every entry that
// changes moves one reference; sums of +-1 do not depend on their order.
constexpr int kForkCols = 32, kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const nvfp4_cache c, const int32_t* parent)
{
    __shared__ int32_t old[kMaxLanes][kForkCols];
    __shared__ int par[kMaxLanes], olen[kMaxLanes];
    pdl_begin();
    const int tid = threadIdx.x, x = tid % kForkCols, y = tid / kForkCols;
    const int col = blockIdx.x * kForkCols + x;
    if (tid < c.lanes) {
        int p = parent[tid];
        if (p < -1 || p >= c.lanes) {
            p = -1;
            atomicOr(&g_cache_status, kRefused);
        }
        par[tid] = p;
        olen[tid] = c.len[tid];
    }
    if (col < c.max_pages)
        for (int b = y; b < c.lanes; b += kForkThreads / kForkCols)
            old[b][x] = c.table[(int64_t)b * c.max_pages + col];
    __syncthreads();
    if (blockIdx.x == 0 && tid < c.lanes) c.len[tid] = par[tid] >= 0 ? olen[par[tid]] : 0;
    if (col >= c.max_pages) return;
    for (int b = y; b < c.lanes; b += kForkThreads / kForkCols) {
        const int was = old[b][x], now = par[b] >= 0 ? old[par[b]][x] : -1;
        if (was == now) continue;
        c.table[(int64_t)b * c.max_pages + col] = now;
        if (now >= 0 && now < c.pages) atomicAdd(c.ref + now, 1);
        if (was >= 0 && was < c.pages) atomicSub(c.ref + was, 1);
    }
}

// ------------------------------------------------------------- reserve
// One launch plans, copies and applies.  Every CTA reads the same inputs and
// comes to the same plan: how many pages each lane takes (a copy of its shared
// last page, then, up to len + want, one for each shared entry and each missing
// one); the n-th page taken is the n-th free one.
//   Nothing shared: CTA 0 applies the plan.  A CTA that reads later, when tables
//   have changed, still finds nothing shared (the new entries' counts are 1).
//   Shared pages: every CTA counts in when it has read all it needs, copies its
//   share of the last pages' filled slots -- per (layer, k or v, head) one
//   contiguous run -- and the last to count in applies the plan.
constexpr int kResThreads = 512;
constexpr int kResWarps = kResThreads / 32;
constexpr int kResStep = 8 * kResThreads;  // page ids looked at in one step

struct Plan {
    int need[kMaxLanes], first[kMaxLanes], copy[kMaxLanes], last[kMaxLanes], dst[kMaxLanes], fill[kMaxLanes],
        col[kMaxLanes];
    int lo[kMaxLanes];         // [lo, first): entries behind the length that are there
    int shared[kMaxLanes];     // of those, the ones to replace
    int at[kMaxLanes];         // the next entry to look at when they are
    int start[kMaxLanes + 1];  // pages taken before lane b
    int ids[kResStep];         // the free pages of a step, where entries are replaced
    int count[kResWarps];
    int bad, left, copies, replaces, last_in;
};

// Whether lane b gives up page p, in its column col: another holder is left when the
// lanes before b that hold it too, where they ask for room, have had their turn.
__device__ __forceinline__ bool gives_up(const nvfp4_cache& c, const Plan& s, int b, int col, int p)
{
    if (p >= c.pages) return false;
    const int r = c.ref[p];
    if (r <= 1) return false;
    int before = 0;
#pragma unroll 8
    for (int o = 0; o < b; ++o) {  // (loads in flight together)
        const bool in = col >= s.lo[o] && col < s.first[o];
        const int held = in ? c.table[(int64_t)o * c.max_pages + col] : -1;
        before += s.last[o] == p || held == p;
    }
    return r - before > 1;
}

// Walk the free pages in order of their ids, until `total` of them have gone
// by: take(rank, page, before) for each, then, for the whole CTA, step(before,
// after) with the ranks that a step's pages have.  Returns whether there are so
// many (all threads).
template <class Take, class Step>
__device__ bool walk_free(const nvfp4_cache& c, int total, Plan& s, Take take, Step step)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int given = 0;
    for (int base = 0; base < c.pages && given < total; base += kResStep) {
        // 8 neighbours a thread, loads in flight together
        const int p0 = base + 8 * tid;
        int n = 0;
        unsigned free = 0;
        int r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = p0 + i < c.pages ? c.ref[p0 + i] : 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) free |= r[i] == 0 ? 1u << i : 0u;
        n = __popc(free);
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) s.count[warp] = incl;
        __syncthreads();  // every thread has read its ids' counts
        int before = lane < kResWarps ? s.count[lane] : 0, all = before;
#pragma unroll
        for (int off = 1; off < kResWarps; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, all, off);
            if (lane >= off) all += o;
        }
        before = __shfl_sync(0xffffffffu, all - before, warp);
        all = __shfl_sync(0xffffffffu, all, kResWarps - 1);
        int rank = given + before + incl - n;
        for (; free && rank < total; free &= free - 1) take(rank++, p0 + __ffs(free) - 1, given);
        step(given, min(given + all, total));
        given += all;
        __syncthreads();
    }
    return given >= total;
}

// The filled slots of the copied pages, in every layer: per (lane, layer, k or v,
// head) one contiguous run, in pieces of kPiece 16-byte vectors, a warp each with
// all its loads in flight.  (Threads in line over all vectors spent half the
// issue slots on finding their places: fork and reserve of eight beams with three
// 12 MB copies 23.4 us, now 20.1, of which the copies' bytes take 11.)
constexpr int kPiece = 256;

__device__ __forceinline__ void copy_slots(const nvfp4_cache& c, const Plan& s)
{
    const int lane = threadIdx.x & 31;
    const int64_t page = (int64_t)c.page_size * (c.head_dim / 8);  // vectors of a page and head
    const int64_t runs = (int64_t)c.layers * 2 * c.kv_heads, warps = (int64_t)gridDim.x * kResWarps;
    int64_t i = (int64_t)blockIdx.x + (int64_t)(threadIdx.x >> 5) * gridDim.x;  // neighbours in different CTAs
    for (int b = 0; b < c.lanes; ++b) {
        if (!s.copy[b]) continue;
        const int n = s.fill[b] * (c.head_dim / 8), pieces = (n + kPiece - 1) / kPiece;
        const int64_t all = runs * pieces;
        for (; i < all; i += warps) {
            const int64_t r = all < ((int64_t)1 << 31) ? (int64_t)((uint32_t)i / (uint32_t)pieces) : i / pieces;
            const int v0 = (int)(i - r * pieces) * kPiece + lane, h = (int)(r % c.kv_heads);
            const int64_t q = r / c.kv_heads, at = q / 2 * c.pages;
            uint4* pool = (uint4*)(q & 1 ? c.v : c.k) + h * page;
            const uint4* from = pool + (at + s.last[b]) * c.kv_heads * page;
            uint4* to = pool + (at + s.dst[b]) * c.kv_heads * page;
            uint4 x[kPiece / 32];
#pragma unroll
            for (int z = 0; z < kPiece / 32; ++z)
                if (v0 + 32 * z < n) x[z] = from[v0 + 32 * z];
#pragma unroll
            for (int z = 0; z < kPiece / 32; ++z)
                if (v0 + 32 * z < n) to[v0 + 32 * z] = x[z];
        }
        i -= all;
    }
}

__global__ void __launch_bounds__(kResThreads) reserve_kernel(const nvfp4_cache c, const int32_t* want, int32_t* ok)
{
    __shared__ Plan s;
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(c.page_size) - 1;
    if (tid == 0) {
        s.bad = 0;
        s.left = 0;
        s.copies = 0;
        s.replaces = 0;
    }
    if (tid < kMaxLanes) {
        s.lo[tid] = 0;
        s.first[tid] = 0;
        s.shared[tid] = 0;
        s.need[tid] = 0;
        s.copy[tid] = 0;
        s.last[tid] = -1;
        s.dst[tid] = -1;
    }
    __syncthreads();
    // a warp per lane: the missing entries, and its partly filled last page
    for (int b = warp; b < c.lanes; b += kResWarps) {
        const int w = want[b], n = max(c.len[b], 0);
        if (w <= 0) continue;
        const int32_t* row = c.table + (int64_t)b * c.max_pages;
        const int64_t end = (int64_t)n + w;
        if (end > (int64_t)c.max_pages << shift) {
            if (lane == 0) s.bad = 1;
            continue;
        }
        const int c0 = (n + c.page_size - 1) >> shift, c1 = (int)((end + c.page_size - 1) >> shift);
        const bool partly = n & (c.page_size - 1);
        const int p = partly ? row[n >> shift] : -1;
        bool bad = partly && (p < 0 || p >= c.pages);
        int first = c1;  // entries from here on are -1: a lane's pages come first
        for (int q = c0; q < c1; q += 32) {
            const int e = q + lane < c1 ? row[q + lane] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, e < 0);
            bad = bad || __any_sync(0xffffffffu, e >= c.pages && (m == 0 || lane < __ffs(m)));
            if (m) {
                first = q + __ffs(m) - 1;
                break;
            }
        }
        if (bad) {  // a slot would have no page, or one outside the pool: the lane is left out
            if (lane == 0) {
                s.left = 1;
                if (blockIdx.x == 0) atomicOr(&g_cache_status, kRefused);
            }
        } else if (lane == 0) {
            s.need[b] = c1 - first;
            s.lo[b] = s.at[b] = c0;
            s.first[b] = first;
            s.fill[b] = n & (c.page_size - 1);
            s.col[b] = n >> shift;
            s.last[b] = p;
        }
    }
    __syncthreads();
    // what of it is shared, in lane order: all but the last holder take a page of their own
    if (tid < kMaxLanes && s.last[tid] >= 0 && gives_up(c, s, tid, s.col[tid], s.last[tid])) {
        s.copy[tid] = 1;
        s.copies = 1;
    }
    for (int b = warp; b < c.lanes; b += kResWarps) {
        const int32_t* row = c.table + (int64_t)b * c.max_pages;
        int n = 0;
        for (int q = s.lo[b]; q < s.first[b]; q += 32) {
            const int col = q + lane;
            n += __popc(__ballot_sync(0xffffffffu, col < s.first[b] && gives_up(c, s, b, col, row[col])));
        }
        if (lane == 0 && n) {
            s.shared[b] = n;
            s.need[b] += n;
            s.replaces = 1;
        }
    }
    __syncthreads();
    if (warp == 0) {
        // sums over the lanes, two a thread, held at one more than there are pages
        const long long x0 = s.need[2 * lane] + s.copy[2 * lane], x1 = s.need[2 * lane + 1] + s.copy[2 * lane + 1];
        long long incl = x0 + x1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const long long most = (long long)c.pages + 1;
        s.start[2 * lane] = (int)min(incl - x0 - x1, most);
        s.start[2 * lane + 1] = (int)min(incl - x1, most);
        if (lane == 31) s.start[kMaxLanes] = (int)min(incl, most);
    }
    __syncthreads();
    const int total = s.start[kMaxLanes];
    bool enough = !s.bad && total <= c.pages, apply = blockIdx.x == 0;
    unsigned* counter = (unsigned*)c.scratch + 4 * c.lanes;
    auto no_step = [](int, int) {};
    auto lane_of = [&](int rank) {
        int b = 0;
        while (s.start[b + 1] <= rank) ++b;
        return b;
    };
    if (s.copies || s.replaces) {
        if (enough && s.copies)
            enough = walk_free(c, total, s, [&](int rank, int page, int) {
                const int b = lane_of(rank);
                if (s.copy[b] && rank == s.start[b]) s.dst[b] = page;
            }, no_step);
        __syncthreads();
        if (tid == 0) s.last_in = count_in(counter) == gridDim.x - 1;
        __syncthreads();
        apply = s.last_in;
        if (enough) copy_slots(c, s);
    }
    if (!apply) return;
    if (enough)
        enough = walk_free(c, total, s, [](int, int, int) {}, no_step);
    if (enough && !s.replaces) {
        walk_free(c, total, s, [&](int rank, int page, int) {
            const int b = lane_of(rank);
            const int nth = rank - s.start[b] - s.copy[b];
            c.table[(int64_t)b * c.max_pages + (nth < 0 ? s.col[b] : s.first[b] + nth)] = page;
            c.ref[page] = 1;
        }, no_step);
    } else if (enough) {
        // The entries to replace, marked -2 - page, from the last lane to the first:
        // a lane's are known by the entries of the lanes before it.
        for (int b = c.lanes - 1; b >= 0; --b) {
            if (!s.shared[b]) continue;
            int32_t* row = c.table + (int64_t)b * c.max_pages;
            for (int q = s.lo[b] + tid; q < s.first[b]; q += kResThreads) {
                const int p = row[q];
                if (gives_up(c, s, b, q, p)) row[q] = -2 - p;
            }
            __syncthreads();
        }
        // A step's free pages in order; a warp per lane gives its entries theirs.
        walk_free(c, total, s, [&](int rank, int page, int before) { s.ids[rank - before] = page; },
                  [&](int r0, int r1) {
            __syncthreads();
            for (int b = warp; b < c.lanes; b += kResWarps) {
                int r = max(s.start[b], r0);
                const int end = min(s.start[b + 1], r1);
                if (r >= end) continue;
                int32_t* row = c.table + (int64_t)b * c.max_pages;
                if (s.copy[b] && r == s.start[b]) {
                    if (lane == 0) {
                        row[s.col[b]] = s.ids[r - r0];
                        c.ref[s.ids[r - r0]] = 1;
                    }
                    ++r;
                }
                int q = s.at[b];
                while (r < end && q < c.max_pages) {
                    const int col = q + lane, e = col < s.first[b] ? row[col] : -1;
                    const unsigned m = __ballot_sync(0xffffffffu, e < 0);
                    const int mine = r + __popc(m & ((1u << lane) - 1));
                    const bool takes = e < 0 && mine < end && col < c.max_pages;
                    if (takes) {
                        const int page = s.ids[mine - r0];
                        row[col] = page;
                        c.ref[page] = 1;
                        if (e < -1) atomicSub(c.ref + (-2 - e), 1);
                    }
                    const unsigned done = __ballot_sync(0xffffffffu, takes);
                    r += __popc(done);
                    q = done == m ? q + 32 : q + 32 - __clz(done);
                }
                __syncwarp();
                if (lane == 0) s.at[b] = q;
            }
        });
    }
    if (enough && tid < c.lanes && s.copy[tid]) atomicSub(c.ref + s.last[tid], 1);
    if (tid == 0) {
        if (ok) *ok = enough && !s.left ? 1 : 0;
        if (!enough) atomicOr(&g_cache_status, kNoPages);
        if (s.copies || s.replaces) *counter = 0u;
    }
}

// ---------------------------------------------------------------- trim
// Lane blockIdx.x gives up its pages from column `keep` on; its pages come
// first in the row, so the scan ends with the first stretch without one.
__device__ void release_from(const nvfp4_cache& c, int b, int keep, int tid, int threads)
{
    int32_t* row = c.table + (int64_t)b * c.max_pages;
    for (int q = keep; q < c.max_pages; q += threads) {
        const int col = q + tid;
        const int p = col < c.max_pages ? row[col] : -1;
        if (p >= 0) {
            row[col] = -1;
            if (p < c.pages) atomicSub(c.ref + p, 1);
        }
        if (!__syncthreads_or(p >= 0)) return;
    }
}

__global__ void __launch_bounds__(256) trim_kernel(const nvfp4_cache c, const int32_t* new_len)
{
    pdl_begin();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n = min(max(c.len[b], 0), max(new_len[b], 0));
    __syncthreads();  // everyone has read the length
    if (tid == 0) c.len[b] = n;
    release_from(c, b, (n + c.page_size - 1) / c.page_size, tid, 256);
}

// ------------------------------------------------------------- compact
// Moves and commit in one launch.  A group of head_dim / 8 threads owns one
// (lane, layer, k or v, head) and moves its slots in ascending order, up to 8
// at a time: sources ascend strictly and none lies before its target, so a
// later source is never an earlier target of another batch.  The last CTA to
// have read its lane commits lengths and releases pages.
constexpr int kMoveThreads = 256;

struct MoveLane {
    int32_t page_of[NVFP4_ATTN_MAX_ROWS];  // source: page id of path[j]'s slot, and the row in it
    int32_t row_of[NVFP4_ATTN_MAX_ROWS];
    int32_t to_page[NVFP4_ATTN_MAX_ROWS];
    int32_t to_row[NVFP4_ATTN_MAX_ROWS];
    int count;  // slots to look at, from `first` on; 0: none moves
    int first;  // the slots before it lie where they belong
    int len;    // before the commit
    int good;
};

// Whether lane b's count and path can be committed (all threads of a CTA ask).
__device__ void read_lane(const nvfp4_cache& c, int b, const int32_t* count, const int32_t* path, int ld, int tid,
                          MoveLane& m)
{
    const int shift = __ffs(c.page_size) - 1;
    const int n = max(c.len[b], 0), k = count[b];
    const int s = path && tid < ld ? path[(int64_t)b * ld + tid] : 0;
    const int before = path && tid && tid < ld ? path[(int64_t)b * ld + tid - 1] : -1;
    const int32_t* row = c.table + (int64_t)b * c.max_pages;
    const int64_t cap = (int64_t)c.max_pages << shift;
    bool fine = k >= 0 && (!path || k <= ld) && (int64_t)n + k <= cap;
    if (tid == 0) {
        m.first = NVFP4_ATTN_MAX_ROWS;
        m.len = n;
    }
    __syncthreads();
    if (path && fine && tid < k) {
        fine = s > before && s < NVFP4_ATTN_MAX_ROWS && (int64_t)n + s < cap;
        if (fine) {
            const int from = n + s, to = n + tid;
            const int fp = row[from >> shift], tp = row[to >> shift];
            fine = fp >= 0 && fp < c.pages && tp >= 0 && tp < c.pages && (s == tid || c.ref[tp] == 1);
            m.page_of[tid] = fp;
            m.row_of[tid] = from & (c.page_size - 1);
            m.to_page[tid] = tp;
            m.to_row[tid] = to & (c.page_size - 1);
            if (s != tid) atomicMin(&m.first, tid);
        }
    } else if (!path && fine && k > 0) {
        // kept as they lie: the slots need pages
        for (int q = (n >> shift) + tid; q <= (n + k - 1) >> shift; q += blockDim.x)
            fine = fine && row[q] >= 0 && row[q] < c.pages;
    }
    m.count = path ? k : 0;  // the same in every thread
    m.good = __syncthreads_and(fine);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const nvfp4_cache c, const int32_t* count,
                                                               const int32_t* path, int ld)
{
    __shared__ MoveLane m;
    __shared__ int s_last;
    constexpr int kVec = D / 8, kGroups = kMoveThreads / kVec;
    pdl_begin();
    const int tid = threadIdx.x;
    const int b = blockIdx.y;
    read_lane(c, b, count, path, ld, tid, m);
    // What the commit changes has been read: count in before the moves, which go
    // on while the last CTA commits.  Each lane's new length, or -1, is in scratch.
    unsigned* counter = (unsigned*)c.scratch + 4 * c.lanes;
    if (tid == 0) {
        if (blockIdx.x == 0) c.scratch[b] = m.good ? m.len + count[b] : -1;
        s_last = count_in(counter) == gridDim.x * gridDim.y - 1;
    }
    if (path && m.good) {
        const int64_t segs = (int64_t)c.layers * 2 * c.kv_heads;
        const int64_t run = (int64_t)c.page_size * D;
        for (int64_t s = (int64_t)blockIdx.x * kGroups + tid / kVec; s < segs; s += (int64_t)gridDim.x * kGroups) {
            const int h = (int)(s % c.kv_heads), kv = (int)(s / c.kv_heads & 1);
            const int64_t layer = s / c.kv_heads / 2;
            uint4* base = (uint4*)((uint16_t*)(kv ? c.v : c.k) + (layer * c.pages * c.kv_heads + h) * run) + tid % kVec;
            const int64_t page = (int64_t)c.kv_heads * run / 8;
            for (int j = m.first; j < m.count; j += 8) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i < m.count) x[i] = base[m.page_of[j + i] * page + m.row_of[j + i] * kVec];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i < m.count) base[m.to_page[j + i] * page + m.to_row[j + i] * kVec] = x[i];
            }
        }
    }
    __syncthreads();
    if (!s_last) return;
    const int lane = tid & 31;
    for (int l = tid >> 5; l < c.lanes; l += kMoveThreads / 32) {
        const int n = __ldcg(c.scratch + l);
        if (n < 0) {
            if (lane == 0) atomicOr(&g_cache_status, kRefused);
            continue;
        }
        if (lane == 0) c.len[l] = n;
        int32_t* row = c.table + (int64_t)l * c.max_pages;
        bool more = true;  // a lane's pages come first: the scan ends with the first stretch without one
        for (int q = (n + c.page_size - 1) / c.page_size; more && q < c.max_pages; q += 32) {
            const int p = q + lane < c.max_pages ? row[q + lane] : -1;
            if (p >= 0) {
                row[q + lane] = -1;
                if (p < c.pages) atomicSub(c.ref + p, 1);
            }
            more = __any_sync(0xffffffffu, p >= 0);
        }
    }
    if (tid == 0) *counter = 0u;
}

}  // namespace

int read_and_clear_cache_status(unsigned* status)
{
    unsigned v = 0;
    NVFP4_CUDA_TRY(cudaDeviceSynchronize());
    NVFP4_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_cache_status, sizeof v));
    if (v != 0) {
        const unsigned zero = 0;
        NVFP4_CUDA_TRY(cudaMemcpyToSymbol(g_cache_status, &zero, sizeof zero));
    }
    *status = v;
    return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

static bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

extern "C" int nvfp4_cache_fork(const nvfp4_cache* cache, const int32_t* parent, cudaStream_t stream)
{
    const int st = check_cache(cache);
    if (st != NVFP4_OK) return st;
    if (!parent) return NVFP4_ERR_ARG;
    if (!aligned4(parent)) return NVFP4_ERR_ALIGN;
    const unsigned grid = (unsigned)((cache->max_pages + kForkCols - 1) / kForkCols);
    NVFP4_CUDA_TRY(launch_pdl(fork_kernel, dim3(grid), dim3(kForkThreads), 0, stream, *cache, parent));
    return NVFP4_OK;
}

extern "C" int nvfp4_cache_reserve(const nvfp4_cache* cache, const int32_t* want, int32_t* ok, cudaStream_t stream)
{
    int st = check_cache(cache);
    if (st != NVFP4_OK) return st;
    if (!want) return NVFP4_ERR_ARG;
    if (!aligned4(want) || !aligned4(ok)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    NVFP4_CUDA_TRY(launch_pdl(reserve_kernel, dim3((unsigned)(2 * sms)), dim3(kResThreads), 0, stream, *cache, want, ok));
    return NVFP4_OK;
}

extern "C" int nvfp4_cache_trim(const nvfp4_cache* cache, const int32_t* new_len, cudaStream_t stream)
{
    const int st = check_cache(cache);
    if (st != NVFP4_OK) return st;
    if (!new_len) return NVFP4_ERR_ARG;
    if (!aligned4(new_len)) return NVFP4_ERR_ALIGN;
    NVFP4_CUDA_TRY(launch_pdl(trim_kernel, dim3((unsigned)cache->lanes), dim3(256), 0, stream, *cache, new_len));
    return NVFP4_OK;
}

extern "C" int nvfp4_cache_compact(const nvfp4_cache* cache, const int32_t* count, const int32_t* path, int ld_path,
                                   cudaStream_t stream)
{
    int st = check_cache(cache);
    if (st != NVFP4_OK) return st;
    if (!count) return NVFP4_ERR_ARG;
    if (path && (ld_path < 1 || ld_path > NVFP4_ATTN_MAX_ROWS)) return NVFP4_ERR_SHAPE;
    if (!aligned4(count) || !aligned4(path)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    auto launch = [&](auto kernel, int D) {
        const int64_t groups = kMoveThreads / (D / 8), segs = (int64_t)cache->layers * 2 * cache->kv_heads;
        int64_t gx = (segs + groups - 1) / groups;
        const int64_t cap = (8 * sms + cache->lanes - 1) / cache->lanes;  // about 8 CTAs an SM, of which 3 are resident
        if (gx > cap) gx = cap;
        const dim3 grid = path ? dim3((unsigned)gx, (unsigned)cache->lanes) : dim3(1, (unsigned)cache->lanes);
        return launch_pdl(kernel, grid, dim3(kMoveThreads), 0, stream, *cache, count, path, ld_path);
    };
    NVFP4_CUDA_TRY(cache->head_dim == 64    ? launch(compact_kernel<64>, 64)
                   : cache->head_dim == 128 ? launch(compact_kernel<128>, 128)
                                            : launch(compact_kernel<256>, 256));
    return NVFP4_OK;
}
