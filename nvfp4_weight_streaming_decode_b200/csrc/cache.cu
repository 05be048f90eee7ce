// cache.cu -- page operations of the paged cache: fork (beams reordered,
// sequences shared, lanes freed), reserve (new pages, copy of shared last
// pages), compact (the accepted drafts of a verified tree moved together) and
// trim.  All state -- page tables, lengths, reference counts -- is device
// memory, so a decode step that forks, reserves and commits needs no host
// round trip and can be captured in a graph.  There is no free list: a page is
// free when its reference count is 0, and the lowest free ids are taken first,
// so the answer does not depend on scheduling.
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
// One CTA plans: how many pages each lane takes (a copy of its shared last
// page, then the missing entries up to len + want), then the n-th page taken
// is the n-th free one.  The copies go to scratch for the second kernel:
// scratch[4 b ..] = {source page, destination page, filled slots, unused}.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const nvfp4_cache c, const int32_t* want,
                                                                    int32_t* ok)
{
    __shared__ int s_need[kMaxLanes], s_first[kMaxLanes], s_copy[kMaxLanes], s_col[kMaxLanes], s_last[kMaxLanes];
    __shared__ int s_start[kMaxLanes + 1];
    __shared__ int s_bad, s_count[kPlanThreads / 32];
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(c.page_size) - 1;
    if (tid == 0) s_bad = 0;
    if (tid < kMaxLanes) {
        s_need[tid] = 0;
        s_copy[tid] = 0;
        s_last[tid] = -1;
    }
    __syncthreads();
    // a warp per lane: the missing entries
    for (int b = warp; b < c.lanes; b += kPlanThreads / 32) {
        const int w = want[b], n = max(c.len[b], 0);
        if (w <= 0) continue;
        const int32_t* row = c.table + (int64_t)b * c.max_pages;
        const int64_t end = (int64_t)n + w;
        if (end > (int64_t)c.max_pages << shift) {
            if (lane == 0) s_bad = 1;
            continue;
        }
        const int c0 = (n + c.page_size - 1) >> shift, c1 = (int)((end + c.page_size - 1) >> shift);
        int first = c1;  // entries from here on are -1: a lane's pages come first
        for (int q = c0; q < c1; q += 32) {
            const int e = q + lane < c1 ? row[q + lane] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, e < 0);
            if (m) {
                first = q + __ffs(m) - 1;
                break;
            }
        }
        if (lane == 0) {
            s_need[b] = c1 - first;
            s_first[b] = first;
            if (n & (c.page_size - 1)) {
                const int p = row[n >> shift];
                s_col[b] = n >> shift;
                if (p >= 0 && p < c.pages)
                    s_last[b] = p;
                else
                    atomicOr(&g_cache_status, kRefused);
            }
        }
    }
    __syncthreads();
    // which lanes copy their last page: in lane order, all but the last holder
    if (tid < c.lanes && s_last[tid] >= 0) {
        int before = 0;
        for (int b = 0; b < tid; ++b) before += s_last[b] == s_last[tid];
        s_copy[tid] = c.ref[s_last[tid]] - before > 1;
    }
    __syncthreads();
    if (tid == 0) {
        int64_t sum = 0;
        for (int b = 0; b < c.lanes; ++b) {
            s_start[b] = (int)sum;
            sum += s_need[b] + s_copy[b];
            if (sum > c.pages) sum = (int64_t)c.pages + 1;  // more than there are: refused below
        }
        s_start[c.lanes] = (int)sum;
    }
    __syncthreads();
    const int total = s_start[c.lanes];
    // Free pages in order of their ids, 4 ids per thread and step: count until
    // there are enough, then hand them out.
    bool enough = total == 0 && !s_bad;
    if (!enough && !s_bad) {
        int seen = 0;
        for (int base = 0; base < c.pages && seen < total; base += 4 * kPlanThreads) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = base + 4 * tid + i;
                n += p < c.pages && c.ref[p] == 0;
            }
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) s_count[warp] = n;
            __syncthreads();
            for (int i = 0; i < kPlanThreads / 32; ++i) seen += s_count[i];
            __syncthreads();
        }
        enough = seen >= total;
    }
    if (tid < c.lanes) {
        c.scratch[4 * tid] = enough && s_copy[tid] ? s_last[tid] : -1;
        c.scratch[4 * tid + 2] = max(c.len[tid], 0) & (c.page_size - 1);
    }
    if (tid == 0) {
        if (ok) *ok = enough ? 1 : 0;
        if (!enough) atomicOr(&g_cache_status, kNoPages);
    }
    if (!enough || total == 0) return;
    __syncthreads();
    int given = 0;
    for (int base = 0; given < total; base += 4 * kPlanThreads) {
        int n = 0;
        unsigned freem = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = base + 4 * tid + i;
            if (p < c.pages && c.ref[p] == 0) {
                freem |= 1u << i;
                ++n;
            }
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) s_count[warp] = incl;
        __syncthreads();  // every thread has read its ids' counts
        int rank = given + incl - n, all = 0;
        for (int i = 0; i < kPlanThreads / 32; ++i) {
            if (i < warp) rank += s_count[i];
            all += s_count[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!((freem >> i) & 1)) continue;
            if (rank < total) {
                int b = 0;
                while (s_start[b + 1] <= rank) ++b;
                int nth = rank - s_start[b];
                const int p = base + 4 * tid + i;
                int col;
                if (s_copy[b] && nth == 0) {
                    col = s_col[b];
                    c.scratch[4 * b + 1] = p;
                } else {
                    col = s_first[b] + nth - s_copy[b];
                }
                c.table[(int64_t)b * c.max_pages + col] = p;
                c.ref[p] = 1;
            }
            ++rank;
        }
        given += all;
        __syncthreads();
    }
    if (tid < c.lanes && s_copy[tid]) atomicSub(c.ref + s_last[tid], 1);
}

// The planned copies: the filled slots of a page, per (layer, k or v, head) one
// contiguous run, spread over the grid.
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const nvfp4_cache c)
{
    __shared__ int lanes_of[kMaxLanes];
    __shared__ int s_n;
    pdl_begin();
    const int tid = threadIdx.x;
    if (tid == 0) {
        int n = 0;
        for (int b = 0; b < c.lanes; ++b)
            if (c.scratch[4 * b] >= 0) lanes_of[n++] = b;
        s_n = n;
    }
    __syncthreads();
    const int64_t per = (int64_t)c.layers * 2 * c.kv_heads;
    const int64_t segs = per * s_n;
    for (int64_t s = blockIdx.x; s < segs; s += gridDim.x) {
        const int b = lanes_of[s / per];
        const int64_t r = s % per;
        const int h = (int)(r % c.kv_heads), kv = (int)(r / c.kv_heads & 1);
        const int64_t layer = r / c.kv_heads / 2;
        const int64_t run = (int64_t)c.page_size * c.head_dim;  // elements of a page and head
        uint16_t* pool = (uint16_t*)(kv ? c.v : c.k);
        const int64_t at = layer * c.pages;
        const uint4* src = (const uint4*)(pool + ((at + c.scratch[4 * b]) * c.kv_heads + h) * run);
        uint4* dst = (uint4*)(pool + ((at + c.scratch[4 * b + 1]) * c.kv_heads + h) * run);
        const int n = c.scratch[4 * b + 2] * (c.head_dim / 8);
        for (int i = tid; i < n; i += kCopyThreads) dst[i] = src[i];
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
// finish commits lengths and releases pages.
constexpr int kMoveThreads = 256;

struct MoveLane {
    int32_t page_of[NVFP4_ATTN_MAX_ROWS];  // source: page id of path[j]'s slot, and the row in it
    int32_t row_of[NVFP4_ATTN_MAX_ROWS];
    int32_t to_page[NVFP4_ATTN_MAX_ROWS];
    int32_t to_row[NVFP4_ATTN_MAX_ROWS];
    int count;  // slots to look at, from `first` on; 0: none moves
    int first;  // the slots before it lie where they belong
    int good;
};

// Whether lane b's count and path can be committed (all threads of a CTA ask).
__device__ void read_lane(const nvfp4_cache& c, int b, const int32_t* count, const int32_t* path, int ld, int tid,
                          MoveLane& m)
{
    const int shift = __ffs(c.page_size) - 1;
    const int n = max(c.len[b], 0), k = count[b];
    if (tid == 0) {
        m.good = k >= 0 && (!path || k <= ld) && (int64_t)n + k <= (int64_t)c.max_pages << shift;
        m.count = 0;
        m.first = NVFP4_ATTN_MAX_ROWS;
    }
    __syncthreads();
    if (path && m.good && tid < k) {
        const int32_t* row = c.table + (int64_t)b * c.max_pages;
        const int s = path[(int64_t)b * ld + tid];
        const int before = tid ? path[(int64_t)b * ld + tid - 1] : -1;
        bool fine = s > before && s < NVFP4_ATTN_MAX_ROWS && (int64_t)n + s < (int64_t)c.max_pages << shift;
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
        if (!fine) atomicAnd(&m.good, 0);
    } else if (!path && m.good && k > 0) {
        // kept as they lie: the slots need pages
        const int32_t* row = c.table + (int64_t)b * c.max_pages;
        bool fine = true;
        for (int q = (n >> shift) + tid; q <= (n + k - 1) >> shift; q += blockDim.x)
            fine = fine && row[q] >= 0 && row[q] < c.pages;
        if (!fine) atomicAnd(&m.good, 0);
    }
    __syncthreads();
    if (tid == 0 && path && m.good) m.count = k;
    __syncthreads();
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
    // The last CTA commits, a warp per lane: every CTA has read lengths, paths
    // and tables by then, and left its lane's verdict in scratch.
    unsigned* counter = (unsigned*)c.scratch + 4 * c.lanes;
    if (tid == 0) {
        if (blockIdx.x == 0) c.scratch[4 * b + 3] = m.good;
        s_last = count_in(counter) == gridDim.x * gridDim.y - 1;
    }
    __syncthreads();
    if (!s_last) return;
    const int lane = tid & 31;
    for (int l = tid >> 5; l < c.lanes; l += kMoveThreads / 32) {
        if (!__ldcg(c.scratch + 4 * l + 3)) {
            if (lane == 0) atomicOr(&g_cache_status, kRefused);
            continue;
        }
        const int n = max(c.len[l], 0) + count[l];
        __syncwarp();
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
    NVFP4_CUDA_TRY(launch_pdl(reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, *cache, want, ok));
    NVFP4_CUDA_TRY(launch_pdl(page_copy_kernel, dim3((unsigned)(8 * sms)), dim3(kCopyThreads), 0, stream, *cache));
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
        const int64_t cap = (8 * sms + cache->lanes - 1) / cache->lanes;  // one wave of resident CTAs
        if (gx > cap) gx = cap;
        const dim3 grid = path ? dim3((unsigned)gx, (unsigned)cache->lanes) : dim3(1, (unsigned)cache->lanes);
        return launch_pdl(kernel, grid, dim3(kMoveThreads), 0, stream, *cache, count, path, ld_path);
    };
    NVFP4_CUDA_TRY(cache->head_dim == 64    ? launch(compact_kernel<64>, 64)
                   : cache->head_dim == 128 ? launch(compact_kernel<128>, 128)
                                            : launch(compact_kernel<256>, 256));
    return NVFP4_OK;
}
