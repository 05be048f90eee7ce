// beam.cu -- beam selection over the head's logits: log-softmax of every row,
// the running scores added, and the best candidates of each group of beams,
// in one launch that reads the logits once.
//
// Within a row candidates rank as their logits do, so no row needs more than
// its `beams` largest logits, and its normaliser: row m is cut into S slices,
// one CTA each, which reads its slice once for the maximum and the sum of
// exp(x - max) -- running, a thread at a time -- and then again, from L2 and only
// the threads that have one, for its `beams` best (value, index).  The last CTA of a group
// to finish (counter, acquire/release) joins the normalisers in slice order and
// ranks the group's beams * S * beams candidates by 64-bit scores.
//
// Selecting k of n values, in a slice and in the merge alike: the k-th largest
// of a warp's 32 thread maxima bounds the answer from below (k different
// elements reach it); the highest of the warps' bounds leaves few
// elements above it (some 60 for k = 8), so one more pass collects those and
// each counts how many rank before it.  (k > 32: the k-th of all maxima.)  When ties push more than
// kListCap elements over the bound, k rounds of a block-wide maximum decide.
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"

// Bound by its chain of steps (read, join warps, collect, rank, count in, merge:
// 24,000 cycles), not by the 39 MB that 64 rows of 151,936 are: 16.4 us, 0.37 of
// the measured copy rate; 8 rows 13 us, 4 rows of 1,000 7.7 us.
namespace nvfp4 {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kChunk = 16;                              // logits a thread takes at a time
constexpr int kStride = 4 * kBeamThreads;               // columns of one round of float4
constexpr int kParts = 16;                              // of a thread's columns, for the second reading
constexpr int kCtasPerSm = 3;
constexpr int kWarps = kBeamThreads / 32;
constexpr int kListCap = 512;
constexpr int kHeld = 8;                                // candidates a merging thread holds
constexpr int kMaxRows = NVFP4_TOPK_MAX_ROWS;

struct alignas(16) SlicePart {
    double sum;  // of exp(x - top)
    float top;   // -inf: the slice has nothing finite
    float unused;
};

struct BeamParams {
    const float* logits;
    long long ldv;
    int V, groups, beams, S, slice;
    const float* scores;
    const uint8_t* finished;
    int eos;
    float* scores_out;
    int32_t *parent, *token;
    uint8_t* finished_out;
    SlicePart* part;    // [rows][S]
    float* cand_x;      // [rows][S][beams]
    int32_t* cand_v;    // their columns, -1: none
    unsigned* counters; // [groups]
};

// 2^x by the exponential unit, within about 2^-22 of itself.  With x = (logit -
// maximum) log2(e) rounded, a term is off by 2^-24 (1 + |x|) more: those far
// below the maximum, where that grows, hardly count in the sum.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (a - ref) log2(e) and (b - ref) log2(e), as pairs.
__device__ __forceinline__ float2 scaled(float a, float b, float ref)
{
    float2 r;
    asm("{\n .reg .b64 v, m, l;\n mov.b64 v, {%2, %3};\n mov.b64 m, {%4, %4};\n mov.b64 l, {%5, %5};\n"
        " add.rn.f32x2 v, v, m;\n mul.rn.f32x2 v, v, l;\n mov.b64 {%0, %1}, v;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a), "f"(b), "f"(-ref), "f"(1.4426950408889634f));
    return r;
}

// An order on (value, place): the larger value first, equal ones by lower place.
template <class T>
__device__ __forceinline__ bool before(T a, uint32_t ia, T b, uint32_t ib)
{
    return a > b || (a == b && ia < ib);
}

template <class T>
struct ListShared {
    T top[kBeamThreads];
    T val[kListCap];
    uint32_t place[kListCap];
    T wval[kWarps];
    uint32_t wplace[kWarps];
    T bound;
    int count;
};

// The value as bits that order as it does.
__device__ __forceinline__ uint32_t order_bits(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A warp's bound: the k-th largest (k <= 32) of its lanes' values goes to *out.
__device__ __forceinline__ void warp_kth(int k, float mine, int lane, float* out)
{
    // k - 1 times the largest leaves (one lane of it); the largest of the rest
    uint32_t key = order_bits(mine);
    for (int i = 1; i < k; ++i) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, key);
        if (lane == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) key = 0u;
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    if (lane == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) *out = mine;
}
__device__ __forceinline__ void warp_kth(int k, double mine, int lane, double* out)
{
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const double o = __shfl_sync(0xffffffffu, mine, i);
        rank += o > mine || (o == mine && i < lane);
    }
    if (rank == k - 1) *out = mine;
}

// The k best of the block's elements under `before`, to emit(rank, value,
// place).  above(bound, f) calls f(value, place) for the calling thread's
// elements from `bound` up, each(f) for all; both leave out -inf and NaN.  `mine`
// is the thread's largest element, or `none`.  For k <= 32 the callers have put
// warp_kth of it into sh.top[warp] and zeroed sh.count before a barrier.
// Returns how many there are, at most k.
template <class T, class Above, class Each, class Emit>
__device__ int block_best(int k, T mine, T none, Above above, Each each, Emit emit, ListShared<T>& sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    T bound;  // none: too few threads hold elements, take all
    if (k <= 32) {
        bound = sh.top[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) bound = sh.top[w] > bound ? sh.top[w] : bound;
    } else {
        __syncthreads();
        sh.top[tid] = mine;
        if (tid == 0) sh.bound = none;
        __syncthreads();
        int rank = 0;
        for (int i = 0; i < kBeamThreads; ++i) {
            const T o = sh.top[i];
            rank += o > mine || (o == mine && i < tid);
        }
        if (rank == k - 1) sh.bound = mine;
        __syncthreads();
        bound = sh.bound;
    }
    if (mine >= bound)
        above(bound, [&](T v, uint32_t place) {
            const int pos = atomicAdd(&sh.count, 1);
            if (pos < kListCap) {
                sh.val[pos] = v;
                sh.place[pos] = place;
            }
        });
    __syncthreads();
    const int n = sh.count;
    if (n <= kListCap) {
        // eight threads count for one element
        for (int i0 = 0; i0 < n; i0 += kBeamThreads / 8) {
            const int i = i0 + (tid >> 3);
            const bool in = i < n;
            const T v = in ? sh.val[i] : none;
            const uint32_t p = in ? sh.place[i] : 0u;
            int r = 0;
#pragma unroll 4
            for (int j = tid & 7; j < n; j += 8) r += before(sh.val[j], sh.place[j], v, p);
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            r += __shfl_xor_sync(0xffffffffu, r, 4);
            if (in && (tid & 7) == 0 && r < k) emit(r, v, p);
        }
        __syncthreads();
        return n < k ? n : k;
    }
    // many ties: one winner a round, each below the one before
    T last = none;
    uint32_t lastp = 0;
    for (int r = 0; r < k; ++r) {
        T bv = none;
        uint32_t bp = 0xFFFFFFFFu;
        each([&](T v, uint32_t place) {
            if ((r == 0 || before(last, lastp, v, place)) && before(v, place, bv, bp)) {
                bv = v;
                bp = place;
            }
        });
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const T ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const uint32_t op = __shfl_xor_sync(0xffffffffu, bp, off);
            if (before(ov, op, bv, bp)) {
                bv = ov;
                bp = op;
            }
        }
        if (lane == 0) {
            sh.wval[warp] = bv;
            sh.wplace[warp] = bp;
        }
        __syncthreads();
        bv = sh.wval[0];
        bp = sh.wplace[0];
        for (int w = 1; w < kWarps; ++w)
            if (before(sh.wval[w], sh.wplace[w], bv, bp)) {
                bv = sh.wval[w];
                bp = sh.wplace[w];
            }
        __syncthreads();
        if (tid == 0) emit(r, bv, bp);  // n > kListCap >= k: a round never comes up empty
        last = bv;
        lastp = bp;
    }
    __syncthreads();
    return k;
}

__global__ void __launch_bounds__(kBeamThreads, kCtasPerSm) beam_kernel(const BeamParams p)
{
    __shared__ union {
        ListShared<float> f;
        ListShared<double> d;
    } sh;
    __shared__ float s_part[kParts][kBeamThreads];
    __shared__ float s_w[kWarps];
    __shared__ double s_d[kWarps];
    __shared__ double s_lse[kMaxRows], s_cum[kMaxRows];
    __shared__ bool s_over[kMaxRows];
    __shared__ int s_last;
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x, m = blockIdx.y, g = m / p.beams;
    const float kNone = __int_as_float(0xff800000);
    const bool done = p.finished && p.finished[m] != 0;
    const long long at = (long long)m * p.S + s;
    if (!done) {
        // 1. The thread's running maximum and sum of exp(x - maximum) over its
        // columns lo + 4 tid + 1024 i + (0..3): once through memory, a chunk of
        // loads in flight at a time.
        const int lo = s * p.slice, n = min(p.slice, p.V - lo);
        const float* x = p.logits + (long long)m * p.ldv + lo;
        auto four = [&](int q) {  // columns q .. q + 3 of the slice, -inf behind it
            float4 v = make_float4(kNone, kNone, kNone, kNone);
            if (q + 4 <= n) {
                v = __ldg(reinterpret_cast<const float4*>(x + q));
            } else if (q < n) {
                v.x = x[q];
                if (q + 1 < n) v.y = x[q + 1];
                if (q + 2 < n) v.z = x[q + 2];
            }
            return v;
        };
        // The maxima of up to kParts parts of the columns stay in shared memory: the
        // selection reads only parts that hold something for it again.
        const int rounds = (n + kChunk / 4 * kStride - 1) / (kChunk / 4 * kStride), per_part = (rounds + kParts - 1) / kParts;
        float mine = kNone, acc = 0.f, part_top = kNone;
        for (int c = 0; c < rounds; ++c) {
            const int q0 = 4 * tid + c * (kChunk / 4 * kStride);
            float4 v[kChunk / 4];
#pragma unroll
            for (int i = 0; i < kChunk / 4; ++i) v[i] = four(q0 + i * kStride);
            float here = kNone;
#pragma unroll
            for (int i = 0; i < kChunk / 4; ++i)
                here = fmaxf(fmaxf(fmaxf(here, v[i].x), fmaxf(v[i].y, v[i].z)), v[i].w);
            part_top = fmaxf(part_top, here);
            if ((c + 1) % per_part == 0 || c + 1 == rounds) {
                s_part[c / per_part][tid] = part_top;
                part_top = kNone;
            }
            const float top = fmaxf(mine, here);
            const float ref = top == kNone ? 0.f : top;  // nothing but -inf so far (or NaN, which the sum keeps)
            float e0 = 0.f, e1 = 0.f;
#pragma unroll
            for (int i = 0; i < kChunk / 4; ++i) {
                // (x - maximum) log2(e), two at a time
                const float2 a = scaled(v[i].x, v[i].y, ref), b = scaled(v[i].z, v[i].w, ref);
                e0 += exp2_fast(a.x) + exp2_fast(a.y);
                e1 += exp2_fast(b.x) + exp2_fast(b.y);
            }
            acc = acc * (mine == top ? 1.f : expf(mine - top)) + (e0 + e1);
            mine = top;
        }
        // 2. the warps' maxima, sums and bounds for the selection; 64 bits from here
        // on.  The joined normaliser is mostly good to 2^-22 or better (the exponentials'
        // own error averages out) and never worse than 2^-16: 43 rounds of a thread at
        // the most, each a sum and perhaps a rescale, and arguments of up to 20 in log2.
        float top = mine;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        double sum = (double)acc * (double)(mine == top ? 1.f : expf(mine - top));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
            s_w[warp] = top;
            s_d[warp] = sum;
        }
        if (tid == 0) sh.f.count = 0;
        if (p.beams <= 32) warp_kth(p.beams, mine, lane, &sh.f.top[warp]);
        __syncthreads();
        if (warp == kWarps - 1) {  // the slice's, from the warps'
            const float wt = lane < kWarps ? s_w[lane] : kNone;
            double ws = lane < kWarps ? s_d[lane] : 0.0;
            float all = wt;
#pragma unroll
            for (int off = kWarps / 2; off > 0; off >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, off));
            ws *= (double)(wt == all ? 1.f : expf(wt - all));
#pragma unroll
            for (int off = kWarps / 2; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
            if (lane == 0) {
                p.part[at].sum = ws;
                p.part[at].top = all;
            }
        }
        // 3. the slice's best
        float* cx = p.cand_x + at * p.beams;
        int32_t* cv = p.cand_v + at * p.beams;
        const int got = block_best<float>(
            p.beams, mine, kNone,
            [&](float bound, auto f) {
                bound = fmaxf(bound, -FLT_MAX);  // never -inf
                // this thread has one: through its parts that do again (L2 holds them)
                // -- each lane its own next one, so that a warp waits for memory about once
                uint32_t todo = 0;
                for (int c = 0; c * per_part < rounds; ++c) todo |= s_part[c][tid] >= bound ? 1u << c : 0u;
                for (int c = 0, end = 0; todo || c < end; ++c) {
                    if (c >= end) {
                        const int part = __ffs(todo) - 1;
                        todo &= todo - 1;
                        c = part * per_part;
                        end = min(c + per_part, rounds);
                    }
                    const int q0 = 4 * tid + c * (kChunk / 4 * kStride);
                    float4 v[kChunk / 4];
#pragma unroll
                    for (int i = 0; i < kChunk / 4; ++i) v[i] = four(q0 + i * kStride);
                    uint32_t hits = 0;
#pragma unroll
                    for (int i = 0; i < kChunk / 4; ++i)
                        hits |= (v[i].x >= bound ? 1u << 4 * i : 0u) | (v[i].y >= bound ? 2u << 4 * i : 0u) |
                                (v[i].z >= bound ? 4u << 4 * i : 0u) | (v[i].w >= bound ? 8u << 4 * i : 0u);
                    for (; hits; hits &= hits - 1) {  // (each lane its own next hit, for the same reason)
                        const int i = __ffs(hits) - 1, q = q0 + (i >> 2) * kStride + (i & 3);
                        f(__ldg(x + q), (uint32_t)(lo + q));
                    }
                }
            },
            [&](auto f) {
                for (int q = tid; q < n; q += kBeamThreads) {
                    const float v = x[q];
                    if (v > kNone) f(v, (uint32_t)(lo + q));
                }
            },
            [&](int rank, float v, uint32_t place) {
                cx[rank] = v;
                cv[rank] = (int32_t)place;
            },
            sh.f);
        if (tid >= got && tid < p.beams) cv[tid] = -1;
    }
    // 4. the group's last CTA merges
    __syncthreads();
    if (tid == 0) s_last = count_in(p.counters + g) == (unsigned)(p.beams * p.S - 1);
    __syncthreads();
    if (!s_last) return;
    // Candidate i of the group is place q = i % per of row w = i / per.  Up to
    // kHeld per thread are fetched at once, before the normalisers they need.
    const int per = p.S * p.beams, n = p.beams * per;
    const bool held = n <= kHeld * kBeamThreads;
    float hx[kHeld];
    int hv[kHeld];
    const long long cells = (long long)g * p.beams * per;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = tid + j * kBeamThreads;
        hv[j] = -1;
        if (held && i < n) {
            hv[j] = __ldcg(p.cand_v + cells + i);
            hx[j] = __ldcg(p.cand_x + cells + i);
        }
    }
    if (tid == 0) sh.d.count = 0;
    for (int w = warp; w < p.beams; w += kWarps) {
        const int row = g * p.beams + w;
        const bool over = p.finished && p.finished[row] != 0;
        double norm = 0.0;
        if (!over) {
            // joined in lane order, two slices a lane held, any further ones in turn
            const float4* part = reinterpret_cast<const float4*>(p.part + (long long)row * p.S);
            const float4 none4 = make_float4(0.f, 0.f, kNone, 0.f);
            const float4 q0 = lane < p.S ? __ldcg(part + lane) : none4;
            const float4 q1 = lane + 32 < p.S ? __ldcg(part + lane + 32) : none4;
            float top = fmaxf(q0.z, q1.z);
            for (int i = lane + 64; i < p.S; i += 32) top = fmaxf(top, __ldcg(part + i).z);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            auto term = [&](const float4& q) {
                return __hiloint2double(__float_as_int(q.y), __float_as_int(q.x)) * (double)expf(q.z - top);
            };
            double sum = lane < p.S ? term(q0) : 0.0;
            if (lane + 32 < p.S) sum += term(q1);
            for (int i = lane + 64; i < p.S; i += 32) sum += term(__ldcg(part + i));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            norm = (double)top + log(sum);
        }
        if (lane == 0) {
            s_lse[w] = norm;
            s_cum[w] = (double)p.scores[row];
            s_over[w] = over;
        }
    }
    __syncthreads();
    const double dnone = -INFINITY;
    // its 64-bit score (none: not a candidate) and w * V + v
    auto cand = [&](int i, float x, int v, double& key, uint32_t& place) {
        const int w = i / per;
        const bool over = s_over[w];
        if (over) v = i == w * per ? p.eos : -1;
        place = (uint32_t)w * (uint32_t)p.V + (uint32_t)(v < 0 ? 0 : v);
        key = over ? s_cum[w] : s_cum[w] + ((double)x - s_lse[w]);
        if (v < 0 || !(key > dnone)) key = dnone;  // NaN too
    };
    double hk[kHeld];
    uint32_t hp[kHeld];
    double mine = dnone;
    if (held) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            hk[j] = dnone;
            hp[j] = 0u;
            const int i = tid + j * kBeamThreads;
            if (i < n) cand(i, hx[j], hv[j], hk[j], hp[j]);
            mine = fmax(mine, hk[j]);
        }
    }
    auto each_cand = [&](auto f) {
        if (held) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (hk[j] > dnone) f(hk[j], hp[j]);
        } else {
            for (int i = tid; i < n; i += kBeamThreads) {
                double key;
                uint32_t place;
                cand(i, __ldcg(p.cand_x + cells + i), __ldcg(p.cand_v + cells + i), key, place);
                if (key > dnone) f(key, place);
            }
        }
    };
    if (!held) each_cand([&](double key, uint32_t) { mine = fmax(mine, key); });
    if (p.beams <= 32) warp_kth(p.beams, mine, lane, &sh.d.top[warp]);
    __syncthreads();
    const int o = g * p.beams;
    __shared__ float o_score[kMaxRows];
    __shared__ int o_parent[kMaxRows], o_token[kMaxRows], o_done[kMaxRows];
    const int got = block_best<double>(
        p.beams, mine, dnone,
        [&](double bound, auto f) {
            each_cand([&](double key, uint32_t place) {
                if (key >= bound) f(key, place);
            });
        },
        each_cand,
        [&](int rank, double key, uint32_t place) {
            const int w = (int)(place / (uint32_t)p.V), v = (int)(place - (uint32_t)w * (uint32_t)p.V);
            o_score[rank] = (float)key;
            o_parent[rank] = o + w;
            o_token[rank] = v;
            o_done[rank] = v == p.eos || (p.finished && p.finished[o + w] != 0);
        },
        sh.d);
    // scores and finished may be the outputs' own memory: written when all is read
    if (tid < p.beams) {
        const bool real = tid < got;
        p.scores_out[o + tid] = real ? o_score[tid] : kNone;
        p.parent[o + tid] = real ? o_parent[tid] : -1;
        p.token[o + tid] = real ? o_token[tid] : -1;
        if (p.finished_out) p.finished_out[o + tid] = real ? (uint8_t)o_done[tid] : 0;
    }
    if (tid == 0) p.counters[g] = 0u;
}

struct BeamSplit {
    int S, slice;
    size_t part, x, v, counters, bytes;  // offsets into the workspace
};

int beam_split(int groups, int beams, int64_t V, int sms, BeamSplit* b)
{
    if (groups < 1 || beams < 1 || groups > kMaxRows || beams > kMaxRows || groups * beams > kMaxRows)
        return NVFP4_ERR_M;
    if (V < 1 || V > (1 << 20)) return NVFP4_ERR_SHAPE;
    const int rows = groups * beams;
    // One turn of the GPU at three CTAs an SM (two to four measure the same), slices of at least 2048 logits, and
    // where it costs no more than three quarters of the CTAs, few enough
    // candidates for the merge to hold in registers (beyond, it fetches them
    // three times).
    int64_t S = (int64_t)kCtasPerSm * sms / rows;
    const int64_t most = (V + 2047) / 2048, held = kHeld * kBeamThreads / (beams * beams);
    if (S > most) S = most;
    if (S > held) S = held > (S + 3) / 4 ? held : (S + 3) / 4;
    if (S < 1) S = 1;
    int64_t slice = (V + S - 1) / S;
    slice = (slice + 3) / 4 * 4;
    b->S = (int)((V + slice - 1) / slice);
    b->slice = (int)slice;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t cells = (size_t)rows * b->S;
    b->counters = 0;
    b->part = up(sizeof(unsigned) * kMaxRows);
    b->x = b->part + up(cells * sizeof(SlicePart));
    b->v = b->x + up(cells * beams * sizeof(float));
    b->bytes = b->v + up(cells * beams * sizeof(int32_t));
    return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int nvfp4_beam_select_workspace(int groups, int beams, int64_t V, int sm_count, size_t* bytes)
{
    if (!bytes || sm_count < 1) return NVFP4_ERR_ARG;
    BeamSplit b;
    const int st = beam_split(groups, beams, V, sm_count, &b);
    if (st == NVFP4_OK) *bytes = b.bytes;
    return st;
}

extern "C" int nvfp4_beam_select(const float* logits, int groups, int beams, int64_t V, int64_t ldv,
                                 const float* scores, const uint8_t* finished, int eos, float* scores_out,
                                 int32_t* parent, int32_t* token, uint8_t* finished_out, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream)
{
    if (!logits || !scores || !scores_out || !parent || !token || !workspace) return NVFP4_ERR_ARG;
    BeamSplit b;
    int st = beam_split(groups, beams, V, 1, &b);  // the limits, before any CUDA call
    if (st != NVFP4_OK) return st;
    if (ldv < V || ldv > ((int64_t)1 << 40) || (finished && (eos < 0 || eos >= V))) return NVFP4_ERR_SHAPE;
    if (!aligned16(logits) || (ldv & 3) || !aligned16(workspace) ||
        (((uintptr_t)scores | (uintptr_t)scores_out | (uintptr_t)parent | (uintptr_t)token) & 3))
        return NVFP4_ERR_ALIGN;
    int sms = 0;
    st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    beam_split(groups, beams, V, sms, &b);
    if (workspace_bytes < b.bytes) return NVFP4_ERR_SCRATCH;
    BeamParams p;
    p.logits = logits;
    p.ldv = ldv;
    p.V = (int)V;
    p.groups = groups;
    p.beams = beams;
    p.S = b.S;
    p.slice = b.slice;
    p.scores = scores;
    p.finished = finished;
    p.eos = eos;
    p.scores_out = scores_out;
    p.parent = parent;
    p.token = token;
    p.finished_out = finished_out;
    uint8_t* w = (uint8_t*)workspace;
    p.counters = (unsigned*)(w + b.counters);
    p.part = (SlicePart*)(w + b.part);
    p.cand_x = (float*)(w + b.x);
    p.cand_v = (int32_t*)(w + b.v);
    NVFP4_CUDA_TRY(launch_pdl(beam_kernel, dim3((unsigned)b.S, (unsigned)(groups * beams)), dim3(kBeamThreads), 0,
                              stream, p));
    return NVFP4_OK;
}
