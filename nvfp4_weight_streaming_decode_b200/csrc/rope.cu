// rope.cu -- rotary positions with several axes on the q/k/v projection's FP32
// output, and the append of its keys and values to the paged cache, in one
// pass: every value of y is read once and every bf16 result written once.
//
// A row's angles a_i = pos * f_i are formed and reduced to [-pi, pi] in 64 bits
// (n = rint(a / 2 pi), r = a - n 2 pi with 2 pi split in two doubles), because
// at position 10^6 a 32-bit product has lost the phase; sine and cosine of the
// reduced angle are 32-bit.  They are shared by all heads of the row, so a CTA
// computes the row's table once into shared memory and then streams its heads.
//
// Bound by memory for a prompt (8,193 rows of 40 + 2 x 8 heads of 128: 62 us, 5.7
// TB/s, 0.87 of the measured copy rate), by its chain of small loads for a round
// (8 rows of 15,360: 3.3 us; 64 rows of 32 heads of 256: 3.5 us).  Each result is
// rounded to bf16 once, the type the attention's products take.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"

namespace nvfp4 {

__device__ unsigned int g_rope_status;

namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
    nvfp4_cache c;
    nvfp4_rope_args a;
    int heads_per_cta;
};

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint4 r;
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    r.x = *reinterpret_cast<uint32_t*>(&h[0]);
    r.y = *reinterpret_cast<uint32_t*>(&h[1]);
    r.z = *reinterpret_cast<uint32_t*>(&h[2]);
    r.w = *reinterpret_cast<uint32_t*>(&h[3]);
    return r;
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// grid: (chunks of heads, rows).  A thread takes 16 values of a head at a time:
// 8 values and their 8 partners (halves), or 16 neighbours.
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p)
{
    __shared__ float2 turn[128];  // (cos, sin) per pair
    __shared__ int s_lane, s_slot;
    __shared__ int64_t s_dst;     // element offset of the row's slot in the layer, head 0; -1: none
    const nvfp4_cache& c = p.c;
    const nvfp4_rope_args& a = p.a;
    pdl_begin();
    const int tid = threadIdx.x, row = blockIdx.y;
    const int half = a.rot_dim / 2, D = c.head_dim;
    if (tid == 0) s_lane = -1;
    __syncthreads();
    if (tid < c.lanes) {
        int lo, hi;
        lane_rows(a.row_start, tid, a.rows, lo, hi);
        if (row >= lo && row < hi) {
            s_lane = tid;
            s_slot = row - lo;
        }
    }
    if (tid < half) {
        int axis = a.pair_axis ? a.pair_axis[tid] : 0;
        if (axis >= a.axes) axis = a.axes - 1;
        const double ang = (double)a.positions[axis * a.ldp + row] * a.inv_freq[tid];
        const double n = rint(ang * 0.15915494309189535);
        const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, ang));
        float sn, cs;
        sincosf((float)r, &sn, &cs);
        turn[tid] = make_float2(cs, sn);
    }
    __syncthreads();
    if (s_lane < 0) return;  // behind the last lane's rows
    if (tid == 0) {
        const int shift = __ffs(c.page_size) - 1;
        const int64_t slot = (int64_t)max(c.len[s_lane], 0) + s_slot;
        int64_t dst = -1;
        if (slot < (int64_t)c.max_pages << shift) {
            const int pg = c.table[(int64_t)s_lane * c.max_pages + (slot >> shift)];
            if (pg >= 0 && pg < c.pages && c.ref[pg] == 1)
                dst = (((int64_t)a.layer * c.pages + pg) * c.kv_heads * c.page_size + (slot & (c.page_size - 1))) * D;
        }
        if (dst < 0) atomicOr(&g_rope_status, 1u);
        s_dst = dst;
    }
    __syncthreads();
    const int64_t dst = s_dst;
    const int units = D / 16;
    const int heads = a.q_heads + 2 * c.kv_heads;
    const int h0 = blockIdx.x * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, heads);
    const float* y = a.y + (int64_t)row * a.ldy;
    for (int u = h0 * units + tid; u < h1 * units; u += kRopeThreads) {
        const int h = u / units, w = u % units;
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + c.kv_heads;
        const bool rotated = !is_v && w < half / 8;
        const bool halves = rotated && a.style == NVFP4_ROPE_HALVES;
        // the two runs of 8 values
        const int e0 = halves ? 8 * w : 16 * w;
        const int e1 = halves ? half + 8 * w : 16 * w + 8;
        // (a head's values past rot_dim are runs of 16 from rot_dim = 16 (half / 8) on)
        float x0[8], x1[8];
        load8(y + (int64_t)h * D + e0, x0);
        load8(y + (int64_t)h * D + e1, x1);
        if (rotated) {
            if (halves) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 t = turn[8 * w + i];
                    const float u0 = x0[i], u1 = x1[i];
                    x0[i] = u0 * t.x - u1 * t.y;
                    x1[i] = u1 * t.x + u0 * t.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 t = turn[8 * w + i];
                    float* z = i < 4 ? x0 + 2 * i : x1 + 2 * (i - 4);
                    const float u0 = z[0], u1 = z[1];
                    z[0] = u0 * t.x - u1 * t.y;
                    z[1] = u1 * t.x + u0 * t.y;
                }
            }
        }
        uint16_t* out;
        if (is_q) {
            out = (uint16_t*)a.q + (int64_t)row * a.ldq + (int64_t)h * D;
        } else {
            if (dst < 0) continue;
            const int kh = is_v ? h - a.q_heads - c.kv_heads : h - a.q_heads;
            out = (uint16_t*)(is_v ? c.v : c.k) + dst + (int64_t)kh * c.page_size * D;
        }
        *reinterpret_cast<uint4*>(out + e0) = pack8(x0);
        *reinterpret_cast<uint4*>(out + e1) = pack8(x1);
    }
}

}  // namespace

int read_and_clear_rope_status(unsigned* status)
{
    unsigned v = 0;
    NVFP4_CUDA_TRY(cudaDeviceSynchronize());
    NVFP4_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_rope_status, sizeof v));
    if (v != 0) {
        const unsigned zero = 0;
        NVFP4_CUDA_TRY(cudaMemcpyToSymbol(g_rope_status, &zero, sizeof zero));
    }
    *status = v;
    return NVFP4_OK;
}

int validate_rope(const nvfp4_rope_args* a)
{
    if (!a) return NVFP4_ERR_ARG;
    const nvfp4_cache* c = a->cache;
    const int st = check_cache(c);
    if (st != NVFP4_OK) return st;
    if (!a->y || !a->q || (a->rot_dim > 0 && (!a->positions || !a->inv_freq))) return NVFP4_ERR_ARG;
    if (a->style != NVFP4_ROPE_HALVES && a->style != NVFP4_ROPE_ADJACENT) return NVFP4_ERR_ARG;
    if (a->rows < 1 || a->rows > 65535 || (!a->row_start && a->rows > c->lanes)) return NVFP4_ERR_M;
    const int64_t D = c->head_dim;
    if (a->layer < 0 || a->layer >= c->layers || a->q_heads < 1 || a->q_heads > 8192 || a->q_heads % c->kv_heads ||
        a->rot_dim < 0 || a->rot_dim > D || a->rot_dim % 16 ||
        (a->rot_dim > 0 && (a->axes < 1 || a->axes > 4 || a->ldp < a->rows)) ||
        a->ldy < (a->q_heads + 2 * (int64_t)c->kv_heads) * D || a->ldq < a->q_heads * D ||
        a->ldy > ((int64_t)1 << 40) || a->ldq > ((int64_t)1 << 40))
        return NVFP4_ERR_SHAPE;
    if (!aligned16(a->y) || !aligned16(a->q) || (a->ldy & 3) || (a->ldq & 7) ||
        (((uintptr_t)a->row_start | (uintptr_t)a->positions) & 3) || ((uintptr_t)a->inv_freq & 7))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int launch_rope(const nvfp4_rope_args* a, cudaStream_t stream)
{
    int sms = 0;
    const int st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    RopeParams p = {};
    p.c = *a->cache;
    p.a = *a;
    const int heads = a->q_heads + 2 * p.c.kv_heads;
    // few rows: split the heads so that the grid covers the SMs about twice
    int per = heads * a->rows / (2 * sms);
    const int least = kRopeThreads * 16 / p.c.head_dim;  // heads that give every thread one unit
    p.heads_per_cta = per < least ? least : (per > heads ? heads : per);
    const dim3 grid((unsigned)((heads + p.heads_per_cta - 1) / p.heads_per_cta), (unsigned)a->rows);
    NVFP4_CUDA_TRY(launch_pdl(rope_append_kernel, grid, dim3(kRopeThreads), 0, stream, p));
    return NVFP4_OK;
}

}  // namespace nvfp4

extern "C" int nvfp4_rope_append(const nvfp4_rope_args* args, cudaStream_t stream)
{
    const int st = nvfp4::validate_rope(args);
    return st != NVFP4_OK ? st : nvfp4::launch_rope(args, stream);
}
