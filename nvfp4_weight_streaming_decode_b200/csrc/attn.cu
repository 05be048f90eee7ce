// attn.cu -- attention of decode rows and drafted trees over the paged cache.
//
// For a query row the scores over the visible slots pass through a softmax
// held as a running maximum and sum, so keys and values are read once:
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
// One CTA per (row, query head); each of its warps takes every fourth slot and
// the warps' states are joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"

namespace nvfp4 {

__device__ unsigned int g_attn_status;

namespace {

struct AttnParams {
    nvfp4_cache c;
    nvfp4_attn_args a;
};

template <int D>
__global__ void __launch_bounds__(128) attn_kernel(const AttnParams p)
{
    constexpr int kPer = D / 32;
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    const nvfp4_cache& c = p.c;
    const nvfp4_attn_args& a = p.a;
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, row = blockIdx.y;
    int b = -1, i = 0, n = 0;
    for (int l = 0; l < c.lanes; ++l) {
        int lo, hi;
        lane_rows(a.row_start, l, a.rows, lo, hi);
        if (row >= lo && row < hi) {
            b = l;
            i = row - lo;
            n = hi - lo;
            break;
        }
    }
    if (b < 0) return;
    const int shift = __ffs(c.page_size) - 1;
    const int len = max(c.len[b], 0);
    const uint64_t mask = a.mask ? a.mask[row] : (i >= 63 ? ~0ull : (2ull << i) - 1);
    const int kh = h / (a.q_heads / c.kv_heads);
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + (int64_t)row * a.ldq + (int64_t)h * D;
    float qr[kPer], o[kPer];
    for (int e = 0; e < kPer; ++e) {
        qr[e] = __bfloat162float(q[lane + 32 * e]) * a.scale;
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int64_t end = (int64_t)len + n;
    for (int64_t s = warp; s < end; s += 4) {
        if (s >= len && !((mask >> (s - len)) & 1)) continue;
        const int64_t col = s >> shift;
        const int pg = col < c.max_pages ? c.table[(int64_t)b * c.max_pages + col] : -1;
        if (pg < 0 || pg >= c.pages) {
            if (lane == 0) atomicOr(&g_attn_status, 1u);
            continue;
        }
        const int64_t at =
            ((((int64_t)a.layer * c.pages + pg) * c.kv_heads + kh) * c.page_size + (s & (c.page_size - 1))) * D;
        const __nv_bfloat16* k = (const __nv_bfloat16*)c.k + at;
        const __nv_bfloat16* v = (const __nv_bfloat16*)c.v + at;
        float x = 0.f;
        for (int e = 0; e < kPer; ++e) x += qr[e] * __bfloat162float(k[lane + 32 * e]);
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const float mn = fmaxf(m, x);
        const float w = x == -INFINITY ? 0.f : expf(x - mn), f = m == -INFINITY ? 0.f : expf(m - mn);
        l = l * f + w;
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * f + w * __bfloat162float(v[lane + 32 * e]);
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    for (int e = 0; e < kPer; ++e) s_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.f, f[4];
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < 4; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - top);
        sum += s_l[w] * f[w];
    }
    const bool any = !(sum == 0.f);
    for (int e = tid; e < D; e += 128) {
        float acc = 0.f;
        for (int w = 0; w < 4; ++w)
            if (f[w] != 0.f) acc += s_o[w][e] * f[w];
        ((__nv_bfloat16*)a.out)[(int64_t)row * a.ldo + (int64_t)h * D + e] = __float2bfloat16(any ? acc / sum : 0.f);
    }
    if (tid == 0 && a.lse) a.lse[(int64_t)row * a.q_heads + h] = any ? top + logf(sum) : -INFINITY;
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

static size_t attn_workspace(int rows, int q_heads, int kv_heads, int head_dim, int sms)
{
    (void)rows;
    (void)q_heads;
    (void)kv_heads;
    (void)head_dim;
    (void)sms;
    return 16;
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
        a->ldq > ((int64_t)1 << 40) || a->ldo > ((int64_t)1 << 40))
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
    const int st = sm_count(&sms);
    if (st != NVFP4_OK) return st;
    if (a->workspace_bytes < attn_workspace(a->rows, a->q_heads, p.c.kv_heads, p.c.head_dim, sms))
        return NVFP4_ERR_SCRATCH;
    const dim3 grid((unsigned)a->q_heads, (unsigned)a->rows);
    NVFP4_CUDA_TRY(p.c.head_dim == 64    ? launch_pdl(attn_kernel<64>, grid, dim3(128), 0, stream, p)
                   : p.c.head_dim == 128 ? launch_pdl(attn_kernel<128>, grid, dim3(128), 0, stream, p)
                                         : launch_pdl(attn_kernel<256>, grid, dim3(128), 0, stream, p));
    return NVFP4_OK;
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
    *bytes = nvfp4::attn_workspace(rows, q_heads, kv_heads, head_dim, sm_count);
    return NVFP4_OK;
}

extern "C" int nvfp4_attn_tree(const nvfp4_attn_args* args, cudaStream_t stream)
{
    const int st = nvfp4::validate_attn(args);
    return st != NVFP4_OK ? st : nvfp4::launch_attn(args, stream);
}
