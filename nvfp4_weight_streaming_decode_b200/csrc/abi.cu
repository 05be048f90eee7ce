// abi.cu -- status codes, argument checks and small queries of the C ABI.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "layout.cuh"

namespace nvfp4 {

static thread_local int t_last_cuda_error = 0;

int fail_cuda(cudaError_t e)
{
    t_last_cuda_error = (int)e;
    cudaGetLastError();  // clear a sticky-free error so the next call starts clean
    return NVFP4_ERR_CUDA;
}

int check_m(int M) { return (M >= 1 && M <= kMaxM) ? NVFP4_OK : NVFP4_ERR_M; }

int check_shape(int64_t N, int64_t K)
{
    if (N < 1 || K < 16 || (K % 16) != 0) return NVFP4_ERR_SHAPE;
    // keep every byte offset and element index well inside int64
    if (N > ((int64_t)1 << 31) || K > ((int64_t)1 << 31) || (N / kTileN + 1) * (K / kChunkK + 1) > ((int64_t)1 << 40))
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

int check_cache(const nvfp4_cache* c)
{
    if (!c || !c->k || !c->v || !c->table || !c->len || !c->ref || !c->scratch) return NVFP4_ERR_ARG;
    const bool page_ok = c->page_size >= 16 && c->page_size <= 256 && (c->page_size & (c->page_size - 1)) == 0;
    const bool dim_ok = c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256;
    if (!page_ok || !dim_ok || c->lanes < 1 || c->lanes > NVFP4_CACHE_MAX_LANES || c->kv_heads < 1 ||
        c->kv_heads > 256 || c->layers < 1 || c->pages < 1 || c->pages > (1 << 24) || c->max_pages < 1 ||
        c->max_pages > (1 << 20) || (int64_t)c->max_pages * c->page_size > ((int64_t)1 << 30) ||
        (int64_t)c->pages * c->kv_heads * c->page_size >= ((int64_t)1 << 32))
        return NVFP4_ERR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v)) return NVFP4_ERR_ALIGN;
    if ((((uintptr_t)c->table | (uintptr_t)c->len | (uintptr_t)c->ref | (uintptr_t)c->scratch) & 3) != 0)
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int sm_count(int* out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    NVFP4_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return NVFP4_ERR_ARG;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        NVFP4_CUDA_TRY(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
        known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return NVFP4_OK;
}

Geometry geometry(int64_t N, int64_t K)
{
    Geometry g;
    g.n_tiles = (N + kTileN - 1) / kTileN;
    g.k_chunks = (K + kChunkK - 1) / kChunkK;
    g.units = g.n_tiles * g.k_chunks;
    return g;
}

}  // namespace nvfp4

extern "C" const char* nvfp4_status_string(int status)
{
    switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_ARG: return "invalid argument (NULL pointer, bad kind or count)";
    case NVFP4_ERR_M: return "M out of range for this entry point (1..8; nvfp4_gemm_decode also takes 9..64)";
    case NVFP4_ERR_SHAPE: return "bad shape: need N >= 1, K >= 16, K % 16 == 0";
    case NVFP4_ERR_ALIGN: return "device pointer not 16-byte aligned";
    case NVFP4_ERR_BAD_SCALE: return "scale plane holds an E4M3 NaN code (0x7F or 0xFF)";
    case NVFP4_ERR_CUDA: return "CUDA runtime error (see nvfp4_last_cuda_error)";
    case NVFP4_ERR_CAPTURE: return "first use of the device inside a stream capture";
    case NVFP4_ERR_DEVICE: return "a kernel's bounded wait gave up (see nvfp4_device_status)";
    case NVFP4_ERR_SCRATCH: return "needs more scratch than the no-alloc entry point's static array holds";
    default: return "unknown status";
    }
}

extern "C" int nvfp4_last_cuda_error(void) { return nvfp4::t_last_cuda_error; }

extern "C" int nvfp4_device_status(void)
{
    int v = 0;
    int st = nvfp4::read_and_clear_device_status(&v);
    if (st != NVFP4_OK) return st;
    unsigned vv = 0;
    st = nvfp4::read_and_clear_verify_status(&vv);
    if (st != NVFP4_OK) return st;
    unsigned vg = 0;
    st = nvfp4::read_and_clear_grouped_status(&vg);
    if (st != NVFP4_OK) return st;
    unsigned vc = 0, vr = 0, va = 0;
    st = nvfp4::read_and_clear_cache_status(&vc);
    if (st == NVFP4_OK) st = nvfp4::read_and_clear_rope_status(&vr);
    if (st == NVFP4_OK) st = nvfp4::read_and_clear_attn_status(&va);
    if (st != NVFP4_OK) return st;
    // verify kernel: 8 = a streaming warp gave up, 16 = its MMA thread did;
    // grouped kernel: 32 = an invalid route, 64 = a bounded wait gave up;
    // cache kernels: 128 = refused content, 256 = too few pages, 512 = an attention wait gave up
    return v | (int)(vv << 3) | (int)(vg << 5) | (int)((vc | vr | va) << 7);
}

extern "C" int nvfp4_version(void) { return 100; }
