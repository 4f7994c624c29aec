// paged_attention.cu -- attention of one new token per sequence over a paged key-value cache: moe_paged_attention.
#include "common.cuh"
#include "paged_cache.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int PA_WARPS = 8;

struct AttnArgs {
    const __nv_bfloat16* q;
    long long q_stride;
    int B, q_heads, M, window;
    CachePools c;
    const int32_t* table;
    const int32_t* lengths;
    float scale;
    __nv_bfloat16* out;
    float* lse;
};

// One element of a row of the cache.
template <bool FP8>
__device__ __forceinline__ float element(const void* pool, const uint8_t* scales, long long line, int dim, int d) {
    if (!FP8) return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[line * dim + d]);
    return e4m3_value(static_cast<const uint8_t*>(pool)[line * dim + d]) * e8m0_value(scales[line * (dim / 32) + d / 32]);
}

// A block per sequence and query head; its warps take the positions in turn, a lane every 32nd element.
template <bool FP8>
__global__ void __launch_bounds__(32 * PA_WARPS) attention_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float part[PA_WARPS][MOE_CACHE_MAX_DIM];
    __shared__ float part_m[PA_WARPS], part_l[PA_WARPS];
    const int h = blockIdx.x, b = blockIdx.y, dim = a.c.dim, lane = lane_id(), warp = threadIdx.x / 32;
    const int kv = h / (a.q_heads / a.c.heads);
    int n = a.lengths[b];
    if (n > (long long)a.M * a.c.page_size) {
        n = a.M * a.c.page_size;
        if (threadIdx.x == 0) raise_device_error(MOE_DEVERR_BAD_ID);
    }
    const int first = a.window > 0 && n > a.window ? n - a.window : 0;
    float q[8], acc[8], m = -INFINITY, l = 0.0f;
    for (int i = 0; i < 8; i++) {
        const int d = lane + 32 * i;
        q[i] = d < dim ? __bfloat162float(a.q[b * a.q_stride + (long long)h * dim + d]) * a.scale : 0.0f;
        acc[i] = 0.0f;
    }
    for (int j = first + warp; j < n; j += PA_WARPS) {
        const int page = a.table[(long long)b * a.M + j / a.c.page_size];
        if ((unsigned)page >= (unsigned)a.c.pages) {
            if (lane == 0) raise_device_error(MOE_DEVERR_BAD_ID);
            continue;
        }
        const long long line = ((long long)page * a.c.heads + kv) * a.c.page_size + j % a.c.page_size;
        float s = 0.0f;
        for (int i = 0; i < 8; i++)
            if (lane + 32 * i < dim) s += q[i] * element<FP8>(a.c.k, a.c.k_scales, line, dim, lane + 32 * i);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
        const float top = fmaxf(m, s), keep = m == -INFINITY ? 0.0f : expf(m - top), p = expf(s - top);
        m = top;
        l = l * keep + p;
        for (int i = 0; i < 8; i++)
            if (lane + 32 * i < dim) acc[i] = acc[i] * keep + p * element<FP8>(a.c.v, a.c.v_scales, line, dim, lane + 32 * i);
    }
    for (int i = 0; i < 8; i++) part[warp][lane + 32 * i] = acc[i];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < PA_WARPS; w++) top = fmaxf(top, part_m[w]);
    for (int w = 0; w < PA_WARPS; w++)
        if (part_l[w] != 0.0f) total += part_l[w] * expf(part_m[w] - top);
    const long long o = (long long)b * a.q_heads + h;
    for (int d = threadIdx.x; d < dim; d += 32 * PA_WARPS) {
        float v = 0.0f;
        for (int w = 0; w < PA_WARPS; w++)
            if (part_l[w] != 0.0f) v += part[w][d] * expf(part_m[w] - top);
        a.out[o * dim + d] = __float2bfloat16_rn(total != 0.0f ? v / total : 0.0f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[o] = total != 0.0f ? top + logf(total) : -INFINITY;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_paged_attention_workspace_size(int B, int q_heads, int heads, int dim) {
    if (B < 0 || B > 65535 || heads < 1 || q_heads < 1 || q_heads % heads || dim < 1 || dim > MOE_CACHE_MAX_DIM) return 0;
    return 256;
}

extern "C" moe_status moe_paged_attention(const void* q, long long q_stride, int B, int q_heads, const void* k_pages,
                                          const uint8_t* k_scales, const void* v_pages, const uint8_t* v_scales,
                                          moe_dtype dtype, int pages, int heads, int page_size, int dim,
                                          const int32_t* table, int M, const int32_t* lengths, float scale, int window,
                                          void* out, float* lse, void* workspace, size_t workspace_bytes,
                                          moe_stream_t stream) {
    using namespace moe;
    const CachePools c = {const_cast<void*>(k_pages), const_cast<void*>(v_pages), const_cast<uint8_t*>(k_scales),
                          const_cast<uint8_t*>(v_scales), pages, heads, page_size, dim};
    if (B < 0 || q_heads < 1 || window < 0 || !isfinite(scale) || heads < 1 || q_heads % heads) return MOE_ERR_INVALID_ARG;
    const moe_status st = moe_host::check_cache(c, dtype, M);
    if (st != MOE_OK) return st;
    if (B > 65535 || q_heads / heads > 1024) return MOE_ERR_UNSUPPORTED;
    if (B > 0 && (!q || !table || !lengths || !out)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_paged_attention_workspace_size(B, q_heads, heads, dim)) return MOE_ERR_WORKSPACE;
    if (q_stride % 8 || !moe_host::aligned(q, 16) || !moe_host::aligned(out, 16) || !moe_host::aligned(lse, 4) ||
        !moe_host::aligned(table, 4) || !moe_host::aligned(lengths, 4) || !moe_host::aligned(workspace, 16))
        return MOE_ERR_ALIGNMENT;
    if (B == 0) return MOE_OK;
    const AttnArgs a = {static_cast<const __nv_bfloat16*>(q), q_stride, B, q_heads, M, window, c, table, lengths, scale,
                        static_cast<__nv_bfloat16*>(out), lse};
    const dim3 grid(q_heads, B);
    if (dtype == MOE_MXFP8) attention_kernel<true><<<grid, 32 * PA_WARPS, 0, moe_host::as_stream(stream)>>>(a);
    else attention_kernel<false><<<grid, 32 * PA_WARPS, 0, moe_host::as_stream(stream)>>>(a);
    return moe_host::launch_status();
}
