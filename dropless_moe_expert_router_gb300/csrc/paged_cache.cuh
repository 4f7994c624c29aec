// paged_cache.cuh -- the pools of a paged key-value cache, for the kernels that write and read them.
#pragma once

#include "common.cuh"

constexpr int MOE_CACHE_MAX_PAGE = 4096;   // positions in a page
constexpr int MOE_CACHE_MAX_DIM = 256;

namespace moe {

// Pages [pages, heads, page_size, dim] of keys and values, and (MXFP8) their scales, dim / 32 bytes a row.
struct CachePools {
    void* k;
    void* v;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int pages, heads, page_size, dim;
};

// Value of an E8M0 byte: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Two E4M3 codes as two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// Four E4M3 codes as floats (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t four, float* f) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t h = e4m3x2_to_f16x2((four >> (16 * i)) & 0xffffu);
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

}  // namespace moe

namespace moe_host {

inline moe_status check_cache(const moe::CachePools& c, moe_dtype dtype, int M) {
    if (dtype != MOE_BF16 && dtype != MOE_MXFP8) return MOE_ERR_INVALID_ARG;
    if (c.pages < 1 || c.heads < 1 || c.dim < 1 || c.page_size < 1 || M < 1 || !c.k || !c.v) return MOE_ERR_INVALID_ARG;
    if (dtype == MOE_MXFP8 && (!c.k_scales || !c.v_scales)) return MOE_ERR_INVALID_ARG;
    if (c.dim % (dtype == MOE_MXFP8 ? 32 : 16) || c.dim > MOE_CACHE_MAX_DIM || c.page_size > MOE_CACHE_MAX_PAGE ||
        (long long)M * c.page_size >= (1ll << 31))
        return MOE_ERR_UNSUPPORTED;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return MOE_ERR_ALIGNMENT;
    if (dtype == MOE_MXFP8) {
        // (a row's scales are read together: a power of two of them at a time)
        const int row = c.dim / 32, a = row % 8 == 0 ? 8 : row % 4 == 0 ? 4 : row % 2 == 0 ? 2 : 1;
        if (!aligned(c.k_scales, a) || !aligned(c.v_scales, a)) return MOE_ERR_ALIGNMENT;
    }
    return MOE_OK;
}

}  // namespace moe_host
