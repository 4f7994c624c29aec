// grad_norm.cu -- global gradient norm over many tensors, and clipping by it: moe_grad_norm_clip.
//
// norm = sqrt(sum of all g^2), c = min(1, max_norm / (norm + eps)), out = g c. Two kernels a
// group of tensors: the first sums the squares (a partial sum per CTA), the second adds the
// partial sums up -- every CTA all of them, in one fixed order -- and scales. The scale depends on every
// gradient, so what does not stay in L2 is read twice: three passes over the bytes bound large lists,
// two launches small ones. Measured: 2.8 GB of bf16 in six tensors 1274-1284 us, 6.6 TB/s over the three
// passes (a copy runs at 6.78); 40 tensors of 24 M elements in all, bf16 and fp32, 32.5 us; six tensors of a small layer 8-9 us.
// The list of tensors travels in the kernels' parameters. Its elements, in blocks of GN_BLOCK, are cut
// into one equal stretch per CTA whatever the tensors' sizes, so ragged lists keep every CTA busy. The
// second kernel walks each stretch from its end: what the first one read last is in L2 still.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int GN_GROUP = 96;          // tensors per launch (the table is a kernel parameter)
constexpr int GN_BLOCK = 2048;        // elements per block
constexpr int GN_THREADS = 256;
constexpr int GN_CTAS = 1216;         // partial sums per group: the grids at most

struct GradTable {
    const void* in[GN_GROUP];
    void* out[GN_GROUP];
    long long count[GN_GROUP];
    int first[GN_GROUP + 1];          // first block of each tensor
    uint8_t f32[GN_GROUP];
    int n;
};

// The tensor that a block belongs to.
__device__ __forceinline__ int tensor_of(const GradTable& g, int block) {
    int lo = 0, hi = g.n - 1;         // last tensor that starts at or before the block (never an empty one)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Sum over the CTA in a fixed order, the same in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    if (lane_id() == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < GN_THREADS / 32; w++) v += red[w];
    return v;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// 16 bytes as floats and back
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4], const float*) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8], const __nv_bfloat16*) { bf16x8_to_f32(v, f); }
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) { return f32_to_bf16x8(f); }

// Elements before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, long long m) {
    const int h = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T);
    return h < m ? h : (int)m;
}

// Squares of the m elements at p added to eight sums per thread: 16-byte pieces, four in flight, the
// elements before the first boundary and after the last one singly.
template <typename T>
__device__ __forceinline__ void sumsq_piece(const T* p, long long m, float (&acc)[8]) {
    constexpr int VEC = 16 / sizeof(T);
    const int h = head_of(p, m);
    const long long n = (m - h) / VEC;
    const uint4* q = reinterpret_cast<const uint4*>(p + h);
    long long j = threadIdx.x;
    for (; j + 3 * GN_THREADS < n; j += 4 * GN_THREADS) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) v[u] = __ldg(q + j + u * GN_THREADS);
#pragma unroll
        for (int u = 0; u < 4; u++) {
            float f[VEC];
            unpack(v[u], f, p);
#pragma unroll
            for (int k = 0; k < VEC; k++) acc[(u & 1) * (8 - VEC) + k] = fmaf(f[k], f[k], acc[(u & 1) * (8 - VEC) + k]);
        }
    }
    for (; j < n; j += GN_THREADS) {
        float f[VEC];
        unpack(__ldg(q + j), f, p);
#pragma unroll
        for (int k = 0; k < VEC; k++) acc[k] = fmaf(f[k], f[k], acc[k]);
    }
    const long long tail = h + n * VEC;
    const int rest = h + (int)(m - tail);                   // (both below VEC: one element a thread)
    if ((int)threadIdx.x < rest) {
        const long long k = (int)threadIdx.x < h ? threadIdx.x : tail + threadIdx.x - h;
        const float f = to_f(p[k]);
        acc[0] = fmaf(f, f, acc[0]);
    }
}

// out = in * c, from the end on; in and out may be the same. Pieces of 16 bytes where both are aligned alike.
template <typename T>
__device__ __forceinline__ void scale_piece(const T* p, T* o, long long m, float c) {
    constexpr int VEC = 16 / sizeof(T);
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
        for (long long j = threadIdx.x; j < m; j += GN_THREADS) put(o + j, to_f(p[j]) * c);
        return;
    }
    const int h = head_of(p, m);
    const long long n = (m - h) / VEC;
    const uint4* q = reinterpret_cast<const uint4*>(p + h);
    uint4* d = reinterpret_cast<uint4*>(o + h);
    auto one = [&](const uint4& v) {
        float f[VEC];
        unpack(v, f, p);
#pragma unroll
        for (int k = 0; k < VEC; k++) f[k] *= c;
        return pack(f);
    };
    long long j = n - 1 - (long long)threadIdx.x;
    for (; j - 3 * GN_THREADS >= 0; j -= 4 * GN_THREADS) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) v[u] = __ldcs(q + j - u * GN_THREADS);
#pragma unroll
        for (int u = 0; u < 4; u++) __stcs(d + j - u * GN_THREADS, one(v[u]));
    }
    for (; j >= 0; j -= GN_THREADS) __stcs(d + j, one(__ldcs(q + j)));
    const long long tail = h + n * VEC;
    const int rest = h + (int)(m - tail);
    if ((int)threadIdx.x < rest) {
        const long long k = (int)threadIdx.x < h ? threadIdx.x : tail + threadIdx.x - h;
        put(o + k, to_f(p[k]) * c);
    }
}

__global__ void __launch_bounds__(GN_THREADS) grad_sumsq_kernel(const __grid_constant__ GradTable g, float* partial) {
    __shared__ float red[GN_THREADS / 32];
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const int blocks = g.first[g.n];
    int b = (int)((long long)blocks * blockIdx.x / gridDim.x);
    const int end = (int)((long long)blocks * (blockIdx.x + 1) / gridDim.x);
    for (int i = tensor_of(g, b); b < end; i++) {
        const int stop = min(end, g.first[i + 1]);
        const long long at = (long long)(b - g.first[i]) * GN_BLOCK;
        const long long m = min((long long)(stop - g.first[i]) * GN_BLOCK, g.count[i]) - at;
        if (g.f32[i]) sumsq_piece(static_cast<const float*>(g.in[i]) + at, m, acc);
        else sumsq_piece(static_cast<const __nv_bfloat16*>(g.in[i]) + at, m, acc);
        b = stop;
    }
    pdl_trigger();
    const float s = cta_sum(((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])), red);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// partial: n_partial sums. norm_out: written by CTA 0, null for the groups after the first.
__global__ void __launch_bounds__(GN_THREADS) grad_scale_kernel(const __grid_constant__ GradTable g, const float* partial,
                                                                int n_partial, float max_norm, float eps,
                                                                float* norm_out) {
    __shared__ float red[GN_THREADS / 32];
    const int blocks = g.first[g.n];
    const int begin = (int)((long long)blocks * blockIdx.x / gridDim.x);
    int b = (int)((long long)blocks * (blockIdx.x + 1) / gridDim.x);
    const int last = b > begin ? tensor_of(g, b - 1) : 0;
    pdl_wait();
    float v = 0.0f;
    for (int j = threadIdx.x; j < n_partial; j += GN_THREADS) v += __ldcg(partial + j);
    const float norm = sqrtf(cta_sum(v, red));
    // (within the bound nothing is divided: 0 / 0 and inf / inf are no scale. A NaN norm is within no bound, and stays.)
    const float c = norm + eps <= max_norm ? 1.0f : max_norm / (norm + eps);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    for (int i = last; b > begin; i--) {
        const int start = max(begin, g.first[i]);
        if (c != 1.0f || g.in[i] != g.out[i]) {
            const long long at = (long long)(start - g.first[i]) * GN_BLOCK;
            const long long m = min((long long)(b - g.first[i]) * GN_BLOCK, g.count[i]) - at;
            if (g.f32[i])
                scale_piece(static_cast<const float*>(g.in[i]) + at, static_cast<float*>(g.out[i]) + at, m, c);
            else
                scale_piece(static_cast<const __nv_bfloat16*>(g.in[i]) + at, static_cast<__nv_bfloat16*>(g.out[i]) + at, m, c);
        }
        b = start;
    }
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_grad_norm_workspace_size(int n) {
    using namespace moe;
    if (n < 0) return 0;
    const size_t groups = n == 0 ? 1 : ((size_t)n + GN_GROUP - 1) / GN_GROUP;
    return groups * GN_CTAS * sizeof(float);
}

extern "C" moe_status moe_grad_norm_clip(const void* const* grads, const long long* counts, const int* dtypes,
                                         void* const* outs, int n, float max_norm, float eps, float* norm_out,
                                         void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    if (n < 0 || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !norm_out) return MOE_ERR_INVALID_ARG;
    if (n > 0 && (!grads || !counts || !dtypes)) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; i++) {
        if (counts[i] < 0 || (dtypes[i] != MOE_BF16 && dtypes[i] != MOE_F32)) return MOE_ERR_INVALID_ARG;
        if (counts[i] > 0 && (!grads[i] || (outs && !outs[i]))) return MOE_ERR_INVALID_ARG;
        if (counts[i] > ((long long)1 << 35)) return MOE_ERR_UNSUPPORTED;   // (blocks are counted in 32 bits)
    }
    if (!workspace || workspace_bytes < moe_grad_norm_workspace_size(n)) return MOE_ERR_WORKSPACE;
    if (!moe_host::aligned(workspace, 16) || !moe_host::aligned(norm_out, 4)) return MOE_ERR_ALIGNMENT;
    for (int i = 0; i < n; i++) {
        const size_t a = dtypes[i] == MOE_F32 ? 4 : 2;
        if (counts[i] > 0 && (!moe_host::aligned(grads[i], a) || (outs && !moe_host::aligned(outs[i], a))))
            return MOE_ERR_ALIGNMENT;
    }
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int most = sms * 8 < GN_CTAS ? sms * 8 : GN_CTAS;
    const cudaStream_t s = moe_host::as_stream(stream);
    float* partial = static_cast<float*>(workspace);
    auto table = [&](int i0) {
        GradTable g;
        g.n = 0;
        int blocks = 0;
        for (int i = i0; i < n && i < i0 + GN_GROUP; i++) {
            if (counts[i] == 0) continue;
            g.in[g.n] = grads[i];
            g.out[g.n] = outs ? outs[i] : nullptr;
            g.count[g.n] = counts[i];
            g.f32[g.n] = dtypes[i] == MOE_F32;
            g.first[g.n] = blocks;
            blocks += (int)((counts[i] + GN_BLOCK - 1) / GN_BLOCK);
            g.n++;
        }
        g.first[g.n] = blocks;
        return g;
    };
    // four blocks a CTA at least (its threads' loads in flight): fewer partial sums for everybody to read
    auto ctas = [&](const GradTable& g) {
        const int c = (g.first[g.n] + 3) / 4;
        return c < most ? c : most;
    };
    int n_partial = 0;
    for (int i0 = 0; i0 < n; i0 += GN_GROUP) {
        const GradTable g = table(i0);
        if (!g.n) continue;
        grad_sumsq_kernel<<<ctas(g), GN_THREADS, 0, s>>>(g, partial + n_partial);
        n_partial += ctas(g);
    }
    bool told = false;
    for (int i0 = 0; i0 < n && outs; i0 += GN_GROUP) {
        const GradTable g = table(i0);
        if (!g.n) continue;
        if (moe_host::launch_pdl(grad_scale_kernel, dim3(ctas(g)), dim3(GN_THREADS), 0, s, g, (const float*)partial, n_partial,
                                 max_norm, eps, told ? (float*)nullptr : norm_out) != cudaSuccess)
            return MOE_ERR_CUDA;
        told = true;
    }
    if (!told) {
        GradTable g;
        g.n = 0;
        g.first[0] = 0;
        if (moe_host::launch_pdl(grad_scale_kernel, dim3(1), dim3(GN_THREADS), 0, s, g, (const float*)partial, n_partial, max_norm,
                                 eps, norm_out) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return moe_host::launch_status();
}
