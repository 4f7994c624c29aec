// layer_norm.cu -- the layer norm of a pre-norm block and its backward pass: moe_layer_norm and
// moe_layer_norm_backward.
//
// Forward, per row: s = x (+ residual), mean = sum s / H, rstd = 1 / sqrt(sum (s - mean)^2 / H + eps),
// y = (s - mean) rstd w + b. Backward, with xh = (s - mean) rstd and g = dy w:
// dx = rstd (g - sum(g) / H - xh sum(g xh) / H) (+ dx_add), dw = sum_t dy xh, db = sum_t dy.
// Each operand is read once and each output written once: the bytes bound both directions.
#include "common.cuh"

namespace moe {
namespace {

constexpr int LN_HMAX = 65536;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Sum over the CTA, the same in every thread; red: 32 floats, free again after the next barrier.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if (lane_id() == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane_id() < (unsigned)warps ? red[lane_id()] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// One CTA per row; a row that does not fit in registers is read again for each sum.
template <typename T, typename W>
__global__ void __launch_bounds__(256) ln_forward_kernel(const T* x, const T* residual, int H, const W* __restrict__ w,
                                                         const W* __restrict__ b, float eps, T* sum, T* y,
                                                         float* mean_out, float* rstd_out) {
    __shared__ float red[2][32];
    const long long base = (long long)blockIdx.x * H;
    float a = 0.0f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
        float v = to_f(x[base + i]);
        if (residual) {
            const T r = from_f<T>(v + to_f(residual[base + i]));
            sum[base + i] = r;
            v = to_f(r);
        }
        a += v;
    }
    const T* s = residual ? sum : x;
    const float mean = cta_sum(a, red[0]) / (float)H;
    a = 0.0f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
        const float d = to_f(s[base + i]) - mean;
        a = fmaf(d, d, a);
    }
    const float rstd = 1.0f / sqrtf(cta_sum(a, red[1]) / (float)H + eps);
    for (int i = threadIdx.x; i < H; i += blockDim.x)
        y[base + i] = from_f<T>(fmaf((to_f(s[base + i]) - mean) * rstd, to_f(w[i]), b ? to_f(b[i]) : 0.0f));
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[blockIdx.x] = mean;
        if (rstd_out) rstd_out[blockIdx.x] = rstd;
    }
}

// dx, one CTA per row.
template <typename T, typename W>
__global__ void __launch_bounds__(256) ln_backward_dx_kernel(const T* dy, const T* __restrict__ s, int H,
                                                             const W* __restrict__ w, const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const T* dx_add, T* dx) {
    __shared__ float red[2][32];
    const long long base = (long long)blockIdx.x * H;
    const float m = mean[blockIdx.x], r = rstd[blockIdx.x];
    float a = 0.0f, c = 0.0f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
        const float g = to_f(dy[base + i]) * to_f(w[i]);
        a += g;
        c = fmaf(g, (to_f(s[base + i]) - m) * r, c);
    }
    a = cta_sum(a, red[0]) / (float)H;
    c = cta_sum(c, red[1]) / (float)H;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
        const float g = to_f(dy[base + i]) * to_f(w[i]);
        float v = r * (g - a - (to_f(s[base + i]) - m) * r * c);
        if (dx_add) v += to_f(dx_add[base + i]);
        dx[base + i] = from_f<T>(v);
    }
}

// dweight and dbias, one thread per column.
template <typename T, typename W>
__global__ void __launch_bounds__(32) ln_backward_w_kernel(const T* dy, const T* __restrict__ s, int rows, int H,
                                                           const float* __restrict__ mean, const float* __restrict__ rstd,
                                                           W* dw, W* db) {
    const int i = blockIdx.x * 32 + threadIdx.x;
    if (i >= H) return;
    float a = 0.0f, c = 0.0f;
    for (int t = 0; t < rows; t++) {
        const float g = to_f(dy[(long long)t * H + i]);
        a = fmaf(g, (to_f(s[(long long)t * H + i]) - mean[t]) * rstd[t], a);
        c += g;
    }
    if (dw) dw[i] = from_f<W>(a);
    if (db) db[i] = from_f<W>(c);
}

bool ln_type(int d) { return d == MOE_BF16 || d == MOE_F32; }
size_t ln_size(int d) { return d == MOE_BF16 ? 2 : 4; }

template <typename T, typename W>
moe_status ln_forward(const void* x, const void* residual, int rows, int H, const void* w, const void* b, float eps,
                      void* sum, void* y, float* mean, float* rstd, cudaStream_t s) {
    ln_forward_kernel<T, W><<<rows, 256, 0, s>>>((const T*)x, (const T*)residual, H, (const W*)w, (const W*)b, eps,
                                                 (T*)sum, (T*)y, mean, rstd);
    return moe_host::launch_status();
}

template <typename T, typename W>
moe_status ln_backward(const void* dy, const void* sv, int rows, int H, const void* w, const float* mean,
                       const float* rstd, const void* dx_add, void* dx, void* dw, void* db, cudaStream_t s) {
    // (before dx, which may be dy)
    if (dw || db)
        ln_backward_w_kernel<T, W><<<(H + 31) / 32, 32, 0, s>>>((const T*)dy, (const T*)sv, rows, H, mean, rstd, (W*)dw,
                                                                (W*)db);
    if (rows)
        ln_backward_dx_kernel<T, W><<<rows, 256, 0, s>>>((const T*)dy, (const T*)sv, H, (const W*)w, mean, rstd,
                                                         (const T*)dx_add, (T*)dx);
    return moe_host::launch_status();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_layer_norm(const void* x, const void* residual, int T, int H, moe_dtype dtype,
                                     const void* weight, const void* bias, moe_dtype w_dtype, float eps, void* sum,
                                     void* y, float* mean, float* rstd, moe_stream_t stream) {
    using namespace moe;
    if (T < 0 || H < 1 || !(eps >= 0.0f) || !ln_type(dtype) || !ln_type(w_dtype)) return MOE_ERR_INVALID_ARG;
    if ((residual == nullptr) != (sum == nullptr) && T > 0) return MOE_ERR_INVALID_ARG;
    if (H > LN_HMAX) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || !weight || !y) return MOE_ERR_INVALID_ARG;
    const size_t a = ln_size(dtype), aw = ln_size(w_dtype);
    if (!moe_host::aligned(x, a) || !moe_host::aligned(residual, a) || !moe_host::aligned(sum, a) ||
        !moe_host::aligned(y, a) || !moe_host::aligned(weight, aw) || !moe_host::aligned(bias, aw) ||
        !moe_host::aligned(mean, 4) || !moe_host::aligned(rstd, 4))
        return MOE_ERR_ALIGNMENT;
    const cudaStream_t s = moe_host::as_stream(stream);
#define MOE_LN(T_, W_) return ln_forward<T_, W_>(x, residual, T, H, weight, bias, eps, sum, y, mean, rstd, s)
    if (dtype == MOE_BF16) {
        if (w_dtype == MOE_BF16) MOE_LN(__nv_bfloat16, __nv_bfloat16);
        MOE_LN(__nv_bfloat16, float);
    }
    if (w_dtype == MOE_BF16) MOE_LN(float, __nv_bfloat16);
    MOE_LN(float, float);
#undef MOE_LN
}

extern "C" size_t moe_layer_norm_backward_workspace_size(int T, int H) {
    if (T < 0 || H < 1 || H > moe::LN_HMAX) return 0;
    return 16;
}

extern "C" moe_status moe_layer_norm_backward(const void* dy, const void* s, int T, int H, moe_dtype dtype,
                                              const void* weight, moe_dtype w_dtype, const float* mean,
                                              const float* rstd, const void* dx_add, void* dx, void* dweight,
                                              void* dbias, void* workspace, size_t workspace_bytes,
                                              moe_stream_t stream) {
    using namespace moe;
    if (T < 0 || H < 1 || !ln_type(dtype) || !ln_type(w_dtype)) return MOE_ERR_INVALID_ARG;
    if (H > LN_HMAX) return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!dy || !s || !weight || !mean || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_layer_norm_backward_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
    const size_t a = ln_size(dtype), aw = ln_size(w_dtype);
    if (!moe_host::aligned(dy, a) || !moe_host::aligned(s, a) || !moe_host::aligned(dx_add, a) ||
        !moe_host::aligned(dx, a) || !moe_host::aligned(weight, aw) || !moe_host::aligned(dweight, aw) ||
        !moe_host::aligned(dbias, aw) || !moe_host::aligned(mean, 4) || !moe_host::aligned(rstd, 4) ||
        !moe_host::aligned(workspace, 16))
        return MOE_ERR_ALIGNMENT;
    const cudaStream_t st = moe_host::as_stream(stream);
#define MOE_LNB(T_, W_) return ln_backward<T_, W_>(dy, s, T, H, weight, mean, rstd, dx_add, dx, dweight, dbias, st)
    if (dtype == MOE_BF16) {
        if (w_dtype == MOE_BF16) MOE_LNB(__nv_bfloat16, __nv_bfloat16);
        MOE_LNB(__nv_bfloat16, float);
    }
    if (w_dtype == MOE_BF16) MOE_LNB(float, __nv_bfloat16);
    MOE_LNB(float, float);
#undef MOE_LNB
}
