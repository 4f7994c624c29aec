// few_tokens.cu -- the whole MoE layer for a few tokens (a decoding step): moe_layer_few_tokens.
//
// For every valid route (t, k) with expert e = ids[t,k]:
//   h = silu(x[t] W1[e]) * (x[t] W3[e]);   y[t] = bf16( sum_k p[t,k] (h W2[e]) )
// Every weight of the chosen experts is read once and used for the few tokens that chose
// them, so the time is the weights' bytes over the memory's rate.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int FEW_TMAX = 64;         // tokens
constexpr int FEW_KMAX = 128;        // routes per token
constexpr int FEW_ROUTES = 4096;     // T * K
constexpr int FEW_EMAX = 8192;       // experts

// ---------------------------------------------------------------------------
// First kernel, one CTA per token: the router's selection (unless the caller gave ids and
// probs), and for MXFP8 the token's row-wise 1x32 quantisation.
//
// Selection: a thread holds V logits as order-preserving keys (expert i * 256 + thread). Up to
// 256 experts, each logit's rank is counted directly against the row. Above, the K-th largest
// key is found by a search over its 32 bits, two bits a step (three counts of keys at or above a
// bound per step), then the keys above it and the lowest-index ones equal to it are ranked among
// themselves.
// ---------------------------------------------------------------------------
constexpr int PREP_THREADS = 256;
constexpr int PREP_WARPS = PREP_THREADS / 32;

struct PrepSmem {
    unsigned key[PREP_THREADS];
    unsigned list_key[FEW_KMAX];
    int list_idx[FEW_KMAX];
    unsigned cnt[2][3];
    float red[2][PREP_WARPS];
    int n;
};

// Larger float -> larger unsigned; -0 and +0 are one key.
__device__ __forceinline__ unsigned order_key(float f) {
    unsigned u = __float_as_uint(f);
    if ((u << 1) == 0) u = 0;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
    return (k & 0x80000000u) ? __uint_as_float(k & 0x7fffffffu) : __uint_as_float(~k);
}

template <bool MAX>
__device__ __forceinline__ float prep_reduce(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(FULL, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (lane_id() == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < PREP_WARPS; w++) v = MAX ? fmaxf(v, red[w]) : v + red[w];
    return v;
}

struct PrepArgs {
    const __nv_bfloat16* x;
    const float* logits;      // null: ids and probs are the caller's
    int H, E, K;
    void* ids;
    bool i16, renorm;
    float* probs;
    uint8_t* xq;              // MXFP8: codes [T, H] and scales [T, H / 32] of x; else null
    uint8_t* xs;
};

template <int V>
__device__ void prep_route(const PrepArgs& p, int t, PrepSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31;
    const float* row = p.logits + (long long)t * p.E;
    unsigned key[V];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = i * PREP_THREADS + tid;
        key[i] = 0u;          // below every logit's key
        if (e < p.E) {
            const float f = __ldg(row + e);
            key[i] = order_key(f);
            m = fmaxf(m, f);
        }
    }
    if (tid == 0) sm.n = 0;
    if (tid < 6) sm.cnt[tid / 3][tid % 3] = 0u;
    m = prep_reduce<true>(m, sm.red[0]);
    float den = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < V; i++)
            if (key[i]) den += expf(key_value(key[i]) - m);
        den = prep_reduce<false>(den, sm.red[1]);
    }
    if (V == 1) {
        sm.key[tid] = key[0];
        __syncthreads();
        int r = 0;
        for (int j = 0; j < p.E; j++) r += (sm.key[j] > key[0]) || (sm.key[j] == key[0] && j < tid);
        if (tid < p.E && r < p.K) {
            sm.list_key[r] = key[0];
            sm.list_idx[r] = tid;
        }
        __syncthreads();
    } else {
        // the largest bound with at least K keys at or above it: the K-th largest key
        unsigned kth = 0u, above = 0u;    // above: keys > kth, once the search is done
        for (int sh = 30, step = 0; sh >= 0; sh -= 2, step ^= 1) {
            unsigned c[3] = {0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < V; i++)
#pragma unroll
                for (int j = 0; j < 3; j++) c[j] += key[i] >= kth + ((unsigned)(j + 1) << sh);
#pragma unroll
            for (int j = 0; j < 3; j++) {
                c[j] = __reduce_add_sync(FULL, c[j]);
                if (lane == 0 && c[j]) atomicAdd(&sm.cnt[step][j], c[j]);
            }
            __syncthreads();
            unsigned d = 0u;
#pragma unroll
            for (int j = 0; j < 3; j++) d += sm.cnt[step][j] >= (unsigned)p.K;
            kth += d << sh;
            if (tid < 3) sm.cnt[step ^ 1][tid] = 0u;
            __syncthreads();
        }
        // how many of the keys equal to it belong to the K largest
        {
            unsigned c = 0u;
#pragma unroll
            for (int i = 0; i < V; i++) c += key[i] > kth;
            c = __reduce_add_sync(FULL, c);
            if (lane == 0 && c) atomicAdd(&sm.cnt[0][0], c);   // (cleared by the search's last step)
            if (tid == 0) sm.cnt[1][1] = 0u;
            __syncthreads();
            above = sm.cnt[0][0];
        }
        const unsigned ties = (unsigned)p.K - above;
        // the keys equal to kth with the lowest expert indices: the index bound by bisection
        int lo = 0, hi = p.E - 1;         // smallest b with at least `ties` equal keys at indices <= b
        int step = 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tid == 0) sm.cnt[step ^ 1][1] = 0u;
            unsigned c = 0u;
#pragma unroll
            for (int i = 0; i < V; i++) c += key[i] == kth && i * PREP_THREADS + tid <= mid;
            c = __reduce_add_sync(FULL, c);
            if (lane == 0 && c) atomicAdd(&sm.cnt[step][1], c);
            __syncthreads();
            if (sm.cnt[step][1] >= ties) hi = mid;
            else lo = mid + 1;
            step ^= 1;
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int e = i * PREP_THREADS + tid;
            if (e < p.E && (key[i] > kth || (key[i] == kth && e <= lo))) {
                const int pos = atomicAdd(&sm.n, 1);
                if (pos < FEW_KMAX) {     // (NaN logits aside, exactly K keys come here)
                    sm.list_key[pos] = key[i];
                    sm.list_idx[pos] = e;
                }
            }
        }
        __syncthreads();
    }
    if (p.renorm) {
        for (int j = tid; j < p.K; j += PREP_THREADS) den += expf(key_value(sm.list_key[j]) - m);
        den = prep_reduce<false>(den, sm.red[1]);
    }
    for (int j = tid; j < p.K; j += PREP_THREADS) {
        const unsigned k = sm.list_key[j];
        const int e = sm.list_idx[j];
        int r = j;
        if (V > 1) {
            r = 0;
            for (int i = 0; i < p.K; i++) r += sm.list_key[i] > k || (sm.list_key[i] == k && sm.list_idx[i] < e);
        }
        const long long o = (long long)t * p.K + r;
        if (p.i16) static_cast<int16_t*>(p.ids)[o] = (int16_t)e;
        else static_cast<int32_t*>(p.ids)[o] = e;
        p.probs[o] = expf(key_value(k) - m) / den;
    }
}

template <int V>
__global__ void __launch_bounds__(PREP_THREADS) few_prep_kernel(PrepArgs p) {
    __shared__ PrepSmem sm;
    const int t = blockIdx.x;
    if (p.logits) prep_route<V>(p, t, sm);
    if (p.xq) {
        const int lane = (int)lane_id();
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (long long)t * p.H);
        const int H8 = p.H >> 3;
        for (int j0 = threadIdx.x & ~31; j0 < H8; j0 += PREP_THREADS) {     // warp-uniform
            const int j = j0 + lane;
            float f[8];
            bf16x8_to_f32(j < H8 ? __ldg(src + j) : make_uint4(0, 0, 0, 0), f);
            int sb;
            const uint2 code = quant8_in_quad(f, &sb);
            if (j < H8) {
                reinterpret_cast<uint2*>(p.xq)[(long long)t * H8 + j] = code;
                if ((lane & 3) == 0) p.xs[(long long)t * (p.H >> 5) + (j >> 2)] = (uint8_t)sb;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The expert MLP, one warp per dot product.
// ---------------------------------------------------------------------------
// Dot product over n elements of two rows (bf16, or E4M3 codes with a scale byte per 32), by a warp.
template <bool FP8>
__device__ __forceinline__ float warp_dot(const void* a, const uint8_t* as, const void* b, const uint8_t* bs, int n) {
    const int lane = (int)lane_id();
    float acc = 0.0f;
    for (int j = lane; j < n / 8; j += 32) {
        if constexpr (FP8) {
            const uint2 u = __ldg(static_cast<const uint2*>(a) + j), v = __ldg(static_cast<const uint2*>(b) + j);
            const uint32_t uw[2] = {u.x, u.y}, vw[2] = {v.x, v.y};
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++)
                s = fmaf(e4m3_value((uw[i / 4] >> (8 * (i % 4))) & 0xffu), e4m3_value((vw[i / 4] >> (8 * (i % 4))) & 0xffu), s);
            acc += s * exp2f((float)((int)as[j / 4] - 127)) * exp2f((float)((int)bs[j / 4] - 127));
        } else {
            float f[8], g[8];
            bf16x8_to_f32(__ldg(static_cast<const uint4*>(a) + j), f);
            bf16x8_to_f32(__ldg(static_cast<const uint4*>(b) + j), g);
#pragma unroll
            for (int i = 0; i < 8; i++) acc = fmaf(f[i], g[i], acc);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(FULL, acc, o);
    return acc;
}

struct FewArgs {
    const void* x;            // [T, H] bf16 or E4M3
    const uint8_t* xs;
    const void* w13;
    const uint8_t* w13s;
    const void* w2;
    const uint8_t* w2s;
    const void* ids;
    const float* probs;
    bool i16;
    int T, H, K, E, F;
    void* h;                  // [T * K, F] bf16 or E4M3
    uint8_t* hs;
    __nv_bfloat16* y;
};

// h of one route and 32 columns of F per CTA (8 warps, four columns each).
template <bool FP8>
__global__ void __launch_bounds__(256) few_up_kernel(FewArgs p) {
    __shared__ float col[32];
    const int r = blockIdx.x, f0 = blockIdx.y * 32, warp = threadIdx.x >> 5, lane = (int)lane_id();
    const int t = r / p.K;
    const int e = load_id(p.ids, r, p.i16);
    if (e < 0 || e >= p.E) {
        if (e != -1 && threadIdx.x == 0 && blockIdx.y == 0) raise_device_error(MOE_DEVERR_BAD_ID);
        return;
    }
    const size_t esz = FP8 ? 1 : 2;
    const char* x = static_cast<const char*>(p.x) + (size_t)t * p.H * esz;
    const uint8_t* xs = FP8 ? p.xs + (size_t)t * (p.H / 32) : nullptr;
    for (int i = 0; i < 4; i++) {
        const int f = f0 + warp * 4 + i;
        const size_t row = (size_t)e * 2 * p.F + f / 128 * 256 + f % 128;
        const char* w = static_cast<const char*>(p.w13);
        const float a = warp_dot<FP8>(x, xs, w + row * p.H * esz, FP8 ? p.w13s + row * (p.H / 32) : nullptr, p.H);
        const float b = warp_dot<FP8>(x, xs, w + (row + 128) * p.H * esz,
                                      FP8 ? p.w13s + (row + 128) * (p.H / 32) : nullptr, p.H);
        if (lane == 0) col[warp * 4 + i] = a / (1.0f + expf(-a)) * b;
    }
    __syncthreads();
    if (warp == 0) {
        const float h = col[lane];
        const size_t o = (size_t)r * p.F + f0 + lane;
        if constexpr (FP8) {
            float amax = fabsf(h);
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o2));
            const int sb = e8m0_scale_byte(amax);
            static_cast<uint8_t*>(p.h)[o] = (uint8_t)f32x2_to_e4m3x2(h * e8m0_inv_scale(sb), 0.0f);
            if (lane == 0) p.hs[o / 32] = (uint8_t)sb;
        } else {
            static_cast<__nv_bfloat16*>(p.h)[o] = __float2bfloat16_rn(h);
        }
    }
}

// y of one token and 32 columns of H per CTA (8 warps, four columns each).
template <bool FP8>
__global__ void __launch_bounds__(256) few_down_kernel(FewArgs p) {
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = (int)lane_id();
    const size_t esz = FP8 ? 1 : 2;
    for (int i = 0; i < 4; i++) {
        const int c = blockIdx.y * 32 + warp * 4 + i;
        float acc = 0.0f;
        for (int k = 0; k < p.K; k++) {
            const int r = t * p.K + k, e = load_id(p.ids, r, p.i16);
            if (e < 0 || e >= p.E) continue;
            const size_t row = (size_t)e * p.H + c;
            const float d = warp_dot<FP8>(static_cast<const char*>(p.h) + (size_t)r * p.F * esz,
                                          FP8 ? p.hs + (size_t)r * (p.F / 32) : nullptr,
                                          static_cast<const char*>(p.w2) + row * p.F * esz,
                                          FP8 ? p.w2s + row * (p.F / 32) : nullptr, p.F);
            acc = fmaf(__ldg(p.probs + r), d, acc);
        }
        if (lane == 0) p.y[(size_t)t * p.H + c] = __float2bfloat16_rn(acc);
    }
}

// Workspace: x's codes and scales (MXFP8), h (and its scales), each region 128-byte aligned.
struct FewLayout {
    size_t xq, xs, h, hs, bytes;
};

FewLayout few_layout(int T, int K, int H, int F, bool fp8) {
    auto up = [](size_t v) { return (v + 127) & ~(size_t)127; };
    FewLayout l{};
    size_t o = 0;
    l.xq = o;
    o += fp8 ? up((size_t)T * H) : 0;
    l.xs = o;
    o += fp8 ? up((size_t)T * (H / 32)) : 0;
    l.h = o;
    o += up((size_t)T * K * F * (fp8 ? 1 : 2));
    l.hs = o;
    o += fp8 ? up((size_t)T * K * (F / 32)) : 0;
    l.bytes = o;
    return l;
}

moe_status few_sizes(int T, int K, int E, int H, int F, moe_dtype dtype) {
    if (dtype != MOE_BF16 && dtype != MOE_MXFP8) return MOE_ERR_INVALID_ARG;
    if (T < 0 || K < 1 || E < 1 || K > E || H < 128 || F < 128) return MOE_ERR_INVALID_ARG;
    const int step = dtype == MOE_MXFP8 ? 512 : 128;    // (MXFP8: whole 16-byte pieces of scales)
    if (H % step || F % step) return MOE_ERR_UNSUPPORTED;
    if (T > FEW_TMAX || K > FEW_KMAX || (long long)T * K > FEW_ROUTES || E > FEW_EMAX) return MOE_ERR_UNSUPPORTED;
    if ((long long)E * 2 * F > 0x7fffffffLL || (long long)E * H > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <bool FP8>
moe_status few_launch(FewArgs a, const PrepArgs& p, cudaStream_t s) {
    if (p.logits || p.xq) {
        const int V = p.logits ? (p.E + PREP_THREADS - 1) / PREP_THREADS : 1;
        if (V <= 1) few_prep_kernel<1><<<a.T, PREP_THREADS, 0, s>>>(p);
        else if (V <= 4) few_prep_kernel<4><<<a.T, PREP_THREADS, 0, s>>>(p);
        else if (V <= 12) few_prep_kernel<12><<<a.T, PREP_THREADS, 0, s>>>(p);
        else few_prep_kernel<32><<<a.T, PREP_THREADS, 0, s>>>(p);
    }
    few_up_kernel<FP8><<<dim3(a.T * a.K, a.F / 32), 256, 0, s>>>(a);
    few_down_kernel<FP8><<<dim3(a.T, a.H / 32), 256, 0, s>>>(a);
    return moe_host::launch_status();
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_layer_few_tokens_workspace_size(int T, int K, int E, int H, int F, moe_dtype dtype) {
    using namespace moe;
    if (few_sizes(T, K, E, H, F, dtype) != MOE_OK) return 0;
    return few_layout(T, K, H, F, dtype == MOE_MXFP8).bytes;
}

extern "C" moe_status moe_layer_few_tokens(const void* x, int T, int H, const float* logits, int K, int E, int F,
                                           const void* w13_packed, const uint8_t* w13_scales, const void* w2_packed,
                                           const uint8_t* w2_scales, moe_dtype dtype, void* ids, moe_dtype id_dtype,
                                           float* probs, void* y, unsigned flags, void* workspace,
                                           size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    if (id_dtype != MOE_I16 && id_dtype != MOE_I32) return MOE_ERR_INVALID_ARG;
    if (flags & ~MOE_ROUTE_RENORM) return MOE_ERR_INVALID_ARG;
    const moe_status st = few_sizes(T, K, E, H, F, dtype);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const bool fp8 = dtype == MOE_MXFP8;
    if (!x || !w13_packed || !w2_packed || !ids || !probs || !y) return MOE_ERR_INVALID_ARG;
    if (fp8 && (!w13_scales || !w2_scales)) return MOE_ERR_INVALID_ARG;
    const FewLayout l = few_layout(T, K, H, F, fp8);
    if (!workspace || workspace_bytes < l.bytes) return MOE_ERR_WORKSPACE;
    if (!moe_host::aligned(x, 16) || !moe_host::aligned(w13_packed, 128) || !moe_host::aligned(w2_packed, 128) ||
        !moe_host::aligned(workspace, 128) || !moe_host::aligned(y, 16) || !moe_host::aligned(logits, 4) ||
        !moe_host::aligned(probs, 4) || !moe_host::aligned(ids, id_dtype == MOE_I16 ? 2 : 4) ||
        (fp8 && (!moe_host::aligned(w13_scales, 16) || !moe_host::aligned(w2_scales, 16))))
        return MOE_ERR_ALIGNMENT;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrepArgs p{};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.logits = logits;
    p.H = H;
    p.E = E;
    p.K = K;
    p.ids = ids;
    p.i16 = id_dtype == MOE_I16;
    p.renorm = (flags & MOE_ROUTE_RENORM) != 0;
    p.probs = probs;
    p.xq = fp8 ? ws + l.xq : nullptr;
    p.xs = fp8 ? ws + l.xs : nullptr;
    FewArgs a{};
    a.x = fp8 ? p.xq : x;
    a.xs = p.xs;
    a.w13 = w13_packed;
    a.w13s = w13_scales;
    a.w2 = w2_packed;
    a.w2s = w2_scales;
    a.ids = ids;
    a.probs = probs;
    a.i16 = p.i16;
    a.T = T;
    a.H = H;
    a.K = K;
    a.E = E;
    a.F = F;
    a.h = ws + l.h;
    a.hs = fp8 ? ws + l.hs : nullptr;
    a.y = static_cast<__nv_bfloat16*>(y);
    const cudaStream_t s = moe_host::as_stream(stream);
    return fp8 ? few_launch<true>(a, p, s) : few_launch<false>(a, p, s);
}
