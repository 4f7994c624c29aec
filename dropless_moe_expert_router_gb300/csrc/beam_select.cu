// beam_select.cu -- selection of a beam search's step: moe_beam_select.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int BS_THREADS = 512;
constexpr int BS_MAX_K = 64;
constexpr int BS_MAX_W = 64;

struct BeamArgs {
    const void* logits;
    const float* scores;
    const uint8_t* done;
    int pad, N, W, V, K;
    float* out_scores;
    int32_t* parents;
    int32_t* tokens;
};

template <typename T>
__device__ __forceinline__ float logit(const void* p, long long i);
template <>
__device__ __forceinline__ float logit<float>(const void* p, long long i) { return __ldg(static_cast<const float*>(p) + i); }
template <>
__device__ __forceinline__ float logit<__nv_bfloat16>(const void* p, long long i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// A block per search: every beam's lse, then K times the largest candidate below the last one.
template <typename T>
__global__ void __launch_bounds__(BS_THREADS) beam_select_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ double lse[BS_MAX_W], red_v[BS_THREADS / 32];
    __shared__ long long red_i[BS_THREADS / 32];
    __shared__ float red[BS_THREADS / 32];
    const int n = blockIdx.x, warp = threadIdx.x / 32;
    const long long row0 = (long long)n * a.W;
    for (int w = 0; w < a.W; w++) {
        float top = -INFINITY;
        bool bad = false;
        for (int t = threadIdx.x; t < a.V; t += BS_THREADS) {
            const float x = logit<T>(a.logits, (row0 + w) * a.V + t);
            bad = bad || x != x;
            top = fmaxf(top, x);
        }
        if (bad) top = INFINITY;
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        if (lane_id() == 0) red[warp] = top;
        __syncthreads();
        for (int i = 0; i < BS_THREADS / 32; i++) top = fmaxf(top, red[i]);
        double sum = 0.0;
        if (isfinite(top))
            for (int t = threadIdx.x; t < a.V; t += BS_THREADS) sum += exp((double)logit<T>(a.logits, (row0 + w) * a.V + t) - top);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (lane_id() == 0) red_v[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < BS_THREADS / 32; i++) sum += red_v[i];
            // (not finite: the beam has no candidate)
            lse[w] = isfinite(top) && isfinite(a.scores[row0 + w]) ? top + log(sum) : INFINITY;
        }
        __syncthreads();
    }
    double last_v = INFINITY;
    long long last_i = -1;
    for (int k = 0; k < a.K; k++) {
        double best_v = -INFINITY;
        long long best_i = 1ll << 62;
        for (int w = 0; w < a.W; w++) {
            const double score = a.scores[row0 + w];
            const bool is_done = a.done && a.done[row0 + w];
            for (int t = threadIdx.x; t < a.V; t += BS_THREADS) {
                double v = -INFINITY;
                if (is_done) {
                    if (t == a.pad && isfinite(score)) v = score;
                } else if (lse[w] != INFINITY) {
                    v = score + ((double)logit<T>(a.logits, (row0 + w) * a.V + t) - lse[w]);
                }
                const long long i = (long long)w * a.V + t;
                if ((v < last_v || (v == last_v && i > last_i)) && (v > best_v || (v == best_v && i < best_i))) {
                    best_v = v;
                    best_i = i;
                }
            }
        }
        auto join = [&](double v, long long i) {
            if (v > best_v || (v == best_v && i < best_i)) {
                best_v = v;
                best_i = i;
            }
        };
        for (int o = 16; o > 0; o >>= 1) {
            const double v = __shfl_xor_sync(FULL, best_v, o);
            const long long i = __shfl_xor_sync(FULL, best_i, o);
            join(v, i);
        }
        __syncthreads();
        if (lane_id() == 0) {
            red_v[warp] = best_v;
            red_i[warp] = best_i;
        }
        __syncthreads();
        for (int i = 0; i < BS_THREADS / 32; i++) join(red_v[i], red_i[i]);
        last_v = best_v;
        last_i = best_i;
        if (threadIdx.x == 0) {
            const long long o = (long long)n * a.K + k;
            a.out_scores[o] = (float)best_v;
            a.parents[o] = (int)(row0 + best_i / a.V);
            a.tokens[o] = (int)(best_i % a.V);
        }
    }
}

bool refused(int N, int W, int V, int K) {
    return N < 0 || W < 1 || W > BS_MAX_W || V < 1 || V >= (1 << 24) || (long long)N * W >= (1 << 24) || K < 1 ||
           K > BS_MAX_K || (long long)K > (long long)W * V;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_beam_select_workspace_size(int N, int W, int V, int K) {
    return moe::refused(N, W, V, K) ? 0 : 256;
}

extern "C" moe_status moe_beam_select(const void* logits, moe_dtype dtype, const float* scores, const uint8_t* done, int pad,
                                      int N, int W, int V, int K, float* out_scores, int32_t* parents, int32_t* tokens,
                                      void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    if ((dtype != MOE_BF16 && dtype != MOE_F32) || N < 0 || W < 1 || V < 1 || K < 1 || (long long)K > (long long)W * V)
        return MOE_ERR_INVALID_ARG;
    if (done && (pad < 0 || pad >= V)) return MOE_ERR_INVALID_ARG;
    if (refused(N, W, V, K)) return MOE_ERR_UNSUPPORTED;
    if (N > 0 && (!logits || !scores || !out_scores || !parents || !tokens)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_beam_select_workspace_size(N, W, V, K)) return MOE_ERR_WORKSPACE;
    if (!moe_host::aligned(logits, 16) || !moe_host::aligned(scores, 4) || !moe_host::aligned(out_scores, 4) ||
        !moe_host::aligned(parents, 4) || !moe_host::aligned(tokens, 4) || !moe_host::aligned(workspace, 16))
        return MOE_ERR_ALIGNMENT;
    if (N == 0) return MOE_OK;
    const BeamArgs a = {logits, scores, done, pad, N, W, V, K, out_scores, parents, tokens};
    if (dtype == MOE_F32) beam_select_kernel<float><<<N, BS_THREADS, 0, moe_host::as_stream(stream)>>>(a);
    else beam_select_kernel<__nv_bfloat16><<<N, BS_THREADS, 0, moe_host::as_stream(stream)>>>(a);
    return moe_host::launch_status();
}
