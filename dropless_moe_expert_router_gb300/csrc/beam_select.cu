// beam_select.cu -- selection of a beam search's step: moe_beam_select.
//
// For every beam lse = ln sum exp(logits), and over a search's beams the K largest score + (logit - lse). The logits
// are read once: DRAM bounds large vocabularies, two launches small ones. Two kernels:
//
// 1. A block holds a chunk of 8192 logits of one beam in registers. It leaves the chunk's maximum and sum of
//    exponentials, and its K largest logits in order (within a beam the order does not depend on lse). For these it
//    takes the K-th largest of its 256 threads' maxima, found bit by bit with a counting barrier: no fewer than K logits are that large,
//    and but for ties to it they are in fewer than K threads, so few are left to be ranked against each other. Where more tie than
//    the buffer holds, the first ones are taken in order.
// 2. A block per search, set up while the first kernel runs, joins the sums in 64 bits and the chunks' lists: it drops
//    what fp32 bounds show to be behind K others, and ranks the rest by its value in 64 bits.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int BS_THREADS = 256;      // of the first kernel
constexpr int BS_HELD = 32;          // logits a thread holds
constexpr int BS_CHUNK = BS_THREADS * BS_HELD;
constexpr int BS_CAP = 2048;         // > (BS_MAX_K - 1) * BS_HELD: what lies above the K-th largest maximum fits
constexpr int BS_JOIN = 512;         // threads of the second
constexpr int BS_EACH = 8;           // list entries a thread of it looks at together
constexpr int BS_MAX_K = 64;
constexpr int BS_MAX_W = 64;

struct BeamArgs {
    const void* logits;
    const float* scores;
    const uint8_t* done;
    int pad, W, V, K, chunks;
    float* out_scores;
    int32_t* parents;
    int32_t* tokens;
    float2* part;                    // [rows, chunks] maximum, sum of exp relative to it
    unsigned long long* list;        // [rows, chunks, K] order of the logit, then of the lowest token; 0: none
};

__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Whole numbers in the order of floats (-0 below +0), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }

// The largest number that at least K threads of the block have or exceed (K of them at most above it; 0 if there is none).
__device__ __forceinline__ uint32_t kth_largest(uint32_t mine, int K, int lowest_bit) {
    uint32_t t = 0u;
    for (int bit = 31; bit >= lowest_bit; bit--) {
        const uint32_t tried = t | (1u << bit);
        const int n = __syncthreads_count(mine >= tried);
        if (n >= K) t = tried;
        if (n == K) break;
    }
    // (below zero, the numbers of values without lower bits have ones there)
    return t & 0x80000000u ? t : t | ((1u << lowest_bit) - 1u);
}

// A thread's logits: pieces of 16 bytes, THREADS pieces apart.
template <typename T>
struct Held;
template <>
struct Held<float> {
    static constexpr int VEC = 4, PIECES = BS_HELD / 4, LOWEST_BIT = 0;
    float v[PIECES][VEC];
    __device__ __forceinline__ float at(int i, int e) const { return v[i][e]; }
    __device__ __forceinline__ void load(int i, const float* p) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p));
        v[i][0] = x.x;
        v[i][1] = x.y;
        v[i][2] = x.z;
        v[i][3] = x.w;
    }
    __device__ __forceinline__ void some(int i, const float* p, int first, int end) {
#pragma unroll
        for (int e = 0; e < VEC; e++) v[i][e] = e >= first && e < end ? __ldg(p + e) : -INFINITY;
    }
    __device__ __forceinline__ float top(int i) const { return fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])); }
};
template <>
struct Held<__nv_bfloat16> {
    static constexpr int VEC = 8, PIECES = BS_HELD / 8, LOWEST_BIT = 16;
    uint4 v[PIECES];
    __device__ __forceinline__ uint32_t word(int i, int w) const { return w == 0 ? v[i].x : w == 1 ? v[i].y : w == 2 ? v[i].z : v[i].w; }
    __device__ __forceinline__ float at(int i, int e) const {
        return __uint_as_float(e & 1 ? word(i, e >> 1) & 0xffff0000u : word(i, e >> 1) << 16);
    }
    __device__ __forceinline__ void load(int i, const __nv_bfloat16* p) { v[i] = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void some(int i, const __nv_bfloat16* p, int first, int end) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            const uint32_t x = e >= first && e < end ? (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + e) : 0xff80u;
            w[e >> 1] = e & 1 ? w[e >> 1] | (x << 16) : x;
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float top(int i) const {
        const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v[i]);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
        return fmaxf(f.x, f.y);
    }
};

template <typename T>
__global__ void __launch_bounds__(BS_THREADS) beam_chunk_kernel(const __grid_constant__ BeamArgs a) {
    using H = Held<T>;
    __shared__ unsigned long long buf[BS_CAP];
    __shared__ float2 warps[BS_THREADS / 32];
    __shared__ int count, scan[BS_THREADS / 32];
    const int chunk = blockIdx.x % a.chunks, warp = threadIdx.x / 32;
    const long long row = blockIdx.x / a.chunks, start = row * a.V;
    // pieces are counted from the last 16-byte boundary at or before the row
    const int skew = (int)(start % H::VEC);
    const T* const base = static_cast<const T*>(a.logits) + (start - skew);
    const int p0 = chunk * (BS_THREADS * H::PIECES) + threadIdx.x;
    pdl_trigger();
    if (threadIdx.x == 0) count = 0;

    H h;
    float top = -INFINITY, tops[H::PIECES];
#pragma unroll
    for (int i = 0; i < H::PIECES; i++) {
        const int at = (p0 + i * BS_THREADS) * H::VEC - skew;        // token of the piece's first element
        const T* const p = base + (at + skew);
        if (at >= 0 && at + H::VEC <= a.V) h.load(i, p);
        else h.some(i, p, max(0, -at), min(H::VEC, a.V - at));
    }
#pragma unroll
    for (int i = 0; i < H::PIECES; i++) {
        tops[i] = h.top(i);
        top = fmaxf(top, tops[i]);
    }
    // sum of exponentials, relative to the thread's maximum (where that is -inf: 0, or NaN if there is one)
    constexpr float LOG2E = 1.44269504088896340736f;
    {
        const float sub = top == -INFINITY ? 0.0f : top;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < H::PIECES; i++)
#pragma unroll
            for (int e = 0; e < H::VEC; e++) sum[e & 3] += pow2((h.at(i, e) - sub) * LOG2E);
        float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        float m = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        if (top != -INFINITY) s *= pow2((top - m) * LOG2E);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
        if (lane_id() == 0) warps[warp] = make_float2(m, s);
    }

    const float least = of_order(kth_largest(order_of(top), a.K, H::LOWEST_BIT));
    if (threadIdx.x == 0) {                                          // (the counting barrier stands between)
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int w = 0; w < BS_THREADS / 32; w++) m = fmaxf(m, warps[w].x);
#pragma unroll
        for (int w = 0; w < BS_THREADS / 32; w++) s += warps[w].x == -INFINITY ? warps[w].y : warps[w].y * pow2((warps[w].x - m) * LOG2E);
        a.part[blockIdx.x] = make_float2(m, s);
    }
    // what is that large; `strictly`: larger
    auto gather = [&](bool strictly) {
        if (top < least) return;
#pragma unroll
        for (int i = 0; i < H::PIECES; i++) {
            if (tops[i] < least) continue;
            const int at = (p0 + i * BS_THREADS) * H::VEC - skew;
#pragma unroll
            for (int e = 0; e < H::VEC; e++) {
                const float x = h.at(i, e);
                if (strictly ? x > least : x >= least) {
                    if ((unsigned)(at + e) < (unsigned)a.V) {
                        const int slot = atomicAdd(&count, 1);
                        if (slot < BS_CAP)
                            buf[slot] = (unsigned long long)order_of(x + 0.0f) << 32 | (0xffffffffu - (uint32_t)(at + e));
                    }
                }
            }
        }
    };
    gather(false);
    __syncthreads();
    int n = count;
    if (n > BS_CAP) {
        // too many ties: those above, and the first K of the ties in the tokens' order
        __syncthreads();
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        gather(true);
        int before = 0;
#pragma unroll
        for (int i = 0; i < H::PIECES; i++) {
            if (before >= a.K) break;
            const int at = (p0 + i * BS_THREADS) * H::VEC - skew;
            int mine = 0;
#pragma unroll
            for (int e = 0; e < H::VEC; e++) mine += h.at(i, e) == least && (unsigned)(at + e) < (unsigned)a.V;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, upto, o);
                if ((int)lane_id() >= o) upto += v;
            }
            __syncthreads();
            if (lane_id() == 31) scan[warp] = upto;
            __syncthreads();
            int rank = before + upto - mine;
            for (int w = 0; w < BS_THREADS / 32; w++) {
                if (w < warp) rank += scan[w];
                before += scan[w];
            }
#pragma unroll
            for (int e = 0; e < H::VEC; e++)
                if (h.at(i, e) == least && (unsigned)(at + e) < (unsigned)a.V && rank++ < a.K) {
                    const int slot = atomicAdd(&count, 1);
                    if (slot < BS_CAP)
                        buf[slot] = (unsigned long long)order_of(least + 0.0f) << 32 | (0xffffffffu - (uint32_t)(at + e));
                }
        }
        __syncthreads();
        n = min(count, BS_CAP);
    }
    unsigned long long* const list = a.list + (long long)blockIdx.x * a.K;
    for (int i = threadIdx.x; i < n; i += BS_THREADS) {
        const unsigned long long mine = buf[i];
        int rank = 0;
        for (int k = 0; k < n; k++) rank += buf[k] > mine;
        if (rank < a.K) list[rank] = mine;
    }
    for (int k = n + threadIdx.x; k < a.K; k += BS_THREADS) list[k] = 0ull;
}

struct Joined {
    double best[BS_MAX_K];
    int best_at[BS_MAX_K];
    double lse[BS_MAX_W];            // of a beam that lives; else NaN
    float score[BS_MAX_W], off[BS_MAX_W];
    int state[BS_MAX_W];             // 0: lives, 1: done, 2: has no candidate
    int count;
    double v[BS_JOIN * BS_EACH + BS_MAX_K];
    int at[BS_JOIN * BS_EACH + BS_MAX_K];
};

__global__ void __launch_bounds__(BS_JOIN) beam_join_kernel(const __grid_constant__ BeamArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Joined& s = *reinterpret_cast<Joined*>(raw);
    const int warp = threadIdx.x / 32;
    const long long row0 = (long long)blockIdx.x * a.W;
    pdl_wait();
    for (int w = warp; w < a.W; w += BS_JOIN / 32) {
        const float2* part = a.part + (row0 + w) * a.chunks;
        float m = -INFINITY;
        for (int c = lane_id(); c < a.chunks; c += 32) m = fmaxf(m, __ldcg(part + c).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        double sum = 0.0;
        for (int c = lane_id(); c < a.chunks; c += 32) {
            const float2 x = __ldcg(part + c);
            sum += x.x == -INFINITY || x.x == m ? (double)x.y : x.y * exp((double)x.x - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (lane_id() == 0) {
            const float score = a.scores[row0 + w];
            const double lse = m + log(sum);
            const bool fine = isfinite(score), done = a.done && a.done[row0 + w];
            s.score[w] = score;
            s.lse[w] = lse;
            s.off[w] = (float)(score - lse);
            s.state[w] = done && fine ? 1 : !done && fine && isfinite(lse) ? 0 : 2;
        }
    }
    __syncthreads();

    const int per_beam = a.chunks * a.K;
    const long long total = (long long)a.W * per_beam;
    // list entry i: its beam and token, and x, its logit (a done or dead beam's: its score, or -inf); false: none
    auto entry = [&](long long i, int& w, int& token, float& x) {
        if (i >= total) return false;
        w = (int)(i / per_beam);
        const int k = (int)(i - (long long)w * per_beam);
        if (s.state[w] == 0) {
            const unsigned long long key = __ldcg(a.list + row0 * per_beam + i);
            if (key == 0ull) return false;
            token = (int)(0xffffffffu - (uint32_t)key);
            x = of_order((uint32_t)(key >> 32));
            return true;
        }
        if (k >= a.K || k >= a.V) return false;
        token = k;
        x = -INFINITY;
        if (s.state[w] == 1) {
            token = k == 0 ? a.pad : k - 1 < a.pad ? k - 1 : k;
            if (k == 0) x = s.score[w];
        }
        return true;
    };
    auto value = [&](int w, float x) {
        return x == -INFINITY ? (double)-INFINITY : s.state[w] ? (double)x : (double)s.score[w] + ((double)x - s.lse[w]);
    };
    int kept = 0;
    for (long long i0 = 0; i0 < total; i0 += BS_JOIN * BS_EACH) {
        float hi[BS_EACH];
        float low = -INFINITY;                                       // the largest lower bound of the thread's entries
        if (threadIdx.x == 0) s.count = 0;
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            int w, token;
            float x;
            hi[e] = __uint_as_float(0x7fc00000u);
            if (!entry(i0 + e * BS_JOIN + threadIdx.x, w, token, x)) continue;
            float lo = x;
            hi[e] = x;
            if (s.state[w] == 0 && x != -INFINITY) {
                // |value - v| < 2^-22 (|off| + |x|) with the roundings of off and of the sum
                const float v = s.off[w] + x, eps = (fabsf(s.off[w]) + fabsf(x)) * 0x1p-21f;
                const bool fine = isfinite(v) && isfinite(eps);
                lo = fine ? v - eps : -INFINITY;
                hi[e] = fine ? v + eps : INFINITY;
            }
            low = fmaxf(low, lo);
        }
        if ((int)threadIdx.x < kept) low = fmaxf(low, __double2float_rd(s.best[threadIdx.x]));
        const float least = of_order(kth_largest(order_of(low), a.K, 0));
        __syncthreads();
        auto push = [&](double v, int at) {
            const int slot = atomicAdd(&s.count, 1);
            s.v[slot] = v;
            s.at[slot] = at;
        };
        if ((int)threadIdx.x < kept) push(s.best[threadIdx.x], s.best_at[threadIdx.x]);
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            int w, token;
            float x;
            if (!(hi[e] >= least) || !entry(i0 + e * BS_JOIN + threadIdx.x, w, token, x)) continue;
            push(value(w, x), w * a.V + token);
        }
        __syncthreads();
        const int n = s.count;
        for (int i = threadIdx.x; i < n; i += BS_JOIN) {
            const double v = s.v[i];
            const int at = s.at[i];
            int rank = 0;
            for (int k = 0; k < n; k++) rank += s.v[k] > v || (s.v[k] == v && s.at[k] < at);
            if (rank < a.K) {
                s.best[rank] = v;
                s.best_at[rank] = at;
            }
        }
        kept = min(n, a.K);
        __syncthreads();
    }
    if ((int)threadIdx.x < a.K) {
        const long long o = (long long)blockIdx.x * a.K + threadIdx.x;
        const int at = s.best_at[threadIdx.x], w = at / a.V;
        a.out_scores[o] = (float)s.best[threadIdx.x];
        a.parents[o] = (int)(row0 + w);
        a.tokens[o] = at - w * a.V;
    }
}

// Chunks of a row: 16-byte pieces that hold V logits wherever the row begins, in blocks' shares.
int chunks_of(int V, int vec) {
    const int pieces = (V + 2 * vec - 2) / vec, share = BS_CHUNK / vec;
    return (pieces + share - 1) / share;
}

bool refused(int N, int W, int V, int K) {
    return N < 0 || W < 1 || W > BS_MAX_W || V < 1 || V >= (1 << 24) || (long long)N * W >= (1 << 24) || K < 1 ||
           K > BS_MAX_K || (long long)K > (long long)W * V || (long long)N * W * chunks_of(V, 8) >= (1ll << 31);
}

// (bf16 rows take at least as many chunks as fp32 ones)
size_t list_bytes(int N, int W, int V, int K) { return (size_t)N * W * chunks_of(V, 8) * K * sizeof(unsigned long long); }

template <typename T>
moe_status launch(BeamArgs a, int N, cudaStream_t s) {
    static moe_host::PerDevice smem;
    a.chunks = chunks_of(a.V, Held<T>::VEC);
    beam_chunk_kernel<T><<<(unsigned)((long long)N * a.W * a.chunks), BS_THREADS, 0, s>>>(a);
    const moe_status st = moe_host::launch_status();
    if (st != MOE_OK) return st;
    if (!moe_host::allow_smem(beam_join_kernel, sizeof(Joined), smem) ||
        moe_host::launch_pdl(beam_join_kernel, dim3(N), dim3(BS_JOIN), sizeof(Joined), s, a) != cudaSuccess)
        return MOE_ERR_CUDA;
    return moe_host::launch_status();
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_beam_select_workspace_size(int N, int W, int V, int K) {
    using namespace moe;
    if (refused(N, W, V, K)) return 0;
    const size_t rows = (size_t)(N ? N : 1) * W;
    return list_bytes(N ? N : 1, W, V, K) + rows * chunks_of(V, 8) * sizeof(float2);
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
    BeamArgs a = {logits, scores, done, pad, W, V, K, 0, out_scores, parents, tokens, nullptr, nullptr};
    a.list = static_cast<unsigned long long*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + list_bytes(N, W, V, K));
    return dtype == MOE_F32 ? launch<float>(a, N, moe_host::as_stream(stream)) : launch<__nv_bfloat16>(a, N, moe_host::as_stream(stream));
}
