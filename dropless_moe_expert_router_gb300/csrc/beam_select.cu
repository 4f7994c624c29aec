// beam_select.cu -- selection of a beam search's step: moe_beam_select.
//
// For every beam lse = ln sum exp(logits), and over a search's beams the K largest score + (logit - lse). The logits
// are read once: DRAM bounds large vocabularies, two launches small ones. Two kernels:
//
// 1. A block holds a chunk of one beam's logits in registers (8192 fp32, 16384 bf16). It leaves the chunk's maximum and sum of
//    exponentials, and its K largest logits in order (within a beam the order does not depend on lse). For these it
//    takes the K-th largest of the maxima of 64 groups of four threads, found bit by bit by one warp: no fewer than K logits are
//    that large, and few more as a rule, which are ranked against each other. Where they are more than the buffer
//    holds, the K-th largest logit itself is found the same way, and of what ties with it the first ones in order.
// 2. A block per search, set up while the first kernel runs, joins the sums in 64 bits and the chunks' lists: it drops
//    what fp32 bounds show to be behind K others, and ranks the rest by its value in 64 bits.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int BS_THREADS = 256;      // of the first kernel
constexpr int BS_GROUPS = BS_THREADS / 4;
constexpr int BS_CAP = 1024;         // logits that are ranked against each other
constexpr int BS_JOIN = 256;         // threads of the second
constexpr int BS_BEAM = 8;           // of them that join a beam's sums
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

// Two floats in one register pair: added or multiplied by one instruction.
struct Two {
    unsigned long long v;
    __device__ __forceinline__ Two(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ void get(float& x, float& y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
    __device__ __forceinline__ Two& operator+=(const Two& o) {
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(o.v));
        return *this;
    }
    __device__ __forceinline__ Two& operator*=(const Two& o) {
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(o.v));
        return *this;
    }
};

// Whole numbers in the order of floats (-0 below +0), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }

// (below zero, the numbers of values without lower bits have ones there)
__device__ __forceinline__ uint32_t filled(uint32_t t, int lowest_bit) {
    return t & 0x80000000u ? t : t | ((1u << lowest_bit) - 1u);
}

// Of two numbers a lane of one warp, the largest t that at least K have or exceed, or a smaller one that K of them do;
// its bits from lowest_bit on are looked for, so with more of them it is the smaller the fewer.
__device__ __forceinline__ uint32_t kth_largest(uint32_t x, uint32_t y, int K, int lowest_bit) {
    uint32_t t = 0u;
    for (int bit = 31; bit >= lowest_bit; bit--) {
        const uint32_t tried = t | (1u << bit);
        const int n = __popc(__ballot_sync(FULL, x >= tried)) + __popc(__ballot_sync(FULL, y >= tried));
        if (n >= K) t = tried;
        if (n == K) break;
    }
    return max(t, 0x007fffffu);      // (not below -inf, where NaN's numbers are)
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A thread's logits: pieces of 16 bytes, THREADS pieces apart.
template <typename T>
struct Held;
template <>
struct Held<float> {
    static constexpr int VEC = 4, PIECES = 8, LOWEST_BIT = 0;
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
    // f(x, e) for the elements [first, end) of the piece at p, all of them where it is whole
    template <typename F>
    static __device__ __forceinline__ void each(const float* p, bool whole, int first, int end, F f) {
        if (whole) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p));
            f(x.x, 0);
            f(x.y, 1);
            f(x.z, 2);
            f(x.w, 3);
        } else {
#pragma unroll 1
            for (int e = first; e < end; e++) f(__ldg(p + e), e);
        }
    }
    __device__ __forceinline__ float top(int i) const { return fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])); }
};
template <>
struct Held<__nv_bfloat16> {
    static constexpr int VEC = 8, PIECES = 8, LOWEST_BIT = 16;
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
    template <typename F>
    static __device__ __forceinline__ void each(const __nv_bfloat16* p, bool whole, int first, int end, F f) {
        if (whole) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < VEC; e++) f(__uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16), e);
        } else {
#pragma unroll 1
            for (int e = first; e < end; e++) f(__bfloat162float(p[e]), e);
        }
    }
    __device__ __forceinline__ float top(int i) const {
        const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v[i]);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
        return fmaxf(f.x, f.y);
    }
};

__device__ __forceinline__ unsigned long long key_of(float x, int token) {
    return (unsigned long long)order_of(x + 0.0f) << 32 | (0xffffffffu - (uint32_t)token);
}

// The K largest of a chunk where many tie, or lie above the groups' threshold: the K-th largest logit is found bit by
// bit; those above it are fewer than K, and of what ties with it the first K in the tokens' order are taken, piece by piece.
// The chunk is read again for it (from L2). Returns their number, in buf.
template <typename T>
__device__ __noinline__ int exactly_largest(const T* row, int first, int V, int K, unsigned long long* buf, int* count, int* scan) {
    using H = Held<T>;
    const int warp = threadIdx.x / 32;
    auto sum = [&](int mine) {
        mine = __reduce_add_sync(FULL, mine);
        __syncthreads();
        if (lane_id() == 0) scan[warp] = mine;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < BS_THREADS / 32; w++) all += scan[w];
        return all;
    };
    auto read = [&](int i, int e, int& token, uint32_t& x) {
        token = first + i * BS_THREADS * H::VEC + e;
        if ((unsigned)token >= (unsigned)V) return false;
        x = order_of(to_float(row[token]) + 0.0f);
        return true;
    };
    int token;
    uint32_t x, t = 0u;
    for (int bit = 31; bit >= H::LOWEST_BIT; bit--) {
        const uint32_t tried = t | (1u << bit);
        int mine = 0;
        for (int i = 0; i < H::PIECES; i++)
            for (int e = 0; e < H::VEC; e++) mine += read(i, e, token, x) && x >= tried;
        if (sum(mine) >= K) t = tried;
    }
    t = filled(t, H::LOWEST_BIT);
    __syncthreads();
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    auto push = [&](uint32_t x, int token) {
        const int slot = atomicAdd(count, 1);
        if (slot < BS_CAP) buf[slot] = (unsigned long long)x << 32 | (0xffffffffu - (uint32_t)token);
    };
    int before = 0;
    for (int i = 0; i < H::PIECES; i++) {
        int mine = 0;
        for (int e = 0; e < H::VEC; e++) {
            if (!read(i, e, token, x)) continue;
            if (x > t) push(x, token);
            mine += x == t;
        }
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
        for (int e = 0; e < H::VEC; e++)
            if (read(i, e, token, x) && x == t && rank++ < K) push(x, token);
    }
    __syncthreads();
    return min(*count, BS_CAP);
}

template <typename T>
__global__ void __launch_bounds__(BS_THREADS, 4) beam_chunk_kernel(const __grid_constant__ BeamArgs a) {
    using H = Held<T>;
    __shared__ unsigned long long buf[BS_CAP];
    __shared__ float2 warps[BS_THREADS / 32];
    __shared__ uint32_t groups[BS_GROUPS], threshold;
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
    const int at0 = p0 * H::VEC - skew;                              // token of the first piece's first element
    const T* const piece0 = base + (at0 + skew);
    constexpr int STEP = BS_THREADS * H::VEC;                        // tokens between a thread's pieces
    const int chunk_at = chunk * H::PIECES * STEP - skew;
    if (chunk_at >= 0 && chunk_at + H::PIECES * STEP <= a.V) {
#pragma unroll
        for (int i = 0; i < H::PIECES; i++) h.load(i, piece0 + i * STEP);
    } else {
#pragma unroll
        for (int i = 0; i < H::PIECES; i++) {
            const int at = at0 + i * STEP;
            if (at >= 0 && at + H::VEC <= a.V) h.load(i, piece0 + i * STEP);
            else h.some(i, piece0 + i * STEP, max(0, -at), min(H::VEC, a.V - at));
        }
    }
#pragma unroll
    for (int i = 0; i < H::PIECES; i++) {
        tops[i] = h.top(i);
        top = fmaxf(top, tops[i]);
    }
    // the threshold, by the first warp while the others sum
    float four = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
    four = fmaxf(four, __shfl_xor_sync(FULL, four, 2));
    if ((threadIdx.x & 3) == 0) groups[threadIdx.x / 4] = order_of(four);
    __syncthreads();
    if (warp == 0) {
        const uint32_t t = kth_largest(groups[lane_id()], groups[lane_id() + 32], a.K, 12);
        if (lane_id() == 0) threshold = t;
    }
    // sum of exponentials, relative to the thread's maximum (where that is -inf: 0, or NaN if there is one)
    constexpr float LOG2E = 1.44269504088896340736f;
    {
        const float sub = top == -INFINITY ? 0.0f : top;
        const Two minus(-sub, -sub), log2e(LOG2E, LOG2E);
        Two sum0(0.0f, 0.0f), sum1(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < H::PIECES; i++)
#pragma unroll
            for (int e = 0; e < H::VEC; e += 2) {
                Two x(h.at(i, e), h.at(i, e + 1));
                x += minus;
                x *= log2e;
                float x0, x1;
                x.get(x0, x1);
                (e & 2 ? sum1 : sum0) += Two(pow2(x0), pow2(x1));
            }
        sum0 += sum1;
        float s, s1;
        sum0.get(s, s1);
        s += s1;
        float m = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        if (top != -INFINITY) s *= pow2((top - m) * LOG2E);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
        if (lane_id() == 0) warps[warp] = make_float2(m, s);
    }
    __syncthreads();
    if (warp == BS_THREADS / 32 - 1) {
        const float2 x = lane_id() < BS_THREADS / 32 ? warps[lane_id()] : make_float2(-INFINITY, 0.0f);
        float m = x.x;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        float v = x.x == -INFINITY ? x.y : x.y * pow2((x.x - m) * LOG2E);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
        if (lane_id() == 0) a.part[blockIdx.x] = make_float2(m, v);
    }
    const float least = of_order(threshold);
    // (the few pieces that hold one are read again: a loop's code, not eight pieces' in line)
    unsigned hits = 0u;
#pragma unroll
    for (int i = 0; i < H::PIECES; i++) hits |= (unsigned)(tops[i] >= least) << i;
    while (hits) {
        const int i = __ffs(hits) - 1;
        hits &= hits - 1;
        const int at = at0 + i * STEP;
        H::each(piece0 + i * STEP, at >= 0 && at + H::VEC <= a.V, max(0, -at), min(H::VEC, a.V - at), [&](float x, int e) {
            if (x >= least) {
                const int slot = atomicAdd(&count, 1);
                if (slot < BS_CAP) buf[slot] = key_of(x, at + e);
            }
        });
    }
    __syncthreads();
    int n = count;
    if (n > BS_CAP) n = exactly_largest<T>(base + skew, at0, a.V, a.K, buf, &count, scan);
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
    unsigned long long best[BS_MAX_K];
    int best_at[BS_MAX_K];
    double lse[BS_MAX_W];            // of a beam that lives
    float score[BS_MAX_W], off[BS_MAX_W], m[BS_MAX_W];
    int state[BS_MAX_W];             // 0: lives, 1: done, 2: has no candidate
    uint32_t groups[64], threshold;
    int count;
    unsigned long long v[BS_JOIN * BS_EACH + BS_MAX_K];
    int at[BS_JOIN * BS_EACH + BS_MAX_K];
};

// Whole numbers in the order of doubles (-0 as +0), and back.
__device__ __forceinline__ unsigned long long order_of(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x == 0.0 ? 0.0 : x);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double of_order(unsigned long long u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

// (What takes 64 bits is slow on this device: a logarithm a beam, all in one warp, and the survivors' values.)
__global__ void __launch_bounds__(BS_JOIN) beam_join_kernel(const __grid_constant__ BeamArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Joined& s = *reinterpret_cast<Joined*>(raw);
    const long long row0 = (long long)blockIdx.x * a.W;
    const int per_beam = a.chunks * a.K, total = a.W * per_beam;
    const unsigned long long* const list = a.list + row0 * per_beam;
    pdl_wait();
    // the first entries are on their way while the sums are joined
    unsigned long long ahead[BS_EACH];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            const int i = i0 + e * BS_JOIN + threadIdx.x;
            ahead[e] = i < total ? __ldcg(list + i) : 0ull;
        }
    };
    fetch(0);
    for (int w0 = 0; w0 < a.W; w0 += BS_JOIN / BS_BEAM) {
        const int w = w0 + threadIdx.x / BS_BEAM, l = threadIdx.x % BS_BEAM;
        const float2* part = a.part + (row0 + min(w, a.W - 1)) * a.chunks;
        float m = -INFINITY;
        for (int c = l; c < a.chunks; c += BS_BEAM) m = fmaxf(m, __ldcg(part + c).x);
#pragma unroll
        for (int o = BS_BEAM / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        double sum = 0.0;
        for (int c = l; c < a.chunks; c += BS_BEAM) {
            const float2 x = __ldcg(part + c);
            sum += x.x == -INFINITY || x.x == m ? x.y : x.y * expf(x.x - m);
        }
#pragma unroll
        for (int o = BS_BEAM / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (l == 0 && w < a.W) {
            s.m[w] = m;
            s.lse[w] = sum;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.W) {
        const int w = threadIdx.x;
        const float score = a.scores[row0 + w];
        const double lse = s.m[w] + log(s.lse[w]);
        const bool fine = isfinite(score), done = a.done && a.done[row0 + w];
        s.score[w] = score;
        s.lse[w] = lse;
        s.off[w] = (float)(score - lse);
        s.state[w] = done && fine ? 1 : !done && fine && isfinite(lse) ? 0 : 2;
    }
    __syncthreads();

    // list entry i, its key read: its beam and token, and x, its logit (a done or dead beam's: its score, or -inf); false: none
    auto entry = [&](int i, unsigned long long key, int& w, int& token, float& x) {
        if (i >= total) return false;
        w = i / per_beam;
        const int k = i - w * per_beam;
        if (s.state[w] == 0) {
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
    for (int i0 = 0; i0 < total; i0 += BS_JOIN * BS_EACH) {
        if (i0) fetch(i0);
        float hi[BS_EACH];
        float low = -INFINITY;                                       // the largest lower bound of the thread's entries
        if (threadIdx.x == 0) s.count = 0;
        const int turns = min(BS_EACH, (total - i0 + BS_JOIN - 1) / BS_JOIN);
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            hi[e] = __uint_as_float(0x7fc00000u);
            if (e >= turns) continue;
            int w, token;
            float x;
            if (!entry(i0 + e * BS_JOIN + threadIdx.x, ahead[e], w, token, x)) continue;
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
        if ((int)threadIdx.x < kept) low = fmaxf(low, __double2float_rd(of_order(s.best[threadIdx.x])));
        low = fmaxf(low, __shfl_xor_sync(FULL, low, 1));
        low = fmaxf(low, __shfl_xor_sync(FULL, low, 2));
        if ((threadIdx.x & 3) == 0) s.groups[threadIdx.x / 4] = order_of(low);
        __syncthreads();
        if (threadIdx.x < 32) {
            const uint32_t t = kth_largest(s.groups[lane_id()], s.groups[lane_id() + 32], a.K, 10);
            if (lane_id() == 0) s.threshold = t;
        }
        __syncthreads();
        const float least = of_order(s.threshold);
        auto push = [&](unsigned long long v, int at) {
            const int slot = atomicAdd(&s.count, 1);
            s.v[slot] = v;
            s.at[slot] = at;
        };
        if ((int)threadIdx.x < kept) push(s.best[threadIdx.x], s.best_at[threadIdx.x]);
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            if (!(hi[e] >= least)) continue;
            int w, token;
            float x;
            if (entry(i0 + e * BS_JOIN + threadIdx.x, ahead[e], w, token, x)) push(order_of(value(w, x)), w * a.V + token);
        }
        __syncthreads();
        const int n = s.count;
        for (int i = threadIdx.x; i < n; i += BS_JOIN) {
            const unsigned long long v = s.v[i];
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
        a.out_scores[o] = (float)of_order(s.best[threadIdx.x]);
        a.parents[o] = (int)(row0 + w);
        a.tokens[o] = at - w * a.V;
    }
}

// Chunks of a row: 16-byte pieces that hold V logits wherever the row begins, in blocks' shares.
template <typename T>
int chunks_of(int V) {
    using H = Held<T>;
    const int pieces = V % H::VEC ? (V + 2 * H::VEC - 2) / H::VEC : V / H::VEC, share = BS_THREADS * H::PIECES;
    return (pieces + share - 1) / share;
}
// (fp32 rows take at least as many as bf16 ones: the workspace is for either)
int most_chunks(int V) { return chunks_of<float>(V); }

bool refused(int N, int W, int V, int K) {
    return N < 0 || W < 1 || W > BS_MAX_W || V < 1 || V >= (1 << 24) || (long long)N * W >= (1 << 24) || K < 1 ||
           K > BS_MAX_K || (long long)K > (long long)W * V || (long long)N * W * most_chunks(V) >= (1ll << 31);
}

size_t list_bytes(int N, int W, int V, int K) { return (size_t)N * W * most_chunks(V) * K * sizeof(unsigned long long); }

template <typename T>
moe_status launch(BeamArgs a, int N, cudaStream_t s) {
    static moe_host::PerDevice smem;
    a.chunks = chunks_of<T>(a.V);
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
    return list_bytes(N ? N : 1, W, V, K) + rows * most_chunks(V) * sizeof(float2);
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
