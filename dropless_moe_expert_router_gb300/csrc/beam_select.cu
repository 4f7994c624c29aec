// beam_select.cu -- selection of a beam search's step: moe_beam_select.
//
// For every beam lse = ln sum exp(logits), and over a search's beams the K largest score + (logit - lse). The logits
// are read once: DRAM bounds large vocabularies, two launches small ones. Two kernels:
//
// 1. All rows' logits, in units of 2048 16-byte pieces, are cut into one equal stretch per block. Every thread copies its
//    own eight pieces of a unit to a ring in shared memory, two units ahead and across rows, so loads are in flight all
//    the time and the code is one short loop (eight pieces in registers in line took half as long again: it does not
//    stay in the instruction cache). A unit is the same logits of a row wherever the row lies and whichever block has it, and
//    its maximum and sum of exponentials are its own, so rows with the same logits have the same sums. Where rows begin off 16 bytes
//    (V no multiple of a piece), the ring holds the aligned pieces around a unit and the threads read theirs across two of them.
//    Besides, a block leaves for each row of its stretch the K largest logits in order (within a beam the order does not
//    depend on lse). What is below a threshold is passed over a piece at a time by the piece's maximum.
//    The first threshold is the K-th largest of the maxima of 64 groups of four threads in the row's first unit, found bit by bit by one
//    warp: no fewer than K logits are that large. Later ones are the K-th largest found so far. Where more than the buffer
//    holds pass, the unit's K-th largest itself is found bit by bit, and of what ties with it the first ones are taken in order.
// 2. A block per search, set up while the first kernel runs, joins the units' sums, in their order, and the lists: it drops
//    what fp32 bounds show to be behind K others, and ranks the rest by its value in two floats, of 46 bits or more
//    (this device's 64-bit units are slow: a logarithm and the sums took 5 us in them).
//
// Measured (one GB300, GPU time): 32 searches of 8 beams over 131072 bf16 logits, K = 16: 24.7-25.1 us (67 MB, 9.9 us at the copy's rate;
// 131071 logits, rows off 16 bytes: 31), of which the first kernel takes 19 and the second 6 behind it, a chain of latencies. The first issues 2.1 instructions a cycle of
// 4; a fifth of its warps' waits are at the block's barriers (two a row for the threshold, three a look), the rest is spread over
// reads of the ring, powers and fixed latencies. Two packed adds, a packed product, two powers and two unpackings for two logits are a third
// of its instructions, thresholds and ranks of each stretch the most of the rest. 1 search of 4 beams over 32000 fp32: 9 us.
#include "common.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int BS_THREADS = 256;      // of the first kernel
constexpr int BS_HELD = 8;           // a thread's 16-byte pieces of a unit
constexpr int BS_GROUPS = BS_THREADS / 4;
constexpr int BS_CAP = 1024;         // logits that are ranked against each other
constexpr int BS_CHECK = 16;         // units between two looks at how many there are, at most
constexpr int BS_STAGE = BS_HELD * BS_THREADS + 1;   // pieces of a unit in the ring, and the one behind
constexpr int BS_CTAS = 3;           // blocks an SM
constexpr int BS_RING = 2;           // units on their way or looked at
constexpr int BS_MAX_CTAS = 1024;    // blocks at most: what the workspace has room for
constexpr int BS_JOIN = 256;         // threads of the second
constexpr int BS_BEAM = 8;           // of them that join a beam's sums
constexpr int BS_EACH = 4;           // lists a warp of it looks at together
constexpr int BS_MAX_K = 64;
constexpr int BS_MAX_W = 64;

struct BeamArgs {
    const void* logits;
    const float* scores;
    const uint8_t* done;
    int pad, W, V, K;
    int units, segments;             // units of a row; stretches that a row is in at most
    int ctas, each, longer;          // blocks; units of a block's stretch, one more for the first `longer` of them
    long long count;                 // logits in all
    float* out_scores;
    int32_t* parents;
    int32_t* tokens;
    float2* part;                    // [row][unit] maximum, sum of exp relative to it
    // of block g's part of row r, at g + r (no two have the same): [K] order of the logit, then of the lowest token; 0: none
    unsigned long long* list;
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
    // += 2^((x + shift) scale), 2^((y + shift) scale)
    __device__ __forceinline__ void add_pow2(float x, float y, const Two& shift, const Two& scale) {
        asm("{\n .reg .b64 t;\n .reg .f32 a, b;\n mov.b64 t, {%1, %2};\n add.rn.f32x2 t, t, %3;\n mul.rn.f32x2 t, t, %4;\n"
            " mov.b64 {a, b}, t;\n ex2.approx.ftz.f32 a, a;\n ex2.approx.ftz.f32 b, b;\n mov.b64 t, {a, b};\n add.rn.f32x2 %0, %0, t;\n}"
            : "+l"(v) : "f"(x), "f"(y), "l"(shift.v), "l"(scale.v));
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
    // (the bits that all have in common it has too)
    const uint32_t any = __reduce_or_sync(FULL, x | y), all = __reduce_and_sync(FULL, x & y), differ = any ^ all;
    if (differ == 0u) return x;
    const int first = 31 - __clz(differ);
    uint32_t t = first == 31 ? 0u : any >> (first + 1) << (first + 1);
    for (int bit = first; bit >= lowest_bit; bit--) {
        const uint32_t tried = t | (1u << bit);
        const int n = __popc(__ballot_sync(FULL, x >= tried)) + __popc(__ballot_sync(FULL, y >= tried));
        if (n >= K) t = tried;
        if (n == K) break;
    }
    return max(t, 0x007fffffu);      // (not below -inf, where NaN's numbers are)
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A piece: 16 bytes of logits.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int VEC = 4, LOWEST_BIT = 0;
    float v[VEC];
    __device__ __forceinline__ float at(int e) const { return v[e]; }
    __device__ __forceinline__ float pick(int e) const { return e & 2 ? (e & 1 ? v[3] : v[2]) : (e & 1 ? v[1] : v[0]); }
    __device__ __forceinline__ void put(const uint4& x) {
        v[0] = __uint_as_float(x.x);
        v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z);
        v[3] = __uint_as_float(x.w);
    }
    // the one that begins so many elements behind a boundary (two 16-byte reads: short ones meet the same banks)
    __device__ __forceinline__ void put_from(const uint4* at, int skew) {
        const uint4 x = at[0], y = at[1];
        const bool two = skew & 2, one = skew & 1;
        const uint32_t w0 = two ? x.z : x.x, w1 = two ? x.w : x.y, w2 = two ? y.x : x.z, w3 = two ? y.y : x.w, w4 = two ? y.z : y.x;
        put(make_uint4(one ? w1 : w0, one ? w2 : w1, one ? w3 : w2, one ? w4 : w3));
    }
    // -inf from element end on
    __device__ __forceinline__ void cut(int end) {
#pragma unroll
        for (int e = 0; e < VEC; e++) v[e] = e < end ? v[e] : -INFINITY;
    }
    __device__ __forceinline__ float top() const { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int VEC = 8, LOWEST_BIT = 16;
    uint4 v;
    __device__ __forceinline__ uint32_t word(int w) const { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; }
    __device__ __forceinline__ float at(int e) const { return __uint_as_float(e & 1 ? word(e >> 1) & 0xffff0000u : word(e >> 1) << 16); }
    __device__ __forceinline__ float pick(int e) const {
        const uint32_t w = e & 4 ? (e & 2 ? v.w : v.z) : (e & 2 ? v.y : v.x);
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ void put(const uint4& x) { v = x; }
    __device__ __forceinline__ void put_from(const uint4* at, int skew) {
        const uint4 x = at[0], y = at[1];
        const bool four = skew & 4, two = skew & 2;
        const uint32_t w0 = four ? x.z : x.x, w1 = four ? x.w : x.y, w2 = four ? y.x : x.z, w3 = four ? y.y : x.w, w4 = four ? y.z : y.x,
                       w5 = four ? y.w : y.y;
        const uint32_t z0 = two ? w1 : w0, z1 = two ? w2 : w1, z2 = two ? w3 : w2, z3 = two ? w4 : w3, z4 = two ? w5 : w4;
        const int bits = 16 * (skew & 1);
        v = make_uint4(__funnelshift_r(z0, z1, bits), __funnelshift_r(z1, z2, bits), __funnelshift_r(z2, z3, bits), __funnelshift_r(z3, z4, bits));
    }
    __device__ __forceinline__ void cut(int end) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = 2 * i >= end ? 0xff80ff80u : 2 * i + 1 >= end ? (word(i) & 0xffffu) | 0xff800000u : word(i);
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float top() const {
        const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
        return fmaxf(f.x, f.y);
    }
};

__device__ __forceinline__ unsigned long long key_of(float x, int token) {
    return (unsigned long long)order_of(x + 0.0f) << 32 | (0xffffffffu - (uint32_t)token);
}

// The K largest of some units where many tie, or are above the threshold: the K-th largest logit is found bit by
// bit; those above it are fewer than K, and of what ties with it the first K in the tokens' order are taken, piece by piece.
// The units are read again for it (from L2). They go behind the `kept` in buf; returns how many there are with those.
template <typename T>
__device__ __noinline__ int exactly_largest(const T* row, int first, int pieces, int V, int K, unsigned long long* buf, int kept, int* count,
                                            int* scan) {
    using P = Piece<T>;
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
        token = first + i * BS_THREADS * P::VEC + e;
        if ((unsigned)token >= (unsigned)V) return false;
        x = order_of(to_float(row[token]) + 0.0f);
        return true;
    };
    int token;
    uint32_t x, t = 0u;
    for (int bit = 31; bit >= P::LOWEST_BIT; bit--) {
        const uint32_t tried = t | (1u << bit);
        int mine = 0;
        for (int i = 0; i < pieces; i++)
            for (int e = 0; e < P::VEC; e++) mine += read(i, e, token, x) && x >= tried;
        if (sum(mine) >= K) t = tried;
    }
    t = filled(t, P::LOWEST_BIT);
    __syncthreads();
    if (threadIdx.x == 0) *count = kept;
    __syncthreads();
    auto push = [&](uint32_t x, int token) {
        const int slot = atomicAdd(count, 1);
        if (slot < BS_CAP) buf[slot] = (unsigned long long)x << 32 | (0xffffffffu - (uint32_t)token);
    };
    int before = 0;
    for (int i = 0; i < pieces; i++) {
        int mine = 0;
        for (int e = 0; e < P::VEC; e++) {
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
        for (int e = 0; e < P::VEC; e++)
            if (read(i, e, token, x) && x == t && rank++ < K) push(x, token);
    }
    __syncthreads();
    return min(*count, BS_CAP);
}

// best[rank] = key for the n keys of buf with a rank below K (all keys are different): four threads a key where they are
// few, a warp where they are more, which share the others.
__device__ __forceinline__ void rank_keys(const unsigned long long* buf, int n, int K, unsigned long long* best) {
    if (n <= 64) {
        static_assert(BS_THREADS == 4 * 64, "four threads a key");
        if ((int)(threadIdx.x & ~31u) >= 4 * n) return;                 // (whole warps)
        const int i = min((int)threadIdx.x / 4, n - 1);
        const unsigned long long key = buf[i];
        int above = 0;
#pragma unroll 4
        for (int k = threadIdx.x & 3; k < n; k += 4) above += buf[k] > key;
        above += __shfl_xor_sync(FULL, above, 1);
        above += __shfl_xor_sync(FULL, above, 2);
        if ((threadIdx.x & 3) == 0 && (int)threadIdx.x / 4 < n && above < K) best[above] = key;
        return;
    }
    for (int i = threadIdx.x / 32; i < n; i += BS_THREADS / 32) {
        const unsigned long long key = buf[i];
        int above = 0;
        for (int k = lane_id(); k < n; k += 32) above += buf[k] > key;
        above = __reduce_add_sync(FULL, above);
        if (above < K && lane_id() == 0) best[above] = key;
    }
}

// APART: rows begin off 16-byte boundaries.
template <typename T, bool APART>
__global__ void __launch_bounds__(BS_THREADS, BS_CTAS) beam_rows_kernel(const __grid_constant__ BeamArgs a) {
    using P = Piece<T>;
    extern __shared__ __align__(16) uint4 ring[];                      // [BS_RING][BS_STAGE]
    __shared__ unsigned long long buf[BS_CAP], best[BS_MAX_K];
    __shared__ float2 sums[BS_CHECK][BS_THREADS / 32];                 // of the units since the last look, a warp's share each
    __shared__ uint32_t groups[BS_GROUPS], threshold;
    __shared__ int count, scan[BS_THREADS / 32];
    constexpr float LOG2E = 1.44269504088896340736f;
    constexpr int STEP = BS_THREADS * P::VEC, UNIT = BS_HELD * STEP;   // tokens between a thread's pieces, and of a unit
    const int warp = threadIdx.x / 32;
    pdl_trigger();
    const int begin = (int)blockIdx.x * a.each + min((int)blockIdx.x, a.longer), end = begin + a.each + ((int)blockIdx.x < a.longer);
    long long row = begin / a.units;
    int u = begin - (int)row * a.units;
    // tokens from the last 16-byte boundary at or before the row to its first
    auto skew_of = [&](long long r) { return APART ? (int)(r * a.V % P::VEC) : 0; };

    // the loading walk: a unit at a time, a thread the pieces at its places from the boundary on (APART: and one behind all)
    const T* ld_base = static_cast<const T*>(a.logits) + row * a.V;    // token t's logit: base[t]
    long long ld_row = row;
    int ld_left = end - begin, ld_u = u, ld_skew = skew_of(row), ld_stage = 0;
    auto issue = [&]() {
        if (ld_left > 0) {
            ld_left--;
            const int t = ld_u * UNIT + (int)threadIdx.x * P::VEC - ld_skew;
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + ld_stage * BS_STAGE + threadIdx.x);
            // what lies behind the logits is zeros and not read, what lies behind the row is not copied
            auto some = [&](int i) {
                if (t + i * STEP >= a.V) return;
                const long long left = a.count - ld_row * a.V - (t + i * STEP);
                const int bytes = APART ? (int)min(16ll, left * (long long)sizeof(T)) : 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * BS_THREADS * 16), "l"(ld_base + t + i * STEP), "r"(bytes) : "memory");
            };
            if ((ld_u + 1) * UNIT <= a.V) {
#pragma unroll
                for (int i = 0; i < BS_HELD; i++)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * BS_THREADS * 16), "l"(ld_base + t + i * STEP) : "memory");
            } else {
#pragma unroll 1
                for (int i = 0; i < BS_HELD; i++) some(i);
            }
            if (APART && threadIdx.x == 0) some(BS_HELD);
            if (++ld_u == a.units) {
                ld_u = 0;
                ld_row++;
                ld_base += a.V;
                ld_skew = skew_of(ld_row);
            }
        }
        ld_stage = ld_stage + 1 == BS_RING ? 0 : ld_stage + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < BS_RING; i++) issue();
    int stage = 0;
    const T* base = static_cast<const T*>(a.logits) + row * a.V;

    for (int at = begin; at < end; row++, base += a.V, u = 0) {
        const int u0 = u, u1 = min(a.units, u + (end - at)), skew = skew_of(row);
        at += u1 - u;
        float least = -INFINITY;
        int kept = 0, looked = 0;                                      // in buf at the last look, and units before it
        for (; u < u1; u++) {
            asm volatile("cp.async.wait_group %0;" ::"n"(BS_RING - 1) : "memory");
            if (APART) __syncthreads();                                // (a thread's piece is of two threads' copies)
            const int token = u * UNIT + (int)threadIdx.x * P::VEC;    // of the thread's first piece's first element
            const uint4* const mine = ring + stage * BS_STAGE + threadIdx.x;
            auto read = [&](P& q, int i) {
                if (APART) q.put_from(mine + i * BS_THREADS, skew);
                else q.put(mine[i * BS_THREADS]);
            };
            P p[BS_HELD];
#pragma unroll
            for (int i = 0; i < BS_HELD; i++) read(p[i], i);
            if ((u + 1) * UNIT > a.V) {
#pragma unroll
                for (int i = 0; i < BS_HELD; i++) {                    // (cutting what is whole or absent word by word, too: 30.6 us in place of 24.7)
                    if (APART) p[i].cut(a.V - (token + i * STEP));
                    else if (token + i * STEP >= a.V) p[i].cut(0);
                }
            }
            float tops[BS_HELD], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < BS_HELD; i++) {
                tops[i] = p[i].top();
                top = fmaxf(top, tops[i]);
            }
            if (u == u0) {
                // the first threshold, by the first warp while the others sum
                float four = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                four = fmaxf(four, __shfl_xor_sync(FULL, four, 2));
                if ((threadIdx.x & 3) == 0) groups[threadIdx.x / 4] = order_of(four);
                if (threadIdx.x == 0) count = 0;
                __syncthreads();
                if (warp == 0) {
                    const uint32_t t = kth_largest(groups[lane_id()], groups[lane_id() + 32], a.K, 12);
                    if (lane_id() == 0) threshold = t;
                }
            }
            // the unit's sum, each thread's relative to its own maximum (where that is -inf: 0, or NaN if there is one), then the
            // warp's, in an order that is the same for all units
            {
                const float sub = top == -INFINITY ? 0.0f : -top;
                const Two minus(sub, sub), log2e(LOG2E, LOG2E);
                Two sum0(0.0f, 0.0f), sum1(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < BS_HELD; i++)
#pragma unroll
                    for (int e = 0; e < P::VEC; e += 2)
                        (e & 2 ? sum1 : sum0).add_pow2(p[i].at(e), p[i].at(e + 1), minus, log2e);
                sum0 += sum1;
                float s0, s1;
                sum0.get(s0, s1);
                const float high = of_order(__reduce_max_sync(FULL, order_of(top)));
                float sum = s0 + s1;
                if (top != -INFINITY) sum *= pow2((top - high) * LOG2E);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
                if (lane_id() == 0) sums[u - u0 - looked][warp] = make_float2(high, sum);
            }
            if (u == u0) {
                __syncthreads();
                least = of_order(threshold);
            }
            // (the few pieces that hold one are read again: a loop's code, not eight pieces' in line)
            unsigned hits = 0u;
#pragma unroll
            for (int i = 0; i < BS_HELD; i++) hits |= (unsigned)(tops[i] >= least) << i;
            while (hits) {
                const int i = __ffs(hits) - 1, t = token + i * STEP;
                hits &= hits - 1;
                P q;
                read(q, i);
                unsigned found = 0u;
#pragma unroll
                for (int e = 0; e < P::VEC; e++) found |= (unsigned)(q.at(e) >= least) << e;
                while (found) {
                    const int e = __ffs(found) - 1;
                    found &= found - 1;
                    if ((unsigned)(t + e) >= (unsigned)a.V) continue;
                    const int to = atomicAdd(&count, 1);
                    if (to < BS_CAP) buf[to] = key_of(q.pick(e), t + e);
                }
            }
            if (APART) __syncthreads();
            issue();
            stage = stage + 1 == BS_RING ? 0 : stage + 1;
            const bool more = u + 1 < u1;
            const int done = u - u0 + 1;                               // units of the row; looked at after 2, 8, 24, ... of them
            if (more && done != 2 && done != 8 && done - looked < BS_CHECK) continue;
            // every few units: the K largest so far in order, the last of them the threshold
            __syncthreads();
            int n = count;
            if ((int)threadIdx.x < done - looked) {                    // the units' sums, of the warps in their order
                const float2* const x = sums[threadIdx.x];
                float high = -INFINITY, v = 0.0f;
#pragma unroll
                for (int w = 0; w < BS_THREADS / 32; w++) high = fmaxf(high, x[w].x);
#pragma unroll
                for (int w = 0; w < BS_THREADS / 32; w++) v += x[w].x == -INFINITY ? x[w].y : x[w].y * pow2((x[w].x - high) * LOG2E);
                a.part[row * a.units + u0 + looked + threadIdx.x] = make_float2(high, v);
            }
            __syncthreads();                                           // (nobody adds to it before all have read it)
            if (n > BS_CAP) {
                n = exactly_largest<T>(base, token - (done - looked - 1) * UNIT, (done - looked) * BS_HELD, a.V, a.K, buf, kept, &count, scan);
            }
            rank_keys(buf, n, a.K, best);
            n = min(n, a.K);
            __syncthreads();
            if ((int)threadIdx.x < n) buf[threadIdx.x] = best[threadIdx.x];
            if (threadIdx.x == 0) count = n;
            // (what ties with it comes later in the row, and behind it: the next number up is the least that counts)
            if (n == a.K) least = of_order((uint32_t)(best[n - 1] >> 32) + 1u);
            __syncthreads();
            kept = n;
            looked = done;
        }
        const long long to = blockIdx.x + row;
        if ((int)threadIdx.x < a.K) a.list[to * a.K + threadIdx.x] = (int)threadIdx.x < kept ? buf[threadIdx.x] : 0ull;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A number as the sum of two floats, the first the sum rounded; where that is not finite, the second is 0.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair pair_of(float x, float y) {            // x + y exactly (Knuth's two-sum)
    const float h = __fadd_rn(x, y), z = __fsub_rn(h, x);
    return {h, isfinite(h) ? __fadd_rn(__fsub_rn(x, __fsub_rn(h, z)), __fsub_rn(y, z)) : 0.0f};
}
__device__ __forceinline__ Pair plus(Pair x, float y) {
    const Pair s = pair_of(x.h, y);
    const float l = __fadd_rn(s.l, x.l), h = __fadd_rn(s.h, l);
    return {h, isfinite(h) ? __fsub_rn(l, __fsub_rn(h, s.h)) : 0.0f};
}
__device__ __forceinline__ Pair plus(Pair x, Pair y) {
    const Pair s = pair_of(x.h, y.h);
    const float l = __fadd_rn(s.l, __fadd_rn(x.l, y.l)), h = __fadd_rn(s.h, l);
    return {h, isfinite(h) ? __fsub_rn(l, __fsub_rn(h, s.h)) : 0.0f};
}

// ln of a normal positive number: ln(2^k f) = k ln 2 + 2 atanh z with f in [0.7, 1.42), z = (f - 1) / (f + 1) and the series of
// atanh. Only k ln 2 and 2 z are taken in two floats: the rest is below 2^-8 and the series ends below 2^-35.
__device__ __forceinline__ Pair ln(Pair x) {
    const uint32_t u = __float_as_uint(x.h);
    int k = (int)(u >> 23) - 127;
    float f = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
    if (f > 1.41421356f) {
        f *= 0.5f;
        k++;
    }
    const float n = __fsub_rn(f, 1.0f);                                // exact
    const Pair d = pair_of(f, 1.0f);
    const float z = __fdiv_rn(n, d.h);
    const float zl = __fdiv_rn(__fsub_rn(__fmaf_rn(-z, d.h, n), __fmul_rn(z, d.l)), d.h);
    const float w = z * z;
    const float rest = z * w * (2.0f / 3 + w * (2.0f / 5 + w * (2.0f / 7 + w * (2.0f / 9 + w * (2.0f / 11 + w * (2.0f / 13))))));
    // ln 2 = 0x1.62e4p-1 + ...: 16 bits, whose product with k is exact, and what is left
    const Pair a = pair_of(__fmul_rn((float)k, 0x1.62e4p-1f), 2.0f * z);
    const float l = a.l + ((float)k * (float)(0.69314718055994530942 - 0x1.62e4p-1) + (2.0f * zl + rest + x.l / x.h));
    const float h = __fadd_rn(a.h, l);
    return {h, __fsub_rn(l, __fsub_rn(h, a.h))};
}

struct Joined {
    unsigned long long best[BS_MAX_K];
    int best_at[BS_MAX_K];
    Pair lse[BS_MAX_W];              // of a beam that lives
    float score[BS_MAX_W], off[BS_MAX_W];
    int first[BS_MAX_W], parts[BS_MAX_W];
    int state[BS_MAX_W];             // 0: lives, 1: done, 2: has no candidate
    uint32_t low[BS_JOIN], threshold;
    int count;
    unsigned long long v[BS_JOIN * BS_EACH * 2 + BS_MAX_K];
    int at[BS_JOIN * BS_EACH * 2 + BS_MAX_K];
};

__global__ void __launch_bounds__(BS_JOIN) beam_join_kernel(const __grid_constant__ BeamArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Joined& s = *reinterpret_cast<Joined*>(raw);
    const long long row0 = (long long)blockIdx.x * a.W;
    const int lists = a.W * a.segments, warp = threadIdx.x / 32;
    constexpr int TOGETHER = BS_JOIN / 32 * BS_EACH;
    // (the scores were there before the first kernel began, which this one runs beside)
    if ((int)threadIdx.x < a.W) {
        // the block that has unit f
        auto block_of = [&](int f) {
            const int border = a.longer * (a.each + 1);
            return f < border ? f / (a.each + 1) : a.longer + (f - border) / a.each;
        };
        const long long row = row0 + threadIdx.x;
        const int f = (int)row * a.units, g0 = block_of(f), g1 = block_of(f + a.units - 1);
        s.first[threadIdx.x] = g0;
        s.parts[threadIdx.x] = g1 - g0 + 1;
        s.score[threadIdx.x] = a.scores[row];
        s.state[threadIdx.x] = a.done && a.done[row];
    }
    // the beam and the part of list l, as far as a thread looks at them together
    int list_w[BS_EACH], list_part[BS_EACH];
    auto place = [&](int l0) {
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            const int l = l0 + e * (BS_JOIN / 32) + warp;
            list_w[e] = l < lists ? l / a.segments : -1;
            list_part[e] = l - list_w[e] * a.segments;
        }
    };
    place(0);
    __syncthreads();
    pdl_wait();
    // the first lists are on their way while the sums are joined: entries lane and lane + 32
    unsigned long long ahead[BS_EACH][2];
    auto fetch = [&]() {
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            ahead[e][0] = ahead[e][1] = 0ull;
            const int w = list_w[e], part = list_part[e];
            if (w >= 0 && part < s.parts[w]) {
                const unsigned long long* const list = a.list + (row0 + w + s.first[w] + part) * a.K;
                if ((int)lane_id() < a.K) ahead[e][0] = __ldcg(list + lane_id());
                if ((int)lane_id() + 32 < a.K) ahead[e][1] = __ldcg(list + lane_id() + 32);
            }
        }
    };
    fetch();
    for (int w0 = 0; w0 < a.W; w0 += BS_JOIN / BS_BEAM) {
        const int w = w0 + threadIdx.x / BS_BEAM, l = threadIdx.x % BS_BEAM;
        const int units = w < a.W ? a.units : 0;
        const float2* part = a.part + (row0 + w) * a.units;
        const float2 mine = l < units ? __ldcg(part + l) : make_float2(-INFINITY, 0.0f);
        float m = mine.x;
        for (int c = l + BS_BEAM; c < units; c += BS_BEAM) m = fmaxf(m, __ldcg(part + c).x);
#pragma unroll
        for (int o = BS_BEAM / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        Pair sum = {0.0f, 0.0f};
        for (int c = l; c < units; c += BS_BEAM) {
            const float2 x = c == l ? mine : __ldcg(part + c);
            sum = plus(sum, x.x == -INFINITY || x.x == m ? x.y : x.y * expf(x.x - m));
        }
#pragma unroll
        for (int o = BS_BEAM / 2; o > 0; o >>= 1)
            sum = plus(sum, Pair{__shfl_xor_sync(FULL, sum.h, o), __shfl_xor_sync(FULL, sum.l, o)});
        if (l == 0 && w < a.W) {
            // (the sum is at least one, where it is one of numbers)
            const float score = s.score[w];
            const bool fine = isfinite(score), done = s.state[w], lives = sum.h >= 1.0f && isfinite(sum.h) && isfinite(m);
            const Pair lse = lives ? plus(ln(sum), m) : Pair{0.0f, 0.0f};
            s.lse[w] = lse;
            s.off[w] = score - lse.h;
            s.state[w] = done && fine ? 1 : !done && fine && lives && isfinite(lse.h) ? 0 : 2;
        }
    }
    __syncthreads();

    // entry k of a beam's list, its key read: the token, and x, its logit (a done or dead beam's, in the place of its
    // first list: its score, or -inf); false: none
    auto entry = [&](int w, int part, int k, unsigned long long key, int& token, float& x) {
        if (s.state[w] == 0) {
            if (key == 0ull) return false;
            token = (int)(0xffffffffu - (uint32_t)key);
            x = of_order((uint32_t)(key >> 32));
            return true;
        }
        if (part > 0 || k >= a.K || k >= a.V) return false;
        token = k;
        x = -INFINITY;
        if (s.state[w] == 1) {
            token = k == 0 ? a.pad : k - 1 < a.pad ? k - 1 : k;
            if (k == 0) x = s.score[w];
        }
        return true;
    };
    // its value as a number in the values' order
    auto value = [&](int w, float x) {
        Pair v = {x, 0.0f};
        if (x != -INFINITY && s.state[w] == 0) {
            const Pair lse = s.lse[w];
            v = plus(plus(pair_of(x, -lse.h), -lse.l), s.score[w]);
        }
        return (unsigned long long)order_of(v.h + 0.0f) << 32 | order_of(v.l + 0.0f);
    };
    int kept = 0;
    for (int l0 = 0; l0 < lists; l0 += TOGETHER) {
        if (l0) {
            place(l0);
            fetch();
        }
        float hi[BS_EACH][2];
        float low = -INFINITY;                                       // the largest lower bound of the thread's entries
        if (threadIdx.x == 0) s.count = 0;
#pragma unroll
        for (int e = 0; e < BS_EACH; e++) {
            hi[e][0] = hi[e][1] = __uint_as_float(0x7fc00000u);
            const int w = list_w[e];
            if (w < 0) continue;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                int token;
                float x;
                if (!entry(w, list_part[e], lane_id() + 32 * h, ahead[e][h], token, x)) continue;
                float lo = x;
                hi[e][h] = x;
                if (s.state[w] == 0 && x != -INFINITY) {
                    // |value - v| < 2^-22 (|off| + |x|) + |lse| 2^-24 with the roundings of off, of lse and of the sum
                    const float v = s.off[w] + x, eps = (fabsf(s.off[w]) + fabsf(x) + fabsf(s.lse[w].h)) * 0x1p-21f;
                    const bool fine = isfinite(v) && isfinite(eps);
                    lo = fine ? v - eps : -INFINITY;
                    hi[e][h] = fine ? v + eps : INFINITY;
                }
                low = fmaxf(low, lo);
            }
        }
        if ((int)threadIdx.x < kept) {
            const float best = of_order((uint32_t)(s.best[threadIdx.x] >> 32));
            low = fmaxf(low, best - fabsf(best) * 0x1p-22f);
        }
        s.low[threadIdx.x] = order_of(low);
        __syncthreads();
        if (warp == 0) {
            // the K-th largest of the threads', or a number a little below it: 14 bits below the first in which those above
            // -inf differ
            constexpr uint32_t NONE = 0x007fffffu;
            uint32_t x[BS_JOIN / 32], any = 0u, all = 0xffffffffu;
            int some = 0;
#pragma unroll
            for (int i = 0; i < BS_JOIN / 32; i++) {
                x[i] = s.low[i * 32 + lane_id()];
                if (x[i] > NONE) {
                    any |= x[i];
                    all &= x[i];
                }
                some += __popc(__ballot_sync(FULL, x[i] > NONE));
            }
            any = __reduce_or_sync(FULL, any);
            const uint32_t differ = any ^ __reduce_and_sync(FULL, all);
            uint32_t t = NONE;
            if (some >= a.K) {
                const int top = differ ? 31 - __clz(differ) : 0;
                t = top == 31 ? 0u : any >> (top + 1) << (top + 1);
                for (int bit = top; bit >= max(0, top - 14); bit--) {
                    const uint32_t tried = t | (1u << bit);
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < BS_JOIN / 32; i++) n += __popc(__ballot_sync(FULL, x[i] >= tried));
                    if (n >= a.K) t = tried;
                    if (n == a.K) break;
                }
            }
            if (lane_id() == 0) s.threshold = max(t, NONE);
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
        for (int e = 0; e < BS_EACH; e++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (!(hi[e][h] >= least)) continue;
                int token;
                float x;
                if (entry(list_w[e], list_part[e], lane_id() + 32 * h, ahead[e][h], token, x))
                    push(value(list_w[e], x), list_w[e] * a.V + token);
            }
        __syncthreads();
        const int n = s.count;
        for (int i = warp; i < n; i += BS_JOIN / 32) {
            const unsigned long long v = s.v[i];
            const int at = s.at[i];
            int above = 0;
            for (int k = lane_id(); k < n; k += 32) above += s.v[k] > v || (s.v[k] == v && s.at[k] < at);
            above = __reduce_add_sync(FULL, above);
            if (above < a.K && lane_id() == 0) {
                s.best[above] = v;
                s.best_at[above] = at;
            }
        }
        kept = min(n, a.K);
        __syncthreads();
    }
    if ((int)threadIdx.x < a.K) {
        const long long o = (long long)blockIdx.x * a.K + threadIdx.x;
        const int at = s.best_at[threadIdx.x], w = at / a.V;
        a.out_scores[o] = of_order((uint32_t)(s.best[threadIdx.x] >> 32));
        a.parents[o] = (int)(row0 + w);
        a.tokens[o] = at - w * a.V;
    }
}

// Units of a row: so many 16-byte pieces from its first logit on.
template <typename T>
int units_of(int V) {
    constexpr int UNIT = BS_THREADS * BS_HELD * Piece<T>::VEC;
    return (V + UNIT - 1) / UNIT;
}

bool refused(int N, int W, int V, int K) {
    return N < 0 || W < 1 || W > BS_MAX_W || V < 1 || V >= (1 << 24) || (long long)N * W >= (1 << 24) || K < 1 ||
           K > BS_MAX_K || (long long)K > (long long)W * V || (long long)N * W * units_of<float>(V) >= (1ll << 31);
}

size_t slots(int N, int W) { return (size_t)N * W + BS_MAX_CTAS; }

template <typename T, bool APART>
moe_status launch(BeamArgs a, int N, cudaStream_t s) {
    static moe_host::PerDevice ring, smem, sms_of;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const int sms = sms_of.get(dev, [&] {
        int n = 0;
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
    });
    if (sms == 0) return MOE_ERR_CUDA;
    a.units = units_of<T>(a.V);
    const int total = N * a.W * a.units, most = sms * BS_CTAS < BS_MAX_CTAS ? sms * BS_CTAS : BS_MAX_CTAS;
    a.ctas = total < most ? total : most;
    a.each = total / a.ctas;
    a.longer = total % a.ctas;
    // the stretches that a row's units can lie in
    const int parts = (a.units - 1 + a.each - 1) / a.each + 1;
    a.segments = parts < a.units ? parts : a.units;
    a.count = (long long)N * a.W * a.V;
    constexpr int RING = BS_RING * BS_STAGE * sizeof(uint4);
    if (!moe_host::allow_smem(beam_rows_kernel<T, APART>, RING, ring)) return MOE_ERR_CUDA;
    beam_rows_kernel<T, APART><<<a.ctas, BS_THREADS, RING, s>>>(a);
    const moe_status st = moe_host::launch_status();
    if (st != MOE_OK) return st;
    if (!moe_host::allow_smem(beam_join_kernel, sizeof(Joined), smem) ||
        moe_host::launch_pdl(beam_join_kernel, dim3(N), dim3(BS_JOIN), sizeof(Joined), s, a) != cudaSuccess)
        return MOE_ERR_CUDA;
    return moe_host::launch_status();
}

template <typename T>
moe_status launch_of(const BeamArgs& a, int N, cudaStream_t s) {
    return a.V % Piece<T>::VEC ? launch<T, true>(a, N, s) : launch<T, false>(a, N, s);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_beam_select_workspace_size(int N, int W, int V, int K) {
    using namespace moe;
    if (refused(N, W, V, K)) return 0;
    return slots(N, W) * K * sizeof(unsigned long long) + (size_t)N * W * units_of<float>(V) * sizeof(float2);
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
    BeamArgs a = {logits, scores, done, pad, W, V, K, 0, 0, 0, 0, 0, 0, out_scores, parents, tokens, nullptr, nullptr};
    a.list = static_cast<unsigned long long*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + slots(N, W) * K * sizeof(unsigned long long));
    return dtype == MOE_F32 ? launch_of<float>(a, N, moe_host::as_stream(stream)) : launch_of<__nv_bfloat16>(a, N, moe_host::as_stream(stream));
}
