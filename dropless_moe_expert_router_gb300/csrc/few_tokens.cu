// few_tokens.cu -- the whole MoE layer for a few tokens (a decoding step): moe_layer_few_tokens. Three
// kernels: routing (and x's quantisation), up projection, down projection and combine.
//
// For every valid route (t, k) with expert e = ids[t,k]:
//   h = silu(x[t] W1[e]) * (x[t] W3[e]);   y[t] = bf16( sum_k p[t,k] (h W2[e]) )
// Every weight of the chosen experts is read once and used for the few tokens that chose
// them, so the time is the weights' bytes over the memory's rate plus a part that does not shrink with them: 10 to
// 15 us from the routing through two dependent kernels' starts and joins with few experts, about 23 us with 2,304
// (routing takes 9 us of its own there, against 4 to 5; how the rest divides between the plans, the kernels' change
// and the joins is not measured). Measured on a GPU that copies 6.78 TB/s (whole layer, SM clock 2070 MHz; the
// share is that of the weights' bytes at that rate):
//   1 token, 8 experts, top-2, 4096 x 14336, bf16         114-120 us   0.87-0.91   (0.70 GB)
//   32 tokens of the same (all experts)                   408-425 us   0.98-1.0    (2.8 GB)
//   8 tokens, 32 experts, top-4, 7168 x 2048, MXFP8       151-168 us   0.84-0.93   (0.95 GB)
//   5 tokens, 2,304 experts, top-36, 512 x 512, bf16        62-66 us   0.61-0.65   (0.27 GB)
//   1 token, 8 experts, top-2, 256 x 512, bf16              14-15 us   starts and joins (1.6 MB)
#include "common.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int FEW_TMAX = 64;         // tokens
constexpr int FEW_KMAX = 128;        // routes per token
constexpr int FEW_ROUTES = 4096;     // T * K
constexpr int FEW_EMAX = 8192;       // experts

// ---------------------------------------------------------------------------
// First kernel. CTA t < T: token t's selection (unless the caller gave ids and probs). MXFP8: the CTAs
// after those quantise x row-wise 1x32, PREP_QUANT elements of a row each. 4 to 5 us (9 with 2,304 experts), all
// of it latency: hence counting and ranking, a fixed number of steps, in place of K rounds of a maximum each.
//
// Selection: a thread holds V logits as order-preserving keys (expert i * 256 + thread). Up to 256
// experts, each logit's rank is counted directly against the row. Above, the K-th largest of the
// threads' own largest keys bounds the row's K-th largest from below; the keys at or above it,
// normally a few more than K, are listed and ranked among themselves. A row with more than PREP_CAND
// of them (many equal logits) takes an exact search instead: the K-th largest key by its 32 bits, two a
// step, then the keys above it and the lowest-index ones equal to it.
// ---------------------------------------------------------------------------
constexpr int PREP_THREADS = 256;
constexpr int PREP_WARPS = PREP_THREADS / 32;
constexpr int PREP_CAND = 256;
constexpr int PREP_QUANT = PREP_THREADS * 8;

struct PrepSmem {
    uint4 key[PREP_THREADS / 4];            // each thread's largest key
    unsigned long long list[PREP_CAND];     // key, then the complement of the expert's index
    unsigned bound;
    unsigned cnt[2];
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

__device__ __forceinline__ unsigned long long list_entry(unsigned key, int e) {
    return ((unsigned long long)key << 32) | (unsigned)~e;
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
    int T, H, E, K;
    void* ids;
    bool i16, renorm;
    float* probs;
    uint8_t* xq;              // MXFP8: codes [T, H] and scales [T, H / 32] of x; else null
    uint8_t* xs;
    unsigned* count;          // the second kernel's counters, zeroed here
    int n_count;
};

// The K largest keys of the row (lower index first among equals) into the list, whatever the ties.
__device__ __noinline__ void prep_exact(const float* row, int E, int K, PrepSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31;
    // (few rows come here: the keys are made anew in each step)
    auto count = [&](unsigned* to, auto pred) {
        unsigned c = 0u;
        for (int e = tid; e < E; e += PREP_THREADS) c += pred(order_key(__ldg(row + e)), e);
        c = __reduce_add_sync(FULL, c);
        if (lane == 0 && c) atomicAdd(to, c);
    };
    __syncthreads();                  // (every thread has read the list's length)
    if (tid < 2) sm.cnt[tid] = 0u;
    if (tid == 0) sm.n = 0;
    __syncthreads();
    // the largest bound with at least K keys at or above it: the K-th largest key
    unsigned kth = 0u;
    int step = 0;
    for (int sh = 31; sh >= 0; sh--, step ^= 1) {
        const unsigned bound = kth | (1u << sh);
        count(&sm.cnt[step], [&](unsigned k, int) { return k >= bound; });
        __syncthreads();
        if (sm.cnt[step] >= (unsigned)K) kth = bound;
        if (tid == 0) sm.cnt[step ^ 1] = 0u;
        __syncthreads();
    }
    // how many of the keys equal to it belong to the K largest: those with the lowest expert
    // indices, the index bound by bisection
    count(&sm.cnt[step], [&](unsigned k, int) { return k > kth; });
    __syncthreads();
    const unsigned ties = (unsigned)K - sm.cnt[step];
    int lo = 0, hi = E - 1;           // smallest b with at least `ties` equal keys at indices <= b
    while (lo < hi) {
        step ^= 1;
        __syncthreads();
        if (tid == 0) sm.cnt[step] = 0u;
        __syncthreads();
        const int mid = (lo + hi) >> 1;
        count(&sm.cnt[step], [&](unsigned k, int e) { return k == kth && e <= mid; });
        __syncthreads();
        if (sm.cnt[step] >= ties) hi = mid;
        else lo = mid + 1;
    }
    for (int e = tid; e < E; e += PREP_THREADS) {
        const unsigned k = order_key(__ldg(row + e));
        if (k > kth || (k == kth && e <= lo)) {
            const int pos = atomicAdd(&sm.n, 1);
            if (pos < PREP_CAND) sm.list[pos] = list_entry(k, e);     // (NaN logits aside, exactly K come here)
        }
    }
    __syncthreads();
}

// The sum of num over the chosen (rank >= 0) in the order of their ranks: which thread has which entry of the list is
// chance. (Inlined, with its barrier, it made the whole kernel slower: the 2,304-expert layer 63.5 -> 66.4 us.)
__device__ __noinline__ float prep_ordered_sum(float num, int rank, int K, PrepSmem& sm) {
    float* by_rank = reinterpret_cast<float*>(sm.key);        // (every thread is done with the keys)
    if (rank >= 0) by_rank[rank] = num;
    __syncthreads();
    return prep_reduce<false>((int)threadIdx.x < K ? by_rank[threadIdx.x] : 0.0f, sm.red[1]);
}

template <int V>
__device__ void prep_route(const PrepArgs& p, int t, PrepSmem& sm) {
    const int tid = threadIdx.x;
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
    if (tid == 0) {
        sm.n = 0;
        sm.bound = 0u;
    }
    m = prep_reduce<true>(m, sm.red[0]);
    float den = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < V; i++)
            if (key[i]) den += expf(key_value(key[i]) - m);
        den = prep_reduce<false>(den, sm.red[1]);
    }
    // the row's largest key of each thread (V = 1: its only one), ranked against the others'
    unsigned top = key[0];
#pragma unroll
    for (int i = 1; i < V; i++) top = max(top, key[i]);
    reinterpret_cast<unsigned*>(sm.key)[tid] = top;
    __syncthreads();
    int above = 0, equal = 0;             // V = 1: equal keys before this one; else all of them
#pragma unroll 4
    for (int j = 0; j < (min(p.E, PREP_THREADS) + 3) / 4; j++) {      // (keys past E are 0, below all)
        const uint4 q = sm.key[j];
        const unsigned k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 4; u++) {
            above += k[u] > top;
            equal += k[u] == top && (V > 1 || 4 * j + u < tid);
        }
    }
    int n = p.K;              // length of the list
    int rank = above + equal;
    unsigned long long mine = list_entry(top, tid);
    bool chosen = V == 1 && tid < p.E && rank < p.K;
    if (V > 1) {
        if (above < p.K && p.K <= above + equal) sm.bound = top;      // (the same from every such thread)
        __syncthreads();
        const unsigned bound = sm.bound;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (key[i] >= bound && i * PREP_THREADS + tid < p.E) {
                const int pos = atomicAdd(&sm.n, 1);
                if (pos < PREP_CAND) sm.list[pos] = list_entry(key[i], i * PREP_THREADS + tid);
            }
        __syncthreads();
        n = sm.n;
        if (n > PREP_CAND) {
            prep_exact(row, p.E, p.K, sm);
            n = p.K;
        }
        // ranks within the list; the first K are the selection
        if (tid < n) {
            mine = sm.list[tid];
            rank = 0;
#pragma unroll 8
            for (int i = 0; i < n; i++) rank += sm.list[i] > mine;
            chosen = rank < p.K;
        }
    }
    const unsigned k = (unsigned)(mine >> 32);
    const int e = (int)~(unsigned)mine;
    const float num = chosen ? expf(key_value(k) - m) : 0.0f;
    if (p.renorm) den = V > 1 ? prep_ordered_sum(num, chosen ? rank : -1, p.K, sm) : prep_reduce<false>(num, sm.red[1]);
    if (chosen) {
        const long long o = (long long)t * p.K + rank;
        if (p.i16) static_cast<int16_t*>(p.ids)[o] = (int16_t)e;
        else static_cast<int32_t*>(p.ids)[o] = e;
        p.probs[o] = num / den;
    }
}

template <int V>
__global__ void __launch_bounds__(PREP_THREADS) few_prep_kernel(PrepArgs p) {
    __shared__ PrepSmem sm;
    pdl_trigger();            // the second kernel sets up meanwhile
    const int t = blockIdx.x;
    if (t < p.T) {
        if (t == 0)
            for (int i = threadIdx.x; i < p.n_count; i += PREP_THREADS) p.count[i] = 0u;
        if (p.logits) prep_route<V>(p, t, sm);
        return;
    }
    const int per = (p.H + PREP_QUANT - 1) / PREP_QUANT;
    const int row = (t - p.T) / per, j = ((t - p.T) % per) * PREP_THREADS + threadIdx.x;
    const int H8 = p.H >> 3;
    float f[8];
    bf16x8_to_f32(j < H8 ? __ldg(reinterpret_cast<const uint4*>(p.x + (long long)row * p.H) + j) : make_uint4(0, 0, 0, 0), f);
    int sb;
    const uint2 code = quant8_in_quad(f, &sb);
    if (j < H8) {
        reinterpret_cast<uint2*>(p.xq)[(long long)row * H8 + j] = code;
        if ((threadIdx.x & 3) == 0) p.xs[(long long)row * (p.H >> 5) + (j >> 2)] = (uint8_t)sb;
    }
}

// ---------------------------------------------------------------------------
// The expert MLP and the combine: two kernels, one persistent CTA per SM each.
//
// Every weight row is streamed once, as the A operand (128 rows) of tcgen05.mma; the few tokens
// are the B operand, so a tile's accumulator is [128 weight rows][tokens] in TMEM (with the weights as
// B the M = 128 rows of A would be padding, and a token's worth of MMA would cost as much as 128). The
// weights' bytes bound the kernels: a producer warp keeps a ring of up to FEW_STAGES stages of two 16 KB
// weight tiles in flight per SM. By themselves, from a cold L2: up 470 MB in 80 us (5.9 TB/s; tensor pipe
// 4 % busy at 1 token, 8 % at 32), down 235 MB in 53 us (its start and its joins weigh more), MXFP8 up 424 MB in 76 us.
// MXFP8 comes near a second bound: the MMA warp spends 324 cycles on a k-block's MMAs, 160 on its scale
// copies and about 175 on barriers, 0.33 us per 16 KB, 7.5 TB/s over 152 SMs.
//
// Up: a tile is 64 columns of W1 and the same 64 of W3 of one expert, over all of H; the tokens
//   operand is all of x (T rows, zero rows past them), the chosen tokens' columns are read. h goes
//   to the workspace, the rows of an expert side by side.
// Down: a tile is 128 output columns of W2, over all chosen experts one after the other; a CTA adds
//   p * (its part of h W2) up over the experts in shared memory.
// Either walk (tile, expert, k-block) is cut into gridDim.x equal pieces wherever that beats whole
// tiles, so that any number of experts and tiles keeps every SM busy to the end. CTAs that share a tile
// leave partial sums, and the last to arrive adds them, in the order of the CTAs: the result does
// not depend on who is last.
// The down kernel is launched while the up kernel runs: its CTAs start as SMs fall free, make the
// plan and fill their rings with weights, which depend on the routing alone, and only then wait for h. (One
// kernel with a barrier between the two halves was slower: it has to be launched cooperatively, which
// alone took 3 us longer.)
//
// Warps: 0 TMA producer, 1 TMEM and MMA issue, 2-5 epilogue (one TMEM lane quarter each), 6 (MXFP8)
// the scales: loads a group of k-blocks' scale bytes and rearranges them for tcgen05.cp.
// ---------------------------------------------------------------------------
constexpr int FEW_STAGES = 6;              // most ring stages
constexpr int FEW_KPS = 2;                 // k-blocks in a stage
constexpr int FEW_A_BYTES = 128 * 128;     // a weight tile: 128 rows of 128 bytes
constexpr int FEW_ACC_COLS = 64;           // TMEM columns of one accumulator: tokens
constexpr int FEW_SF_KB = 8;               // MXFP8: k-blocks in a group of scales (4 bytes a row each)
constexpr int FEW_SF_SLOTS = 4;            // groups of scales in flight (short tiles have a group each)
constexpr int FEW_SF_BYTES = FEW_SF_KB * 1024;   // a slot: landed 4 FEW_SF_KB bytes a row, rearranged FEW_SF_KB x (A 512 | B 512)
constexpr int FEW_XCH = 16;                // tokens whose W3 products the epilogue exchanges at a time (tmem_wait16)
constexpr int FEW_MIN_KB = 2;              // k-blocks that a CTA takes at least
constexpr int FEW_GRID_MAX = 256;          // CTAs that the workspace has room for
constexpr int FEW_ONE_JOIN = 512;          // down: most CTAs of a tile x tokens that are joined in one step: one SM reads
                                           // them all (64 tokens, H = 256, 64 experts, F = 1024: 50 us, in two steps 45;
                                           // at 1024 24 tokens, H = 512, F = 2048 take 39.9 us instead of 36.4)
constexpr int FEW_SHARE = 32;              // up: CTAs that share a tile at most (the last to arrive reads all their sums)
constexpr int FEW_JOIN_KB = 8;             // joining partial sums costs about as much as this many k-blocks
constexpr size_t FEW_SMEM_MAX = 227 * 1024;

struct FewArgs {
    const void* ids;
    const float* probs;
    bool i16;
    int T, H, K, E, F;
    int nb;                   // B rows of a stage: T rounded up to 16
    int stages;
    int a_max;                // most experts chosen: min(E, T K)
    void* h;                  // [T K, F] bf16 or E4M3
    uint8_t* hs;              // MXFP8: [T K, F / 32]
    float* part;              // [2 gridDim.x][T][128] partial sums of shared output tiles
    unsigned* count;          // arrivals at shared tiles (down: by tile, H / 128; up: by first CTA, FEW_GRID_MAX) and
                              // at a tile's groups of CTAs (down: by the first one's slot, 2 FEW_GRID_MAX); zeroed before
    __nv_bfloat16* y;
};

// Shared memory past the ring.
struct FewSmem {
    uint64_t full[FEW_STAGES], empty[FEW_STAGES], tfull[2], tempty[2], done;
    uint64_t sf_full[FEW_SF_SLOTS], sf_ready[FEW_SF_SLOTS], sf_empty[FEW_SF_SLOTS];
    uint32_t tmem, abort_flag;
    int A, slots, routes, ticket;
    int scan[2][8];
    float xch[2][FEW_XCH][64];
};

__host__ __device__ constexpr size_t few_up16(size_t v) { return (v + 15) & ~(size_t)15; }

// Bytes of shared memory past the ring: FewSmem, MXFP8 scale slots, output sums, the plan.
__host__ __device__ inline size_t few_fixed_smem(int T, int K, int a_max, bool fp8) {
    return few_up16(sizeof(FewSmem)) + (fp8 ? (size_t)FEW_SF_SLOTS * FEW_SF_BYTES : 0) + (size_t)T * 128 * 4 +
           few_up16((size_t)a_max * 8) + few_up16((size_t)a_max * 4) + few_up16((size_t)(a_max + 1) * 4) +
           few_up16((size_t)T * K * 4);
}

// The chosen experts: id, first row of h, which tokens; and each route's weight.
struct FewPlan {
    const unsigned long long* mask;
    const int* e;
    const int* off;
    const float* w;
    int A;
    int kbs;                  // k-blocks of a tile (down: of all its experts)
    int W;                    // k-blocks of the whole walk
    int unit;                 // it is cut at multiples of this many
    int parts;                // CTAs that take a piece each: base units, the first `more` of them one more
    int base, more;

    __device__ void cut(int n) {
        parts = n;
        base = W / unit / n;
        more = W / unit - base * n;
    }
    // first k-block of CTA c's piece (c >= parts: the end)
    __device__ int begin_of(int c) const { return c >= parts ? W : unit * (base * c + min(c, more)); }
    // the CTA whose piece has k-block w
    __device__ int owner(int w) const {
        const int u = w / unit, longer = more * (base + 1);
        return u < longer ? u / (base + 1) : more + (u - longer) / base;
    }
    // Partial sums have two slots per CTA: 0 for the first tile that it works on, 1 for its last. Of a
    // tile's CTAs only the first (c0) can have it as its last.
    __device__ int slot_of(int c, int tile) const { return 2 * c + (begin_of(c) / kbs != tile); }
};

// A run of k-blocks of one tile: the unit that all warps walk in the same order.
struct FewRun {
    int a;                    // index among the chosen experts
    int tile;                 // up: expert * (F / 64) + 64-column tile of F; down: 128-column tile of H
    int kb0, nkb;
    int row0, row1;           // weight rows of the two 64-row halves
    int brow, bn;             // tokens operand: first row, rows loaded
};

template <bool FP8, bool DOWN>
struct FewWalk {
    const FewArgs& p;
    const FewPlan& pl;
    int at, end;              // k-blocks
    __device__ FewWalk(const FewArgs& p_, const FewPlan& pl_) : p(p_), pl(pl_) {
        at = pl.begin_of(blockIdx.x);
        end = pl.begin_of(blockIdx.x + 1);
    }
    __device__ bool next(FewRun& r) {
        constexpr int BK = FP8 ? 128 : 64;
        if (at >= end) return false;
        const int kbs = (DOWN ? p.F : p.H) / BK;      // of a tile and expert
        const int q = at / kbs;
        r.kb0 = at - q * kbs;
        r.nkb = min(kbs - r.kb0, end - at);
        at += r.nkb;
        if constexpr (DOWN) {
            r.tile = q / pl.A;
            r.a = q - r.tile * pl.A;
            r.row0 = pl.e[r.a] * p.H + r.tile * 128;
            r.row1 = r.row0 + 64;
            r.brow = pl.off[r.a];
            r.bn = (pl.off[r.a + 1] - r.brow + 15) & ~15;
        } else {
            const int ft = p.F / 64;
            r.tile = q;
            r.a = q / ft;
            const int c = (q - r.a * ft) * 64;
            r.row0 = pl.e[r.a] * 2 * p.F + c / 128 * 256 + c % 128;
            r.row1 = r.row0 + 128;
            r.brow = 0;
            r.bn = p.nb;
        }
        return true;
    }
};

// A weight tile, read once by the whole GPU: first to leave L2, so that what the next call needs again
// (the kernels' code, x, the workspace) stays.
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_weights(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%3, %4}], [%2], %5;" ::"r"(ptx::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_addr(bar)), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Whether all 128 epilogue threads say yes: what they decide on is the same in all of them.
__device__ __forceinline__ bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred P, Q;\n setp.ne.b32 P, %1, 0;\n barrier.cta.red.and.pred Q, 1, 128, P;\n"
        " selp.u32 %0, 1, 0, Q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// One TMEM column (dynamic) of this warp's lane quarter.
__device__ __forceinline__ uint32_t tmem_ld_x1(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    return v;
}

// 16 consecutive TMEM columns of this warp's lane quarter.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The loads into r have completed (r passes through, so that no use of it moves ahead of the wait).
__device__ __forceinline__ void tmem_wait16(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// v[j] = the sum over the CTAs i = i0, i0 + di, ... < n of their partial sums of token t0 + j dt (< T): the
// first CTA's at `first`, the others' at `rest`, `stride` apart. UN CTAs' loads in flight.
template <int NT, int UN>
__device__ __forceinline__ void few_add_parts(float4 (&v)[NT], const float4* first, const float4* rest, size_t stride,
                                              int i0, int di, int n, int t0, int dt, int T) {
#pragma unroll
    for (int j = 0; j < NT; j++) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (; i0 < n; i0 += UN * di) {
        float4 u[UN][NT];
#pragma unroll
        for (int k = 0; k < UN; k++) {
            const int i = i0 + k * di;
            const float4* from = i == 0 ? first : rest + stride * (i - 1);
#pragma unroll
            for (int j = 0; j < NT; j++)
                u[k][j] = i < n && t0 + j * dt < T ? __ldcg(from + (t0 + j * dt) * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < UN; k++)
#pragma unroll
            for (int j = 0; j < NT; j++) {
                v[j].x += u[k][j].x;
                v[j].y += u[k][j].y;
                v[j].z += u[k][j].z;
                v[j].w += u[k][j].w;
            }
    }
}

template <bool FP8>
constexpr int few_threads() { return FP8 ? 224 : 192; }

__device__ __forceinline__ int few_id(const FewArgs& p, int r) {
    return p.i16 ? (int)__ldcg(static_cast<const short*>(p.ids) + r) : __ldcg(static_cast<const int*>(p.ids) + r);
}

// The plan, the same in every CTA: experts in ascending order, an expert's tokens in ascending order.
// scratch: 8 E bytes (token masks), 2 E (an expert's index among the chosen) and 2 T K (the routes), in the ring.
// Up: waits for the first kernel, whose the routes are, and then lets the down kernel start, which therefore
// finds them written. (Routes are read past L1, which is not kept in line with the other kernels.)
template <int THREADS, bool DOWN>
__device__ void few_plan(const FewArgs& p, FewSmem& sm, uint8_t* scratch, unsigned long long* s_mask, int* s_e,
                         int* s_off, float* s_w) {
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(scratch);
    uint16_t* index = reinterpret_cast<uint16_t*>(scratch + (size_t)p.E * 8);
    uint16_t* id = index + p.E;
    constexpr uint16_t NONE = 0xffff;
    constexpr int B = 8;              // routes a thread has in flight
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < p.E; e += THREADS) mask[e] = 0ull;
    if (tid == 0) sm.routes = 0;
    __syncthreads();
    if constexpr (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    const int R = p.T * p.K;
    int valid = 0;
    float w_own[B];                   // (down) its first routes' weights
    for (int r0 = tid; r0 < R; r0 += B * THREADS) {
        int e[B];
#pragma unroll
        for (int u = 0; u < B; u++) {
            const int r = r0 + u * THREADS;
            e[u] = r < R ? few_id(p, r) : -1;
            if (DOWN && r0 == tid) w_own[u] = r < R ? __ldcg(p.probs + r) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < B; u++) {
            const int r = r0 + u * THREADS;
            if (r >= R) break;
            const bool ok = e[u] >= 0 && e[u] < p.E;
            id[r] = ok ? (uint16_t)e[u] : NONE;
            if (ok) {
                // (by words: 64-bit atomics on shared memory retry where routes meet)
                atomicOr(reinterpret_cast<unsigned*>(mask + e[u]) + (r / p.K >> 5), 1u << (r / p.K & 31));
                valid++;
            } else if (!DOWN && e[u] != -1 && blockIdx.x == 0) {
                raise_device_error(MOE_DEVERR_BAD_ID);
            }
        }
    }
    if (valid) atomicAdd(&sm.routes, valid);
    __syncthreads();
    // exclusive scan of (chosen, tokens) over the experts, a stretch of them per thread
    const int per = (p.E + THREADS - 1) / THREADS;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    int n = 0, m = 0;
    for (int e = e0; e < e1; e++) {
        const unsigned long long b = mask[e];
        n += b != 0ull;
        m += __popcll(b);
    }
    int sn = n, sm_ = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(FULL, sn, d), c = __shfl_up_sync(FULL, sm_, d);
        if (lane >= d) {
            sn += a;
            sm_ += c;
        }
    }
    if (lane == 31) {
        sm.scan[0][warp] = sn;
        sm.scan[1][warp] = sm_;
    }
    __syncthreads();
    int a = sn - n, o = sm_ - m;
    for (int i = 0; i < warp; i++) {
        a += sm.scan[0][i];
        o += sm.scan[1][i];
    }
    for (int e = e0; e < e1; e++) {
        const unsigned long long b = mask[e];
        if (!b) continue;
        s_mask[a] = b;
        s_e[a] = e;
        s_off[a] = o;
        index[e] = (uint16_t)a;
        a++;
        o += __popcll(b);
    }
    if (tid == THREADS - 1) {
        sm.A = a;
        sm.slots = o;
        s_off[a] = o;
    }
    __syncthreads();
    if (!DOWN) {
        ptx::fence_proxy_async_smem();
        return;
    }
    // each route's weight at its row of h; an expert that a token names more than once has one row,
    // weighted with the sum (in ascending k)
    const bool repeated = sm.slots != sm.routes;
    for (int r0 = tid; r0 < R; r0 += B * THREADS) {
        float w[B];
#pragma unroll
        for (int u = 0; u < B; u++) {
            const int r = r0 + u * THREADS;
            w[u] = r0 == tid ? w_own[u] : r < R ? __ldcg(p.probs + r) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < B; u++) {
            const int r = r0 + u * THREADS;
            if (r >= R || id[r] == NONE) continue;
            const int e = id[r], t = r / p.K;
            if (repeated) {
                bool first = true;
                for (int j = t * p.K; j < r; j++) first = first && id[j] != e;
                if (!first) continue;
                for (int j = r + 1; j < (t + 1) * p.K; j++)
                    if (id[j] == e) w[u] += __ldcg(p.probs + j);
            }
            s_w[s_off[index[e]] + __popcll(mask[e] & ((1ull << t) - 1))] = w[u];
        }
    }
    ptx::fence_proxy_async_smem();     // the ring, used as scratch here, is TMA's from now on
}

template <bool FP8, bool DOWN>
__global__ void __launch_bounds__(few_threads<FP8>(), 1)
    few_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                    const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmST,
                    const FewArgs p) {
    constexpr int THREADS = few_threads<FP8>();
    constexpr int BK = FP8 ? 128 : 64;
    constexpr int TMEM_COLS = FP8 ? 256 : 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = p.stages;
    const int stage_bytes = FEW_KPS * (FEW_A_BYTES + p.nb * 128);      // FEW_KPS weight tiles, then tokens
    uint8_t* at = ring + (size_t)stages * stage_bytes;
    uint8_t* sfring = at;                                            // MXFP8
    at += FP8 ? FEW_SF_SLOTS * FEW_SF_BYTES : 0;
    FewSmem& sm = *reinterpret_cast<FewSmem*>(at);
    at += few_up16(sizeof(FewSmem));
    float* acc = reinterpret_cast<float*>(at);                       // [T][128] output sums
    at += (size_t)p.T * 512;
    unsigned long long* s_mask = reinterpret_cast<unsigned long long*>(at);
    at += few_up16((size_t)p.a_max * 8);
    int* s_e = reinterpret_cast<int*>(at);
    at += few_up16((size_t)p.a_max * 4);
    int* s_off = reinterpret_cast<int*>(at);
    at += few_up16((size_t)(p.a_max + 1) * 4);
    float* s_w = reinterpret_cast<float*>(at);
    volatile uint32_t* s_abort = &sm.abort_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < FEW_STAGES; s++) {
            ptx::mbar_init(&sm.full[s], 1);
            ptx::mbar_init(&sm.empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            ptx::mbar_init(&sm.tfull[s], 1);
            ptx::mbar_init(&sm.tempty[s], 4);
        }
        for (int s = 0; s < FEW_SF_SLOTS; s++) {
            ptx::mbar_init(&sm.sf_full[s], 1);
            ptx::mbar_init(&sm.sf_ready[s], 1);
            ptx::mbar_init(&sm.sf_empty[s], 1);
        }
        ptx::mbar_init(&sm.done, 1);
        sm.abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tmW);
        ptx::prefetch_tmap(&tmT);
        if constexpr (FP8) {
            ptx::prefetch_tmap(&tmSW);
            ptx::prefetch_tmap(&tmST);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc(&sm.tmem, TMEM_COLS);
        ptx::tmem_relinquish();
    }
    few_plan<THREADS, DOWN>(p, sm, ring, s_mask, s_e, s_off, s_w);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    FewPlan pl{s_mask, s_e, s_off, s_w, sm.A, 0, 0, 1, 1, 0, 0};
    if constexpr (DOWN) {
        pl.kbs = pl.A * (p.F / BK);
        pl.W = (p.H / 128) * pl.kbs;
        // n CTAs take W / n k-blocks of about 0.36 us each, then the last of a tile reads n / (H / 128) sums
        // of about 0.1 us each, 5 ns a token where that is more: the n that makes the sum least
        const float least = sqrtf((float)pl.W * (float)(p.H / 128) * (p.T <= 20 ? 3.6f : 72.0f / (float)p.T));
        pl.cut(max(1, min(min((int)gridDim.x, pl.W / FEW_MIN_KB), (int)least)));
    } else {
        const int tiles = pl.A * (p.F / 64), G = gridDim.x;
        pl.kbs = p.H / BK;
        pl.W = tiles * pl.kbs;
        // whole tiles, or equal pieces with the shared tiles joined: whichever ends first
        const int join = FEW_JOIN_KB + sm.slots / (2 * max(pl.A, 1));       // (and half of one for each token)
        // n pieces of W / n k-blocks of about 0.36 us each, then the last of a tile reads n / tiles sums of about
        // 0.02 us a token each (of 8 tokens at least): the n that makes the sum least (64 tokens of one expert, H =
        // 7168, F = 128: 84 us with 32 CTAs a tile, 37 so; 1 token, F = 256: 28 and 20)
        const float m = (float)sm.slots / (float)max(pl.A, 1);
        const int least = (int)sqrtf(18.0f * (float)pl.W * (float)tiles / fmaxf(m, 8.0f));
        const int pieces = max(1, min(min(G, pl.W / FEW_MIN_KB), min(tiles * FEW_SHARE, max(tiles, least))));
        const bool whole = (tiles + G - 1) / G * pl.kbs <= (pl.W + pieces - 1) / pieces + join;
        pl.unit = whole ? pl.kbs : 1;
        pl.cut(whole ? max(1, min(G, tiles)) : pieces);
    }

    if (warp == 0) {
        // ------------------------------------------------------------ producer (one lane)
        if (lane == 0) {
            FewWalk<FP8, DOWN> wk(p, pl);
            FewRun r;
            const uint64_t policy = evict_first_policy();
            int stage = 0, issued = 0, kb = 0;
            uint32_t phase = 0;
            bool ok = true, have = wk.next(r);
            // a stage: k-blocks k and, if the run has it, k + 1
            auto load_a = [&](int st, const FewRun& q, int k) {
                uint8_t* sa = ring + (size_t)st * stage_bytes;
                const int n = min(FEW_KPS, q.nkb - k);
                ptx::mbar_arrive_expect_tx(&sm.full[st], n * (FEW_A_BYTES + q.bn * 128));
                for (int i = 0; i < n; i++, sa += FEW_A_BYTES) {
                    tma_load_weights(sa, &tmW, &sm.full[st], (q.kb0 + k + i) * BK, q.row0, policy);
                    tma_load_weights(sa + FEW_A_BYTES / 2, &tmW, &sm.full[st], (q.kb0 + k + i) * BK, q.row1, policy);
                }
            };
            auto load_b = [&](int st, const FewRun& q, int k) {
                uint8_t* sb = ring + (size_t)st * stage_bytes + FEW_KPS * FEW_A_BYTES;
                const int n = min(FEW_KPS, q.nkb - k);
                for (int i = 0; i < n; i++, sb += p.nb * 128) {
                    if constexpr (DOWN) {
                        for (int j = 0; j < q.bn; j += 16)
                            ptx::tma_load_2d(sb + j * 128, &tmT, &sm.full[st], (q.kb0 + k + i) * BK, q.brow + j);
                    } else {
                        ptx::tma_load_2d(sb, &tmT, &sm.full[st], (q.kb0 + k + i) * BK, 0);
                    }
                }
            };
            auto step = [&]() {
                issued++;
                if (++stage == stages) { stage = 0; phase ^= 1u; }
                if ((kb += FEW_KPS) >= r.nkb) { kb = 0; have = wk.next(r); }
            };
            if constexpr (DOWN) {
                // the ring's worth of weights, then (once h is written) their tokens operand
                FewWalk<FP8, DOWN> wb = wk;
                FewRun rb = r;
                int sb = 0, kbb = 0, n = 0;
                for (; have && n < stages; n++) {
                    load_a(stage, r, kb);
                    step();
                }
                pdl_wait();
                for (int i = 0; i < n; i++) {
                    load_b(sb++, rb, kbb);
                    if ((kbb += FEW_KPS) >= rb.nkb) { kbb = 0; wb.next(rb); }
                }
            }
            while (have) {
                ok = ptx::wait_parity(&sm.empty[stage], phase ^ 1u, s_abort);
                if (!ok) break;
                load_a(stage, r, kb);
                load_b(stage, r, kb);
                step();
            }
            if (!ok) {
                // give the loads already issued a bounded chance to land before the CTA exits
                for (int i = 0; i < stages && i < issued; i++) {
                    if (--stage < 0) { stage = stages - 1; phase ^= 1u; }
                    volatile uint32_t never = 0u;
                    ptx::wait_parity(&sm.full[stage], phase, &never, 100000000ull);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one lane)
        // An SM's share of the memory's rate brings a 16 KB tile about every 690 cycles; a k-block's four
        // MMAs take 320, its two copies of scales 160, and a stage's wait and commit 350, one after the
        // other: hence two k-blocks a stage, and one lane that does nothing else.
        if (lane == 0) {
            FewWalk<FP8, DOWN> wk(p, pl);
            FewRun r;
            int stage = 0, buf = 0, sslot = 0;
            uint32_t phase = 0, tphase = 0, sphase = 0;
            const uint64_t a_desc = ptx::sdesc_k_sw128(ptx::smem_addr(ring));
            const uint64_t sf_desc = ptx::sdesc_plain(ptx::smem_addr(sfring));
            bool ok = true;
            while (ok && wk.next(r)) {
                ok = ptx::wait_parity(&sm.tempty[buf], tphase ^ 1u, s_abort);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * FEW_ACC_COLS);
                const uint32_t idesc = FP8 ? ptx::idesc_mxf8(128, r.bn, 0, 0) : ptx::idesc_bf16(128, r.bn);
                for (int k0 = 0; k0 < r.nkb; k0 += FEW_KPS) {
                    const uint64_t ad0 = a_desc + (uint64_t)(stage * (stage_bytes / 16));
                    const uint64_t bd0 = ad0 + FEW_KPS * FEW_A_BYTES / 16;
                    ok = ptx::wait_parity(&sm.full[stage], phase, s_abort);
                    if (!ok) break;
#pragma unroll
                    for (int u = 0; u < FEW_KPS; u++) {
                        const int kb = k0 + u;
                        if (kb >= r.nkb) break;
                        const uint64_t ad = ad0 + u * FEW_A_BYTES / 16, bd = bd0 + (uint64_t)(u * p.nb * 8);
                        if constexpr (FP8) {
                            const int gw = (r.kb0 + kb) & (FEW_SF_KB - 1);
                            const uint32_t sf_t = tmem + (uint32_t)(2 * FEW_ACC_COLS);
                            if (kb == 0 || gw == 0) {
                                // a group's scales to TMEM at once; the slot in shared memory is free after that
                                ok = ptx::wait_parity(&sm.sf_ready[sslot], sphase, s_abort);
                                if (!ok) break;
                                const uint64_t sd = sf_desc + (uint64_t)(sslot * (FEW_SF_BYTES / 16));
                                const int end = min(FEW_SF_KB, gw + r.nkb - kb);
                                for (int w = gw; w < end; w++) {
                                    ptx::tc_cp_32x128b_warpx4(sf_t + 8 * w, sd + 64 * w);
                                    ptx::tc_cp_32x128b_warpx4(sf_t + 8 * w + 4, sd + 64 * w + 32);
                                }
                                ptx::tc_commit(&sm.sf_empty[sslot]);
                                if (++sslot == FEW_SF_SLOTS) { sslot = 0; sphase ^= 1u; }
                            }
                            const uint32_t sf = sf_t + (uint32_t)gw * 8;
#pragma unroll
                            for (int k = 0; k < 4; k++)      // (scale ids k: bits 29-30 of A's, 4-5 of B's)
                                ptx::mma_mxf8(d, ad + 2 * k, bd + 2 * k, idesc | (uint32_t)(k << 29) | (uint32_t)(k << 4),
                                              sf, sf + 4, (kb | k) != 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; k++) ptx::mma_f16(d, ad + 2 * k, bd + 2 * k, idesc, (kb | k) != 0);
                        }
                    }
                    if (!ok) break;
                    ptx::tc_commit(&sm.empty[stage]);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::tc_commit(&sm.tfull[buf]);
                buf ^= 1;
                if (buf == 0) tphase ^= 1u;
            }
            // every MMA issued has completed before TMEM is released
            ptx::tc_commit(&sm.done);
            volatile uint32_t never = 0u;
            ptx::wait_parity(&sm.done, 0u, &never, 100000000ull);
        }
        __syncwarp();
    } else if (FP8 && warp == 6) {
        // ------------------------------------------------------------ scales (MXFP8)
        // A group is the scale bytes of FEW_SF_KB k-blocks of every row of a tile: 128 weight rows, bn token
        // rows. Landed, it is rearranged in place into a chunk per k-block for tcgen05.cp .32x128b: the
        // word of row 32 j + lane at lane * 4 + j; first the weights' 512 bytes, then the tokens'. Loads
        // and rearranging do not wait for one another.
        if constexpr (FP8) {
            struct Cursor {
                FewWalk<FP8, DOWN> wk;
                FewRun r;
                int kb;
                bool have;
            };
            auto advance = [](Cursor& c) {
                c.kb += FEW_SF_KB - ((c.r.kb0 + c.kb) & (FEW_SF_KB - 1));
                if (c.kb >= c.r.nkb) {
                    c.kb = 0;
                    c.have = c.wk.next(c.r);
                }
            };
            Cursor ld{FewWalk<FP8, DOWN>(p, pl), FewRun{}, 0, false};
            ld.have = ld.wk.next(ld.r);
            int ld_slot = 0, pr_slot = 0, loaded = 0;
            uint32_t ld_phase = 0, pr_phase = 0;
            if constexpr (DOWN) pdl_wait();       // (h's scales; the weights' wait with them)
            uint64_t t_idle = ptx::globaltimer_ns();
            while (ld.have || loaded > 0) {
                bool progress = false;
                if (ld.have && loaded < FEW_SF_SLOTS &&
                    __all_sync(FULL, ptx::mbar_test_wait(&sm.sf_empty[ld_slot], ld_phase ^ 1u))) {
                    if (lane == 0) {
                        uint8_t* sf = sfring + (size_t)ld_slot * FEW_SF_BYTES;
                        constexpr int RB = FEW_SF_KB * 4;            // bytes of a row
                        const int kx = (ld.r.kb0 + ld.kb) / FEW_SF_KB * RB;
                        ptx::mbar_arrive_expect_tx(&sm.sf_full[ld_slot], (128 + ld.r.bn) * RB);
                        ptx::tma_load_2d(sf, &tmSW, &sm.sf_full[ld_slot], kx, ld.r.row0);
                        ptx::tma_load_2d(sf + 64 * RB, &tmSW, &sm.sf_full[ld_slot], kx, ld.r.row1);
                        if constexpr (DOWN) {
                            for (int i = 0; i < ld.r.bn; i += 16)
                                ptx::tma_load_2d(sf + (128 + i) * RB, &tmST, &sm.sf_full[ld_slot], kx, ld.r.brow + i);
                        } else {
                            ptx::tma_load_2d(sf + 128 * RB, &tmST, &sm.sf_full[ld_slot], kx, 0);
                        }
                    }
                    __syncwarp();
                    loaded++;
                    advance(ld);
                    if (++ld_slot == FEW_SF_SLOTS) { ld_slot = 0; ld_phase ^= 1u; }
                    progress = true;
                }
                if (loaded > 0 && __all_sync(FULL, ptx::mbar_test_wait(&sm.sf_full[pr_slot], pr_phase))) {
                    uint8_t* sf = sfring + (size_t)pr_slot * FEW_SF_BYTES;
                    const uint4* l = reinterpret_cast<const uint4*>(sf);
                    constexpr int Q = FEW_SF_KB / 4;
                    uint4 v[6][Q];                   // row 32 j + lane: words of k-blocks 4 i ..
#pragma unroll
                    for (int j = 0; j < 6; j++)
#pragma unroll
                        for (int i = 0; i < Q; i++) v[j][i] = l[(32 * j + lane) * Q + i];
                    __syncwarp();
                    uint4* out = reinterpret_cast<uint4*>(sf);
#pragma unroll
                    for (int w = 0; w < FEW_SF_KB; w++) {
                        auto word = [w](const uint4 (&q)[Q]) {
                            const uint4& u = q[w / 4];
                            return w % 4 == 0 ? u.x : w % 4 == 1 ? u.y : w % 4 == 2 ? u.z : u.w;
                        };
                        out[w * 64 + lane] = make_uint4(word(v[0]), word(v[1]), word(v[2]), word(v[3]));
                        out[w * 64 + 32 + lane] = make_uint4(word(v[4]), word(v[5]), 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&sm.sf_ready[pr_slot]);
                    loaded--;
                    if (++pr_slot == FEW_SF_SLOTS) { pr_slot = 0; pr_phase ^= 1u; }
                    progress = true;
                }
                if (progress) {
                    t_idle = ptx::globaltimer_ns();
                } else if (__any_sync(FULL, *s_abort != 0u)) {
                    break;
                } else if (__any_sync(FULL, ptx::globaltimer_ns() - t_idle > ptx::WAIT_LIMIT_NS)) {
                    *s_abort = 1u;
                    raise_device_error(MOE_DEVERR_TIMEOUT);
                    break;
                }
            }
            for (int i = 0; i < loaded; i++) {     // loads in flight land before the CTA exits
                volatile uint32_t never = 0u;
                ptx::wait_parity(&sm.sf_full[pr_slot], pr_phase, &never, 100000000ull);
                if (++pr_slot == FEW_SF_SLOTS) { pr_slot = 0; pr_phase ^= 1u; }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (4 warps)
        const int q = warp & 3;                         // TMEM lane quarter
        const int row = q * 32 + lane;                  // weight row of the tile
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
        FewWalk<FP8, DOWN> wk(p, pl);
        FewRun r;
        int buf = 0;
        uint32_t tphase = 0;
        bool ok = true, have = wk.next(r);
        auto release = [&]() {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sm.tempty[buf]);
            buf ^= 1;
            if (buf == 0) tphase ^= 1u;
        };
        // Counts this CTA's partial sums as written (all four warps', by the barrier) and makes those counted
        // before visible: how many these are.
        auto arrive = [&](unsigned* count) {
            epi_sync();
            if (threadIdx.x == 64) {
                unsigned n;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(n) : "l"(count), "r"(1u) : "memory");
                sm.ticket = (int)n;
            }
            epi_sync();
            return sm.ticket;
        };
        if constexpr (!DOWN) {
        // lanes 0-63 hold the gate products, 64-127 the same columns' linear ones; FEW_XCH tokens at a
        // time, two exchange buffers in turn
        int xb = 0;
        while (have) {
            ok = ptx::wait_parity(&sm.tfull[buf], tphase, s_abort);
            ok = epi_all(ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const unsigned long long tokens = pl.mask[r.a];
            const int m_a = pl.off[r.a + 1] - pl.off[r.a];
            const size_t slot = (size_t)p.T * 128;
            // the next up to 16 tokens' columns of the accumulator
            auto load16 = [&](unsigned long long& m, uint32_t* v) {
#pragma unroll
                for (int i = 0; i < FEW_XCH; i++) v[i] = 0u;
#pragma unroll
                for (int i = 0; i < FEW_XCH; i++) {
                    if (!m) break;                       // uniform
                    v[i] = tmem_ld_x1(tq + (uint32_t)(buf * FEW_ACC_COLS + __ffsll((long long)m) - 1));
                    m &= m - 1;
                }
                tmem_wait16(v);
            };
            const bool whole = r.nkb == pl.kbs;
            bool mine = true;
            int c0 = 0, c1 = 0;
            if (!whole) {
                c0 = pl.owner(r.tile * pl.kbs);
                c1 = pl.owner((r.tile + 1) * pl.kbs - 1);
                float* to = p.part + pl.slot_of(blockIdx.x, r.tile) * slot + row;
                unsigned long long m = tokens;
                for (int i0 = 0; i0 < m_a; i0 += FEW_XCH) {
                    uint32_t v[FEW_XCH];
                    load16(m, v);
#pragma unroll
                    for (int i = 0; i < FEW_XCH; i++)
                        if (i0 + i < m_a) __stcg(to + (i0 + i) * 128, __uint_as_float(v[i]));
                }
                release();
                mine = arrive(p.count + p.H / 128 + c0) == c1 - c0;
            }
            if (mine) {
                unsigned long long m = tokens;
                for (int i0 = 0; i0 < m_a; i0 += FEW_XCH) {
                    uint32_t v[FEW_XCH];
                    const int n = min(FEW_XCH, m_a - i0);
                    if (whole) {
                        load16(m, v);
                    } else {
                        float f[FEW_XCH];
#pragma unroll
                        for (int i = 0; i < FEW_XCH; i++) f[i] = 0.0f;
                        const float* from = p.part + pl.slot_of(c0, r.tile) * slot + i0 * 128 + row;
#pragma unroll 4
                        for (int c = c0; c <= c1; c++) {
#pragma unroll
                            for (int i = 0; i < FEW_XCH; i++)
                                if (i < n) f[i] += __ldcg(from + i * 128);
                            from = p.part + (2 * (c + 1)) * slot + i0 * 128 + row;
                        }
#pragma unroll
                        for (int i = 0; i < FEW_XCH; i++) v[i] = __float_as_uint(f[i]);
                    }
                    // gate and linear lanes each finish every other token: the other half's value comes through
                    // shared memory
                    const int col = row & 63;
                    const bool gate = q < 2;
                    const int other = gate ? 1 : 0;          // parity of the tokens that go over
#pragma unroll
                    for (int i = 0; i < FEW_XCH; i += 2) {
                        if (i + other >= n) break;
                        sm.xch[xb][i + other][col] = __uint_as_float(gate ? v[i + 1] : v[i]);
                    }
                    epi_sync();
                    size_t o = (size_t)(pl.off[r.a] + i0 + 1 - other) * p.F + r.tile % (p.F / 64) * 64 + col;
#pragma unroll
                    for (int i = 0; i < FEW_XCH; i += 2, o += 2 * p.F) {
                        if (i + 1 - other >= n) break;
                        const float here = __uint_as_float(gate ? v[i] : v[i + 1]), there = sm.xch[xb][i + 1 - other][col];
                        const float ga = gate ? here : there, li = gate ? there : here;
                        const float h = __fdividef(ga, 1.0f + __expf(-ga)) * li;
                        if constexpr (FP8) {
                            const float amax = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(fabsf(h))));
                            const int sbyte = e8m0_scale_byte(amax);
                            static_cast<uint8_t*>(p.h)[o] = (uint8_t)f32x2_to_e4m3x2(h * e8m0_inv_scale(sbyte), 0.0f);
                            if (lane == 0) p.hs[o >> 5] = (uint8_t)sbyte;
                        } else {
                            static_cast<__nv_bfloat16*>(p.h)[o] = __float2bfloat16_rn(h);
                        }
                    }
                    xb ^= 1;
                }
            }
            if (whole) release();
            have = wk.next(r);
        }
        } else {
        int tile = -1;
        auto flush = [&]() {
            const int c0 = pl.owner(tile * pl.kbs), c1 = pl.owner((tile + 1) * pl.kbs - 1);
            __nv_bfloat16* y = p.y + tile * 128 + row;
            if (c0 == c1) {
                for (int t = 0; t < p.T; t++) y[(size_t)t * p.H] = __float2bfloat16_rn(acc[t * 128 + row]);
                return;
            }
            const size_t slot = (size_t)p.T * 128;
            float* to = p.part + pl.slot_of(blockIdx.x, tile) * slot + row;
            for (int t = 0; t < p.T; t++) __stcg(to + t * 128, acc[t * 128 + row]);
            auto put = [&](int t, const float4& v) {
                __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
                *reinterpret_cast<uint2*>(p.y + (size_t)t * p.H + tile * 128 + 4 * lane) = *reinterpret_cast<uint2*>(o);
            };
            // four rows a lane; up to 32 loads in flight per warp
            const float4* first = reinterpret_cast<const float4*>(p.part + pl.slot_of(c0, tile) * slot) + lane;
            int n = c1 - c0 + 1, apart = 1;            // sums to add: of every apart-th CTA
            if (n * p.T > FEW_ONE_JOIN) {
                // in two steps: the last of a group of CTAs adds the group's sums up into its first one's
                apart = (int)ceilf(sqrtf((float)n));
                const int g = ((int)blockIdx.x - c0) / apart, m0 = c0 + g * apart, m = min(apart, c1 + 1 - m0);
                const int own = pl.slot_of(m0, tile);
                if (arrive(p.count + p.H / 128 + FEW_GRID_MAX + own) != m - 1) return;
                float4* sum = reinterpret_cast<float4*>(p.part + own * slot) + lane;
                const float4* others = reinterpret_cast<const float4*>(p.part + (size_t)2 * (m0 + 1) * slot) + lane;
                for (int t0 = q; t0 < p.T; t0 += 32) {
                    float4 v[8];
                    few_add_parts<8, 4>(v, sum, others, slot / 2, 0, 1, m, t0, 4, p.T);
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (t0 + 4 * j < p.T) __stcg(sum + (t0 + 4 * j) * 32, v[j]);
                }
                n = (n + apart - 1) / apart;
            }
            if (arrive(p.count + tile) != n - 1) return;
            const float4* rest = reinterpret_cast<const float4*>(p.part + (size_t)2 * (c0 + apart) * slot) + lane;
            const size_t stride = apart * (slot / 2);
            if (apart == 1 && p.T <= 4) {
                // a quarter of the CTAs' sums per warp, then the four warps' in order
                float4 v[4];
                few_add_parts<4, 8>(v, first, rest, slot / 2, q, 4, n, 0, 1, p.T);
                float4* x = reinterpret_cast<float4*>(sm.xch);      // [warp][token][lane]
#pragma unroll
                for (int t = 0; t < 4; t++) x[(q * 4 + t) * 32 + lane] = v[t];
                epi_sync();
                if (q < p.T) {
                    float4 a = x[q * 32 + lane];
#pragma unroll
                    for (int w = 1; w < 4; w++) {
                        const float4 b = x[(w * 4 + q) * 32 + lane];
                        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
                    }
                    put(q, a);
                }
                epi_sync();
            } else if (apart == 1 && p.T <= 16) {
                // a warp per token
                float4 v[4];
                few_add_parts<4, 8>(v, first, rest, slot / 2, 0, 1, n, q, 4, p.T);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (q + 4 * j < p.T) put(q + 4 * j, v[j]);
            } else {
                for (int t0 = q; t0 < p.T; t0 += 32) {
                    float4 v[8];
                    few_add_parts<8, 4>(v, first, rest, stride, 0, 1, n, t0, 4, p.T);
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (t0 + 4 * j < p.T) put(t0 + 4 * j, v[j]);
                }
            }
        };
        while (have) {
            if (r.tile != tile) {
                if (tile >= 0) flush();
                tile = r.tile;
                for (int t = 0; t < p.T; t++) acc[t * 128 + row] = 0.0f;
            }
            ok = ptx::wait_parity(&sm.tfull[buf], tphase, s_abort);
            ok = epi_all(ok);
            if (!ok) break;
            ptx::tc_fence_after();
            unsigned long long m = pl.mask[r.a];
            const int m_a = pl.off[r.a + 1] - pl.off[r.a];
            const float* wt = pl.w + pl.off[r.a];
            for (int i0 = 0; i0 < m_a; i0 += 16) {
                uint32_t v[16];
                tmem_ld_x16(tq + (uint32_t)(buf * FEW_ACC_COLS + i0), v);
                tmem_wait16(v);
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    if (i0 + i >= m_a) break;
                    const int t = __ffsll((long long)m) - 1;
                    m &= m - 1;
                    acc[t * 128 + row] = fmaf(wt[i0 + i], __uint_as_float(v[i]), acc[t * 128 + row]);
                }
            }
            release();
            have = wk.next(r);
        }
        if (ok && tile >= 0) flush();
        if (pl.A == 0) {
            // no valid route at all: zeros
            for (long long i = (long long)blockIdx.x * 128 + row; i < (long long)p.T * p.H; i += (long long)gridDim.x * 128)
                p.y[i] = __float2bfloat16_rn(0.0f);
        }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Workspace: counters, x's codes and scales (MXFP8), h (and its scales), partial sums; each region
// 128-byte aligned.
struct FewLayout {
    size_t count, xq, xs, h, hs, part, bytes;
};

int few_sms() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}


FewLayout few_layout(int T, int K, int H, int F, bool fp8) {
    auto up = [](size_t v) { return (v + 127) & ~(size_t)127; };
    FewLayout l{};
    size_t o = 0;
    l.count = o;
    o += up((size_t)(H / 128 + 3 * FEW_GRID_MAX) * 4);
    l.xq = o;
    o += fp8 ? up((size_t)T * H) : 0;
    l.xs = o;
    o += fp8 ? up((size_t)T * (H / 32)) : 0;
    l.h = o;
    o += up((size_t)T * K * F * (fp8 ? 1 : 2));
    l.hs = o;
    o += fp8 ? up((size_t)T * K * (F / 32)) : 0;
    l.part = o;
    o += (size_t)2 * FEW_GRID_MAX * T * 128 * 4;
    l.bytes = o;
    return l;
}

// Ring stages that fit beside the plan and the output sums, 0 where too few do, or where the plan's
// scratch does not fit them.
int few_stages(int T, int K, int E, bool fp8) {
    const size_t fixed = 1024 + few_fixed_smem(T, K, E < T * K ? E : T * K, fp8);
    const size_t stage = FEW_KPS * (FEW_A_BYTES + (size_t)((T + 15) & ~15) * 128);
    if (fixed + 2 * stage > FEW_SMEM_MAX) return 0;
    const int n = (int)((FEW_SMEM_MAX - fixed) / stage), stages = n < FEW_STAGES ? n : FEW_STAGES;
    return stages * stage < (size_t)E * 10 + (size_t)T * K * 2 ? 0 : stages;
}

moe_status few_sizes(int T, int K, int E, int H, int F, moe_dtype dtype) {
    if (dtype != MOE_BF16 && dtype != MOE_MXFP8) return MOE_ERR_INVALID_ARG;
    if (T < 0 || K < 1 || E < 1 || K > E || H < 128 || F < 128) return MOE_ERR_INVALID_ARG;
    const int step = dtype == MOE_MXFP8 ? 512 : 128;    // (MXFP8: whole 16-byte pieces of scales)
    if (H % step || F % step) return MOE_ERR_UNSUPPORTED;
    if (T > FEW_TMAX || K > FEW_KMAX || (long long)T * K > FEW_ROUTES || E > FEW_EMAX) return MOE_ERR_UNSUPPORTED;
    if ((long long)E * 2 * F > 0x7fffffffLL || (long long)E * H > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (T > 0 && !few_stages(T, K, E, dtype == MOE_MXFP8)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <bool FP8>
moe_status few_launch(FewArgs a, const PrepArgs& p, const void* x, const uint8_t* xs, const void* w13,
                      const uint8_t* w13s, const void* w2, const uint8_t* w2s, cudaStream_t s) {
    a.stages = few_stages(a.T, a.K, a.E, FP8);
    const size_t smem = 1024 + few_fixed_smem(a.T, a.K, a.a_max, FP8) + (size_t)a.stages * FEW_KPS * (FEW_A_BYTES + a.nb * 128);
    CUtensorMap tw13, tw2, tx, th, ts13, ts2, tsx, tsh;
    using moe_host::make_operand_map;
    using moe_host::make_scale_map;
    const uint64_t r13 = (uint64_t)a.E * 2 * a.F, r2 = (uint64_t)a.E * a.H, rh = (uint64_t)a.T * a.K;
    if (!make_operand_map(&tw13, w13, FP8, a.H, r13, 64) || !make_operand_map(&tw2, w2, FP8, a.F, r2, 64) ||
        !make_operand_map(&tx, x, FP8, a.H, a.T, a.nb) || !make_operand_map(&th, a.h, FP8, a.F, rh, 16))
        return MOE_ERR_CUDA;
    if (FP8) {
        if (!make_scale_map(&ts13, w13s, a.H / 32, r13, 64, FEW_SF_KB * 4) || !make_scale_map(&ts2, w2s, a.F / 32, r2, 64, FEW_SF_KB * 4) ||
            !make_scale_map(&tsx, xs, a.H / 32, a.T, a.nb, FEW_SF_KB * 4) || !make_scale_map(&tsh, a.hs, a.F / 32, rh, 16, FEW_SF_KB * 4))
            return MOE_ERR_CUDA;
    } else {
        ts13 = ts2 = tsx = tsh = tw13;
    }
    static moe_host::PerDevice up_smem, down_smem;
    if (!moe_host::allow_smem(few_gemm_kernel<FP8, false>, FEW_SMEM_MAX, up_smem) ||
        !moe_host::allow_smem(few_gemm_kernel<FP8, true>, FEW_SMEM_MAX, down_smem))
        return MOE_ERR_CUDA;
    const int V = p.logits ? (p.E + PREP_THREADS - 1) / PREP_THREADS : 1;
    const int ctas = a.T + (FP8 ? a.T * ((a.H + PREP_QUANT - 1) / PREP_QUANT) : 0);
    if (V <= 1) few_prep_kernel<1><<<ctas, PREP_THREADS, 0, s>>>(p);
    else if (V <= 4) few_prep_kernel<4><<<ctas, PREP_THREADS, 0, s>>>(p);
    else if (V <= 12) few_prep_kernel<12><<<ctas, PREP_THREADS, 0, s>>>(p);
    else few_prep_kernel<32><<<ctas, PREP_THREADS, 0, s>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) return moe_host::launch_status();
    int grid = few_sms();
    if (grid > FEW_GRID_MAX) grid = FEW_GRID_MAX;
    const dim3 block(few_threads<FP8>());
    if (moe_host::launch_pdl(few_gemm_kernel<FP8, false>, dim3((unsigned)grid), block, smem, s, tw13, tx, ts13, tsx, a) !=
            cudaSuccess ||
        moe_host::launch_pdl(few_gemm_kernel<FP8, true>, dim3((unsigned)grid), block, smem, s, tw2, th, ts2, tsh, a) !=
            cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
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
    p.T = T;
    p.H = H;
    p.E = E;
    p.K = K;
    p.ids = ids;
    p.i16 = id_dtype == MOE_I16;
    p.renorm = (flags & MOE_ROUTE_RENORM) != 0;
    p.probs = probs;
    p.xq = fp8 ? ws + l.xq : nullptr;
    p.xs = fp8 ? ws + l.xs : nullptr;
    p.count = reinterpret_cast<unsigned*>(ws + l.count);
    p.n_count = H / 128 + 3 * FEW_GRID_MAX;
    FewArgs a{};
    a.ids = ids;
    a.probs = probs;
    a.i16 = p.i16;
    a.T = T;
    a.H = H;
    a.K = K;
    a.E = E;
    a.F = F;
    a.nb = (T + 15) / 16 * 16;
    a.a_max = E < T * K ? E : T * K;
    a.h = ws + l.h;
    a.hs = fp8 ? ws + l.hs : nullptr;
    a.part = reinterpret_cast<float*>(ws + l.part);
    a.count = p.count;
    a.y = static_cast<__nv_bfloat16*>(y);
    const cudaStream_t s = moe_host::as_stream(stream);
    return fp8 ? few_launch<true>(a, p, p.xq, p.xs, w13_packed, w13_scales, w2_packed, w2_scales, s)
               : few_launch<false>(a, p, x, nullptr, w13_packed, nullptr, w2_packed, nullptr, s);
}
