// paged_attention.cu -- attention of one new token per sequence over a paged key-value cache: moe_paged_attention.
//
// For every sequence and key head, with its group of query heads: s = scale q.k over the cached positions,
// out = sum exp(s - m) v / sum exp(s - m), in one pass with a running maximum m. Each cached byte is used by the
// group's heads only (a multiply-add per head and element), so DRAM bounds it: what matters is that every block
// has loads in flight all the time and that all blocks end together.
//
// Split: the positions of all (sequence, key head) pairs, in units of 64, are laid end to end and cut into one
// equal stretch per block (two blocks an SM), whatever the lengths. A pair that lies in one stretch is finished there; of one
// that is cut, each block leaves m, l and the unnormalised output in the workspace, and a second kernel, set up
// while the first one runs, joins them in the blocks' order. So outputs do not depend on timing.
//
// A block's four warps work alone, a tile of 16 or 32 positions of a unit each: a ring of tiles per warp (two of MXFP8 rows of 128
// or 256, three to six of the others: what 24 KB hold) is filled by 16-byte asynchronous copies (rows anywhere, so pages may end inside a tile; absent rows are filled with zeros).
// The products take the cache as the 16-row operand and the heads as the 8 columns, S^T = K Q^T and
// O^T = V^T P^T, so that a key or value passes through one fragment once, whatever the group, and the running
// maximum and scale of a head sit in the lanes that hold its column. P^T is the transpose of the fragment that S^T comes
// out in (movmatrix). These are mma.sync products: a tcgen05 tile of 128 rows would want the softmax
// across 128 lanes of tensor memory and the weights back through shared memory, for a product that DRAM bounds.
//
// MXFP8: codes are converted to halves on the way to the fragments (exact). A block of 32 keys' elements is one
// partial product, scaled by the key's power of two in fp32; q is scaled per head by a power of two to fill fp16's
// range. Values' scales go into the weights, relative to the largest scale that the warp has met, which the sums are
// kept relative to; fp16 weights are scaled by 2^15, so that one loses bits only below 2^-29 of the largest. A tile
// whose scales span more than 2^6 below that takes bf16 values and weights, which have fp32's range.
//
// A bf16 weight is 8 bits: rounded to them, weights would add nearly as much to the outputs' error as the outputs' own rounding does
// (one sequence of 131072: 0.0020 of the outputs, root mean square, in place of 0.0017). So it is two bf16, 16 bits, and two
// products (that sequence 91.7 -> 92.2 us, 64 of 1 to 8192 50.3 -> 50.9; 32 query heads a key head, which the products bound, 84
// -> 93). One fp16, 11 bits, adds 0.4 % of that and stays one: the MXFP8 kernel is bound by its instructions.
//
// Measured (one GB300, GPU time of the call with the join): bf16, 32 x 16384 positions of 8 key heads of 128, 32 query heads
// 321-324 us = 6.63-6.69 TB/s of the cache's bytes (a plain copy runs at 6.78); one sequence of 131072 92 us, of which the join
// is 5 to 6; 64 sequences of 1 to 8192 51 us (38 at the copy's rate). MXFP8, the 32 x 16384: 183 us = 6.0 TB/s, near what DRAM gives
// (about 9 us are the beginning and the join) with 731 instructions a warp and 32 positions, 1.7 a cycle with 8 warps an SM;
// 12 warps take 16-row tiles, and 249 us; a third stage of the ring changes nothing. One sequence of 100: 6.3 us.
#include "common.cuh"
#include "paged_cache.cuh"
#include "scale_words.h"

#include <math.h>

namespace moe {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = 32 * PA_WARPS;
constexpr int PA_MAX_CTAS = 512;                  // blocks at most: what the workspace has room for
constexpr int PA_BEGIN = 2;                       // units that beginning and ending a pair takes as long as
constexpr int PA_MIN_UNITS = 2;                   // of a block's stretch: a shorter one costs more to join than it saves
constexpr int PA_WHOLE = 256;                     // positions that a pair is not cut for
constexpr int PA_SPREAD = 6;                      // exponents below the largest scale that fp16 weights take

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
    float* part;                                  // [2 * ctas][8 NB][DP] unnormalised outputs
    float2* part_ml;                              // [2 * ctas][8 NB]
    int4* cut;                                    // [ctas] the pair that a block begins and does not end
    int tiles_of_heads;                           // tiles of 8 NB query heads in a group
    int whole;                                    // pairs are not cut: a stretch is of pairs, not of units
    uint32_t page_mul, page_shift;                // p / page_size = (p page_mul >> 32) >> page_shift (0: pages of one)
};

template <bool FP8, int DP, int NB>
struct Cfg {
    static constexpr int ROW = DP * (FP8 ? 1 : 2);             // bytes of a row in shared memory
    static constexpr int CHUNKS = ROW / 16;
    static constexpr int SUB = ROW <= 128 && NB < 4 ? 2 : 1;   // 16-row operands of a tile: short rows go two at a time
    static constexpr int TILE = 16 * SUB;                      // positions of a warp's tile
    static constexpr int UNIT = PA_WARPS * TILE;               // positions of a block's unit
    static constexpr int KV = 2 * TILE * ROW;
    static constexpr int STAGE = KV + (FP8 ? 2 * TILE * 16 : 0);   // and a 16-byte slot for each row's scales
    static constexpr int STAGES = DP == 256 && !FP8 ? 3 : (96 * 1024 / PA_WARPS) / STAGE > 6 ? 6 : (96 * 1024 / PA_WARPS) / STAGE;
    static_assert(STAGES >= 2, "a tile is on its way while another is taken");
    static constexpr int PREP = FP8 ? DP / 32 * TILE * (4 + 2) : 0;  // a tile's scales as the products take them
    static constexpr int HALF = DP / 2;                        // elements joined at a time
    static constexpr int JOIN = PA_WARPS * 8 * (HALF + 4) * 4;
    static constexpr int ML = PA_WARPS * 8 * NB * 2 * 4;
    static constexpr int SMEM = PA_WARPS * (STAGES * STAGE + PREP + 64) + JOIN + ML;
    static constexpr int CTAS = SMEM + 1024 <= 114 * 1024 ? 2 : 1;
    static constexpr int SLOT = 8 * NB * DP;                   // floats of a partial output
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes (0: zeros instead) to shared memory.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 2^e for e <= 127, in fp32's subnormals too (ex2.approx.ftz has none).
__device__ __forceinline__ float two_to(int e) {
    return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : e >= -149 ? 1u << (e + 149) : 0u);
}
// Shared memory by pointers: the compiler orders these between the barriers as it likes.
template <typename T>
__device__ __forceinline__ T get(const uint8_t* p) { return *reinterpret_cast<const T*>(p); }
template <typename T>
__device__ __forceinline__ void put(uint8_t* p, T v) { *reinterpret_cast<T*>(p) = v; }
// 2, 4 or 8 words that begin on a boundary of their size (16 bytes at most).
template <int N>
__device__ __forceinline__ void get_all(const uint8_t* p, uint32_t (&w)[N]) {
    if (N == 2) {
        const uint2 x = get<uint2>(p);
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; i++) {
            const uint4 x = get<uint4>(p + 16 * i);
            w[4 * i] = x.x;
            w[(4 * i + 1) % N] = x.y;
            w[(4 * i + 2) % N] = x.z;
            w[(4 * i + 3) % N] = x.w;
        }
    }
}
// Whether one of the four bytes is 255.
__device__ __forceinline__ bool has_255(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & x & 0x80808080u; }
// Codes 0 and 1 of a word, codes 2 and 3, as two halves each (exact).
__device__ __forceinline__ void halves(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}
// Two halves that came from codes as two bf16 (exact).
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// Two weights as two bf16 each, 16 bits of them in all: cut off, and what is left. That is never 0 beside a first part that is
// not, so that an infinite value times both stays what it is.
__device__ __forceinline__ void split2(float x, float y, uint32_t& first, uint32_t& left) {
    const uint32_t cx = __float_as_uint(x) & 0xffff0000u, cy = __float_as_uint(y) & 0xffff0000u;
    const float fx = __uint_as_float(cx), fy = __uint_as_float(cy);
    first = (cx >> 16) | cy;
    left = pack2<false>(fmaxf(x - fx, fx * 0x1p-24f), fmaxf(y - fy, fy * 0x1p-24f));
}
template <bool F16>
__device__ __forceinline__ uint32_t times2(uint32_t x, uint32_t y) {
    if (F16) {
        const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// ---------------------------------------------------------------- the walk over units
// Positions [first, n) of sequence b.
__device__ __forceinline__ void range_of(const AttnArgs& a, int b, int& first, int& n) {
    n = max(0, __ldg(a.lengths + b));
    const long long most = (long long)a.M * a.c.page_size;
    if (n > most) {
        n = (int)most;
        if (threadIdx.x == 0) raise_device_error(MOE_DEVERR_BAD_ID);
    }
    first = a.window > 0 && n > a.window ? n - a.window : 0;
}
// A pair's units: one at least, which writes the output of a sequence without positions. On the line that is cut into
// stretches PA_BEGIN steps stand before them: what a block takes for a pair however few units it has of it.
// (Positions are counted in 31 bits, those up to a unit's end in 32.)
__device__ __forceinline__ int units_of(int first, int n, int unit) {
    return max(1, (int)(((uint32_t)(n - first) + (uint32_t)unit - 1u) / (uint32_t)unit));
}

struct Walk {
    int b, pair, first, n, units;                 // pair: of a sequence's key heads and tiles of query heads
    int at, u, u1;                                // the segment's first step of the pair; its units [u, u1)
    long long left;                               // steps (whole: pairs) of the stretch from this segment on

    __device__ __forceinline__ void cut(const AttnArgs& a) {
        u = a.whole ? 0 : max(0, at - PA_BEGIN);
        u1 = a.whole ? units : (int)max(0ll, min((long long)units, at + left - PA_BEGIN));
    }
    // The next segment with a unit in it (left is 0 behind the last).
    __device__ __forceinline__ void next(const AttnArgs& a, int pairs, int unit) {
        do {
            left -= a.whole ? 1 : min((long long)units + PA_BEGIN - at, left);
            at = 0;
            if (left <= 0) return;
            if (++pair == pairs) {
                pair = 0;
                b++;
                range_of(a, b, first, n);
                units = units_of(first, n, unit);
            }
            cut(a);
        } while (u1 <= u);
    }
};

// The first segment of this block's stretch, and in total the steps (whole: pairs) of all. Every thread calls it.
__device__ __forceinline__ Walk walk_begin(const AttnArgs& a, int pairs, int unit, long long* red, long long& total, int& ctas) {
    const int per = (a.B + PA_THREADS - 1) / PA_THREADS, b0 = min(a.B, per * (int)threadIdx.x), b1 = min(a.B, b0 + per);
    const int warp = threadIdx.x / 32;
    long long mine = 0;
    int first, n;
    for (int b = b0; b < b1; b++) {
        if (!a.whole) range_of(a, b, first, n);
        mine += (long long)pairs * (a.whole ? 1 : PA_BEGIN + units_of(first, n, unit));
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(FULL, upto, o);
        if ((int)lane_id() >= o) upto += v;
    }
    if (lane_id() == 31) red[warp] = upto;
    __syncthreads();
    total = 0;
    long long before = 0;
#pragma unroll
    for (int w = 0; w < PA_WARPS; w++) {
        if (w < warp) before += red[w];
        total += red[w];
    }
    // (a short total is left to fewer blocks; whole pairs to as many as there are)
    const long long fill = a.whole ? total : (total + PA_MIN_UNITS - 1) / PA_MIN_UNITS;
    ctas = (int)min((long long)gridDim.x, fill);
    Walk w;
    w.b = a.B;
    w.left = 0;
    if ((int)blockIdx.x >= ctas) return w;
    const long long from = total * blockIdx.x / ctas;
    w.left = total * (blockIdx.x + 1) / ctas - from;
    // the thread whose sequences hold the first unit finds it
    long long at = before + upto - mine;
    __syncthreads();
    if (from >= at && from < at + mine) {
        for (int b = b0; b < b1; b++) {
            range_of(a, b, first, n);
            const int steps = a.whole ? 1 : PA_BEGIN + units_of(first, n, unit);
            const long long here = (long long)pairs * steps;
            if (from < at + here) {
                red[0] = b;
                red[1] = (from - at) / steps;
                red[2] = (from - at) % steps;
                break;
            }
            at += here;
        }
    }
    __syncthreads();
    w.b = (int)red[0];
    w.pair = (int)red[1];
    w.at = (int)red[2];
    range_of(a, w.b, w.first, w.n);
    w.units = units_of(w.first, w.n, unit);
    w.cut(a);
    if (w.u1 <= w.u) w.next(a, pairs, unit);
    __syncthreads();
    return w;
}

// ---------------------------------------------------------------- the kernel
template <bool FP8, int DP, int NB>
__global__ void __launch_bounds__(PA_THREADS, (Cfg<FP8, DP, NB>::CTAS)) attention_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<FP8, DP, NB>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = lane_id(), j = lane & 3, r8 = lane >> 2;
    const int dim = a.c.dim, group = a.q_heads / a.c.heads, pairs = a.c.heads * a.tiles_of_heads;
    const int row_bytes = dim * (FP8 ? 1 : 2), row_scales = dim / 32;
    const long long lines = (long long)a.c.pages * a.c.heads * a.c.page_size;
    // the bytes of a row's scales that there are, four and four
    const uint32_t keep0 = row_scales >= 4 ? 0xffffffffu : (1u << (8 * row_scales)) - 1u;
    const uint32_t keep1 = row_scales >= 8 ? 0xffffffffu : row_scales > 4 ? (1u << (8 * (row_scales - 4))) - 1u : 0u;
    uint8_t* const ring_at = smem + warp * (C::STAGES * C::STAGE);
    const uint32_t ring = saddr(ring_at);
    uint8_t* const prep = smem + PA_WARPS * C::STAGES * C::STAGE + warp * C::PREP;    // fp32 [TILE][DP/32], then 16-bit [TILE/2][DP/32][2]
    uint32_t* const seen = reinterpret_cast<uint32_t*>(smem + PA_WARPS * (C::STAGES * C::STAGE + C::PREP)) + warp * 16;  // of a stage's rows
    float* const join = reinterpret_cast<float*>(smem + PA_WARPS * (C::STAGES * C::STAGE + C::PREP + 64));
    float2* const ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(join) + C::JOIN);
    if (FP8) {
        for (int i = lane; i < C::PREP / 4; i += 32) put(prep + 4 * i, 0u);
        __syncwarp();
    }
    long long total;
    int ctas;
    Walk w = walk_begin(a, pairs, C::UNIT, reinterpret_cast<long long*>(join), total, ctas);
    if (threadIdx.x == 0 && !a.whole) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    pdl_trigger();
    if (w.left <= 0) return;

    // -------- the loading walk, a tile ahead of the copies: its rows' pages are on their way
    Walk ld = w;
    int ld_u = w.u, ld_page = -1, ld_off = 0, ld_kv = w.pair / a.tiles_of_heads;
    bool ld_in = false, ld_more = true;
    auto look = [&]() {                            // finds the next tile of this warp that has a position
        ld_more = false;
        while (ld.left > 0) {
            if (ld_u == ld.u1) {
                ld.next(a, pairs, C::UNIT);
                ld_u = ld.u;
                ld_kv = ld.pair / a.tiles_of_heads;
                continue;
            }
            const uint32_t t = (uint32_t)ld.first + (uint32_t)ld_u * C::UNIT + warp * C::TILE;
            ld_u++;
            if (t >= (uint32_t)ld.n) continue;
            const uint32_t p = t + (lane & (C::TILE - 1));
            ld_in = p < (uint32_t)ld.n;
            const int col = a.page_mul ? (int)(__umulhi(p, a.page_mul) >> a.page_shift) : (int)p;
            ld_off = (int)p - col * a.c.page_size;
            ld_page = ld_in ? __ldg(a.table + (long long)ld.b * a.M + col) : -1;
            ld_more = true;
            return;
        }
    };
    const int ld_chunk = lane % C::CHUNKS, ld_row = lane / C::CHUNKS;
    int fill = 0;                                  // the stage that is filled next
    auto issue = [&]() {
        if (ld_more) {
            const bool ok = ld_in && (unsigned)ld_page < (unsigned)a.c.pages;
            if (ld_in && !ok) raise_device_error(MOE_DEVERR_BAD_ID);
            const long long line = ok ? ((long long)ld_page * a.c.heads + ld_kv) * a.c.page_size + ld_off : 0;
            const long long row_at = line * row_bytes;
            const unsigned rows = __ballot_sync(FULL, ok) & (C::TILE == 32 ? FULL : 0xffffu);
            const uint32_t at = ring + fill * C::STAGE;
            constexpr int PER = 32 / C::CHUNKS;    // rows that an instruction of the warp copies
            const char* const kp = static_cast<const char*>(a.c.k) + ld_chunk * 16;
            const char* const vp = static_cast<const char*>(a.c.v) + ld_chunk * 16;
            // a row's chunk in a tile of keys or values, where the fragments' reads meet all banks
            auto kx = [&](int row) { return !FP8 ? row & 7 : DP == 64 ? ((row >> 1) & 1) << 1 : (row & 3) << 1; };
            auto vx = [&](int row) { return !FP8 ? row & 7 : DP == 64 ? ((row >> 1) & 1) << 1 : ((row >> 1) & 3) << 1; };
            // Sixteen rows that follow one another (a page, or a part of it) need one address.
            const long long half = __shfl_sync(FULL, line, lane & 16 & (C::TILE - 1));
            const bool run = __all_sync(FULL, ok && line == half + (lane & 15)) && row_bytes == C::ROW;
            if (run) {
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    const long long from = __shfl_sync(FULL, row_at, x * 16) + ld_row * C::ROW;
#pragma unroll
                    for (int i = 0; i < 16 / PER; i++) {
                        const int row = x * 16 + i * PER + ld_row;
                        copy16(at + row * C::ROW + (ld_chunk ^ kx(row)) * 16, kp + from + i * PER * C::ROW);
                        copy16(at + (C::TILE + row) * C::ROW + (ld_chunk ^ vx(row)) * 16, vp + from + i * PER * C::ROW);
                    }
                }
            } else {
                const unsigned mine = ld_chunk * 16 < row_bytes ? rows >> ld_row : 0u;
#pragma unroll
                for (int i = 0; i < C::TILE / PER; i++) {
                    const int row = i * PER + ld_row;
                    const long long from = __shfl_sync(FULL, row_at, row);
                    // (a chunk that is not there is zeros, and its address the pool's first)
                    const bool there = (mine >> (i * PER)) & 1;
                    copy16(at + row * C::ROW + (ld_chunk ^ kx(row)) * 16, there ? kp + from : static_cast<const char*>(a.c.k), there);
                    copy16(at + (C::TILE + row) * C::ROW + (ld_chunk ^ vx(row)) * 16, there ? vp + from : static_cast<const char*>(a.c.v), there);
                }
            }
            if (FP8) {
                // a lane's row: the words that hold its scales, and where in them they begin
                const long long scales_at = line * row_scales;
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    const bool is_v = C::SUB == 2 ? x == 1 : lane >= 16;
                    const uint8_t* const base = (is_v ? a.c.v_scales : a.c.k_scales) + scales_at;
                    const uint32_t slot = at + C::KV + (x * 32 + lane) * 16;
                    uint8_t* const here = ring_at + (slot - ring);
                    if (row_scales == DP / 32 && DP >= 128) {          // whole words
#pragma unroll
                        for (int i = 0; i < DP / 128; i++) copy4(slot + 4 * i, base + 4 * i, ok);
                        put(here + 12, 0u);
                    } else if (ok && scales_at_an_end(line, lines)) {
#pragma unroll 1
                        for (int i = 0; i < row_scales; i++) put(here + i, __ldg(base + i));
                        put(here + 12, 0u);
                    } else {
                        const ScaleWords w = scale_words(reinterpret_cast<uintptr_t>(base), row_scales);
#pragma unroll
                        for (int i = 0; i < (DP / 32 + 6) / 4; i++)
                            if (i < w.words) copy4(slot + 4 * i, base - w.skip + 4 * i, ok);
                        put(here + 12, ok ? 8u * w.skip : 0u);
                    }
                }
            }
            if (lane == 0) seen[fill] = rows;
            look();
        }
        copies_commit();
        fill = fill + 1 == C::STAGES ? 0 : fill + 1;
    };
    look();
#pragma unroll 1
    for (int i = 0; i < C::STAGES; i++) issue();

    const float log2_scale = a.scale * 1.44269504088896340736f;
    uint32_t qf[NB][DP / 16][2];
    auto load_q = [&]() {                          // the heads of a segment
        const int kv = w.pair / a.tiles_of_heads, h0 = (w.pair - kv * a.tiles_of_heads) * 8 * NB;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int h = h0 + nb * 8 + r8;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + w.b * a.q_stride + (long long)(kv * group + h) * dim);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ks++) {
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    // (MXFP8: a lane's elements of a 32-element block are its eight codes of a row)
                    const int d = FP8 ? (ks / 2) * 32 + j * 8 + (ks % 2) * 4 + e * 2 : ks * 16 + j * 2 + e * 8;
                    qf[nb][ks][e] = h < group && d < dim ? __ldg(src + d / 2) : 0u;
                }
            }
        }
    };
    load_q();
    int take = 0;
    while (w.left > 0) {
        float to_s[NB][2];                         // from the products to scores in powers of two, of columns 2j and 2j + 1
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            to_s[nb][0] = to_s[nb][1] = log2_scale;
            if (FP8) {
                float top = 0.0f;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ks++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&qf[nb][ks][e]));
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                // by 2^shift the largest element is in [2^14, 2^15); two steps, for either may leave fp32's exponents
                int shift = 14 + 127 - (int)(__float_as_uint(top) >> 23);
                if (!(top > 0.0f) || isinf(top)) shift = 0;
                const float f1 = __uint_as_float((uint32_t)(127 + shift / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + shift - shift / 2) << 23);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ks++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&qf[nb][ks][e]));
                        qf[nb][ks][e] = pack2<true>(f.x * f1 * f2, f.y * f1 * f2);
                    }
                const float i1 = __uint_as_float((uint32_t)(127 - shift / 2) << 23), i2 = __uint_as_float((uint32_t)(127 - shift + shift / 2) << 23);
                const float back = log2_scale * i1 * i2;
                to_s[nb][0] = __shfl_sync(FULL, back, j * 8);
                to_s[nb][1] = __shfl_sync(FULL, back, j * 8 + 4);
            }
        }
        float m[NB][2], l[NB][2], o[NB][DP / 16][4];
        int vref = 0;                              // o is relative to 2^(vref - 127) (MXFP8)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
            for (int d = 0; d < DP / 16; d++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[nb][d][e] = 0.0f;
        }
        const int my_end = min(w.u1, (int)(((uint32_t)max(0, w.n - w.first - warp * C::TILE) + C::UNIT - 1u) / C::UNIT));
#pragma unroll 1
        for (int u = w.u; u < my_end; u++) {
            copies_wait<C::STAGES - 1>();
            __syncwarp();
            const uint8_t* const tile = ring_at + take * C::STAGE;
            const uint32_t kt = ring + take * C::STAGE, vt = kt + C::TILE * C::ROW;
            const uint32_t rows = seen[take];
            bool wide = false;                     // (MXFP8) this tile's scales span more than fp16 weights take
            if (FP8) {
                // the tile's scales, a lane a row (and, of 16 rows, a side); what a shorter row has not is 0, in least 255
                constexpr int BLOCKS = DP / 32;
                uint32_t most = 0u, least = 255u, word[C::SUB][2];
                bool nan = false;
                const bool here = (rows >> (lane & (C::TILE - 1))) & 1;
                auto byte_of = [&](int x, int i) { return (word[x][i >> 2] >> (8 * (i & 3))) & 0xffu; };
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    const uint4 slot = get<uint4>(tile + C::KV + (x * 32 + lane) * 16);
                    word[x][0] = __funnelshift_r(slot.x, slot.y, slot.w) & keep0;
                    word[x][1] = DP == 256 ? __funnelshift_r(slot.y, slot.z, slot.w) & keep1 : 0u;
                    nan = nan || has_255(word[x][0]) || (DP == 256 && has_255(word[x][1]));
                    if (C::SUB == 2 ? x == 1 : lane >= 16) {
#pragma unroll
                        for (int i = 0; i < BLOCKS; i++) {
                            most = max(most, byte_of(x, i));
                            least = min(least, ((i < 4 ? word[x][0] | ~keep0 : word[x][1] | ~keep1) >> (8 * (i & 3))) & 0xffu);
                        }
                    }
                }
                nan = __any_sync(FULL, nan);
                if (nan) {
                    most = 0u;
                    for (int x = 0; x < C::SUB; x++)
                        for (int i = 0; i < BLOCKS; i++)
                            if ((C::SUB == 2 ? x == 1 : lane >= 16) && byte_of(x, i) != 255u) most = max(most, byte_of(x, i));
                }
                most = __reduce_max_sync(FULL, most);
                least = __reduce_min_sync(FULL, here ? least : 255u);
                if ((int)most > vref) {
                    const float f = two_to(vref - (int)most);
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int d = 0; d < DP / 16; d++)
#pragma unroll
                            for (int e = 0; e < 4; e++) o[nb][d][e] *= f;
                    vref = (int)most;
                }
                wide = vref - (int)least > PA_SPREAD;
                const int bias = (wide ? 127 : 15) - vref, step = wide ? 7 : 10;
                const int row = lane & (C::TILE - 1);
                uint8_t *const ks = prep + row * BLOCKS * 4, *const vs = prep + C::TILE * BLOCKS * 4 + (row >> 1) * BLOCKS * 4 + (row & 1) * 2;
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    if (C::SUB == 2 ? x == 0 : lane < 16) {
                        uint32_t b[BLOCKS];        // (2^-127 is half of the least normal number)
#pragma unroll
                        for (int i = 0; i < BLOCKS; i++) b[i] = max(byte_of(x, i) << 23, 0x00400000u);
#pragma unroll
                        for (int i = 0; i < BLOCKS; i += 2) put(ks + 4 * i, make_uint2(b[i], b[i + 1]));
                    } else {
#pragma unroll
                        for (int i = 0; i < BLOCKS; i++) put(vs + 4 * i, (uint16_t)(max(0, bias + (int)byte_of(x, i)) << step));
                    }
                }
                if (nan) {
                    for (int x = 0; x < C::SUB; x++)
                        for (int i = 0; i < BLOCKS; i++) {
                            if (byte_of(x, i) != 255u) continue;
                            if (C::SUB == 2 ? x == 0 : lane < 16) put(ks + 4 * i, 0x7fc00000u);
                            else put(vs + 4 * i, (uint16_t)(wide ? 0x7fc0u : 0x7e00u));
                        }
                }
                __syncwarp();
            }
            // S^T = K Q^T
            float s[C::SUB][NB][4];
#pragma unroll
            for (int x = 0; x < C::SUB; x++)
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int e = 0; e < 4; e++) s[x][nb][e] = 0.0f;
            if (!FP8) {
                const int row = lane & 15;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ks++)
#pragma unroll
                    for (int x = 0; x < C::SUB; x++) {
                        uint32_t f[4];
                        ldmatrix(f, kt + (x * 16 + row) * C::ROW + (((2 * ks + (lane >> 4)) ^ (row & 7)) * 16));
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) mma<false>(s[x][nb], f, qf[nb][ks][0], qf[nb][ks][1]);
                    }
            } else {
                const int sw = DP == 64 ? ((r8 >> 1) & 1) << 1 : (r8 & 3) << 1;               // (row r8 + 8 has the same)
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    uint32_t scale0[DP / 32], scale1[DP / 32];
                    get_all(prep + (x * 16 + r8) * (DP / 32) * 4, scale0);
                    get_all(prep + (x * 16 + r8 + 8) * (DP / 32) * 4, scale1);
#pragma unroll
                    for (int i = 0; i < DP / 32; i++) {
                        const uint8_t* const at = tile + (x * 16 + r8) * C::ROW + (((2 * i + (j >> 1)) ^ sw) * 16) + (j & 1) * 8;
                        const uint2 top = get<uint2>(at), bot = get<uint2>(at + 8 * C::ROW);
                        float part[NB][4];
                        uint32_t f[4], g[4];
                        halves(top.x, f[0], f[2]);
                        halves(bot.x, f[1], f[3]);
                        halves(top.y, g[0], g[2]);
                        halves(bot.y, g[1], g[3]);
                        const float k0 = __uint_as_float(scale0[i]), k1 = __uint_as_float(scale1[i]);
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) {
                            part[nb][0] = part[nb][1] = part[nb][2] = part[nb][3] = 0.0f;
                            mma<true>(part[nb], f, qf[nb][2 * i][0], qf[nb][2 * i][1]);
                            mma<true>(part[nb], g, qf[nb][2 * i + 1][0], qf[nb][2 * i + 1][1]);
                            s[x][nb][0] = fmaf(k0, part[nb][0], s[x][nb][0]);
                            s[x][nb][1] = fmaf(k0, part[nb][1], s[x][nb][1]);
                            s[x][nb][2] = fmaf(k1, part[nb][2], s[x][nb][2]);
                            s[x][nb][3] = fmaf(k1, part[nb][3], s[x][nb][3]);
                        }
                    }
                }
            }
            // weights
            bool rises = false;
#pragma unroll
            for (int x = 0; x < C::SUB; x++) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        s[x][nb][e] *= to_s[nb][e];
                        s[x][nb][2 + e] *= to_s[nb][e];
                    }
                if (rows != (C::TILE == 32 ? FULL : 0xffffu)) {
                    const bool in0 = (rows >> (x * 16 + r8)) & 1, in1 = (rows >> (x * 16 + r8 + 8)) & 1;
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            if (!in0) s[x][nb][e] = -INFINITY;
                            if (!in1) s[x][nb][2 + e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int e = 0; e < 2; e++) rises = rises || fmaxf(s[x][nb][e], s[x][nb][2 + e]) > m[nb][e];
            }
            if (__any_sync(FULL, rises)) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
                    float keep[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        float top = fmaxf(s[0][nb][e], s[0][nb][2 + e]);
                        if (C::SUB == 2) top = fmaxf(top, fmaxf(s[C::SUB - 1][nb][e], s[C::SUB - 1][nb][2 + e]));
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, 16));
                        top = fmaxf(top, m[nb][e]);
                        keep[e] = top == -INFINITY ? 1.0f : pow2(m[nb][e] - top);
                        m[nb][e] = top;
                        l[nb][e] *= keep[e];
                    }
#pragma unroll
                    for (int d = 0; d < DP / 16; d++) {
                        o[nb][d][0] *= keep[0];
                        o[nb][d][1] *= keep[1];
                        o[nb][d][2] *= keep[0];
                        o[nb][d][3] *= keep[1];
                    }
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float sub = m[nb][e] == -INFINITY ? 0.0f : FP8 ? m[nb][e] - 15.0f : m[nb][e];
#pragma unroll
                    for (int x = 0; x < C::SUB; x++) {
                        s[x][nb][e] = pow2(s[x][nb][e] - sub);
                        s[x][nb][2 + e] = pow2(s[x][nb][2 + e] - sub);
                        l[nb][e] += s[x][nb][e] + s[x][nb][2 + e];
                    }
                }
            // O^T += V^T P^T
            if (!FP8) {
                const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int x = 0; x < C::SUB; x++) {
                    uint32_t b0[NB][2], b1[NB][2];
#pragma unroll
                    for (int nb = 0; nb < NB; nb++) {
                        split2(s[x][nb][0], s[x][nb][1], b0[nb][0], b0[nb][1]);
                        split2(s[x][nb][2], s[x][nb][3], b1[nb][0], b1[nb][1]);
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            b0[nb][w] = transposed(b0[nb][w]);
                            b1[nb][w] = transposed(b1[nb][w]);
                        }
                    }
#pragma unroll
                    for (int d = 0; d < DP / 16; d++) {
                        uint32_t f[4];
                        ldmatrix_t(f, vt + (x * 16 + row) * C::ROW + (((2 * d + ((lane >> 3) & 1)) ^ (row & 7)) * 16));
#pragma unroll
                        for (int nb = 0; nb < NB; nb++)
#pragma unroll
                            for (int w = 0; w < 2; w++) mma<false>(o[nb][d], f, b0[nb][w], b1[nb][w]);
                    }
                }
            } else {
                auto values = [&](auto wide_tag) {
                    constexpr bool F16 = !decltype(wide_tag)::value;
                    constexpr int PARTS = F16 ? 1 : 2;                 // of a weight
#pragma unroll
                    for (int x = 0; x < C::SUB; x++) {
                        uint32_t b0[NB][PARTS], b1[NB][PARTS];
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) {
                            if constexpr (F16) {
                                b0[nb][0] = pack2<true>(s[x][nb][0], s[x][nb][1]);
                                b1[nb][0] = pack2<true>(s[x][nb][2], s[x][nb][3]);
                            } else {
                                split2(s[x][nb][0], s[x][nb][1], b0[nb][0], b0[nb][1]);
                                split2(s[x][nb][2], s[x][nb][3], b1[nb][0], b1[nb][1]);
                            }
#pragma unroll
                            for (int w = 0; w < PARTS; w++) {
                                b0[nb][w] = transposed(b0[nb][w]);
                                b1[nb][w] = transposed(b1[nb][w]);
                            }
                        }
                        uint32_t factor0[DP / 32], factor1[DP / 32];   // of rows 2j, 2j + 1 and 2j + 8, 2j + 9, two 16-bit numbers each
                        const uint8_t* const factors = prep + C::TILE * (DP / 32) * 4 + (x * 8 + j) * (DP / 32) * 4;
                        get_all(factors, factor0);
                        get_all(factors + 4 * (DP / 32) * 4, factor1);
#pragma unroll
                        for (int i = 0; i < DP / 32; i++) {
                            const uint32_t f0 = factor0[i], f1 = factor1[i];
                            uint32_t c[4];         // codes 4 r8 .. 4 r8 + 3 of the block, rows 2j, 2j + 1, 2j + 8, 2j + 9
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const int row = 2 * j + (e & 1) + (e >> 1) * 8;
                                const int sw = DP == 64 ? ((row >> 1) & 1) << 1 : ((row >> 1) & 3) << 1;
                                c[e] = get<uint32_t>(tile + (C::TILE + x * 16 + row) * C::ROW + (((2 * i + (r8 >> 2)) ^ sw) * 16) + (r8 & 3) * 4);
                            }
                            uint32_t p0[NB][PARTS], p1[NB][PARTS];
#pragma unroll
                            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                                for (int w = 0; w < PARTS; w++) {
                                    p0[nb][w] = times2<F16>(b0[nb][w], f0);
                                    p1[nb][w] = times2<F16>(b1[nb][w], f1);
                                }
#pragma unroll
                            for (int h = 0; h < 2; h++) {  // codes 4 r8 + 2h and 4 r8 + 2h + 1: rows r8 and r8 + 8 of the operand
                                uint32_t f[4];
                                const uint32_t sel = h ? 0x7362u : 0x5140u;
                                halves(__byte_perm(c[0], c[1], sel), f[0], f[1]);
                                halves(__byte_perm(c[2], c[3], sel), f[2], f[3]);
                                if (!F16) {
#pragma unroll
                                    for (int e = 0; e < 4; e++) f[e] = to_bf16x2(f[e]);
                                }
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                                    for (int w = 0; w < PARTS; w++) mma<F16>(o[nb][2 * i + h], f, p0[nb][w], p1[nb][w]);
                            }
                        }
                    }
                };
                if (wide) values(std::true_type());
                else values(std::false_type());
            }
            __syncwarp();
            take = take + 1 == C::STAGES ? 0 : take + 1;
            issue();
        }

        // -------- the warps' sums joined, while the next segment's heads are on their way
        const Walk now = w;
        w.next(a, pairs, C::UNIT);
        if (w.left > 0) load_q();
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                l[nb][e] += __shfl_xor_sync(FULL, l[nb][e], 4);
                l[nb][e] += __shfl_xor_sync(FULL, l[nb][e], 8);
                l[nb][e] += __shfl_xor_sync(FULL, l[nb][e], 16);
                if (FP8) l[nb][e] *= 0x1p-15f;         // (from here on without the fp16 weights' factor)
                if (r8 == 0) ml[warp * 8 * NB + nb * 8 + 2 * j + e] = make_float2(m[nb][e], l[nb][e]);
            }
        __syncthreads();
        const int kv = now.pair / a.tiles_of_heads, h0 = (now.pair - kv * a.tiles_of_heads) * 8 * NB;
        const bool cut = now.u > 0 || now.u1 < now.units;
        const int slot = 2 * blockIdx.x + (now.u > 0 ? 0 : 1);
        const float o_scale = FP8 ? two_to(vref - 127) : 1.0f;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float top = -INFINITY;
#pragma unroll
                for (int v = 0; v < PA_WARPS; v++) top = fmaxf(top, ml[v * 8 * NB + nb * 8 + 2 * j + e].x);
                f[e] = top == -INFINITY ? 1.0f : pow2(m[nb][e] - top);
                if (FP8) f[e] *= 0x1p-15f;
            }
#pragma unroll
            for (int half = 0; half < 2; half++) {
                float* const mine = join + warp * 8 * (C::HALF + 4);
#pragma unroll
                for (int d = 0; d < C::HALF / 16; d++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int at = FP8 ? (d / 2) * 32 + r8 * 4 + (d % 2) * 2 + (e >> 1) : d * 16 + r8 + (e >> 1) * 8;
                        mine[(2 * j + (e & 1)) * (C::HALF + 4) + at] = o[nb][half * (C::HALF / 16) + d][e] * f[e & 1] * o_scale;
                    }
                __syncthreads();
                // eight elements of a head a thread and turn
                for (int i = threadIdx.x; i < 8 * C::HALF / 8; i += PA_THREADS) {
                    const int h = i / (C::HALF / 8), d = (i - h * (C::HALF / 8)) * 8;
                    float top = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int v = 0; v < PA_WARPS; v++) top = fmaxf(top, ml[v * 8 * NB + nb * 8 + h].x);
#pragma unroll
                    for (int v = 0; v < PA_WARPS; v++) {
                        const float2 x = ml[v * 8 * NB + nb * 8 + h];
                        sum += top == -INFINITY ? x.y : x.y * pow2(x.x - top);
                    }
                    float v8[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) v8[e] = 0.0f;
#pragma unroll
                    for (int v = 0; v < PA_WARPS; v++)
#pragma unroll
                        for (int e = 0; e < 8; e++) v8[e] += join[(v * 8 + h) * (C::HALF + 4) + d + e];
                    const int head = h0 + nb * 8 + h, at = half * C::HALF + d;
                    if (head < group && at < dim) {
                        if (!cut) {
                            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                            for (int e = 0; e < 8; e++) v8[e] *= inv;
                            const long long row = (long long)now.b * a.q_heads + kv * group + head;
                            *reinterpret_cast<uint4*>(a.out + row * dim + at) = f32_to_bf16x8(v8);
                            if (a.lse && at == 0)
                                a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
                        } else {
                            float* const to = a.part + (long long)slot * C::SLOT + (nb * 8 + h) * DP + at;
                            *reinterpret_cast<float4*>(to) = make_float4(v8[0], v8[1], v8[2], v8[3]);
                            *reinterpret_cast<float4*>(to + 4) = make_float4(v8[4], v8[5], v8[6], v8[7]);
                            if (at == 0) a.part_ml[slot * 8 * NB + nb * 8 + h] = make_float2(top, sum);
                        }
                    }
                }
                __syncthreads();
            }
        }
        if (now.u == 0 && now.u1 < now.units && threadIdx.x == 0) {
            // the block that has the pair's last step: the largest whose stretch begins at or before it
            const long long begin = total * (blockIdx.x + 1) / ctas - now.left - now.at, end = begin + PA_BEGIN + now.units - 1;
            const int last = (int)(((end + 1) * ctas - 1) / total);
            a.cut[blockIdx.x] = make_int4(now.b, now.pair, last - (int)blockIdx.x, 0);
        }
    }
    copies_wait<0>();
}

// Pairs that were cut: block (i, g) joins four heads of the one that begins in block i of the first kernel. Its threads
// take four elements of a head each, in groups that share the pieces out; a piece's loads do not wait for the maxima.
constexpr int PA_JOIN = 512;
constexpr int PA_JOIN_HEADS = 4;

template <bool FP8, int DP, int NB>
__global__ void __launch_bounds__(PA_JOIN) attention_join_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<FP8, DP, NB>;
    constexpr int LANES = DP / 4, GROUPS = PA_JOIN / LANES / PA_JOIN_HEADS, AHEAD = 8;
    __shared__ float factor[PA_JOIN_HEADS][PA_MAX_CTAS], sums[PA_JOIN_HEADS], tops[PA_JOIN_HEADS];
    __shared__ float4 joined[GROUPS][PA_JOIN_HEADS][LANES];
    const int lane = threadIdx.x % LANES, at = threadIdx.x / LANES, hh = at % PA_JOIN_HEADS, g = at / PA_JOIN_HEADS;
    const int h = blockIdx.y * PA_JOIN_HEADS + hh, warp = threadIdx.x / 32;
    pdl_wait();
    const int4 cut = __ldcg(a.cut + blockIdx.x);
    if (cut.x < 0) return;
    // the first piece is in the block's second slot; the blocks after it have theirs in their first
    const int parts = cut.z + 1;
    auto slot_of = [&](int k) { return (long long)(k ? 2 * (blockIdx.x + k) : 2 * blockIdx.x + 1); };
    auto piece = [&](int k) {
        return k < parts ? __ldcg(reinterpret_cast<const float4*>(a.part + slot_of(k) * C::SLOT + h * DP) + lane) : make_float4(0, 0, 0, 0);
    };
    float4 y[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; e++) y[e] = piece(g + e * GROUPS);
    if (warp < PA_JOIN_HEADS) {
        const float2* const ml = a.part_ml + blockIdx.y * PA_JOIN_HEADS + warp;
        float top = -INFINITY, sum = 0.0f;
        for (int k = lane_id(); k < parts; k += 32) top = fmaxf(top, __ldcg(ml + slot_of(k) * 8 * NB).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        for (int k = lane_id(); k < parts; k += 32) {
            const float2 x = __ldcg(ml + slot_of(k) * 8 * NB);
            const float f = top == -INFINITY ? 1.0f : pow2(x.x - top);
            factor[warp][k] = f;
            sum += x.y * f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (lane_id() == 0) {
            tops[warp] = top;
            sums[warp] = sum;
        }
    }
    __syncthreads();
    float4 v = make_float4(0, 0, 0, 0);
    for (int k0 = g; k0 < parts; k0 += AHEAD * GROUPS) {
#pragma unroll
        for (int e = 0; e < AHEAD; e++) {
            const int k = k0 + e * GROUPS;
            if (k >= parts) break;
            const float f = factor[hh][k];
            v.x += y[e].x * f;
            v.y += y[e].y * f;
            v.z += y[e].z * f;
            v.w += y[e].w * f;
        }
#pragma unroll
        for (int e = 0; e < AHEAD; e++) y[e] = piece(k0 + (AHEAD + e) * GROUPS);
    }
    joined[g][hh][lane] = v;
    __syncthreads();
    const int kv = cut.y / a.tiles_of_heads, group = a.q_heads / a.c.heads, head = (cut.y - kv * a.tiles_of_heads) * 8 * NB + h;
    if (g > 0 || head >= group) return;
#pragma unroll
    for (int e = 1; e < GROUPS; e++) {
        const float4 o = joined[e][hh][lane];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    const long long row = (long long)cut.x * a.q_heads + kv * group + head;
    const float sum = sums[hh], inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (lane * 4 < a.c.dim) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), up = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(a.out + row * a.c.dim + lane * 4) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&up));
    }
    if (a.lse && lane == 0)
        a.lse[row] = sum == 0.0f ? -INFINITY : (tops[hh] + log2f(sum)) * 0.69314718055994530942f;
}

// Blocks of 8 query heads that a warp holds at once, by the group: what does not fit is another pass over the cache.
int head_blocks(int group, int dim) { return group <= 8 ? 1 : group <= 16 || dim > 128 ? 2 : 4; }
int padded(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

size_t part_bytes(int nb, int dp) { return (size_t)2 * PA_MAX_CTAS * 8 * nb * dp * sizeof(float); }
size_t ml_bytes(int nb) { return (size_t)2 * PA_MAX_CTAS * 8 * nb * sizeof(float2); }

template <bool FP8, int DP, int NB>
moe_status launch(const AttnArgs& a, cudaStream_t s) {
    using C = Cfg<FP8, DP, NB>;
    static moe_host::PerDevice smem, sms_of;
    if (!moe_host::allow_smem(attention_kernel<FP8, DP, NB>, C::SMEM, smem)) return MOE_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const int sms = sms_of.get(dev, [&] {
        int n = 0;
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
    });
    if (sms == 0) return MOE_ERR_CUDA;
    // stretches of at least PA_MIN_UNITS steps, as far as the table's room for positions tells
    const long long room = (long long)a.M * a.c.page_size, pairs = (long long)a.B * a.c.heads * a.tiles_of_heads;
    const long long steps = (((a.window > 0 && a.window < room ? a.window : room) + C::UNIT - 1) / C::UNIT + PA_BEGIN) * pairs;
    const long long fill = a.whole ? pairs : (steps + PA_MIN_UNITS - 1) / PA_MIN_UNITS;
    long long ctas = (long long)sms * C::CTAS;
    if (ctas > PA_MAX_CTAS) ctas = PA_MAX_CTAS;
    if (ctas > fill) ctas = fill;
    attention_kernel<FP8, DP, NB><<<(unsigned)ctas, PA_THREADS, C::SMEM, s>>>(a);
    const moe_status st = moe_host::launch_status();
    if (st != MOE_OK || a.whole) return st;
    if (moe_host::launch_pdl(attention_join_kernel<FP8, DP, NB>, dim3((unsigned)ctas, 8 * NB / PA_JOIN_HEADS), dim3(PA_JOIN), 0, s, a) != cudaSuccess)
        return MOE_ERR_CUDA;
    return moe_host::launch_status();
}

template <bool FP8>
moe_status launch_of(const AttnArgs& a, int nb, cudaStream_t s) {
    switch (padded(a.c.dim)) {
        case 64: return nb == 1 ? launch<FP8, 64, 1>(a, s) : nb == 2 ? launch<FP8, 64, 2>(a, s) : launch<FP8, 64, 4>(a, s);
        case 128: return nb == 1 ? launch<FP8, 128, 1>(a, s) : nb == 2 ? launch<FP8, 128, 2>(a, s) : launch<FP8, 128, 4>(a, s);
        default: return nb == 1 ? launch<FP8, 256, 1>(a, s) : launch<FP8, 256, 2>(a, s);
    }
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_paged_attention_workspace_size(int B, int q_heads, int heads, int dim) {
    using namespace moe;
    if (B < 0 || B > 65535 || heads < 1 || q_heads < 1 || q_heads % heads || q_heads / heads > 1024 || dim < 1 ||
        dim > MOE_CACHE_MAX_DIM)
        return 0;
    const int nb = head_blocks(q_heads / heads, dim);
    return part_bytes(nb, padded(dim)) + ml_bytes(nb) + PA_MAX_CTAS * sizeof(int4);
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
    const int nb = head_blocks(q_heads / heads, dim), dp = padded(dim);
    AttnArgs a = {static_cast<const __nv_bfloat16*>(q), q_stride, B, q_heads, M, window, c, table, lengths, scale,
                  static_cast<__nv_bfloat16*>(out), lse, nullptr, nullptr, nullptr, 0, 0, 0, 0};
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.part = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + part_bytes(nb, dp));
    a.cut = reinterpret_cast<int4*>(ws + part_bytes(nb, dp) + ml_bytes(nb));
    a.tiles_of_heads = (q_heads / heads + 8 * nb - 1) / (8 * nb);
    const long long room = (long long)M * page_size, most = window > 0 && window < room ? window : room;
    a.whole = most <= PA_WHOLE;
    // division by the page size: with 2^(k-1) < page_size <= 2^k and mul = ceil(2^(31+k) / page_size), p mul / 2^(31+k)
    // exceeds p / page_size by less than 2^31 2^k / 2^(31+k) / page_size = 1 / page_size for p < 2^31
    int k = 0;
    while ((1 << k) < page_size) k++;
    a.page_mul = k ? (uint32_t)(((1ull << (31 + k)) + (uint32_t)page_size - 1) / (uint32_t)page_size) : 0u;
    a.page_shift = k ? k - 1 : 0;
    const cudaStream_t s = moe_host::as_stream(stream);
    return dtype == MOE_MXFP8 ? launch_of<true>(a, nb, s) : launch_of<false>(a, nb, s);
}
