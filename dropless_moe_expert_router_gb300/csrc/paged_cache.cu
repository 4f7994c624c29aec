// paged_cache.cu -- the paged key-value cache around the attention of a decoding step: moe_cache_append,
// moe_cache_gather, moe_cache_copy_pages, moe_cache_fork, moe_cache_compact.
//
// Append and gather move rows between [n, heads, dim] and the pages: every byte once, 8 elements a thread, so
// DRAM bounds long prompts and one launch a decoding step. Copies of pages are plain copies. Fork and compact
// are index work on a table and a mark a page, a few hundred kilobytes: latency bounds them. They run as one block
// with the marks in shared memory where those fit and the table is not long, else as one cluster of eight blocks with
// the marks in the workspace, phases parted by cluster barriers. So a whole call is one launch.
//
// Measured (one GB300): append of 64 tokens 2.8 us; 8192 tokens of 8 heads of 128 into MXFP8 13.4 to 15.5 us and back 13 us (7.5 us of
// bytes each at the copy's rate; 3.4 waves of blocks for the append, whose 52 registers let four of them on an SM, and 2.2 for the
// gather, each a chain of position, table and row), bf16 14.0 and 14.3 (9.9); fork of 4 beams 6 us, of 32 x 8 beams over
// 33,000 table entries 14.5 us; the copies of 88 pages in four layers 9 us, of 2,100 pages in two 24 to 33 us.
#include "common.cuh"
#include "paged_cache.cuh"

#include <cooperative_groups.h>

namespace moe {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ rows in and out
constexpr int RW_THREADS = 256;

struct RowsArgs {
    void* k;                      // [n, heads, dim] bf16
    void* v;
    long long k_stride, v_stride; // elements between tokens
    const int32_t* rows;
    const int32_t* positions;
    const int32_t* table;
    int n, S, M;
    CachePools c;
};

// The element of a pool at which token i's position begins in the first head's pages; -1: skipped or bad.
__device__ __forceinline__ long long place_of(const RowsArgs& a, int i) {
    const int pos = __ldg(a.positions + i);
    const int row = a.rows ? __ldg(a.rows + i) : i;
    if (pos < 0 || row < 0) return -1;
    const int col = pos / a.c.page_size;
    const int p = row < a.S && col < a.M ? __ldg(a.table + (long long)row * a.M + col) : -1;
    if ((unsigned)p < (unsigned)a.c.pages) return ((long long)p * a.c.heads * a.c.page_size + (pos - col * a.c.page_size)) * a.c.dim;
    raise_device_error(MOE_DEVERR_BAD_ID);
    return -1;
}

// A thread moves one piece (8 elements of a side and head) of EACH tokens, so what depends on the piece is found once; four
// neighbours share a 32-element block. A block's threads are a token's pieces (blockIdx.y: 256 of them), or those of
// several tokens side by side where a token has fewer; its tokens are looked up once, by a thread each.
template <bool FP8, bool WRITE, int EACH>
__global__ void __launch_bounds__(RW_THREADS) cache_rows_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ long long places[RW_THREADS / 4 * EACH];    // (a token has four pieces at least)
    const int dim8 = a.c.dim / 8, side = a.c.heads * dim8, per_token = 2 * side;
    const int beside = max(1, RW_THREADS / per_token);     // tokens side by side
    const int token0 = blockIdx.x * beside * EACH;
    if ((int)threadIdx.x < beside * EACH) places[threadIdx.x] = token0 + (int)threadIdx.x < a.n ? place_of(a, token0 + threadIdx.x) : -1;
    __syncthreads();
    const int sub = per_token < RW_THREADS ? (int)threadIdx.x / per_token : 0;
    const int piece = blockIdx.y * RW_THREADS + threadIdx.x - sub * per_token;
    const bool mine = sub < beside && piece < per_token, is_v = piece >= side;
    const int in_side = is_v ? piece - side : piece, head = in_side / dim8, d8 = in_side - head * dim8;
    const long long stride = 2 * (is_v ? a.v_stride : a.k_stride), step = beside * stride;
    char* const dense = static_cast<char*>(is_v ? a.v : a.k) + (long long)(token0 + sub) * stride + 16ll * in_side;
    const long long in_page = (long long)head * a.c.page_size * a.c.dim + 8 * d8;
    char* const pool = static_cast<char*>(is_v ? a.c.v : a.c.k) + (FP8 ? 1 : 2) * in_page;
    uint8_t* const scale = FP8 ? (is_v ? a.c.v_scales : a.c.k_scales) + in_page / 32 : nullptr;     // (dim is whole blocks)
    long long place[EACH];
    uint4 v[EACH];
#pragma unroll
    for (int e = 0; e < EACH; e++) {
        place[e] = mine ? places[e * beside + sub] : -1;
        v[e] = make_uint4(0, 0, 0, 0);
        if (place[e] < 0) continue;
        if (WRITE) {
            v[e] = __ldg(reinterpret_cast<const uint4*>(dense + e * step));
        } else if (FP8) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(pool + place[e]));
            v[e] = make_uint4(q.x, q.y, __ldg(scale + (place[e] >> 5)), 0u);
        } else {
            v[e] = __ldg(reinterpret_cast<const uint4*>(pool + 2 * place[e]));
        }
    }
#pragma unroll
    for (int e = 0; e < EACH; e++) {
        float f[8];
        const bool ok = place[e] >= 0;
        if (WRITE && FP8) {
            int byte;
            bf16x8_to_f32(v[e], f);
            const uint2 q = quant8_in_quad(f, &byte);
            if (ok) {
                *reinterpret_cast<uint2*>(pool + place[e]) = q;
                if ((d8 & 3) == 0) scale[place[e] >> 5] = (uint8_t)byte;
            }
        } else if (WRITE) {
            if (ok) *reinterpret_cast<uint4*>(pool + 2 * place[e]) = v[e];
        } else if (mine && token0 + e * beside + sub < a.n) {
            if (FP8) {
                const float s = e8m0_value(v[e].z);
                e4m3x4_to_f32(v[e].x, f);
                e4m3x4_to_f32(v[e].y, f + 4);
#pragma unroll
                for (int k = 0; k < 8; k++) f[k] *= s;
                v[e] = ok ? f32_to_bf16x8(f) : make_uint4(0, 0, 0, 0);
            }
            *reinterpret_cast<uint4*>(dense + e * step) = v[e];
        }
    }
}

// ------------------------------------------------------------------ copies of pages
constexpr int CP_THREADS = 256;
constexpr int CP_GROUP = 128;        // pools a launch (their table is a kernel parameter)
constexpr int CP_PIECE = 16384;      // bytes a block copies at a time: four 16-byte loads a thread in flight
constexpr int CP_PAIRS = 2048;       // pairs looked at together

struct CopyTable {
    char* at[CP_GROUP];
    long long bytes[CP_GROUP];       // a page's
    int first[CP_GROUP + 1];         // first piece of each pool
    int n;
};

__device__ __forceinline__ void copy_piece(const char* from, char* to, int bytes, bool wide) {
    if (wide) {
        const uint4* s = reinterpret_cast<const uint4*>(from);
        uint4* d = reinterpret_cast<uint4*>(to);
        const int n = bytes / 16;
        uint4 v[CP_PIECE / 16 / CP_THREADS];
#pragma unroll
        for (int u = 0; u < CP_PIECE / 16 / CP_THREADS; u++) {
            const int j = threadIdx.x + u * CP_THREADS;
            if (j < n) v[u] = __ldg(s + j);
        }
#pragma unroll
        for (int u = 0; u < CP_PIECE / 16 / CP_THREADS; u++) {
            const int j = threadIdx.x + u * CP_THREADS;
            if (j < n) d[j] = v[u];
        }
    } else {
        for (int j = threadIdx.x; j < bytes; j += CP_THREADS) to[j] = from[j];
    }
}

// Every block reads the list, 2048 pairs at a time, and keeps those that are to be copied; their pieces go round
// the blocks, so a long list of few pairs costs its reading and keeps every block busy.
__global__ void __launch_bounds__(CP_THREADS) copy_pages_kernel(const __grid_constant__ CopyTable t, const int32_t* src,
                                                                const int32_t* dst, int n, int pages) {
    __shared__ int2 pair[CP_PAIRS];
    __shared__ int warp_count[CP_THREADS / 32];
    const int pieces = t.first[t.n];
    long long before = 0;                                  // pieces of the pairs of earlier rounds
    for (int p0 = 0; p0 < n; p0 += CP_PAIRS) {
        int count = 0;
        for (int q = 0; q < CP_PAIRS && p0 + q < n; q += CP_THREADS) {
            const int p = p0 + q + threadIdx.x;
            int s = -1, d = -1;
            if (p < n) {
                s = __ldg(src + p);
                d = __ldg(dst + p);
                if ((s < -1 || s >= pages || d < -1 || d >= pages) && blockIdx.x == 0) raise_device_error(MOE_DEVERR_BAD_ID);
            }
            const bool ok = (unsigned)s < (unsigned)pages && (unsigned)d < (unsigned)pages;
            const unsigned who = __ballot_sync(FULL, ok);
            __syncthreads();
            if (lane_id() == 0) warp_count[threadIdx.x / 32] = __popc(who);
            __syncthreads();
            int mine = count, all = 0;
            for (int w = 0; w < CP_THREADS / 32; w++) {
                if (w < (int)threadIdx.x / 32) mine += warp_count[w];
                all += warp_count[w];
            }
            if (ok) pair[mine + __popc(who & lanemask_lt())] = make_int2(s, d);
            count += all;
        }
        __syncthreads();
        const long long todo = (long long)count * pieces;
        // the first piece at or after `before` that is this block's
        for (long long j = (blockIdx.x + (long long)gridDim.x - before % gridDim.x) % gridDim.x; j < todo; j += gridDim.x) {
            const int2 sd = pair[j / pieces];
            const int piece = (int)(j % pieces);
            int lo = 0, hi = t.n - 1;                      // the pool that the piece is of
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (t.first[mid] <= piece) lo = mid;
                else hi = mid - 1;
            }
            const long long at = (long long)(piece - t.first[lo]) * CP_PIECE, b = t.bytes[lo];
            const int m = (int)min(b - at, (long long)CP_PIECE);
            const bool wide = (b % 16) == 0 && (reinterpret_cast<uintptr_t>(t.at[lo]) % 16) == 0;
            copy_piece(t.at[lo] + sd.x * b + at, t.at[lo] + sd.y * b + at, m, wide);
        }
        before += todo;
    }
}

// ------------------------------------------------------------------ fork and compact
constexpr int PG_THREADS = 1024;
constexpr int PG_CTAS = 8;           // blocks of the cluster
constexpr int PG_FLIGHT = 8;         // table entries that a thread has in flight
constexpr int PG_NEAR = 4096;        // entries of the list of pages that shared memory holds
constexpr size_t PG_SMEM = 200 * 1024;
constexpr long long PG_ONE = 16;     // table entries a thread of the single block (32: 20 us against the cluster's 14.5)

// Workspace: marks [pages], list [pages], counts [64] (int32), then for a fork offsets [rows].
struct PagesWork {
    uint32_t* mark;
    int32_t* list;
    int32_t* count;
    int32_t* row;
};

__host__ __device__ inline PagesWork pages_work(void* ws, int pages) {
    PagesWork w;
    w.mark = static_cast<uint32_t*>(ws);
    w.list = static_cast<int32_t*>(ws) + pages;
    w.count = w.list + pages;
    w.row = w.count + 64;
    return w;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    __syncthreads();
    if (lane_id() == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[lane_id() & (PG_THREADS / 32 - 1)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// Exclusive prefix sum over the block; *all: the total.
__device__ __forceinline__ int block_scan(int v, int* red, int* all) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, x, o);
        if ((int)lane_id() >= o) x += y;
    }
    __syncthreads();
    if (lane_id() == 31) red[threadIdx.x / 32] = x;
    __syncthreads();
    int w = red[lane_id()];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, w, o);
        if ((int)lane_id() >= o) w += y;
    }
    *all = __shfl_sync(FULL, w, 31);
    const int before = __shfl_sync(FULL, w, max(0, (int)threadIdx.x / 32 - 1));
    return (threadIdx.x < 32 ? 0 : before) + x - v;
}

struct ForkArgs {
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* parents;
    const int32_t* rooms;
    int S, M, S_new, pages, page_size, room;
    int32_t* new_table;
    int32_t* new_lengths;
    int32_t* src;
    int32_t* dst;
    int32_t* used;
    PagesWork w;
};

// The chunk of the pages that block b of the cluster looks at.
__device__ __forceinline__ void chunk_of(int pages, int b, int ctas, int* lo, int* hi) {
    *lo = (int)((long long)pages * b / ctas);
    *hi = (int)((long long)pages * (b + 1) / ctas);
}

__device__ __forceinline__ int parent_of(const ForkArgs& a, int i) { return a.parents ? __ldg(a.parents + i) : i; }

__device__ __forceinline__ int length_of(const ForkArgs& a, int par) {
    const int l = par >= 0 && par < a.S ? __ldg(a.lengths + par) : 0;
    return l < 0 ? 0 : (int)min((long long)l, (long long)a.M * a.page_size);
}

// The marks and the list of pages given out: in shared memory (ONE: a single block), or in the workspace.
template <bool ONE>
struct Marks {
    uint32_t* m;
    int32_t* near;                   // ONE: the list's first PG_NEAR entries
    int32_t* far;
    __device__ __forceinline__ uint32_t get(int p) const { return ONE ? m[p] : __ldcg(m + p); }
    __device__ __forceinline__ int32_t* entry(int k) const { return ONE && k < PG_NEAR ? near + k : far + k; }
    __device__ __forceinline__ int32_t listed(int k) const { return ONE && k < PG_NEAR ? near[k] : __ldcg(far + k); }
};
template <bool ONE>
__device__ __forceinline__ void all_blocks() {
    if (ONE) __syncthreads();
    else cg::this_cluster().sync();
}
// f(e, i, j) for the entries of rows of M columns, PG_FLIGHT of them at a time by load(i, j) first.
template <typename Load, typename Use>
__device__ __forceinline__ void entries(long long total, int M, int thread, int threads, Load load, Use use) {
    const int di = threads / M, dj = threads - di * M;
    int i = thread / M, j = thread - i * M;
    for (long long e = thread; e < total;) {
        int32_t v[PG_FLIGHT];
        int vi[PG_FLIGHT], vj[PG_FLIGHT];
#pragma unroll
        for (int k = 0; k < PG_FLIGHT; k++) {
            vi[k] = i;
            vj[k] = j;
            v[k] = e + (long long)k * threads < total ? load(i, j) : -1;
            i += di;
            j += dj;
            if (j >= M) {
                j -= M;
                i++;
            }
        }
#pragma unroll
        for (int k = 0; k < PG_FLIGHT; k++)
            if (e + (long long)k * threads < total) use(vi[k], vj[k], v[k]);
        e += (long long)PG_FLIGHT * threads;
    }
}

// What row i, its pages copied and marked, needs: bit 30 a copy of its last page, below it the pages in all.
template <bool ONE>
__device__ __forceinline__ int needs_of(const ForkArgs& a, const Marks<ONE>& marks, int i, int* held_out, int* last_out) {
    const int par = parent_of(a, i);
    const int l = length_of(a, par), ps = a.page_size;
    const int held = l / ps + (l % ps != 0);               // (l + ps passes 2^31)
    *held_out = held;
    *last_out = -1;
    if (par < 0 || par >= a.S) return 0;
    const int room = max(0, a.rooms ? __ldg(a.rooms + i) : a.room);
    if (room == 0) return 0;
    const long long end = min(((long long)l + room + ps - 1) / ps, (long long)a.M);
    int need = (int)end - held;
    if (l % ps) {
        const int page = __ldcg(a.new_table + (long long)i * a.M + held - 1);
        *last_out = page;
        const uint32_t key = (uint32_t)(l - (held - 1) * ps) * a.S_new + (a.S_new - i);
        if (page >= 0 && marks.get(page) != key) need = (need + 1) | (1 << 30);
    }
    return need;
}

template <bool ONE>
__global__ void __launch_bounds__(PG_THREADS) cache_fork_kernel(const __grid_constant__ ForkArgs a) {
    extern __shared__ __align__(16) uint32_t pg_smem[];
    __shared__ int red[PG_THREADS / 32];
    const Marks<ONE> marks = {ONE ? pg_smem + PG_NEAR : a.w.mark, reinterpret_cast<int32_t*>(pg_smem), a.w.list};
    const int ctas = gridDim.x, b = blockIdx.x, ps = a.page_size;
    const int thread = b * PG_THREADS + threadIdx.x, threads = ctas * PG_THREADS;
    for (int p = thread; p < a.pages; p += threads) marks.m[p] = 0u;
    all_blocks<ONE>();

    // rows: the parents' pages, each marked with the most positions that a row has in it, the first such row
    for (int i = thread; i < a.S_new; i += threads) {
        const int par = parent_of(a, i), l = length_of(a, par);
        a.new_lengths[i] = l;
        if (par < -1 || par >= a.S || (par >= 0 && __ldg(a.lengths + par) > l)) raise_device_error(MOE_DEVERR_BAD_ID);
    }
    entries((long long)a.S_new * a.M, a.M, thread, threads,
            [&](int i, int j) {
                const int par = parent_of(a, i);
                return par >= 0 && par < a.S ? __ldg(a.table + (long long)par * a.M + j) : -1;
            },
            [&](int i, int j, int page) {
                const int l = length_of(a, parent_of(a, i));
                if ((long long)j * ps < l) {
                    if ((unsigned)page < (unsigned)a.pages) {
                        const uint32_t fill = (uint32_t)min(l - j * ps, ps);
                        atomicMax(marks.m + page, fill * a.S_new + (a.S_new - i));
                    } else {
                        raise_device_error(MOE_DEVERR_BAD_ID);
                        page = -1;
                    }
                } else {
                    page = -1;
                }
                a.new_table[(long long)i * a.M + j] = page;
            });
    all_blocks<ONE>();

    // free pages of this block's chunk, and (block 0) where each row's pages start among those that are given out
    int lo, hi;
    chunk_of(a.pages, b, ctas, &lo, &hi);
    int n = 0;
    for (int p = lo + threadIdx.x; p < hi; p += PG_THREADS) n += marks.get(p) == 0u;
    n = block_sum(n, red);
    if (!ONE && threadIdx.x == 0) a.w.count[b] = n;
    int wanted = 0, free_before = 0, free_all = n;
    if (b == 0) {
        for (int i0 = 0; i0 < a.S_new; i0 += PG_THREADS) {
            const int i = i0 + threadIdx.x;
            int held = 0, last, all;
            const int need = i < a.S_new ? needs_of(a, marks, i, &held, &last) & ~(1 << 30) : 0;
            const int at = wanted + block_scan(need, red, &all);
            if (i < a.S_new) a.w.row[i] = at;
            wanted += all;
        }
        if (!ONE && threadIdx.x == 0) a.w.count[PG_CTAS] = wanted;
    }
    if (!ONE) {
        all_blocks<ONE>();
        wanted = __ldcg(a.w.count + PG_CTAS);
        free_all = 0;
        for (int c = 0; c < ctas; c++) {
            const int f = __ldcg(a.w.count + c);
            if (c < b) free_before += f;
            free_all += f;
        }
    }
    // the free pages that are given out, in order
    for (int p0 = lo; p0 < hi && free_before < wanted; p0 += PG_THREADS) {
        const int p = p0 + threadIdx.x;
        const int is_free = p < hi && marks.get(p) == 0u;
        int all;
        const int at = free_before + block_scan(is_free, red, &all);
        if (is_free && at < wanted) *marks.entry(at) = p;
        free_before += all;
    }
    all_blocks<ONE>();

    for (int i = thread; i < a.S_new; i += threads) {
        int held, last;
        const int need = needs_of(a, marks, i, &held, &last), pages = need & ~(1 << 30);
        const bool copy = need >> 30;
        const int start = pages ? __ldcg(a.w.row + i) : 0;
        int from = -1, to = -1;
        for (int k = 0; k < pages; k++) {
            const int page = start + k < free_all ? marks.listed(start + k) : -1;
            if (copy && k == 0) {
                from = page >= 0 ? last : -1;
                to = page;
            }
            a.new_table[(long long)i * a.M + held - copy + k] = page;
        }
        a.src[i] = from;
        a.dst[i] = to;
    }
    if (thread == 0) {
        *a.used = (int)min((long long)a.pages - free_all + wanted, 0x7fffffffll);
        if (wanted > free_all) raise_device_error(MOE_DEVERR_NO_PAGE);
    }
}

struct CompactArgs {
    const int32_t* table;
    int pages, moves;
    long long entries;
    int32_t* new_table;
    int32_t* src;
    int32_t* dst;
    int32_t* used;
    PagesWork w;
};

template <bool ONE>
__global__ void __launch_bounds__(PG_THREADS) cache_compact_kernel(const __grid_constant__ CompactArgs a) {
    extern __shared__ __align__(16) uint32_t pg_smem[];
    __shared__ int red[PG_THREADS / 32];
    const Marks<ONE> marks = {ONE ? pg_smem + PG_NEAR : a.w.mark, reinterpret_cast<int32_t*>(pg_smem), a.w.list};
    const int ctas = gridDim.x, b = blockIdx.x;
    const int thread = b * PG_THREADS + threadIdx.x, threads = ctas * PG_THREADS;
    for (int p = thread; p < a.pages; p += threads) marks.m[p] = 0u;
    all_blocks<ONE>();
    entries(a.entries, 1, thread, threads, [&](int i, int) { return a.table[i]; },
            [&](int, int, int page) {
                if ((unsigned)page < (unsigned)a.pages) marks.m[page] = 1u;
                else if (page != -1) raise_device_error(MOE_DEVERR_BAD_ID);
            });
    all_blocks<ONE>();
    int lo, hi;
    chunk_of(a.pages, b, ctas, &lo, &hi);
    int n = 0;
    for (int p = lo + threadIdx.x; p < hi; p += PG_THREADS) n += marks.get(p) != 0u;
    n = block_sum(n, red);
    int live = n, before = 0;        // live pages in all, and before this chunk
    if (!ONE) {
        if (threadIdx.x == 0) a.w.count[b] = n;
        all_blocks<ONE>();
        live = 0;
        for (int c = 0; c < ctas; c++) {
            const int f = __ldcg(a.w.count + c);
            if (c < b) before += f;
            live += f;
        }
    }
    int below = 0;                   // live pages below number `live`
    for (int c = 0; c < ctas; c++) {
        int clo, chi;
        chunk_of(a.pages, c, ctas, &clo, &chi);
        if (chi <= live) {
            below += ONE ? n : __ldcg(a.w.count + c);
        } else {
            int m = 0;
            for (int p = clo + threadIdx.x; p < live; p += PG_THREADS) m += marks.get(p) != 0u;
            below += block_sum(m, red);
            break;
        }
    }
    const int moved = live - below;
    // (marks below `live` stay as they are: other blocks may still count them)
    for (int p0 = lo; p0 < hi; p0 += PG_THREADS) {
        const int p = p0 + threadIdx.x;
        const int is_live = p < hi && marks.get(p) != 0u;
        int all;
        const int lives = before + block_scan(is_live, red, &all);       // live pages below p
        before += all;
        if (p >= hi) continue;
        if (is_live && p >= live) {
            a.src[lives - below] = p;
            marks.m[p] = 2u + (uint32_t)(lives - below);
        } else if (!is_live && p < live) {
            a.dst[p - lives] = p;
            *marks.entry(p - lives) = p;
        }
    }
    for (int j = moved + thread; j < a.moves; j += threads) {
        a.src[j] = -1;
        a.dst[j] = -1;
    }
    if (thread == 0) *a.used = live;
    all_blocks<ONE>();
    entries(a.entries, 1, thread, threads, [&](int i, int) { return a.table[i]; },
            [&](int i, int, int page) {
                if ((unsigned)page < (unsigned)a.pages) {
                    const uint32_t m = marks.get(page);
                    if (m >= 2u) page = marks.listed((int)(m - 2u));
                } else {
                    page = -1;
                }
                a.new_table[i] = page;
            });
}

// One block where the marks fit its shared memory and its threads have few entries each; a cluster above.
template <typename Args>
moe_status launch_pages(void (*one)(const Args), void (*many)(const Args), moe_host::PerDevice& done, const Args& a, int pages,
                        long long entries, cudaStream_t s) {
    const size_t smem = (PG_NEAR + (size_t)pages) * sizeof(uint32_t);
    if (smem <= PG_SMEM && entries <= PG_ONE * PG_THREADS) {
        if (!moe_host::allow_smem(one, smem, done)) return MOE_ERR_CUDA;
        one<<<1, PG_THREADS, smem, s>>>(a);
        return moe_host::launch_status();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(PG_CTAS);
    cfg.blockDim = dim3(PG_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PG_CTAS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, many, a) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return moe_host::launch_status();
}

moe_status rows_call(RowsArgs a, moe_dtype dtype, bool write, moe_stream_t stream) {
    const long long total = (long long)a.n * 2 * a.c.heads * (a.c.dim / 8);
    const long long per_token = 2ll * a.c.heads * (a.c.dim / 8), beside = per_token < RW_THREADS ? RW_THREADS / per_token : 1;
    // Four tokens a thread (four loads in flight) from 512 blocks of one on; one, for latency, below. One against four, us, of
    // tokens of 8 heads of 128 into MXFP8 and back: 64 3.1 3.1 / 3.6 3.6, 256 3.2 3.2 / 3.6 3.6, 512 (512 blocks) 3.7 3.6 / 3.6 3.2,
    // 1024 4.1 4.1 / 3.7 3.7, 4096 11.3 11.5 / 8.7 8.3, 8192 20.4 20.7 / 15.5 13.5; bf16 into bf16: 256 3.1 / 3.1, 1024 3.7 / 3.7,
    // 4096 11.4 / 8.9.
    const int each = total >= 512ll * RW_THREADS ? 4 : 1;
    const long long ctas = (a.n + beside * each - 1) / (beside * each), rows = (per_token + RW_THREADS - 1) / RW_THREADS;
    if (rows > 65535) return MOE_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ctas, (unsigned)rows);
    const cudaStream_t s = moe_host::as_stream(stream);
    auto go = [&](auto kernel) { kernel<<<grid, RW_THREADS, 0, s>>>(a); };
    if (dtype == MOE_MXFP8) {
        if (write) each == 4 ? go(cache_rows_kernel<true, true, 4>) : go(cache_rows_kernel<true, true, 1>);
        else each == 4 ? go(cache_rows_kernel<true, false, 4>) : go(cache_rows_kernel<true, false, 1>);
    } else {
        if (write) each == 4 ? go(cache_rows_kernel<false, true, 4>) : go(cache_rows_kernel<false, true, 1>);
        else each == 4 ? go(cache_rows_kernel<false, false, 4>) : go(cache_rows_kernel<false, false, 1>);
    }
    return moe_host::launch_status();
}

moe_status rows_check(const void* k, const void* v, long long k_stride, long long v_stride, int n, const int32_t* rows,
                      const int32_t* positions, const int32_t* table, int S, int M, const CachePools& c, moe_dtype dtype) {
    if (n < 0 || S < 0) return MOE_ERR_INVALID_ARG;
    const moe_status st = moe_host::check_cache(c, dtype, M);
    if (st != MOE_OK) return st;
    if (n > 1 << 30) return MOE_ERR_UNSUPPORTED;                       // (tokens are counted in 32 bits)
    if (!rows && n > S) return MOE_ERR_INVALID_ARG;
    if (n > 0 && (!k || !v || !positions || !table)) return MOE_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || !moe_host::aligned(k, 16) || !moe_host::aligned(v, 16) || !moe_host::aligned(rows, 4) ||
        !moe_host::aligned(positions, 4) || !moe_host::aligned(table, 4))
        return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_cache_append(const void* k, const void* v, long long k_stride, long long v_stride, int n,
                                       const int32_t* rows, const int32_t* positions, const int32_t* table, int S, int M,
                                       moe_dtype dtype, int pages, int heads, int page_size, int dim, void* k_pages,
                                       uint8_t* k_scales, void* v_pages, uint8_t* v_scales, moe_stream_t stream) {
    using namespace moe;
    const CachePools c = {k_pages, v_pages, k_scales, v_scales, pages, heads, page_size, dim};
    const moe_status st = rows_check(k, v, k_stride, v_stride, n, rows, positions, table, S, M, c, dtype);
    if (st != MOE_OK || n == 0) return st;
    const RowsArgs a = {const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride, rows, positions, table, n, S, M, c};
    return rows_call(a, dtype, true, stream);
}

extern "C" moe_status moe_cache_gather(void* k, void* v, int n, const int32_t* rows, const int32_t* positions,
                                       const int32_t* table, int S, int M, moe_dtype dtype, int pages, int heads,
                                       int page_size, int dim, const void* k_pages, const uint8_t* k_scales,
                                       const void* v_pages, const uint8_t* v_scales, moe_stream_t stream) {
    using namespace moe;
    const CachePools c = {const_cast<void*>(k_pages), const_cast<void*>(v_pages), const_cast<uint8_t*>(k_scales),
                          const_cast<uint8_t*>(v_scales), pages, heads, page_size, dim};
    const long long stride = (long long)heads * dim;
    const moe_status st = rows_check(k, v, 0, 0, n, rows, positions, table, S, M, c, dtype);
    if (st != MOE_OK || n == 0) return st;
    const RowsArgs a = {k, v, stride, stride, rows, positions, table, n, S, M, c};
    return rows_call(a, dtype, false, stream);
}

extern "C" size_t moe_cache_pages_workspace_size(int pages, int rows) {
    if (pages < 1 || rows < 0) return 0;
    return sizeof(int32_t) * (2 * (size_t)pages + 64 + (size_t)rows);
}

static moe_status pages_check(int S, int M, int rows, int pages, const void* workspace, size_t workspace_bytes) {
    if (S < 0 || M < 1 || rows < 0 || pages < 1) return MOE_ERR_INVALID_ARG;
    if (pages > 1 << 30) return MOE_ERR_UNSUPPORTED;                   // (strides over them are counted in 32 bits)
    if (!workspace || workspace_bytes < moe_cache_pages_workspace_size(pages, rows)) return MOE_ERR_WORKSPACE;
    return moe_host::aligned(workspace, 16) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

extern "C" moe_status moe_cache_fork(const int32_t* table, const int32_t* lengths, int S, int M, const int32_t* parents,
                                     int S_new, int pages, int page_size, int room, const int32_t* rooms,
                                     int32_t* new_table, int32_t* new_lengths, int32_t* src, int32_t* dst, int32_t* used,
                                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    if (S_new < 0 || S < 0 || M < 1 || pages < 1 || page_size < 1 || page_size > MOE_CACHE_MAX_PAGE ||
        (long long)M * page_size >= (1ll << 31) || (long long)page_size * S_new >= (1ll << 31) - S_new || (long long)M * S_new >= (1ll << 31))
        return MOE_ERR_INVALID_ARG;
    if (!parents && S_new != S) return MOE_ERR_INVALID_ARG;
    if ((S > 0 && (!table || !lengths)) || !used) return MOE_ERR_INVALID_ARG;
    if (S_new > 0 && (!new_table || !new_lengths || !src || !dst)) return MOE_ERR_INVALID_ARG;
    const moe_status st = pages_check(S, M, S_new, pages, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    for (const void* p : {(const void*)table, (const void*)lengths, (const void*)parents, (const void*)rooms,
                          (const void*)new_table, (const void*)new_lengths, (const void*)src, (const void*)dst, (const void*)used})
        if (!moe_host::aligned(p, 4)) return MOE_ERR_ALIGNMENT;
    const ForkArgs a = {table, lengths, parents, rooms, S, M, S_new, pages, page_size, room, new_table, new_lengths, src, dst,
                        used, pages_work(workspace, pages)};
    static moe_host::PerDevice done;
    return launch_pages(cache_fork_kernel<true>, cache_fork_kernel<false>, done, a, pages, (long long)S_new * M,
                        moe_host::as_stream(stream));
}

extern "C" moe_status moe_cache_compact(const int32_t* table, int S, int M, int pages, int32_t* new_table, int32_t* src,
                                        int32_t* dst, int32_t* used, void* workspace, size_t workspace_bytes,
                                        moe_stream_t stream) {
    using namespace moe;
    if ((S > 0 && (!table || !new_table)) || !used || (pages > 1 && (!src || !dst))) return MOE_ERR_INVALID_ARG;
    const moe_status st = pages_check(S, M, 0, pages, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    for (const void* p : {(const void*)table, (const void*)new_table, (const void*)src, (const void*)dst, (const void*)used})
        if (!moe_host::aligned(p, 4)) return MOE_ERR_ALIGNMENT;
    const long long entries = (long long)S * M;
    const CompactArgs a = {table, pages, pages / 2, entries, new_table, src, dst, used, pages_work(workspace, pages)};
    static moe_host::PerDevice done;
    if (entries >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    return launch_pages(cache_compact_kernel<true>, cache_compact_kernel<false>, done, a, pages, entries, moe_host::as_stream(stream));
}

extern "C" moe_status moe_cache_copy_pages(void* const* tensors, const long long* page_bytes, int n_tensors,
                                           const int32_t* src, const int32_t* dst, int n, int pages, moe_stream_t stream) {
    using namespace moe;
    if (n < 0 || n_tensors < 0 || pages < 1) return MOE_ERR_INVALID_ARG;
    if (n > 0 && (!src || !dst)) return MOE_ERR_INVALID_ARG;
    if (n_tensors > 0 && (!tensors || !page_bytes)) return MOE_ERR_INVALID_ARG;
    if (n > 1 << 30) return MOE_ERR_UNSUPPORTED;                       // (pairs are counted in 32 bits)
    for (int i = 0; i < n_tensors; i++) {
        if (!tensors[i] || page_bytes[i] < 1) return MOE_ERR_INVALID_ARG;
        if (page_bytes[i] > (1ll << 32)) return MOE_ERR_UNSUPPORTED;   // (pieces are counted in 32 bits)
    }
    if (!moe_host::aligned(src, 4) || !moe_host::aligned(dst, 4)) return MOE_ERR_ALIGNMENT;
    if (n == 0) return MOE_OK;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i0 = 0; i0 < n_tensors; i0 += CP_GROUP) {
        CopyTable t;
        t.n = 0;
        int pieces = 0;
        for (int i = i0; i < n_tensors && i < i0 + CP_GROUP; i++) {
            t.at[t.n] = static_cast<char*>(tensors[i]);
            t.bytes[t.n] = page_bytes[i];
            t.first[t.n] = pieces;
            pieces += (int)((page_bytes[i] + CP_PIECE - 1) / CP_PIECE);
            t.n++;
        }
        t.first[t.n] = pieces;
        const long long most = (long long)n * pieces, fill = sms * 6;
        copy_pages_kernel<<<(unsigned)(most < fill ? most : fill), CP_THREADS, 0, moe_host::as_stream(stream)>>>(t, src, dst, n, pages);
    }
    return moe_host::launch_status();
}
