// paged_cache.cu -- the paged key-value cache around the attention of a decoding step: moe_cache_append,
// moe_cache_gather, moe_cache_copy_pages, moe_cache_fork, moe_cache_compact.
//
// Append and gather move rows between [n, heads, dim] and the pages: every byte once, 8 elements a thread, so
// DRAM bounds long prompts and one launch a decoding step. Copies of pages are plain copies. Fork and compact
// are index work on a table and a mark a page, a few hundred kilobytes: latency bounds them. They run as
// one cluster of blocks whose phases are parted by cluster barriers, so a whole call is one launch.
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

// The page of token i's position and the offset in it; false: skipped or bad.
__device__ __forceinline__ bool place_of(const RowsArgs& a, int i, int* page, int* offset) {
    const int pos = __ldg(a.positions + i);
    const int row = a.rows ? __ldg(a.rows + i) : i;
    if (pos < 0 || row < 0) return false;
    const int col = pos / a.c.page_size;
    const int p = row < a.S && col < a.M ? __ldg(a.table + (long long)row * a.M + col) : -1;
    *page = p;
    *offset = pos - col * a.c.page_size;
    if ((unsigned)p < (unsigned)a.c.pages) return true;
    raise_device_error(MOE_DEVERR_BAD_ID);
    return false;
}

// A thread moves 8 elements of one token, head and side; four neighbours share a 32-element block.
template <bool FP8, bool WRITE>
__global__ void __launch_bounds__(RW_THREADS) cache_rows_kernel(const __grid_constant__ RowsArgs a) {
    const int dim8 = a.c.dim / 8, side = a.c.heads * dim8, per_token = 2 * side;
    const long long total = (long long)a.n * per_token;
    // (whole warps go round together: the quantiser's lanes exchange their maxima)
    for (long long base = (long long)blockIdx.x * RW_THREADS; base < total; base += (long long)gridDim.x * RW_THREADS) {
        const long long at = base + threadIdx.x;
        const int i = (int)(at / per_token);
        const int rest = (int)(at - (long long)i * per_token);
        const bool is_v = rest >= side;
        const int in_side = is_v ? rest - side : rest;
        int page = 0, offset = 0;
        const bool ok = at < total && place_of(a, i, &page, &offset);
        char* const dense = static_cast<char*>(is_v ? a.v : a.k) + 2 * ((long long)i * (is_v ? a.v_stride : a.k_stride) + 8 * in_side);
        const int head = in_side / dim8, d8 = in_side - head * dim8;
        const long long line = ((long long)page * a.c.heads + head) * a.c.page_size + offset;
        char* const pool = static_cast<char*>(is_v ? a.c.v : a.c.k);
        if (!FP8) {
            uint4* const at_pool = reinterpret_cast<uint4*>(pool + 2 * (line * a.c.dim + 8 * d8));
            if (WRITE) {
                if (ok) *at_pool = __ldg(reinterpret_cast<const uint4*>(dense));
            } else if (at < total) {
                *reinterpret_cast<uint4*>(dense) = ok ? __ldg(at_pool) : make_uint4(0, 0, 0, 0);
            }
        } else {
            uint2* const at_pool = reinterpret_cast<uint2*>(pool + line * a.c.dim + 8 * d8);
            uint8_t* const at_scale = (is_v ? a.c.v_scales : a.c.k_scales) + line * (a.c.dim / 32) + d8 / 4;
            float f[8];
            if (WRITE) {
                bf16x8_to_f32(ok ? __ldg(reinterpret_cast<const uint4*>(dense)) : make_uint4(0, 0, 0, 0), f);
                int byte;
                const uint2 q = quant8_in_quad(f, &byte);
                if (ok) {
                    *at_pool = q;
                    if ((d8 & 3) == 0) *at_scale = (uint8_t)byte;
                }
            } else if (at < total) {
                uint4 out = make_uint4(0, 0, 0, 0);
                if (ok) {
                    const uint2 q = __ldg(at_pool);
                    const float s = e8m0_value(__ldg(at_scale));
                    e4m3x4_to_f32(q.x, f);
                    e4m3x4_to_f32(q.y, f + 4);
#pragma unroll
                    for (int e = 0; e < 8; e++) f[e] *= s;
                    out = f32_to_bf16x8(f);
                }
                *reinterpret_cast<uint4*>(dense) = out;
            }
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
constexpr int PG_CTAS = 8;           // blocks of the cluster at most

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

// What row i, its pages copied and marked, needs: bit 30 a copy of its last page, below it the pages in all.
__device__ __forceinline__ int needs_of(const ForkArgs& a, int i, int* held_out) {
    const int par = parent_of(a, i);
    const int l = length_of(a, par), ps = a.page_size;
    const int held = (l + ps - 1) / ps;
    *held_out = held;
    if (par < 0 || par >= a.S) return 0;
    const int room = max(0, a.rooms ? __ldg(a.rooms + i) : a.room);
    if (room == 0) return 0;
    const long long end = min(((long long)l + room + ps - 1) / ps, (long long)a.M);
    int need = (int)end - held;
    if (l % ps) {
        const int page = __ldcg(a.new_table + (long long)i * a.M + held - 1);
        const uint32_t key = (uint32_t)(l - (held - 1) * ps) * a.S_new + (a.S_new - i);
        if (page >= 0 && __ldcg(a.w.mark + page) != key) need = (need + 1) | (1 << 30);
    }
    return need;
}

__global__ void __launch_bounds__(PG_THREADS) cache_fork_kernel(const __grid_constant__ ForkArgs a) {
    __shared__ int red[PG_THREADS / 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = gridDim.x, b = blockIdx.x, ps = a.page_size;
    const int thread = b * PG_THREADS + threadIdx.x, threads = ctas * PG_THREADS;
    for (int p = thread; p < a.pages; p += threads) a.w.mark[p] = 0u;
    cluster.sync();

    // rows: the parents' pages, each marked with the most positions that a row has in it, the first such row
    for (int i = thread / 32; i < a.S_new; i += threads / 32) {
        const int par = parent_of(a, i);
        const bool bad = par < -1 || par >= a.S;
        const int l = length_of(a, par);
        if (lane_id() == 0) {
            a.new_lengths[i] = l;
            if (bad || (par >= 0 && !bad && __ldg(a.lengths + par) > l)) raise_device_error(MOE_DEVERR_BAD_ID);
        }
        for (int j = lane_id(); j < a.M; j += 32) {
            int page = -1;
            if ((long long)j * ps < l) {
                page = __ldg(a.table + (long long)par * a.M + j);
                if ((unsigned)page < (unsigned)a.pages) {
                    const uint32_t fill = (uint32_t)min(l - j * ps, ps);
                    atomicMax(a.w.mark + page, fill * a.S_new + (a.S_new - i));
                } else {
                    raise_device_error(MOE_DEVERR_BAD_ID);
                    page = -1;
                }
            }
            a.new_table[(long long)i * a.M + j] = page;
        }
    }
    cluster.sync();

    // free pages of this block's chunk, and (block 0) where each row's pages start among those that are given out
    int lo, hi;
    chunk_of(a.pages, b, ctas, &lo, &hi);
    int n = 0;
    for (int p = lo + threadIdx.x; p < hi; p += PG_THREADS) n += __ldcg(a.w.mark + p) == 0u;
    n = block_sum(n, red);
    if (threadIdx.x == 0) a.w.count[b] = n;
    if (b == 0) {
        int base = 0;
        for (int i0 = 0; i0 < a.S_new; i0 += PG_THREADS) {
            const int i = i0 + threadIdx.x;
            int held = 0, all;
            const int need = i < a.S_new ? needs_of(a, i, &held) & ~(1 << 30) : 0;
            const int at = base + block_scan(need, red, &all);
            if (i < a.S_new) a.w.row[i] = at;
            base += all;
        }
        if (threadIdx.x == 0) a.w.count[PG_CTAS] = base;
    }
    cluster.sync();

    // the free pages that are given out, in order
    const int wanted = __ldcg(a.w.count + PG_CTAS);
    int free_before = 0, free_all = 0;
    for (int c = 0; c < ctas; c++) {
        const int f = __ldcg(a.w.count + c);
        if (c < b) free_before += f;
        free_all += f;
    }
    for (int p0 = lo; p0 < hi && free_before < wanted; p0 += PG_THREADS) {
        const int p = p0 + threadIdx.x;
        const int is_free = p < hi && __ldcg(a.w.mark + p) == 0u;
        int all;
        const int at = free_before + block_scan(is_free, red, &all);
        if (is_free && at < wanted) a.w.list[at] = p;
        free_before += all;
    }
    cluster.sync();

    for (int i = thread; i < a.S_new; i += threads) {
        int held;
        const int need = needs_of(a, i, &held), pages = need & ~(1 << 30);
        const bool copy = need >> 30;
        int from = -1, to = -1;
        for (int k = 0; k < pages; k++) {
            const int at = __ldcg(a.w.row + i) + k;
            const int page = at < free_all ? __ldcg(a.w.list + at) : -1;
            int32_t* entry = a.new_table + (long long)i * a.M + held - copy + k;
            if (copy && k == 0) {
                from = page >= 0 ? __ldcg(entry) : -1;
                to = page;
            }
            *entry = page;
        }
        a.src[i] = from;
        a.dst[i] = to;
    }
    if (thread == 0) {
        *a.used = a.pages - free_all + wanted;
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

__global__ void __launch_bounds__(PG_THREADS) cache_compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int red[PG_THREADS / 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = gridDim.x, b = blockIdx.x;
    const int thread = b * PG_THREADS + threadIdx.x, threads = ctas * PG_THREADS;
    for (int p = thread; p < a.pages; p += threads) a.w.mark[p] = 0u;
    cluster.sync();
    for (long long j = thread; j < a.entries; j += threads) {
        const int page = a.table[j];
        if ((unsigned)page < (unsigned)a.pages) a.w.mark[page] = 1u;
        else if (page != -1) raise_device_error(MOE_DEVERR_BAD_ID);
    }
    cluster.sync();
    int lo, hi;
    chunk_of(a.pages, b, ctas, &lo, &hi);
    int n = 0;
    for (int p = lo + threadIdx.x; p < hi; p += PG_THREADS) n += __ldcg(a.w.mark + p) != 0u;
    n = block_sum(n, red);
    if (threadIdx.x == 0) a.w.count[b] = n;
    cluster.sync();

    // live pages in all, before this chunk, and below that number of all
    int live = 0, before = 0;
    for (int c = 0; c < ctas; c++) {
        const int f = __ldcg(a.w.count + c);
        if (c < b) before += f;
        live += f;
    }
    int below = 0;
    for (int c = 0; c < ctas; c++) {
        int clo, chi;
        chunk_of(a.pages, c, ctas, &clo, &chi);
        if (chi <= live) {
            below += __ldcg(a.w.count + c);
        } else {
            int m = 0;
            for (int p = clo + threadIdx.x; p < live; p += PG_THREADS) m += __ldcg(a.w.mark + p) != 0u;
            below += block_sum(m, red);
            break;
        }
    }
    const int moved = live - below;
    // (marks below `live` stay as they are: other blocks may still count them)
    for (int p0 = lo; p0 < hi; p0 += PG_THREADS) {
        const int p = p0 + threadIdx.x;
        const int is_live = p < hi && __ldcg(a.w.mark + p) != 0u;
        int all;
        const int lives = before + block_scan(is_live, red, &all);       // live pages below p
        before += all;
        if (p >= hi) continue;
        if (is_live && p >= live) {
            a.src[lives - below] = p;
            a.w.mark[p] = 2u + (uint32_t)(lives - below);
        } else if (!is_live && p < live) {
            a.dst[p - lives] = p;
        }
    }
    for (int j = moved + thread; j < a.moves; j += threads) {
        a.src[j] = -1;
        a.dst[j] = -1;
    }
    if (thread == 0) *a.used = live;
    cluster.sync();
    for (long long j = thread; j < a.entries; j += threads) {
        int page = a.table[j];
        if ((unsigned)page < (unsigned)a.pages) {
            const uint32_t m = __ldcg(a.w.mark + page);
            if (m >= 2u) page = __ldcg(a.dst + (m - 2u));
        } else {
            page = -1;
        }
        a.new_table[j] = page;
    }
}

template <typename Args>
moe_status launch_cluster(void (*kernel)(const Args), const Args& a, int ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(PG_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return moe_host::launch_status();
}

// Blocks of the cluster: one where its threads have a handful of entries each.
int pages_ctas(long long work) { return work <= 8 * PG_THREADS ? 1 : PG_CTAS; }

moe_status rows_call(RowsArgs a, moe_dtype dtype, bool write, moe_stream_t stream) {
    const long long total = (long long)a.n * 2 * a.c.heads * (a.c.dim / 8);
    const long long ctas = (total + RW_THREADS - 1) / RW_THREADS;
    const dim3 grid((unsigned)(ctas < (1 << 20) ? ctas : (1 << 20)));
    const cudaStream_t s = moe_host::as_stream(stream);
    if (dtype == MOE_MXFP8) {
        if (write) cache_rows_kernel<true, true><<<grid, RW_THREADS, 0, s>>>(a);
        else cache_rows_kernel<true, false><<<grid, RW_THREADS, 0, s>>>(a);
    } else {
        if (write) cache_rows_kernel<false, true><<<grid, RW_THREADS, 0, s>>>(a);
        else cache_rows_kernel<false, false><<<grid, RW_THREADS, 0, s>>>(a);
    }
    return moe_host::launch_status();
}

moe_status rows_check(const void* k, const void* v, long long k_stride, long long v_stride, int n, const int32_t* rows,
                      const int32_t* positions, const int32_t* table, int S, int M, const CachePools& c, moe_dtype dtype) {
    if (n < 0 || S < 0) return MOE_ERR_INVALID_ARG;
    const moe_status st = moe_host::check_cache(c, dtype, M);
    if (st != MOE_OK) return st;
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
    if (!workspace || workspace_bytes < moe_cache_pages_workspace_size(pages, rows)) return MOE_ERR_WORKSPACE;
    return moe_host::aligned(workspace, 16) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

extern "C" moe_status moe_cache_fork(const int32_t* table, const int32_t* lengths, int S, int M, const int32_t* parents,
                                     int S_new, int pages, int page_size, int room, const int32_t* rooms,
                                     int32_t* new_table, int32_t* new_lengths, int32_t* src, int32_t* dst, int32_t* used,
                                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    if (S_new < 0 || S < 0 || M < 1 || pages < 1 || page_size < 1 || page_size > MOE_CACHE_MAX_PAGE ||
        (long long)M * page_size >= (1ll << 31) || (long long)page_size * S_new >= (1ll << 31) - S_new)
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
    return launch_cluster(cache_fork_kernel, a, pages_ctas((long long)S_new * M + pages), moe_host::as_stream(stream));
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
    return launch_cluster(cache_compact_kernel, a, pages_ctas(entries + pages), moe_host::as_stream(stream));
}

extern "C" moe_status moe_cache_copy_pages(void* const* tensors, const long long* page_bytes, int n_tensors,
                                           const int32_t* src, const int32_t* dst, int n, int pages, moe_stream_t stream) {
    using namespace moe;
    if (n < 0 || n_tensors < 0 || pages < 1) return MOE_ERR_INVALID_ARG;
    if (n > 0 && (!src || !dst)) return MOE_ERR_INVALID_ARG;
    if (n_tensors > 0 && (!tensors || !page_bytes)) return MOE_ERR_INVALID_ARG;
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
