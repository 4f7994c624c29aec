// layer_norm.cu -- the layer norm of a pre-norm block and its backward pass: moe_layer_norm and
// moe_layer_norm_backward.
//
// Forward, per row: s = x (+ residual), mean = sum s / H, rstd = 1 / sqrt(sum (s - mean)^2 / H + eps),
// y = (s - mean) rstd w + b. Backward, with xh = (s - mean) rstd and g = dy w:
// dx = rstd (g - sum(g) / H - xh sum(g xh) / H) (+ dx_add), dw = sum_t dy xh, db = sum_t dy.
// Each operand is read once and each output written once: the bytes bound both directions. A single row
// is latency: 3.8 us at 1 x 4096.
#include "common.cuh"
#include "sm100_ptx.cuh"

#include <initializer_list>

namespace moe {
namespace {

constexpr int LN_HMAX = 65536;
constexpr int LN_STAGES = 6;              // most ring stages of the kernels that go through shared memory
constexpr size_t LN_SMEM = 220 * 1024;    // their dynamic shared memory at most

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive elements, moved in pieces of 16 bytes at most; bf16 pairs stay packed in registers.
template <typename T, int VEC>
struct alignas(VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16) Vec {
    T v[VEC];
    __device__ __forceinline__ float get(int j) const { return to_f(v[j]); }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int j = 0; j < VEC; j++) v[j] = from_f<T>(f[j]);
    }
};
template <int VEC>
struct alignas(VEC * 2 < 16 ? VEC * 2 : 16) VecBf16 {
    uint32_t v[VEC / 2];
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[j], f[j + 1]);
            v[j / 2] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
};
template <>
struct Vec<__nv_bfloat16, 8> : VecBf16<8> {};
template <>
struct Vec<__nv_bfloat16, 4> : VecBf16<4> {};

// Sums of N values over a row's threads (a warp, or the CTA), the same in every thread. red: 32 N floats,
// free again once every thread has passed another such sum through other memory.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], bool warp_row, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; n++) v[n] += __shfl_xor_sync(FULL, v[n], o);
    if (warp_row) return;
    const int warps = blockDim.x >> 5, lane = (int)lane_id();
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; n++) red[n * 32 + (threadIdx.x >> 5)] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = lane < warps ? red[n * 32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; n++) v[n] += __shfl_xor_sync(FULL, v[n], o);
}

// ---------------------------------------------------------------------------
// Forward, the row in registers: a row belongs to a warp (warp_row: 8 rows a CTA) or to a CTA, NV
// pieces of VEC elements per thread, piece i at i * threads + thread. CTAs walk the rows with the
// grid's stride; weight and bias come from L1. For short rows, and for rows off the 16-byte boundary where
// they are short or few or not off it alike; the others take the ring below (ln_shape has the rules; 8192 x 4096
// with a residual took 57 us this way, 47 us by the ring).
// ---------------------------------------------------------------------------
template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(512) ln_forward_kernel(const T* x, const T* residual, int rows, int H, bool warp_row,
                                                         const W* __restrict__ w, const W* __restrict__ b, float eps,
                                                         T* sum, T* y, float* mean_out, float* rstd_out) {
    __shared__ float red[2][32];
    const int tpr = warp_row ? 32 : blockDim.x;
    const int me = threadIdx.x % tpr, groups = blockDim.x / tpr;
    const int n = H / VEC;
    for (long long t = (long long)blockIdx.x * groups + threadIdx.x / tpr; t < rows; t += (long long)gridDim.x * groups) {
        const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(x + t * H);
        Vec<T, VEC> xv[NV], rv[NV];
        float f[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = me + i * tpr;
            if (c < n) {
                xv[i] = xr[c];
                if (residual) rv[i] = reinterpret_cast<const Vec<T, VEC>*>(residual + t * H)[c];
            }
        }
        float m[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = me + i * tpr;
            if (c >= n) continue;
            if (residual) {
#pragma unroll
                for (int j = 0; j < VEC; j++) f[i][j] = xv[i].get(j) + rv[i].get(j);
                xv[i].set(f[i]);
                reinterpret_cast<Vec<T, VEC>*>(sum + t * H)[c] = xv[i];
            }
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                f[i][j] = xv[i].get(j);
                m[0] += f[i][j];
            }
        }
        row_sum(m, warp_row, red[0]);
        const float mean = m[0] / (float)H;
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (me + i * tpr < n)
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    f[i][j] -= mean;
                    q[0] = fmaf(f[i][j], f[i][j], q[0]);
                }
        row_sum(q, warp_row, red[1]);
        const float rstd = 1.0f / sqrtf(q[0] / (float)H + eps);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = me + i * tpr;
            if (c < n) {
                const Vec<W, VEC> wv = reinterpret_cast<const Vec<W, VEC>*>(w)[c];
                Vec<W, VEC> bv;
                if (b) bv = reinterpret_cast<const Vec<W, VEC>*>(b)[c];
                Vec<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; j++) f[i][j] = fmaf(f[i][j] * rstd, wv.get(j), b ? bv.get(j) : 0.0f);
                o.set(f[i]);
                reinterpret_cast<Vec<T, VEC>*>(y + t * H)[c] = o;
            }
        }
        if (me == 0) {
            if (mean_out) mean_out[t] = mean;
            if (rstd_out) rstd_out[t] = rstd;
        }
    }
}

// Forward for rows too long for the ring: a CTA per row, which is read again for each sum (from L2). 1000 x 40000 bf16
// with a residual 76 us (floor 47; element by element 200).
template <typename T, typename W, int VEC>
__global__ void __launch_bounds__(512) ln_forward_long_kernel(const T* x, const T* residual, int H,
                                                              const W* __restrict__ w, const W* __restrict__ b,
                                                              float eps, T* sum, T* y, float* mean_out,
                                                              float* rstd_out) {
    __shared__ float red[2][32];
    using V = Vec<T, VEC>;
    const long long base = (long long)blockIdx.x * H;
    const int n = H / VEC;
    float a[1] = {0.0f};
#pragma unroll(VEC == 1 ? 1 : 2)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        V v = reinterpret_cast<const V*>(x + base)[i];
        if (residual) {
            const V r = reinterpret_cast<const V*>(residual + base)[i];
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) f[j] = v.get(j) + r.get(j);
            v.set(f);
            reinterpret_cast<V*>(sum + base)[i] = v;
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) a[0] += v.get(j);
    }
    const T* s = residual ? sum : x;
    row_sum(a, false, red[0]);
    const float mean = a[0] / (float)H;
    a[0] = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const V v = reinterpret_cast<const V*>(s + base)[i];
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            const float d = v.get(j) - mean;
            a[0] = fmaf(d, d, a[0]);
        }
    }
    row_sum(a, false, red[1]);
    const float rstd = 1.0f / sqrtf(a[0] / (float)H + eps);
#pragma unroll(VEC == 1 ? 1 : 2)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const V v = reinterpret_cast<const V*>(s + base)[i];
        const Vec<W, VEC> wv = reinterpret_cast<const Vec<W, VEC>*>(w)[i];
        Vec<W, VEC> bv;
        if (b) bv = reinterpret_cast<const Vec<W, VEC>*>(b)[i];
        V o;
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) f[j] = fmaf((v.get(j) - mean) * rstd, wv.get(j), b ? bv.get(j) : 0.0f);
        o.set(f);
        reinterpret_cast<V*>(y + base)[i] = o;
    }
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[blockIdx.x] = mean;
        if (rstd_out) rstd_out[blockIdx.x] = rstd;
    }
}

// ---------------------------------------------------------------------------
// Backward, the row in registers (laid out as in the forward). A thread's columns are the same in
// every row, so dweight and dbias add up in its registers over the CTA's rows and leave as one
// partial sum per CTA: part [gridDim.x][2][H]. The next row's loads are issued before this row's
// sums (PRE), so that a CTA that fills its SM has a row in flight at all times.
// ---------------------------------------------------------------------------
template <typename T, typename W, int VEC, int NV, bool PRE>
__global__ void __launch_bounds__(512, 1) ln_backward_kernel(const T* dy, const T* __restrict__ s, int rows, int H,
                                                             bool warp_row, const W* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const T* add, T* dx,
                                                             float* part) {
    extern __shared__ float cols[];       // warp_row: [2][H], the CTA's sums
    __shared__ float red[2][64];
    using V = Vec<T, VEC>;
    const int tpr = warp_row ? 32 : blockDim.x;
    const int me = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int n = H / VEC;
    Vec<W, VEC> wv[NV];
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (me + i * tpr < n) wv[i] = reinterpret_cast<const Vec<W, VEC>*>(w)[me + i * tpr];
#pragma unroll
        for (int j = 0; j < VEC; j++) dw[i][j] = db[i][j] = 0.0f;
    }
    V gv[NV], sv[NV], av[NV];
    float m = 0.0f, r = 0.0f;
    auto load = [&](long long t, V* g_, V* s_, V* a_, float& m_, float& r_) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = me + i * tpr;
            if (c < n) {
                g_[i] = reinterpret_cast<const V*>(dy + t * H)[c];
                s_[i] = reinterpret_cast<const V*>(s + t * H)[c];
                if (add) a_[i] = reinterpret_cast<const V*>(add + t * H)[c];
            }
        }
        m_ = __ldg(mean + t);
        r_ = __ldg(rstd + t);
    };
    const long long step = (long long)gridDim.x * groups;
    long long t = (long long)blockIdx.x * groups + group;
    if (PRE && t < rows) load(t, gv, sv, av, m, r);
    for (int buf = 0; t < rows; t += step, buf ^= 1) {
        V gn[NV], sn[NV], an[NV];
        float mn = 0.0f, rn = 0.0f;
        if (PRE) {
            if (t + step < rows) load(t + step, gn, sn, an, mn, rn);
        } else {
            load(t, gv, sv, av, m, r);
        }
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (me + i * tpr < n)
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const float d = gv[i].get(j), xh = (sv[i].get(j) - m) * r, g = d * wv[i].get(j);
                    sums[0] += g;
                    sums[1] = fmaf(g, xh, sums[1]);
                    dw[i][j] = fmaf(d, xh, dw[i][j]);
                    db[i][j] += d;
                }
        row_sum(sums, warp_row, red[buf]);
        const float a = sums[0] / (float)H, c2 = sums[1] / (float)H;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = me + i * tpr;
            if (c < n) {
                V o;
                float f[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const float xh = (sv[i].get(j) - m) * r, g = gv[i].get(j) * wv[i].get(j);
                    f[j] = r * (g - a - xh * c2);
                    if (add) f[j] += av[i].get(j);
                }
                o.set(f);
                reinterpret_cast<V*>(dx + t * H)[c] = o;
            }
        }
        if (PRE) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                gv[i] = gn[i];
                sv[i] = sn[i];
                av[i] = an[i];
            }
            m = mn;
            r = rn;
        }
    }
    if (!part) return;
    float* out = part + (size_t)blockIdx.x * 2 * H;
    if (warp_row) {
        // the warps' sums one after the other, in a fixed order
        for (int k = 0; k < groups; k++) {
            if (group == k)
#pragma unroll
                for (int i = 0; i < NV; i++)
                    if (me + i * tpr < n)
#pragma unroll
                        for (int j = 0; j < VEC; j++) {
                            const int c = (me + i * tpr) * VEC + j;
                            cols[c] = k ? cols[c] + dw[i][j] : dw[i][j];
                            cols[H + c] = k ? cols[H + c] + db[i][j] : db[i][j];
                        }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * H; c += blockDim.x) out[c] = cols[c];
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (me + i * tpr < n) {
                const int c = (me + i * tpr) * VEC;
                Vec<float, VEC> o;
                o.set(dw[i]);
                *reinterpret_cast<Vec<float, VEC>*>(out + c) = o;
                o.set(db[i]);
                *reinterpret_cast<Vec<float, VEC>*>(out + H + c) = o;
            }
    }
}

// ---------------------------------------------------------------------------
// Rows through shared memory. A CTA takes R consecutive rows at a time; their operands arrive by
// bulk copies, a ring of stages ahead, so that enough bytes are in flight without holding them in
// registers, and one barrier per R rows joins the warps' sums (it also says that everybody has
// read the stage before: in the forward thread 0 refills it then). Thread pieces as above: piece i at
// i * threads + thread.
// ---------------------------------------------------------------------------
// Rows of a CTA and their parts. Where every row starts on a 16-byte boundary, piece c is its elements c * VEC
// ... and a CTA takes R consecutive rows at a time. Else (ODD; every row tensor is off the boundary alike) a row
// is `head` elements up to its first boundary, n pieces, which the bulk copies bring, and `tail` elements past the
// last one; a lane for each of those, in the CTA's last warp, moves them itself, a group of rows ahead. Rows t and
// t + period start alike: a CTA takes only rows of one head, so that a thread's columns are the same in all.
template <bool ODD>
struct LnRows {
    int n, head;
    int edge;                         // the column of this thread's single element, or -1
    int period, first;                // row(u) = u * period + first
    long long count;                  // rows of this head
    __device__ LnRows(const void* base, int size, int rows, int H, int period_, int tpr) : n(H * size / 16), head(0), edge(-1), period(1), first(0), count(rows) {
        if constexpr (ODD) {
            const int vec = 16 / size;
            period = period_;
            first = (int)(blockIdx.x % period);
            count = ((long long)rows - first + period - 1) / period;
            head = vec - 1 - (int)(((reinterpret_cast<uintptr_t>(base) & 15) / size + (long long)first * H + vec - 1) % vec);
            n = (H - head) / vec;
            const int q = tpr - 1 - (int)threadIdx.x, tail = H - head - n * vec;
            if (q >= 0 && q < head) edge = q;
            else if (q >= 8 && q - 8 < tail) edge = head + n * vec + q - 8;
        }
    }
    __device__ long long row(long long u) const { return ODD ? u * period + first : u; }
    __device__ long long begin() const { return ODD ? blockIdx.x / period : blockIdx.x; }
    __device__ long long step() const { return ODD ? gridDim.x / period : gridDim.x; }
    __device__ bool single() const { return ODD && edge >= 0; }
};

// Columns of weight or bias that belong to piece c.
template <typename W, int VEC, bool ODD>
__device__ __forceinline__ Vec<W, VEC> ln_column(const LnRows<ODD>& l, const W* w, int c) {
    if constexpr (ODD) {
        Vec<W, VEC> v;
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) f[j] = to_f(w[l.head + c * VEC + j]);
        v.set(f);
        return v;
    } else {
        return reinterpret_cast<const Vec<W, VEC>*>(w)[c];
    }
}

struct LnRing {
    uint64_t full[LN_STAGES];
    uint32_t abort_flag;
};

__device__ __forceinline__ void ring_init(LnRing& ring, int stages) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; i++) ptx::mbar_init(&ring.full[i], 1);
        ring.abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    __syncthreads();
}

// After a wait that gave up: the copies in flight get a bounded chance to land (`done` groups were begun).
__device__ __forceinline__ void ring_drain(LnRing& ring, int stages, int done) {
    if (threadIdx.x == 0 && *(volatile uint32_t*)&ring.abort_flag) {
        volatile uint32_t never = 0u;
        for (int i = 0; i < stages && i < done; i++)
            ptx::wait_parity(&ring.full[(done - 1 - i) % stages], (uint32_t)(((done - 1 - i) / stages) & 1), &never, 100000000ull);
    }
}

// Forward. The variance is joined from each warp's sum of squares about its own mean (no cancellation,
// one barrier): sum (s - mean)^2 = sum over warps of (their M2 + n_w (mean_w - mean)^2). 8192 x 4096 bf16
// with a residual, 268 MB: 47-48 us, 5.6-5.7 TB/s; a device-to-device copy of as many bytes takes 48 us.
template <typename T, typename W, int VEC, int NV, int R, bool ODD>
__global__ void __launch_bounds__(512, NV == 2 && R == 1 ? 2 : 1) ln_forward_ring_kernel(const T* x, const T* residual, int rows, int H,
                                                              const W* __restrict__ w, const W* __restrict__ b,
                                                              float eps, T* sum, T* y, float* mean_out, float* rstd_out,
                                                              int stages, int period, uint32_t rb) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LnRing ring;
    __shared__ float2 red[2][16 * R];         // (mean, M2) of every warp and row
    __shared__ float count[16];               // elements of a row that a warp has
    using V = Vec<T, VEC>;
    const LnRows<ODD> l(x, sizeof(T), rows, H, period, blockDim.x);
    const int tpr = blockDim.x, me = threadIdx.x, n = l.n, lane = (int)lane_id();
    const int entry = lane & (16 * R - 1);    // this lane's of red: warp entry / R, row entry % R
    const int nt = residual ? 2 : 1;
    const uint32_t stage_bytes = nt * R * rb;
    const long long groups = (l.count + R - 1) / R, step = l.step();
    auto issue = [&](long long g, int st) {
        uint8_t* d = smem + (size_t)st * stage_bytes;
        const long long u = g * R;
        const int nr = (int)(l.count - u < R ? l.count - u : R);
        if constexpr (ODD) {
            const uint32_t nb = (uint32_t)l.n * 16u;
            ptx::mbar_arrive_expect_tx(&ring.full[st], nt * nr * nb);
#pragma unroll
            for (int k = 0; k < R; k++) {
                if (k >= nr) continue;
                const long long at = l.row(u + k) * H + l.head;
                ptx::bulk_load(d + k * rb, x + at, nb, &ring.full[st]);
                if (residual) ptx::bulk_load(d + (R + k) * rb, residual + at, nb, &ring.full[st]);
            }
        } else {
            const uint32_t nb = (uint32_t)nr * rb;
            ptx::mbar_arrive_expect_tx(&ring.full[st], nt * nb);
            ptx::bulk_load(d, x + u * H, nb, &ring.full[st]);
            if (residual) ptx::bulk_load(d + R * rb, residual + u * H, nb, &ring.full[st]);
        }
    };
    ring_init(ring, stages);
    if (me == 0)
        for (int i = 0; i < stages; i++)
            if (l.begin() + i * step < groups) issue(l.begin() + i * step, i);
    Vec<W, VEC> wv[NV], bv[NV];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = me + i * tpr;
        if (c < n) {
            mine += VEC;
            wv[i] = ln_column<W, VEC>(l, w, c);
            if (b) bv[i] = ln_column<W, VEC>(l, b, c);
        }
    }
    // single elements: (x, residual) of the group to come
    float ew = 0.0f, eb = 0.0f, ex[R], er[R];
    auto fetch = [&](long long g) {
#pragma unroll
        for (int k = 0; k < R; k++)
            if (l.single() && g * R + k < l.count) {
                const long long at = l.row(g * R + k) * H + l.edge;
                ex[k] = to_f(x[at]);
                if (residual) er[k] = to_f(residual[at]);
            }
    };
    if (l.single()) {
        mine++;
        ew = to_f(w[l.edge]);
        if (b) eb = to_f(b[l.edge]);
        fetch(l.begin());
    }
    const int nw = __reduce_add_sync(FULL, mine);
    if (me < 16) count[me] = 0.0f;
    for (int i = me; i < 2 * 16 * R; i += tpr) (&red[0][0])[i] = make_float2(0.0f, 0.0f);
    __syncthreads();
    if (lane == 0) count[me >> 5] = (float)nw;
    const float per_nw = nw ? 1.0f / (float)nw : 0.0f, per_h = 1.0f / (float)H;
    int st = 0, done = 0;
    uint32_t phase = 0;
    for (long long g = l.begin(); g < groups; g += step, done++) {
        ptx::wait_parity(&ring.full[st], phase, &ring.abort_flag);
        const uint8_t* base = smem + (size_t)st * stage_bytes;
        const int nr = (int)(l.count - g * R < R ? l.count - g * R : R);
        float2* rd = red[done & 1];
        V xv[R][NV];
        float sw[R], qw[R], es[R];
#pragma unroll
        for (int k = 0; k < R; k++) {
            sw[k] = 0.0f;
            if (k >= nr) continue;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = me + i * tpr;
                if (c >= n) continue;
                xv[k][i] = reinterpret_cast<const V*>(base + (size_t)k * rb)[c];
                if (residual) {
                    const V rv = reinterpret_cast<const V*>(base + (size_t)(R + k) * rb)[c];
                    float f[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; j++) f[j] = xv[k][i].get(j) + rv.get(j);
                    xv[k][i].set(f);
                    reinterpret_cast<V*>(sum + l.row(g * R + k) * H + l.head)[c] = xv[k][i];
                }
#pragma unroll
                for (int j = 0; j < VEC; j++) sw[k] += xv[k][i].get(j);
            }
            if (l.single()) {
                es[k] = ex[k];
                if (residual) {
                    const T v = from_f<T>(ex[k] + er[k]);
                    sum[l.row(g * R + k) * H + l.edge] = v;
                    es[k] = to_f(v);
                }
                sw[k] += es[k];
            }
        }
        if (l.single()) fetch(g + step);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < R; k++) sw[k] += __shfl_xor_sync(FULL, sw[k], o);
#pragma unroll
        for (int k = 0; k < R; k++) {
            qw[k] = 0.0f;
            sw[k] *= per_nw;                            // the warp's mean
            if (k >= nr) continue;
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (me + i * tpr < n)
#pragma unroll
                    for (int j = 0; j < VEC; j++) {
                        const float d = xv[k][i].get(j) - sw[k];
                        qw[k] = fmaf(d, d, qw[k]);
                    }
            if (l.single()) qw[k] = fmaf(es[k] - sw[k], es[k] - sw[k], qw[k]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < R; k++) qw[k] += __shfl_xor_sync(FULL, qw[k], o);
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < R; k++) {
                rd[(me >> 5) * R + k] = make_float2(sw[k], qw[k]);
            }
        __syncthreads();
        if (me == 0 && done > 0 && g + (stages - 1) * step < groups)
            issue(g + (stages - 1) * step, st == 0 ? stages - 1 : st - 1);      // the stage before this one
        // every warp joins the warps' sums, an entry a lane
        const float2 e = rd[entry];
        const float ce = count[entry / R];
        float sum_e = ce * e.x;
#pragma unroll
        for (int o = R; o < 16 * R; o <<= 1) sum_e += __shfl_xor_sync(FULL, sum_e, o);
        const float mean_e = sum_e * per_h, d_e = e.x - mean_e;
        float m2_e = fmaf(ce * d_e, d_e, e.y);
#pragma unroll
        for (int o = R; o < 16 * R; o <<= 1) m2_e += __shfl_xor_sync(FULL, m2_e, o);
        const float rstd_e = rsqrtf(fmaf(m2_e, per_h, eps));
#pragma unroll
        for (int k = 0; k < R; k++) {
            const float mean = __shfl_sync(FULL, mean_e, k), rstd = __shfl_sync(FULL, rstd_e, k);
            if (k >= nr) continue;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = me + i * tpr;
                if (c >= n) continue;
                V o;
                float f[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    f[j] = fmaf((xv[k][i].get(j) - mean) * rstd, wv[i].get(j), b ? bv[i].get(j) : 0.0f);
                o.set(f);
                reinterpret_cast<V*>(y + l.row(g * R + k) * H + l.head)[c] = o;
            }
            if (l.single()) y[l.row(g * R + k) * H + l.edge] = from_f<T>(fmaf((es[k] - mean) * rstd, ew, eb));
            if (me == 0) {
                if (mean_out) mean_out[l.row(g * R + k)] = mean;
                if (rstd_out) rstd_out[l.row(g * R + k)] = rstd;
            }
        }
        if (++st == stages) { st = 0; phase ^= 1u; }
    }
    ring_drain(ring, stages, done);
}

// Sums of 2 R values over the first `threads` (512 at most) threads of the CTA, one barrier, the same in each. The first
// step hands half of the values to either half of a warp; then every warp joins the warps' sums, two
// values a lane. red: 16 R pairs, zero where there is no warp.
template <int R>
__device__ __forceinline__ void cta_sums(float (&v)[2 * R], float2* red, int threads) {
    const int lane = (int)lane_id();
#pragma unroll
    for (int k = 0; k < R; k++) {
        const float mine = lane < 16 ? v[2 * k] : v[2 * k + 1], other = lane < 16 ? v[2 * k + 1] : v[2 * k];
        v[2 * k] = mine + __shfl_xor_sync(FULL, other, 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < R; k++) v[2 * k] += __shfl_xor_sync(FULL, v[2 * k], o);
    if ((lane & 15) == 0)
#pragma unroll
        for (int k = 0; k < R; k++) reinterpret_cast<float*>(red)[((threadIdx.x >> 5) * R + k) * 2 + (lane >> 4)] = v[2 * k];
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    float2 e = red[lane & (16 * R - 1)];
#pragma unroll
    for (int o = R; o < 16 * R; o <<= 1) {
        e.x += __shfl_xor_sync(FULL, e.x, o);
        e.y += __shfl_xor_sync(FULL, e.y, o);
    }
#pragma unroll
    for (int k = 0; k < R; k++) {
        v[2 * k] = __shfl_sync(FULL, e.x, k);
        v[2 * k + 1] = __shfl_sync(FULL, e.y, k);
    }
}

// Backward. A warp of its own fills the ring, a stage per row, as soon as the computing warps have let go of
// the row that was there; those take R rows at a time. dweight and dbias add up in the threads' registers
// over the CTA's rows and leave as one partial sum per CTA: part [gridDim.x][2][H]. 8192 x 7168 bf16 with
// dx_add, 470 MB: 86-89 us with the columns' kernel, 5.4 TB/s; a copy of as many bytes takes 77 us. (Refilled by
// thread 0 between the barriers, as in the forward, it took 98 us.) xh is (s - mean) rstd in both passes: one fma
// s rstd - mean rstd would save 1 us of that and lose |mean| rstd units of xh's last place.
template <typename T, typename W, int VEC, int NV, int R, bool ODD>
__global__ void __launch_bounds__(544) ln_backward_ring_kernel(const T* dy, const T* s, int rows, int H,
                                                               const W* __restrict__ w, const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, const T* add, T* dx,
                                                               float* part, int stages, int period, uint32_t rb) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[LN_STAGES], empty[LN_STAGES];
    __shared__ uint32_t abort_flag;
    __shared__ float2 red[2][16 * R];
    __shared__ float4 own[ODD ? R : 1][ODD ? 16 : 1];     // single elements of the group at hand, each its own thread's
    using V = Vec<T, VEC>;
    const LnRows<ODD> l(s, sizeof(T), rows, H, period, blockDim.x - 32);
    const int tpr = blockDim.x - 32, me = threadIdx.x, n = l.n;
    const int nt = add ? 3 : 2;
    const uint32_t stage_bytes = nt * rb;
    const long long groups = (l.count + R - 1) / R, step = l.step();
    for (int i = me; i < 2 * 16 * R; i += blockDim.x) (&red[0][0])[i] = make_float2(0.0f, 0.0f);
    if (me == 0) {
        for (int i = 0; i < stages; i++) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], tpr >> 5);
        }
        abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    int st = 0;
    uint32_t phase = 0;
    if (me >= tpr) {
        if (me == tpr) {
            int issued = 0;
            bool ok = true;
            for (long long g = l.begin(); g < groups && ok; g += step)
                for (long long u = g * R; u < l.count && u < (g + 1) * R; u++) {
                    ok = ptx::wait_parity(&empty[st], phase ^ 1u, &abort_flag);
                    if (!ok) break;
                    uint8_t* d = smem + (size_t)st * stage_bytes;
                    const long long at = l.row(u) * H + l.head;
                    const uint32_t nb = ODD ? (uint32_t)l.n * 16u : rb;
                    ptx::mbar_arrive_expect_tx(&full[st], nt * nb);
                    ptx::bulk_load(d, dy + at, nb, &full[st]);
                    ptx::bulk_load(d + rb, s + at, nb, &full[st]);
                    if (add) ptx::bulk_load(d + 2 * rb, add + at, nb, &full[st]);
                    issued++;
                    if (++st == stages) { st = 0; phase ^= 1u; }
                }
            if (!ok) {       // the copies in flight get a bounded chance to land
                for (int i = 0; i < stages && i < issued; i++) {
                    if (--st < 0) { st = stages - 1; phase ^= 1u; }
                    volatile uint32_t never = 0u;
                    ptx::wait_parity(&full[st], phase, &never, 100000000ull);
                }
            }
        }
        return;
    }
    Vec<W, VEC> wv[NV];
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (me + i * tpr < n) wv[i] = ln_column<W, VEC>(l, w, me + i * tpr);
#pragma unroll
        for (int j = 0; j < VEC; j++) dw[i][j] = db[i][j] = 0.0f;
    }
    // the rows' statistics, one group ahead
    const float per_h = 1.0f / (float)H;
    float m[R], r[R], mn[R], rn[R];
    auto stats = [&](long long g, float* a, float* c) {
#pragma unroll
        for (int k = 0; k < R; k++) {
            const long long t = l.row(g * R + k < l.count ? g * R + k : l.count - 1);
            a[k] = __ldg(mean + t);
            c[k] = __ldg(rstd + t);
        }
    };
    // single elements: (dy, s, add) of the group to come
    float ew = 0.0f, edw = 0.0f, edb = 0.0f, eg[R], es[R], ea[R];
    auto fetch = [&](long long g) {
#pragma unroll
        for (int k = 0; k < R; k++)
            if (l.single() && g * R + k < l.count) {
                const long long at = l.row(g * R + k) * H + l.edge;
                eg[k] = to_f(dy[at]);
                es[k] = to_f(s[at]);
                if (add) ea[k] = to_f(add[at]);
            }
    };
    if (l.single()) {
        ew = to_f(w[l.edge]);
        fetch(l.begin());
    }
    if (l.begin() < groups) stats(l.begin(), m, r);
    int buf = 0;
    for (long long g = l.begin(); g < groups; g += step, buf ^= 1) {
        if (g + step < groups) stats(g + step, mn, rn);
        const int nr = (int)(l.count - g * R < R ? l.count - g * R : R);
        float sums[2 * R];
        int at[R];
#pragma unroll
        for (int k = 0; k < R; k++) {
            sums[2 * k] = sums[2 * k + 1] = 0.0f;
            at[k] = st;
            if (k >= nr) continue;
            ptx::wait_parity(&full[st], phase, &abort_flag);
            if (++st == stages) { st = 0; phase ^= 1u; }
            const V* gr = reinterpret_cast<const V*>(smem + (size_t)at[k] * stage_bytes);
            const V* sr = reinterpret_cast<const V*>(smem + (size_t)at[k] * stage_bytes + rb);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = me + i * tpr;
                if (c >= n) continue;
                const V gv = gr[c], sv = sr[c];
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const float d = gv.get(j), xh = (sv.get(j) - m[k]) * r[k], q = d * wv[i].get(j);
                    sums[2 * k] += q;
                    sums[2 * k + 1] = fmaf(q, xh, sums[2 * k + 1]);
                    dw[i][j] = fmaf(d, xh, dw[i][j]);
                    db[i][j] += d;
                }
            }
        }
        if (l.single()) {
#pragma unroll
            for (int k = 0; k < R; k++) {
                if (k >= nr) continue;
                const float xh = (es[k] - m[k]) * r[k], q = eg[k] * ew;
                sums[2 * k] += q;
                sums[2 * k + 1] = fmaf(q, xh, sums[2 * k + 1]);
                edw = fmaf(eg[k], xh, edw);
                edb += eg[k];
                own[k][tpr - 1 - me] = make_float4(eg[k], es[k], add ? ea[k] : 0.0f, 0.0f);
            }
            fetch(g + step);
        }
        cta_sums<R>(sums, red[buf], tpr);
#pragma unroll
        for (int k = 0; k < R; k++) {
            if (k >= nr) continue;
            const V* gr = reinterpret_cast<const V*>(smem + (size_t)at[k] * stage_bytes);
            const V* sr = reinterpret_cast<const V*>(smem + (size_t)at[k] * stage_bytes + rb);
            const V* ar = reinterpret_cast<const V*>(smem + (size_t)at[k] * stage_bytes + 2 * rb);
            const float a = sums[2 * k] * per_h, c2 = sums[2 * k + 1] * per_h;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = me + i * tpr;
                if (c >= n) continue;
                const V gv = gr[c], sv = sr[c];
                V av, o;
                if (add) av = ar[c];
                float f[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const float xh = (sv.get(j) - m[k]) * r[k];
                    f[j] = r[k] * fmaf(-xh, c2, fmaf(gv.get(j), wv[i].get(j), -a));
                    if (add) f[j] += av.get(j);
                }
                o.set(f);
                reinterpret_cast<V*>(dx + l.row(g * R + k) * H + l.head)[c] = o;
            }
            if (l.single()) {
                const float4 e = own[k][tpr - 1 - me];
                const float xh = (e.y - m[k]) * r[k];
                dx[l.row(g * R + k) * H + l.edge] = from_f<T>(r[k] * fmaf(-xh, c2, fmaf(e.x, ew, -a)) + e.z);
            }
            __syncwarp();
            if (lane_id() == 0) ptx::mbar_arrive(&empty[at[k]]);
            m[k] = mn[k];
            r[k] = rn[k];
        }
    }
    pdl_trigger();
    if (!part) return;
    float* out = part + (size_t)blockIdx.x * 2 * H;
    if constexpr (ODD) {
        // by way of the ring, for whole lines (the computing warps have read all of it)
        float* o = reinterpret_cast<float*>(smem);
        const int np = n * VEC;
        asm volatile("bar.sync 1, %0;" ::"r"(tpr) : "memory");
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (me + i * tpr < n) {
                const int c = (me + i * tpr) * VEC;
#pragma unroll
                for (int j = 0; j < VEC; j += 4) {
                    *reinterpret_cast<float4*>(o + c + j) = make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
                    *reinterpret_cast<float4*>(o + np + c + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
                }
            }
        if (l.single()) {
            out[l.edge] = edw;
            out[H + l.edge] = edb;
        }
        asm volatile("bar.sync 1, %0;" ::"r"(tpr) : "memory");
#pragma unroll 4
        for (int i = me; i < np; i += tpr) {
            out[l.head + i] = o[i];
            out[H + l.head + i] = o[np + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (me + i * tpr < n) {
                const int c = (me + i * tpr) * VEC;
                Vec<float, VEC> o;
                o.set(dw[i]);
                *reinterpret_cast<Vec<float, VEC>*>(out + c) = o;
                o.set(db[i]);
                *reinterpret_cast<Vec<float, VEC>*>(out + H + c) = o;
            }
    }
}

// Backward for rows too long for the ring (bf16 above 8192 columns): dx with the row read twice (from L2 the second
// time) ... Together with the kernel below 3000 x 16384 bf16 with dx_add takes 128 us (floor 58; two more reads of
// the operands than that; element by element 264).
template <typename T, typename W, int VEC>
__global__ void __launch_bounds__(512) ln_backward_long_kernel(const T* dy, const T* __restrict__ s, int H,
                                                               const W* __restrict__ w, const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, const T* add, T* dx) {
    __shared__ float red[64];
    using V = Vec<T, VEC>;
    const long long base = (long long)blockIdx.x * H;
    const int n = H / VEC;
    const float m = mean[blockIdx.x], r = rstd[blockIdx.x];
    float sums[2] = {0.0f, 0.0f};
#pragma unroll(VEC == 1 ? 1 : 2)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const V gv = reinterpret_cast<const V*>(dy + base)[i], sv = reinterpret_cast<const V*>(s + base)[i];
        const Vec<W, VEC> wv = reinterpret_cast<const Vec<W, VEC>*>(w)[i];
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            const float g = gv.get(j) * wv.get(j);
            sums[0] += g;
            sums[1] = fmaf(g, (sv.get(j) - m) * r, sums[1]);
        }
    }
    row_sum(sums, false, red);
    const float a = sums[0] / (float)H, c = sums[1] / (float)H;
#pragma unroll(VEC == 1 ? 1 : 2)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const V gv = reinterpret_cast<const V*>(dy + base)[i], sv = reinterpret_cast<const V*>(s + base)[i];
        const Vec<W, VEC> wv = reinterpret_cast<const Vec<W, VEC>*>(w)[i];
        V av, o;
        if (add) av = reinterpret_cast<const V*>(add + base)[i];
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            f[j] = r * (gv.get(j) * wv.get(j) - a - (sv.get(j) - m) * r * c);
            if (add) f[j] += av.get(j);
        }
        o.set(f);
        reinterpret_cast<V*>(dx + base)[i] = o;
    }
}

// ... and the partial sums of dweight and dbias, a slice of the rows per blockIdx.y, VEC columns a thread, four rows
// of loads in flight.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) ln_backward_long_w_kernel(const T* dy, const T* __restrict__ s, int rows, int H,
                                                                 const float* __restrict__ mean,
                                                                 const float* __restrict__ rstd, float* part) {
    using V = Vec<T, VEC>;
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= H / VEC) return;
    float a[VEC], c[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) a[j] = c[j] = 0.0f;
#pragma unroll 4
    for (long long t = blockIdx.y; t < rows; t += gridDim.y) {
        const V gv = reinterpret_cast<const V*>(dy + t * H)[i], sv = reinterpret_cast<const V*>(s + t * H)[i];
        const float m = mean[t], r = rstd[t];
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            a[j] = fmaf(gv.get(j), (sv.get(j) - m) * r, a[j]);
            c[j] += gv.get(j);
        }
    }
    float* out = part + (size_t)blockIdx.y * 2 * H + (size_t)i * VEC;
#pragma unroll
    for (int j = 0; j < VEC; j++) {
        out[j] = a[j];
        out[H + j] = c[j];
    }
}

// dweight and dbias from n partial sums, 32 columns per CTA: thread row y adds partials y, y + 32, ...
// Latency, mostly: 8.7 MB in 6.8-7.1 us from a cold L2 (152 partial sums of 7168 columns).
template <typename W>
__global__ void __launch_bounds__(1024) ln_columns_kernel(const float* __restrict__ part, int n, int H, W* dw, W* db) {
    __shared__ float red[2][32][33];
    pdl_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float a = 0.0f, b = 0.0f;
    if (c < H) {
        constexpr int B = 8;                           // of either in flight, the last ones too
        const float* p = part + (size_t)y * 2 * H + c;
        const size_t step = (size_t)64 * H;
        for (int left = n - y; left > 0; left -= 32 * B) {
            float u[B], v[B];
#pragma unroll
            for (int k = 0; k < B; k++, p += step) {
                u[k] = left > 32 * k ? p[0] : 0.0f;
                v[k] = left > 32 * k ? p[H] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < B; k++) {
                a += u[k];
                b += v[k];
            }
        }
    }
    red[0][y][x] = a;
    red[1][y][x] = b;
    __syncthreads();
    if (y < 2 && c < H) {
        float v = 0.0f;
        for (int i = 0; i < 32; i++) v += red[y][i][x];
        W* out = y ? db : dw;
        if (out) out[c] = from_f<W>(v);
    }
}

bool ln_type(int d) { return d == MOE_BF16 || d == MOE_F32; }
size_t ln_size(int d) { return d == MOE_BF16 ? 2 : 4; }

int ln_sms() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

constexpr int LN_PARTS = 1024;            // most partial sums of dweight and dbias

// The row tensors (null: not there) and the columns' (weight, bias) against 16 bytes. alike: the rows' are
// off the boundary alike; wide: every row and column starts on it.
struct LnAlign {
    bool alike = true, wide = true;
    LnAlign(std::initializer_list<const void*> row_tensors, std::initializer_list<const void*> columns, int H, int vec) {
        const uintptr_t first = reinterpret_cast<uintptr_t>(*row_tensors.begin()) & 15;
        for (const void* q : row_tensors) alike = alike && (!q || (reinterpret_cast<uintptr_t>(q) & 15) == first);
        wide = alike && first == 0 && H % vec == 0;
        for (const void* q : columns) wide = wide && moe_host::aligned(q, 16);
    }
};

// How a row is spread over threads: pieces of vec elements, nv a thread, a warp or a CTA per row. nv = 0: it
// does not fit. ring: it goes through shared memory; odd: with rows off the 16-byte boundary.
// Both sides of the rules, in us (bf16 unless said; forward with a residual, backward with dx_add):
//   on the boundary, a warp per row up to 32 pieces: forward 8192 x 256 5.0 (ring 7.3), but 8192 x 512 9.8
//     (7.1); backward 8192 x 256 11.5 (13.4) but 1000 x 256 9.1 (7.5) and 64 x 256 7.8 (5.0)
//   off it, forward, element by element: 777 x 511 3.9 (ring 6.1), 8192 x 255 10.7 (11.8), but 777 x 777 6.5
//     (5.7), 8192 x 1021 42 (18), 777 x 5001 25 (11.7)
//   off it, backward, element by element: 2000 x 1021 13.4 (15.3), 8192 x 511 22.5 (24.8), 777 x 1021 fp32 8.4
//     (9.1), but 8192 x 1021 46 (29), 2000 x 777 fp32 12.1 (11.1), 777 x 5001 36 (19.4)
struct LnShape {
    int nv, threads;
    bool warp_row, ring, odd;
    int period;               // rows t and t + period start alike on the 16-byte boundary
    uint32_t row_bytes;       // of a row in the ring
};

LnShape ln_shape(int H, int size, const LnAlign& a, bool forward, int rows) {
    const int vec = 16 / size;
    auto cta = [&](int n, int nv) { return LnShape{nv, (((n + nv - 1) / nv) + 31) / 32 * 32, false, false, false, 1, 0u}; };
    auto ring = [&](int n, bool odd) {
        LnShape l = cta(n, n <= 1024 ? 2 : 4);
        l.ring = true;
        l.odd = odd;
        while (odd && (long long)l.period * H % vec) l.period *= 2;
        l.row_bytes = odd ? (uint32_t)n * 16u : (uint32_t)(H * size);
        return l;
    };
    const int most = forward || vec == 4 ? 2048 : 1024;      // pieces
    if (a.wide) {
        const int n = H / vec;
        if (n <= 32 && (forward || rows > 2000)) return {1, 256, true, false, false, 1, 0u};
        return n <= most ? ring(n, false) : LnShape{0, 512, false, false, false, 1, 0u};
    }
    // Element by element while that fits a few registers a thread and the rows are short or few, else whole
    // pieces by the ring where they are off the boundary alike.
    if (H <= 128) return {4, 256, true, false, false, 1, 0u};
    const long long all = (long long)rows * H;
    const bool little = forward ? H * size <= 512 || all <= 1 << 19 : H * size <= 1024 || all * size <= 1 << 22;
    if (a.alike && H / vec <= most && !(little && H <= 2048)) return ring(H / vec, true);
    if (H <= 2048) return cta(H, 4);
    if (H <= 8192) return cta(H, 16);
    return {0, 512, false, false, false, 1, 0u};
}

// Rows per group, ring stages and CTAs per SM of the ring kernels, row_bytes of operands per row.
struct LnRingShape {
    int rows, stages, ctas;
    size_t smem;
};

// Forward: a stage is a group of two rows where two CTAs of three such stages fit an SM, else one row. Not
// 32 CTAs of one warp, whose starts cost more than they hide: 8192 x 264 bf16 8.2 us, with 16 of them 6.9.
LnRingShape ln_forward_ring(size_t row_bytes, const LnShape& l) {
    LnRingShape r;
    r.rows = l.nv == 4 || 2 * 3 * 2 * row_bytes > LN_SMEM ? 1 : 2;
    r.stages = 3 * r.rows * row_bytes <= LN_SMEM ? 3 : 2;
    r.smem = r.stages * r.rows * row_bytes;
    const int fit = (int)(LN_SMEM / (r.smem + 2048)), most = l.threads < 64 ? 16 : 1024 / l.threads;
    r.ctas = fit < most ? (fit < 1 ? 1 : fit) : most;
    return r;
}

// Backward: a stage is a row; two rows a group where three fit (long fp32 rows go singly, and rows off the
// boundary of more than 4 KB: 3000 x 8191 61 us by twos, singly 56.6, but 777 x 1021 fp32 8.7 and 9.8. Off the
// boundary the bf16 instance spills 44 to 52 bytes with two rows, 20 with one).
LnRingShape ln_backward_ring(size_t row_bytes, const LnShape& l) {
    LnRingShape r;
    const int most = l.threads > 256 ? 1 : 512 / l.threads;     // (128 registers a thread)
    r.ctas = most;
    while (r.ctas > 1 && r.ctas * (4 * row_bytes + 2048) > LN_SMEM) r.ctas--;
    r.stages = (int)((LN_SMEM / r.ctas - 2048) / row_bytes);
    if (r.stages > LN_STAGES) r.stages = LN_STAGES;
    r.rows = l.nv == 4 || r.stages < 3 || (l.odd && l.row_bytes > 4096) ? 1 : 2;
    r.smem = r.stages * row_bytes;
    return r;
}

// CTAs of a ring kernel: the same number for each of the period's rows.
int ln_ring_grid(int rows, int group, int period, long long most) {
    const long long of_one = (((long long)rows + period - 1) / period + group - 1) / group;
    most /= period;
    return (int)(of_one < most ? of_one : most) * period;
}

template <typename T, typename W>
moe_status ln_forward(const void* x, const void* residual, int rows, int H, const void* w, const void* b, float eps,
                      void* sum, void* y, float* mean, float* rstd, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(T);
    const LnAlign align({x, residual, sum, y}, {w, b}, H, VEC);
    const bool wide = align.wide;
    const LnShape l = ln_shape(H, sizeof(T), align, true, rows);
    if (l.ring) {
        const LnRingShape r = ln_forward_ring((size_t)(residual ? 2 : 1) * l.row_bytes, l);
        const int grid = ln_ring_grid(rows, r.rows, l.period, (long long)ln_sms() * r.ctas);
#define MOE_LN_FR(nv, R, odd)                                                                                         \
    {                                                                                                                 \
        static moe_host::PerDevice allowed;                                                                           \
        auto kern = ln_forward_ring_kernel<T, W, VEC, nv, R, odd>;                                                    \
        if (!moe_host::allow_smem(kern, LN_SMEM, allowed)) return MOE_ERR_CUDA;                                       \
        kern<<<grid, l.threads, r.smem, s>>>((const T*)x, (const T*)residual, rows, H, (const W*)w, (const W*)b, eps, \
                                             (T*)sum, (T*)y, mean, rstd, r.stages, l.period, l.row_bytes);            \
    }
        if (l.nv == 2 && r.rows == 2) {
            if (l.odd) MOE_LN_FR(2, 2, true)
            else MOE_LN_FR(2, 2, false)
        } else if (l.nv == 2) {
            if (l.odd) MOE_LN_FR(2, 1, true)
            else MOE_LN_FR(2, 1, false)
        } else {
            if (l.odd) MOE_LN_FR(4, 1, true)
            else MOE_LN_FR(4, 1, false)
        }
#undef MOE_LN_FR
        return moe_host::launch_status();
    }
    const long long ctas = l.warp_row ? ((long long)rows + 7) / 8 : rows;
    // as many CTAs as are resident at 2048 threads an SM: a CTA's rows share its weights
    const long long most = (long long)ln_sms() * (2048 / l.threads);
    const int grid = (int)(ctas < most ? ctas : most);
#define MOE_LN_F(vec, nv)                                                                                             \
    ln_forward_kernel<T, W, vec, nv><<<grid, l.threads, 0, s>>>((const T*)x, (const T*)residual, rows, H, l.warp_row, \
                                                                (const W*)w, (const W*)b, eps, (T*)sum, (T*)y, mean, rstd)
#define MOE_LN_FL(vec)                                                                                              \
    ln_forward_long_kernel<T, W, vec><<<rows, 512, 0, s>>>((const T*)x, (const T*)residual, H, (const W*)w, (const W*)b, \
                                                           eps, (T*)sum, (T*)y, mean, rstd)
    if (l.nv == 0 && wide) MOE_LN_FL(VEC);
    else if (l.nv == 0) MOE_LN_FL(1);
    else if (wide) MOE_LN_F(VEC, 1);
    else if (l.nv == 4) MOE_LN_F(1, 4);
    else MOE_LN_F(1, 16);
#undef MOE_LN_F
#undef MOE_LN_FL
    return moe_host::launch_status();
}

template <typename T, typename W>
moe_status ln_backward(const void* dy, const void* sv, int rows, int H, const void* w, const float* mean,
                       const float* rstd, const void* add, void* dx, void* dw, void* db, float* part, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(T);
    const LnAlign align({dy, sv, add, dx}, {w}, H, VEC);
    const bool wide = align.wide;
    const LnShape l = ln_shape(H, sizeof(T), align, false, rows);
    const bool sums = dw || db;
    int n_part = 0;
    if (rows == 0) {
    } else if (l.nv == 0) {
#define MOE_LN_BL(vec)                                                                                              \
    {                                                                                                               \
        if (sums) { /* (before dx, which may be dy) */                                                              \
            /* eight rows a CTA at least; four CTAs an SM, more of the narrow ones */                               \
            const int cols = (H / vec + 255) / 256, most = (vec == 1 ? 24 : 4) * ln_sms() / cols + 1;               \
            n_part = (rows + 7) / 8 < most ? (rows + 7) / 8 : most;                                                 \
            if (n_part > LN_PARTS) n_part = LN_PARTS;                                                               \
            ln_backward_long_w_kernel<T, vec><<<dim3(cols, n_part), 256, 0, s>>>((const T*)dy, (const T*)sv, rows, H, \
                                                                                 mean, rstd, part);                 \
        }                                                                                                           \
        ln_backward_long_kernel<T, W, vec><<<rows, 512, 0, s>>>((const T*)dy, (const T*)sv, H, (const W*)w, mean, rstd, \
                                                                (const T*)add, (T*)dx);                             \
    }
        if (wide) MOE_LN_BL(VEC)
        else MOE_LN_BL(1)
#undef MOE_LN_BL
    } else if (l.ring) {
        LnRingShape r = ln_backward_ring((size_t)(add ? 3 : 2) * l.row_bytes, l);
        if (l.odd && r.smem < (size_t)H * 8) r.smem = (size_t)H * 8;       // (its partial sums leave by it)
        const int sms = ln_sms();
        if (sms * r.ctas > LN_PARTS) r.ctas = LN_PARTS / sms;
        n_part = ln_ring_grid(rows, r.rows, l.period, (long long)sms * r.ctas);
#define MOE_LN_BR(nv, R, odd)                                                                                       \
    {                                                                                                               \
        static moe_host::PerDevice allowed;                                                                         \
        auto kern = ln_backward_ring_kernel<T, W, VEC, nv, R, odd>;                                                 \
        if (!moe_host::allow_smem(kern, LN_SMEM, allowed)) return MOE_ERR_CUDA;                                     \
        kern<<<n_part, l.threads + 32, r.smem, s>>>((const T*)dy, (const T*)sv, rows, H, (const W*)w, mean, rstd,        \
                                               (const T*)add, (T*)dx, sums ? part : nullptr, r.stages, l.period,    \
                                               l.row_bytes);                                                        \
    }
        if (l.nv == 4) {
            if constexpr (VEC == 4) {
                if (l.odd) MOE_LN_BR(4, 1, true)
                else MOE_LN_BR(4, 1, false)
            }
        } else if (r.rows == 2) {
            if (l.odd) MOE_LN_BR(2, 2, true)
            else MOE_LN_BR(2, 2, false)
        } else {
            if (l.odd) MOE_LN_BR(2, 1, true)
            else MOE_LN_BR(2, 1, false)
        }
#undef MOE_LN_BR
    } else {
        const long long ctas = l.warp_row ? ((long long)rows + 7) / 8 : rows;
        long long most = (long long)ln_sms() * (512 / l.threads > 1 ? 512 / l.threads : 1);
        if (most > LN_PARTS) most = LN_PARTS;
        n_part = (int)(ctas < most ? ctas : most);
        const size_t smem = l.warp_row ? (size_t)H * 8 : 0;
#define MOE_LN_B(vec, nv, pre)                                                                                        \
    ln_backward_kernel<T, W, vec, nv, pre><<<n_part, l.threads, smem, s>>>((const T*)dy, (const T*)sv, rows, H,       \
                                                                           l.warp_row, (const W*)w, mean, rstd,       \
                                                                           (const T*)add, (T*)dx, sums ? part : nullptr)
        if (wide) MOE_LN_B(VEC, 1, true);
        else if (l.nv == 4) MOE_LN_B(1, 4, true);
        else MOE_LN_B(1, 16, false);
#undef MOE_LN_B
    }
    if (sums && moe_host::launch_pdl(ln_columns_kernel<W>, dim3((H + 31) / 32), dim3(1024), 0, s, (const float*)part, n_part,
                                     H, (W*)dw, (W*)db) != cudaSuccess)
        return MOE_ERR_CUDA;
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
    return (size_t)moe::LN_PARTS * 2 * H * sizeof(float);
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
#define MOE_LNB(T_, W_) return ln_backward<T_, W_>(dy, s, T, H, weight, mean, rstd, dx_add, dx, dweight, dbias, (float*)workspace, st)
    if (dtype == MOE_BF16) {
        if (w_dtype == MOE_BF16) MOE_LNB(__nv_bfloat16, __nv_bfloat16);
        MOE_LNB(__nv_bfloat16, float);
    }
    if (w_dtype == MOE_BF16) MOE_LNB(float, __nv_bfloat16);
    MOE_LNB(float, float);
#undef MOE_LNB
}
