/*
 * moe_gb300.h -- C ABI of the single-GPU dropless Mixture-of-Experts layer
 * hot path for NVIDIA GB300 (sm_103a).
 *
 * The path: router top-K -> permute (dispatch into expert-contiguous order,
 * optionally quantising to MXFP8 on the way) -> grouped SwiGLU expert MLP
 * (two ragged grouped GEMMs, BF16 or MXFP8) -> probability-weighted
 * unpermute/combine back to token order; plus the grouped backward GEMMs.
 *
 * Sources (cited by page title and section):
 *   [SPARSER] "Sparser MoE end-to-end" (harryzhou2000 blog)
 *   [TEJAX]   "Dropless MoE acceleration in JAX with NVIDIA Transformer Engine"
 *             (news.bpdata.com)
 *   [CLARITY] "NVIDIA's unoptimized DeepSeek-V3 baseline spends 84% of kernel
 *             time moving tokens between GPUs" (theclarity.today)
 *
 * Conventions shared by every entry point:
 *  - Ownership: the caller allocates every buffer (device memory unless stated)
 *    and keeps it alive until the enqueued work has finished. The library never
 *    allocates, never synchronises and never copies device->host in the calls
 *    below, except moe_get_device_errors. Group sizes stay on the device
 *    ([TEJAX] "Optimization 1: Grouped GEMM": shapes must not need the CPU, so
 *    CUDA graphs stay usable); every call is safe to capture in a CUDA graph.
 *  - Streams: work is enqueued on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) and nowhere else.
 *  - Layouts are row-major. bf16 tensors are passed as raw 16-bit payloads.
 *    Device pointers must be 16-byte aligned; operands of the grouped GEMMs
 *    (x_perm, h, packed weights and their scales) must be 128-byte aligned.
 *  - Capacity: permuted buffers have R_cap = T*K rows. Only the first
 *    R = group_offsets[E] rows are written or read; the rest are unspecified.
 *  - Errors: argument checks are synchronous and return a status without
 *    enqueuing anything. A failed launch returns MOE_ERR_CUDA. Conditions found
 *    on the device never trap: they set bits in a device error word that
 *    moe_get_device_errors reads.
 *  - T = 0 (no tokens) is legal and enqueues nothing.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *moe_stream_t;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* bad shape, null pointer or flag combination */
    MOE_ERR_UNSUPPORTED = 2,   /* legal but not implemented (e.g. H % 128 != 0 for the GEMM) */
    MOE_ERR_WORKSPACE = 3,     /* workspace missing or too small */
    MOE_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    MOE_ERR_ALIGNMENT = 5,     /* a pointer is not aligned as required */
    MOE_ERR_DEVICE = 6         /* the device error word is non-zero (moe_get_device_errors) */
} moe_status;

typedef enum {
    MOE_I16 = 0,   /* int16 expert ids (E <= 32767) */
    MOE_I32 = 1,   /* int32 expert ids */
    MOE_BF16 = 2,  /* bfloat16 operands */
    MOE_MXFP8 = 3, /* E4M3 payloads with one E8M0 scale byte per 32 elements */
    MOE_F32 = 4    /* fp32 (layer norm, gradient norm, beam selection) */
} moe_dtype;

/* flags */
#define MOE_ROUTE_RENORM 1u        /* probs normalised over the K selected experts */
#define MOE_PERMUTE_FUSE_MXFP8 2u  /* permute writes MXFP8 rows instead of bf16 rows */
#define MOE_QUANT_COLWISE 4u       /* group-aware 32x1 blocks along rows (wgrad operands) */

/* device error bits */
#define MOE_DEVERR_BAD_ID 1u       /* an expert id outside [-1, E) was seen (treated as invalid) */
#define MOE_DEVERR_TIMEOUT 2u      /* a bounded wait inside a kernel gave up */
#define MOE_DEVERR_NO_PAGE 4u      /* the cache's pool had fewer free pages than its sequences needed */

/* ------------------------------------------------------------------------
 * Router top-K ([SPARSER] "Preserve a compact route": radix/threshold
 * selection with bounded histogram passes for large E and K, a separate fast
 * path for small top-k, and routes carried as a dense [T, K] id list rather
 * than a [T, E] map; [TEJAX] "Optimization 2": router kernels assign tokens
 * before dispatch).
 *
 * logits [T, E] fp32. For every row: the K experts with the largest logits,
 * ties to the lower expert index (-0 and +0 are equal), written to ids[T, K]
 * in that order (int16 or int32 per id_dtype); probs[T, K] fp32 is the softmax
 * over all E logits taken at the selected expert, or, with MOE_ROUTE_RENORM,
 * the softmax over the K selected logits. The router never emits -1.
 * Requires 1 <= K <= E, K <= 128, E <= 8192, no NaN
 * logits (NaN rows give unspecified ids). Small E (<= 256) and K (<= 16) use a
 * warp-per-row arg-max path; E % 4 == 0, E <= 2304 with 16-byte aligned logits
 * use a warp-per-row threshold select; the rest use the radix-select path (a
 * CTA per row). All paths give the same ids and the same probs up to fp32
 * rounding order.
 * ------------------------------------------------------------------------ */
moe_status moe_route_topk(const float *logits, int T, int E, int K,
                          void *ids, moe_dtype id_dtype, float *probs,
                          unsigned flags, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Router backward ([SPARSER] "The workload changes the bottleneck" names a
 * router backward among the kernels, "Preserve a compact route" a backward
 * beside the forward; neither defines it). The gradient of moe_route_topk's
 * probs with respect to the logits, the selection held fixed (top-K is
 * piecewise constant): for row t, S = its valid ids (0 <= id < E; others
 * skipped), g[k] = dprobs[t,k], G_e = sum of g[k] over the k with ids[t,k] = e,
 * p the softmax over all E (with MOE_ROUTE_RENORM: over S, and 0 off S),
 * s = sum over valid k of g[k] p_{ids[t,k]}:
 *   dlogits[t,e] = p_e (G_e - s)       (0 off S with MOE_ROUTE_RENORM).
 * logits [T, E] fp32 (the forward's input), ids [T, K] int16/int32, dprobs
 * [T, K] fp32 in; dlogits [T, E] fp32 out (every element written). Same size
 * limits as moe_route_topk (K <= 128); fp32 arithmetic, within 1e-6 absolute
 * of the exact value for logits of the workloads' scale.
 * ------------------------------------------------------------------------ */
moe_status moe_route_topk_backward(const float *logits, const void *ids, moe_dtype id_dtype,
                                   const float *dprobs, int T, int E, int K,
                                   unsigned flags, float *dlogits, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Sigmoid-score routing with a per-expert selection bias ([SPARSER] "The
 * workload changes the bottleneck": the router's score transformation and
 * top-k selection; "Preserve a compact route": bias statistics carried with
 * compact routes; the pages define neither, the DeepSeek-style reading is
 * taken). For every row t and expert e:
 *   s_e = 1 / (1 + exp(-logits[t,e]))      (fp32)
 *   key_e = s_e + expert_bias[e]            (fp32; bias NULL means 0)
 * ids[t, 0..K) = the K largest keys, in descending order, ties to the lower
 * expert index; probs[t,k] = s at ids[t,k], or with MOE_ROUTE_RENORM that
 * score divided by the sum of the K selected scores. The bias steers only the
 * selection; its statistics (valid routes per expert) are the group_sizes that
 * moe_permute writes. logits [T, E] fp32, expert_bias [E] fp32 (optional) in;
 * ids [T, K] int16/int32 and probs [T, K] fp32 out. One warp per row, keys in
 * registers. Requires 1 <= K <= E, E <= 1024 and K <= 64 (else
 * MOE_ERR_UNSUPPORTED), no NaN logits or biases, finite biases. The score is
 * CUDA's fp32 logistic (within 2 ulp of the correctly rounded value), so two
 * keys within a few ulp of each other may be ordered either way.
 * ------------------------------------------------------------------------ */
moe_status moe_route_sigmoid_topk(const float *logits, const float *expert_bias, int T, int E,
                                  int K, void *ids, moe_dtype id_dtype, float *probs,
                                  unsigned flags, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Backward of moe_route_sigmoid_topk's probs with respect to the logits, the
 * selection held fixed. Row t: S = its distinct valid ids, G_e = sum of
 * dprobs[t,k] over the k with ids[t,k] = e, s_e the score above, Z = sum over
 * S of s_e, c = sum over S of G_e s_e / Z:
 *   dlogits[t,e] = G_e s_e (1 - s_e)                  (e in S)
 *   dlogits[t,e] = s_e (1 - s_e) (G_e - c) / Z        (e in S, MOE_ROUTE_RENORM)
 * and 0 off S (the bias has no gradient path). logits [T, E], ids [T, K],
 * dprobs [T, K] in; dlogits [T, E] fp32 out (every element written).
 * Requires 1 <= K <= min(E, 128).
 * ------------------------------------------------------------------------ */
moe_status moe_route_sigmoid_topk_backward(const float *logits, const void *ids, moe_dtype id_dtype,
                                           const float *dprobs, int T, int E, int K,
                                           unsigned flags, float *dlogits, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Permute / dispatch ([TEJAX] "Dropless vs capacity-based MoE": every routed
 * token is processed, nothing dropped or padded; MoE-layer figure: tokens are
 * grouped per expert and combine restores token order; [SPARSER] "Remove work
 * that has no selected route": local processing visits only the selected
 * slots, found by a warp ballot; invalid routes (-1) are preserved).
 *
 * A device-side counting sort of the T*K routes by expert:
 *   group_sizes[E]      number of valid routes per expert (int32)
 *   group_offsets[E+1]  exclusive scan of group_sizes; group_offsets[E] = R
 *   row_map[T, K]       destination row of route (t, k), -1 if invalid (int32)
 *   perm_src[R_cap]     source token of each destination row (int32; rows >= R untouched)
 *   x_perm[R_cap, H]    x_perm[row_map[t,k]] = x[t] bit for bit (bf16), or with
 *                       MOE_PERMUTE_FUSE_MXFP8: E4M3 payload bytes, with
 *   x_perm_scales[R_cap, H/32]  the row-wise 1x32 E8M0 scale bytes (else NULL).
 * Route (t, k) is valid iff 0 <= ids[t,k] < E; ids outside [-1, E) also set
 * MOE_DEVERR_BAD_ID. Within an expert, rows are in ascending t*K + k order
 * (deterministic; no dependence on atomic ordering). The MXFP8 rule: per 32
 * consecutive elements, scale byte = clamp(floor(log2(amax)) - 8 + 127, 0, 254)
 * (127 for an all-zero block), payload = E4M3(x / 2^(byte-127)) rounded to
 * nearest even and saturated to +-448.
 * Requires H % 32 == 0, 1 <= K <= min(E, 128), E <= 19370 (above 64
 * experts the count kernel keeps a 64-bit token mask and a count per expert in
 * shared memory; larger E gets MOE_ERR_UNSUPPORTED), and a workspace of
 * moe_permute_workspace_size(T, K, E) bytes (16-byte aligned; its contents
 * need not be initialised and are overwritten).
 * ------------------------------------------------------------------------ */
size_t moe_permute_workspace_size(int T, int K, int E);

/* Number of kernels moe_permute launches for this shape (2 when the per-expert,
 * per-token-tile count table is small enough to be scanned inside the scatter
 * kernel, else 3; 0 for T == 0; -1 for invalid sizes). Host-only, no GPU work;
 * not an operation of the pages, a count for launch accounting. */
int moe_permute_kernel_launches(int T, int K, int E);

moe_status moe_permute(const void *x, int T, int H,
                       const void *ids, moe_dtype id_dtype, int K, int E,
                       void *x_perm, uint8_t *x_perm_scales,
                       int32_t *group_sizes, int32_t *group_offsets,
                       int32_t *row_map, int32_t *perm_src,
                       unsigned flags, void *workspace, size_t workspace_bytes,
                       moe_stream_t stream);

/* ------------------------------------------------------------------------
 * moe_permute_noalloc: moe_permute without a caller workspace. (The pages
 * describe nothing like it; it exists for callers of this library.)
 *
 * Some callers cannot allocate device memory: a serving process that reserves
 * all of its GPU memory at start-up and forbids any later cudaMalloc, a plug-in
 * whose host application owns the CUDA allocator and offers C code no hook
 * into it, or code that must not risk the implicit device synchronisation
 * cudaMalloc / cudaFree may perform. This entry point takes the same arguments
 * as moe_permute minus the workspace and allocates nothing: its scratch is a
 * static device array of moe_permute_noalloc_max_scratch() bytes (4 MiB),
 * held by every GPU that loads the library until the process exits.
 *  - Its argument checks (shapes, dtypes, null pointers, alignment) come first
 *    and report what moe_permute reports; then it returns MOE_ERR_WORKSPACE,
 *    without enqueuing anything, when moe_permute_workspace_size(T, K, E)
 *    exceeds that maximum.
 *  - Every call looks up the array's device address on the current device
 *    (cudaGetSymbolAddress), so no address outlives a device reset. The first
 *    call on a device may load the library's device code: make that first call
 *    before any stream capture.
 *  - All calls on a device share the one array, and it keeps the last call's
 *    contents (nothing in it needs to start at zero: each call rewrites what it
 *    reads). Calls that overlap on the GPU (other streams, or other host threads
 *    on the same device) race on it: serialise them.
 * Outputs, requirements and errors are otherwise those of moe_permute.
 * ------------------------------------------------------------------------ */
size_t moe_permute_noalloc_max_scratch(void);

moe_status moe_permute_noalloc(const void *x, int T, int H,
                               const void *ids, moe_dtype id_dtype, int K, int E,
                               void *x_perm, uint8_t *x_perm_scales,
                               int32_t *group_sizes, int32_t *group_offsets,
                               int32_t *row_map, int32_t *perm_src,
                               unsigned flags, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Expert-parallel dispatch metadata ([TEJAX] "Optimization 2: Expert
 * parallelism to fuse Dispatch and Combine"; [SPARSER] "Remove work that has
 * no selected route": only selected routes travel, each destination receives
 * the rows of its own experts).
 *
 * G ranks, E_loc experts per rank (rank g owns experts g*E_loc ..
 * g*E_loc + E_loc - 1). Every source rank sends, from its moe_permute order,
 * the rows of the destination's experts (they are contiguous there); the
 * destination receives them source by source and, within a source, expert by
 * expert. recv_counts [G][E_loc] int32 (device): rows received from source s
 * for local expert j (the exchanged group sizes). Writes ids [R_cap] int32
 * (device): the local expert of each received row r, i.e. j of the segment
 * (s, j) that holds r when the segments are laid end to end in that order;
 * rows past the last segment get -1. moe_permute of the received rows with
 * these ids (K = 1, E = E_loc) gives the local experts' contiguous order.
 * Requires G * E_loc <= 4096; a negative count is read as 0 and sets
 * MOE_DEVERR_BAD_ID. Enqueues one kernel; the host never reads the counts.
 * ------------------------------------------------------------------------ */
moe_status moe_ep_recv_expert_ids(const int32_t *recv_counts, int G, int E_loc,
                                  long long R_cap, int32_t *ids, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Group-aware MXFP8 quantisation ([TEJAX] "Transformer Engine building
 * blocks": group-aware MXFP8 quantization feeding the MXFP8 grouped GEMM).
 *
 * x [R_cap, H] bf16, rows [group_offsets[e], group_offsets[e+1]) forming
 * group e; only rows < group_offsets[E] are read or written.
 *  - default (row-wise 1x32): q[R_cap, H] E4M3, scales[R_cap, H/32].
 *  - MOE_QUANT_COLWISE (32x1 along rows, for the weight-gradient GEMMs whose
 *    contraction runs over a group's rows): blocks start at each group's first
 *    row and never cross a group; a partial last block takes its amax over its
 *    valid rows. q[R_cap, H]; scales[E + R_cap/32 + 1, H] where block b of
 *    group e is scale row e + group_offsets[e]/32 + b (rows no block uses are
 *    left untouched).
 * Same scale/payload rule as moe_permute. Requires H % 32 == 0.
 * ------------------------------------------------------------------------ */
moe_status moe_quant_mxfp8_grouped(const void *x, int R_cap, int H,
                                   const int32_t *group_offsets, int E,
                                   uint8_t *q, uint8_t *scales,
                                   unsigned flags, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * NVFP4 operands ([TEJAX] "Measured training impact with JAX + Transformer
 * Engine" and [WITTY] "What to watch" name NVFP4 as a planned addition and do
 * not define it; NVIDIA's published format is taken). Elements E2M1 (0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives); 16 consecutive elements of a row
 * share one E4M3 decode scale; the tensor has one fp32 encode scale
 * S = 448 * 6 / amax (1 when amax is 0, at most FLT_MAX); a value decodes as
 * e2m1 * e4m3(scale) / S. Encoder, in fp32 with one rounding per operation:
 *   scale = E4M3(round to nearest even, saturating)((amax_block / 6) * S)
 *   code  = E2M1(round to nearest even, saturating to 6, sign kept)(x * (S / e4m3(scale))),
 *           0 when e4m3(scale) is 0.
 * Packing: element 2i in the low nibble of byte i, 2i+1 in the high nibble.
 *
 * moe_amax_bf16: *amax = max |x| over rows [0, n) of x [rows, cols] bf16, with
 *   n = rows, or min(rows, *valid_rows) when valid_rows (a device int, e.g.
 *   &group_offsets[E]) is given; cols % 8 == 0; amax is zeroed on the stream
 *   first. moe_quant_nvfp4: the same rows of x quantised with the encode scale of
 *   the device *amax: q [rows, cols/2] packed codes (8-byte aligned), scales
 *   [rows, cols/16]; rows past n are not written; cols % 16 == 0.
 * ------------------------------------------------------------------------ */
moe_status moe_amax_bf16(const void *x, long long rows, int cols, const int32_t *valid_rows,
                         float *amax, moe_stream_t stream);
moe_status moe_quant_nvfp4(const void *x, long long rows, int cols, const int32_t *valid_rows,
                           const float *amax, uint8_t *q, uint8_t *scales, moe_stream_t stream);

/* moe_permute_nvfp4: moe_permute (same routing outputs, workspace and rules)
 * whose scatter writes NVFP4 rows: first *x_amax = max |x| over the tokens
 * with at least one valid route (exactly the amax of the rows x_perm
 * receives; zeroed on the stream first), then each row is quantised with that
 * amax's encode scale as it is copied: x_perm_q [T*K, H/2] packed E2M1 (4-byte
 * aligned), x_perm_scales [T*K, H/16] E4M3 -- the bytes moe_quant_nvfp4 would
 * write from the bf16 permuted rows. One kernel more than moe_permute. */
moe_status moe_permute_nvfp4(const void *x, int T, int H, const void *ids, moe_dtype id_dtype,
                             int K, int E, float *x_amax, void *x_perm_q, uint8_t *x_perm_scales,
                             int32_t *group_sizes, int32_t *group_offsets, int32_t *row_map,
                             int32_t *perm_src, void *workspace, size_t workspace_bytes,
                             moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Grouped SwiGLU expert MLP ([TEJAX] "Optimization 1: Grouped GEMM": one
 * kernel covers all experts, each with its actual token count, computing only
 * valid regions, with the counts kept on the device; MoE-layer figure: the
 * grouped MLP is two grouped GEMMs on variable-length groups; "Transformer
 * Engine building blocks": MXFP8 grouped GEMM on Blackwell).
 *
 * For each expert e and each row r in [group_offsets[e], group_offsets[e+1]):
 *   a = x_perm[r] W1[e],  b = x_perm[r] W3[e]       (fp32 accumulation)
 *   h[r] = silu(a) * b    rounded to bf16, or (MXFP8) quantised 1x32 along F
 *   y_perm[r] = h[r] W2[e]  rounded to bf16
 * Rows >= group_offsets[E] are never written. Logical weights: W1, W3 [E, H, F]
 * and W2 [E, F, H] bf16; the GEMMs read them packed once by
 * moe_prepare_weights (outside the hot path):
 *   w13_packed [E][2F][H]: per 256-row tile j, rows 0..127 = columns
 *              128j..128j+127 of W1 transposed, rows 128..255 the same of W3;
 *   w2_packed  [E][H][F] = W2 transposed per expert;
 * bf16, or MXFP8 (E4M3 bytes, plus E8M0 scales [E][2F][H/32] and [E][H][F/32]
 * with blocks of 32 along the contraction dimension).
 * Activations: x_perm [R_cap, H] bf16, or MXFP8 E4M3 with x_scales
 * [R_cap, H/32] (as written by moe_permute with MOE_PERMUTE_FUSE_MXFP8);
 * h [R_cap, F] (caller-allocated intermediate, kept for the backward pass)
 * bf16, or E4M3 with h_scales [R_cap, F/32]; y_perm [R_cap, H] bf16.
 * Requires H % 256 == 0 and F % 128 == 0 (MXFP8: H % 512 == 0 and F % 512 == 0),
 * x_perm, h and the packed weights 128-byte aligned, scales 16-byte aligned,
 * E small enough for the group table to fit in shared memory (bf16: E <= 4200,
 * MXFP8: E <= 1150). moe_grouped_gemm_up / _down run the two halves alone.
 * ------------------------------------------------------------------------ */
size_t moe_packed_weights_bytes(int E, int H, int F, moe_dtype dtype, int which);
/* which: 0 = w13 payload, 1 = w13 scales, 2 = w2 payload, 3 = w2 scales (0 bytes for bf16) */

moe_status moe_prepare_weights(const void *w1, const void *w3, const void *w2, int E, int H, int F,
                               moe_dtype dtype, void *w13_packed, uint8_t *w13_scales,
                               void *w2_packed, uint8_t *w2_scales, moe_stream_t stream);

moe_status moe_grouped_swiglu_gemm(const void *x_perm, const uint8_t *x_scales,
                                   const void *w13_packed, const uint8_t *w13_scales,
                                   const void *w2_packed, const uint8_t *w2_scales, moe_dtype dtype,
                                   const int32_t *group_offsets, int E, int H, int F, int R_cap,
                                   void *h, uint8_t *h_scales, void *y_perm, moe_stream_t stream);

/* moe_grouped_gemm_up also saves, when the pointers are not NULL, what the
 * backward pass needs: ab_save [R_cap, 2F] bf16, the pre-activations a and b in
 * the interleaved layout of w13_packed (per 256 columns: 128 of a, then the
 * same 128 columns of b); h_bf16_save [R_cap, F] bf16, a bf16 copy of h (MXFP8
 * only, for the column-wise quantisation of the weight gradient). */
moe_status moe_grouped_gemm_up(const void *x_perm, const uint8_t *x_scales, const void *w13_packed,
                               const uint8_t *w13_scales, moe_dtype dtype,
                               const int32_t *group_offsets, int E, int H, int F, int R_cap,
                               void *h, uint8_t *h_scales, void *ab_save, void *h_bf16_save,
                               moe_stream_t stream);

moe_status moe_grouped_gemm_down(const void *h, const uint8_t *h_scales, const void *w2_packed,
                                 const uint8_t *w2_scales, moe_dtype dtype,
                                 const int32_t *group_offsets, int E, int H, int F, int R_cap,
                                 void *y_perm, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * The grouped SwiGLU MLP's two GEMMs on NVFP4 operands (tcgen05 kind
 * mxf4nvf4: E2M1 x E2M1 with a UE4M3 scale per 16 elements, fp32
 * accumulation, the two tensors' encode scales divided out in the epilogue).
 * Operands as moe_quant_nvfp4 writes them: x_q [R_cap, H/2] + x_scales
 * [R_cap, H/16] with the device x_amax; weights in the packed layouts of
 * moe_grouped_gemm_up (w13 [E][2F][H]) and down (w2 [E][H][F]) quantised
 * row-wise along the contraction dimension, each stacked tensor with one amax.
 * moe_grouped_gemm_up_nvfp4 writes h [R_cap, F] bf16 = silu(a) * b, the
 * optional ab_save like moe_grouped_gemm_up, and *h_amax = max |h| over the
 * rows it wrote (zeroed on the stream first), which moe_quant_nvfp4 takes to
 * quantise h for moe_grouped_gemm_down_nvfp4 (y_perm [R_cap, H] bf16).
 * Requires H % 256 == 0 and F % 256 == 0 (128-byte k-blocks of 256 elements);
 * operand bases 128-byte aligned, scales 16-byte aligned.
 * ------------------------------------------------------------------------ */
moe_status moe_grouped_gemm_up_nvfp4(const void *x_q, const uint8_t *x_scales, const float *x_amax,
                                     const void *w13_q, const uint8_t *w13_scales, const float *w13_amax,
                                     const int32_t *group_offsets, int E, int H, int F, int R_cap,
                                     void *h, float *h_amax, void *ab_save, moe_stream_t stream);
moe_status moe_grouped_gemm_down_nvfp4(const void *h_q, const uint8_t *h_scales, const float *h_amax,
                                       const void *w2_q, const uint8_t *w2_scales, const float *w2_amax,
                                       const int32_t *group_offsets, int E, int H, int F, int R_cap,
                                       void *y_perm, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Grouped backward of the SwiGLU expert MLP (the training step of [TEJAX]
 * "Measured training impact", on the same ragged groups as the forward).
 *
 * For each expert e and row r of its group, with a, b the saved bf16
 * pre-activations (ab_save of moe_grouped_gemm_up) and dy the gradient of y_perm:
 *   dh = dy W2[e]^T;  da = dh * b * silu'(a);  db = dh * silu(a)
 *       (silu'(a) = s(a) (1 + a (1 - s(a))), s the logistic function)
 *   dx = da W1[e]^T + db W3[e]^T
 *   dW2[e] = h_e^T dy_e;  dW1[e] = x_e^T da_e;  dW3[e] = x_e^T db_e
 * (fp32 accumulation, bf16 outputs). Backward weights, packed once by
 * moe_prepare_weights_bwd: w2_bwd [E][F][H] (= W2) and w13t [E][H][2F] (row h =
 * W1[e][h] and W3[e][h] interleaved per 128 columns), bf16 or MXFP8 with blocks
 * along H and along 2F respectively.
 *
 * moe_grouped_swiglu_dgrad: dy [R_cap, H] (bf16, or MXFP8 row-wise: E4M3 +
 *   dy_scales [R_cap, H/32]) -> dab [R_cap, 2F] bf16 = (da | db) interleaved per
 *   128 columns like ab. Requires F % 256 == 0. Optional (both or neither, NULL
 *   skips): dab_q [R_cap, 2F] E4M3 bytes (32-byte aligned) and dab_scales
 *   [R_cap, 2F/32] E8M0, the row-wise MXFP8 of the bf16 dab (1x32 blocks along
 *   2F, as moe_quant_mxfp8_grouped writes it), for moe_grouped_gemm_dx.
 * moe_grouped_gemm_dx: dab (bf16, or MXFP8 row-wise along 2F) -> dx [R_cap, H] bf16.
 * moe_grouped_transpose: makes a weight-gradient operand: for x [R_cap, C] bf16
 *   (or, with src_rows != NULL, x [*, C] read at row src_rows[r], e.g. the
 *   tokens through perm_src), xT[c][P_e + i] = x[off[e] + i][c] for i < m_e, with
 *   P_e = 128 * (e + off[e] / 128) and zeros up to P_e + 128 * ceil(m_e / 128);
 *   xT is [C][Kpad], Kpad = moe_grouped_transpose_kpad(R_cap, E) (a multiple of
 *   512 at least 128 * (E + ceil(R_cap / 128) + 1)). MXFP8 output:
 *   group-aware 32-row blocks (starting at each group's first row, a partial
 *   block taking its amax over valid rows), E4M3 payload in xT and E8M0 scales
 *   xT_scales[c][P_e / 32 + b] ([C][Kpad/32]). Requires C % 64 == 0.
 * moe_grouped_gemm_wgrad: aT [M][Kpad], bT [N][Kpad] from moe_grouped_transpose
 *   -> dw [E][M][N] bf16 with dw[e] = sum over group e's rows of a^T b; with dw2
 *   != NULL the output is split: columns [256j, 256j+128) of each row go to
 *   dw [E][M][N/2] and [256j+128, 256j+256) to dw2 (so bT = transposed dab gives
 *   dW1 and dW3 in their logical layouts). An expert with no rows gets zeros.
 *   Requires M % 128 == 0, N % 256 == 0.
 * ------------------------------------------------------------------------ */
moe_status moe_prepare_weights_bwd(const void *w1, const void *w3, const void *w2, int E, int H, int F,
                                   moe_dtype dtype, void *w2_bwd, uint8_t *w2_bwd_scales,
                                   void *w13t, uint8_t *w13t_scales, moe_stream_t stream);

moe_status moe_grouped_swiglu_dgrad(const void *dy, const uint8_t *dy_scales, const void *w2_bwd,
                                    const uint8_t *w2_bwd_scales, const void *ab, moe_dtype dtype,
                                    const int32_t *group_offsets, int E, int H, int F, int R_cap,
                                    void *dab, uint8_t *dab_q, uint8_t *dab_scales,
                                    moe_stream_t stream);

moe_status moe_grouped_gemm_dx(const void *dab, const uint8_t *dab_scales, const void *w13t,
                               const uint8_t *w13t_scales, moe_dtype dtype,
                               const int32_t *group_offsets, int E, int H, int F, int R_cap,
                               void *dx, moe_stream_t stream);

size_t moe_grouped_transpose_kpad(int R_cap, int E);

moe_status moe_grouped_transpose(const void *x, const int32_t *src_rows, int R_cap, int C,
                                 const int32_t *group_offsets, int E, moe_dtype out_dtype,
                                 void *xT, uint8_t *xT_scales, moe_stream_t stream);

moe_status moe_grouped_gemm_wgrad(const void *aT, const uint8_t *aT_scales, const void *bT,
                                  const uint8_t *bT_scales, moe_dtype dtype,
                                  const int32_t *group_offsets, int E, int M, int N, int R_cap,
                                  void *dw, void *dw2, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Unpermute / combine ([TEJAX] "Optimization 2": results are routed back and
 * accumulated; [SPARSER] "Remove work that has no selected route": combine is a
 * pull-and-reduce over each token's selected rows).
 *
 * y[t, :] = bf16( sum over k = 0..K-1 with row_map[t,k] >= 0 of
 *                 probs[t,k] * y_perm[row_map[t,k], :] )
 * accumulated in fp32 in ascending k; a token with no valid route gets zeros.
 * y_perm [R_cap, H] bf16, row_map [T, K] int32, probs [T, K] fp32, y [T, H] bf16.
 * Requires H % 8 == 0.
 * ------------------------------------------------------------------------ */
moe_status moe_unpermute_combine(const void *y_perm, const int32_t *row_map,
                                 const float *probs, int T, int K, int H,
                                 void *y, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Combine backward: the adjoint of moe_unpermute_combine (the chain rule
 * through y[t] = sum_k p[t,k] y_perm[row_map[t,k]]; the pages give the
 * forward, [TEJAX] "Optimization 2", and name training, not this step).
 * For every valid route (t, k) with row r = row_map[t,k]:
 *   dy_perm[r]   = bf16(p[t,k] * dy[t])                  (one rounding)
 *   dprobs[t,k]  = sum_j dy[t,j] * y_perm[r,j]            (fp32 accumulation)
 * and dprobs[t,k] = 0 for invalid routes. dy [T, H] bf16, y_perm [R_cap, H]
 * bf16 (the forward's), row_map [T, K], probs [T, K] fp32 in; dy_perm
 * [R_cap, H] bf16 (rows no route maps to are not written) and dprobs [T, K]
 * fp32 out. Requires H % 8 == 0, 1 <= K <= 128; 16-byte aligned rows.
 * Optional (both or neither; NULL skips): dy_perm_q [R_cap, H] E4M3 bytes
 * (8-byte aligned) and dy_perm_scales [R_cap, H/32] E8M0 bytes, the row-wise
 * MXFP8 quantisation (1x32 blocks along H, as moe_quant_mxfp8_grouped writes
 * it) of the bf16 dy_perm values, for the next grouped GEMM; requires
 * H % 32 == 0. Same rows written as dy_perm.
 * ------------------------------------------------------------------------ */
moe_status moe_unpermute_combine_backward(const void *dy, const void *y_perm,
                                          const int32_t *row_map, const float *probs,
                                          int T, int K, int H, void *dy_perm,
                                          float *dprobs, uint8_t *dy_perm_q,
                                          uint8_t *dy_perm_scales, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Permute backward: the adjoint of moe_permute's row copies, dx[t] = bf16(sum
 * over the valid k, ascending, of dx_perm[row_map[t,k]]) with fp32
 * accumulation; tokens without a valid route get 0. dx_perm [R_cap, H] bf16,
 * row_map [T, K] in; dx [T, H] bf16 out. Requires H % 8 == 0, 1 <= K <= 128.
 * ------------------------------------------------------------------------ */
moe_status moe_permute_backward(const void *dx_perm, const int32_t *row_map,
                                int T, int K, int H, void *dx, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * The whole layer for a few tokens (a decoding step): router, up projection, and down
 * projection with the combine, three kernels that overlap, on the same packed weights
 * as the grouped GEMMs.
 * (The pages describe training batches and no such call.)
 *
 * x [T, H] bf16, logits [T, E] fp32. ids [T, K] and probs [T, K] as
 * moe_route_topk gives them (same flags), written; with logits NULL they are
 * inputs instead (any router's; an id outside [0, E) is an invalid route, outside
 * [-1, E) it also sets MOE_DEVERR_BAD_ID). For every valid route (t, k), e = ids[t,k]:
 *   a = x[t] W1[e],  b = x[t] W3[e]                       (fp32 accumulation)
 *   h = silu(a) * b, rounded to bf16, or (MXFP8) quantised 1x32 along F
 *   y[t] = bf16( sum over the valid k of probs[t,k] * (h W2[e]) )
 * with the sums over F and k in fp32 and one rounding at the end (the batched path
 * rounds every route's row to bf16 before the combine). MXFP8: x is quantised 1x32
 * along H first, as moe_permute does. A token without a valid route gets zeros.
 * w13_packed, w2_packed and their scales: moe_prepare_weights, dtype MOE_BF16 or
 * MOE_MXFP8. Outputs do not depend on the timing of the GPU's blocks.
 * Requires 0 <= T <= 64, 1 <= K <= min(E, 128), T * K <= 4096, E <= 8192 (MXFP8: with
 * E > 2304, T * K above 2048 may not fit shared memory; above: MOE_ERR_UNSUPPORTED),
 * H % 128 == 0 and F % 128 == 0 (MXFP8: both % 512), the packed weights and the workspace
 * 128-byte aligned, x, y and the scales 16-byte, ids and probs to their element. workspace: moe_layer_few_tokens_workspace_size bytes (0 for sizes
 * that are refused); its contents need not be initialised, and calls that share one
 * must not overlap. Every wait inside is bounded (MOE_DEVERR_TIMEOUT).
 * ------------------------------------------------------------------------ */
size_t moe_layer_few_tokens_workspace_size(int T, int K, int E, int H, int F, moe_dtype dtype);

moe_status moe_layer_few_tokens(const void *x, int T, int H, const float *logits, int K, int E, int F,
                                const void *w13_packed, const uint8_t *w13_scales,
                                const void *w2_packed, const uint8_t *w2_scales, moe_dtype dtype,
                                void *ids, moe_dtype id_dtype, float *probs, void *y,
                                unsigned flags, void *workspace, size_t workspace_bytes,
                                moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm around the layer (the norm of a pre-norm block; the pages do not
 * describe one). For every row t of x [T, H] (dtype MOE_BF16 or MOE_F32):
 *   s = x[t], or with residual [T, H]: s = round(x[t] + residual[t]) to dtype, also
 *       written to sum [T, H] (required with residual, NULL without)
 *   mean[t] = sum s / H;  rstd[t] = 1 / sqrt(sum (s - mean)^2 / H + eps)   (fp32)
 *   y[t] = round((s - mean) * rstd * weight + bias)
 * weight, bias [H] of dtype w_dtype (MOE_BF16 or MOE_F32); bias may be NULL (0). mean, rstd
 * [T] fp32, NULL to skip. y, sum of dtype; sum may be x or residual itself, y may be any
 * of them too. Pointers aligned to their elements (16 bytes and a row of whole 16-byte
 * pieces take the wide path). Requires T >= 0, 1 <= H <= 65536, eps >= 0.
 * ------------------------------------------------------------------------ */
moe_status moe_layer_norm(const void *x, const void *residual, int T, int H, moe_dtype dtype,
                          const void *weight, const void *bias, moe_dtype w_dtype, float eps,
                          void *sum, void *y, float *mean, float *rstd, moe_stream_t stream);

/* Its backward pass: s [T, H] (the normalised stream: x, or sum), dy [T, H], the forward's
 * mean and rstd, weight. With xh = (s - mean) rstd and g = dy * weight:
 *   dx[t] = round( rstd (g - sum(g)/H - xh sum(g xh)/H) + dx_add[t] )
 *   dweight = round(sum over t of dy xh),  dbias = round(sum over t of dy)
 * dx_add [T, H] (the gradient that reaches s past the norm) may be NULL, dx may be dy or
 * dx_add itself. dweight [H] and dbias [H] (each NULL to skip) of w_dtype; T = 0 writes
 * zeros to them. Sums in fp32, in an order that depends on the sizes and the device only.
 * workspace: moe_layer_norm_backward_workspace_size bytes, 16-byte aligned, not
 * initialised. Same limits as the forward. */
size_t moe_layer_norm_backward_workspace_size(int T, int H);

moe_status moe_layer_norm_backward(const void *dy, const void *s, int T, int H, moe_dtype dtype,
                                   const void *weight, moe_dtype w_dtype, const float *mean,
                                   const float *rstd, const void *dx_add, void *dx, void *dweight,
                                   void *dbias, void *workspace, size_t workspace_bytes,
                                   moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping by it (the step between
 * the layer's backward pass and an optimiser; the pages do not describe it).
 *   norm = sqrt( sum over the n tensors of sum g^2 )                       (fp32)
 *   c = 1 if norm + eps <= max_norm, else max_norm / (norm + eps);   outs[i] = round(grads[i] * c)
 * grads, counts, dtypes, outs are host arrays of n entries: device pointers (aligned to
 * their element), element counts (0 is legal, the pointer is then not used), MOE_BF16 or
 * MOE_F32. outs NULL: only the norm. outs[i] may be grads[i] (in place: with c = 1 nothing
 * is written) and has the type of grads[i]. *norm_out (device fp32). A NaN in a gradient
 * makes norm and every output NaN; an infinite norm gives c = 0 (0 * inf is NaN), but with
 * max_norm infinite too c = 1: such a bound only measures. The tensors must not overlap. Squares
 * are summed in fp32 (values above about 1e19 overflow to an infinite norm, those below
 * about 1e-19 lose bits and below 1e-23 vanish) in an order that
 * depends on the sizes and the device only. The host never reads the norm. Requires n >= 0,
 * max_norm >= 0, eps >= 0 (not NaN). workspace: moe_grad_norm_workspace_size(n) bytes,
 * 16-byte aligned, not initialised. The host arrays are read during the call only.
 * ------------------------------------------------------------------------ */
size_t moe_grad_norm_workspace_size(int n);

moe_status moe_grad_norm_clip(const void *const *grads, const long long *counts,
                              const int *dtypes, void *const *outs, int n, float max_norm,
                              float eps, float *norm_out, void *workspace,
                              size_t workspace_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged key-value cache (a decoding step's attention around the layer; the pages
 * do not describe one). One layer's cache is two pools of pages, keys and values
 * [pages, heads, page_size, dim], of dtype MOE_BF16, or MOE_MXFP8 with scales
 * [pages, heads, page_size, dim/32] (the row rule of moe_permute along dim). A table
 * [S, M] int32 gives the pages of S sequences: position p of sequence s is offset
 * p % page_size of page table[s, p / page_size]. -1 marks no page. A page id outside
 * [-1, pages) where a position is read or written, or -1 there, sets MOE_DEVERR_BAD_ID;
 * the position is then left out. Many rows may name one page. The calls below require
 * 1 <= pages, heads, dim % 16 == 0 (MXFP8: % 32), dim <= 256, 1 <= page_size <= 4096,
 * 1 <= M, M * page_size < 2^31; tables, lengths and positions 4-byte aligned, everything
 * else 16-byte (scales: to the largest power of two that divides dim / 32, 8 at most).
 *
 * moe_cache_append: k, v [n, heads, dim] bf16, tokens k_stride and v_stride elements apart
 * (multiples of 8; slices of one projection), to position positions[i] of sequence rows[i]
 * (rows NULL: of sequence i, n <= S). A negative position or row is skipped (padding); a
 * position at or past M * page_size or a row >= S is a bad id. The (page, offset) pairs of one
 * call must be distinct. MXFP8 quantises on the way. n <= 2^30.
 * moe_cache_gather: the same positions read back, k, v [n, heads, dim] bf16 contiguous
 * (MXFP8: code times scale, exact within bf16's range), zeros for the positions that are skipped or
 * bad.
 * ------------------------------------------------------------------------ */
moe_status moe_cache_append(const void *k, const void *v, long long k_stride, long long v_stride,
                            int n, const int32_t *rows, const int32_t *positions,
                            const int32_t *table, int S, int M, moe_dtype dtype, int pages,
                            int heads, int page_size, int dim, void *k_pages, uint8_t *k_scales,
                            void *v_pages, uint8_t *v_scales, moe_stream_t stream);

moe_status moe_cache_gather(void *k, void *v, int n, const int32_t *rows, const int32_t *positions,
                            const int32_t *table, int S, int M, moe_dtype dtype, int pages,
                            int heads, int page_size, int dim, const void *k_pages,
                            const uint8_t *k_scales, const void *v_pages,
                            const uint8_t *v_scales, moe_stream_t stream);

/* Attention of one new token per sequence over the cache. q [B, q_heads, dim] bf16, sequences
 * q_stride elements apart (a multiple of 8); q_heads a multiple of heads, query head h reads
 * key head h / (q_heads / heads). With n = lengths[b] (negative: 0; above M * page_size: that, and
 * MOE_DEVERR_BAD_ID) and first = window > 0 ? max(0, n - window) : 0, over first <= j < n:
 *   s_j = scale q.k_j;  m = max s;  l = sum exp(s_j - m);  out = round(sum exp(s_j - m) v_j / l)
 *   lse = m + ln l
 * out [B, q_heads, dim] bf16, lse [B, q_heads] fp32 (NULL to skip). Without a position: out 0,
 * lse -inf. What lies in the pages beside these positions does not matter (NaN among it). Sums,
 * maxima and the joined parts are fp32; the weights exp(s - m) meet the values as two bf16 (16 bits)
 * beside bf16 values and where the scales of MXFP8 ones lie far apart, as fp16 (11 bits) beside other
 * MXFP8 ones; l is summed before that. Sums of exp(s - m) |v| beyond fp32's range give infinities.
 * Outputs depend on the sizes, lengths and the device, not on timing. Requires B <= 65535,
 * q_heads / heads <= 1024, finite scale, window >= 0. workspace:
 * moe_paged_attention_workspace_size bytes (0 for refused sizes), 16-byte aligned, not
 * initialised; calls that share one must not overlap. */
size_t moe_paged_attention_workspace_size(int B, int q_heads, int heads, int dim);

moe_status moe_paged_attention(const void *q, long long q_stride, int B, int q_heads,
                               const void *k_pages, const uint8_t *k_scales, const void *v_pages,
                               const uint8_t *v_scales, moe_dtype dtype, int pages, int heads,
                               int page_size, int dim, const int32_t *table, int M,
                               const int32_t *lengths, float scale, int window, void *out,
                               float *lse, void *workspace, size_t workspace_bytes,
                               moe_stream_t stream);

/* Page bookkeeping on the device: no counts of pages are kept, a page is free when no row of the
 * table names it.
 *
 * moe_cache_fork: S_new sequences that go on from parents [S_new] (NULL: each from itself, S_new
 * = S). Row i of new_table [S_new, M] is row parents[i] of table, cut to the pages that
 * lengths[parents[i]] positions take; new_lengths[i] is that length; parent -1 (or outside
 * [-1, S): a bad id) gives an empty row of length 0. Then every row with a parent gets room
 * for `room` more positions (rooms [S_new], where given, instead; negative: 0): a page that it
 * would write in but shares is replaced by a free one and (src[i], dst[i]) says what to copy (-1, -1 where
 * nothing is); the row that keeps a shared page is the one with most positions in it, then the
 * first. The pages behind are free ones too (up to M). Free pages go out in ascending order, to
 * rows in ascending order, the copied page first. Pages that no row names any more are free.
 * *used: the pages named in the end, and those that were missing: then *used > pages and
 * MOE_DEVERR_NO_PAGE is set, and the entries are -1, that of a last page that could not be copied
 * among them, so the new row has lost the positions in it. table and lengths still have all; a caller
 * that finds *used > pages copies nothing and goes on from those. Outputs must not overlap inputs.
 * Requires (page_size + 1) * S_new < 2^31, M * S_new < 2^31 (compact: M * S), pages <= 2^30.
 *
 * moe_cache_compact: the named pages renumbered to 0 .. *used - 1: the i-th page at or above
 * *used goes to the i-th hole below it. new_table: the rows with the new numbers; src, dst
 * [pages / 2]: the moves, in order, -1 behind the last. A bad id in the table becomes -1. new_table
 * may be table.
 *
 * moe_cache_copy_pages: page dst[i] = page src[i] for n <= 2^30 pairs, in n_tensors pools (host arrays of
 * device pointers and bytes a page); pairs with -1 are skipped, ids outside [-1, pages) are
 * skipped and bad. No page may be the destination of two pairs, nor of one and the source of
 * another (the lists of the two calls above are so). The host arrays are read during the call only.
 *
 * workspace: moe_cache_pages_workspace_size bytes (rows: of the new table), 16-byte aligned, not
 * initialised; calls that share one must not overlap. */
size_t moe_cache_pages_workspace_size(int pages, int rows);

moe_status moe_cache_fork(const int32_t *table, const int32_t *lengths, int S, int M,
                          const int32_t *parents, int S_new, int pages, int page_size, int room,
                          const int32_t *rooms, int32_t *new_table, int32_t *new_lengths,
                          int32_t *src, int32_t *dst, int32_t *used, void *workspace,
                          size_t workspace_bytes, moe_stream_t stream);

moe_status moe_cache_compact(const int32_t *table, int S, int M, int pages, int32_t *new_table,
                             int32_t *src, int32_t *dst, int32_t *used, void *workspace,
                             size_t workspace_bytes, moe_stream_t stream);

moe_status moe_cache_copy_pages(void *const *tensors, const long long *page_bytes, int n_tensors,
                                const int32_t *src, const int32_t *dst, int n, int pages,
                                moe_stream_t stream);

/* Selection of a beam search's step. logits [N, W, V] (MOE_F32 or MOE_BF16), scores [N, W] fp32.
 * Candidate (w, t) of search n: scores[n,w] + (logits[n,w,t] - lse), lse = ln sum exp(logits[n,w]); of a
 * beam whose score or lse is not finite: -inf. done [N, W] bytes (NULL: none): a beam that is
 * done has one candidate, token pad with its score as it is, and -inf elsewhere. The K largest in
 * order, ties to the lower w, then the lower t: out_scores [N, K] fp32, parents [N, K] = n * W + w,
 * tokens [N, K]. lse is summed in fp32, the same pieces of a row apart wherever it lies (equal
 * beams have equal candidates, and a search its scores whatever stands beside it); it, the joined
 * sums and the candidates are held in two floats (46 bits or more; a candidate that fp32 rounds
 * to -inf counts as -inf) and rounded once. Requires 1 <= W <= 64, 1 <= V < 2^24,
 * N * W < 2^24, 1 <= K <= 64, K <= W * V, 0 <= pad < V with done. workspace:
 * moe_beam_select_workspace_size bytes (0 for refused sizes), 16-byte aligned, not initialised; calls that
 * share one must not overlap. */
size_t moe_beam_select_workspace_size(int N, int W, int V, int K);

moe_status moe_beam_select(const void *logits, moe_dtype dtype, const float *scores,
                           const uint8_t *done, int pad, int N, int W, int V, int K,
                           float *out_scores, int32_t *parents, int32_t *tokens, void *workspace,
                           size_t workspace_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Device error word. Copies the word to *flags_out (synchronising the device)
 * and clears it when `clear` is non-zero. Not for the hot path. Returns
 * MOE_ERR_DEVICE when the word was non-zero.
 * ------------------------------------------------------------------------ */
moe_status moe_get_device_errors(uint32_t *flags_out, int clear);

/* Self-test of the bounded waits the grouped GEMM uses for its pipeline barriers:
 * launches one warp that waits on a barrier nothing arrives on; after limit_us
 * microseconds (1 .. 1,000,000) the wait gives up, sets MOE_DEVERR_TIMEOUT in the
 * device error word and the kernel returns, leaving the context usable. */
moe_status moe_debug_bounded_wait_selftest(uint32_t limit_us, moe_stream_t stream);

/* Human-readable name of a status code (static storage). */
const char *moe_status_string(moe_status status);

/* Device address of page-locked host memory (cudaHostAlloc / pinned): on systems with a
 * unified address space the library's kernels can read their inputs from, and write their
 * outputs to, such memory directly (moe_permute's x, moe_unpermute_combine's y), so a caller
 * whose tensors live on the host needs no separate copy in or out. Writes *dev_ptr and returns
 * MOE_OK when host_ptr lies in page-locked memory the current device can address,
 * MOE_ERR_UNSUPPORTED otherwise (plain pageable memory, no mapping), MOE_ERR_INVALID_ARG for
 * null pointers. No work is enqueued. (The pages describe no such call.) */
moe_status moe_host_mapped_pointer(const void *host_ptr, void **dev_ptr);

/* Byte sizes of the compact route ([SPARSER] "Preserve a compact route":
 * [T, K] ids instead of a [T, E] map): ids of the given dtype, and fp32 probs. */
size_t moe_route_ids_bytes(int T, int K, moe_dtype id_dtype);
size_t moe_route_probs_bytes(int T, int K);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
