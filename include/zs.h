/*
 * zs.h -- C ABI of libzs: the zonal scatter of the geometric initial
 * embedding (GIE) of an SO(3)-equivariant interatomic potential, lmax = 3,
 * forward and backward, with the stable destination CSR it walks.
 *
 * What the operation is: deepmd-kit pull request "fused Triton zonal scatter
 * for the GIE head (DP_GIE_SCATTER_INFER)", section "What" (forward bullet:
 * a node-parallel walk of the stable destination CSR that accumulates the
 * message without materialising the (E, D-1, C) surface and writes the
 * padded (N, D, C) node layout with a zero scalar row; backward bullet: one
 * edge-parallel pass giving the (E, D-1) coupling and (E, lmax, C) radial
 * gradients; last bullet: the reduction follows the stable-sort CSR order)
 * and section "Boundary and layout contract" (contiguous inputs, the packed
 * lmax = 3 row layout of degree groups 3/5/7).
 *
 * Notation: D = 16 node rows, R = 15 zonal rows, rows 0..2 are degree 1,
 * rows 3..7 degree 2, rows 8..14 degree 3; radial slot s = degree - 1.
 *   coup  (E, 15)     fp32, row-major, contiguous
 *   rad   (E, 3, C)   fp32, row-major, contiguous
 *   out   (N, 16, C)  fp32, row-major, contiguous
 *   g     (N, 16, C)  fp32 cotangent of out (row 0 is never read)
 * Every entry point with an lmax argument also takes the other ladders
 * lmax = 1..5 (an extension of the pages' operator, same definitions):
 * D = (lmax+1)^2, R = D - 1, degree l holding rows [l^2 - 1, (l+1)^2 - 1),
 * coup (E, R), rad (E, lmax, C), out and g (N, D, C).  C = 32 with 16-byte
 * aligned operands takes the vectorised kernels at every lmax (tuned at
 * lmax = 3); every other shape takes per-channel kernels.
 *   forward:  out[n,0,c] = 0,
 *             out[n,1+r,c] = sum over CSR positions j of node n, in order,
 *                            of coup[e,r] * rad[e,s(r),c], e = perm[j]
 *   backward: d_coup[e,r]  = sum_c g[dst[e],1+r,c] * rad[e,s(r),c]
 *             d_rad[e,s,c] = sum over rows r of slot s of g[dst[e],1+r,c] * coup[e,r]
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller.  Inputs are
 *     only read.  Outputs are fully overwritten (the caller need not zero
 *     them).  The library never allocates or frees memory; scratch comes from
 *     the caller's workspace, sized by the matching *_workspace_bytes query.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and is asynchronous: no entry point synchronises the
 *     host.  A status other than ZS_OK means nothing was enqueued, except
 *     ZS_ERR_CUDA, which reports a failed launch (see zs_last_error()).
 *   - E = 0 and N = 0 are valid.  Sizes are limited to E < 2^31 (perm and
 *     row_ptr are int32); all address arithmetic inside is 64-bit.
 *   - Results are bitwise deterministic run to run for the same inputs.
 *   - Destinations outside [0, N) belong to no node (reading of the pages,
 *     which leave them undefined): the CSR build counts them and places them
 *     after all valid edges; the backward gives those edges zero gradients.
 *   - Operands are contiguous row-major arrays (the coupling rows may be
 *     strided through the *_ld entry points).  As on the pages, where the
 *     inputs are flattened to contiguous before they enter the operator, a
 *     caller holding a sliced view of the radial operand makes it
 *     contiguous first; the PyTorch operators over this library do that.
 *   - Any C >= 1 is accepted.  C == 32 with 16-byte aligned float4 operands
 *     (rad and out in the forward; g, rad and d_rad in the backward) takes
 *     the vectorised path; every other case takes a per-channel path with
 *     the same results up to fp32 rounding order.
 */
#ifndef ZS_H_
#define ZS_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ZS_API __attribute__((visibility("default")))
#else
#define ZS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, spelled without the CUDA headers. */
typedef struct CUstream_st* zs_stream_t;

typedef enum zs_status {
    ZS_OK = 0,
    ZS_ERR_INVALID_ARG = 1,  /* null pointer with nonzero size, negative size, E >= 2^31, C < 1, workspace too small */
    ZS_ERR_UNSUPPORTED = 2,  /* lmax outside 1..5 */
    ZS_ERR_CUDA = 3,         /* a CUDA call or launch failed; zs_last_error() has the message */
    ZS_ERR_TIMEOUT = 4       /* a bounded device wait ran out (see zs_check_timeouts) */
} zs_status;

/* Static, human-readable name of a status code. */
ZS_API const char* zs_status_string(int status);

/* Message of the last ZS_ERR_* returned on the calling host thread ("" if none). */
ZS_API const char* zs_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
ZS_API int zs_version(void);

/*
 * Bytes of device workspace zs_build_csr needs for E edges and N nodes
 * (0 when E == 0).  The workspace must be 256-byte aligned.
 */
ZS_API size_t zs_build_csr_workspace_bytes(int64_t E, int32_t N);

/*
 * Stable destination CSR ("stable-sort CSR order", pull request "fused
 * Triton zonal scatter for the GIE head", section "What").
 *   dst            (E,)   int32 destination node of each edge
 *   row_ptr        (N+1,) int32 out: node n owns CSR positions [row_ptr[n], row_ptr[n+1])
 *   perm           (E,)   int32 out: edge id at each CSR position; within a node,
 *                         edge ids ascend (stable); edges with dst outside [0, N)
 *                         fill positions [row_ptr[N], E) in ascending edge order
 *   bad_dst_count  (1,)   int32 out, may be NULL: number of edges with dst outside [0, N)
 *   workspace             device scratch of zs_build_csr_workspace_bytes(E, N) bytes
 * The result is bit-identical to a sequential counting sort.
 */
ZS_API zs_status zs_build_csr(const int32_t* dst, int64_t E, int32_t N,
                       int32_t* row_ptr, int32_t* perm, int32_t* bad_dst_count,
                       void* workspace, size_t workspace_bytes, zs_stream_t stream);

/*
 * Bytes of device workspace zs_forward needs at lmax = 3 (partial sums of
 * nodes whose edges are split across work units, and flags that mark them
 * written).  256-byte alignment required; its contents need not start at
 * zero.
 */
ZS_API size_t zs_forward_workspace_bytes(int64_t E, int32_t N, int32_t C);

/*
 * The same for any ladder lmax = 1..5 (0 for an lmax outside that range);
 * equal to zs_forward_workspace_bytes at lmax = 3.
 */
ZS_API size_t zs_forward_workspace_bytes_lmax(int64_t E, int32_t N, int32_t C, int32_t lmax);

/*
 * Forward zonal scatter (pull request "fused Triton zonal scatter for the
 * GIE head", section "What", forward bullet).
 *   coup (E,15), rad (E,3,C)  inputs, indexed by edge id
 *   row_ptr (N+1,), perm (E,) a CSR as produced by zs_build_csr; positions
 *                             row_ptr[N]..E-1 are ignored
 *   E                         length of perm and number of rows of coup/rad
 *   lmax                      1..5 (else ZS_ERR_UNSUPPORTED); the workspace is
 *                             zs_forward_workspace_bytes_lmax(E, N, C, lmax)
 *   out (N,16,C)              output, fully written: row 0 and the rows of
 *                             nodes without edges are exact zeros
 * Each node's sum is formed in fp32 in a fixed order: CSR order within
 * fixed windows of positions, windows combined in ascending order.
 */
ZS_API zs_status zs_forward(const float* coup, const float* rad,
                     const int32_t* row_ptr, const int32_t* perm,
                     int64_t E, int32_t N, int32_t C, int32_t lmax,
                     float* out, void* workspace, size_t workspace_bytes,
                     zs_stream_t stream);

/*
 * zs_forward with coupling rows coup_ld floats apart (coup_ld >= D-1; row e
 * at coup + e * coup_ld, any 4-byte alignment): for instance the m = 0
 * segment of a packed Wigner band, read in place.  The banded storage of
 * the pull request "banded Wigner-D storage for the fused inference
 * consumers" keeps, per edge, three segments of the (E, 3*D-2) band, and
 * the GIE zonal coupling reads its m = 0 segment (section "What"); the
 * pages print no segment offsets, so the caller passes the pointer to the
 * first zonal row (the degree-1 entries after the degree-0 one) and the
 * band's row length, 3*D-2.  Results are bit-identical to zs_forward on the
 * same values stored contiguously.  Other arguments as zs_forward;
 * ZS_ERR_INVALID_ARG for coup_ld < D-1.
 */
ZS_API zs_status zs_forward_ld(const float* coup, int64_t coup_ld, const float* rad,
                               const int32_t* row_ptr, const int32_t* perm,
                               int64_t E, int32_t N, int32_t C, int32_t lmax,
                               float* out, void* workspace, size_t workspace_bytes, zs_stream_t stream);

/*
 * Forward with the degree normalisation fused in.  The pages apply an
 * inverse-square-root degree normalisation to the operator's output in the
 * traced graph, so that its own cotangent keeps flowing (pull request
 * "fused Triton zonal scatter for the GIE head", section "What", third
 * bullet, and its sequence diagram); here the per-node factor is applied
 * as the node is written, saving a pass over the (N, D, C) output.
 *   node_scale (N,)   per-node factor s[n] (for instance 1/sqrt of a
 *                     degree); any finite or non-finite value
 *   out (N, D, C)     out[n,1+r,c] = s[n] * (the zs_forward value), row 0
 *                     zero; nodes without edges are zero whatever s[n]
 *   out_raw (N, D, C) may be NULL; else also receives the unscaled
 *                     zs_forward result (what zs_backward_scaled needs for
 *                     the scale's gradient)
 * Other arguments, workspace, errors and summation order as zs_forward;
 * out equals zs_forward's result times s[n] rounded once (bitwise).
 */
ZS_API zs_status zs_forward_scaled(const float* coup, const float* rad,
                                   const int32_t* row_ptr, const int32_t* perm, const float* node_scale,
                                   int64_t E, int32_t N, int32_t C, int32_t lmax,
                                   float* out, float* out_raw, void* workspace, size_t workspace_bytes,
                                   zs_stream_t stream);

/*
 * Backward of zs_forward_scaled, edge order: for the cotangent g of the
 * scaled out,
 *   d_coup[e,r]  = s[dst[e]] * (zs_backward's d_coup with the same g)
 *   d_rad[e,l,c] = s[dst[e]] * (zs_backward's d_rad)
 *   d_scale[n]   = sum over rows 1..D-1 and channels of g[n,r,c] * out_raw[n,r,c]
 * node_scale (N,) as given to the forward; out_raw (N, D, C) the forward's
 * unscaled result, needed only when d_scale is not NULL; d_scale (N,) may
 * be NULL.  Each product of a gradient and s is rounded once.  Errors as
 * zs_backward, plus ZS_ERR_INVALID_ARG for a NULL node_scale, or a d_scale
 * without out_raw.  Needs no workspace.
 */
ZS_API zs_status zs_backward_scaled(const float* g, const float* coup, const float* rad, const int32_t* dst,
                                    const float* node_scale, const float* out_raw,
                                    int64_t E, int32_t N, int32_t C, int32_t lmax,
                                    float* d_coup, float* d_rad, float* d_scale, zs_stream_t stream);

/*
 * Backward of the zonal scatter (pull request "fused Triton zonal scatter
 * for the GIE head", section "What", backward bullet): one edge-parallel
 * pass writing both operand gradients.
 *   g (N,16,C)     cotangent of out; row 0 is not read
 *   coup, rad, dst the forward's inputs, indexed by edge id
 *   d_coup (E,15)  output, fully written
 *   d_rad (E,3,C)  output, fully written
 * Edges with dst outside [0, N) get zero gradients.  Needs no workspace.
 */
ZS_API zs_status zs_backward(const float* g, const float* coup, const float* rad,
                      const int32_t* dst, int64_t E, int32_t N, int32_t C, int32_t lmax,
                      float* d_coup, float* d_rad, zs_stream_t stream);

/*
 * zs_backward with coupling rows coup_ld floats apart and coupling-gradient
 * rows d_coup_ld floats apart (both >= D-1, any 4-byte alignment), so that
 * both can live in a packed band's m = 0 segment (see zs_forward_ld); only
 * the D-1 entries of each d_coup row are written.  Bit-identical to
 * zs_backward on contiguous copies.
 */
ZS_API zs_status zs_backward_ld(const float* g, const float* coup, int64_t coup_ld, const float* rad,
                                const int32_t* dst, int64_t E, int32_t N, int32_t C, int32_t lmax,
                                float* d_coup, int64_t d_coup_ld, float* d_rad, zs_stream_t stream);

/*
 * Backward of the zonal scatter with the edges visited in destination (CSR)
 * order: the same d_coup and d_rad as zs_backward, written for every edge,
 * for callers that already hold the forward's CSR.  Each node's cotangent
 * rows g[n] are read once per run of its edges instead of once per edge.
 *   g (N,16,C), coup (E,15), rad (E,3,C)  as for zs_backward
 *   row_ptr (N+1,), perm (E,)             the CSR zs_build_csr returned for
 *                                         the edges' destinations; perm must
 *                                         be a permutation of [0, E)
 *   d_coup (E,15), d_rad (E,3,C)          outputs, fully written; edges at
 *                                         positions >= row_ptr[N] (no node)
 *                                         get zero gradients
 * Needs no workspace.  Gradients agree with zs_backward's to fp32 rounding
 * (each is bitwise reproducible run to run).
 */
ZS_API zs_status zs_backward_csr(const float* g, const float* coup, const float* rad,
                                 const int32_t* row_ptr, const int32_t* perm,
                                 int64_t E, int32_t N, int32_t C, int32_t lmax,
                                 float* d_coup, float* d_rad, zs_stream_t stream);

/*
 * zs_forward without a workspace argument, for callers that cannot allocate
 * device memory: code that must not call cudaMalloc or a caching allocator
 * (for instance inside a region where allocation is forbidden or would
 * synchronise, or a host framework that owns all device memory and passes
 * in only the tensors).  The pages have no counterpart; this is a
 * convenience of this library.
 *   Arguments, results and errors as zs_forward (caller still passes the
 *   inputs and out).  The partial sums zs_forward keeps in its workspace
 *   live instead in one static device array of 4 MiB that every GPU
 *   loading the library holds until the process exits.  The single-kernel
 *   path (C == 32, rad 16-byte aligned, and out 16-byte aligned when
 *   lmax == 3; coup may have any 4-byte alignment) needs about 8 * R * 32
 *   bytes per SM whatever E is (R = (lmax+1)^2 - 1 rows, 3.8 KB at
 *   lmax 3); every other shape needs 8 * R * C + 12 bytes per 256 edges.
 *   A call that would need more returns ZS_ERR_INVALID_ARG and enqueues
 *   nothing.
 *   The first call on each device (and the first after a cudaDeviceReset)
 *   looks up the array's device address with cudaGetSymbolAddress, with
 *   that device current; make that first call before any stream capture.
 *   Every call shares the array: calls whose kernels overlap on the GPU
 *   (other streams, other host threads) race and give wrong results.
 *   Nothing in the array needs to start at zero.
 */
ZS_API zs_status zs_forward_noalloc(const float* coup, const float* rad,
                                    const int32_t* row_ptr, const int32_t* perm,
                                    int64_t E, int32_t N, int32_t C, int32_t lmax,
                                    float* out, zs_stream_t stream);

/*
 * Registers a caller-owned 32-bit word that the kernels set to 1 when a
 * bounded wait runs out (see zs_check_timeouts), so that a caller can see a
 * timeout without synchronising the device: for instance page-locked host
 * memory that the host reads at any time, or device memory that it copies
 * back asynchronously.  The word is only written (never cleared) by the
 * library; the caller clears it.
 *   flag   device memory, or page-locked host memory the device reaches at
 *          the same address (cudaHostAlloc / cudaMallocHost on a system
 *          with unified addressing), 4-byte aligned; NULL unregisters
 * Applies to the current device and to kernels enqueued after the call
 * (a synchronous copy to a device symbol: call it at set-up, not during
 * stream capture).  The word must stay valid until it is unregistered.
 * ZS_ERR_INVALID_ARG for memory the device cannot reach at that address.
 * The pages have no counterpart.
 */
ZS_API zs_status zs_set_timeout_flag(uint32_t* flag);

/*
 * Reads and clears the device-side count of bounded waits that ran out.
 * The kernels that stream operands with asynchronous bulk copies wait for
 * them with an iteration limit; a wait that reaches its limit is counted
 * and the kernel returns instead of hanging the GPU (its outputs are then
 * undefined), and the word registered with zs_set_timeout_flag, if any, is
 * set.  Synchronises the device.  Returns ZS_ERR_TIMEOUT when any
 * wait ran out since the previous call, ZS_OK otherwise.
 */
ZS_API zs_status zs_check_timeouts(void);

/*
 * Self-test of the bounded waits (the pages have no counterpart): enqueues a
 * one-warp kernel that waits on an mbarrier nothing completes, giving up
 * after max_spins tries (1 <= max_spins <= 2^16).  The wait records one
 * timeout, which the next
 * zs_check_timeouts() reports as ZS_ERR_TIMEOUT.  Nothing faults or hangs.
 */
ZS_API zs_status zs_selftest_bounded_wait(uint32_t max_spins, zs_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Training operators of a species-resolved update block: products grouped by
 * a CSR, residual norms with a gate, and the AdamW step.  The pages have no
 * counterpart.  The conventions at the top hold for them too (device
 * pointers, caller-owned memory, asynchronous, bitwise deterministic), except
 * that their operands may be 16-bit, as each dtype argument says; every sum
 * is formed in 32 bits and each result rounded once.
 */
typedef enum zs_dtype {
    ZS_F32 = 0,
    ZS_BF16 = 1,
    ZS_F16 = 2
} zs_dtype;

/*
 * Matrix products grouped by a CSR over rows: with (row_ptr, perm) the CSR
 * zs_build_csr gives for the group of each row (its species, or species and
 * degree), g(i) the group of row i,
 *   y[i,:] = w[g(i)] x[i,:]        y[i,n] = sum_k w[g(i),n,k] * x[i,k]
 * Rows stay in their own order; the gather and the scatter happen inside.
 *   dtype            zs_dtype of x, w and y (one type for all three)
 *   x (M, K)         rows x_ld elements apart (x_ld >= K)
 *   w (G, N, K)      contiguous
 *   row_ptr (G+1,)   group g owns positions [row_ptr[g], row_ptr[g+1])
 *   perm (M,)        row at each position, each row once as zs_build_csr
 *                    gives them; NULL: position p is row p
 *   y (M, N)         rows y_ld elements apart (y_ld >= N), fully written:
 *                    rows at positions >= row_ptr[G] (no group) are zeros
 * M, K and N up to 2^31 - 2^16, K >= 1, N >= 1, G >= 0.  Values outside a
 * row's own group never reach its result.  Sums are in fp32, in a fixed order
 * for given sizes.  Those of the tensor cores, whose additions truncate, come out
 * up to 2^-16 of their terms' magnitudes low for 16-bit operands and about 2^-22
 * for fp32 ones, each of whose terms is known to 2^-24.  An fp32 value that is
 * not finite makes the results that it reaches not finite: NaN, or the infinity
 * that the sum is.
 */
ZS_API zs_status zs_grouped_matmul(int32_t dtype, const void* x, int64_t x_ld, const void* w,
                                   const int32_t* row_ptr, const int32_t* perm,
                                   int64_t M, int32_t K, int32_t N, int32_t G,
                                   void* y, int64_t y_ld, zs_stream_t stream);

/*
 * Gradient of zs_grouped_matmul in x:  dx[i,:] = w[g(i)]^T dy[i,:].
 *   dy (M, N) rows dy_ld apart, dx (M, K) rows dx_ld apart, fully written
 *   (rows of no group are zeros).  Other arguments as above.
 */
ZS_API zs_status zs_grouped_matmul_dx(int32_t dtype, const void* dy, int64_t dy_ld, const void* w,
                                      const int32_t* row_ptr, const int32_t* perm,
                                      int64_t M, int32_t K, int32_t N, int32_t G,
                                      void* dx, int64_t dx_ld, zs_stream_t stream);

/*
 * The two above with a workspace, in which rows that do not start on 16-byte
 * boundaries (odd K or N, views at odd offsets), and 16-bit rows that perm
 * gathers for 1280 columns or more, are laid out anew before the products: up to
 * four times as fast for the former from a few hundred rows on.  Same results.
 *   workspace  zs_grouped_matmul_workspace_bytes(dtype, M, K, N, G) bytes,
 *              256-byte aligned; its contents need not start at zero.  What
 *              does not fit, or NULL, is not used.
 */
ZS_API size_t zs_grouped_matmul_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G);
ZS_API zs_status zs_grouped_matmul_ws(int32_t dtype, const void* x, int64_t x_ld, const void* w,
                                      const int32_t* row_ptr, const int32_t* perm,
                                      int64_t M, int32_t K, int32_t N, int32_t G,
                                      void* y, int64_t y_ld, void* workspace, size_t workspace_bytes,
                                      zs_stream_t stream);
ZS_API zs_status zs_grouped_matmul_dx_ws(int32_t dtype, const void* dy, int64_t dy_ld, const void* w,
                                         const int32_t* row_ptr, const int32_t* perm,
                                         int64_t M, int32_t K, int32_t N, int32_t G,
                                         void* dx, int64_t dx_ld, void* workspace, size_t workspace_bytes,
                                         zs_stream_t stream);

/*
 * Gradient of zs_grouped_matmul in w:  dw[g] = sum over rows i of group g of
 * dy[i,:]^T x[i,:].
 *   dw (G, N, K)  contiguous, of the operands' type, fully written (a group
 *                 without rows gets zeros)
 *   workspace     zs_grouped_matmul_dw_workspace_bytes(dtype, M, K, N, G)
 *                 bytes at least, 256-byte aligned; its contents need not start
 *                 at zero.  Where it has zs_grouped_matmul_dw_copy_bytes() more,
 *                 operands are laid out anew as above (for gathered rows: of 64
 *                 tiles of 128 x 256 weights or more).
 */
ZS_API size_t zs_grouped_matmul_dw_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G);
ZS_API size_t zs_grouped_matmul_dw_copy_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G);
ZS_API zs_status zs_grouped_matmul_dw(int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                                      const int32_t* row_ptr, const int32_t* perm,
                                      int64_t M, int32_t K, int32_t N, int32_t G,
                                      void* dw, void* workspace, size_t workspace_bytes, zs_stream_t stream);

/* Row norms: v / sqrt(mean(v^2) + eps), or the same of v - mean(v). */
typedef enum zs_norm_kind {
    ZS_NORM_RMS = 0,
    ZS_NORM_LAYER = 1
} zs_norm_kind;

/*
 * The norms around a block fused with its gate, residual scale and residual
 * sum: with q = sigmoid(gate) (1 without a gate),
 *   y = x + scale * q * (norm(h) * w_post)      the residual stream
 *   u = norm(y) * w_pre                         the next block's input
 * y enters its norm unrounded.
 *   dtype        zs_dtype of h, x, gate, y and u
 *   h, x (M, C)  rows h_ld, x_ld elements apart
 *   gate         (M, gate_cols), rows gate_ld apart; gate_cols is C (a gate
 *                for each channel), 1 (one for each row) or, with gate NULL, 0
 *   w_post, scale, w_pre (C,)  fp32
 *   y, u (M, C)  contiguous, fully written
 *   stats (M, 4) fp32, may be NULL: mean and 1/root of h, then of y (means 0
 *                for ZS_NORM_RMS); what the backward reads; 16-byte aligned
 * 1 <= C <= 8192 (else ZS_ERR_UNSUPPORTED), eps >= 0.
 */
ZS_API zs_status zs_norm_gate_residual(int32_t dtype, int32_t kind, const void* h, int64_t h_ld,
                                       const void* x, int64_t x_ld, const void* gate, int64_t gate_ld,
                                       int32_t gate_cols, const float* w_post, const float* scale,
                                       const float* w_pre, float eps, int64_t M, int32_t C,
                                       void* y, void* u, float* stats, zs_stream_t stream);

/*
 * Backward of zs_norm_gate_residual for the cotangents dy of y and du of u
 * (either may be NULL: zeros).
 *   dh, dx (M, C)  contiguous; dgate (M, gate_cols) contiguous, NULL without
 *                  a gate; all of the operands' type
 *   dw_post, dscale, dw_pre (C,)  fp32
 *   workspace      zs_norm_gate_residual_backward_workspace_bytes(M, C)
 *                  bytes, 256-byte aligned
 * Every output is fully written (M = 0 gives zero dw_post, dscale, dw_pre).
 */
ZS_API size_t zs_norm_gate_residual_backward_workspace_bytes(int64_t M, int32_t C);
ZS_API zs_status zs_norm_gate_residual_backward(int32_t dtype, int32_t kind, const void* dy, int64_t dy_ld,
                                                const void* du, int64_t du_ld, const void* h, int64_t h_ld,
                                                const void* x, int64_t x_ld, const void* gate, int64_t gate_ld,
                                                int32_t gate_cols, const float* w_post, const float* scale,
                                                const float* w_pre, const float* stats, int64_t M, int32_t C,
                                                void* dh, void* dx, void* dgate, float* dw_post, float* dscale,
                                                float* dw_pre, void* workspace, size_t workspace_bytes,
                                                zs_stream_t stream);

/*
 * One tensor of an AdamW step: numel contiguous elements of each array.
 * With 32-bit states exp_avg and exp_avg_sq are fp32 and the scales unused.
 * With 8-bit states they hold e4m3 codes, with one fp32 scale for each block
 * of 256 elements (the last one may be short): exp_avg the first moment,
 * exp_avg_sq the square root of the second.
 */
typedef struct zs_adamw_tensor {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* exp_avg_scale;
    float* exp_avg_sq_scale;
    int64_t numel;
} zs_adamw_tensor;

typedef struct zs_adamw_hyper {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;   /* 1 for the first step */
} zs_adamw_hyper;

/*
 * One AdamW step over many tensors, in place.  For every element, in fp32
 * with each operation rounded once, in this order:
 *   g = grad * grad_scale
 *   m = beta1 * m + (1 - beta1) * g
 *   v = beta2 * v + (1 - beta2) * (g * g)
 *   p = p * (1 - lr * weight_decay)
 *       - (lr / (1 - beta1^step)) * (m / (sqrt(v) * (1 / sqrt(1 - beta2^step)) + eps))
 * (the constants are formed in 64 bits and rounded once), p rounded to the
 * parameter's type.  8-bit states read m = code * scale, and sqrt(v) = code *
 * scale squared; they are written with scale = top / 448, top the largest
 * finite magnitude in the block, code the e4m3 value nearest to the value
 * times (1 / top) * 448 (ties to even); a positive root is held as at least
 * the smallest positive code, so that a held first moment never meets a zero
 * denominator; a value that is not finite is held as NaN and leaves the rest
 * of its block alone; a block whose top is below 1e-30 is held as zeros.
 *   tensors      HOST array of `count` entries; read before the call returns
 *   dtype        zs_dtype of the parameters and gradients (every tensor)
 *   state_bits   32 or 8 (every tensor)
 *   hyper        host; step >= 1, 0 <= beta < 1, eps >= 0
 *   grad_scale   (1,) fp32 on the device, may be NULL (1): the reciprocal of a
 *                loss scale, a clipping factor
 * The arrays of one call must not overlap.  Tensors of any element alignment;
 * 16-byte aligned ones take wide loads.  Captured in a graph, a call replays with
 * the step, the rates and the addresses of its capture.
 * Rounded to nearest, a code moves only where a step changes its value by more
 * than half the distance to the next code, about 3 to 6 %: with beta2 = 0.999 no
 * root ever falls against the largest of its block, and a first moment may
 * stay some 30 to 60 % off a constant gradient.  A training run with 8-bit
 * states takes zs_adamw_step_seeded.
 */
ZS_API zs_status zs_adamw_step(const zs_adamw_tensor* tensors, int32_t count, int32_t dtype, int32_t state_bits,
                               const zs_adamw_hyper* hyper, const float* grad_scale, zs_stream_t stream);

/*
 * The same step with 8-bit codes rounded at random, up with the probability of
 * the distance to the code below: a held state is its value on average, however
 * little a step changes it (32-bit states: the same as zs_adamw_step).  The
 * random numbers follow from the arguments: with all products and sums modulo
 * 2^64 (key) and 2^32 (x), element i of a tensor, after tensors that fill n
 * chunks of 2048 elements (a last one of each may be short), has c = 2048 n + i and
 *   key = seed ^ (step * 0x9e3779b97f4a7c15)
 *   twice: key = (key ^ key >> 32) * 0xd6e8feb86659fd93;  key = key ^ key >> 32
 *   x = low(c) ^ (low(key) + high(c) * 0x9e3779b9)
 *   x = (x ^ x >> 16) * 0x7feb352d;  x = ((x ^ x >> 15) + high(key)) * 0x846ca68b
 *   x = x ^ x >> 16
 * with low and high 32 bits.  With k the low 16 bits of x for the first moment,
 * the high 16 for the root, and t = |q| + 2^-6 rounded to fp32 where |q| < 2^-6
 * (|q| elsewhere), the code is that of t's bits plus 16 k + 8, cut to their
 * first 12, less what was added (448 at most), with q's sign.
 */
ZS_API zs_status zs_adamw_step_seeded(const zs_adamw_tensor* tensors, int32_t count, int32_t dtype, int32_t state_bits,
                                      const zs_adamw_hyper* hyper, uint64_t seed, const float* grad_scale,
                                      zs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_H_ */
