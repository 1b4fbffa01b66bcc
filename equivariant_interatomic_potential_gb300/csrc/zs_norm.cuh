// The norms around a block fused with its gate, residual scale and residual
// sum, and their backward:
//   nh = norm(h), q = sigmoid(gate), a = scale * w_post
//   y = x + q a nh,  ny = norm(y),  u = ny * w_pre
// and for the cotangents dy, du
//   dx = dy + norm'(du * w_pre; ny, ry),  dh = norm'(dx q a; nh, rh)
//   dgate = dx q a nh (1 - q)
//   dw_pre = sum_rows du ny, and with B = sum_rows dx q nh:
//   dw_post = scale * B, dscale = w_post * B
// with norm'(d; n, r) = r (d - mean(d n) n), minus r mean(d) for the layer
// norm.  The backward forms y again from x, h and the gate (as many bytes as
// reading y, and unrounded), and keeps only four floats a row.
//
// Bound by HBM.  A row lives in the registers of 8 to 256 threads, or of a
// cluster of CTAs that exchange their sums through distributed shared memory,
// each thread holding up to NV pieces of VEC elements, so that every operand
// is read once.  Rows go round the CTAs of a persistent grid, whose threads
// keep the parameters of their columns, and in the backward the running
// column sums, in registers; the pieces of the next rows are on their way
// into shared memory meanwhile, each thread's own ones into slots that it
// alone reads, so that no barrier stands between the copy and its use.
//
// Rows that do not start on 16-byte boundaries (odd channel counts) are still
// read in 16-byte pieces of memory: a row's first and last piece bring some of
// its neighbours' elements along, which count as zeros (at the two ends of
// the matrix they go element by element, as they always do when stored).  The distance `phase` of a row's start past a
// boundary repeats every VEC rows, so a thread that steps by a multiple of
// VEC rows keeps its columns.  That needs all operands to be at the same
// phase; where they are not (views at odd offsets), VEC is 1.
#pragma once

#include <initializer_list>

#include "zs_tma.cuh"
#include "zs_types.cuh"

namespace zs {

constexpr int kNormMaxC = 8192;
constexpr int kNormThreads = 256;     // of a CTA, at most
constexpr int kNormWideThreads = 384; // of a CTA of the backward with 16 elements a thread: one CTA an SM, 168 registers
constexpr int kNormWarps = kNormWideThreads / 32;
constexpr int kNormCluster = 8;       // CTAs that share a row, at most
constexpr int kNormCtas = 608;        // of the backward, at most: rows of the partial column sums

struct NormShape {
    int64_t M;
    int32_t C;
    int32_t tpr;        // threads that hold a row: 8, 16, or a multiple of 32
    int32_t cluster;    // CTAs that hold a row (1: a CTA holds one or more rows)
    int32_t gate_cols;  // 0, 1 or C
    int32_t layer;      // subtract the mean
    float eps, inv_c;
};

struct NormView {
    const void* p;
    int64_t ld;
};

struct NormArgs {
    NormShape s;
    NormView dy, du, h, x, gate;
    const float *w_post, *scale, *w_pre;
    const float4* stats_in;
    void *out0, *out1, *out2;   // y, u  |  dh, dx, dgate
    float4* stats_out;
    float *dw_post, *dscale, *dw_pre, *partial;
};

// How a thread's columns are laid out: piece k covers the VEC columns from
// (k * tpr + lane) * VEC - phase on.
struct NormLane {
    int tpr, lane, C, phase;
};

template <typename T, int VEC, int NV, bool kEdges>
struct NormCols {
    static constexpr int E = VEC * NV;
    static_assert(VEC == 1 || VEC == kVec<T>, "whole 16-byte pieces or single elements");

    static __device__ __forceinline__ int start(const NormLane& l, int k) {
        return (k * l.tpr + l.lane) * VEC - (kEdges ? l.phase : 0);
    }
    static __device__ __forceinline__ bool whole(const NormLane& l, int c0) {
        return !kEdges || (c0 >= 0 && c0 + VEC <= l.C);
    }
    // f(i, c) for this thread's columns c of the row, element i of its E
    template <typename F>
    static __device__ __forceinline__ void for_columns(const NormLane& l, F&& f) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = start(l, k);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (kEdges ? (unsigned)(c0 + i) < (unsigned)l.C : c0 < l.C) f(k * VEC + i, c0 + i);
        }
    }
    template <typename F>
    static __device__ __forceinline__ void columns(float (&v)[E], const NormLane& l, F&& f) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = 0.f;
        for_columns(l, [&](int i, int c) { v[i] = f(c); });
    }
    // Zero outside the row.
    static __device__ __forceinline__ void clear_outside(float (&v)[E], const NormLane& l) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = start(l, k);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (!(kEdges ? (unsigned)(c0 + i) < (unsigned)l.C : c0 < l.C)) v[k * VEC + i] = 0.f;
        }
    }
    static __device__ __forceinline__ void store(T* row, const float (&f)[E], const NormLane& l) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = start(l, k);
            if (c0 >= l.C) continue;
            if constexpr (VEC == 1) {
                row[c0] = from_f32<T>(f[k]);
            } else {
                float q[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[i] = f[k * VEC + i];
                if (whole(l, c0)) {
                    st_piece(row + c0, pack<T>(q));
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if ((unsigned)(c0 + i) < (unsigned)l.C) row[c0 + i] = from_f32<T>(q[i]);
                }
            }
        }
    }
};

// The rows on their way: S stages of NA operands, NV pieces each, in shared
// memory; a piece of this thread lies `stride` (a slot for each thread of the
// CTA) after the one before.
template <typename T, int VEC, int NV, int NA, bool kEdges, int S>
struct NormRing {
    using Co = NormCols<T, VEC, NV, kEdges>;
    static constexpr int kSlot = VEC == 1 ? 4 : 16;
    unsigned char* mine;    // this thread's first slot
    uint32_t mine_s;        // its shared address
    uint32_t stride;
    uint4 mask[kEdges ? NV : 1];

    __device__ __forceinline__ void init(unsigned char* smem) {
        mine = smem + threadIdx.x * kSlot;
        mine_s = (uint32_t)__cvta_generic_to_shared(mine);
        stride = blockDim.x * kSlot;
        // pieces outside the row are never copied: they stay zero
        for (int i = 0; i < S * NA * NV; ++i) {
            if constexpr (VEC == 1) *reinterpret_cast<uint32_t*>(mine + i * stride) = 0;
            else *reinterpret_cast<uint4*>(mine + i * stride) = make_uint4(0, 0, 0, 0);
        }
    }
    // Row r of the M rows of v on its way into a stage.
    __device__ __forceinline__ void issue(int stage, int a, const NormView& v, int64_t r, int64_t M, const NormLane& l) {
        const T* row = static_cast<const T*>(v.p) + r * v.ld;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = Co::start(l, k);
            if (c0 >= l.C) continue;
            const uint32_t slot = ((stage * NA + a) * NV + k) * stride;
            if constexpr (VEC == 1) {
                *reinterpret_cast<T*>(mine + slot) = row[c0];
            } else if (Co::whole(l, c0) || (r * v.ld + c0 >= 0 && c0 + VEC <= (M - 1 - r) * v.ld + l.C)) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(mine_s + slot), "l"(row + c0) : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if ((unsigned)(c0 + i) < (unsigned)l.C) *reinterpret_cast<T*>(mine + slot + i * sizeof(T)) = row[c0 + i];
            }
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // All but the last S - 1 groups have landed.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" :: "n"(S - 1) : "memory"); }
    static __device__ __forceinline__ void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }

    // Which bits of this thread's pieces are the row's (the phase is set).
    __device__ __forceinline__ void cut(const NormLane& l) {
        if constexpr (kEdges) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c0 = Co::start(l, k);
                uint32_t* m = &mask[k].x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        m[j] = (unsigned)(c0 + j) < (unsigned)l.C ? 0xffffffffu : 0u;
                    } else {
                        m[j] = ((unsigned)(c0 + 2 * j) < (unsigned)l.C ? 0xffffu : 0u) |
                               ((unsigned)(c0 + 2 * j + 1) < (unsigned)l.C ? 0xffff0000u : 0u);
                    }
                }
            }
        }
    }
    // The elements of operand a in a stage; a neighbour's count as zeros.
    __device__ __forceinline__ void open(int stage, int a, float (&f)[Co::E]) const {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const unsigned char* slot = mine + ((stage * NA + a) * NV + k) * stride;
            if constexpr (VEC == 1) {
                f[k] = to_f32(*reinterpret_cast<const T*>(slot));
            } else {
                float q[VEC];
                uint4 raw = *reinterpret_cast<const uint4*>(slot);
                if constexpr (kEdges) raw = make_uint4(raw.x & mask[k].x, raw.y & mask[k].y, raw.z & mask[k].z, raw.w & mask[k].w);
                unpack<T>(raw, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[k * VEC + i] = q[i];
            }
        }
    }
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums over the threads of a row.  Rows of up to 32 threads stay within a
// warp.  Wider ones go through shared memory: `red` holds two rounds of a
// float4 for each warp of each CTA of the row, taken in turn, so that one
// barrier a round is enough: who writes a round's slots again has passed the
// barrier of the round between.  Every thread adds them in the same order.
// Between the CTAs of a cluster the parts travel as asynchronous stores that
// count on the receiver's mbarrier (a cluster barrier would also wait for the
// rows' results to reach L2).
struct NormSums {
    float4 red[2][kNormCluster * kNormWarps];
    uint64_t bars[2];
    // Thread 0, before the first barrier of the CTA and the cluster.
    __device__ __forceinline__ void begin() {
        mbar_init(smem_u32(&bars[0]), 1);
        mbar_init(smem_u32(&bars[1]), 1);
        mbar_fence_init();
    }
};
template <int NQ>
__device__ __forceinline__ void row_sum(float (&q)[NQ], const NormShape& s, NormSums& sums, int& round) {
    static_assert(NQ <= 4, "a float4 per warp");
    const int lim = s.tpr < 32 ? s.tpr : 32;
    for (int o = lim >> 1; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) q[i] += __shfl_xor_sync(0xffffffffu, q[i], o);
    }
    if (s.tpr <= 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per_row = s.tpr >> 5;
    float4* slot = sums.red[round & 1];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float* ve = &v.x;
#pragma unroll
    for (int i = 0; i < NQ; ++i) ve[i] = q[i];
    int first;
    if (s.cluster == 1) {
        first = warp / per_row * per_row;
        if (lane == 0) slot[warp] = v;
        __syncthreads();
    } else {
        first = 0;
        uint32_t rank;
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        const uint32_t bar = smem_u32(&sums.bars[round & 1]);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, per_row * 16);
        if (lane < s.cluster) {   // lane i sends this warp's part to CTA i
            uint32_t there, bar_there;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(slot + rank * (blockDim.x >> 5) + warp)), "r"(lane));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar_there) : "r"(bar), "r"(lane));
            asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                         :: "r"(there), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar_there) : "memory");
        }
        mbar_wait(bar, (uint32_t)(round >> 1) & 1);
        __syncwarp();
    }
    ++round;
#pragma unroll
    for (int i = 0; i < NQ; ++i) q[i] = 0.f;
    for (int w = 0; w < per_row; ++w) {
        const float4 p = slot[first + w];
        const float* pe = &p.x;
#pragma unroll
        for (int i = 0; i < NQ; ++i) q[i] += pe[i];
    }
}

// Where a thread stands: its row group within the CTA, and the persistent
// grid's step.
struct NormPlace {
    int sub, rows;
    int64_t first, step;
    int lane;
    int64_t group;    // of the grid: CTA or cluster
    __device__ __forceinline__ explicit NormPlace(const NormShape& s) {
        if (s.cluster == 1) {
            sub = threadIdx.x / s.tpr;
            rows = blockDim.x / s.tpr;
            lane = threadIdx.x - sub * s.tpr;
            group = blockIdx.x;
            step = (int64_t)gridDim.x * rows;
        } else {
            sub = 0;
            rows = 1;
            lane = blockIdx.x % s.cluster * blockDim.x + threadIdx.x;
            group = blockIdx.x / s.cluster;
            step = gridDim.x / s.cluster;
        }
        first = group * rows;
    }
};

// A gate of a whole row.
__device__ __forceinline__ float sigmoid(float z) { return __frcp_rn(1.f + expf(-z)); }
// A gate of one element.  In 16 bits (half an ulp 2^-12 or more of what the
// result is rounded to) known to about |z| 2^-24 of itself at z < 0 and better
// at z > 0, in a quarter of the instructions (4097 x 1031 fp16: forward 25 ->
// 19 us, backward 38 -> 34).  In fp32 -z log2(e) is formed in two parts, of
// which the second one multiplies the power of two by 1 + part ln(2), so that
// the error stays at a few ulps whatever z (65536 x 512 fp32: forward 120 us,
// backward 208; one part 121 and 208, with the functions of a row's gate 138
// and 252).  Beyond +-100, where the gate is 1 or 0, z does not grow: infinities.
template <typename T>
__device__ __forceinline__ float element_sigmoid(float z) {
    if constexpr (sizeof(T) == 4) {
        constexpr float kLog2E = 1.4426950408889634f, kRest = 1.4426950408889634 - (double)kLog2E;
        float e, q;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(z), "f"(100.f));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(z), "f"(-100.f));
        const float t = -z * kLog2E, rest = fmaf(-z, kRest, fmaf(-z, kLog2E, -t));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
        e *= fmaf(rest, 0.6931471805599453f, 1.f);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));
        return q;
    } else {
        return __fdividef(1.f, 1.f + __expf(-z));
    }
}

// How a row is spread: over as many threads as need nv pieces each, with the
// largest nv up to `most` unless a smaller one takes a tenth fewer slots.
constexpr int norm_threads(int elements, bool backward) { return backward && elements > 8 ? kNormWideThreads : kNormThreads; }
struct NormPlan {
    int nv, tpr, cluster, threads, rows;
};
inline NormPlan norm_plan(int32_t C, int vec, bool edges, int most, bool backward) {
    const int pieces = (C + (edges ? vec - 1 : 0) + vec - 1) / vec;   // a phase may add one
    NormPlan best = {};
    int least = 0;
    for (int nv = most; nv >= 1; nv /= 2) {
        NormPlan p;
        p.nv = nv;
        int t = (pieces + nv - 1) / nv;
        const int threads = norm_threads(vec * nv, backward);
        p.cluster = (t + threads - 1) / threads;
        if (p.cluster > kNormCluster) continue;
        if (t <= 32) {
            p.tpr = t <= 8 ? 8 : t <= 16 ? 16 : 32;
        } else {
            t = (t + p.cluster - 1) / p.cluster;
            p.tpr = p.cluster * ((t + 31) / 32 * 32);
        }
        p.rows = p.cluster > 1 ? 1 : threads / p.tpr;
        p.threads = p.cluster > 1 ? p.tpr / p.cluster : p.rows * p.tpr;
        if (least == 0 || p.tpr * nv * 10 < least * 9) best = p, least = p.tpr * nv;
    }
    return least || most >= 4 ? best : norm_plan(C, vec, edges, 2 * most, backward);   // the row takes more pieces a thread
}
// Groups of rows (CTAs, or clusters) for M rows, `most` at most: a multiple of
// 8 where a group takes several rounds, so that its phase stays.
inline int norm_groups(int64_t M, int rows, int most) {
    const int64_t need = (M + rows - 1) / rows;
    return (int)(need <= most ? need : imax(8, most / 8 * 8));
}

template <typename K>
inline void norm_launch(K kernel, int groups, const NormPlan& p, size_t smem, cudaStream_t s, const NormArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(groups * p.cluster);
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kernel, a);
}

// 16-byte pieces can be used (whole rows, or all operands at one phase) for
// these (pointer, row stride) pairs; NULLs are skipped.
struct NormAccess {
    bool wide, edges;
};
template <typename T>
NormAccess norm_access(int32_t C, std::initializer_list<NormView> views) {
    NormAccess a{true, C % kVec<T> != 0};
    int64_t at = -1, step = -1;
    for (const NormView& v : views) {
        if (!v.p) continue;
        const int64_t x = (int64_t)(reinterpret_cast<uintptr_t>(v.p) & 15u), y = v.ld * (int64_t)sizeof(T) & 15;
        if (at < 0) at = x, step = y;
        if (x != at || y != step) a.wide = false;
        if (x != 0 || y != 0) a.edges = true;
    }
    return a;
}

template <typename T>
zs_status norm_forward(NormArgs& a, cudaStream_t s);
template <typename T>
zs_status norm_backward(NormArgs& a, cudaStream_t s);

}  // namespace zs
