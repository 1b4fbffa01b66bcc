// Backward of the residual norms (zs_norm.cuh has the formulas and the layout).
#include <initializer_list>

#include "zs_norm.cuh"

namespace zs {

namespace {

#ifndef MOSTB
#define MOSTB 2
#endif
constexpr int kMostB = MOSTB;
constexpr int kSumCols = 32, kSumRows = 16;   // shape of the CTAs that add the CTAs' column sums

template <int E>
constexpr int kMinCtas = E > 8 ? 1 : 2;

template <typename T, int VEC, int NV, bool kEdges, bool kGate>
__global__ void __launch_bounds__(kNormThreads, kMinCtas<VEC * NV>) norm_bwd(const NormArgs a) {
    using Co = NormCols<T, VEC, NV, kEdges>;
    constexpr int E = Co::E;
    __shared__ NormSums sums;
    extern __shared__ float cols[];   // [rows][C]: the row groups' column sums at the end
    int round = 0;
    const NormShape& s = a.s;
    const NormPlace at(s);
    NormLane l{s.tpr, at.lane, s.C, 0};
    struct Row {
        typename Co::Raw h, x, g, dy, du;
        float4 st;
        T gate;
    };
    auto load = [&](Row& w, int64_t r) {
        if (r >= s.M) return;   // threads past the last row only keep the barriers company
        if (a.du.p) Co::load(w.du, a.du, r, s.M, l);
        Co::load(w.h, a.h, r, s.M, l);
        Co::load(w.x, a.x, r, s.M, l);
        if constexpr (kGate) Co::load(w.g, a.gate, r, s.M, l);
        else if (s.gate_cols) w.gate = static_cast<const T*>(a.gate.p)[r * a.gate.ld];
        if (a.dy.p) Co::load(w.dy, a.dy, r, s.M, l);
        w.st = __ldg(a.stats_in + r);
    };
    if (s.cluster > 1) cluster_barrier();   // every CTA of the row runs before another writes to it
    pdl_wait();
    pdl_trigger();
    int64_t r = at.first + at.sub;
    if (kEdges) l.phase = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.h.p) + r * a.h.ld) & 15u) / sizeof(T));
    Row cur = {};
    load(cur, r);
    float pa[E], wr[E], sum_b[E], sum_pre[E];
    Co::columns(pa, l, [&](int c) { return __ldg(a.scale + c) * __ldg(a.w_post + c); });
    Co::columns(wr, l, [&](int c) { return __ldg(a.w_pre + c); });
#pragma unroll
    for (int i = 0; i < E; ++i) sum_b[i] = sum_pre[i] = 0.f;
    // every thread of the CTA goes round as often: the row sums may hold a barrier
    for (int64_t r0 = at.first; r0 < s.M; r0 += at.step, r += at.step) {
        const bool live = r < s.M;
        Row next = {};
        load(next, r + at.step);
        float nh[E], ny[E], q[kGate ? E : 1], d[E];
        Co::open(cur.h, nh, l);
        Co::open(cur.x, ny, l);
        if constexpr (kGate) {
            Co::open(cur.g, q, l);
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = sigmoid(q[i]);
        } else {
            q[0] = s.gate_cols ? sigmoid(to_f32(cur.gate)) : 1.f;
        }
        auto gate = [&](int i) { return q[kGate ? i : 0]; };
#pragma unroll
        for (int i = 0; i < E; ++i) {
            nh[i] = (nh[i] - cur.st.x) * cur.st.y;
            ny[i] = (fmaf(gate(i) * pa[i], nh[i], ny[i]) - cur.st.z) * cur.st.w;
        }
        if (a.du.p) {
            Co::open(cur.du, d, l);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = 0.f;
        }
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (live) sum_pre[i] = fmaf(d[i], ny[i], sum_pre[i]);
            d[i] *= wr[i];
            m[0] = fmaf(d[i], ny[i], m[0]);   // d is zero outside the row
            m[1] += d[i];
        }
        row_sum(m, s, sums, round);
        const float dn = -m[0] * s.inv_c, dm = s.layer ? -m[1] * s.inv_c : 0.f;
        float dx[E];
        if (a.dy.p) {
            Co::open(cur.dy, dx, l);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) dx[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) dx[i] = fmaf(cur.st.w, fmaf(dn, ny[i], d[i] + dm), dx[i]);
        if (live) Co::store(static_cast<T*>(a.out1) + r * s.C, dx, l);
        Co::clear_outside(dx, l);
        float b[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dx[i] *= gate(i);                       // from here dx q
            ny[i] = dx[i] * nh[i];                  // a row's part of B
            if (live) sum_b[i] += ny[i];
            d[i] = dx[i] * pa[i];
            b[0] = fmaf(d[i], nh[i], b[0]);
            b[1] += d[i];
            if constexpr (kGate) ny[i] *= pa[i] * (1.f - q[i]);   // the gate's gradient
        }
        row_sum(b, s, sums, round);
        const float hn = -b[0] * s.inv_c, hm = s.layer ? -b[1] * s.inv_c : 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = cur.st.y * fmaf(hn, nh[i], d[i] + hm);
        if (live) {
            Co::store(static_cast<T*>(a.out0) + r * s.C, d, l);
            if constexpr (kGate) Co::store(static_cast<T*>(a.out2) + r * s.C, ny, l);
            else if (s.gate_cols && l.lane == 0) static_cast<T*>(a.out2)[r] = from_f32<T>(b[0] * (1.f - q[0]));
        }
        cur = next;
    }
    // the group's column sums: its rows' (which may be at other phases) added in order
    float* mine = a.partial + at.group * 2 * s.C;
    if (at.rows == 1) {
        Co::for_columns(l, [&](int i, int c) {
            mine[c] = sum_b[i];
            mine[s.C + c] = sum_pre[i];
        });
    } else {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (w) __syncthreads();
            Co::for_columns(l, [&](int i, int c) { cols[at.sub * s.C + c] = w ? sum_pre[i] : sum_b[i]; });
            __syncthreads();
            for (int c = threadIdx.x; c < s.C; c += blockDim.x) {
                float total = cols[c];
                for (int o = 1; o < at.rows; ++o) total += cols[o * s.C + c];
                mine[w * s.C + c] = total;
            }
        }
    }
    if (s.cluster > 1) cluster_barrier();   // no CTA leaves while another may write to it
}

// The gradients of the parameters from the CTAs' column sums, added in order:
// 16 threads a column, then their sums in order.
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_column_sums(const NormArgs a, int ctas) {
    __shared__ float part[kSumRows][kSumCols];
    const int j = threadIdx.x % kSumCols, k = threadIdx.x / kSumCols, C = a.s.C;
    const int col = blockIdx.x * kSumCols + j;   // of 2 C
    pdl_wait();
    pdl_trigger();
    float v = 0.f;
    if (col < 2 * C)
#pragma unroll 8
        for (int i = k; i < ctas; i += kSumRows) v += __ldg(a.partial + (int64_t)i * 2 * C + col);
    part[k][j] = v;
    __syncthreads();
    if (k == 0 && col < 2 * C) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) v += part[i][j];
        if (col < C) {
            a.dw_post[col] = __ldg(a.scale + col) * v;
            a.dscale[col] = __ldg(a.w_post + col) * v;
        } else {
            a.dw_pre[col - C] = v;
        }
    }
}

template <typename T, int VEC, int NV, bool kEdges>
zs_status launch_bwd(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    const char* fn = "zs_norm_gate_residual_backward";
    const int groups = norm_groups(a.s.M, p.rows, imin(kNormCtas, num_sms() * kMinCtas<VEC * NV>) / p.cluster);
    if (groups > 0) {
        const size_t smem = p.rows > 1 ? (size_t)p.rows * a.s.C * 4 : 0;
        if (a.s.gate_cols > 1) norm_launch(norm_bwd<T, VEC, NV, kEdges, true>, groups, p, smem, s, a);
        else norm_launch(norm_bwd<T, VEC, NV, kEdges, false>, groups, p, smem, s, a);
        if (zs_status st = check_launch(fn)) return st;
    }
    launch(norm_column_sums, dim3((2 * a.s.C + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumRows), 0, s, a, groups);
    return check_launch(fn);
}

template <typename T, bool kEdges>
zs_status dispatch_wide(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (p.nv == 1) return launch_bwd<T, V, 1, kEdges>(p, a, s);
    return launch_bwd<T, V, 2, kEdges>(p, a, s);
}

// Operands at different phases: element by element.
template <typename T>
zs_status launch_single(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    if (p.nv <= 2) return launch_bwd<T, 1, 2, false>(p, a, s);
    return launch_bwd<T, 1, 16, false>(p, a, s);
}

template <typename T>
zs_status dispatch(NormArgs& a, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const int64_t C = a.s.C;
    const bool full = a.s.gate_cols > 1;
    const NormAccess w = norm_access<T>(a.s.C, {a.h, a.x, a.dy, a.du, full ? a.gate : NormView{nullptr, 0}, {a.out0, C},
                                                {a.out1, C}, {full ? a.out2 : nullptr, C}});
    const NormPlan p = w.wide ? norm_plan(a.s.C, V, w.edges, kMostB) : norm_plan(a.s.C, 1, false, 16);
    a.s.tpr = p.tpr;
    a.s.cluster = p.cluster;
    if (!w.wide) return launch_single<T>(p, a, s);
    return w.edges ? dispatch_wide<T, true>(p, a, s) : dispatch_wide<T, false>(p, a, s);
}

}  // namespace

zs_status norm_backward(int32_t dtype, NormArgs& a, cudaStream_t s) {
    switch (dtype) {
        case ZS_F32: return dispatch<float>(a, s);
        case ZS_BF16: return dispatch<__nv_bfloat16>(a, s);
        default: return dispatch<__half>(a, s);
    }
}

}  // namespace zs
