// Forward of the residual norms (zs_norm.cuh has the formulas and the layout).
#include <initializer_list>

#include "zs_norm.cuh"

namespace zs {

namespace {

template <int E>
constexpr int kMinCtas = E > 8 ? 2 : 3;

// Mean (layer norm) and 1/root of a row's values: the mean first, then the
// centred squares, both over the registers.  v is zero outside the row.
template <typename Co, int E>
__device__ __forceinline__ float2 row_stats(const float (&v)[E], const NormShape& s, const NormLane& l, NormSums& sums, int& round) {
    float a[1] = {0.f};
    float mean = 0.f;
    if (s.layer) {
#pragma unroll
        for (int i = 0; i < E; ++i) a[0] += v[i];
        row_sum(a, s, sums, round);
        mean = a[0] * s.inv_c;
        a[0] = 0.f;
        float d[E];
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = v[i] - mean;
        Co::clear_outside(d, l);
#pragma unroll
        for (int i = 0; i < E; ++i) a[0] = fmaf(d[i], d[i], a[0]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) a[0] = fmaf(v[i], v[i], a[0]);
    }
    row_sum(a, s, sums, round);
    return make_float2(mean, rsqrtf(fmaf(a[0], s.inv_c, s.eps)));
}

template <typename T, int VEC, int NV, bool kEdges, bool kGate>
__global__ void __launch_bounds__(kNormThreads, kMinCtas<VEC * NV>) norm_fwd(const NormArgs a) {
    using Co = NormCols<T, VEC, NV, kEdges>;
    constexpr int E = Co::E;
    __shared__ NormSums sums;
    int round = 0;
    const NormShape& s = a.s;
    const NormPlace at(s);
    NormLane l{s.tpr, at.lane, s.C, 0};
    struct Row {
        typename Co::Raw h, x, g;
        T gate;
    };
    auto load = [&](Row& w, int64_t r) {
        if (r >= s.M) return;   // threads past the last row only keep the barriers company
        Co::load(w.h, a.h, r, s.M, l);
        Co::load(w.x, a.x, r, s.M, l);
        if constexpr (kGate) Co::load(w.g, a.gate, r, s.M, l);
        else if (s.gate_cols) w.gate = static_cast<const T*>(a.gate.p)[r * a.gate.ld];
    };
    if (s.cluster > 1) cluster_barrier();   // every CTA of the row runs before another writes to it
    pdl_wait();
    pdl_trigger();
    int64_t r = at.first + at.sub;
    if (kEdges) l.phase = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.h.p) + r * a.h.ld) & 15u) / sizeof(T));
    Row cur = {};
    load(cur, r);
    float pa[E], wr[E];
    Co::columns(pa, l, [&](int c) { return __ldg(a.scale + c) * __ldg(a.w_post + c); });
    Co::columns(wr, l, [&](int c) { return __ldg(a.w_pre + c); });
    // every thread of the CTA goes round as often: the row sums may hold a barrier
    for (int64_t r0 = at.first; r0 < s.M; r0 += at.step, r += at.step) {
        Row next = {};
        load(next, r + at.step);
        float v[E], yv[E];
        Co::open(cur.h, v, l);
        const float2 hs = row_stats<Co>(v, s, l, sums, round);
        Co::open(cur.x, yv, l);
        if constexpr (kGate) {
            float z[E];
            Co::open(cur.g, z, l);
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = fmaf(sigmoid(z[i]) * pa[i], (v[i] - hs.x) * hs.y, yv[i]);
        } else {
            const float q = s.gate_cols ? sigmoid(to_f32(cur.gate)) : 1.f;
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = fmaf(q * pa[i], (v[i] - hs.x) * hs.y, yv[i]);
        }
        const float2 ys = row_stats<Co>(yv, s, l, sums, round);
        if (r < s.M) {
            Co::store(static_cast<T*>(a.out0) + r * s.C, yv, l);
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = (yv[i] - ys.x) * ys.y * wr[i];
            Co::store(static_cast<T*>(a.out1) + r * s.C, yv, l);
            if (a.stats_out && l.lane == 0) a.stats_out[r] = make_float4(hs.x, hs.y, ys.x, ys.y);
        }
        cur = next;
    }
    if (s.cluster > 1) cluster_barrier();   // no CTA leaves while another may write to it
}

template <typename T, int VEC, int NV, bool kEdges>
zs_status launch_fwd(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    const int groups = norm_groups(a.s.M, p.rows, num_sms() * kMinCtas<VEC * NV> / p.cluster);
    if (a.s.gate_cols > 1) norm_launch(norm_fwd<T, VEC, NV, kEdges, true>, groups, p, 0, s, a);
    else norm_launch(norm_fwd<T, VEC, NV, kEdges, false>, groups, p, 0, s, a);
    return check_launch("zs_norm_gate_residual");
}

template <typename T, bool kEdges>
zs_status dispatch_wide(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (p.nv == 1) return launch_fwd<T, V, 1, kEdges>(p, a, s);
    return launch_fwd<T, V, 2, kEdges>(p, a, s);
}

// Operands at different phases: element by element.
template <typename T>
zs_status launch_single(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    if (p.nv <= 2) return launch_fwd<T, 1, 2, false>(p, a, s);
    return launch_fwd<T, 1, 16, false>(p, a, s);
}

template <typename T>
zs_status dispatch(NormArgs& a, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const int64_t C = a.s.C;
    const NormAccess w = norm_access<T>(a.s.C, {a.h, a.x, a.s.gate_cols > 1 ? a.gate : NormView{nullptr, 0}, {a.out0, C}, {a.out1, C}});
    const NormPlan p = w.wide ? norm_plan(a.s.C, V, w.edges, 2) : norm_plan(a.s.C, 1, false, 16);
    a.s.tpr = p.tpr;
    a.s.cluster = p.cluster;
    if (!w.wide) return launch_single<T>(p, a, s);
    return w.edges ? dispatch_wide<T, true>(p, a, s) : dispatch_wide<T, false>(p, a, s);
}

}  // namespace

zs_status norm_forward(int32_t dtype, NormArgs& a, cudaStream_t s) {
    switch (dtype) {
        case ZS_F32: return dispatch<float>(a, s);
        case ZS_BF16: return dispatch<__nv_bfloat16>(a, s);
        default: return dispatch<__half>(a, s);
    }
}

}  // namespace zs
