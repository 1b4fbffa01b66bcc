// Kernels of the residual norms (zs_norm.cuh has the formulas and the layout),
// instantiated for one element type in each of zs_norm_f32.cu, zs_norm_bf16.cu
// and zs_norm_f16.cu.
#pragma once

#include "zs_norm.cuh"

namespace zs {

namespace {

// CTAs of norm_threads() an SM holds, which sets the registers a thread may
// take, and stages of the rows on their way.
template <int E>
constexpr int kFwdCtas = E > 8 ? 2 : 3;
template <int E>
constexpr int kBwdCtas = E > 8 ? 1 : 2;
constexpr int kFwdStages = 4;
template <int E>
constexpr int kBwdStages = E > 8 ? 3 : 4;

// Mean (kLayer) and 1/root of a row's values: the mean first, then the
// centred squares, both over the registers.  v is zero outside the row.
template <typename Co, bool kLayer, int E>
__device__ __forceinline__ float2 row_stats(const float (&v)[E], const NormShape& s, const NormLane& l, NormSums& sums, int& round) {
    float a[1] = {0.f};
    float mean = 0.f;
    if constexpr (kLayer) {
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
template <bool kLayer>
__device__ __forceinline__ float centred(float v, float mean) { return kLayer ? v - mean : v; }

template <typename T, int VEC, int NV, bool kEdges, bool kGate, bool kLayer>
__global__ void __launch_bounds__(kNormThreads, kFwdCtas<VEC * NV>) norm_fwd(const NormArgs a) {
    using Co = NormCols<T, VEC, NV, kEdges>;
    constexpr int E = Co::E, NA = kGate ? 3 : 2;
    __shared__ NormSums sums;
    extern __shared__ __align__(16) unsigned char smem[];
    int round = 0;
    const NormShape& s = a.s;
    const NormPlace at(s);
    NormLane l{s.tpr, at.lane, s.C, 0};
    constexpr int S = kFwdStages;
    NormRing<T, VEC, NV, NA, kEdges, S> ring;
    ring.init(smem);
    if (threadIdx.x == 0) sums.begin();
    if (s.cluster > 1) cluster_barrier();   // every CTA of the row runs before another writes to it
    pdl_wait();
    pdl_trigger();
    int64_t r = at.first + at.sub, ahead = r;
    if (kEdges) l.phase = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.h.p) + r * a.h.ld) & 15u) / sizeof(T));
    ring.cut(l);
    auto issue = [&](int stage) {
        if (ahead < s.M) {
            ring.issue(stage, 0, a.h, ahead, s.M, l);
            ring.issue(stage, 1, a.x, ahead, s.M, l);
            if constexpr (kGate) ring.issue(stage, 2, a.gate, ahead, s.M, l);
        }
        ring.commit();
        ahead += at.step;
    };
    auto gate_of = [&](int64_t row) {
        return !kGate && s.gate_cols && row < s.M ? static_cast<const T*>(a.gate.p)[row * a.gate.ld] : from_f32<T>(0.f);
    };
    for (int i = 0; i < S - 1; ++i) issue(i);
    T gate = gate_of(r);
    float pa[E], wr[E];
    Co::columns(pa, l, [&](int c) { return __ldg(a.scale + c) * __ldg(a.w_post + c); });
    Co::columns(wr, l, [&](int c) { return __ldg(a.w_pre + c); });
    int stage = 0;
    // every thread of the CTA goes round as often: the row sums may hold a barrier
    for (int64_t r0 = at.first; r0 < s.M; r0 += at.step, r += at.step) {
        issue((stage + S - 1) % S);
        const T gate_next = gate_of(r + at.step);
        ring.wait();
        float v[E], yv[E];
        ring.open(stage, 0, v);
        const float2 hs = row_stats<Co, kLayer>(v, s, l, sums, round);
        ring.open(stage, 1, yv);
        if constexpr (kGate) {
            float z[E];
            ring.open(stage, 2, z);
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = fmaf(element_sigmoid<T>(z[i]) * pa[i], centred<kLayer>(v[i], hs.x) * hs.y, yv[i]);
        } else {
            const float q = s.gate_cols ? sigmoid(to_f32(gate)) : 1.f;
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = fmaf(q * pa[i], centred<kLayer>(v[i], hs.x) * hs.y, yv[i]);
        }
        const float2 ys = row_stats<Co, kLayer>(yv, s, l, sums, round);
        if (r < s.M) {
            Co::store(static_cast<T*>(a.out0) + r * s.C, yv, l);
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = centred<kLayer>(yv[i], ys.x) * ys.y * wr[i];
            Co::store(static_cast<T*>(a.out1) + r * s.C, yv, l);
            if (a.stats_out && l.lane == 0) a.stats_out[r] = make_float4(hs.x, hs.y, ys.x, ys.y);
        }
        gate = gate_next;
        stage = (stage + 1) % S;
    }
    ring.drain();
    if (s.cluster > 1) cluster_barrier();   // no CTA leaves while another may write to it
}

template <typename T, int VEC, int NV, bool kEdges, bool kGate, bool kLayer>
__global__ void __launch_bounds__(norm_threads(VEC * NV, true), kBwdCtas<VEC * NV>) norm_bwd(const NormArgs a) {
    using Co = NormCols<T, VEC, NV, kEdges>;
    constexpr int E = Co::E, NA = kGate ? 5 : 4;
    __shared__ NormSums sums;
    extern __shared__ __align__(16) unsigned char smem[];   // the ring, and at the end the row groups' column sums
    int round = 0;
    const NormShape& s = a.s;
    const NormPlace at(s);
    NormLane l{s.tpr, at.lane, s.C, 0};
    constexpr int S = kBwdStages<E>;
    NormRing<T, VEC, NV, NA, kEdges, S> ring;
    ring.init(smem);
    if (threadIdx.x == 0) sums.begin();
    if (s.cluster > 1) cluster_barrier();   // every CTA of the row runs before another writes to it
    pdl_wait();
    pdl_trigger();
    int64_t r = at.first + at.sub, ahead = r;
    if (kEdges) l.phase = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.h.p) + r * a.h.ld) & 15u) / sizeof(T));
    ring.cut(l);
    auto issue = [&](int stage) {
        if (ahead < s.M) {
            ring.issue(stage, 0, a.h, ahead, s.M, l);
            ring.issue(stage, 1, a.x, ahead, s.M, l);
            if (a.du.p) ring.issue(stage, 2, a.du, ahead, s.M, l);   // else its slots stay zero
            if (a.dy.p) ring.issue(stage, 3, a.dy, ahead, s.M, l);
            if constexpr (kGate) ring.issue(stage, 4, a.gate, ahead, s.M, l);
        }
        ring.commit();
        ahead += at.step;
    };
    auto gate_of = [&](int64_t row) {
        return !kGate && s.gate_cols && row < s.M ? static_cast<const T*>(a.gate.p)[row * a.gate.ld] : from_f32<T>(0.f);
    };
    auto stats_of = [&](int64_t row) { return row < s.M ? __ldg(a.stats_in + row) : make_float4(0.f, 0.f, 0.f, 0.f); };
    for (int i = 0; i < S - 1; ++i) issue(i);
    T gate = gate_of(r);
    float4 st = stats_of(r);
    float pa[E], wr[E], sum_b[E], sum_pre[E];
    Co::columns(pa, l, [&](int c) { return __ldg(a.scale + c) * __ldg(a.w_post + c); });
    Co::columns(wr, l, [&](int c) { return __ldg(a.w_pre + c); });
#pragma unroll
    for (int i = 0; i < E; ++i) sum_b[i] = sum_pre[i] = 0.f;
    int stage = 0;
    // every thread of the CTA goes round as often: the row sums may hold a barrier
    for (int64_t r0 = at.first; r0 < s.M; r0 += at.step, r += at.step) {
        issue((stage + S - 1) % S);
        const T gate_next = gate_of(r + at.step);
        const float4 st_next = stats_of(r + at.step);
        const bool live = r < s.M;
        ring.wait();
        float nh[E], ny[E], q[kGate ? E : 1], d[E];
        ring.open(stage, 0, nh);
        ring.open(stage, 1, ny);
        if constexpr (kGate) {
            ring.open(stage, 4, q);
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = element_sigmoid<T>(q[i]);
        } else {
            q[0] = s.gate_cols ? sigmoid(to_f32(gate)) : 1.f;
        }
        auto gate_at = [&](int i) { return q[kGate ? i : 0]; };
#pragma unroll
        for (int i = 0; i < E; ++i) {
            nh[i] = centred<kLayer>(nh[i], st.x) * st.y;
            ny[i] = centred<kLayer>(fmaf(gate_at(i) * pa[i], nh[i], ny[i]), st.z) * st.w;
        }
        ring.open(stage, 2, d);
        if (!live) {   // a row that is not there adds nothing
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = nh[i] = ny[i] = 0.f;
        }
        float m[kLayer ? 2 : 1] = {};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            sum_pre[i] = fmaf(d[i], ny[i], sum_pre[i]);
            d[i] *= wr[i];
            m[0] = fmaf(d[i], ny[i], m[0]);   // d is zero outside the row
            if constexpr (kLayer) m[1] += d[i];
        }
        row_sum(m, s, sums, round);
        const float dn = -m[0] * s.inv_c;
        float dm = 0.f;
        if constexpr (kLayer) dm = m[1] * s.inv_c;
        float dx[E];
        ring.open(stage, 3, dx);
        if (!live) {   // an infinity of the row that its slots held before would leave NaN
#pragma unroll
            for (int i = 0; i < E; ++i) dx[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) dx[i] = fmaf(st.w, fmaf(dn, ny[i], centred<kLayer>(d[i], dm)), dx[i]);
        if (live) Co::store(static_cast<T*>(a.out1) + r * s.C, dx, l);
        if constexpr (kLayer) Co::clear_outside(dx, l);   // without the means it is zero outside the row
        float b[kLayer ? 2 : 1] = {};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dx[i] *= gate_at(i);                    // from here dx q
            ny[i] = dx[i] * nh[i];                  // a row's part of B
            sum_b[i] += ny[i];
            d[i] = dx[i] * pa[i];
            b[0] = fmaf(d[i], nh[i], b[0]);
            if constexpr (kLayer) b[1] += d[i];
            if constexpr (kGate) ny[i] *= pa[i] * (1.f - q[i]);   // the gate's gradient
        }
        row_sum(b, s, sums, round);
        const float hn = -b[0] * s.inv_c;
        float hm = 0.f;
        if constexpr (kLayer) hm = b[1] * s.inv_c;
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = st.y * fmaf(hn, nh[i], centred<kLayer>(d[i], hm));
        if (live) {
            Co::store(static_cast<T*>(a.out0) + r * s.C, d, l);
            if constexpr (kGate) Co::store(static_cast<T*>(a.out2) + r * s.C, ny, l);
            else if (s.gate_cols && l.lane == 0) static_cast<T*>(a.out2)[r] = from_f32<T>(b[0] * (1.f - q[0]));
        }
        gate = gate_next;
        st = st_next;
        stage = (stage + 1) % S;
    }
    ring.drain();
    // the group's column sums: its rows' (which may be at other phases) added in order
    float* mine = a.partial + at.group * 2 * s.C;
    if (at.rows == 1) {
        Co::for_columns(l, [&](int i, int c) {
            mine[c] = sum_b[i];
            mine[s.C + c] = sum_pre[i];
        });
    } else {
        float* cols = reinterpret_cast<float*>(smem);   // [rows][C]
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            __syncthreads();
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

// The gradients of the parameters from the groups' column sums, added in
// order: kSumRows threads a column, then their sums in order.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_column_sums(const NormArgs a, int groups) {
    __shared__ float part[kSumRows][kSumCols];
    const int j = threadIdx.x % kSumCols, k = threadIdx.x / kSumCols, C = a.s.C;
    const int col = blockIdx.x * kSumCols + j;   // of 2 C
    pdl_wait();
    pdl_trigger();
    float v = 0.f;
    if (col < 2 * C)
#pragma unroll 8
        for (int i = k; i < groups; i += kSumRows) v += __ldg(a.partial + (int64_t)i * 2 * C + col);
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

// Which of the four kernels: a gate for each channel or not, means or not.
template <typename T, int VEC, int NV, bool kEdges, bool kBackward, bool kGate, bool kLayer>
int start(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    constexpr int NA = kBackward ? (kGate ? 5 : 4) : (kGate ? 3 : 2);
    constexpr int S = kBackward ? kBwdStages<VEC * NV> : kFwdStages, kThreads = norm_threads(VEC * NV, kBackward);
    constexpr int per_thread = S * NA * NV * NormRing<T, VEC, NV, NA, kEdges, S>::kSlot;
    int smem = per_thread * p.threads;
    if (kBackward && p.rows > 1) smem = imax(smem, p.rows * a.s.C * 4);
    constexpr int most = imax(per_thread * kThreads, kBackward ? VEC * NV * kThreads * 4 : 0);
    static_assert(most <= 224 * 1024, "the ring fits");
    // as many CTAs as run at once: by their registers (threads), and by their shared memory
    const int by_threads = (kBackward ? kBwdCtas<VEC * NV> : kFwdCtas<VEC * NV>) * kThreads / p.threads;
    const int per_sm = imin(by_threads, imax(1, 224 * 1024 / (smem + 4096)));
    const int ctas = num_sms() * per_sm;
    const int groups = norm_groups(a.s.M, p.rows, (kBackward ? imin(kNormCtas, ctas) : ctas) / p.cluster);
    if (groups == 0) return 0;
    static std::atomic<uint64_t> done[kMaxDevices];
    if constexpr (kBackward) {
        set_smem_limit_once(norm_bwd<T, VEC, NV, kEdges, kGate, kLayer>, most, done);
        norm_launch(norm_bwd<T, VEC, NV, kEdges, kGate, kLayer>, groups, p, smem, s, a);
    } else {
        set_smem_limit_once(norm_fwd<T, VEC, NV, kEdges, kGate, kLayer>, most, done);
        norm_launch(norm_fwd<T, VEC, NV, kEdges, kGate, kLayer>, groups, p, smem, s, a);
    }
    return groups;
}

template <typename T, int VEC, int NV, bool kEdges, bool kBackward>
zs_status start(const NormPlan& p, const NormArgs& a, cudaStream_t s) {
    const char* fn = kBackward ? "zs_norm_gate_residual_backward" : "zs_norm_gate_residual";
    int groups;
    if (a.s.gate_cols > 1) {
        groups = a.s.layer ? start<T, VEC, NV, kEdges, kBackward, true, true>(p, a, s)
                           : start<T, VEC, NV, kEdges, kBackward, true, false>(p, a, s);
    } else {
        groups = a.s.layer ? start<T, VEC, NV, kEdges, kBackward, false, true>(p, a, s)
                           : start<T, VEC, NV, kEdges, kBackward, false, false>(p, a, s);
    }
    if (zs_status st = check_launch(fn)) return st;
    if constexpr (kBackward) {
        launch(norm_column_sums, dim3((2 * a.s.C + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumRows), 0, s, a, groups);
        return check_launch(fn);
    }
    return ZS_OK;
}

template <typename T, bool kBackward>
zs_status dispatch(NormArgs& a, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const int64_t C = a.s.C;
    const bool full = a.s.gate_cols > 1;
    const NormAccess w = norm_access<T>(a.s.C, {a.h, a.x, a.dy, a.du, full ? a.gate : NormView{nullptr, 0}, {a.out0, C},
                                                {a.out1, C}, {full ? a.out2 : nullptr, C}});
    // Two pieces a thread are the faster (32768 x 512 bf16: forward 28 against 48 us, backward 44 against 56), except
    // that the backward, which holds more for each element, takes one where a warp then holds the row (65536 x 256 bf16
    // 57 against 70 us, 647170 x 128 fp32 406 against 418) and where the pieces at a row's ends take registers too
    // (4097 x 1031 fp16 48 against 58).
    const int most = kBackward && (w.edges ? C <= 256 * V : C <= 32 * V) ? 1 : 2;
    const NormPlan p = w.wide ? norm_plan(a.s.C, V, w.edges, most, kBackward) : norm_plan(a.s.C, 1, false, 4, kBackward);
    a.s.tpr = p.tpr;
    a.s.cluster = p.cluster;
    if (!w.wide) {   // operands at different phases: element by element
        if (p.nv <= 2) return start<T, 1, 2, false, kBackward>(p, a, s);
        return start<T, 1, 4, false, kBackward>(p, a, s);
    }
    if (w.edges) return p.nv == 1 ? start<T, V, 1, true, kBackward>(p, a, s) : start<T, V, 2, true, kBackward>(p, a, s);
    return p.nv == 1 ? start<T, V, 1, false, kBackward>(p, a, s) : start<T, V, 2, false, kBackward>(p, a, s);
}

}  // namespace

template <typename T>
zs_status norm_forward(NormArgs& a, cudaStream_t s) { return dispatch<T, false>(a, s); }
template <typename T>
zs_status norm_backward(NormArgs& a, cudaStream_t s) { return dispatch<T, true>(a, s); }

}  // namespace zs
