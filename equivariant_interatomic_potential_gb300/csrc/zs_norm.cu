// C entry points of the residual norms.
#include <initializer_list>

#include "zs_norm.cuh"

namespace zs {

namespace {

// The checks that both directions share; ZS_OK leaves a.s filled.
zs_status check(const char* fn, int32_t dtype, int32_t kind, const NormView& gate, int32_t gate_cols, int64_t M, int32_t C,
                NormArgs& a) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (kind != ZS_NORM_RMS && kind != ZS_NORM_LAYER)
        return fail(ZS_ERR_UNSUPPORTED, "%s: kind %d is not a zs_norm_kind", fn, kind);
    if (M < 0 || C < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld C=%d", fn, (long long)M, C);
    if (C > kNormMaxC) return fail(ZS_ERR_UNSUPPORTED, "%s: C=%d is above %d", fn, C, kNormMaxC);
    if (gate_cols != 0 && gate_cols != 1 && gate_cols != C)
        return fail(ZS_ERR_INVALID_ARG, "%s: gate_cols=%d is none of 0, 1 and C=%d", fn, gate_cols, C);
    if (M > 0 && (gate_cols == 0) != (gate.p == nullptr))
        return fail(ZS_ERR_INVALID_ARG, "%s: a gate pointer goes with gate_cols > 0", fn);
    if (!a.w_post || !a.scale || !a.w_pre) return fail(ZS_ERR_INVALID_ARG, "%s: w_post, scale or w_pre is NULL", fn);
    const uintptr_t el = (uintptr_t)dtype_bytes(dtype) - 1;
    for (const void* p : {gate.p, a.h.p, a.x.p, a.dy.p, a.du.p, (const void*)a.out0, (const void*)a.out1, (const void*)a.out2})
        if (reinterpret_cast<uintptr_t>(p) & el)
            return fail(ZS_ERR_INVALID_ARG, "%s: an array is not aligned to its elements", fn);
    for (const float* p : {a.w_post, a.scale, a.w_pre, (const float*)a.dw_post, (const float*)a.dscale, (const float*)a.dw_pre})
        if (reinterpret_cast<uintptr_t>(p) & 3)
            return fail(ZS_ERR_INVALID_ARG, "%s: an fp32 array is not aligned to its elements", fn);
    for (const NormView& v : {a.h, a.x, a.dy, a.du})
        if (v.p && v.ld < C && M > 1)
            return fail(ZS_ERR_INVALID_ARG, "%s: a row stride of %lld is below C=%d", fn, (long long)v.ld, C);
    if (gate.p && gate.ld < gate_cols && M > 1)
        return fail(ZS_ERR_INVALID_ARG, "%s: gate_ld=%lld is below gate_cols=%d", fn, (long long)gate.ld, gate_cols);
    a.s.M = M;
    a.s.C = C;
    a.s.gate_cols = gate_cols;
    a.s.layer = kind == ZS_NORM_LAYER;
    a.s.inv_c = 1.f / (float)C;
    a.gate = gate;
    return ZS_OK;
}

}  // namespace

}  // namespace zs

extern "C" {

zs_status zs_norm_gate_residual(int32_t dtype, int32_t kind, const void* h, int64_t h_ld, const void* x, int64_t x_ld,
                                const void* gate, int64_t gate_ld, int32_t gate_cols, const float* w_post,
                                const float* scale, const float* w_pre, float eps, int64_t M, int32_t C, void* y,
                                void* u, float* stats, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_norm_gate_residual";
    NormArgs a = {};
    a.h = {h, h_ld};
    a.x = {x, x_ld};
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.out0 = y, a.out1 = u;
    a.stats_out = reinterpret_cast<float4*>(stats);
    if (zs_status st = check(fn, dtype, kind, NormView{gate, gate_ld}, gate_cols, M, C, a)) return st;
    if (!(eps >= 0.f)) return fail(ZS_ERR_INVALID_ARG, "%s: eps=%g", fn, (double)eps);
    if (!aligned16(stats)) return fail(ZS_ERR_INVALID_ARG, "%s: stats is not 16-byte aligned", fn);
    if (M == 0) return ZS_OK;
    if (!h || !x || !y || !u) return fail(ZS_ERR_INVALID_ARG, "%s: NULL h, x, y or u", fn);
    a.s.eps = eps;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == ZS_F32 ? norm_forward<float>(a, s) : dtype == ZS_BF16 ? norm_forward<__nv_bfloat16>(a, s) : norm_forward<__half>(a, s);
}

size_t zs_norm_gate_residual_backward_workspace_bytes(int64_t M, int32_t C) {
    if (M <= 0 || C < 1) return 0;
    return (size_t)zs::imin<int64_t>(M, zs::kNormCtas) * 2 * (size_t)C * 4;
}

zs_status zs_norm_gate_residual_backward(int32_t dtype, int32_t kind, const void* dy, int64_t dy_ld, const void* du,
                                         int64_t du_ld, const void* h, int64_t h_ld, const void* x, int64_t x_ld,
                                         const void* gate, int64_t gate_ld, int32_t gate_cols, const float* w_post,
                                         const float* scale, const float* w_pre, const float* stats, int64_t M,
                                         int32_t C, void* dh, void* dx, void* dgate, float* dw_post, float* dscale,
                                         float* dw_pre, void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_norm_gate_residual_backward";
    NormArgs a = {};
    a.dy = {dy, dy_ld};
    a.du = {du, du_ld};
    a.h = {h, h_ld};
    a.x = {x, x_ld};
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.stats_in = reinterpret_cast<const float4*>(stats);
    a.out0 = dh, a.out1 = dx, a.out2 = dgate;
    a.dw_post = dw_post, a.dscale = dscale, a.dw_pre = dw_pre;
    a.partial = static_cast<float*>(workspace);
    if (zs_status st = check(fn, dtype, kind, NormView{gate, gate_ld}, gate_cols, M, C, a)) return st;
    if (!dw_post || !dscale || !dw_pre) return fail(ZS_ERR_INVALID_ARG, "%s: NULL dw_post, dscale or dw_pre", fn);
    if (M > 0) {
        if (!h || !x || !stats || !dh || !dx || (gate_cols > 0 && !dgate))
            return fail(ZS_ERR_INVALID_ARG, "%s: NULL h, x, stats, dh, dx or dgate", fn);
        if (!aligned16(stats)) return fail(ZS_ERR_INVALID_ARG, "%s: stats is not 16-byte aligned", fn);
        if (workspace_bytes < zs_norm_gate_residual_backward_workspace_bytes(M, C) || !workspace)
            return fail(ZS_ERR_INVALID_ARG, "%s: workspace of %zu bytes is too small", fn, workspace_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return fail(ZS_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == ZS_F32 ? norm_backward<float>(a, s) : dtype == ZS_BF16 ? norm_backward<__nv_bfloat16>(a, s) : norm_backward<__half>(a, s);
}

}  // extern "C"
