// Routing of rows to experts, and the gradient of the logits.
//
// A warp takes a row.  Its lanes hold the experts in ascending order, those of
// a group of experts in neighbouring lanes, so that the lowest lane among equal
// ones has the lowest index.  Scores become unsigned keys that sort like them
// (0: closed), and k rounds of a warp maximum pick the experts.
//
// The choice is that of the scores in 64 bits.  Without a bias and groups it
// goes by the logits themselves, which sort like their scores.  Otherwise scores
// are formed in 32 bits, with a bound of their error; where two neighbours of
// the choice lie closer than that (and are not of one logit and bias), the row is
// done again in 64 bits.  Weights are formed in 32 bits, relative to the largest
// chosen logit where they are renormalised, so that they never are 0 / 0.
//
// What bounds it: instructions, k rounds of about 3 E / 32 of them a row.
#include "zs_types.cuh"

namespace zs {
namespace {

constexpr int kRouteMaxE = 1024, kRouteMaxK = 32, kRouteMaxGroups = 32;
constexpr int kRouteWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

struct RouteShape {
    int64_t M, ld;
    int32_t E, k, groups, per, top_groups, group_top;
    int32_t lanes, each;    // lanes of a group, experts of a lane
    bool sigmoid, renormalise;
    float scale;
};

template <typename F> struct KeyOf;
template <> struct KeyOf<float> {
    using U = uint32_t;
    static __device__ __forceinline__ U bits(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ float value(U b) { return __uint_as_float(b); }
    static __device__ __forceinline__ U max_of_warp(U v) { return __reduce_max_sync(kAll, v); }
};
template <> struct KeyOf<double> {
    using U = unsigned long long;
    static __device__ __forceinline__ U bits(double v) { return (U)__double_as_longlong(v); }
    static __device__ __forceinline__ double value(U b) { return __longlong_as_double((long long)b); }
    static __device__ __forceinline__ U max_of_warp(U v) {
        for (int o = 16; o > 0; o >>= 1) {
            const U w = __shfl_xor_sync(kAll, v, o);
            v = w > v ? w : v;
        }
        return v;
    }
};
// Keys sort like their values; NaN above all, -infinity is 0.
template <typename F>
__device__ __forceinline__ typename KeyOf<F>::U to_key(F v) {
    using U = typename KeyOf<F>::U;
    constexpr U top = (U)1 << (8 * sizeof(U) - 1);
    if (v != v) return ~(U)0;
    if (v == -(F)INFINITY) return 0;
    const U b = KeyOf<F>::bits(v + (F)0);   // -0 is 0
    return b & top ? ~b : b | top;
}
template <typename F>
__device__ __forceinline__ F from_key(typename KeyOf<F>::U k) {
    using U = typename KeyOf<F>::U;
    constexpr U top = (U)1 << (8 * sizeof(U) - 1);
    return KeyOf<F>::value(k & top ? k & ~top : ~k);
}

template <typename F>
__device__ __forceinline__ F sum_of_warp(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float max_of_warp(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// A lane's experts.
struct Lane {
    int group, first, count;
    __device__ __forceinline__ Lane(const RouteShape& s, int lane) {
        group = lane / s.lanes;
        const int at = (lane - group * s.lanes) * s.each;
        first = group * s.per + at;
        count = group < s.groups ? imax(imin(s.per - at, s.each), 0) : 0;
    }
};

template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) { return to_f32(__ldg(row + e)); }

// Keeps the keys of the best groups, zeroes the others.  Returns whether the last group in and the first one out are
// closer than their scores are known, each to `error` and the rounding of its sum.
template <typename F, int V>
__device__ __forceinline__ bool keep_groups(const RouteShape& s, const Lane& l, typename KeyOf<F>::U (&key)[V], F error) {
    using U = typename KeyOf<F>::U;
    U first = 0, second = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const U k = key[i];
        second = k > first ? first : (k > second ? k : second);
        first = k > first ? k : first;
    }
    for (int o = 1; o < s.lanes; o <<= 1) {
        const U a = __shfl_xor_sync(kAll, first, o), b = __shfl_xor_sync(kAll, second, o);
        second = a > first ? (b > first ? b : first) : (a > second ? a : second);
        first = a > first ? a : first;
    }
    U value = 0;
    F size = 0;   // of what the sum is formed of
    if (first) {
        F v = from_key<F>(first);
        size = fabs(v);
        if (first == ~(U)0 || (s.group_top == 2 && second == ~(U)0)) {
            v = (F)NAN;
        } else if (s.group_top == 2 && second) {
            const F w = from_key<F>(second);
            v += w;
            size += fabs(w);
        }
        value = to_key<F>(v);
        if (!value) value = 1;
    }
    int ahead = 0;
    for (int g = 0; g < s.groups; ++g) {
        const U other = __shfl_sync(kAll, value, g * s.lanes);
        ahead += other > value || (other == value && g < l.group);
    }
    const bool kept = l.group < s.groups && ahead < s.top_groups;
    const bool last = kept && ahead == s.top_groups - 1, next = l.group < s.groups && ahead == s.top_groups;
    const unsigned in = __ballot_sync(kAll, last), out = __ballot_sync(kAll, next);
    bool close = false;
    if (in && out) {
        const int p = __ffs(in) - 1, q = __ffs(out) - 1;
        const U a = __shfl_sync(kAll, value, p), b = __shfl_sync(kAll, value, q);
        const F sizes = __shfl_sync(kAll, size, p) + __shfl_sync(kAll, size, q);
        close = a && b && from_key<F>(a) - from_key<F>(b) <= 4 * error + (F)0x1p-22 * sizes;
    }
    if (!kept)
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0;
    return close;
}

// The largest key of the warp, taken out: its expert in `e` (of the lowest index), the key returned (0: none left).
template <typename F, int V>
__device__ __forceinline__ typename KeyOf<F>::U take(const Lane& l, int lane, typename KeyOf<F>::U (&key)[V], int& e) {
    using U = typename KeyOf<F>::U;
    U best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
    const U top = KeyOf<F>::max_of_warp(best);
    if (top == 0) return 0;
    const int winner = __ffs(__ballot_sync(kAll, best == top)) - 1;
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = key[i] == top ? i : at;
    if (lane == winner)
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = i == at ? 0 : key[i];
    e = __shfl_sync(kAll, l.first + at, winner);
    return top;
}

// The row's choice in 64 bits: the expert of choice `lane` (or -1).
template <typename T, int V>
__device__ __noinline__ int choose_in_64_bits(const RouteShape& s, int lane, const T* __restrict__ row, const float* __restrict__ bias) {
    const Lane l(s, lane);
    double z[V], top = -INFINITY;
    for (int i = 0; i < V; ++i) {
        z[i] = i < l.count ? (double)logit(row, l.first + i) : -INFINITY;
        top = z[i] > top ? z[i] : top;
    }
    double sum = 0.0;
    if (!s.sigmoid) {
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
        for (int i = 0; i < V; ++i)
            if (i < l.count && top != -INFINITY) sum += exp(z[i] - top);
        sum = sum_of_warp(sum);
    }
    unsigned long long key[V];
    for (int i = 0; i < V; ++i) {
        key[i] = 0;
        if (i >= l.count || z[i] == -INFINITY) continue;
        const double score = s.sigmoid ? 1.0 / (1.0 + exp(-z[i])) : exp(z[i] - top) / sum;
        key[i] = to_key<double>(score + (bias ? (double)__ldg(bias + l.first + i) : 0.0));
    }
    if (s.top_groups < s.groups) keep_groups<double, V>(s, l, key, 0.0);
    int mine = -1;
    for (int r = 0; r < s.k; ++r) {
        int e = -1;
        if (take<double, V>(l, lane, key, e) == 0) break;
        if (lane == r) mine = e;
    }
    return mine;
}

// Shares of the chosen logits z (lanes with `held`) among themselves: softmax, or sigmoids over their sum.
__device__ __forceinline__ float renormalised(bool sigmoid, bool held, float z) {
    const float top = max_of_warp(held ? z : -INFINITY);
    float t = 0.f;
    if (held) {
        if (sigmoid) t = expf(fminf(z, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(z)));
        else t = expf(z - top);
        if (z != z) t = z;
    }
    const float sum = sum_of_warp(t);
    return held ? t / sum : 0.f;
}
__device__ __forceinline__ float sigmoid_of(float z) { return 1.f / (1.f + expf(-z)); }

template <typename T, int V, bool kScored>
__global__ void __launch_bounds__(kRouteWarps * 32) route_rows(RouteShape s, const T* __restrict__ logits, const float* __restrict__ bias,
                                                               int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (r0 >= s.M) return;
    const T* row = logits + r0 * s.ld;
    const Lane l(s, lane);
    float z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = i < l.count ? logit(row, l.first + i) : -INFINITY;
    float top = 0.f, sum = 1.f;
    const bool whole = !s.sigmoid && (kScored || !s.renormalise);   // scores over all experts are wanted
    if (whole) {
        top = z[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, z[i]);
        top = max_of_warp(top);
    }
    float e[V];
    if (whole) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = z[i] == -INFINITY ? 0.f : expf(z[i] - top);
            sum += e[i];
        }
        sum = sum_of_warp(sum);
    }
    uint32_t key[V];
    float error = 0.f;   // of a score, beside its rounding
    bool close = false;
    if (kScored) {
        const float inv = 1.f / sum;
        // sigmoids: an exponential, a sum and a quotient; softmax: the difference to the largest logit is known to
        // 2^-24 of itself, and an exponential above zero has no difference beyond 104
        error = s.sigmoid ? 0x1p-20f : 0x1p-17f * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float score = s.sigmoid ? sigmoid_of(z[i]) : e[i] * inv;
            key[i] = z[i] == -INFINITY ? 0 : to_key(score + (bias && i < l.count ? __ldg(bias + l.first + i) : 0.f));
        }
        if (s.top_groups < s.groups) close = keep_groups<float, V>(s, l, key, error);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = to_key(z[i]);
    }
    int mine = -1, before = -1;
    float last = 0.f;
    for (int r = 0; r < (kScored ? s.k + 1 : s.k); ++r) {
        int at = -1;
        const uint32_t best = take<float, V>(l, lane, key, at);
        if (best == 0) break;
        if (kScored) {
            const float a = from_key<float>(best);
            if (r > 0 && last - a <= 2.f * error + 0x1p-22f * (fabsf(last) + fabsf(a)) &&
                !(logit(row, before) == logit(row, at) && (!bias || __ldg(bias + before) == __ldg(bias + at))))
                close = true;
            last = a;
            before = at;
        }
        if (lane == r && r < s.k) mine = at;
    }
    if (kScored && close) mine = choose_in_64_bits<T, V>(s, lane, row, bias);
    const bool held = mine >= 0;
    const float zc = held ? logit(row, mine) : -INFINITY;
    float w;
    if (s.renormalise) w = renormalised(s.sigmoid, held, zc);
    else w = !held ? 0.f : s.sigmoid ? sigmoid_of(zc) : expf(zc - top) / sum;
    if (lane < s.k) {
        ids[r0 * s.k + lane] = mine;
        weights[r0 * s.k + lane] = held ? w * s.scale : 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_rows_backward(RouteShape s, const float* __restrict__ dweights,
                                                                        const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                                        T* __restrict__ dlogits) {
    extern __shared__ float buffers[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * kRouteWarps + warp;
    float* g = buffers + warp * s.E;   // gradients by expert
    pdl_wait();
    pdl_trigger();
    if (r0 >= s.M) return;
    const T* row = logits + r0 * s.ld;
    for (int i = lane; i < s.E; i += 32) g[i] = 0.f;
    const int id = lane < s.k ? __ldg(ids + r0 * s.k + lane) : -1;
    const bool held = (uint32_t)id < (uint32_t)s.E;
    const float z = held ? logit(row, id) : -INFINITY;
    const float d = held ? __ldg(dweights + r0 * s.k + lane) * s.scale : 0.f;
    const bool whole = !s.sigmoid && !s.renormalise;
    float top = -INFINITY, sum = 0.f, mean = 0.f, own = d;
    if (whole) {
        for (int i = lane; i < s.E; i += 32) top = fmaxf(top, logit(row, i));
        top = max_of_warp(top);
        for (int i = lane; i < s.E; i += 32) {
            const float v = logit(row, i);
            sum += v == -INFINITY ? 0.f : expf(v - top);
        }
        sum = sum_of_warp(sum);
        mean = sum_of_warp(held ? d * (expf(z - top) / sum) : 0.f);
    } else if (s.renormalise) {
        const float share = renormalised(s.sigmoid, held, z);
        const float all = sum_of_warp(held ? share * d : 0.f);
        own = share * (d - all);
        if (s.sigmoid) own *= sigmoid_of(-z);
    } else {
        own = d * sigmoid_of(z) * sigmoid_of(-z);
    }
    __syncwarp();
    for (int j = 0; j < s.k; ++j) {   // one after another: an expert may be named twice
        if (lane == j && held) g[id] += own;
        __syncwarp();
    }
    T* out = dlogits + r0 * s.E;
    for (int i = lane; i < s.E; i += 32) {
        float v = g[i];
        if (whole) {
            const float zi = logit(row, i);
            v = zi == -INFINITY ? 0.f : expf(zi - top) / sum * (v - mean);
        }
        out[i] = from_f32<T>(v);
    }
}

template <typename T, bool kScored>
zs_status route_launch(const RouteShape& s, const void* logits, const float* bias, int32_t* ids, float* weights, cudaStream_t stream) {
    const dim3 grid((unsigned)((s.M + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    const T* z = static_cast<const T*>(logits);
    if (s.each <= 1) launch(route_rows<T, 1, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    else if (s.each <= 2) launch(route_rows<T, 2, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    else if (s.each <= 4) launch(route_rows<T, 4, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    else if (s.each <= 8) launch(route_rows<T, 8, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    else if (s.each <= 16) launch(route_rows<T, 16, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    else launch(route_rows<T, 32, kScored>, grid, block, 0, stream, s, z, bias, ids, weights);
    return check_launch("route");
}

zs_status check(const char* fn, int32_t dtype, int32_t score, const void* logits, int64_t ld, int64_t M, int32_t E, int32_t k, float scale,
                RouteShape& s) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (score != ZS_SCORE_SOFTMAX && score != ZS_SCORE_SIGMOID)
        return fail(ZS_ERR_UNSUPPORTED, "%s: score %d is not a zs_score_kind", fn, score);
    if (M < 0 || M > ((int64_t)1 << 31) - (1 << 16) || E < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld E=%d", fn, (long long)M, E);
    if (k < 1 || k > E) return fail(ZS_ERR_INVALID_ARG, "%s: k=%d is outside [1, E=%d]", fn, k, E);
    if (E > kRouteMaxE || k > kRouteMaxK)
        return fail(ZS_ERR_UNSUPPORTED, "%s: E=%d is above %d or k=%d above %d", fn, E, kRouteMaxE, k, kRouteMaxK);
    if (!(scale - scale == 0.f)) return fail(ZS_ERR_INVALID_ARG, "%s: scale=%g", fn, (double)scale);
    if (M > 0 && !logits) return fail(ZS_ERR_INVALID_ARG, "%s: logits is NULL", fn);
    if (reinterpret_cast<uintptr_t>(logits) & (uintptr_t)(dtype_bytes(dtype) - 1))
        return fail(ZS_ERR_INVALID_ARG, "%s: logits is not aligned to its elements", fn);
    if (M > 1 && ld < E) return fail(ZS_ERR_INVALID_ARG, "%s: a row stride of logits, %lld, is below E=%d", fn, (long long)ld, E);
    s.M = M, s.ld = ld, s.E = E, s.k = k, s.scale = scale;
    s.sigmoid = score == ZS_SCORE_SIGMOID;
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" {

zs_status zs_route(int32_t dtype, int32_t score, const void* logits, int64_t logits_ld, const float* bias, int64_t M, int32_t E,
                   int32_t k, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renormalise, float scale, int32_t* ids,
                   float* weights, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_route";
    RouteShape s = {};
    if (zs_status st = check(fn, dtype, score, logits, logits_ld, M, E, k, scale, s)) return st;
    if (groups < 1 || E % groups) return fail(ZS_ERR_INVALID_ARG, "%s: groups=%d does not divide E=%d", fn, groups, E);
    if (groups > kRouteMaxGroups) return fail(ZS_ERR_UNSUPPORTED, "%s: groups=%d is above %d", fn, groups, kRouteMaxGroups);
    if (top_groups < 1 || top_groups > groups)
        return fail(ZS_ERR_INVALID_ARG, "%s: top_groups=%d is outside [1, groups=%d]", fn, top_groups, groups);
    if (group_top != 1 && group_top != 2) return fail(ZS_ERR_INVALID_ARG, "%s: group_top=%d is neither 1 nor 2", fn, group_top);
    if ((int64_t)top_groups * (E / groups) < k)
        return fail(ZS_ERR_INVALID_ARG, "%s: k=%d experts are more than %d groups of %d hold", fn, k, top_groups, E / groups);
    if (M > 0 && (!ids || !weights)) return fail(ZS_ERR_INVALID_ARG, "%s: ids or weights is NULL", fn);
    for (const void* p : {(const void*)bias, (const void*)ids, (const void*)weights})
        if (reinterpret_cast<uintptr_t>(p) & 3) return fail(ZS_ERR_INVALID_ARG, "%s: bias, ids or weights is not aligned to its elements", fn);
    s.renormalise = renormalise != 0;
    s.groups = top_groups < groups ? groups : 1;   // where all are kept they make no difference
    s.top_groups = top_groups < groups ? top_groups : 1;
    s.per = E / s.groups;
    s.group_top = group_top;
    int slots = 1;
    while (slots < s.groups) slots *= 2;
    s.lanes = 32 / slots;
    s.each = (s.per + s.lanes - 1) / s.lanes;
    if (s.each > kRouteMaxE / 32)
        return fail(ZS_ERR_UNSUPPORTED, "%s: %d groups of %d experts do not fit 32 lanes of %d", fn, s.groups, s.per, kRouteMaxE / 32);
    if (M == 0) return ZS_OK;
    const bool scored = bias || s.groups > 1;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        return scored ? route_launch<T, true>(s, logits, bias, ids, weights, st) : route_launch<T, false>(s, logits, bias, ids, weights, st);
    };
    return dtype == ZS_F32 ? go(float()) : dtype == ZS_BF16 ? go(__nv_bfloat16()) : go(__half());
}

zs_status zs_route_backward(int32_t dtype, int32_t score, const float* dweights, const void* logits, int64_t logits_ld,
                            const int32_t* ids, int64_t M, int32_t E, int32_t k, int32_t renormalise, float scale, void* dlogits,
                            zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_route_backward";
    RouteShape s = {};
    if (zs_status st = check(fn, dtype, score, logits, logits_ld, M, E, k, scale, s)) return st;
    if (M > 0 && (!dweights || !ids || !dlogits)) return fail(ZS_ERR_INVALID_ARG, "%s: dweights, ids or dlogits is NULL", fn);
    if ((reinterpret_cast<uintptr_t>(dweights) | reinterpret_cast<uintptr_t>(ids)) & 3 ||
        reinterpret_cast<uintptr_t>(dlogits) & (uintptr_t)(dtype_bytes(dtype) - 1))
        return fail(ZS_ERR_INVALID_ARG, "%s: dweights, ids or dlogits is not aligned to its elements", fn);
    if (M == 0) return ZS_OK;
    s.renormalise = renormalise != 0;
    const dim3 grid((unsigned)((M + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    const size_t smem = (size_t)kRouteWarps * E * sizeof(float);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        launch(route_rows_backward<T>, grid, block, smem, st, s, dweights, static_cast<const T*>(logits), ids, static_cast<T*>(dlogits));
    };
    if (dtype == ZS_F32) go(float());
    else if (dtype == ZS_BF16) go(__nv_bfloat16());
    else go(__half());
    return check_launch("route gradient");
}

}  // extern "C"
