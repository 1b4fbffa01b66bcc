// AdamW over many tensors in one launch (up to kTableMax tensors each), with
// states in 32 bits or in e4m3 with a scale per 256 elements.
//
// Bound by HBM: a step reads and writes the parameter and both states and
// reads the gradient once (28 bytes an element in fp32, 22 with 16-bit
// parameters, 16 and 10 with 8-bit states).  The tensors' pointers travel as
// kernel arguments, so a call uploads nothing and owns no memory.  The
// elements of all tensors are cut into chunks of 256 threads x 8 elements;
// a CTA finds its tensor by a binary search over the chunk counts' prefix.
#include <cuda_fp8.h>
#include <math.h>

#include "zs_types.cuh"

namespace zs {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                      // elements of a thread
constexpr int kChunk = kThreads * kPer;
constexpr int kBlock = 256;                  // elements that share a scale: one warp's
static_assert(kBlock == 32 * kPer, "a warp holds one block of an 8-bit state");

// Kernel arguments may take 32764 bytes.  Most calls have few tensors and
// take a short table.
constexpr int kTableShort = 32, kTableMax = 500;

template <int N>
struct Table {
    zs_adamw_tensor t[N];
    int32_t first[N + 1];   // first chunk of each tensor
    int32_t count;
};

struct Consts {
    float beta1, omb1, beta2, omb2, eps, decay, step_size, rbc2;
};

// What the random bits of 8-bit codes are formed from: a key of the seed and
// the step, and the chunks of the list before this table.
struct Dither {
    uint32_t lo, hi;
    int64_t base;
};

// States in 32 bits, in 8 rounded to nearest, and in 8 rounded at random: up
// with the probability of the distance to the code below, so that a state's
// expectation is its value.  To nearest, a root that a step changes by less
// than half a code (with beta2 = 0.999 every one but the block's largest, which
// the scale follows) never moves again.
enum States { kFull, kNearest, kRandom };

constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Tiny = 0.001953125f;   // 2^-9
constexpr float kScaleMin = 1e-30f;

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// m, v (the second moment before its root) -> m, root of v, p.  Every
// operation rounds once (the intrinsics keep the compiler from fusing), so
// that 8-bit codes follow from the formula alone.
__device__ __forceinline__ void update(float& p, float g, float& m, float v, float& r, const Consts& c) {
    m = __fadd_rn(__fmul_rn(c.beta1, m), __fmul_rn(c.omb1, g));
    r = __fsqrt_rn(v);
    const float denom = __fadd_rn(__fmul_rn(r, c.rbc2), c.eps);
    p = __fsub_rn(__fmul_rn(p, c.decay), __fmul_rn(c.step_size, __fdiv_rn(m, denom)));
}
__device__ __forceinline__ float second_moment(float v, float g, const Consts& c) {
    return __fadd_rn(__fmul_rn(c.beta2, v), __fmul_rn(c.omb2, __fmul_rn(g, g)));
}

// Reads or writes `n` (<= kPer) consecutive elements from p + i.
template <typename T>
__device__ __forceinline__ void load(const T* p, int64_t i, int n, bool wide, float (&f)[kPer]) {
    if (wide && n == kPer) {
#pragma unroll
        for (int j = 0; j < kPer; j += kVec<T>) {
            float q[kVec<T>];
            unpack<T>(ld_piece(p + i + j), q);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) f[j + k] = q[k];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) f[j] = j < n ? to_f32(p[i + j]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store(T* p, int64_t i, int n, bool wide, const float (&f)[kPer]) {
    if (wide && n == kPer) {
#pragma unroll
        for (int j = 0; j < kPer; j += kVec<T>) {
            float q[kVec<T>];
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) q[k] = f[j + k];
            st_piece(p + i + j, pack<T>(q));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < n) p[i + j] = from_f32<T>(f[j]);
    }
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t i, int n, bool wide) {
    if (wide && n == kPer) return *reinterpret_cast<const uint2*>(p + i);
    uint2 c = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (j < n) (j < 4 ? c.x : c.y) |= (uint32_t)p[i + j] << (8 * (j & 3));
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int n, bool wide, uint2 c) {
    if (wide && n == kPer) {
        *reinterpret_cast<uint2*>(p + i) = c;
        return;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (j < n) p[i + j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
}
__device__ __forceinline__ void decode(uint2 c, float scale, float (&f)[kPer]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? c.x : c.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        f[2 * j] = __fmul_rn(v.x, scale);
        f[2 * j + 1] = __fmul_rn(v.y, scale);
    }
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 32 random bits of element c of the list: multiply-xorshift rounds, the key
// in their midst too, so that no two steps' bits are the same ones reordered.
__device__ __forceinline__ uint32_t random_bits(uint32_t c, uint32_t lo, uint32_t hi) {
    uint32_t x = c ^ lo;
    x = (x ^ (x >> 16)) * 0x7feb352du;
    x = ((x ^ (x >> 15)) + hi) * 0x846ca68bu;
    return x ^ (x >> 16);
}
// |q| <= 448 or a little above -> the e4m3 value below or above it, by 16 random
// bits.  The last 20 of its 23 bits go, with 2^-6 added first where the codes
// stand 2^-9 apart whatever the exponent.  What is a code stays one.
__device__ __forceinline__ float round_at_random(float q, uint32_t bits16) {
    const float a = fabsf(q), off = a < 0.015625f ? 0.015625f : 0.f;
    const uint32_t t = (__float_as_uint(__fadd_rn(a, off)) + (bits16 << 4) + 8u) & 0xfff00000u;
    return copysignf(__fadd_rn(__uint_as_float(t), -off), q);
}
// The codes of a block (a warp's values, zero past its end) and its scale.
// Blocks of finite values, all but every one, take no care of others.
template <bool kRoot, bool kAtRandom>
__device__ __forceinline__ uint2 encode(const float (&f)[kPer], float& scale, const uint32_t (&bits)[kPer]) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) top = max_or_nan(top, fabsf(f[j]));
    const bool fine = __all_sync(0xffffffffu, finite(top));
    if (!fine) {
        top = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (finite(f[j])) top = fmaxf(top, fabsf(f[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool live = top >= kScaleMin;
    scale = live ? __fmul_rn(top, 1.f / kE4m3Max) : 0.f;
    const float inv = live ? __fmul_rn(__frcp_rn(top), kE4m3Max) : 0.f;
    const float least = live ? kE4m3Tiny : 0.f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
        float2 q;
        float* qe = &q.x;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = f[j + k];
            qe[k] = __fmul_rn(x, inv);
            if (kAtRandom) qe[k] = round_at_random(qe[k], kRoot ? bits[j + k] >> 16 : bits[j + k] & 0xffffu);
            if (kRoot && x > 0.f) qe[k] = fmaxf(qe[k], least);
            if (!fine && !finite(x)) qe[k] = __int_as_float(0x7fc00000);
        }
        w[j / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (16 * ((j / 2) & 1));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ bool aligned(const void* p, unsigned a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// 8-bit states take 88 instructions an element in long chains (roots, quotients, block maxima), so warps count for more than
// the few values that spill: 30 M fp32 elements take 109 us with 4 CTAs an SM, 103 with 5, 102 with 6, and 12 more rounded at random.  32-bit states wait for
// memory, with more loads a warp on their way (200 M bf16: 628 us as the compiler likes, 714 with 5 CTAs).
template <typename T, States kStates, int N>
__global__ void __launch_bounds__(kThreads, kStates == kFull ? 1 : 6)
adamw_step(const __grid_constant__ Table<N> table, Consts c, const float* __restrict__ grad_scale, Dither d) {
    pdl_wait();
    pdl_trigger();
    const int chunk = blockIdx.x;
    int lo = 0, hi = table.count;   // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.first[mid] <= chunk) lo = mid; else hi = mid;
    }
    const zs_adamw_tensor& t = table.t[lo];
    const int64_t i = (int64_t)(chunk - table.first[lo]) * kChunk + threadIdx.x * kPer;
    const int64_t left = t.numel - i;
    const int n = left <= 0 ? 0 : left < kPer ? (int)left : kPer;
    if (__ballot_sync(0xffffffffu, n > 0) == 0) return;   // whole warps: a block of 8-bit states is a warp's
    const float gs = grad_scale ? __ldg(grad_scale) : 1.f;
    T* param = static_cast<T*>(t.param);
    const T* grad = static_cast<const T*>(t.grad);
    float p[kPer], g[kPer], m[kPer], v[kPer], r[kPer];
    load(grad, i, n, aligned(grad, 16), g);
    const bool pw = aligned(param, 16);
    load(param, i, n, pw, p);
    if constexpr (kStates == kFull) {
        float* ma = static_cast<float*>(t.exp_avg);
        float* va = static_cast<float*>(t.exp_avg_sq);
        const bool mw = aligned(ma, 16), vw = aligned(va, 16);
        load(ma, i, n, mw, m);
        load(va, i, n, vw, v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float gj = __fmul_rn(g[j], gs);
            v[j] = second_moment(v[j], gj, c);
            update(p[j], gj, m[j], v[j], r[j], c);
        }
        store(param, i, n, pw, p);
        store(ma, i, n, mw, m);
        store(va, i, n, vw, v);
    } else {
        uint8_t* ma = static_cast<uint8_t*>(t.exp_avg);
        uint8_t* va = static_cast<uint8_t*>(t.exp_avg_sq);
        const bool mw = aligned(ma, 8), vw = aligned(va, 8);
        const int64_t b = i / kBlock;
        const uint2 mc = load_codes(ma, i, n, mw), vc = load_codes(va, i, n, vw);
        decode(mc, t.exp_avg_scale[b], m);
        decode(vc, t.exp_avg_sq_scale[b], r);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float gj = __fmul_rn(g[j], gs);
            update(p[j], gj, m[j], second_moment(__fmul_rn(r[j], r[j]), gj, c), r[j], c);
        }
        store(param, i, n, pw, p);
        uint32_t bits[kPer] = {};
        if constexpr (kStates == kRandom) {
            const int64_t at = (d.base + chunk) * kChunk + threadIdx.x * kPer;
            const uint32_t lo = d.lo + (uint32_t)(at >> 32) * 0x9e3779b9u;
#pragma unroll
            for (int j = 0; j < kPer; ++j) bits[j] = random_bits((uint32_t)at + j, lo, d.hi);
        }
        float ms, rs;
        store_codes(ma, i, n, mw, encode<false, kStates == kRandom>(m, ms, bits));
        store_codes(va, i, n, vw, encode<true, kStates == kRandom>(r, rs, bits));
        if ((threadIdx.x & 31) == 0) {
            t.exp_avg_scale[b] = ms;
            t.exp_avg_sq_scale[b] = rs;
        }
    }
}

template <typename T, States kStates, int N>
zs_status launch_table(const Table<N>& table, const Consts& c, const float* grad_scale, const Dither& d, cudaStream_t s) {
    const int chunks = table.first[table.count];
    if (chunks == 0) return ZS_OK;
    launch(adamw_step<T, kStates, N>, dim3(chunks), dim3(kThreads), 0, s, table, c, grad_scale, d);
    return check_launch("zs_adamw_step");
}

// Cuts the list into tables: kTableMax tensors, or 2^30 chunks, each.
template <typename T, States kStates, int N>
zs_status step_with(const zs_adamw_tensor* tensors, int32_t count, const Consts& c, const float* grad_scale, Dither d,
                    cudaStream_t s) {
    Table<N> table;
    table.count = 0;
    int64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i) {
        const int64_t n = tensors[i].numel;
        if (n == 0) continue;
        const int64_t k = (n + kChunk - 1) / kChunk;
        if (table.count == N || chunks + k > (int64_t(1) << 30)) {
            table.first[table.count] = (int32_t)chunks;
            const zs_status st = launch_table<T, kStates>(table, c, grad_scale, d, s);
            if (st != ZS_OK) return st;
            table.count = 0;
            d.base += chunks;
            chunks = 0;
        }
        table.t[table.count] = tensors[i];
        table.first[table.count++] = (int32_t)chunks;
        chunks += k;
    }
    table.first[table.count] = (int32_t)chunks;
    return launch_table<T, kStates>(table, c, grad_scale, d, s);
}

template <typename T, States kStates>
zs_status step(const zs_adamw_tensor* tensors, int32_t count, const Consts& c, const float* grad_scale, const Dither& d,
               cudaStream_t s) {
    if (count <= kTableShort) return step_with<T, kStates, kTableShort>(tensors, count, c, grad_scale, d, s);
    return step_with<T, kStates, kTableMax>(tensors, count, c, grad_scale, d, s);
}

template <typename T>
zs_status step(States states, const zs_adamw_tensor* tensors, int32_t count, const Consts& c, const float* grad_scale,
               const Dither& d, cudaStream_t s) {
    switch (states) {
        case kFull: return step<T, kFull>(tensors, count, c, grad_scale, d, s);
        case kNearest: return step<T, kNearest>(tensors, count, c, grad_scale, d, s);
        default: return step<T, kRandom>(tensors, count, c, grad_scale, d, s);
    }
}

// seed: NULL rounds to nearest.
zs_status adamw(const char* fn, const zs_adamw_tensor* tensors, int32_t count, int32_t dtype, int32_t state_bits,
                const zs_adamw_hyper* hyper, const uint64_t* seed, const float* grad_scale, zs_stream_t stream) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (state_bits != 32 && state_bits != 8)
        return fail(ZS_ERR_UNSUPPORTED, "%s: states have 32 or 8 bits, not %d", fn, state_bits);
    if (count < 0 || (count > 0 && !tensors) || !hyper)
        return fail(ZS_ERR_INVALID_ARG, "%s: count=%d with a NULL table, or no hyper-parameters", fn, count);
    const zs_adamw_hyper& h = *hyper;
    if (!(h.step >= 1) || !(h.beta1 >= 0 && h.beta1 < 1) || !(h.beta2 >= 0 && h.beta2 < 1) || !(h.eps >= 0) ||
        !isfinite(h.lr) || !isfinite(h.weight_decay) || !isfinite(h.eps))
        return fail(ZS_ERR_INVALID_ARG, "%s: lr=%g beta1=%g beta2=%g eps=%g weight_decay=%g step=%lld", fn, h.lr,
                    h.beta1, h.beta2, h.eps, h.weight_decay, (long long)h.step);
    const uintptr_t el = (uintptr_t)dtype_bytes(dtype) - 1, st = state_bits == 32 ? 3 : 0;
    auto off = [](const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    for (int32_t i = 0; i < count; ++i) {
        const zs_adamw_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > (int64_t(1) << 40))
            return fail(ZS_ERR_INVALID_ARG, "%s: tensor %d has numel=%lld", fn, i, (long long)t.numel);
        if (t.numel == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
            (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
            return fail(ZS_ERR_INVALID_ARG, "%s: tensor %d has a NULL array", fn, i);
        if (off(t.param, el) || off(t.grad, el) || off(t.exp_avg, st) || off(t.exp_avg_sq, st) ||
            (state_bits == 8 && (off(t.exp_avg_scale, 3) || off(t.exp_avg_sq_scale, 3))))
            return fail(ZS_ERR_INVALID_ARG, "%s: tensor %d has an array that is not aligned to its elements", fn, i);
    }
    Consts c;
    c.beta1 = (float)h.beta1;
    c.omb1 = (float)(1.0 - h.beta1);
    c.beta2 = (float)h.beta2;
    c.omb2 = (float)(1.0 - h.beta2);
    c.eps = (float)h.eps;
    c.decay = (float)(1.0 - h.lr * h.weight_decay);
    c.step_size = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
    c.rbc2 = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const States states = state_bits == 32 ? kFull : seed ? kRandom : kNearest;
    Dither d = {};
    if (seed) {
        uint64_t key = *seed ^ ((uint64_t)h.step * 0x9e3779b97f4a7c15ull);
        for (int i = 0; i < 2; ++i) key = (key ^ (key >> 32)) * 0xd6e8feb86659fd93ull;
        key ^= key >> 32;
        d.lo = (uint32_t)key, d.hi = (uint32_t)(key >> 32);
    }
    switch (dtype) {
        case ZS_F32: return step<float>(states, tensors, count, c, grad_scale, d, s);
        case ZS_BF16: return step<__nv_bfloat16>(states, tensors, count, c, grad_scale, d, s);
        default: return step<__half>(states, tensors, count, c, grad_scale, d, s);
    }
}

}  // namespace

}  // namespace zs

extern "C" {

zs_status zs_adamw_step(const zs_adamw_tensor* tensors, int32_t count, int32_t dtype, int32_t state_bits,
                        const zs_adamw_hyper* hyper, const float* grad_scale, zs_stream_t stream) {
    return zs::adamw("zs_adamw_step", tensors, count, dtype, state_bits, hyper, nullptr, grad_scale, stream);
}

zs_status zs_adamw_step_seeded(const zs_adamw_tensor* tensors, int32_t count, int32_t dtype, int32_t state_bits,
                               const zs_adamw_hyper* hyper, uint64_t seed, const float* grad_scale, zs_stream_t stream) {
    return zs::adamw("zs_adamw_step_seeded", tensors, count, dtype, state_bits, hyper, &seed, grad_scale, stream);
}

}  // extern "C"
