// Dropout from a counter-based generator, with an optional residual sum:
//   y = residual + (u >= limit ? h * 65536 / (65536 - limit) : 0)
// limit = round(65536 p), u 16 bits for each element.  Eight elements in a row
// share one output of Philox 4x32 with 10 rounds (J. K. Salmon, M. A. Moraes,
// R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
// the counter is (block number: 64 bits, call, step), the key the seed, so that
// the mask is never stored: the backward pass draws it again from the counters.
//
// Bound by memory: an element costs 4 bytes and more (16-bit, no residual), its
// share of the generator about 6 instructions of the 22 that fit beside it (32
// bits for each element would take all of them).  32768 x 2048 bf16: 47 us, 56
// with a residual, 5.7 and 7.1 TB/s; the second is above the rate of a copy since
// 56 MB of the 134 written are still in L2 at the kernel's end.  Rows at strides,
// and bases off 16-byte boundaries, go element by element: 164 and 173 us.
#include <math.h>

#include "zs_rows.cuh"

namespace zs {
namespace {

constexpr int kDropBlock = 8;       // elements that share a counter
constexpr int kDropThreads = 256;

struct DropKey {
    uint32_t seed[2], call, limit;
    int64_t step;
    const int64_t* step_at;         // added to step; may be NULL
    float factor;
};

__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// The random bits of a block of eight elements.
struct DropBits {
    uint32_t w[4];
    __device__ __forceinline__ DropBits(const DropKey& key, uint32_t step, int64_t block) {
        const uint4 r = philox(make_uint4((uint32_t)block, (uint32_t)((uint64_t)block >> 32), key.call, step), key.seed[0], key.seed[1]);
        w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    }
    __device__ __forceinline__ bool keep(int e, uint32_t limit) const { return ((w[e >> 1] >> (16 * (e & 1))) & 0xffffu) >= limit; }
};

__device__ __forceinline__ uint32_t drop_step(const DropKey& key) {
    return (uint32_t)(key.step + (key.step_at ? *key.step_at : 0));
}

// Element e of a block: dropped ones count nothing, whatever they hold.
template <bool kAdd>
__device__ __forceinline__ float drop(const DropBits& bits, int e, const DropKey& key, float h, float r) {
    if (!bits.keep(e, key.limit)) return kAdd ? r : 0.f;
    return kAdd ? fmaf(h, key.factor, r) : h * key.factor;
}

// Whole blocks of contiguous elements at 16-byte boundaries, the last one element by element.  A thread takes U blocks.
template <typename T, bool kAdd, int U>
__global__ void __launch_bounds__(kDropThreads) drop_flat(int64_t n, DropKey key, const T* __restrict__ h, const T* __restrict__ r,
                                                          T* __restrict__ y) {
    constexpr int V = kVec<T>, N = kDropBlock / V;
    pdl_wait();
    pdl_trigger();
    const uint32_t step = drop_step(key);
    const int64_t first = (int64_t)blockIdx.x * (U * kDropThreads) + threadIdx.x;
    uint4 a[U][N], b[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e0 = (first + u * kDropThreads) * kDropBlock;
        if (e0 + kDropBlock > n) continue;
#pragma unroll
        for (int q = 0; q < N; ++q) {
            a[u][q] = ld_piece(h + e0 + q * V);
            if (kAdd) b[u][q] = ld_piece(r + e0 + q * V);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t block = first + u * kDropThreads, e0 = block * kDropBlock;
        if (e0 >= n) return;
        const DropBits bits(key, step, block);
        if (e0 + kDropBlock <= n) {
#pragma unroll
            for (int q = 0; q < N; ++q) {
                float f[V], g[V] = {};
                unpack<T>(a[u][q], f);
                if (kAdd) unpack<T>(b[u][q], g);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = drop<kAdd>(bits, q * V + i, key, f[i], g[i]);
                st_piece(y + e0 + q * V, pack<T>(f));
            }
        } else {
            for (int e = 0; e0 + e < n; ++e)
                y[e0 + e] = from_f32<T>(drop<kAdd>(bits, e, key, to_f32(h[e0 + e]), kAdd ? to_f32(r[e0 + e]) : 0.f));
        }
    }
}

// Rows at strides, or bases off 16-byte boundaries: a thread for a block, element by element.
template <typename T, bool kAdd>
__global__ void __launch_bounds__(kDropThreads) drop_rows(int64_t n, int32_t C, DropKey key, const T* __restrict__ h, int64_t h_ld,
                                                          const T* __restrict__ r, int64_t r_ld, T* __restrict__ y, int64_t y_ld) {
    pdl_wait();
    pdl_trigger();
    const uint32_t step = drop_step(key);
    const int64_t block = (int64_t)blockIdx.x * kDropThreads + threadIdx.x, e0 = block * kDropBlock;
    if (e0 >= n) return;
    const DropBits bits(key, step, block);
    int64_t row = e0 / C;
    int32_t col = (int32_t)(e0 - row * C);
    float a[kDropBlock], b[kDropBlock];
    int64_t to[kDropBlock];
#pragma unroll
    for (int e = 0; e < kDropBlock; ++e) {
        to[e] = -1;
        if (e0 + e < n) {
            a[e] = to_f32(h[row * h_ld + col]);
            b[e] = kAdd ? to_f32(r[row * r_ld + col]) : 0.f;
            to[e] = row * y_ld + col;
        }
        if (++col == C) col = 0, ++row;
    }
#pragma unroll
    for (int e = 0; e < kDropBlock; ++e)
        if (to[e] >= 0) y[to[e]] = from_f32<T>(drop<kAdd>(bits, e, key, a[e], b[e]));
}

template <typename T, bool kAdd>
void drop_launch(int64_t M, int32_t C, const DropKey& key, const void* h, int64_t h_ld, const void* r, int64_t r_ld, void* y, int64_t y_ld,
                 cudaStream_t s) {
    const int64_t n = M * C, blocks = (n + kDropBlock - 1) / kDropBlock;
    const T *hp = static_cast<const T*>(h), *rp = static_cast<const T*>(r);
    T* yp = static_cast<T*>(y);
    auto grid = [&](int64_t per) { return dim3((unsigned)((blocks + per * kDropThreads - 1) / (per * kDropThreads))); };
    if (!(h_ld == C && r_ld == C && y_ld == C && aligned16(h) && aligned16(r) && aligned16(y)))
        launch(drop_rows<T, kAdd>, grid(1), dim3(kDropThreads), 0, s, n, C, key, hp, h_ld, rp, r_ld, yp, y_ld);
    else if (blocks < (int64_t)num_sms() * 16 * kDropThreads)
        launch(drop_flat<T, kAdd, 1>, grid(1), dim3(kDropThreads), 0, s, n, key, hp, rp, yp);
    else   // two blocks a thread where every SM has more than its fill: 32768 x 2048 bf16 with a residual 61 -> 56 us
        launch(drop_flat<T, kAdd, 2>, grid(2), dim3(kDropThreads), 0, s, n, key, hp, rp, yp);
}

}  // namespace
}  // namespace zs

extern "C" zs_status zs_dropout(int32_t dtype, const void* h, int64_t h_ld, const void* residual, int64_t residual_ld, int64_t M,
                                int32_t C, double p, uint64_t seed, uint32_t call, int64_t step, const int64_t* step_at, void* y,
                                int64_t y_ld, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_dropout";
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (M < 0 || C < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld C=%d", fn, (long long)M, C);
    if (M > kMaxRows || C > kMaxRows || M * C >= ((int64_t)1 << 41))
        return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld or C=%d is above 2^31 - 2^16, or M * C not below 2^41", fn, (long long)M, C);
    if (!(p >= 0.0 && p <= 1.0)) return fail(ZS_ERR_INVALID_ARG, "%s: p=%g is outside [0, 1]", fn, p);
    if (M == 0) return ZS_OK;
    if (zs_status st = check_rows(fn, "h", dtype, h, h_ld, M, C)) return st;
    if (residual)
        if (zs_status st = check_rows(fn, "residual", dtype, residual, residual_ld, M, C)) return st;
    if (zs_status st = check_rows(fn, "y", dtype, y, y_ld, M, C)) return st;
    if (reinterpret_cast<uintptr_t>(step_at) & 7) return fail(ZS_ERR_INVALID_ARG, "%s: step_at is not 8-byte aligned", fn);
    if (M < 2) h_ld = y_ld = residual_ld = C;
    if (!residual) residual_ld = C;
    DropKey key = {};
    key.seed[0] = (uint32_t)seed, key.seed[1] = (uint32_t)(seed >> 32);
    key.call = call, key.step = step, key.step_at = step_at;
    key.limit = (uint32_t)nearbyint(p * 65536.0);
    key.factor = key.limit < 65536u ? (float)(65536.0 / (65536.0 - key.limit)) : 0.f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        if (residual) drop_launch<T, true>(M, C, key, h, h_ld, residual, residual_ld, y, y_ld, s);
        else drop_launch<T, false>(M, C, key, h, h_ld, residual, residual_ld, y, y_ld, s);
    };
    if (dtype == ZS_F32) go(float());
    else if (dtype == ZS_BF16) go(__nv_bfloat16());
    else go(__half());
    return check_launch(fn);
}
