// Grouped products over rows of up to 32 elements on both sides, on the CUDA
// cores: the weights of a group fit shared memory whole, a tile takes one load
// and one store of each row, and many small CTAs have all of them on their way
// at once, which is what such products wait for.  4 x 4 results a thread.
// 65536 rows in 16 groups, fp32: y in 9 us where the tensor cores take 16 (they
// are the faster ones from rows of 64 on).
#include "zs_grouped.cuh"
#include "zs_grouped_walk.cuh"

namespace zs {

namespace {

constexpr int kThreads = 256;
constexpr int kMost = 32;          // elements of a row, on either side
constexpr int kTileRows = 128;         // of a tile
constexpr int kStride = kMost + 4;

struct SmallArgs {
    const void* a;
    int64_t a_ld;
    const void* w;
    void* out;
    int64_t out_ld;
    const int32_t* row_ptr;
    const int32_t* perm;
    int M, G, red, cols;
    bool a_wide, out_wide;         // four elements at a time
};

// Four consecutive elements as fp32 and back (8 or 16 bytes).
template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T v[4];
};
template <typename T>
__device__ __forceinline__ float4 open4(const Four<T>& q) {
    return make_float4(to_f32(q.v[0]), to_f32(q.v[1]), to_f32(q.v[2]), to_f32(q.v[3]));
}

// out = a w^T (w rows as long as the sum, kT false) or a w (kT true).
template <typename T, bool kT>
__global__ void __launch_bounds__(kThreads) small_rows(const SmallArgs a) {
    __shared__ __align__(16) float xs[kTileRows][kStride];
    __shared__ __align__(16) float ws[kMost][kStride];   // [summed-over][column]
    __shared__ int rows[kTileRows];
    pdl_wait();
    pdl_trigger();
    const Groups<kTileRows, 1> gr{a.row_ptr, a.G, a.M, false};
    const int g = gr.find(blockIdx.x, a.G + 1);
    const int b = gr.start(g), e = gr.start(g + 1);
    const int64_t p0 = b + (int64_t)((int)blockIdx.x - (b / kTileRows + g)) * kTileRows;
    if (p0 >= e) return;
    const int n = (int)imin<int64_t>(kTileRows, e - p0);
    if (threadIdx.x < kTileRows) {
        int r = -1;
        if ((int)threadIdx.x < n) {
            r = a.perm ? __ldg(a.perm + p0 + threadIdx.x) : (int)p0 + (int)threadIdx.x;
            if ((uint32_t)r >= (uint32_t)a.M) r = -1;
        }
        rows[threadIdx.x] = r;
    }
    const bool none = g == a.G;
    const int red4 = (a.red + 3) / 4 * 4;
    // the group's weights, while the rows' numbers are on their way
    if (!none) {
        const T* w = static_cast<const T*>(a.w) + (int64_t)g * a.red * a.cols;
        const int all = a.red * a.cols, inner = kT ? a.cols : a.red;
        for (int i0 = threadIdx.x; i0 < all; i0 += 4 * kThreads) {
            T v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(w + imin(i0 + j * kThreads, all - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * kThreads, outer = i / inner, in = i - outer * inner;
                if (i < all) ws[kT ? outer : in][kT ? in : outer] = to_f32(v[j]);
            }
        }
        for (int i = threadIdx.x; i < (red4 - a.red) * kMost; i += kThreads) ws[a.red + i / kMost][i % kMost] = 0.f;
    }
    __syncthreads();
    if (!none) {
        if (a.a_wide) {
            const int quads = a.red / 4, all = n * quads;
            for (int i0 = threadIdx.x; i0 < all; i0 += 4 * kThreads) {
                Four<T> v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = imin(i0 + j * kThreads, all - 1), r = i / quads;
                    v[j] = *reinterpret_cast<const Four<T>*>(static_cast<const T*>(a.a) + imax(rows[r], 0) * a.a_ld + 4 * (i - r * quads));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * kThreads, r = i / quads;
                    if (i < all) *reinterpret_cast<float4*>(&xs[r][4 * (i - r * quads)]) = open4(v[j]);
                }
            }
        } else {
            const int all = n * red4;
            for (int i0 = threadIdx.x; i0 < all; i0 += 8 * kThreads) {
                T v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = imin(i0 + j * kThreads, all - 1), r = i / red4;
                    v[j] = static_cast<const T*>(a.a)[imax(rows[r], 0) * a.a_ld + imin(i - r * red4, a.red - 1)];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + j * kThreads, r = i / red4, c = i - r * red4;
                    if (i < all) xs[r][c] = c < a.red ? to_f32(v[j]) : 0.f;
                }
            }
        }
    }
    __syncthreads();
    const int tx = threadIdx.x % (kMost / 4), ty = threadIdx.x / (kMost / 4);
    float acc[4][4] = {};
    if (!none) {
        for (int k = 0; k < red4; k += 4) {
            float4 x[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = *reinterpret_cast<const float4*>(&xs[4 * ty + i][k]);
                w[i] = *reinterpret_cast<const float4*>(&ws[k + i][4 * tx]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xv[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[i][0] = fmaf(xv[q], w[q].x, acc[i][0]);
                    acc[i][1] = fmaf(xv[q], w[q].y, acc[i][1]);
                    acc[i][2] = fmaf(xv[q], w[q].z, acc[i][2]);
                    acc[i][3] = fmaf(xv[q], w[q].w, acc[i][3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = rows[4 * ty + i], c = 4 * tx;
        if (r < 0) continue;
        T* out = static_cast<T*>(a.out) + r * a.out_ld + c;
        if (a.out_wide && c + 4 <= a.cols) {
            Four<T> q;
#pragma unroll
            for (int j = 0; j < 4; ++j) q.v[j] = from_f32<T>(acc[i][j]);
            *reinterpret_cast<Four<T>*>(out) = q;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.cols) out[j] = from_f32<T>(acc[i][j]);
        }
    }
}

template <typename T>
zs_status rows_of(const char* fn, const SmallArgs& a, bool transposed, cudaStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.M / kTileRows + a.G + 2));
    if (transposed) launch(small_rows<T, true>, grid, dim3(kThreads), 0, s, a);
    else launch(small_rows<T, false>, grid, dim3(kThreads), 0, s, a);
    return check_launch(fn);
}

// dw[g] = sum of dy^T x over the positions of a CTA's units: chunks of kHeld rows
// pass through shared memory (the next one's elements and the one after's row
// numbers on their way in registers), 4 x 4 results a thread; four groups of
// threads share the rows and add their sums at the end.
constexpr int kHeld = 32, kShares = 4, kPer = kThreads / kShares;
__global__ void __launch_bounds__(kThreads) small_weights(const WeightArgs a) {
    constexpr int kLoads = kHeld * kMost / kThreads;
    __shared__ __align__(16) float xs[kHeld][kStride], dys[kHeld][kStride];
    __shared__ __align__(16) float sums[kPer * 16 * 2];
    __shared__ int rows[2][kHeld];
    __shared__ int32_t starts[kGroupsHeld + 2];
    pdl_wait();
    pdl_trigger();
    WeightGroups<float> gr;
    gr.hold(a.row_ptr, a.G, a.M, starts);
    __syncthreads();
    if (threadIdx.x >= kThreads - 32) note_join<float>(a, gr);
    Walk<float, kMost> walk(a, gr);
    const int tx = threadIdx.x % 8, ty = threadIdx.x / 8 % 8, share = threadIdx.x / kPer;
    Segment s;
    while (walk.next(s)) {
        float acc[4][4] = {};
        float xv[kLoads], dv[kLoads];
        auto number = [&](int p) {
            return threadIdx.x < kHeld && p + (int)threadIdx.x < s.p1 ? weight_row(a, p + threadIdx.x) : -1;
        };
        auto fetch = [&](int buf) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int i = threadIdx.x + j * kThreads, r = imax(rows[buf][i / kMost], 0), c = i % kMost;
                xv[j] = static_cast<const float*>(a.x.p)[r * a.x.ld + imin(c, a.K - 1)];
                dv[j] = static_cast<const float*>(a.dy.p)[r * a.dy.ld + imin(c, a.N - 1)];
            }
        };
        int buf = 0, ahead = number(s.p0);
        __syncthreads();
        if (threadIdx.x < kHeld) rows[0][threadIdx.x] = ahead;
        ahead = number(s.p0 + kHeld);
        __syncthreads();
        if (s.p0 < s.p1) fetch(0);
        for (int p = s.p0; p < s.p1; p += kHeld, buf ^= 1) {
            if (threadIdx.x < kHeld) rows[buf ^ 1][threadIdx.x] = ahead;
            ahead = number(p + 2 * kHeld);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int i = threadIdx.x + j * kThreads, r = i / kMost, c = i % kMost;
                const bool in = rows[buf][r] >= 0;
                xs[r][c] = in ? xv[j] : 0.f;
                dys[r][c] = in ? dv[j] : 0.f;
            }
            __syncthreads();
            if (p + kHeld < s.p1) fetch(buf ^ 1);
#pragma unroll
            for (int r = share; r < kHeld; r += kShares) {
                const float4 x = *reinterpret_cast<const float4*>(&xs[r][4 * tx]);
                const float4 d = *reinterpret_cast<const float4*>(&dys[r][4 * ty]);
                const float dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][0] = fmaf(dd[i], x.x, acc[i][0]);
                    acc[i][1] = fmaf(dd[i], x.y, acc[i][1]);
                    acc[i][2] = fmaf(dd[i], x.z, acc[i][2]);
                    acc[i][3] = fmaf(dd[i], x.w, acc[i][3]);
                }
            }
            __syncthreads();
        }
        for (int step = kShares / 2; step > 0; step /= 2) {   // the shares' sums, in a fixed order
            float* mine = sums + (share % step * kPer + threadIdx.x % kPer) * 16;
            if (share >= step && share < 2 * step) {
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[i] = acc[i / 4][i % 4];
            }
            __syncthreads();
            if (share < step) {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] += mine[i];
            }
            __syncthreads();
        }
        if (share == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 4 * ty + i, k = 4 * tx;
                if (n >= a.N) continue;
                float* out = static_cast<float*>(a.dw) + ((int64_t)s.g * a.N + n) * a.K + k;
                float* part = a.partial + (((int64_t)blockIdx.x * 2 + s.part) * kTileM + n) * kMost + k;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k + j >= a.K) continue;
                    (s.whole ? out : part)[j] = acc[i][j];
                }
            }
        }
    }
}

}  // namespace

bool grouped_is_small(int32_t K, int32_t N) { return K <= kMost && N <= kMost; }

zs_status grouped_small_rows(const char* fn, int32_t dtype, int which, const void* a, int64_t a_ld, const void* w,
                             const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out,
                             int64_t out_ld, cudaStream_t s) {
    const int red = which ? N : K, cols = which ? K : N, bytes = 4 * dtype_bytes(dtype);
    auto fours = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld % 4 == 0 || M == 1); };
    if (M / kTileRows + G + 2 >= (int64_t(1) << 31)) return fail(ZS_ERR_INVALID_ARG, "%s: %lld rows in %d groups", fn, (long long)M, G);
    const SmallArgs f{a, a_ld, w, out, out_ld, row_ptr, perm, (int)M, G, red, cols, fours(a, a_ld) && red % 4 == 0, fours(out, out_ld)};
    switch (dtype) {
        case ZS_F32: return rows_of<float>(fn, f, which != 0, s);
        case ZS_BF16: return rows_of<__nv_bfloat16>(fn, f, which != 0, s);
        default: return rows_of<__half>(fn, f, which != 0, s);
    }
}

zs_status grouped_small_weights(const char* fn, const WeightArgs& a, int ctas, cudaStream_t s) {
    launch(small_weights, dim3(ctas), dim3(kThreads), 0, s, a);
    if (zs_status st = check_launch(fn)) return st;
    if (ctas > 1) {
        launch(weights_join<float, kMost>, dim3((a.cuts + kNotes - 1) / kNotes, kMost / kPartRows), dim3(256), 0, s, a);
        return check_launch(fn);
    }
    return ZS_OK;
}

}  // namespace zs
