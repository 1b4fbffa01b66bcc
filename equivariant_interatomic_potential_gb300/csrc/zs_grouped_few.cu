// Grouped products over few rows: what counts is that the weights stream by.
//
// With a handful of rows a group, a tile of 128 rows on the tensor cores is
// mostly empty and its loads come one stage after another.  Here each weight
// is read once, straight into registers, by as many warps as there are pieces
// of the weights to read, and multiplied with up to eight rows held as fp32 in
// shared memory.  Bound by HBM (the weights') until a group has more than
// eight rows, for which its weights are read again, from L2.
#include <type_traits>

#include "zs_grouped.cuh"
#include "zs_types.cuh"

namespace zs {

namespace {

constexpr int kFewRows = 8;        // rows of a pass
constexpr int kFewChunk = 1024;    // summed-over elements of the rows held at a time

struct FewArgs {
    const void* a;      // the rows' operand (x, or dy)
    int64_t a_ld;
    const void* b;      // the weights, or (weight gradient) x
    int64_t b_ld;
    void* out;
    int64_t out_ld;
    const int32_t* row_ptr;
    const int32_t* perm;
    int M, K, N, G;
};

__device__ __forceinline__ int start(const FewArgs& a, int g) {
    if (g > a.G) return a.M;
    const int v = __ldg(a.row_ptr + g);
    return v < 0 ? 0 : v > a.M ? a.M : v;
}
__device__ __forceinline__ int row_at(const FewArgs& a, int p, int e) {
    if (p >= e) return -1;
    const int r = a.perm ? __ldg(a.perm + p) : p;
    return (uint32_t)r < (uint32_t)a.M ? r : -1;
}
// Rows of no group: zeros in columns [c0, c1).
template <typename T>
__device__ __forceinline__ void clear_rows(const FewArgs& a, int b, int e, int c0, int c1) {
    const int w = c1 - c0;
    for (int64_t i = threadIdx.x; i < (int64_t)(e - b) * w; i += blockDim.x) {
        const int r = row_at(a, b + (int)(i / w), e);
        if (r >= 0) static_cast<T*>(a.out)[r * a.out_ld + c0 + i % w] = from_f32<T>(0.f);
    }
}
// Columns [c0, c0 + n) of R rows as fp32, rows kFewChunk apart.  Eight loads a
// thread are on their way at once.
template <typename T, int R>
__device__ __forceinline__ void hold_rows(float* to, const void* from, int64_t ld, const int* rows, int c0, int n) {
    const int all = R * n;
    for (int i0 = threadIdx.x; i0 < all; i0 += 8 * blockDim.x) {
        T v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = imin(i0 + j * (int)blockDim.x, all - 1), r = i / n;
            v[j] = static_cast<const T*>(from)[imax(rows[r], 0) * ld + c0 + (i - r * n)];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * (int)blockDim.x, r = i / n;
            if (i < all) to[r * kFewChunk + (i - r * n)] = rows[r] >= 0 ? to_f32(v[j]) : 0.f;
        }
    }
}
// V consecutive elements as fp32.
template <typename T, int V>
__device__ __forceinline__ void read(const T* p, float (&f)[V]) {
    if constexpr (V == 1) f[0] = to_f32(__ldg(p));
    else unpack<T>(__ldg(reinterpret_cast<const uint4*>(p)), f);
}

// f(std::integral_constant<int, R>) with R the smallest of 1, 2, 4 and 8 that holds n rows.
template <typename F>
__device__ __forceinline__ void with_rows(int n, F&& f) {
    if (n > 4) f(std::integral_constant<int, 8>());
    else if (n > 2) f(std::integral_constant<int, 4>());
    else if (n > 1) f(std::integral_constant<int, 2>());
    else f(std::integral_constant<int, 1>());
}

// y: a warp takes four columns of y (rows of w), its lanes go along K.
constexpr int kFwdCols = 32;
template <typename T, int V>
__global__ void __launch_bounds__(256) few_forward(const FewArgs a) {
    __shared__ __align__(16) float xs[kFewRows * kFewChunk];
    __shared__ int rows[kFewRows];
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.y, b = start(a, g), e = start(a, g + 1), c0 = blockIdx.x * kFwdCols;
    if (b >= e) return;
    if (g == a.G) return clear_rows<T>(a, b, e, c0, imin(c0 + kFwdCols, a.N));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n0 = c0 + 4 * warp;
    const T* w = static_cast<const T*>(a.b) + ((int64_t)g * a.N + n0) * a.K;
    const int cols = imin(4, a.N - n0);
    for (int p = b; p < e; p += kFewRows) {
        __syncthreads();
        if (threadIdx.x < kFewRows) rows[threadIdx.x] = row_at(a, p + threadIdx.x, e);
        with_rows(e - p, [&](auto r_) {
            constexpr int R = decltype(r_)::value;
            float acc[4][R] = {};
            for (int k0 = 0; k0 < a.K; k0 += kFewChunk) {
                const int n = imin(kFewChunk, a.K - k0);
                __syncthreads();
                hold_rows<T, R>(xs, a.a, a.a_ld, rows, k0, n);
                __syncthreads();
                for (int k = lane * V; k < n; k += 32 * V) {
                    float f[4][V];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c < cols) {
                            read<T, V>(w + (int64_t)c * a.K + k0 + k, f[c]);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; ++i) f[c][i] = 0.f;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float x[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) x[i] = xs[r * kFewChunk + k + i];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[c][r] = fmaf(f[c][i], x[i], acc[c][r]);
                    }
                }
            }
            float mine = 0.f;   // lane c R + r ends with column c of row r
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float v = acc[c][r];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane == c * R + r) mine = v;
                }
            const int c = lane / R, r = lane % R;
            if (c < cols && rows[r] >= 0) static_cast<T*>(a.out)[rows[r] * a.out_ld + n0 + c] = from_f32<T>(mine);
        });
    }
}

// dx: kLanes lanes go along K; the rows of w (the sum's elements) are shared by
// the other lanes and the warps of a CTA, and by the CTAs of a cluster, which
// add their parts through distributed shared memory.  Eight lanes (128 bytes of a
// row) give four times the CTAs, for one or a few groups.
constexpr int kDxWarps = 8, kDxCluster = 8;
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <typename T, int V, int kLanes>
__global__ void __launch_bounds__(32 * kDxWarps) few_dx(const FewArgs a) {
    constexpr int kCols = kLanes * V, kShares = kDxWarps * (32 / kLanes);   // columns; threads that share them
    __shared__ float dys[kFewRows * kFewChunk];
    __shared__ float sum[kFewRows][kCols];
    __shared__ int rows[kFewRows];
    float* part = dys;   // [kShares][kCols], once the sums are done
    static_assert(kShares * kCols <= kFewRows * kFewChunk, "the parts fit");
    pdl_wait();
    pdl_trigger();
    const int ctas = gridDim.z, rank = blockIdx.z;
    const int g = blockIdx.y, b = start(a, g), e = start(a, g + 1), c0 = blockIdx.x * kCols;
    if (b >= e) return;                // the whole cluster
    if (g == a.G) {
        if (rank == 0) clear_rows<T>(a, b, e, c0, imin(c0 + kCols, a.K));
        return;
    }
    const int share = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, c = c0 + lane * V;
    const T* w = static_cast<const T*>(a.b) + (int64_t)g * a.N * a.K + c;
    const int per = (a.N + ctas - 1) / ctas, first = rank * per, last = imin(first + per, a.N);
    for (int p = b; p < e; p += kFewRows) {
        __syncthreads();
        if (threadIdx.x < kFewRows) rows[threadIdx.x] = row_at(a, p + threadIdx.x, e);
        with_rows(e - p, [&](auto r_) {
            constexpr int R = decltype(r_)::value;
            float acc[R][V] = {};
            for (int n0 = first; n0 < last; n0 += kFewChunk) {
                const int n = imin(kFewChunk, last - n0);
                __syncthreads();
                hold_rows<T, R>(dys, a.a, a.a_ld, rows, n0, n);
                __syncthreads();
                if (c < a.K) {
                    constexpr int kAtOnce = 8;   // rows of w on their way
                    for (int i0 = share; i0 < n; i0 += kShares * kAtOnce) {
                        float f[kAtOnce][V];
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u)
                            read<T, V>(w + (int64_t)(n0 + imin(i0 + u * kShares, n - 1)) * a.K, f[u]);
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u) {
                            const int i = i0 + u * kShares;
                            if (i >= n) break;
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int j = 0; j < V; ++j) acc[r][j] = fmaf(f[u][j], dys[r * kFewChunk + i], acc[r][j]);
                        }
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < V; ++j) part[share * kCols + lane * V + j] = acc[r][j];
                __syncthreads();
                for (int j = threadIdx.x; j < kCols; j += blockDim.x) {
                    float v = 0.f;
#pragma unroll
                    for (int i = 0; i < kShares; ++i) v += part[i * kCols + j];
                    sum[r][j] = v;
                }
            }
            if (ctas > 1) cluster_barrier();
            else __syncthreads();
            // the CTAs' sums in order: each writes its share of the row's columns
            for (int i = rank * blockDim.x + threadIdx.x; i < R * kCols; i += ctas * blockDim.x) {
                const int r = i / kCols, j = i % kCols;
                float v = 0.f;
                if (ctas == 1) {
                    v = sum[r][j];
                } else {
                    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&sum[r][j]);
                    for (int o = 0; o < ctas; ++o) {
                        uint32_t there;
                        float x;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(o));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
                        v += x;
                    }
                }
                if (c0 + j < a.K && rows[r] >= 0) static_cast<T*>(a.out)[rows[r] * a.out_ld + c0 + j] = from_f32<T>(v);
            }
            if (ctas > 1) cluster_barrier();   // no CTA goes on, or leaves, while another reads its sums
        });
    }
}

// dw: a warp takes eight rows of dw, its lanes go along K; the rows of the
// group pass by through shared memory.
constexpr int kDwWarpRows = 8, kDwRows = 8 * kDwWarpRows, kHeld = 8;
template <typename T, int V>
__global__ void __launch_bounds__(256) few_dw(const FewArgs a, bool x_wide) {
    constexpr int kCols = 32 * V;
    __shared__ __align__(16) float xs[kHeld][kCols];
    __shared__ __align__(16) float dys[kHeld][kDwRows];
    __shared__ int rows[kHeld];
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.z, b = start(a, g), e = start(a, g + 1);
    const int k0 = blockIdx.x * kCols, n0 = blockIdx.y * kDwRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float acc[kDwWarpRows][V] = {};
    for (int p = b; p < e; p += kHeld) {
        __syncthreads();
        if (threadIdx.x < kHeld) rows[threadIdx.x] = row_at(a, p + threadIdx.x, e);
        __syncthreads();
        const int held = imin(kHeld, e - p);
        if (V > 1 && x_wide) {
            for (int i = threadIdx.x; i < held * 32; i += blockDim.x) {
                const int row = rows[i / 32], k = k0 + i % 32 * V;
                float f[V] = {};
                if (row >= 0 && k < a.K) read<T, V>(static_cast<const T*>(a.b) + row * a.b_ld + k, f);
#pragma unroll
                for (int j = 0; j < V; ++j) xs[i / 32][i % 32 * V + j] = f[j];
            }
        } else {
#pragma unroll 4
            for (int i = threadIdx.x; i < held * kCols; i += blockDim.x) {
                const int row = rows[i / kCols], k = k0 + i % kCols;
                xs[i / kCols][i % kCols] = row >= 0 && k < a.K ? to_f32(static_cast<const T*>(a.b)[row * a.b_ld + k]) : 0.f;
            }
        }
#pragma unroll 2
        for (int i = threadIdx.x; i < held * kDwRows; i += blockDim.x) {
            const int row = rows[i / kDwRows], n = n0 + i % kDwRows;
            dys[i / kDwRows][i % kDwRows] = row >= 0 && n < a.N ? to_f32(static_cast<const T*>(a.a)[row * a.a_ld + n]) : 0.f;
        }
        __syncthreads();
        for (int r = 0; r < held; ++r) {
            float x[V], d[kDwWarpRows];
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = xs[r][lane * V + j];
#pragma unroll
            for (int i = 0; i < kDwWarpRows; ++i) d[i] = dys[r][kDwWarpRows * warp + i];
#pragma unroll
            for (int i = 0; i < kDwWarpRows; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[i][j] = fmaf(d[i], x[j], acc[i][j]);
        }
    }
    const int k = k0 + lane * V;
    if (k >= a.K) return;
#pragma unroll
    for (int i = 0; i < kDwWarpRows; ++i) {
        const int n = n0 + kDwWarpRows * warp + i;
        if (n >= a.N) break;
        T* out = static_cast<T*>(a.out) + ((int64_t)g * a.N + n) * a.K + k;
        if constexpr (V == 1) out[0] = from_f32<T>(acc[i][0]);
        else st_piece(out, pack<T>(acc[i]));
    }
}

template <typename T, int V>
zs_status launch_few(const char* fn, const FewArgs& a, int which, cudaStream_t s) {
    auto up = [](int x, int y) { return (unsigned)((x + y - 1) / y); };
    if (which == 0) {
        launch(few_forward<T, V>, dim3(up(a.N, kFwdCols), a.G + 1), dim3(256), 0, s, a);
    } else if (which == 1) {
        // a cluster shares the sum where there are too few CTAs to read the weights with
        const bool narrow = (int64_t)up(a.K, 32 * V) * a.G < 304;
        const unsigned tiles = up(a.K, (narrow ? 8 : 32) * V);
        const unsigned ctas = (int64_t)tiles * a.G < 304 && a.N >= 256 ? kDxCluster : 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles, a.G + 1, ctas);
        cfg.blockDim = dim3(32 * kDxWarps);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = ctas;
        cfg.attrs = attr;
        cfg.numAttrs = ctas > 1 ? 2 : 1;
        cudaLaunchKernelEx(&cfg, narrow ? few_dx<T, V, 8> : few_dx<T, V, 32>, a);
    } else {
        launch(few_dw<T, V>, dim3(up(a.K, 32 * V), up(a.N, kDwRows), a.G), dim3(256), 0, s, a,
               aligned16(a.b) && a.b_ld % kVec<T> == 0);
    }
    return check_launch(fn);
}

template <typename T>
zs_status few(const char* fn, const FewArgs& a, int which, cudaStream_t s) {
    // 16 bytes of a row of the weights (or of their gradient) at a time where its rows allow it
    const void* rows = which == 2 ? a.out : a.b;
    if (aligned16(rows) && a.K % kVec<T> == 0) return launch_few<T, kVec<T>>(fn, a, which, s);
    return launch_few<T, 1>(fn, a, which, s);
}

}  // namespace

// Measured against the tensor-core kernels (us, few / tensor): M = 1, 2048 -> 4096 bf16: y 6.5 / 34, dx 7.9 / 59, dw 5.8 / 12;
// M = 8, 3 groups of 264 -> 2000 fp16: y 5.3 / 7.4, dx 6.8 / 23, dw 4.0 / 7.2; M = 16, 8 groups of 1024 -> 4096 bf16: 22 / 14,
// 45 / 32, 16 / 32; M = 64: 55 / 15, 82 / 32, 31 / 33; M = 24, one group of 143 -> 1264 fp32: 9.9 / 13, 16 / 72, 6 / 9;
// M = 144, 57 groups of 1680 -> 264 fp32: 84 / 106, 69 / 93, 26 / 91, bf16: 71 / 26, 67 / 15, 20 / 38; M = 512, 89 groups of
// 256 -> 256 fp32: 54 / 30, 66 / 30, 29 / 25, bf16 dw 34 / 15.
bool grouped_is_few(int32_t dtype, int which, int64_t M, int32_t N, int32_t G) {
    if (G >= 65535 || N > 65535 * kDwRows) return false;   // of a grid's sides
    if (which == 2) return M <= 32 || M <= 4 * (int64_t)G;
    return M <= kFewRows || (dtype == ZS_F32 && (M <= 4 * kFewRows || (M <= 256 && M <= 4 * (int64_t)G)));
}

zs_status grouped_few(const char* fn, int32_t dtype, int which, const void* a, int64_t a_ld, const void* b, int64_t b_ld,
                      const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out,
                      int64_t out_ld, cudaStream_t s) {
    const FewArgs f{a, a_ld, b, b_ld, out, out_ld, row_ptr, perm, (int)M, K, N, G};
    switch (dtype) {
        case ZS_F32: return few<float>(fn, f, which, s);
        case ZS_BF16: return few<__nv_bfloat16>(fn, f, which, s);
        default: return few<__half>(fn, f, which, s);
    }
}

}  // namespace zs
