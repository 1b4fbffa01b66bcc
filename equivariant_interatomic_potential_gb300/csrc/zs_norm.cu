// The norms around a block fused with its gate, residual scale and residual
// sum, and their backward:
//   nh = norm(h), t = nh * w_post, q = sigmoid(gate)
//   y = x + scale * q * t,  ny = norm(y),  u = ny * w_pre
// and for the cotangents dy, du
//   dny = du * w_pre,           dx = dy + norm'(dny; ny, ry)
//   dnh = dx * scale * q * w_post,  dh = norm'(dnh; nh, rh)
//   dgate = dx * scale * t * q (1 - q)
//   dw_post = sum_rows dx * scale * q * nh, dscale = sum_rows dx * q * t,
//   dw_pre = sum_rows du * ny
// with norm'(d; n, r) = r * (d - mean(d n) n), minus r * mean(d) for the
// layer norm.  The backward forms y again from x, h and the gate (as many
// bytes as reading y, and unrounded), and keeps only four floats a row.
//
// Bound by HBM.  A row lives in the registers of a power of two (8 to 512)
// threads, each holding up to NV pieces of VEC elements, so that every
// operand is read once; rows go round the CTAs of a persistent grid, which
// keep the parameters of their columns, and in the backward the running
// column sums, in registers (rows of more than 4096 channels: the parameters
// in L1, the sums in shared memory).  Each CTA writes its column sums once and a
// second kernel adds them in a fixed order.
#include "zs_types.cuh"

namespace zs {

namespace {

constexpr int kMaxC = 8192;
constexpr int kThreads = 256;     // of a CTA, unless a row takes more
constexpr int kBigThreads = 512;
constexpr int kBwdCtas = 304;     // two for each of the 152 SMs: rows of the partial column sums
constexpr int kSumCols = 32, kSumRows = 16;   // shape of the CTAs that add them

struct Shape {
    int64_t M;
    int32_t C;
    int32_t tpr;        // threads that hold a row
    int32_t gate_cols;  // 0, 1 or C
    int32_t layer;      // subtract the mean
    float eps, inv_c;
};

struct View {
    const void* p;
    int64_t ld;
};

// Elements of a thread: NV pieces of VEC, piece k at column (k * tpr + thread) * VEC.
template <typename T, int VEC, int NV>
struct Cols {
    static constexpr int E = VEC * NV;
    static_assert(VEC == 1 || VEC == kVec<T>, "whole 16-byte pieces or single elements");

    template <typename F>
    static __device__ __forceinline__ void each(int tpr, int lane, int C, F&& f) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = (k * tpr + lane) * VEC;
            if (c0 < C) f(k, c0);
        }
    }
    // A row as it travels: raw pieces, so that loads can be issued well before use.
    struct Raw {
        uint4 v[VEC == 1 ? 1 : NV];
        T s[VEC == 1 ? NV : 1];
    };
    static __device__ __forceinline__ void load(Raw& r, const T* row, int tpr, int lane, int C) {
        each(tpr, lane, C, [&](int k, int c0) {
            if constexpr (VEC == 1) r.s[k] = row[c0];
            else r.v[k] = ld_piece(row + c0);
        });
    }
    static __device__ __forceinline__ void open(const Raw& r, float (&f)[E], int tpr, int lane, int C) {
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = 0.f;
        each(tpr, lane, C, [&](int k, int) {
            if constexpr (VEC == 1) {
                f[k] = to_f32(r.s[k]);
            } else {
                float q[kVec<T>];
                unpack<T>(r.v[k], q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[k * VEC + i] = q[i];
            }
        });
    }
    static __device__ __forceinline__ void store(T* row, const float (&f)[E], int tpr, int lane, int C) {
        each(tpr, lane, C, [&](int k, int c0) {
            if constexpr (VEC == 1) {
                row[c0] = from_f32<T>(f[k]);
            } else {
                float q[kVec<T>];
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[i] = f[k * VEC + i];
                st_piece(row + c0, pack<T>(q));
            }
        });
    }
    static __device__ __forceinline__ void load_params(const float* p, float (&f)[E], int tpr, int lane, int C) {
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = 0.f;
        each(tpr, lane, C, [&](int k, int c0) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[k * VEC + i] = __ldg(p + c0 + i);
        });
    }
    // Zero beyond the row's end, so that sums over a thread's elements need no care.
    static __device__ __forceinline__ void clear_tail(float (&f)[E], int tpr, int lane, int C) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if ((k * tpr + lane) * VEC >= C) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[k * VEC + i] = 0.f;
            }
    }
};

// Sums over the threads of a row.  Rows of up to 32 threads stay within a
// warp; wider ones go through shared memory: `red` holds two rounds of a
// float4 per warp, taken in turn, so that one barrier a round is enough.
template <int NQ>
__device__ __forceinline__ void row_sum(float (&q)[NQ], int tpr, float4* red, int& round) {
    static_assert(NQ <= 4, "a float4 per warp");
    const int lim = tpr < 32 ? tpr : 32;
    for (int o = lim >> 1; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) q[i] += __shfl_xor_sync(0xffffffffu, q[i], o);
    }
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, per_row = tpr >> 5, first = warp / per_row * per_row;
    float4* slot = red + (round & 1) * 32;
    ++round;
    if ((threadIdx.x & 31) == 0) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float* ve = &v.x;
#pragma unroll
        for (int i = 0; i < NQ; ++i) ve[i] = q[i];
        slot[warp] = v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NQ; ++i) q[i] = 0.f;
    for (int w = 0; w < per_row; ++w) {
        const float4 v = slot[first + w];
        const float* ve = &v.x;
#pragma unroll
        for (int i = 0; i < NQ; ++i) q[i] += ve[i];
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __frcp_rn(1.f + expf(-z)); }

// Mean (layer norm) and 1/root of a row's values; zeroes the tail.  Two
// passes over the registers: the mean first, then the centred squares.
template <typename Co, int E>
__device__ __forceinline__ float2 row_stats(float (&v)[E], const Shape& s, int lane, float4* red, int& round) {
    float mean = 0.f;
    if (s.layer) {
        float a[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) a[0] += v[i];
        row_sum(a, s.tpr, red, round);
        mean = a[0] * s.inv_c;
    }
    float d[E];
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = v[i] - mean;
    if (s.layer) Co::clear_tail(d, s.tpr, lane, s.C);
    float a[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) a[0] = fmaf(d[i], d[i], a[0]);
    row_sum(a, s.tpr, red, round);
    return make_float2(mean, rsqrtf(fmaf(a[0], s.inv_c, s.eps)));
}

template <typename T, int VEC, int NV, bool kBig>
__global__ void __launch_bounds__(kBig ? kBigThreads : kThreads) norm_forward(Shape s, View h, View x, View gate,
                                                   const float* __restrict__ w_post, const float* __restrict__ scale,
                                                   const float* __restrict__ w_pre, T* y, T* u, float4* stats) {
    using Co = Cols<T, VEC, NV>;
    constexpr int E = Co::E;
    __shared__ float4 red[64];
    int round = 0;
    const int tpr = s.tpr, lane = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr, rows = blockDim.x / tpr;
    pdl_wait();
    pdl_trigger();
    float wp[E], sc[E], wr[E];
    auto params = [&] {
        Co::load_params(w_post, wp, tpr, lane, s.C);
        Co::load_params(scale, sc, tpr, lane, s.C);
        Co::load_params(w_pre, wr, tpr, lane, s.C);
    };
    if (!kBig) params();
    // every thread of the CTA goes round as often: the row sums may hold a barrier
    for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < s.M; r0 += (int64_t)gridDim.x * rows) {
        const bool live = r0 + sub < s.M;
        const int64_t r = live ? r0 + sub : s.M - 1;
        typename Co::Raw hr, xr, gr;
        Co::load(hr, static_cast<const T*>(h.p) + r * h.ld, tpr, lane, s.C);
        Co::load(xr, static_cast<const T*>(x.p) + r * x.ld, tpr, lane, s.C);
        const T* grow = static_cast<const T*>(gate.p) + r * gate.ld;
        float q_row = 1.f;
        if (s.gate_cols > 1) Co::load(gr, grow, tpr, lane, s.C);
        else if (s.gate_cols == 1) q_row = sigmoid(to_f32(grow[0]));
        if (kBig) params();
        float hv[E], yv[E];
        Co::open(hr, hv, tpr, lane, s.C);
        const float2 hs = row_stats<Co>(hv, s, lane, red, round);
        Co::open(xr, yv, tpr, lane, s.C);
        if (s.gate_cols > 1) {
            float z[E];
            Co::open(gr, z, tpr, lane, s.C);
#pragma unroll
            for (int i = 0; i < E; ++i)
                yv[i] = fmaf(sc[i] * sigmoid(z[i]), (hv[i] - hs.x) * hs.y * wp[i], yv[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) yv[i] = fmaf(sc[i] * q_row, (hv[i] - hs.x) * hs.y * wp[i], yv[i]);
        }
        const float2 ys = row_stats<Co>(yv, s, lane, red, round);
        if (!live) continue;
        Co::store(y + r * s.C, yv, tpr, lane, s.C);
#pragma unroll
        for (int i = 0; i < E; ++i) yv[i] = (yv[i] - ys.x) * ys.y * wr[i];
        Co::store(u + r * s.C, yv, tpr, lane, s.C);
        if (stats && lane == 0) stats[r] = make_float4(hs.x, hs.y, ys.x, ys.y);
    }
}

template <typename T, int VEC, int NV, bool kBig>
__global__ void __launch_bounds__(kBig ? kBigThreads : kThreads) norm_backward(Shape s, View dy, View du, View h, View x, View gate,
                                                   const float* __restrict__ w_post, const float* __restrict__ scale,
                                                   const float* __restrict__ w_pre, const float4* __restrict__ stats,
                                                   T* dh, T* dx, T* dgate, float* partial) {
    using Co = Cols<T, VEC, NV>;
    constexpr int E = Co::E;
    __shared__ float4 red[64];
    // [rows - 1][C]: the column sums of the CTA's other row groups; kBig: [3][C], the running sums
    extern __shared__ float cols[];
    int round = 0;
    const int tpr = s.tpr, lane = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr, rows = blockDim.x / tpr;
    pdl_wait();
    pdl_trigger();
    float wp[E], sc[E], wr[E], sums[kBig ? 1 : 3][E];
    auto params = [&] {
        Co::load_params(w_post, wp, tpr, lane, s.C);
        Co::load_params(scale, sc, tpr, lane, s.C);
        Co::load_params(w_pre, wr, tpr, lane, s.C);
    };
    if constexpr (kBig) {
        Co::each(tpr, lane, s.C, [&](int, int c0) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int w = 0; w < 3; ++w) cols[w * s.C + c0 + i] = 0.f;
        });
    } else {
        params();
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int i = 0; i < E; ++i) sums[w][i] = 0.f;
    }
    // adds a * b to column sum `which` (a thread owns its columns)
    auto add = [&](int which, const float (&a)[E], const float (&b)[E]) {
        if constexpr (kBig) {
            Co::each(tpr, lane, s.C, [&](int k, int c0) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float* c = cols + which * s.C + c0 + i;
                    *c = fmaf(a[k * VEC + i], b[k * VEC + i], *c);
                }
            });
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) sums[which][i] = fmaf(a[i], b[i], sums[which][i]);
        }
    };
    for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < s.M; r0 += (int64_t)gridDim.x * rows) {
        const bool live = r0 + sub < s.M;
        const int64_t r = live ? r0 + sub : s.M - 1;
        typename Co::Raw hr, xr, gr, dyr, dur;
        if (du.p) Co::load(dur, static_cast<const T*>(du.p) + r * du.ld, tpr, lane, s.C);
        Co::load(hr, static_cast<const T*>(h.p) + r * h.ld, tpr, lane, s.C);
        Co::load(xr, static_cast<const T*>(x.p) + r * x.ld, tpr, lane, s.C);
        const T* grow = static_cast<const T*>(gate.p) + r * gate.ld;
        float q_row = 1.f;
        if (s.gate_cols > 1) Co::load(gr, grow, tpr, lane, s.C);
        else if (s.gate_cols == 1) q_row = sigmoid(to_f32(grow[0]));
        if (dy.p) Co::load(dyr, static_cast<const T*>(dy.p) + r * dy.ld, tpr, lane, s.C);
        const float4 st = __ldg(stats + r);
        if (kBig) params();
        float nh[E], ny[E], q[E], d[E];
        Co::open(hr, nh, tpr, lane, s.C);
        Co::open(xr, ny, tpr, lane, s.C);
        if (s.gate_cols > 1) {
            Co::open(gr, q, tpr, lane, s.C);
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = sigmoid(q[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = q_row;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            nh[i] = (nh[i] - st.x) * st.y;
            ny[i] = (fmaf(sc[i] * q[i], nh[i] * wp[i], ny[i]) - st.z) * st.w;
        }
        if (du.p) Co::open(dur, d, tpr, lane, s.C);
        else {
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = 0.f;
        }
        if (live) add(2, d, ny);
        float a[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            d[i] *= wr[i];
            a[0] = fmaf(d[i], ny[i], a[0]);   // d is zero beyond the row's end
            a[1] += d[i];
        }
        row_sum(a, tpr, red, round);
        const float dn = a[0] * s.inv_c, dm = s.layer ? a[1] * s.inv_c : 0.f;
        float dxv[E];
        if (dy.p) Co::open(dyr, dxv, tpr, lane, s.C);
        else {
#pragma unroll
            for (int i = 0; i < E; ++i) dxv[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) dxv[i] = fmaf(st.w, d[i] - dm - dn * ny[i], dxv[i]);
        if (live) Co::store(dx + r * s.C, dxv, tpr, lane, s.C);
        Co::clear_tail(dxv, tpr, lane, s.C);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dxv[i] *= q[i];             // from here dx * q, then dx * q * scale
            ny[i] = nh[i] * wp[i];      // from here t, then the gate's gradient
        }
        if (live) add(1, dxv, ny);
#pragma unroll
        for (int i = 0; i < E; ++i) dxv[i] *= sc[i];
        if (live) add(0, dxv, nh);
        float b[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            ny[i] *= dxv[i] * (1.f - q[i]);
            d[i] = dxv[i] * wp[i];
            b[0] = fmaf(d[i], nh[i], b[0]);
            b[1] += d[i];
            b[2] += ny[i];
        }
        row_sum(b, tpr, red, round);
        const float hn = b[0] * s.inv_c, hm = s.layer ? b[1] * s.inv_c : 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = st.y * (d[i] - hm - hn * nh[i]);
        if (!live) continue;
        Co::store(dh + r * s.C, d, tpr, lane, s.C);
        if (s.gate_cols > 1) Co::store(dgate + r * s.C, ny, tpr, lane, s.C);
        else if (s.gate_cols == 1 && lane == 0) dgate[r] = from_f32<T>(b[2]);
    }
    // the CTA's column sums: its row groups' added in order
    float* mine = partial + (int64_t)blockIdx.x * 3 * s.C;
    if constexpr (kBig) {
        Co::each(tpr, lane, s.C, [&](int, int c0) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int w = 0; w < 3; ++w) mine[w * s.C + c0 + i] = cols[w * s.C + c0 + i];
        });
    } else {
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            if (rows > 1) __syncthreads();
            if (sub > 0)
                Co::each(tpr, lane, s.C, [&](int k, int c0) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) cols[(sub - 1) * s.C + c0 + i] = sums[w][k * VEC + i];
                });
            if (rows > 1) __syncthreads();
            if (sub == 0)
                Co::each(tpr, lane, s.C, [&](int k, int c0) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float total = sums[w][k * VEC + i];
                        for (int o = 0; o < rows - 1; ++o) total += cols[o * s.C + c0 + i];
                        mine[w * s.C + c0 + i] = total;
                    }
                });
        }
    }
}

// out[c] = sum over the CTAs' partial sums, in order: 16 threads a column,
// then their sums in order.
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_column_sums(const float* __restrict__ partial, int ctas, int32_t C,
                                                                       float* dw_post, float* dscale, float* dw_pre) {
    __shared__ float part[kSumRows][kSumCols];
    const int j = threadIdx.x % kSumCols, k = threadIdx.x / kSumCols;
    const int64_t col = (int64_t)blockIdx.x * kSumCols + j;   // of 3 C
    pdl_wait();
    pdl_trigger();
    float a = 0.f;
    if (col < 3 * (int64_t)C)
#pragma unroll 8
        for (int i = k; i < ctas; i += kSumRows) a += __ldg(partial + (int64_t)i * 3 * C + col);
    part[k][j] = a;
    __syncthreads();
    if (k == 0 && col < 3 * (int64_t)C) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) a += part[i][j];
        float* out = col < C ? dw_post : col < 2 * (int64_t)C ? dscale : dw_pre;
        out[col % C] = a;
    }
}

// How a row is spread: the fewest threads (a power of two, at least 8) that
// hold it in up to 16 elements each, then the fewest pieces each.
struct Plan {
    int vec, nv, tpr, threads;
};
inline Plan plan_for(int32_t C, int wide) {
    Plan p;
    p.vec = wide;
    const int most = 16 / wide;
    const int pieces = (C + wide - 1) / wide;
    p.tpr = 8;
    while (p.tpr * most < pieces) p.tpr *= 2;
    p.nv = 1;
    while (p.nv * p.tpr < pieces) p.nv *= wide == 1 ? 4 : 2;
    p.threads = p.tpr > kThreads ? p.tpr : kThreads;
    return p;
}

struct Args {
    Shape s;
    View dy, du, h, x, gate;
    const float *w_post, *scale, *w_pre;
    const float4* stats_in;
    void *out0, *out1, *out2;   // y, u  |  dh, dx, dgate
    float4* stats_out;
    float *dw_post, *dscale, *dw_pre, *partial;
};

template <typename T, int VEC, int NV, bool kBig>
zs_status run_as(const Plan& p, const Args& a, bool backward, cudaStream_t s) {
    const int rows = p.threads / p.tpr;
    const int64_t need = (a.s.M + rows - 1) / rows;
    if (!backward) {
        const int ctas = (int)imin<int64_t>(need, num_sms() * (kBig ? 1 : 4));
        launch(norm_forward<T, VEC, NV, kBig>, dim3(ctas), dim3(p.threads), 0, s, a.s, a.h, a.x, a.gate, a.w_post, a.scale,
               a.w_pre, static_cast<T*>(a.out0), static_cast<T*>(a.out1), a.stats_out);
        return check_launch("zs_norm_gate_residual");
    }
    const int ctas = (int)imin<int64_t>(need, kBwdCtas);
    if (ctas > 0) {
        const int smem = (kBig ? 3 : rows - 1) * a.s.C * 4;
        if (kBig) {
            static std::atomic<uint64_t> done[kMaxDevices];
            set_smem_limit_once(norm_backward<T, VEC, NV, kBig>, 3 * kMaxC * 4, done);
        }
        launch(norm_backward<T, VEC, NV, kBig>, dim3(ctas), dim3(p.threads), smem, s, a.s, a.dy,
               a.du, a.h, a.x, a.gate, a.w_post, a.scale, a.w_pre, a.stats_in, static_cast<T*>(a.out0),
               static_cast<T*>(a.out1), static_cast<T*>(a.out2), a.partial);
        const zs_status st = check_launch("zs_norm_gate_residual_backward");
        if (st != ZS_OK) return st;
    }
    const int sums = (int)((3 * (int64_t)a.s.C + kSumCols - 1) / kSumCols);
    launch(norm_column_sums, dim3(sums), dim3(kSumCols * kSumRows), 0, s, (const float*)a.partial, ctas, a.s.C, a.dw_post,
           a.dscale, a.dw_pre);
    return check_launch("zs_norm_gate_residual_backward");
}

template <typename T, int VEC, int NV>
zs_status run(const Plan& p, const Args& a, bool backward, cudaStream_t s) {
    if constexpr (VEC * NV == 16)
        if (p.tpr > kThreads) return run_as<T, VEC, NV, true>(p, a, backward, s);
    return run_as<T, VEC, NV, false>(p, a, backward, s);
}

template <typename T>
zs_status dispatch(Args& a, bool backward, cudaStream_t s) {
    constexpr int V = kVec<T>;
    auto fits = [&](const View& v) { return !v.p || (aligned16(v.p) && v.ld % V == 0); };
    const bool wide = a.s.C % V == 0 && fits(a.dy) && fits(a.du) && fits(a.h) && fits(a.x) &&
                      (a.s.gate_cols <= 1 || fits(a.gate)) && aligned16(a.out0) && aligned16(a.out1) &&
                      (a.s.gate_cols <= 1 || !a.out2 || aligned16(a.out2));
    const Plan p = plan_for(a.s.C, wide ? V : 1);
    a.s.tpr = p.tpr;
    if (wide) {
        if (p.nv == 1) return run<T, V, 1>(p, a, backward, s);
        if (p.nv == 2) return run<T, V, 2>(p, a, backward, s);
        if constexpr (V == 4) return run<T, V, 4>(p, a, backward, s);
    }
    if (p.nv == 1) return run<T, 1, 1>(p, a, backward, s);
    if (p.nv == 4) return run<T, 1, 4>(p, a, backward, s);
    return run<T, 1, 16>(p, a, backward, s);
}

zs_status dispatch(int32_t dtype, Args& a, bool backward, cudaStream_t s) {
    switch (dtype) {
        case ZS_F32: return dispatch<float>(a, backward, s);
        case ZS_BF16: return dispatch<__nv_bfloat16>(a, backward, s);
        default: return dispatch<__half>(a, backward, s);
    }
}

// The checks that both directions share; ZS_OK leaves a.s filled.
zs_status check(const char* fn, int32_t dtype, int32_t kind, const View& gate, int32_t gate_cols, int64_t M, int32_t C,
                Args& a) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (kind != ZS_NORM_RMS && kind != ZS_NORM_LAYER)
        return fail(ZS_ERR_UNSUPPORTED, "%s: kind %d is not a zs_norm_kind", fn, kind);
    if (M < 0 || C < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld C=%d", fn, (long long)M, C);
    if (C > kMaxC) return fail(ZS_ERR_UNSUPPORTED, "%s: C=%d is above %d", fn, C, kMaxC);
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
    for (const View& v : {a.h, a.x, a.dy, a.du})
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
    Args a = {};
    a.h = {h, h_ld};
    a.x = {x, x_ld};
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.out0 = y, a.out1 = u;
    a.stats_out = reinterpret_cast<float4*>(stats);
    if (zs_status st = check(fn, dtype, kind, View{gate, gate_ld}, gate_cols, M, C, a)) return st;
    if (!(eps >= 0.f)) return fail(ZS_ERR_INVALID_ARG, "%s: eps=%g", fn, (double)eps);
    if (!aligned16(stats)) return fail(ZS_ERR_INVALID_ARG, "%s: stats is not 16-byte aligned", fn);
    if (M == 0) return ZS_OK;
    if (!h || !x || !y || !u) return fail(ZS_ERR_INVALID_ARG, "%s: NULL h, x, y or u", fn);
    a.s.eps = eps;
    return dispatch(dtype, a, false, reinterpret_cast<cudaStream_t>(stream));
}

size_t zs_norm_gate_residual_backward_workspace_bytes(int64_t M, int32_t C) {
    if (M <= 0 || C < 1) return 0;
    return (size_t)zs::imin<int64_t>(M, zs::kBwdCtas) * 3 * (size_t)C * 4;
}

zs_status zs_norm_gate_residual_backward(int32_t dtype, int32_t kind, const void* dy, int64_t dy_ld, const void* du,
                                         int64_t du_ld, const void* h, int64_t h_ld, const void* x, int64_t x_ld,
                                         const void* gate, int64_t gate_ld, int32_t gate_cols, const float* w_post,
                                         const float* scale, const float* w_pre, const float* stats, int64_t M,
                                         int32_t C, void* dh, void* dx, void* dgate, float* dw_post, float* dscale,
                                         float* dw_pre, void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_norm_gate_residual_backward";
    Args a = {};
    a.dy = {dy, dy_ld};
    a.du = {du, du_ld};
    a.h = {h, h_ld};
    a.x = {x, x_ld};
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.stats_in = reinterpret_cast<const float4*>(stats);
    a.out0 = dh, a.out1 = dx, a.out2 = dgate;
    a.dw_post = dw_post, a.dscale = dscale, a.dw_pre = dw_pre;
    a.partial = static_cast<float*>(workspace);
    if (zs_status st = check(fn, dtype, kind, View{gate, gate_ld}, gate_cols, M, C, a)) return st;
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
    return dispatch(dtype, a, true, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
