// Grouped products over rows: y[i] = w[g(i)] x[i], and the gradient in x with
// w transposed.  One persistent kernel: warp 0 brings tiles in by TMA (rows
// of a CSR by gather), or eight more warps read them where TMA cannot (fp32,
// which is cut into bf16 planes on the way, and unaligned rows); warp 1
// issues the products; warps 4 to 7 write finished tiles while the next one
// is being summed.
#include <initializer_list>

#include "zs_grouped.cuh"
#include "zs_mma.cuh"

namespace zs {

namespace {

constexpr int kLoaderWarps = 8;

struct RowsArgs {
    Matrix a;             // rows of the left operand
    Matrix w;             // weights of group 0, rows w.ld apart
    int64_t w_group;      // elements of a group's weights
    const int32_t* row_ptr;
    const int32_t* perm;
    void* out;
    int64_t out_ld;
    bool out_wide;
    int M, G;
    int red, cols;        // summed-over length, output columns
    int items, ntiles;
};

template <typename T, bool kTma, bool kMN, int BN>
struct RowsShape {
    static constexpr int P = kPlanes<T>;
    static constexpr uint32_t kA = kTileM * kBoxRow;
    static constexpr uint32_t kB = (kMN && BN < kBoxCols ? kBoxCols : BN) * kBoxRow;
    static constexpr uint32_t kStage = P * (kA + kB);
    static constexpr int kFixed = 4 * kStageWarp + 1024 + 512;   // staging, alignment, barriers
    static constexpr int kFit = (kSmemMost - kFixed) / (int)kStage;
    static constexpr int S = kFit > 8 ? 8 : kFit;
    static_assert(S >= 2, "two stages at least");
    static constexpr int kSmem = S * (int)kStage + kFixed;
    static constexpr int kThreads = 256 + (kTma ? 0 : 32 * kLoaderWarps);
    static constexpr uint32_t kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
};

struct Item {
    int g, p0, p1, n0;
};
// The item'th tile of output; false when it is empty.
__device__ __forceinline__ bool get_item(const RowsArgs& a, const Groups<kTileM>& gr, int item, int BN, Item& t) {
    const int64_t slot = item / a.ntiles;
    t.n0 = item % a.ntiles * BN;
    t.g = gr.find(slot, a.G + 1);
    const int b = gr.start(t.g), e = gr.start(t.g + 1);
    const int64_t p0 = b + (slot - (b / kTileM + t.g)) * kTileM;
    if (p0 >= e) return false;
    t.p0 = (int)p0;
    t.p1 = (int)imin<int64_t>(p0 + kTileM, e);
    return true;
}

__device__ __forceinline__ int row_at(const RowsArgs& a, int p) {
    if (!a.perm) return p;
    const int r = __ldg(a.perm + p);
    return (uint32_t)r < (uint32_t)a.M ? r : -1;
}

template <typename T, bool kTma, bool kMN, int BN>
__global__ void __launch_bounds__(RowsShape<T, kTma, kMN, BN>::kThreads, 1)
rows_mma(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap w_map, RowsArgs a) {
    using Sh = RowsShape<T, kTma, kMN, BN>;
    constexpr int S = Sh::S;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* staging = ring + S * Sh::kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 4 * kStageWarp);
    volatile int* dead = reinterpret_cast<volatile int*>(bars + 2 * S + 5);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 6);
    const uint32_t full = smem_u32(bars), empty = full + 8 * S, tfull = empty + 8 * S, tempty = tfull + 16, done = tempty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + 8 * i, kTma ? 1 : kLoaderWarps);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 4);
        }
        mbar_init(done, 1);
        *dead = 0;
        mbar_fence_init();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 2) tmem_alloc(smem_u32(tmem_slot), Sh::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Groups<kTileM> gr{a.row_ptr, a.G, a.M};
    const int nk = (a.red + kBoxCols - 1) / kBoxCols;

    if (kTma && warp == 0) {
        RingPos<S> pos;
        int issued = 0;
        for (int item = blockIdx.x; item < a.items && !*dead; item += gridDim.x) {
            Item t;
            if (!get_item(a, gr, item, BN, t) || t.g == a.G) continue;
            // this lane's four rows; the last one again past the end
            int4 rows = make_int4(0, 0, 0, 0);
            const int p = t.p0 + 4 * lane;
            const bool mine = p < t.p1;
            if (a.perm && mine) {
                int* r = &rows.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = imax(row_at(a, imin(p + i, t.p1 - 1)), 0);
            }
            const uint32_t a_bytes = a.perm ? 512u * ((t.p1 - t.p0 + 3) / 4) : Sh::kA;
            const int boxes = kMN ? (imin(BN, a.cols - t.n0) + kBoxCols - 1) / kBoxCols : 1;
            const uint32_t bytes = a_bytes + (kMN ? boxes * kBoxCols * kBoxRow : Sh::kB);
            for (int k = 0; k < nk; ++k, pos.next()) {
                if (!bounded_wait(empty + 8 * pos.stage, pos.phase ^ 1, dead)) break;
                const uint32_t bar = full + 8 * pos.stage, at = smem_u32(ring) + pos.stage * Sh::kStage, bt = at + Sh::kA;
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (a.perm) {
                    if (mine) tma_gather4(at + lane * 512, &a_map, k * kBoxCols, rows, bar);
                } else if (lane == 0) {
                    tma_2d(at, &a_map, k * kBoxCols, t.p0, bar);
                }
                if (kMN) {
                    if (lane < boxes) tma_3d(bt + lane * kBoxCols * kBoxRow, &w_map, t.n0 + lane * kBoxCols, k * kBoxCols, t.g, bar);
                } else if (lane == 0) {
                    tma_3d(bt, &w_map, k * kBoxCols, t.n0, t.g, bar);
                }
                ++issued;
            }
        }
        if (*dead) {   // wait for the copies in flight
            for (int i = 0; i < imin(issued, S); ++i) {
                const int k = issued - 1 - i;
                for (uint32_t n = 0; n < kDrainSpins && !mbar_try_wait(full + 8 * (k % S), (uint32_t)(k / S) & 1); ++n) {}
            }
        }
    } else if (!kTma && warp >= 8) {
        RingPos<S> pos;
        const int w = warp - 8;
        for (int item = blockIdx.x; item < a.items && !*dead; item += gridDim.x) {
            Item t;
            if (!get_item(a, gr, item, BN, t) || t.g == a.G) continue;
            constexpr int kRowsA = kTileM / kLoaderWarps;
            int myrow = -1;   // lane i < 16: the row of tile row 8 i + w
            if (lane < kRowsA && t.p0 + lane * kLoaderWarps + w < t.p1) myrow = row_at(a, t.p0 + lane * kLoaderWarps + w);
            Matrix wm = a.w;
            wm.p = static_cast<const T*>(wm.p) + t.g * a.w_group;
            for (int k = 0; k < nk; ++k, pos.next()) {
                if (!bounded_wait(empty + 8 * pos.stage, pos.phase ^ 1, dead)) break;
                unsigned char* at = ring + pos.stage * Sh::kStage;
                unsigned char* bt = at + Sh::P * Sh::kA;
                const int c = k * kBoxCols + 2 * lane;
                Pair<T> v[kRowsA];
#pragma unroll
                for (int i = 0; i < kRowsA; ++i) {
                    const int r = __shfl_sync(0xffffffffu, myrow, i);
                    if (r >= 0) v[i] = load_pair<T>(a.a, r, c);
                    else v[i].a = v[i].b = from_f32<T>(0.f);
                }
#pragma unroll
                for (int i = 0; i < kRowsA; ++i) store_pair<T>(at, Sh::kA, i * kLoaderWarps + w, lane, v[i]);
                if constexpr (!kMN) {
                    constexpr int kB8 = BN / kLoaderWarps;
                    Pair<T> u[kB8];
#pragma unroll
                    for (int i = 0; i < kB8; ++i) {
                        const int n = t.n0 + i * kLoaderWarps + w;
                        if (n < a.cols) u[i] = load_pair<T>(wm, n, c);
                        else u[i].a = u[i].b = from_f32<T>(0.f);
                    }
#pragma unroll
                    for (int i = 0; i < kB8; ++i) store_pair<T>(bt, Sh::kB, i * kLoaderWarps + w, lane, u[i]);
                } else {
                    constexpr int kR8 = kBoxCols / kLoaderWarps;
                    for (int box = 0; box * kBoxCols < BN && t.n0 + box * kBoxCols < a.cols; ++box) {
                        Pair<T> u[kR8];
#pragma unroll
                        for (int i = 0; i < kR8; ++i) {
                            const int r = k * kBoxCols + i * kLoaderWarps + w;
                            if (r < a.red) u[i] = load_pair<T>(wm, r, t.n0 + box * kBoxCols + 2 * lane);
                            else u[i].a = u[i].b = from_f32<T>(0.f);
                        }
#pragma unroll
                        for (int i = 0; i < kR8; ++i)
                            store_pair<T>(bt + box * kBoxCols * kBoxRow, Sh::kB, i * kLoaderWarps + w, lane, u[i]);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * pos.stage);
            }
        }
    } else if (warp == 1) {
        RingPos<S> pos;
        const uint32_t idesc = instr_desc<T>(false, kMN, BN);
        int n = 0;
        for (int item = blockIdx.x; item < a.items && !*dead; item += gridDim.x) {
            Item t;
            if (!get_item(a, gr, item, BN, t) || t.g == a.G) continue;
            const int buf = n & 1;
            if (!bounded_wait(tempty + 8 * buf, ((n >> 1) & 1) ^ 1, dead)) break;
            tc_fence_after();
            for (int k = 0; k < nk; ++k, pos.next()) {
                if (!bounded_wait(full + 8 * pos.stage, pos.phase, dead)) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t at = smem_u32(ring) + pos.stage * Sh::kStage;
                    const int steps = (imin(kBoxCols, a.red - k * kBoxCols) + 15) / 16;
                    issue_stage<T, false, kMN>(tmem + buf * BN, at, Sh::kA, 0, at + Sh::P * Sh::kA, Sh::kB,
                                               kBoxCols * kBoxRow, idesc, steps, k > 0);
                    tc_commit(empty + 8 * pos.stage);
                }
                __syncwarp();
            }
            if (lane == 0) tc_commit(tfull + 8 * buf);
            __syncwarp();
            ++n;
        }
        if (*dead) {   // wait for the products in flight
            if (lane == 0) tc_commit(done);
            for (uint32_t i = 0; i < kDrainSpins && !mbar_try_wait(done, 0); ++i) {}
        }
    } else if (warp >= 4 && warp < 8) {
        const int q = warp - 4;
        unsigned char* stage = staging + q * kStageWarp;
        int n = 0;
        for (int item = blockIdx.x; item < a.items && !*dead; item += gridDim.x) {
            Item t;
            if (!get_item(a, gr, item, BN, t)) continue;
            const int p = t.p0 + 32 * q + lane;
            const int r = p < t.p1 ? row_at(a, p) : -1;
            T* row = r >= 0 ? static_cast<T*>(a.out) + r * a.out_ld + t.n0 : nullptr;
            const int cols = imin(BN, a.cols - t.n0);
            if (t.g == a.G) {
                store_tile<T>(kNoTile, cols, row, a.out_wide, stage, lane);
                continue;
            }
            const int buf = n & 1;
            if (!bounded_wait(tfull + 8 * buf, (n >> 1) & 1, dead)) break;
            tc_fence_after();
            store_tile<T>(tmem + buf * BN + ((uint32_t)(32 * q) << 16), cols, row, a.out_wide, stage, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty + 8 * buf);
            ++n;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free(tmem, Sh::kTmemCols);
}

template <typename T, bool kTma, bool kMN, int BN>
zs_status launch_rows(const char* fn, RowsArgs a, cudaStream_t s) {
    using Sh = RowsShape<T, kTma, kMN, BN>;
    CUtensorMap a_map = {}, w_map = {};
    if (kTma) {
        constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
        const int w_rows = kMN ? a.red : a.cols;
        if (!encode_boxes(&a_map, bf16, a.a.p, a.red, a.M, a.a.ld, 0, a.perm ? 1 : kTileM) ||
            !encode_boxes(&w_map, bf16, a.w.p, a.w.ld, w_rows, a.w.ld, a.G, kMN ? kBoxCols : BN))
            return fail(ZS_ERR_CUDA, "%s: a tensor map was refused", fn);
    }
    a.ntiles = (a.cols + BN - 1) / BN;
    const int64_t items = ((int64_t)a.M / kTileM + a.G + 2) * a.ntiles;
    if (items >= (int64_t(1) << 31) - 65536) return fail(ZS_ERR_INVALID_ARG, "%s: %lld tiles", fn, (long long)items);
    a.items = (int)items;
    static std::atomic<uint64_t> done[kMaxDevices];
    set_smem_limit_once(rows_mma<T, kTma, kMN, BN>, Sh::kSmem, done);
    launch(rows_mma<T, kTma, kMN, BN>, dim3(imin(a.items, num_sms())), dim3(Sh::kThreads), Sh::kSmem, s, a_map, w_map, a);
    return check_launch(fn);
}

template <typename T, bool kTma, bool kMN>
zs_status launch_rows(const char* fn, const RowsArgs& a, cudaStream_t s) {
    if (a.cols <= 32) return launch_rows<T, kTma, kMN, 32>(fn, a, s);
    if (a.cols <= 64) return launch_rows<T, kTma, kMN, 64>(fn, a, s);
    if constexpr (kTma)
        if ((a.cols + 127) / 128 % 2 == 0) return launch_rows<T, kTma, kMN, 256>(fn, a, s);
    return launch_rows<T, kTma, kMN, 128>(fn, a, s);
}

template <typename T>
zs_status rows_product(const char* fn, RowsArgs a, bool mn, bool aligned, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (aligned) return mn ? launch_rows<T, true, true>(fn, a, s) : launch_rows<T, true, false>(fn, a, s);
    return mn ? launch_rows<T, false, true>(fn, a, s) : launch_rows<T, false, false>(fn, a, s);
}

}  // namespace

unsigned int take_timeouts_grouped_rows() { return take_timeouts_local(); }
cudaError_t set_timeout_flag_grouped_rows(unsigned int* flag) { return set_timeout_flag_local(flag); }

// rows x_ld apart, K the length of a weight row; transposed: the gradient.
zs_status grouped_rows(const char* fn, int32_t dtype, const void* x, int64_t x_ld, const void* w, const int32_t* row_ptr,
                       const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out, int64_t out_ld,
                       bool transposed, cudaStream_t s) {
    const int es = dtype_bytes(dtype), per16 = 16 / es;
    auto at = [&](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    RowsArgs a = {};
    a.red = transposed ? N : K;
    a.cols = transposed ? K : N;
    a.a = {x, x_ld, a.red, at(x, 2 * es) && x_ld % 2 == 0};
    a.w = {w, K, K, at(w, 2 * es) && K % 2 == 0};
    a.w_group = (int64_t)K * N;
    a.row_ptr = row_ptr;
    a.perm = perm;
    a.out = out;
    a.out_ld = out_ld;
    a.out_wide = at(out, 16) && out_ld % per16 == 0 && a.cols % per16 == 0;
    a.M = (int)M;
    a.G = G;
    const bool aligned = at(x, 16) && x_ld % per16 == 0 && at(w, 16) && K % per16 == 0 && G > 0;
    switch (dtype) {
        case ZS_F32: return rows_product<float>(fn, a, transposed, false, s);
        case ZS_BF16: return rows_product<__nv_bfloat16>(fn, a, transposed, aligned, s);
        default: return rows_product<__half>(fn, a, transposed, aligned, s);
    }
}

}  // namespace zs
