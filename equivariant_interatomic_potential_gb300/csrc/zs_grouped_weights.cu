// Grouped products' gradient in the weights: dw[g] = sum over the rows of
// group g of dy[i]^T x[i].
//
// The summed-over direction is the rows', which both operands have across
// their memory rows (MN-major boxes), and the groups' lengths are known on
// the device alone.  A unit of work is 64 positions of one group for one
// 128 x BN tile of the weights; units are numbered tile by tile, and each CTA
// takes an equal range of them, so that skewed groups, few tiles and many
// tiles all keep every SM busy.  A range cuts at most the group it starts in
// and the group it ends in: those two sums go to the workspace in fp32, and a
// second kernel adds, for each group that was cut, its CTAs' parts in order.
#include "zs_grouped.cuh"
#include "zs_mma.cuh"

namespace zs {

namespace {

constexpr int kLoaderWarps = 8;
constexpr int kStep = 64;        // positions of a unit: rows of a box
constexpr int kPartRows = 16;    // rows of a tile that one CTA of the second kernel adds

struct WeightArgs {
    Matrix dy, x;
    const int32_t* row_ptr;
    const int32_t* perm;
    void* dw;
    float* partial;      // [CTA][2][128][BN]
    bool dw_wide;
    int M, G, N, K;
    int ktiles;
    int64_t slots;       // units of a tile, empty ones of no group at its end among them
    int64_t units, per;  // all units, units of a CTA
};

template <typename T, bool kTma, int BN>
struct WeightShape {
    static constexpr int P = kPlanes<T>;
    static constexpr int kBBoxes = BN < kBoxCols ? 1 : BN / kBoxCols;
    static constexpr uint32_t kBox = kStep * kBoxRow;
    static constexpr uint32_t kA = 2 * kBox, kB = kBBoxes * kBox;
    static constexpr uint32_t kStage = P * (kA + kB);
    static constexpr int kFixed = 4 * kStageWarp + 1024 + 512;
    static constexpr int kFit = (kSmemMost - kFixed) / (int)kStage;
    static constexpr int S = kFit > 8 ? 8 : kFit;
    static_assert(S >= 2, "two stages at least");
    static constexpr int kSmem = S * (int)kStage + kFixed;
    static constexpr int kThreads = 256 + (kTma ? 0 : 32 * kLoaderWarps);
    static constexpr uint32_t kTmemCols = 2 * BN;
};

// A maximal run of a CTA's units within one group and one tile.
struct Segment {
    int g, n0, k0;
    int p0, p1;        // positions (p0 == p1: none)
    bool whole;        // all of the group: written as it is
    int part;          // else which of the CTA's two partial tiles
};

// Walks the segments of units [u, end).
template <int BN>
struct Walk {
    const WeightArgs& a;
    Groups<kStep> gr;
    int64_t u, begin, end;
    __device__ __forceinline__ Walk(const WeightArgs& args, int64_t cta)
        : a(args), gr{args.row_ptr, args.G, args.M}, u(cta * args.per), begin(u), end(imin(u + args.per, args.units)) {}
    __device__ __forceinline__ bool next(Segment& s) {
        while (u < end) {
            const int64_t t = u / a.slots, slot = u - t * a.slots;
            const int64_t last = gr.slot(a.G);       // slots of groups
            if (slot >= last) {
                u = (t + 1) * a.slots;
                continue;
            }
            s.g = gr.find(slot, a.G);
            const int64_t g0 = gr.slot(s.g), g1 = gr.slot(s.g + 1);
            const int b = gr.start(s.g), e = gr.start(s.g + 1);
            const int64_t stop = imin(end, t * a.slots + g1);
            s.n0 = (int)(t / a.ktiles) * kTileM;
            s.k0 = (int)(t % a.ktiles) * BN;
            s.whole = slot == g0 && stop == t * a.slots + g1;
            s.part = u == begin ? 0 : 1;
            s.p0 = (int)imin<int64_t>(b + (slot - g0) * kStep, e);
            s.p1 = (int)imin<int64_t>(b + (stop - t * a.slots - g0) * kStep, e);
            u = stop;
            return true;
        }
        return false;
    }
};

__device__ __forceinline__ int row_at(const WeightArgs& a, int p) {
    if (!a.perm) return p;
    const int r = __ldg(a.perm + p);
    return (uint32_t)r < (uint32_t)a.M ? r : -1;
}

template <typename T, bool kTma, int BN>
__global__ void __launch_bounds__(WeightShape<T, kTma, BN>::kThreads, 1)
weights_mma(const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap x_map, const WeightArgs a) {
    using Sh = WeightShape<T, kTma, BN>;
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
    Walk<BN> walk(a, blockIdx.x);
    Segment s;

    if (kTma && warp == 0) {
        RingPos<S> pos;
        int issued = 0;
        while (!*dead && walk.next(s)) {
            const int a_boxes = imin(2, (a.N - s.n0 + kBoxCols - 1) / kBoxCols);
            const int b_boxes = imin(Sh::kBBoxes, (a.K - s.k0 + kBoxCols - 1) / kBoxCols);
            for (int p = s.p0; p < s.p1; p += kStep, pos.next()) {
                // lanes 0..15: four rows each (of 64); the last one again past the end
                const int quads = imin(kStep / 4, (s.p1 - p + 3) / 4);
                int4 rows = make_int4(0, 0, 0, 0);
                if (a.perm && lane < quads) {
                    int* r = &rows.x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = imax(row_at(a, imin(p + 4 * lane + i, s.p1 - 1)), 0);
                }
                if (!bounded_wait(empty + 8 * pos.stage, pos.phase ^ 1, dead)) break;
                const uint32_t bar = full + 8 * pos.stage, at = smem_u32(ring) + pos.stage * Sh::kStage, bt = at + Sh::kA;
                if (lane == 0) mbar_arrive_expect_tx(bar, (a_boxes + b_boxes) * (a.perm ? quads * 512u : Sh::kBox));
                __syncwarp();
                if (a.perm) {
                    if (lane < quads) {
                        for (int i = 0; i < a_boxes; ++i)
                            tma_gather4(at + i * Sh::kBox + lane * 512, &dy_map, s.n0 + i * kBoxCols, rows, bar);
                        for (int i = 0; i < b_boxes; ++i)
                            tma_gather4(bt + i * Sh::kBox + lane * 512, &x_map, s.k0 + i * kBoxCols, rows, bar);
                    }
                } else {
                    if (lane < a_boxes) tma_2d(at + lane * Sh::kBox, &dy_map, s.n0 + lane * kBoxCols, p, bar);
                    if (lane < b_boxes) tma_2d(bt + lane * Sh::kBox, &x_map, s.k0 + lane * kBoxCols, p, bar);
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
        while (!*dead && walk.next(s)) {
            for (int p = s.p0; p < s.p1; p += kStep, pos.next()) {
                constexpr int kRows = kStep / kLoaderWarps;
                int myrow = -1;   // lane i < 8: the row at position p + 8 i + w
                if (lane < kRows && p + lane * kLoaderWarps + w < s.p1) myrow = row_at(a, p + lane * kLoaderWarps + w);
                if (!bounded_wait(empty + 8 * pos.stage, pos.phase ^ 1, dead)) break;
                unsigned char* at = ring + pos.stage * Sh::kStage;
                auto bring = [&](const Matrix& m, unsigned char* to, uint32_t plane, int c0, int boxes) {
                    for (int box = 0; box < boxes && c0 + box * kBoxCols < m.cols; ++box) {
                        Pair<T> v[kRows];
#pragma unroll
                        for (int i = 0; i < kRows; ++i) {
                            const int r = __shfl_sync(0xffffffffu, myrow, i);
                            if (r >= 0) v[i] = load_pair<T>(m, r, c0 + box * kBoxCols + 2 * lane);
                            else v[i].a = v[i].b = from_f32<T>(0.f);
                        }
#pragma unroll
                        for (int i = 0; i < kRows; ++i) store_pair<T>(to + box * Sh::kBox, plane, i * kLoaderWarps + w, lane, v[i]);
                    }
                };
                bring(a.dy, at, Sh::kA, s.n0, 2);
                bring(a.x, at + Sh::P * Sh::kA, Sh::kB, s.k0, Sh::kBBoxes);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * pos.stage);
            }
        }
    } else if (warp == 1) {
        RingPos<S> pos;
        const uint32_t idesc = instr_desc<T>(true, true, BN);
        int n = 0;
        while (!*dead && walk.next(s)) {
            if (s.p0 == s.p1) continue;
            const int buf = n & 1;
            if (!bounded_wait(tempty + 8 * buf, ((n >> 1) & 1) ^ 1, dead)) break;
            tc_fence_after();
            for (int p = s.p0; p < s.p1; p += kStep, pos.next()) {
                if (!bounded_wait(full + 8 * pos.stage, pos.phase, dead)) break;
                const int rows = imin(kStep, s.p1 - p), steps = (rows + 15) / 16;
                unsigned char* at = ring + pos.stage * Sh::kStage;
                if (kTma && rows < 16 * steps) {
                    // positions past the segment's end hold other rows, or nothing: they count as zeros
                    const int chunks = (16 * steps - rows) * (kBoxRow / 16);
                    for (int i = lane; i < chunks * (2 + Sh::kBBoxes); i += 32)
                        *reinterpret_cast<uint4*>(at + (i / chunks) * Sh::kBox + rows * kBoxRow + (i % chunks) * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t aa = smem_u32(at);
                    issue_stage<T, true, true>(tmem + buf * BN, aa, Sh::kA, Sh::kBox, aa + Sh::P * Sh::kA, Sh::kB, Sh::kBox,
                                               idesc, steps, p > s.p0);
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
        const int q = warp - 4, r = 32 * q + lane;
        unsigned char* stage = staging + q * kStageWarp;
        int n = 0;
        while (!*dead && walk.next(s)) {
            const bool some = s.p0 < s.p1;
            const int buf = n & 1;
            if (some) {
                if (!bounded_wait(tfull + 8 * buf, (n >> 1) & 1, dead)) break;
                tc_fence_after();
            }
            const uint32_t from = some ? tmem + buf * BN + ((uint32_t)(32 * q) << 16) : kNoTile;
            const int cols = imin(BN, a.K - s.k0);
            if (s.whole) {
                T* row = s.n0 + r < a.N ? static_cast<T*>(a.dw) + ((int64_t)s.g * a.N + s.n0 + r) * a.K + s.k0 : nullptr;
                store_tile<T>(from, cols, row, a.dw_wide, stage, lane);
            } else {
                float* row = s.n0 + r < a.N ? a.partial + (((int64_t)blockIdx.x * 2 + s.part) * kTileM + r) * BN : nullptr;
                store_tile<float>(from, (cols + 3) / 4 * 4, row, true, stage, lane);
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty + 8 * buf);
                ++n;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free(tmem, Sh::kTmemCols);
}

// Block (x, y): the group and tile that CTA x + 1's range begins inside of, if
// CTA x holds its beginning; rows y * kPartRows .. of the tile.
template <typename T, int BN>
__global__ void __launch_bounds__(256) weights_join(const WeightArgs a) {
    pdl_wait();
    pdl_trigger();
    const Groups<kStep> gr{a.row_ptr, a.G, a.M};
    const int64_t cut = (blockIdx.x + 1) * a.per;
    if (cut >= a.units) return;
    const int64_t t = cut / a.slots, slot = cut - t * a.slots;
    if (slot >= gr.slot(a.G)) return;
    const int g = gr.find(slot, a.G);
    const int64_t u0 = t * a.slots + gr.slot(g), u1 = imin(t * a.slots + gr.slot(g + 1), a.units);
    if (u0 >= cut) return;                          // the group begins with CTA x + 1
    const int64_t first = u0 / a.per, last = (u1 - 1) / a.per;
    if (first != blockIdx.x) return;                // an earlier block adds it
    const int first_part = u0 == first * a.per ? 0 : 1;
    const int n0 = (int)(t / a.ktiles) * kTileM + blockIdx.y * kPartRows, k0 = (int)(t % a.ktiles) * BN;
    const int cols = imin(BN, a.K - k0), rows = imin(kPartRows, a.N - n0);
    for (int i = threadIdx.x; i < rows * BN; i += blockDim.x) {
        const int r = i / BN, c = i % BN;
        if (c >= cols) continue;
        const int64_t at = ((int64_t)blockIdx.y * kPartRows + r) * BN + c;
        float sum = __ldg(a.partial + (first * 2 + first_part) * kTileM * BN + at);
        for (int64_t p = first + 1; p <= last; ++p) sum += __ldg(a.partial + p * 2 * kTileM * BN + at);
        static_cast<T*>(a.dw)[((int64_t)g * a.N + n0 + r) * a.K + k0 + c] = from_f32<T>(sum);
    }
}

// Tiles and ranges of a problem; the same on every device, so that the
// workspace's size is too.
constexpr int kCtas = 152;
struct WeightPlan {
    int bn;
    int64_t tiles, slots, units, per;
    int ctas;
};
WeightPlan weight_plan(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    WeightPlan p;
    p.bn = K <= 32 ? 32 : K <= 64 ? 64 : dtype == ZS_F32 || (K + 127) / 128 % 2 ? 128 : 256;
    p.tiles = (int64_t)((N + kTileM - 1) / kTileM) * ((K + p.bn - 1) / p.bn);
    p.slots = M / kStep + G;
    p.units = p.tiles * p.slots;
    p.per = (p.units + kCtas - 1) / kCtas;
    p.ctas = p.per ? (int)((p.units + p.per - 1) / p.per) : 0;
    return p;
}

template <typename T, bool kTma, int BN>
zs_status launch_weights(const char* fn, WeightArgs a, const WeightPlan& p, cudaStream_t s) {
    using Sh = WeightShape<T, kTma, BN>;
    CUtensorMap dy_map = {}, x_map = {};
    if (kTma) {
        constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
        const int box = a.perm ? 1 : kStep;
        if (!encode_boxes(&dy_map, bf16, a.dy.p, a.N, a.M, a.dy.ld, 0, box) ||
            !encode_boxes(&x_map, bf16, a.x.p, a.K, a.M, a.x.ld, 0, box))
            return fail(ZS_ERR_CUDA, "%s: a tensor map was refused", fn);
    }
    static std::atomic<uint64_t> done[kMaxDevices];
    set_smem_limit_once(weights_mma<T, kTma, BN>, Sh::kSmem, done);
    launch(weights_mma<T, kTma, BN>, dim3(p.ctas), dim3(Sh::kThreads), Sh::kSmem, s, dy_map, x_map, a);
    if (zs_status st = check_launch(fn)) return st;
    if (p.ctas > 1) {
        launch(weights_join<T, BN>, dim3(p.ctas - 1, kTileM / kPartRows), dim3(256), 0, s, a);
        return check_launch(fn);
    }
    return ZS_OK;
}

template <typename T, bool kTma>
zs_status launch_weights(const char* fn, const WeightArgs& a, const WeightPlan& p, cudaStream_t s) {
    if (p.bn == 32) return launch_weights<T, kTma, 32>(fn, a, p, s);
    if (p.bn == 64) return launch_weights<T, kTma, 64>(fn, a, p, s);
    if constexpr (sizeof(T) == 2)
        if (p.bn == 256) return launch_weights<T, kTma, 256>(fn, a, p, s);
    return launch_weights<T, kTma, 128>(fn, a, p, s);
}

}  // namespace

unsigned int take_timeouts_grouped_weights() { return take_timeouts_local(); }
cudaError_t set_timeout_flag_grouped_weights(unsigned int* flag) { return set_timeout_flag_local(flag); }

size_t grouped_weights_workspace(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    const WeightPlan p = weight_plan(dtype, M, K, N, G);
    return p.ctas > 1 ? (size_t)p.ctas * 2 * kTileM * p.bn * 4 : 0;
}

zs_status grouped_weights(const char* fn, int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                          const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dw,
                          void* workspace, cudaStream_t s) {
    const int es = dtype_bytes(dtype), per16 = 16 / es;
    auto at = [&](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const WeightPlan p = weight_plan(dtype, M, K, N, G);
    if (p.units >= (int64_t(1) << 40)) return fail(ZS_ERR_INVALID_ARG, "%s: %lld units", fn, (long long)p.units);
    WeightArgs a = {};
    a.dy = {dy, dy_ld, N, at(dy, 2 * es) && dy_ld % 2 == 0};
    a.x = {x, x_ld, K, at(x, 2 * es) && x_ld % 2 == 0};
    a.row_ptr = row_ptr;
    a.perm = perm;
    a.dw = dw;
    a.partial = static_cast<float*>(workspace);
    a.dw_wide = at(dw, 16) && K % per16 == 0;
    a.M = (int)M, a.G = G, a.N = N, a.K = K;
    a.ktiles = (K + p.bn - 1) / p.bn;
    a.slots = p.slots, a.units = p.units, a.per = p.per;
    const bool aligned = at(dy, 16) && dy_ld % per16 == 0 && at(x, 16) && x_ld % per16 == 0 && M > 0;
    switch (dtype) {
        case ZS_F32: return launch_weights<float, false>(fn, a, p, s);
        case ZS_BF16: return aligned ? launch_weights<__nv_bfloat16, true>(fn, a, p, s)
                                     : launch_weights<__nv_bfloat16, false>(fn, a, p, s);
        default: return aligned ? launch_weights<__half, true>(fn, a, p, s) : launch_weights<__half, false>(fn, a, p, s);
    }
}

}  // namespace zs
