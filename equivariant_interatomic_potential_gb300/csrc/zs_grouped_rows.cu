// Grouped products over rows: y[i] = w[g(i)] x[i], and the gradient in x with
// w transposed.  One persistent kernel: warp 0 brings tiles in by TMA, eight
// more warps copy the rows of a CSR in with cp.async, or two groups of eight
// read everything where neither can (fp32, which is cut into bf16 planes on
// the way, and unaligned rows); warp 1 issues the products (of a pair of CTAs,
// the first one's those of both); warps 4 to 11 write finished tiles while the
// next one is being summed.
//
// 32768 bf16 rows in order, 8 groups of 1024 -> 4096: 170 us (1.62 PFLOP/s) and
// 189 transposed, the tensor cores 70 % active and the power limit reached; 89
// groups of 256 -> 256, gathered: 19 us, of which the weights' copies take 10 and
// the results' way out 4 (0.36 of the copy rate); fp32 at a sixth of the rate.
#include <initializer_list>

#include "zs_grouped.cuh"
#include "zs_mma.cuh"

namespace zs {

namespace {

struct RowsArgs {
    Matrix a;             // rows of the left operand
    Matrix w;             // weights of group 0, rows w.ld apart
    int64_t w_group;      // elements of a group's weights
    const int32_t* row_ptr;
    const int32_t* perm;  // the output rows
    const int32_t* gather;   // the left operand's rows: perm, or NULL where they are in order
    void* out;
    int64_t out_ld;
    bool out_wide;
    int M, G;
    int red, cols;        // summed-over length, output columns
    int items, ntiles;
};

// kPair: two CTAs form a tile of 256 rows together, each with its own 128 rows
// and half of the weights.
template <typename T, bool kTma, bool kMN, int BN, bool kPair>
struct RowsShape {
    static_assert(!kPair || (kTma && BN == 256), "pairs form 256 x 256");
    static constexpr int kTile = kPair ? 2 * kTileM : kTileM;
    static constexpr int kMine = kPair ? BN / 2 : BN;   // columns whose weights this CTA holds
    static constexpr int P = kPlanes<T>, kBox = kStageK<T>;
    static constexpr uint32_t kA = box_bytes<kBox>(kTileM);
    static constexpr int kBoxes = kMN ? (kMine + kBoxMN - 1) / kBoxMN : 1;                       // of the right operand
    static constexpr uint32_t kBoxB = kMN ? box_bytes<kBoxMN>(kBox) : box_bytes<kBox>(kMine);
    static constexpr uint32_t kB = kBoxes * kBoxB;
    static constexpr uint32_t kStage = P * (kA + kB);
    static constexpr int kHalves = BN >= 64 ? 2 : 1;   // warps that share 32 rows of a tile
    static constexpr uint32_t kTmemCols = tmem_cols(2 * kSums<T> * BN);
    // what the loader warps copy into before they turn it: 16 bytes a part, two stages for each of the two groups (or
    // one of unaligned rows, 32 bytes a part)
    using PartsA = BoxParts<T, kTileM, kBox>;
    using PartsB = BoxParts<T, kMN ? kBox : kMine, kMN ? kBoxMN : kBox>;
    static constexpr int kParts = PartsA::kSteps + kBoxes * PartsB::kSteps;
    static constexpr int kSlots = kTma ? 0 : 4 * kParts * 32 * kLoaderWarps * 16;
    static constexpr int kFixed = kSlots + kEpilogueWarps * kStageWarp + 1024 + 4608;   // staging, alignment, barriers and groups
    static constexpr int kFit = (kSmemMost - kFixed) / (int)kStage;
    static constexpr int S = kFit > 8 ? 8 : kFit;
    static_assert(kPlanes<T> == 1 || !kMN || BN == kBoxMN, "the planes of an MN-major operand follow each other");
    static_assert(S >= 2 && Setup<S, kTmemCols, kTile, 1, kPair>::kBytes <= 4608, "two stages at least");
    static constexpr int kSmem = S * (int)kStage + kFixed;
    static constexpr int kThreads = 32 * (4 + kEpilogueWarps + (kPair ? 0 : kTma ? 1 : 2) * kLoaderWarps);
};

struct Item {
    int g, p0, p1, n0;
};
template <int kTile>
using RowGroups = Groups<kTile, 1>;

// The next tile of output with rows in it, from `item` on in steps of `step`.
template <int kTile>
__device__ __forceinline__ bool next_item(const RowsArgs& a, const RowGroups<kTile>& gr, int& item, int step, int BN, Item& t) {
    for (; item < a.items; item += step) {
        const int slot = item / a.ntiles;
        t.n0 = item % a.ntiles * BN;
        t.g = gr.find(slot, a.G + 1);
        const int b = gr.start(t.g), e = gr.start(t.g + 1);
        const int64_t p0 = b + (int64_t)(slot - (b / kTile + t.g)) * kTile;
        if (p0 < e) {
            t.p0 = (int)p0;
            t.p1 = (int)imin<int64_t>(p0 + kTile, e);
            item += step;
            return true;
        }
    }
    return false;
}
// The same without the rows of no group, which take no product.
template <int kTile>
__device__ __forceinline__ bool next_product(const RowsArgs& a, const RowGroups<kTile>& gr, int& item, int step, int BN, Item& t) {
    while (next_item(a, gr, item, step, BN, t))
        if (t.g < a.G) return true;
    return false;
}

__device__ __forceinline__ int row_at(const int32_t* perm, int M, int p) {
    if (!perm) return p;
    const int r = __ldg(perm + p);
    return (uint32_t)r < (uint32_t)M ? r : -1;
}

template <typename T, bool kTma, bool kMN, int BN, bool kPair>
__global__ void __launch_bounds__(RowsShape<T, kTma, kMN, BN, kPair>::kThreads, 1)
rows_mma(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap w_map, const RowsArgs a) {
    using Sh = RowsShape<T, kTma, kMN, BN, kPair>;
    constexpr int S = Sh::S;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* slots = ring + S * Sh::kStage;
    unsigned char* staging = slots + Sh::kSlots;
    Setup<S, Sh::kTmemCols, Sh::kTile, 1, kPair> set;
    set.begin(staging + kEpilogueWarps * kStageWarp, !kTma ? kLoaderWarps : a.gather ? 1 + kCopyWarps : 1, 4 * Sh::kHalves, a.row_ptr, a.G, a.M);
    const RowGroups<Sh::kTile>& gr = set.groups;
    volatile int* dead = set.dead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kBox = Sh::kBox;
    const uint32_t full = kPair ? in_first(set.full) : set.full;   // told to
    const int nk = (a.red + kBox - 1) / kBox;
    constexpr int kPerChunk = (kSums<T> > 1 ? kChunk : kLongSum) / kBox;   // stages between hand-overs to the epilogue
    const int rank = kPair ? (int)cluster_rank() : 0, step = kPair ? gridDim.x / 2 : gridDim.x;
    int item = kPair ? blockIdx.x / 2 : blockIdx.x;
    Item t;

    if (kTma && warp == 0) {
        RingPos<S> pos;
        int issued = 0;
        while (!is_dead(dead) && next_product(a, gr, item, step, BN, t)) {
            auto boxes_from = [&](int n0) { return kMN ? imax(0, imin(Sh::kMine, a.cols - n0) + kBoxMN - 1) / kBoxMN : 1; };
            const int n0 = t.n0 + rank * Sh::kMine, boxes = boxes_from(n0);
            // of a pair, the first CTA's barrier counts both CTAs' bytes
            const uint32_t bytes = (kPair ? 2 : 1) * (a.gather ? 0 : Sh::kA) + (boxes + (kPair ? boxes_from(t.n0 + Sh::kMine) : 0)) * Sh::kBoxB;
            for (int k = 0; k < nk; ++k, ++issued, pos.next()) {
                bounded_wait_on(set.empty + 8 * pos.stage, pos.phase ^ 1, dead);
                if (is_dead(dead)) break;
                const uint32_t at = smem_u32(ring) + pos.stage * Sh::kStage, bt = at + Sh::kA;
                const uint32_t bar = full + 8 * pos.stage;
                if (rank == 0) expect_bytes(set.full + 8 * pos.stage, bytes);
                if (!a.gather) tma_2d<kPair>(at, &a_map, k * kBox, t.p0 + kTileM * rank, bar);
                for (int i = 0; i < boxes; ++i) {
                    if (kMN) tma_3d<kPair>(bt + i * Sh::kBoxB, &w_map, n0 + i * kBoxMN, k * kBox, t.g, bar);
                    else tma_3d<kPair>(bt, &w_map, k * kBox, n0, t.g, bar);
                }
            }
        }
        if (is_dead(dead) && rank == 0) set.drain_copies(issued);
        if (kPair)   // the last arrivals from the first CTA's products
            for (int i = 0; i < S; ++i, pos.next()) bounded_wait_on<true>(set.empty + 8 * pos.stage, pos.phase ^ 1, dead);
    } else if (!kPair && warp >= 4 + kEpilogueWarps) {
        const int w = (warp - 4 - kEpilogueWarps) % kLoaderWarps;
        Item u;
        bool have = (!kTma || a.gather) && next_product(a, gr, item, step, BN, t);
        auto row_of = [&](const Item& x, int i) {   // of the tile's row i
            const int p = x.p0 + i;
            return p < x.p1 ? row_at(a.gather, a.M, p) : -1;
        };
        if constexpr (kTma) {
            constexpr int kPerA = kTileM / kCopyWarps, kPieces = kPerA / 32;   // rows of a warp; a lane holds one of each 32
            const int turn = w / kCopyWarps, first = w % kCopyWarps * kPerA;
            Copies<S> copies(turn);
            int n = 0, row[kPieces], row_next[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) row[i] = have ? row_of(t, first + 32 * i + lane) : -1;
            while (have && !is_dead(dead)) {
                const bool more = next_product(a, gr, item, step, BN, u);
#pragma unroll
                for (int i = 0; i < kPieces; ++i) row_next[i] = more ? row_of(u, first + 32 * i + lane) : -1;
                for (int k = 0; k < nk; ++k) {
                    if (n++ % kCopyGroups != turn) continue;
                    if (!copies.acquire(set.full, set.empty, dead)) break;
                    const uint32_t at = smem_u32(ring) + copies.stage() * Sh::kStage;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) copy_rows<32>(at, a.a, row[i], k * kBox, first + 32 * i, lane);
                    copies.issued();
                }
                t = u;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) row[i] = row_next[i];
                have = more;
            }
            copies.finish(set.full);
        } else {
            // two groups of warps take the stages in turn; while one stage of a group is turned, its next is copied
            // (rows that are not aligned take the room of both)
            constexpr int kPerA = kTileM / kLoaderWarps;
            auto lane_row = [&](const Item& x) { return row_of(x, kPerA * w + lane % kPerA); };
            int row = have ? lane_row(t) : -1;
            const int turn = (warp - 4 - kEpilogueWarps) / kLoaderWarps;
            constexpr uint32_t kStride = 32 * kLoaderWarps * 16;
            const bool aligned = a.a.aligned && a.w.aligned;
            const uint32_t stride = aligned ? kStride : 2 * kStride;
            unsigned char* mine = slots + turn * 2 * Sh::kParts * kStride + (w * 32 + lane) * (aligned ? 16 : 32);
            uint32_t offs_a = 0, offs_b = 0;
            int told = turn;   // the stage to be turned next
            auto turn_stage = [&](unsigned char* from) {
                const int st = told % S;
                if (!bounded_wait(set.empty + 8 * st, (uint32_t)(told / S & 1) ^ 1, dead)) return;
                unsigned char* at = ring + st * Sh::kStage;
                Sh::PartsA::turn(from, stride, aligned, offs_a, at, Sh::kA, w, lane);
                from += Sh::PartsA::kSteps * stride;
#pragma unroll
                for (int i = 0; i < Sh::kBoxes; ++i)
                    Sh::PartsB::turn(from + i * Sh::PartsB::kSteps * stride, stride, aligned, offs_b >> (4 * i * Sh::PartsB::kSteps),
                                     at + Sh::P * Sh::kA + i * Sh::kBoxB, Sh::kB, w, lane);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(set.full + 8 * st);
                told += 2;
            };
            int n = 0, copied = 0;
            while (have && !is_dead(dead)) {
                const bool more = next_product(a, gr, item, step, BN, u);
                const int row_next = more ? lane_row(u) : -1;
                Matrix wm = a.w;
                wm.p = static_cast<const T*>(wm.p) + t.g * a.w_group;
                for (int k = 0; k < nk; ++k) {
                    if ((n++ & 1) != turn) continue;
                    unsigned char* to = mine + (aligned ? (copied & 1) * Sh::kParts * kStride : 0);
                    const uint32_t to_s = smem_u32(to);
                    offs_a = Sh::PartsA::copy(a.a, row, k * kBox, to_s, stride, aligned, lane);
                    const int first = (kMN ? k * kBox : t.n0) + Sh::PartsB::kPer * w + lane % Sh::PartsB::kPer;
                    const int row_b = first < (kMN ? a.red : a.cols) ? first : -1;
                    offs_b = 0;
#pragma unroll
                    for (int i = 0; i < Sh::kBoxes; ++i)
                        offs_b |= Sh::PartsB::copy(wm, row_b, kMN ? t.n0 + i * kBoxMN : k * kBox,
                                                   to_s + (Sh::PartsA::kSteps + i * Sh::PartsB::kSteps) * stride, stride, aligned, lane)
                                  << (4 * i * Sh::PartsB::kSteps);
                    copies_commit();
                    ++copied;
                    if (!aligned) {
                        copies_wait<0>();
                        turn_stage(mine);
                    } else if (copied > 1) {
                        copies_wait<1>();
                        turn_stage(mine + (copied & 1) * Sh::kParts * kStride);
                    }
                }
                t = u;
                row = row_next;
                have = more;
            }
            copies_wait<0>();
            if (aligned && copied > 0 && !is_dead(dead)) turn_stage(mine + ((copied - 1) & 1) * Sh::kParts * kStride);
        }
    } else if (warp == 1 && rank == 0) {   // of a pair, for both
        RingPos<S> pos;
        Buffers<T> bufs;
        int n = 0, buf = 0;   // n of chunks (fp32), or tiles
        bool have = next_product(a, gr, item, step, BN, t);   // which tile it is does not matter here
        while (have && !is_dead(dead)) {
            for (int k = 0; k < nk; ++k, pos.next()) {
                if (k % kPerChunk == 0) {
                    buf = (kSums<T> > 1 || k == 0 ? n : n + 1) & 1;
                    bounded_wait_on<kPair>(set.tempty + 8 * buf, bufs.of(buf, n) ^ 1, dead);
                }
                bounded_wait_on<kPair>(set.full + 8 * pos.stage, pos.phase, dead);
                tc_fence_after();
                const uint32_t at = smem_u32(ring) + pos.stage * Sh::kStage;
                const int steps = (imin(kBox, a.red - k * kBox) + 15) / 16;
                issue_stage<T, false, kMN, BN, kPair>(set.tmem + buf * kSums<T> * BN, at, Sh::kA, 0, at + Sh::P * Sh::kA, Sh::kBoxB,
                                                      steps, k % kPerChunk > 0, set.empty + 8 * pos.stage);
                if (k == 0) have = next_product(a, gr, item, step, BN, t);   // looked for while products run
                if (k % kPerChunk == kPerChunk - 1 || k == nk - 1) {
                    tc_commit<kPair>(set.tfull + 8 * buf);
                    bufs.used(buf);
                    if (kSums<T> > 1 || k == nk - 1) ++n;
                }
            }
        }
        if (is_dead(dead)) set.drain_products();
    } else if (warp >= 4 && warp < 4 + 4 * Sh::kHalves) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        constexpr int kCols = BN / Sh::kHalves;
        unsigned char* stage = staging + (warp - 4) * kStageWarp;
        Buffers<T> bufs;
        int n = 0;
        auto ready = [&](int buf) {
            if (!bounded_wait(set.tfull + 8 * buf, bufs.of(buf, n), dead)) return false;
            bufs.used(buf);
            tc_fence_after();
            return true;
        };
        auto release = [&](int buf) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair) mbar_arrive_there(in_first(set.tempty + 8 * buf));
                else mbar_arrive(set.tempty + 8 * buf);
            }
        };
        while (!is_dead(dead) && next_item(a, gr, item, step, BN, t)) {
            const int p = t.p0 + kTileM * rank + 32 * q + lane;
            const int r = p < t.p1 ? row_at(a.perm, a.M, p) : -1;
            T* row = r >= 0 ? static_cast<T*>(a.out) + r * a.out_ld + t.n0 : nullptr;
            const int c0 = half * kCols, c1 = imin(c0 + kCols, a.cols - t.n0);
            if (t.g == a.G) {
                store_tile<T>(kNoTile, c0, c1, row, a.out_wide, stage, lane);
                continue;
            }
            const uint32_t lanes = set.tmem + ((uint32_t)(32 * q) << 16);
            if constexpr (kSums<T> == 1) {
                const int buf = n & 1, other = buf ^ 1;
                if (!ready(buf)) break;
                bool ok = true;
                for (int k = kPerChunk; k < nk && (ok = ready(other)); k += kPerChunk) {
                    add_tile(lanes + buf * BN, lanes + other * BN, c0, c0 + kCols);
                    release(other);
                }
                if (!ok) break;
                store_tile<T>(lanes + buf * BN, c0, c1, row, a.out_wide, stage, lane);
                release(buf);
                ++n;
            } else {
                static_assert(kSums<T> == 1 || kCols == 32, "a warp's columns of an fp32 tile fit one register array");
                float acc[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = 0.f;
                bool ok = true;
                for (int k = 0; k < nk; k += kPerChunk, ++n) {
                    const int buf = n & 1;
                    if (!(ok = ready(buf))) break;
                    const uint32_t from = lanes + buf * kSums<T> * BN + c0;
                    add_chunk(from, BN, acc);
                    release(buf);
                }
                if (!ok) break;
                if (c0 < c1) emit32<T>(acc, c1 - c0, row ? row + c0 : nullptr, a.out_wide, stage, lane);
            }
        }
    }
    set.end();
}

template <typename T, bool kTma, bool kMN, int BN, bool kPair = false>
zs_status launch_rows(const char* fn, RowsArgs a, cudaStream_t s) {
    using Sh = RowsShape<T, kTma, kMN, BN, kPair>;
    CUtensorMap a_map = {}, w_map = {};
    if (kTma) {
        constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
        const int w_rows = kMN ? a.red : a.cols;
        if (!encode_boxes(&a_map, bf16, a.a.p, a.red, a.M, a.a.ld, 0, kTileM) ||
            !encode_boxes(&w_map, bf16, a.w.p, a.w.cols, w_rows, a.w.ld, a.G, kMN ? kStageK<T> : Sh::kMine))
            return fail(ZS_ERR_CUDA, "%s: a tensor map was refused", fn);
    }
    a.ntiles = (a.cols + BN - 1) / BN;
    const int64_t items = ((int64_t)a.M / Sh::kTile + a.G + 2) * a.ntiles;
    if (items >= (int64_t(1) << 31) - 65536) return fail(ZS_ERR_INVALID_ARG, "%s: %lld tiles", fn, (long long)items);
    a.items = (int)items;
    constexpr auto kernel = rows_mma<T, kTma, kMN, BN, kPair>;
    constexpr int kCtas = kPair ? 2 : 1;
    static std::atomic<uint64_t> done[kMaxDevices];
    set_smem_limit_once(kernel, Sh::kSmem, done);
    launch_clusters(kCtas, kernel, dim3(kCtas * imin(a.items, num_sms() / kCtas)), dim3(Sh::kThreads), Sh::kSmem, s, a_map, w_map, a);
    return check_launch(fn);
}

// Rows of an average group from which on two CTAs form a tile of 256 rows, each
// with half of its weights, where the rows are in order: 32768 bf16 rows, 1024 ->
// 1024, 8 groups 52 us and 55 alone, 16 groups 52 and 61, 1024 -> 4096 170 and
// 192.  Gathered rows are limited by copies of their own (1024 -> 1024 94 and 83
// when that was measured), short groups by tiles that are mostly empty (256 rows: 50 and 40).
constexpr int kPairRows = 512;

// Whether tiles of 64 columns leave the SMs busier than wider ones: few tiles take few rounds, whose length is that of a
// tile's copies and epilogue (about its columns and kTileCost more) as long as the sums are short.  2048 bf16 rows, 256 ->
// 256: 6.6 us and 8.4; 1000 fp16 rows, 131 -> 131: 8.1 and 10.1; but 160 rows, sums of 3760, 784 columns: 77 and 64.
constexpr int kTileCost = 96, kShortSum = 512;
bool narrow_tiles(const RowsArgs& a, int bn) {
    if (a.red > kShortSum) return false;
    const int64_t rows = a.M / kTileM + imin(a.G, a.M);   // tiles of rows, at most
    auto cost = [&](int n) { return (rows * ((a.cols + n - 1) / n) + num_sms() - 1) / num_sms() * (n + kTileCost); };
    return 4 * cost(64) <= 3 * cost(bn);
}

template <typename T, bool kTma, bool kMN>
zs_status launch_rows(const char* fn, const RowsArgs& a, cudaStream_t s) {
    if constexpr (!kMN || sizeof(T) == 2)   // an MN-major plane of fp32 is a box wide
        if (a.cols <= 32) return launch_rows<T, kTma, kMN, 32>(fn, a, s);
    if constexpr (kTma) {
        const bool even = (a.cols + 127) / 128 % 2 == 0;
        if (a.cols > 64 && narrow_tiles(a, even ? 256 : 128)) return launch_rows<T, kTma, kMN, 64>(fn, a, s);
        if (a.cols > 64 && even)
            return !a.gather && a.M >= kPairRows * (int64_t)a.G ? launch_rows<T, kTma, kMN, 256, true>(fn, a, s) : launch_rows<T, kTma, kMN, 256>(fn, a, s);
    }
    if constexpr (sizeof(T) == 2)
        if (a.cols > 64) return launch_rows<T, kTma, kMN, 128>(fn, a, s);
    return launch_rows<T, kTma, kMN, 64>(fn, a, s);
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

// rows x_ld apart, rows of K weights w_ld apart; transposed: the gradient.
zs_status grouped_rows(const char* fn, int32_t dtype, const void* x, int64_t x_ld, const void* w, int64_t w_ld, const int32_t* row_ptr,
                       const int32_t* perm, const int32_t* gather, int64_t M, int32_t K, int32_t N, int32_t G, void* out, int64_t out_ld,
                       bool transposed, cudaStream_t s) {
    const int es = dtype_bytes(dtype), per16 = 16 / es;
    auto at = [&](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    RowsArgs a = {};
    a.red = transposed ? N : K;
    a.cols = transposed ? K : N;
    a.a = {x, x_ld, a.red, at(x, 16) && x_ld % per16 == 0};
    a.w = {w, w_ld, K, at(w, 16) && w_ld % per16 == 0};
    a.w_group = w_ld * N;
    a.row_ptr = row_ptr;
    a.perm = perm;
    a.gather = gather;
    a.out = out;
    a.out_ld = out_ld;
    a.out_wide = at(out, 16) && out_ld % per16 == 0 && a.cols % per16 == 0;
    a.M = (int)M;
    a.G = G;
    const bool aligned = a.a.aligned && a.w.aligned && G > 0;
    switch (dtype) {
        case ZS_F32: return rows_product<float>(fn, a, transposed, false, s);
        case ZS_BF16: return rows_product<__nv_bfloat16>(fn, a, transposed, aligned, s);
        default: return rows_product<__half>(fn, a, transposed, aligned, s);
    }
}

}  // namespace zs
