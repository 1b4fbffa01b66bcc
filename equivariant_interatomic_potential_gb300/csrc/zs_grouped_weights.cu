// Grouped products' gradient in the weights: dw[g] = sum over the rows of
// group g of dy[i]^T x[i].
//
// Both operands have the summed-over direction across their memory rows
// (MN-major boxes); zs_grouped_walk.cuh says how the work is shared out.
//
// 32768 bf16 rows in order, 8 groups of 1024 -> 4096: 238 us (1.16 PFLOP/s), of
// which the copies alone take 214 (48 KB a stage, six boxes); 89 groups of 256 ->
// 256, gathered: 30 us with the joining kernel, bound by the partial tiles.
#include <initializer_list>

#include "zs_grouped.cuh"
#include "zs_grouped_walk.cuh"

namespace zs {

namespace {

template <typename T, bool kTma, int BN>
struct WeightShape {
    static constexpr int P = kPlanes<T>, kUnit = kStageK<T>;
    static constexpr int kABoxes = kTileM / kBoxMN, kBBoxes = (BN + kBoxMN - 1) / kBoxMN;
    static constexpr uint32_t kBox = box_bytes<kBoxMN>(kUnit);
    static constexpr uint32_t kA = kABoxes * kBox, kB = kBBoxes * kBox;
    static constexpr uint32_t kStage = P * (kA + kB);
    // what the loader warps copy into before they turn it, as in the products over rows
    using Parts = BoxParts<T, kUnit, kBoxMN>;
    static constexpr int kParts = (kABoxes + kBBoxes) * Parts::kSteps;
    static constexpr int kSlots = kTma ? 0 : 4 * kParts * 32 * kLoaderWarps * 16;
    static constexpr int kHalves = BN >= 64 ? 2 : 1;   // warps that share 32 rows of a tile
    static constexpr uint32_t kTmemCols = tmem_cols(2 * kSums<T> * BN);
    static constexpr int kFixed = kSlots + kEpilogueWarps * kStageWarp + 1024 + 4608;   // staging, alignment, barriers and groups
    static constexpr int kFit = (kSmemMost - kFixed) / (int)kStage;
    static constexpr int S = kFit > 8 ? 8 : kFit;
    static_assert(kPlanes<T> == 1 || BN == kBoxMN, "the planes of the right operand follow each other");
    static_assert(S >= 2 && Setup<S, kTmemCols, kUnit, kFlush>::kBytes <= 4608, "two stages at least");
    static constexpr int kSmem = S * (int)kStage + kFixed;
    static constexpr int kThreads = 32 * (4 + kEpilogueWarps + (kTma ? 1 : 2) * kLoaderWarps);
};

template <typename T, bool kTma, int BN>
__global__ void __launch_bounds__(WeightShape<T, kTma, BN>::kThreads, 1)
weights_mma(const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap x_map, const WeightArgs a) {
    using Sh = WeightShape<T, kTma, BN>;
    constexpr int S = Sh::S;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* slots = ring + S * Sh::kStage;
    unsigned char* staging = slots + Sh::kSlots;
    constexpr int kUnit = Sh::kUnit;
    Setup<S, Sh::kTmemCols, kUnit, kFlush> set;
    set.begin(staging + kEpilogueWarps * kStageWarp, !kTma ? kLoaderWarps : a.perm ? kCopyWarps : 1, 4 * Sh::kHalves, a.row_ptr, a.G, a.M);
    volatile int* dead = set.dead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Walk<T, BN> walk(a, set.groups);
    Segment s;
    constexpr int kPerChunk = kSums<T> > 1 ? kChunk : kLongSum;   // positions between hand-overs to the epilogue

    if (kTma && warp == 0 && !a.perm) {
        RingPos<S> pos;
        int issued = 0;
        while (!is_dead(dead) && walk.next(s)) {
            const int a_boxes = imin(2, (a.N - s.n0 + kBoxMN - 1) / kBoxMN);
            const int b_boxes = imin(Sh::kBBoxes, (a.K - s.k0 + kBoxMN - 1) / kBoxMN);
            for (int p = s.p0; p < s.p1; p += kUnit, ++issued, pos.next()) {
                bounded_wait_on(set.empty + 8 * pos.stage, pos.phase ^ 1, dead);
                if (is_dead(dead)) break;
                const uint32_t bar = set.full + 8 * pos.stage, at = smem_u32(ring) + pos.stage * Sh::kStage, bt = at + Sh::kA;
                expect_bytes(bar, (a_boxes + b_boxes) * Sh::kBox);
                for (int i = 0; i < a_boxes; ++i) tma_2d(at + i * Sh::kBox, &dy_map, s.n0 + i * kBoxMN, p, bar);
                for (int i = 0; i < b_boxes; ++i) tma_2d(bt + i * Sh::kBox, &x_map, s.k0 + i * kBoxMN, p, bar);
            }
        }
        if (is_dead(dead)) set.drain_copies(issued);
    } else if (warp >= 4 + kEpilogueWarps && (!kTma || a.perm)) {
        const int w = (warp - 4 - kEpilogueWarps) % kLoaderWarps;
        constexpr int kPer = kUnit / (kTma ? kCopyWarps : kLoaderWarps);
        auto row_of = [&](int p) {   // lane i (mod kPer): the row at the warp's position i
            const int at = p + kPer * (kTma ? w % kCopyWarps : w) + lane % kPer;
            return at < s.p1 ? weight_row(a, at) : -1;
        };
        if constexpr (kTma) {
            const int turn = w / kCopyWarps, part = w % kCopyWarps;
            Copies<S> copies(turn);
            int n = 0;
            while (!is_dead(dead) && walk.next(s)) {
                int row = row_of(s.p0);
                for (int p = s.p0; p < s.p1; p += kUnit) {
                    const int mine = row;
                    row = row_of(p + kUnit);
                    if (n++ % kCopyGroups != turn) continue;
                    if (!copies.acquire(set.full, set.empty, dead)) break;
                    const uint32_t at = smem_u32(ring) + copies.stage() * Sh::kStage;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (s.n0 + i * kBoxMN < a.N) copy_rows<kPer>(at + i * Sh::kBox, a.dy, mine, s.n0 + i * kBoxMN, kPer * part, lane);
#pragma unroll
                    for (int i = 0; i < Sh::kBBoxes; ++i)
                        if (s.k0 + i * kBoxMN < a.K) copy_rows<kPer>(at + Sh::kA + i * Sh::kBox, a.x, mine, s.k0 + i * kBoxMN, kPer * part, lane);
                    copies.issued();
                }
            }
            copies.finish(set.full);
        } else {
            // two groups of warps take the stages in turn; while one stage of a group is turned, its next is copied
            // (rows that are not aligned take the room of both)
            using Parts = typename Sh::Parts;
            const int turn = (warp - 4 - kEpilogueWarps) / kLoaderWarps;
            constexpr uint32_t kStride = 32 * kLoaderWarps * 16;
            const bool aligned = a.dy.aligned && a.x.aligned;
            const uint32_t stride = aligned ? kStride : 2 * kStride;
            unsigned char* mine = slots + turn * 2 * Sh::kParts * kStride + (w * 32 + lane) * (aligned ? 16 : 32);
            constexpr int kAll = Sh::kABoxes + Sh::kBBoxes;
            uint32_t offs[kAll] = {};
            int told = turn;   // the stage to be turned next
            auto turn_stage = [&](const unsigned char* from) {
                const int st = told % S;
                if (!bounded_wait(set.empty + 8 * st, (uint32_t)(told / S & 1) ^ 1, dead)) return;
                unsigned char* at = ring + st * Sh::kStage;
#pragma unroll
                for (int i = 0; i < kAll; ++i) {
                    const bool of_a = i < Sh::kABoxes;
                    Parts::turn(from + i * Parts::kSteps * stride, stride, aligned, offs[i],
                                of_a ? at + i * Sh::kBox : at + Sh::P * Sh::kA + (i - Sh::kABoxes) * Sh::kBox,
                                of_a ? Sh::kA : Sh::kB, w, lane);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(set.full + 8 * st);
                told += 2;
            };
            int n = 0, copied = 0;
            while (!is_dead(dead) && walk.next(s)) {
                int row = row_of(s.p0);
                for (int p = s.p0; p < s.p1; p += kUnit) {
                    const int here = row;
                    row = row_of(p + kUnit);
                    if ((n++ & 1) != turn) continue;
                    unsigned char* to = mine + (aligned ? (copied & 1) * Sh::kParts * kStride : 0);
                    const uint32_t to_s = smem_u32(to);
#pragma unroll
                    for (int i = 0; i < kAll; ++i) {
                        const bool of_a = i < Sh::kABoxes;
                        offs[i] = Parts::copy(of_a ? a.dy : a.x, here, of_a ? s.n0 + i * kBoxMN : s.k0 + (i - Sh::kABoxes) * kBoxMN,
                                              to_s + i * Parts::kSteps * stride, stride, aligned, lane);
                    }
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
            }
            copies_wait<0>();
            if (aligned && copied > 0 && !is_dead(dead)) turn_stage(mine + ((copied - 1) & 1) * Sh::kParts * kStride);
        }
    } else if (warp == 1) {
        RingPos<S> pos;
        Buffers<T> bufs;
        int n = 0, buf = 0;   // n of chunks (fp32), or segments
        // a stage's products
        auto products = [&](int p) {
            const int since = (p - s.p0) % kPerChunk, steps = (imin(kUnit, s.p1 - p) + 15) / 16;
            const uint32_t at = smem_u32(ring) + pos.stage * Sh::kStage;
            tc_fence_after();
            issue_stage<T, true, true, BN>(set.tmem + buf * kSums<T> * BN, at, Sh::kA, Sh::kBox, at + Sh::P * Sh::kA, Sh::kBox,
                                           steps, since > 0, set.empty + 8 * pos.stage);
            if (since + kUnit >= kPerChunk || p + kUnit >= s.p1) {
                tc_commit<false>(set.tfull + 8 * buf);
                bufs.used(buf);
                if (kSums<T> > 1 || p + kUnit >= s.p1) ++n;
            }
        };
        auto ready = [&](int p) {
            if ((p - s.p0) % kPerChunk == 0) {
                buf = (kSums<T> > 1 || p == s.p0 ? n : n + 1) & 1;
                bounded_wait_on(set.tempty + 8 * buf, bufs.of(buf, n) ^ 1, dead);
            }
            bounded_wait_on(set.full + 8 * pos.stage, pos.phase, dead);
        };
        while (!is_dead(dead) && walk.next(s)) {
            // positions past the segment's end hold other rows where TMA brought them: they count as zeros
            const bool ragged = kTma && !a.perm && (s.p1 - s.p0) % 16 != 0;
            for (int p = s.p0; p < s.p1; p += kUnit, pos.next()) {
                ready(p);
                if (ragged && p + kUnit > s.p1) {
                    const int rows = s.p1 - p, pieces = (((rows + 15) & ~15) - rows) * (kBoxMN / 8);
                    unsigned char* at = ring + pos.stage * Sh::kStage + rows * (kBoxMN * 2);
                    for (int i = lane; i < pieces * (Sh::kABoxes + Sh::kBBoxes); i += 32)
                        *reinterpret_cast<uint4*>(at + i / pieces * Sh::kBox + i % pieces * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                products(p);
            }
        }
        if (is_dead(dead)) set.drain_products();
    } else if (warp == 3) {
        note_join<T>(a, set.groups);
    } else if (warp >= 4 && warp < 4 + 4 * Sh::kHalves) {
        const int q = warp & 3, half = (warp - 4) >> 2, r = 32 * q + lane;
        constexpr int kMine = BN / Sh::kHalves;
        unsigned char* stage = staging + (warp - 4) * kStageWarp;
        const uint32_t lanes = set.tmem + ((uint32_t)(32 * q) << 16);
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
            if (lane == 0) mbar_arrive(set.tempty + 8 * buf);
        };
        while (!is_dead(dead) && walk.next(s)) {
            const bool some = s.p0 < s.p1, mine = s.n0 + r < a.N;
            const int c0 = half * kMine, c1 = imin(c0 + kMine, a.K - s.k0);
            T* row = mine ? static_cast<T*>(a.dw) + ((int64_t)s.g * a.N + s.n0 + r) * a.K + s.k0 : nullptr;
            float* part = mine ? a.partial + (((int64_t)blockIdx.x * 2 + s.part) * kTileM + r) * BN : nullptr;
            const int c1_part = imin((c1 + 3) / 4 * 4, c0 + kMine);   // whole pieces of a partial tile's rows
            if constexpr (kSums<T> == 1) {
                const int buf = n & 1, other = buf ^ 1;
                bool ok = !some || ready(buf);
                for (int done = kPerChunk; done < s.p1 - s.p0 && (ok = ok && ready(other)); done += kPerChunk) {
                    add_tile(lanes + buf * BN, lanes + other * BN, c0, c0 + kMine);
                    release(other);
                }
                if (!ok) break;
                const uint32_t from = some ? lanes + buf * BN : kNoTile;
                if (s.whole) store_tile<T>(from, c0, c1, row, a.dw_wide, stage, lane);
                else store_tile<float>(from, c0, c1_part, part, true, stage, lane);
                if (some) {
                    release(buf);
                    ++n;
                }
            } else {
                static_assert(kSums<T> == 1 || kMine == 32, "a warp's columns of an fp32 tile fit one register array");
                float acc[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = 0.f;
                bool ok = true;
                for (int p = s.p0; p < s.p1; p += kPerChunk, ++n) {
                    const int buf = n & 1;
                    if (!(ok = ready(buf))) break;
                    const uint32_t from = lanes + buf * kSums<T> * BN + c0;
                    add_chunk(from, BN, acc);
                    release(buf);
                }
                if (!ok) break;
                if (c0 >= c1) continue;
                if (s.whole) emit32<T>(acc, c1 - c0, row ? row + c0 : nullptr, a.dw_wide, stage, lane);
                else emit32<float>(acc, c1_part - c0, part ? part + c0 : nullptr, true, stage, lane);
            }
        }
    }
    set.end();
}

// Tiles and ranges of a problem; the same on every device, so that the
// workspace's size is too.  One CTA for each of the 152 SMs; short rows take
// little room, and four of theirs.
constexpr int kCtas = 152;
constexpr int64_t kL2Bytes = 100 << 20;   // what of an operand stays in L2
struct WeightPlan {
    bool small;          // the CUDA cores form it (zs_grouped_small.cu)
    int bn;
    int64_t slots, units, per;
    int ctas;
};
WeightPlan weight_plan(int32_t dtype, bool tma, int64_t M, int32_t K, int32_t N, int32_t G) {
    WeightPlan p;
    p.small = dtype == ZS_F32 && grouped_is_small(K, N);   // 16 bits: 19 us on the tensor cores, 25 without (65536 rows)
    p.bn = p.small ? 32 : dtype == ZS_F32 ? 64 : K <= 32 ? 32 : K <= 64 ? 64 : (K + 127) / 128 % 2 || !tma ? 128 : 256;
    p.slots = M / (dtype == ZS_F32 ? kStageK<float> : kStageK<__half>) + (int64_t)G * kFlush;
    p.units = p.slots * ((N + kTileM - 1) / kTileM) * ((K + p.bn - 1) / p.bn);
    const int most = p.small ? 4 * kCtas : kCtas;
    p.per = (p.units + most - 1) / most;
    // Where tiles share an operand that L2 does not hold, ranges that start at the same positions of their tiles read it
    // from memory once: 32768 x 4096 and 32768 x 1024 bf16, 128 tiles, take 250 us on 128 SMs so and 272 on all 152 with
    // equal ranges.  Where it does not matter, fewer SMs do: 32768 x 1360 and 32768 x 216 79 and 74 us.
    const int64_t ntiles = (N + kTileM - 1) / kTileM, ktiles = (K + p.bn - 1) / p.bn, tiles = ntiles * ktiles;
    const int64_t row = dtype_bytes(dtype) * imax(ktiles > 1 ? (int64_t)N : 0, ntiles > 1 ? (int64_t)K : 0);
    if (!p.small && M * row > kL2Bytes) {
        const int64_t pieces = most / tiles, rounds = (tiles + most - 1) / most;   // ranges of a tile, or tiles of a range
        const int64_t per = pieces ? (p.slots + pieces - 1) / pieces : p.slots * rounds;
        if ((p.units + per - 1) / per >= most * 4 / 5) p.per = per;
    }
    p.ctas = p.per ? (int)((p.units + p.per - 1) / p.per) : 0;
    return p;
}

template <typename T, bool kTma, int BN>
zs_status launch_weights(const char* fn, WeightArgs a, const WeightPlan& p, cudaStream_t s) {
    using Sh = WeightShape<T, kTma, BN>;
    CUtensorMap dy_map = {}, x_map = {};
    if (kTma) {
        constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
        if (!a.perm && (!encode_boxes(&dy_map, bf16, a.dy.p, a.N, a.M, a.dy.ld, 0, kStageK<T>) ||
                        !encode_boxes(&x_map, bf16, a.x.p, a.K, a.M, a.x.ld, 0, kStageK<T>)))
            return fail(ZS_ERR_CUDA, "%s: a tensor map was refused", fn);
    }
    static std::atomic<uint64_t> done[kMaxDevices];
    set_smem_limit_once(weights_mma<T, kTma, BN>, Sh::kSmem, done);
    launch(weights_mma<T, kTma, BN>, dim3(p.ctas), dim3(Sh::kThreads), Sh::kSmem, s, dy_map, x_map, a);
    if (zs_status st = check_launch(fn)) return st;
    if (p.ctas > 1) {
        launch(weights_join<T, BN>, dim3((a.cuts + kNotes - 1) / kNotes, kTileM / kPartRows), dim3(256), 0, s, a);
        return check_launch(fn);
    }
    return ZS_OK;
}

template <typename T, bool kTma>
zs_status launch_weights(const char* fn, const WeightArgs& a, const WeightPlan& p, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (p.bn == 32) return launch_weights<T, kTma, 32>(fn, a, p, s);
        if constexpr (kTma)
            if (p.bn == 256) return launch_weights<T, kTma, 256>(fn, a, p, s);
        if (p.bn == 128) return launch_weights<T, kTma, 128>(fn, a, p, s);
    }
    return launch_weights<T, kTma, 64>(fn, a, p, s);
}

}  // namespace

unsigned int take_timeouts_grouped_weights() { return take_timeouts_local(); }
cudaError_t set_timeout_flag_grouped_weights(unsigned int* flag) { return set_timeout_flag_local(flag); }

size_t grouped_weights_workspace(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    size_t bytes = 0;
    for (bool tma : {false, true}) {   // which one depends on the operands' alignment
        const WeightPlan p = weight_plan(dtype, tma, M, K, N, G);
        if (p.ctas > 1 && !(tma && dtype == ZS_F32)) bytes = imax(bytes, (size_t)p.ctas * (2 * kTileM * p.bn * 4 + sizeof(JoinTile)));
    }
    return align_up(bytes, 256);
}

zs_status grouped_weights(const char* fn, int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                          const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dw,
                          void* workspace, cudaStream_t s) {
    const int es = dtype_bytes(dtype), per16 = 16 / es;
    auto at = [&](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const bool tma = dtype != ZS_F32 && at(dy, 16) && dy_ld % per16 == 0 && at(x, 16) && x_ld % per16 == 0 && M > 0;
    const WeightPlan p = weight_plan(dtype, tma, M, K, N, G);
    if (p.units + p.per >= int64_t(1) << 31) return fail(ZS_ERR_INVALID_ARG, "%s: %lld units", fn, (long long)p.units);
    WeightArgs a = {};
    a.dy = {dy, dy_ld, N, at(dy, 16) && dy_ld % per16 == 0};
    a.x = {x, x_ld, K, at(x, 16) && x_ld % per16 == 0};
    a.row_ptr = row_ptr;
    a.perm = perm;
    a.dw = dw;
    a.partial = static_cast<float*>(workspace);
    a.cuts = p.ctas - 1;
    a.joins = reinterpret_cast<JoinTile*>(a.partial + (int64_t)p.ctas * 2 * kTileM * p.bn);
    a.dw_wide = at(dw, 16) && K % per16 == 0;
    a.M = (int)M, a.G = G, a.N = N, a.K = K;
    a.ktiles = (K + p.bn - 1) / p.bn;
    a.slots = (int)p.slots, a.units = (int)p.units, a.per = (int)p.per;
    if (p.small) return grouped_small_weights(fn, a, p.ctas, s);
    switch (dtype) {
        case ZS_F32: return launch_weights<float, false>(fn, a, p, s);
        case ZS_BF16: return tma ? launch_weights<__nv_bfloat16, true>(fn, a, p, s)
                                     : launch_weights<__nv_bfloat16, false>(fn, a, p, s);
        default: return tma ? launch_weights<__half, true>(fn, a, p, s) : launch_weights<__half, false>(fn, a, p, s);
    }
}

}  // namespace zs
