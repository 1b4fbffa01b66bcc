// How the gradient in the weights is shared out, whichever kernel forms it: the
// summed-over direction is the rows', whose groups' lengths are known on the
// device alone.  A unit of work is a stage's positions of one group for one
// 128 x BN tile of the weights; units are numbered tile by tile, and each CTA
// takes an equal range of them, so that skewed groups, few tiles and many
// tiles all keep every SM busy.  (Each group also counts kFlush units for
// writing its tile.)  A range cuts at most the group it starts in and the
// group it ends in: those two sums go to the workspace in fp32, and a second
// kernel adds, for each group that was cut, its CTAs' parts in order.  Which
// ones they are the first kernel notes down (note_join): to find it anew in
// each block of the second was a chain of loads that took it 5 us
// more (32768 rows of 89 groups, 256 x 256 bf16 weights).
#pragma once

#include "zs_mma.cuh"

namespace zs {

constexpr int kFlush = 2;        // units that writing a tile costs
constexpr int kPartRows = 4;     // rows of a tile that one CTA of the second kernel adds
template <typename T>
using WeightGroups = Groups<kStageK<T>, kFlush>;   // a unit's positions are a stage's

// A group that is cut where a CTA's range ends and that starts in this range.
struct JoinTile {
    int g;        // -1: none
    int tile;     // of the weights
    int last;     // the CTA that holds its end
    int part;     // which of the first CTA's partial tiles
};

struct WeightArgs {
    Matrix dy, x;
    const int32_t* row_ptr;
    const int32_t* perm;
    void* dw;
    float* partial;      // [CTA][2][128][BN]
    JoinTile* joins;     // [CTA]
    int cuts;            // ranges that end before the units do
    bool dw_wide;
    int M, G, N, K;
    int ktiles;
    int slots;           // units of a tile, empty ones of no group at its end among them
    int units, per;      // all units, units of a CTA
};

// The part of one group's sum for one tile that a CTA forms.
struct Segment {
    int g, n0, k0;
    int p0, p1;        // positions (none: an empty group, whose sum is zero)
    bool whole;        // all of the group's positions: written as it is
    int part;          // else which of the CTA's two partial tiles
};

// Walks the segments of a CTA's units.  Whole warps.
template <typename T, int BN>
struct Walk {
    const WeightArgs& a;
    const WeightGroups<T>& gr;
    int u, begin, end, last;
    __device__ __forceinline__ Walk(const WeightArgs& args, const WeightGroups<T>& groups)
        : a(args), gr(groups), u(blockIdx.x * args.per), begin(u), end(imin(u + args.per, args.units)), last(groups.slot(args.G)) {}
    __device__ __forceinline__ bool next(Segment& s) {
        while (u < end) {
            const int t = u / a.slots, first = t * a.slots, slot = u - first, from = u;
            if (slot >= last) {          // units of no group
                u = first + a.slots;
                continue;
            }
            s.g = gr.find(slot, a.G);
            const int g0 = gr.slot(s.g), b = gr.start(s.g), e = gr.start(s.g + 1);
            u = imin(end, first + gr.slot(s.g + 1));
            s.n0 = t / a.ktiles * kTileM;
            s.k0 = t % a.ktiles * BN;
            s.p0 = (int)imin<int64_t>(b + (int64_t)(slot - g0) * kStageK<T>, e);
            s.p1 = (int)imin<int64_t>(b + (int64_t)(u - first - g0) * kStageK<T>, e);
            s.whole = s.p0 == b && s.p1 == e;
            s.part = from == begin ? 0 : 1;
            if (s.p0 < s.p1 || (b == e && slot == g0)) return true;   // else only units that count for writing
        }
        return false;
    }
};

__device__ __forceinline__ int weight_row(const WeightArgs& a, int p) {
    if (!a.perm) return p;
    const int r = __ldg(a.perm + p);
    return (uint32_t)r < (uint32_t)a.M ? r : -1;
}

// Notes down what is cut at the end of this CTA's range.  By a whole warp, which waits for nothing.
template <typename T>
__device__ __forceinline__ void note_join(const WeightArgs& a, const WeightGroups<T>& gr) {
    JoinTile j = {-1, 0, 0, 0};
    const int cut = (blockIdx.x + 1) * a.per;
    if (cut < a.units) {
        const int t = cut / a.slots, slot = cut - t * a.slots;
        if (slot < gr.slot(a.G)) {
            const int g = gr.find(slot, a.G);
            const int b = gr.start(g), e = gr.start(g + 1);
            const int u0 = t * a.slots + gr.slot(g), u1 = u0 + (e - b + kStageK<T> - 1) / kStageK<T>;   // units with positions
            // it is cut here, and no earlier range holds positions of it
            if (u0 < cut && u1 > cut && u0 / a.per == (int)blockIdx.x)
                j = {g, t, (u1 - 1) / a.per, u0 != (int)blockIdx.x * a.per};
        }
    }
    if ((threadIdx.x & 31) == 0 && blockIdx.x + 1 < gridDim.x) a.joins[blockIdx.x] = j;
}

// Adds the parts of a group that is cut, the first one formed by CTA `first`:
// rows y * kPartRows .. of its tile, 4 columns a thread.
template <typename T, int BN>
__device__ __forceinline__ void join_tile(const WeightArgs& a, int4 note, int first) {
    const int g = note.x, t = note.y, last = note.z, first_part = note.w;
    if (g < 0) return;
    const int n0 = t / a.ktiles * kTileM + blockIdx.y * kPartRows, k0 = t % a.ktiles * BN;
    const int cols = imin(BN, a.K - k0), rows = imin(kPartRows, a.N - n0);
    constexpr int64_t kTile = (int64_t)kTileM * BN;
    // a thread adds four columns over its share of the parts, then the shares' sums are added in order
    constexpr int kItems = kPartRows * BN / 4, kShares = 256 / kItems;
    static_assert(kItems <= 256 && 256 % kItems == 0, "whole shares");
    __shared__ float4 sums[256];
    const int item = threadIdx.x % kItems, share = threadIdx.x / kItems;
    const int r = item / (BN / 4), c = item % (BN / 4) * 4;
    const bool in = r < rows && c < cols;
    const int parts = last - first + 1, each = (parts + kShares - 1) / kShares;
    const int p0 = first + share * each, p1 = imin(p0 + each, last + 1);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
        const float* at = a.partial + ((int64_t)blockIdx.y * kPartRows + r) * BN + c;
#pragma unroll 8
        for (int p = p0; p < p1; ++p)
            sum = f4_add(sum, ld_ro4(at + ((int64_t)p * 2 + (p == first ? first_part : 0)) * kTile));
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (share == 0 && in) {
#pragma unroll
        for (int i = 1; i < kShares; ++i) sum = f4_add(sum, sums[i * kItems + item]);
        T* out = static_cast<T*>(a.dw) + ((int64_t)g * a.N + n0 + r) * a.K + k0 + c;
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) out[j] = from_f32<T>(v[j]);
    }
    __syncthreads();   // sums
}

// Block (x, y): what was cut of which one of CTAs kNotes x .. formed the first
// part (often nothing: a block that only looks and leaves takes its time too).
constexpr int kNotes = 4;
template <typename T, int BN>
__global__ void __launch_bounds__(256) weights_join(const WeightArgs a) {
    pdl_wait();
    pdl_trigger();
    int4 notes[kNotes];
#pragma unroll
    for (int i = 0; i < kNotes; ++i) {
        const int x = blockIdx.x * kNotes + i;
        notes[i] = x < a.cuts ? __ldg(reinterpret_cast<const int4*>(a.joins) + x) : make_int4(-1, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kNotes; ++i) join_tile<T, BN>(a, notes[i], blockIdx.x * kNotes + i);
}

// The gradient in fp32 where grouped_is_small() (zs_grouped_small.cu): one tile of 32 columns.
zs_status grouped_small_weights(const char* fn, const WeightArgs& a, int ctas, cudaStream_t s);

}  // namespace zs
