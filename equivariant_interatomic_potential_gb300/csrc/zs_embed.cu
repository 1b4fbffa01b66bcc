// Embedding: rows of a table by id, scaled, and the table's gradient from a
// CSR of the ids.
//
// Forward: y[i] = scale * w[ids[i]], one pass that writes M C elements and
// reads the rows it needs (move_rows).  Bound by what it writes: 647170 rows of
// 96 floats of a table of 3 MB in 43 us, 5.8 TB/s.
//
// Gradient: dw[v] = scale * sum of dy[perm[j]] over the positions j of CSR row
// v.  A row of dw is written once and a row of dy read once, both C elements,
// so that "position j" and "end of row v" cost the same: they are merged into
// one list of M + V items (the end of row v comes after its positions, as item
// row_ptr[v + 1] + v) that is cut into equal shares, however skewed the ids
// and however many rows of the table have none.  A CTA takes one share of the
// list and up to 256 pieces of the columns: it stages its part of row_ptr and
// perm in shared memory, its threads (a share of the CTA's items and a piece
// each) walk their items, six rows on their way while six are added, and what is
// cut between its threads is added up in shared memory.  What is cut between
// CTAs goes to the workspace in fp32 and is added up by a second kernel in the
// CTAs' order.  All sums are in fp32 and in an order that follows from the sizes
// and the ids.  As many CTAs as run at once: the search for a share's first row
// and the staging take about 5 us, in which nothing else runs (24 CTAs an SM: 71
// instead of 46 us).  Both kernels, 647170 rows of 96 floats, skewed over 7921
// ids: 47 us, 5.4 TB/s; 16384 rows of 1024 bf16 and a table of 50021: 33 us, 4.2
// TB/s, of which the join is about 4.
#include "zs_rows.cuh"

namespace zs {
namespace {

struct IdSource {
    static constexpr bool kScaled = true, kAgain = true;   // rows are read again: they may stay in L1
    const int32_t* ids;
    int32_t V;
    __device__ __forceinline__ int32_t row(int32_t i, bool) const {
        const int32_t v = __ldg(ids + i);
        return (uint32_t)v < (uint32_t)V ? v : -1;
    }
};

template <typename T, bool kWhole>
zs_status embed_forward(const void* w, int64_t w_ld, int32_t V, const int32_t* ids, int64_t M, int32_t C, float scale, void* y,
                        int64_t y_ld, cudaStream_t s) {
    constexpr int U = 4;
    const MoveShape shape = move_rows_shape<T, kWhole>(M, C, U);
    launch(move_rows<T, kWhole, U, IdSource>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape, IdSource{ids, V},
           Rows<T>(w, V, w_ld, C), scale, static_cast<T*>(y), y_ld);
    return check_launch("embedding");
}

// ------------------------------------------------------------------ gradient

constexpr int kSumThreads = 256;
constexpr int kSumBatch = 6;         // rows of dy that a thread loads at a time (of 80 registers: 32 to 46 bytes are spilled
                                     // for 16-bit rows of whole pieces and fp32 rows of others, 4 for fp32 ones of whole pieces)
constexpr int kSumMaxC = 1 << 23;    // columns (of the grids)
constexpr int kSumItems = 4096;      // most items of a CTA (staged in shared memory)
constexpr int kSumCluster = 8;       // CTAs of a cluster, which adds up what is cut between them itself: where they
constexpr int kSumFew = 32;          // have no more than kSumFew items a thread (512 rows, 89 ids, 128 bf16: 6.1 us with
                                     // one kernel, 7.3 with two; 2000 rows, 300 ids, 256: 11 with few CTAs, 7.4 with two)
constexpr int kSumCtas = 3;          // CTAs an SM that the shares are made for: as many as run at once

struct SumShape {
    int64_t M, items;                // items: M + V
    int32_t V, C, P;
    int32_t cols;                    // pieces of a CTA, of P
    int32_t units, per_unit;         // shares of a CTA's items, items of each
    int32_t ctas, ctas_y;
    bool cluster;                    // few CTAs: a cluster of them adds up what is cut itself
    FastDiv by_cols;
    int64_t share() const { return (int64_t)units * per_unit; }
};

inline SumShape sum_shape(int64_t M, int32_t V, int32_t C, int vec) {
    SumShape s = {};
    s.M = M;
    s.V = V;
    s.C = C;
    s.items = M + V;
    s.P = (C + vec - 1) / vec;
    // Columns are cut so that few threads idle: of 256, P of them in each of as many units as fit.  Up to four CTAs a row more
    // than the least are tried, until five threads of six have work (132 pieces: one CTA has 132 at work, of three each 220).
    const int least = (s.P + kSumThreads - 1) / kSumThreads;
    int64_t best = 0;
    for (int y = least; y <= imin(least + 4, s.P) && best < (int64_t)kSumThreads * 5 / 6 * 1000; ++y) {
        const int cols = (s.P + y - 1) / y, units = kSumThreads / cols;
        const int64_t busy = (int64_t)s.P * units * 1000 / y;   // threads of a CTA, on average, in thousandths
        if (busy > best) best = busy, s.cols = cols, s.units = units, s.ctas_y = y;
    }
    const int64_t few = (s.items + kSumCluster * s.units - 1) / (kSumCluster * s.units);
    s.cluster = few <= imin(kSumFew, kSumItems / s.units);
    const int64_t target = imax<int64_t>(1, (int64_t)num_sms() * kSumCtas / s.ctas_y);
    const int64_t per = s.cluster ? few : (s.items + target * s.units - 1) / (target * s.units);
    s.per_unit = (int32_t)imax<int64_t>(imin<int64_t>(imax<int64_t>(per, kSumBatch), kSumItems / s.units), 1);
    s.ctas = (int32_t)((s.items + s.share() - 1) / s.share());
    s.by_cols = FastDiv((uint32_t)s.cols);
    return s;
}

// Of each CTA of the first kernel: the row that it closes and others have begun (or -1), and the CTA that began it.
struct SumNote {
    int32_t row, first;
};

// Rows that end before item d of the merged list: how many v have row_ptr[v + 1] + v < d.  By `kSumThreads / 2` threads,
// the two halves of the CTA with a d each: rounds of as many samples at even distances, two of them for 16000 rows.
__device__ __forceinline__ int rows_before(const int32_t* row_ptr, int32_t V, int64_t d, int (*first)[kSumThreads / 64]) {
    constexpr int N = kSumThreads / 2;
    const int t = threadIdx.x % N, half = threadIdx.x / N, lane = threadIdx.x & 31;
    int64_t lo = 0, hi = V;
    while (__syncthreads_or(lo < hi)) {
        const int64_t step = (hi - lo + N - 1) / N, at = lo + t * step;
        const bool ge = lo < hi && (at >= hi || (int64_t)__ldg(row_ptr + at + 1) + at >= d);
        const unsigned m = __ballot_sync(0xffffffffu, ge);
        if (lane == 0) first[half][t >> 5] = m ? (t & ~31) + __ffs(m) - 1 : N;   // the first sample that is not before d
        __syncthreads();
        if (lo >= hi) continue;
        int f = N;
#pragma unroll
        for (int w = 0; w < N / 32; ++w) f = imin(f, first[half][w]);
        hi = imin(lo + f * step, hi);
        if (f > 0) lo += (f - 1) * step + 1;
        if (lo > hi) lo = hi;
    }
    return (int)lo;
}

template <typename T, bool kWhole, bool kCluster>
__global__ void __launch_bounds__(kSumThreads, kSumCtas) sum_rows(SumShape s, Rows<T> dy, const int32_t* __restrict__ row_ptr,
                                                                  const int32_t* __restrict__ perm, float scale, T* __restrict__ dw,
                                                                  float* __restrict__ head, float* __restrict__ tail,
                                                                  SumNote* __restrict__ notes) {
    using R = Row<T, kWhole, sizeof(T) == 4>;
    // rows at a time; of words that are shifted one (and the next ones' in flight): 16384 of 50021, 1023 bf16: 47 us, two 59
    constexpr int VEC = R::N, kBatch = R::kOnePhase ? kSumBatch : 1;
    __shared__ int32_t staged[kSumItems + 8];        // row_ptr[v0 .. v1 + 1], then perm[j0 .. j1)
    __shared__ int32_t bound[2];
    __shared__ int32_t unit_row[kSumThreads + 1];    // rows that end before each unit
    __shared__ float open[kSumThreads * VEC];        // sums of rows that a unit leaves open
    __shared__ int samples[2][kSumThreads / 64];
    __shared__ int32_t begun_by;                     // the CTA that began the row which ends here and was begun before, or -1
    const int tid = threadIdx.x;
    const int64_t share = (int64_t)s.units * s.per_unit;
    const int64_t d0 = blockIdx.x * share, d1 = imin(d0 + share, s.items);
    pdl_wait();
    pdl_trigger();
    const int32_t held = __ldg(row_ptr + s.V);       // positions of some id: those behind are not read
    if (gridDim.x == 1) {
        if (tid == 0) bound[0] = 0, bound[1] = s.V;
    } else {
        const int v = rows_before(row_ptr, s.V, tid < kSumThreads / 2 ? d0 : d1, samples);
        if (tid % (kSumThreads / 2) == 0) bound[tid / (kSumThreads / 2)] = v;
    }
    __syncthreads();
    const int v0 = bound[0], v1 = bound[1];
    const int64_t j0 = imax<int64_t>(imin(d0 - v0, s.M), 0), j1 = imax(imin(d1 - v1, s.M), j0);
    // v1 - v0 rows end here and one more may be open: v1 - v0 + 2 bounds, and j1 - j0 positions, together at most the
    // share and two (and no more than fits, whatever row_ptr holds)
    const int rows = imax(imin(v1 - v0, kSumItems), 0), bounds = rows + 2;
    const int count = (int)imax<int64_t>(imin<int64_t>(imin<int64_t>(j1, held) - j0, kSumItems + 8 - bounds), 0);
    for (int i = tid; i < bounds; i += kSumThreads) staged[i] = v0 + i <= s.V ? __ldg(row_ptr + v0 + i) : (int32_t)s.M;
    int32_t* sperm = staged + bounds;
    for (int i = tid; i < count; i += kSumThreads) sperm[i] = __ldg(perm + j0 + i);
    __syncthreads();
    if (tid == 0) {                                  // items are below 2^32
        const int64_t begin = (int64_t)staged[0] + v0;
        begun_by = rows > 0 && begin < d0 ? (int32_t)((uint32_t)imax<int64_t>(begin, 0) / (uint32_t)share) : -1;
    }
    // where each unit starts: rows that end before it
    for (int i = tid; i <= s.units; i += kSumThreads) {
        const int64_t d = imin(d0 + (int64_t)i * s.per_unit, d1);
        int lo = 0, hi = rows;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)staged[mid + 1] + v0 + mid < d) lo = mid + 1;
            else hi = mid;
        }
        unit_row[i] = lo;
    }
    __syncthreads();

    const int unit = (int)s.by_cols.quotient((uint32_t)tid), col = tid - unit * s.cols;
    const int64_t c = (int64_t)blockIdx.y * s.cols + col;
    const int32_t e = (int32_t)imin<int64_t>(R::kStrided ? c : c * VEC, s.C);
    auto column = [&](int64_t c, int i) { return R::kStrided ? c + (int64_t)i * s.P : c * VEC + i; };   // element i of piece c
    const bool live = unit < s.units && c < s.P;
    float acc[VEC] = {};
    bool cut = false;                 // the unit closes a row that others have begun
    float begun[VEC] = {};            // and its own part of that row
    int begun_row = 0;
    if (live) {
        const int64_t e0 = imin(d0 + (int64_t)unit * s.per_unit, d1), e1 = imin(e0 + s.per_unit, d1);
        int r = unit_row[unit];       // row v0 + r is open
        const int r_end = unit_row[unit + 1];
        const int first = r;
        // positions within the CTA's
        int p = (int)imax<int64_t>(imin<int64_t>(e0 - (v0 + r) - j0, count), 0);
        const int p_end = (int)imax<int64_t>(imin<int64_t>(e1 - (v0 + r_end) - j0, count), p);
        const bool entered = (int64_t)staged[r] < j0 + p;   // its first row has begun before
        auto close = [&]() {
            if (r == first && entered) {
                cut = true;
                begun_row = r;
#pragma unroll
                for (int i = 0; i < VEC; ++i) begun[i] = acc[i];
            } else {
                // a row of nothing but zeros in its own phase, in which it may have a piece more
                T* to = dw + (int64_t)(v0 + r) * s.C;
                const bool empty = !kWhole && !R::kStrided && staged[r] == staged[r + 1];
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = acc[i] * scale;
                R::template store<true, false>(to, empty ? R::column(to, (int32_t)c) : e, s.C, pack<T>(f));
                if (empty && c == s.P - 1) R::template store<true>(to, R::column(to, s.P), s.C, R::zero());
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
            ++r;
        };
        auto load = [&](typename R::Loaded(&v)[kBatch], int p) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                v[u] = {};
                if (p + u < p_end) {
                    const int32_t i = sperm[p + u];
                    if ((uint64_t)(int64_t)i < (uint64_t)s.M) v[u] = R::template load<false>(dy, i, e, s.C);
                }
            }
        };
        typename R::Loaded v[kBatch], next[kBatch];
        load(v, p);
        for (; p < p_end; p += kBatch) {
            load(next, p + kBatch);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (p + u >= p_end) break;
                while (r < r_end && j0 + p + u >= (int64_t)staged[r + 1]) close();
                float f[VEC];
                unpack<T>(R::join(v[u]), f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += f[i];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) v[u] = next[u];
        }
        while (r < r_end) close();
#pragma unroll
        for (int i = 0; i < VEC; ++i) open[tid * VEC + i] = acc[i];
    }
    __syncthreads();

    // Sums of units [from, unit) that left row v0 + r open, added in their order.
    auto earlier = [&](int r, float (&sum)[VEC]) {
        int from = unit;
        while (from > 0 && unit_row[from] == r) --from;   // down to the unit that begins the row, or to the CTA's first
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
        for (int q = from; q < unit; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] += open[(q * s.cols + col) * VEC + i];
    };
    // Without the ways that Row::store takes by a row's phase: with these, behind the threads of a warp that had gone all of
    // them (its rows at a phase of 0, then odd, then even ones, and their last pieces) the last pieces' threads went on with
    // values that were not theirs, and left out or misplaced parts of the row that is joined below (7 of 137000 gradients).
    const int64_t at = (int64_t)blockIdx.x * s.C;
    if (live && cut) {
        float sum[VEC];
        earlier(begun_row, sum);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += begun[i];
        if ((int64_t)staged[begun_row] + v0 + begun_row >= d0) {   // begun in this CTA
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] *= scale;
            T* to = dw + (int64_t)(v0 + begun_row) * s.C;
            if constexpr (kWhole) {
                R::template store<true>(to, e, s.C, pack<T>(sum));
            } else {   // a store for each element: few rows are cut
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (column(c, i) < s.C) to[column(c, i)] = from_f32<T>(sum[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (kWhole || column(c, i) < s.C) head[at + column(c, i)] = sum[i];
        }
    }
    if (live && unit == s.units - 1) {
        const int r = unit_row[s.units];
        float sum[VEC];
        if (unit_row[unit] == r) {
            earlier(r, sum);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += sum[i];
        }
        if ((int64_t)staged[r] + v0 + r < d1)   // the row goes on in the next CTA
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (kWhole || column(c, i) < s.C) tail[at + column(c, i)] = acc[i];
    }
    const int first = begun_by;
    if (!kCluster) {
        if (tid == 0 && blockIdx.y == 0) notes[blockIdx.x] = SumNote{first < 0 ? -1 : v0, imax(first, 0)};
        return;
    }
    cluster_barrier();
    if (first < 0) return;
    const int64_t c0 = (int64_t)blockIdx.y * s.cols;
    for (int t = tid; t < s.cols * VEC; t += kSumThreads) {
        const int i = R::kStrided ? (int)s.by_cols.quotient((uint32_t)t) : t % VEC;
        const int64_t piece = c0 + (R::kStrided ? t - i * s.cols : t / VEC), q = column(piece, i);
        if (piece >= s.P || q >= s.C) continue;
        float sum = 0.f;
        for (int b = first; b < (int)blockIdx.x; ++b) sum += __ldcg(tail + (int64_t)b * s.C + q);
        sum += __ldcg(head + (int64_t)blockIdx.x * s.C + q);
        dw[(int64_t)v0 * s.C + q] = from_f32<T>(sum * scale);
    }
}

// For each CTA that closes a row which others have begun: the parts in their order, by slices of threads, the slices in
// theirs.  W floats at a time where rows of C are whole vectors of them.
constexpr int kJoinBatch = 8;
template <typename T, int W>
__global__ void __launch_bounds__(kSumThreads) join_rows(int32_t C, int32_t wide, float scale, const float* __restrict__ head,
                                                         const float* __restrict__ tail, const SumNote* __restrict__ notes,
                                                         T* __restrict__ dw) {
    using Vec = typename std::conditional<W == 4, float4, float>::type;
    __shared__ Vec part[kSumThreads];
    pdl_wait();
    pdl_trigger();
    const SumNote note = notes[blockIdx.x];
    if (note.row < 0) return;
    const int64_t c0 = (int64_t)blockIdx.y * wide;
    const int cols = (int)imin<int64_t>(wide, C - c0) / W;       // vectors of this CTA
    const int slices = kSumThreads / cols, slice = threadIdx.x / cols, col = threadIdx.x - slice * cols;
    const int last = blockIdx.x, n = last - note.first;   // tails of the CTAs [first, last), then the head of the last
    const int each = (n + slices - 1) / slices;
    auto at = [&](const float* p, int64_t q) { return reinterpret_cast<const Vec*>(p + q * C + c0)[col]; };
    auto add = [](Vec& a, Vec b) {
        if constexpr (W == 4) a = f4_add(a, b);
        else a += b;
    };
    Vec sum = {};
    if (slice < slices) {
        int q = note.first + imin(slice * each, n);
        const int end = note.first + imin((slice + 1) * each, n);
        for (; q < end; q += kJoinBatch) {
            Vec v[kJoinBatch];
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u) v[u] = q + u < end ? at(tail, q + u) : Vec{};
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u) add(sum, v[u]);
        }
    }
    if (n > 1) {
        part[threadIdx.x] = sum;
        __syncthreads();
    }
    if (slice > 0) return;
    for (int k = 1; k < imin(slices, n); ++k) add(sum, part[k * cols + col]);
    add(sum, at(head, last));
    T* out = dw + (int64_t)note.row * C + c0 + col * W;
    if constexpr (W == 4) {
        const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = from_f32<T>(f[i] * scale);
    } else {
        *out = from_f32<T>(sum * scale);
    }
}

size_t sum_workspace(const SumShape& s) {
    return 2 * align_up((size_t)s.ctas * s.C * 4, 256) + align_up((size_t)s.ctas * sizeof(SumNote), 256);
}

template <typename T, bool kWhole>
zs_status embed_backward(const void* dy, int64_t dy_ld, const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t V, int32_t C,
                         float scale, void* dw, void* workspace, cudaStream_t stream) {
    const SumShape s = sum_shape(M, V, C, kVec<T>);
    float* head = static_cast<float*>(workspace);
    const size_t each = align_up((size_t)s.ctas * C * 4, 256);
    float* tail = reinterpret_cast<float*>(static_cast<char*>(workspace) + each);
    SumNote* notes = reinterpret_cast<SumNote*>(static_cast<char*>(workspace) + 2 * each);
    const dim3 grid(s.ctas, s.ctas_y), block(kSumThreads);
    const Rows<T> rows(dy, M, dy_ld, C);
    T* to = static_cast<T*>(dw);
    if (s.cluster) launch_clusters(s.ctas, sum_rows<T, kWhole, true>, grid, block, 0, stream, s, rows, row_ptr, perm, scale, to, head, tail, notes);
    else launch(sum_rows<T, kWhole, false>, grid, block, 0, stream, s, rows, row_ptr, perm, scale, to, head, tail, notes);
    if (zs_status st = check_launch("embedding gradient")) return st;
    if (!s.cluster && s.ctas > 1) {
        // as few columns a CTA as its threads are slices of many parts (11841 rows of one id, 256 bf16: 256 columns 17 us, 64
        // 11), while those without a row do not take longer to start (16384 of 50021, 1024 bf16: 64 columns 39, 256 34)
        int wide = 64;
        while (wide < 256 && (int64_t)s.ctas * ((C + wide - 1) / wide) > 2048) wide *= 2;
        const dim3 columns(s.ctas, (C + wide - 1) / wide);
        auto join = C % 4 ? join_rows<T, 1> : join_rows<T, 4>;
        launch(join, columns, block, 0, stream, C, wide, scale, (const float*)head, (const float*)tail, (const SumNote*)notes, to);
        return check_launch("embedding gradient (join)");
    }
    return ZS_OK;
}

zs_status check(const char* fn, int32_t dtype, int64_t M, int32_t V, int32_t C, float scale) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (M < 0 || V < 0 || C < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld V=%d C=%d", fn, (long long)M, V, C);
    if (M > kMaxRows || V > kMaxRows || C > kMaxRows)
        return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld, V=%d or C=%d is above 2^31 - 2^16", fn, (long long)M, V, C);
    if (!(scale - scale == 0.f)) return fail(ZS_ERR_INVALID_ARG, "%s: scale=%g", fn, (double)scale);
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" {

zs_status zs_embedding(int32_t dtype, const void* w, int64_t w_ld, const int32_t* ids, int64_t M, int32_t V, int32_t C, float scale,
                       void* y, int64_t y_ld, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_embedding";
    if (zs_status st = check(fn, dtype, M, V, C, scale)) return st;
    if (M == 0) return ZS_OK;
    if (zs_status st = check_rows(fn, "w", dtype, w, w_ld, V, C)) return st;
    if (zs_status st = check_rows(fn, "y", dtype, y, y_ld, M, C)) return st;
    if (zs_status st = check_words(fn, "ids", ids, M)) return st;
    if (V < 2) w_ld = C;
    if (M < 2) y_ld = C;
    const bool whole = whole_pieces(dtype, C, {{w, w_ld}, {y, y_ld}});
    return ZS_ROWS_DISPATCH(embed_forward, dtype, whole, w, w_ld, V, ids, M, C, scale, y, y_ld, reinterpret_cast<cudaStream_t>(stream));
}

size_t zs_embedding_backward_workspace_bytes(int32_t dtype, int64_t M, int32_t V, int32_t C) {
    using namespace zs;
    if (!known_dtype(dtype) || M < 0 || V < 1 || C < 1 || M > kMaxRows || V > kMaxRows || C > kSumMaxC) return 0;
    return sum_workspace(sum_shape(M, V, C, 16 / dtype_bytes(dtype)));
}

zs_status zs_embedding_backward(int32_t dtype, const void* dy, int64_t dy_ld, const int32_t* row_ptr, const int32_t* perm, int64_t M,
                                int32_t V, int32_t C, float scale, void* dw, void* workspace, size_t workspace_bytes,
                                zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_embedding_backward";
    if (zs_status st = check(fn, dtype, M, V, C, scale)) return st;
    if (C > kSumMaxC) return fail(ZS_ERR_UNSUPPORTED, "%s: C=%d is above %d", fn, C, kSumMaxC);
    if (V == 0) return ZS_OK;
    if (zs_status st = check_rows(fn, "dy", dtype, dy, dy_ld, M, C)) return st;
    if (zs_status st = check_rows(fn, "dw", dtype, dw, C, V, C)) return st;
    if (zs_status st = check_words(fn, "row_ptr", row_ptr, V)) return st;
    if (zs_status st = check_words(fn, "perm", perm, M)) return st;
    if (!workspace || workspace_bytes < zs_embedding_backward_workspace_bytes(dtype, M, V, C))
        return fail(ZS_ERR_INVALID_ARG, "%s: workspace of %zu bytes is too small", fn, workspace_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(ZS_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (M < 2) dy_ld = C;
    const bool whole = whole_pieces(dtype, C, {{dy, dy_ld}, {dw, C}});
    return ZS_ROWS_DISPATCH(embed_backward, dtype, whole, dy, dy_ld, row_ptr, perm, M, V, C, scale, dw, workspace,
                            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
