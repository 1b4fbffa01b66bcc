// Embedding: rows of a table by id, scaled, and the table's gradient from a
// CSR of the ids.
//
// Forward: y[i] = scale * w[ids[i]], one pass that writes M C elements and
// reads the rows it needs (move_rows).
//
// Gradient: dw[v] = scale * sum of dy[perm[j]] over the positions j of CSR row
// v.  A row of dw is written once and a row of dy read once, both C elements,
// so that "position j" and "end of row v" cost the same: they are merged into
// one list of M + V items (the end of row v comes after its positions, as item
// row_ptr[v + 1] + v) that is cut into equal shares, however skewed the ids
// and however many rows of the table have none.  A CTA takes one share of the
// list and up to 256 pieces of the columns: it stages its part of row_ptr and
// perm in shared memory, its threads (a share of the CTA's items and a piece
// each) walk their items with eight loads in flight, and what is cut between
// its threads is added up in shared memory.  What is cut between CTAs goes to
// the workspace in fp32 and is added up by a second kernel in the CTAs' order.
// All sums are in fp32 and in an order that follows from the sizes.
#include "zs_rows.cuh"

namespace zs {
namespace {

struct IdSource {
    static constexpr bool kScaled = true;
    const int32_t* ids;
    int32_t V;
    __device__ __forceinline__ int64_t row(int64_t i, bool) const {
        const int32_t v = __ldg(ids + i);
        return (uint32_t)v < (uint32_t)V ? v : -1;
    }
};

template <typename T, int VEC>
zs_status embed_forward(const void* w, int64_t w_ld, int32_t V, const int32_t* ids, int64_t M, int32_t C, float scale, void* y,
                        int64_t y_ld, cudaStream_t s) {
    constexpr int U = VEC == 1 ? 8 : 2;
    const MoveShape shape = move_shape(M, C / VEC, U);
    launch(move_rows<T, VEC, U, IdSource>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape, IdSource{ids, V},
           static_cast<const T*>(w), w_ld, scale, static_cast<T*>(y), y_ld);
    return check_launch("embedding");
}

// ------------------------------------------------------------------ gradient

constexpr int kSumThreads = 256;
constexpr int kSumBatch = 8;         // rows of dy in flight for a thread
constexpr int kSumItems = 4096;      // most items of a CTA (staged in shared memory)
constexpr int kSumCtas = 6;          // CTAs an SM that the shares are made for

struct SumShape {
    int64_t M, items;                // items: M + V
    int32_t V, C, P;
    int32_t cols;                    // pieces of a CTA, of P
    int32_t units, per_unit;         // shares of a CTA's items, items of each
    int32_t ctas, ctas_y;
    FastDiv by_cols;
    int64_t share() const { return (int64_t)units * per_unit; }
};

inline SumShape sum_shape(int64_t M, int32_t V, int32_t C, int vec) {
    SumShape s = {};
    s.M = M;
    s.V = V;
    s.C = C;
    s.items = M + V;
    s.P = C / vec;
    s.cols = imin(s.P, kSumThreads);
    s.units = kSumThreads / s.cols;
    s.ctas_y = (s.P + s.cols - 1) / s.cols;
    const int64_t target = imax<int64_t>(1, (int64_t)num_sms() * kSumCtas / s.ctas_y);
    const int64_t per = (s.items + target * s.units - 1) / (target * s.units);
    s.per_unit = (int32_t)imax<int64_t>(imin<int64_t>(imax<int64_t>(per, kSumBatch), kSumItems / s.units), 1);
    s.ctas = (int32_t)((s.items + s.share() - 1) / s.share());
    s.by_cols = FastDiv((uint32_t)s.cols);
    return s;
}

// Of each CTA of the first kernel: the row that it closes and others have begun (or -1), and the CTA that began it.
struct SumNote {
    int32_t row, first;
};

// Rows that end before item d of the merged list: how many v have row_ptr[v + 1] + v < d.  Whole warp.
__device__ __forceinline__ int rows_before(const int32_t* row_ptr, int32_t V, int64_t d, int lane) {
    int lo = 0, hi = V;
    while (lo < hi) {
        const int step = ((hi - lo) + 31) >> 5;
        const int64_t at = (int64_t)lo + (int64_t)lane * step;
        const bool ge = at >= hi || (int64_t)__ldg(row_ptr + at + 1) + at >= d;
        const unsigned m = __ballot_sync(0xffffffffu, ge);
        if (m == 0) {
            lo += 31 * step + 1;
        } else {
            const int f = __ffs(m) - 1;
            hi = (int)imin<int64_t>((int64_t)lo + (int64_t)f * step, hi);
            if (f > 0) lo += (f - 1) * step + 1;
        }
    }
    return lo;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads) sum_rows(SumShape s, const T* __restrict__ dy, int64_t dy_ld,
                                                        const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ perm,
                                                        float scale, T* __restrict__ dw, float* __restrict__ head,
                                                        float* __restrict__ tail, SumNote* __restrict__ notes) {
    using R = Row<T, VEC>;
    __shared__ int32_t staged[kSumItems + 8];        // row_ptr[v0 .. v1 + 1], then perm[j0 .. j1)
    __shared__ int32_t bound[2];
    __shared__ int32_t unit_row[kSumThreads + 1];    // rows that end before each unit
    __shared__ float open[kSumThreads * VEC];        // sums of rows that a unit leaves open
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t share = (int64_t)s.units * s.per_unit;
    const int64_t d0 = blockIdx.x * share, d1 = imin(d0 + share, s.items);
    pdl_wait();
    pdl_trigger();
    if (warp < 2) {
        const int v = rows_before(row_ptr, s.V, warp ? d1 : d0, lane);
        if (lane == 0) bound[warp] = v;
    }
    __syncthreads();
    const int v0 = bound[0], v1 = bound[1];
    const int64_t j0 = imax<int64_t>(imin(d0 - v0, s.M), 0), j1 = imax(imin(d1 - v1, s.M), j0);
    // v1 - v0 rows end here and one more may be open: v1 - v0 + 2 bounds, and j1 - j0 positions, together at most the
    // share and two (and no more than fits, whatever row_ptr holds)
    const int rows = imax(imin(v1 - v0, kSumItems), 0), bounds = rows + 2;
    const int count = (int)imin<int64_t>(j1 - j0, kSumItems + 8 - bounds);
    for (int i = tid; i < bounds; i += kSumThreads) staged[i] = v0 + i <= s.V ? __ldg(row_ptr + v0 + i) : (int32_t)s.M;
    int32_t* sperm = staged + bounds;
    for (int i = tid; i < count; i += kSumThreads) sperm[i] = __ldg(perm + j0 + i);
    __syncthreads();
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
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = acc[i] * scale;
                R::store(dw + (int64_t)(v0 + r) * s.C, c, R::rounded(f));
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
            ++r;
        };
        for (; p < p_end; p += kSumBatch) {
            typename R::Raw v[kSumBatch];
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u) {
                v[u] = R::zero();
                if (p + u < p_end) {
                    const int32_t i = sperm[p + u];
                    if ((uint64_t)(int64_t)i < (uint64_t)s.M) v[u] = R::load_once(dy + (int64_t)i * dy_ld, c);
                }
            }
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u) {
                if (p + u >= p_end) break;
                while (r < r_end && j0 + p + u >= (int64_t)staged[r + 1]) close();
                float f[VEC];
                R::floats(v[u], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += f[i];
            }
        }
        while (r < r_end) close();
#pragma unroll
        for (int i = 0; i < VEC; ++i) open[tid * VEC + i] = acc[i];
    }
    __syncthreads();
    if (!live) return;

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
    const int64_t at = (int64_t)blockIdx.x * s.C + c * VEC;
    if (cut) {
        float sum[VEC];
        earlier(begun_row, sum);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += begun[i];
        if ((int64_t)staged[begun_row] + v0 + begun_row >= d0) {   // begun in this CTA
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] *= scale;
            R::store(dw + (int64_t)(v0 + begun_row) * s.C, c, R::rounded(sum));
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) head[at + i] = sum[i];
        }
    }
    if (unit == s.units - 1) {
        const int r = unit_row[s.units];
        float sum[VEC];
        if (unit_row[unit] == r) {
            earlier(r, sum);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += sum[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) tail[at + i] = acc[i];
    }
    if (tid == 0 && blockIdx.y == 0) {
        // the row that is open at the CTA's start, if it was begun before and ends here
        const int64_t begin = (int64_t)staged[0] + v0;
        const bool closes = rows > 0 && begin < d0;
        notes[blockIdx.x] = SumNote{closes ? v0 : -1, closes ? (int32_t)imax<int64_t>(begin / share, 0) : 0};
    }
}

// A CTA for each CTA that closes a row which others have begun: the parts in
// their order, by slices of threads and the slices in theirs.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) join_rows(int32_t C, int cols, float scale, const float* __restrict__ head,
                                                         const float* __restrict__ tail, const SumNote* __restrict__ notes,
                                                         T* __restrict__ dw) {
    __shared__ float part[kSumThreads];
    pdl_wait();
    pdl_trigger();
    const SumNote note = notes[blockIdx.x];
    if (note.row < 0) return;
    const int slices = kSumThreads / cols, slice = threadIdx.x / cols, col = threadIdx.x - slice * cols;
    const int last = blockIdx.x, n = last - note.first;   // tails of the CTAs [first, last), then the head of the last
    const int each = (n + slices - 1) / slices;
    for (int64_t c = (int64_t)blockIdx.y * cols + col; c - col < C; c += (int64_t)gridDim.y * cols) {
        float sum = 0.f;
        if (slice < slices && c < C) {
            const int a = note.first + imin(slice * each, n), b = note.first + imin((slice + 1) * each, n);
            int q = a;
            for (; q + kSumBatch <= b; q += kSumBatch) {
                float v[kSumBatch];
#pragma unroll
                for (int u = 0; u < kSumBatch; ++u) v[u] = tail[(int64_t)(q + u) * C + c];
#pragma unroll
                for (int u = 0; u < kSumBatch; ++u) sum += v[u];
            }
            for (; q < b; ++q) sum += tail[(int64_t)q * C + c];
        }
        part[threadIdx.x] = sum;
        __syncthreads();
        if (slice == 0 && c < C) {
            for (int k = 1; k < slices; ++k) sum += part[k * cols + col];
            sum += head[(int64_t)last * C + c];
            dw[(int64_t)note.row * C + c] = from_f32<T>(sum * scale);
        }
        __syncthreads();
    }
}

size_t sum_workspace(const SumShape& s) {
    return 2 * align_up((size_t)s.ctas * s.C * 4, 256) + align_up((size_t)s.ctas * sizeof(SumNote), 256);
}

template <typename T, int VEC>
zs_status embed_backward(const void* dy, int64_t dy_ld, const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t V, int32_t C,
                         float scale, void* dw, void* workspace, cudaStream_t stream) {
    const SumShape s = sum_shape(M, V, C, VEC);
    float* head = static_cast<float*>(workspace);
    const size_t each = align_up((size_t)s.ctas * C * 4, 256);
    float* tail = reinterpret_cast<float*>(static_cast<char*>(workspace) + each);
    SumNote* notes = reinterpret_cast<SumNote*>(static_cast<char*>(workspace) + 2 * each);
    launch(sum_rows<T, VEC>, dim3(s.ctas, s.ctas_y), dim3(kSumThreads), 0, stream, s, static_cast<const T*>(dy), dy_ld, row_ptr, perm,
           scale, static_cast<T*>(dw), head, tail, notes);
    if (zs_status st = check_launch("embedding gradient")) return st;
    if (s.ctas > 1) {
        const int cols = imin(C, 32);
        const int32_t ctas_y = (int32_t)imin<int64_t>(64, (C + cols - 1) / cols);
        launch(join_rows<T>, dim3(s.ctas, ctas_y), dim3(kSumThreads), 0, stream, C, cols, scale, (const float*)head, (const float*)tail,
               (const SumNote*)notes, static_cast<T*>(dw));
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
    if (!known_dtype(dtype) || M < 0 || V < 1 || C < 1 || M > kMaxRows || V > kMaxRows || C > kMaxRows) return 0;
    const int vec = 16 / dtype_bytes(dtype);
    const size_t elements = sum_workspace(sum_shape(M, V, C, 1));
    return C % vec ? elements : imax(elements, sum_workspace(sum_shape(M, V, C, vec)));
}

zs_status zs_embedding_backward(int32_t dtype, const void* dy, int64_t dy_ld, const int32_t* row_ptr, const int32_t* perm, int64_t M,
                                int32_t V, int32_t C, float scale, void* dw, void* workspace, size_t workspace_bytes,
                                zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_embedding_backward";
    if (zs_status st = check(fn, dtype, M, V, C, scale)) return st;
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
