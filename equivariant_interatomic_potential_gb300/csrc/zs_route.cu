// Routing of rows to experts, and the gradient of the logits.
//
// A warp takes a row (a thread where experts are few and rows many, see
// route_rows_of_few).  Its lanes hold up to V experts each in ascending order,
// those of a group of experts in neighbouring lanes, so that the lowest lane
// among equal ones has the lowest index.  Values become unsigned keys that sort
// like them (0: closed), the last bits of a key the expert's place in its lane.
// A lane sorts its keys by a network of minima and maxima and lays them down in
// shared memory; then k rounds of a warp maximum over the lanes' first keys pick
// the experts, and the lane that a round took from moves on to its next key.
//
// The choice is that of the scores in 64 bits.  Without a bias and groups it
// goes by the logits themselves, which sort like their scores.  Keys hold values
// to a bound that is known (the place's bits, and the error of scores, which are
// formed in 32 bits); where two neighbours of the choice, or two groups at its
// border, lie closer than that (and are not of one logit and bias), the few
// candidates are put in order in 64 bits, a lane each: one row in some hundred of
// ordinary ones.  Where there are more than 32, with NaN, for a softmax with a
// bias, and where a softmax's scores are below 2^-1000 (which a division by the
// row's sum may make alike), all of the row is done in 64 bits.  Weights are
// formed in 32 bits, relative to the largest chosen logit where they are
// renormalised, so that they never are 0 / 0.
//
// What bounds it: the instructions of this way of choosing.  32768 rows of 256
// experts, 8 choices, 4 of 8 groups: 870 a row (25 for each choice, 140 for
// sigmoids and a bias, 160 for groups), 33 us where the bytes are 5.  48 warps of
// 40 registers an SM issue in two of three cycles: a warp lives for one row,
// whose loads and rounds only other warps hide.  An unsorted lane (rounds that
// look at all V keys) took 77 us, several rows a warp 45 (too few CTAs to even
// out).
#include "zs_types.cuh"

namespace zs {
namespace {

constexpr int kRouteMaxE = 1024, kRouteMaxK = 32, kRouteMaxGroups = 32;
constexpr int kRouteWarps = 4;
template <int V> constexpr int kBackWarps = V <= 8 ? 8 : 4;   // of the gradient: 65536 rows of 64 14 us at 8, 17 at 4; of 1024 105 and 92
constexpr int kRouteFew = 16, kRouteFewRows = 4096;   // experts whose row a thread takes, and rows from which on
constexpr unsigned kAll = 0xffffffffu;

struct RouteShape {
    int64_t M, ld;
    int32_t E, k, groups, per, top_groups, group_top;
    int32_t lanes, each;    // lanes of a group (a power of two), experts of a lane
    int32_t lane_bits;      // log2 of lanes
    int32_t width;          // the least power of two that holds k
    bool sigmoid, renormalise;
    bool wide, wide_bias;   // a lane's logits and biases are whole 16-byte pieces
    float scale;
};

template <typename F> struct KeyOf;
template <> struct KeyOf<float> {
    using U = uint32_t;
    static __device__ __forceinline__ U bits(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ float value(U b) { return __uint_as_float(b); }
    static __device__ __forceinline__ U max_of_warp(U v) { return __reduce_max_sync(kAll, v); }
};
template <> struct KeyOf<double> {
    using U = unsigned long long;
    static __device__ __forceinline__ U bits(double v) { return (U)__double_as_longlong(v); }
    static __device__ __forceinline__ double value(U b) { return __longlong_as_double((long long)b); }
    static __device__ __forceinline__ U max_of_warp(U v) {
        for (int o = 16; o > 0; o >>= 1) {
            const U w = __shfl_xor_sync(kAll, v, o);
            v = w > v ? w : v;
        }
        return v;
    }
};
// Keys sort like their values; NaN above all, -infinity is 0.
template <typename F>
__device__ __forceinline__ typename KeyOf<F>::U to_key(F v) {
    using U = typename KeyOf<F>::U;
    constexpr U top = (U)1 << (8 * sizeof(U) - 1);
    if (v != v) return ~(U)0;
    if (v == -(F)INFINITY) return 0;
    const U b = KeyOf<F>::bits(v + (F)0);   // -0 is 0
    return b & top ? ~b : b | top;
}
template <typename F>
__device__ __forceinline__ F from_key(typename KeyOf<F>::U k) {
    using U = typename KeyOf<F>::U;
    constexpr U top = (U)1 << (8 * sizeof(U) - 1);
    return KeyOf<F>::value(k & top ? k & ~top : ~k);
}

// 2^x and 1 / x by one instruction each (2 ulps and 1, numbers below the normal ones as 0).
__device__ __forceinline__ float exp2_quick(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_quick(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504088896341f;

template <typename F>
__device__ __forceinline__ F sum_of_warp(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float max_of_warp(float v) {   // NaN are passed over
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// A lane's experts.
struct Lane {
    int group, first, count;
    __device__ __forceinline__ Lane(const RouteShape& s, int lane) {
        group = lane >> s.lane_bits;
        const int at = (lane & (s.lanes - 1)) * s.each;
        first = group * s.per + at;
        count = group < s.groups ? imax(imin(s.per - at, s.each), 0) : 0;
    }
};

template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) { return to_f32(__ldg(row + e)); }

// A lane's keys, the largest first: Batcher's merge exchange sort, V a power of two, its steps as templates so that every
// index is known and the keys stay in registers (of 32 keys, loops were not unrolled: 65536 rows of 1024 fp32 288 us, now 107).
template <int P, int K, int V>
__device__ __forceinline__ void sort_step(uint32_t (&key)[V]) {
    if constexpr (P < V) {
#pragma unroll
        for (int x = K % P; x < V - K; ++x)
            if ((x - K % P) / K % 2 == 0 && x / (2 * P) == (x + K) / (2 * P)) {
                const uint32_t a = key[x], b = key[x + K];
                key[x] = max(a, b);
                key[x + K] = min(a, b);
            }
        if constexpr (K > 1) sort_step<P, K / 2>(key);
        else sort_step<2 * P, 2 * P>(key);
    }
}
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V]) {
    sort_step<1, 1>(key);
}

// The two largest keys of a lane's group, from those of its lanes.
template <typename U>
__device__ __forceinline__ void two_of_group(const RouteShape& s, U& first, U& second) {
    for (int o = 1; o < s.lanes; o <<= 1) {
        const U a = __shfl_xor_sync(kAll, first, o), b = __shfl_xor_sync(kAll, second, o);
        second = max(min(a, first), a > first ? b : second);
        first = max(a, first);
    }
}
// What the choice goes by, in 64 bits: -infinity where it is closed.  `top` and `sum` for a softmax with a bias.
template <bool kScored>
__device__ __forceinline__ double score_in_64_bits(const RouteShape& s, double z, double top, double sum, const float* __restrict__ bias,
                                                   int e) {
    if (!kScored || z == -INFINITY) return z;
    const double a = s.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - top) / sum;
    return bias ? a + (double)__ldg(bias + e) : a;
}

// A softmax's exponentials sort like its scores, and their sums like the scores', where the division by the row's sum, at most
// 1024, loses nothing of them.
constexpr double kLeastExp = 0x1p-1000;

// The `need` groups of the mask `groups` with the largest values, as a mask: lane g holds group g's.  NaN are above all,
// equal ones go by their number.
__device__ __forceinline__ unsigned best_groups(unsigned groups, int need, int lane, double value) {
    const unsigned long long own = to_key<double>(value);
    int ahead = 0;
    for (unsigned m = groups; m; m &= m - 1) {
        const int g = __ffs(m) - 1;
        const unsigned long long v = __shfl_sync(kAll, own, g);
        ahead += v > own || (v == own && g < lane);
    }
    return __ballot_sync(kAll, (groups >> lane & 1u) && ahead < need);
}

// The row's choice in 64 bits: the expert of choice `lane` (or -1).
template <typename T, int V, bool kScored>
__device__ __noinline__ int choose_in_64_bits(const RouteShape& s, int lane, const T* __restrict__ row, const float* __restrict__ bias) {
    using U = unsigned long long;
    const Lane l(s, lane);
    U key[V];
    double top = -INFINITY, sum = 0.0;
    if (kScored && !s.sigmoid) {
#pragma unroll 1
        for (int i = 0; i < l.count; ++i) top = fmax(top, (double)logit(row, l.first + i));
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll 1
        for (int i = 0; i < l.count; ++i) {
            const float z = logit(row, l.first + i);
            if (z != -INFINITY) sum += exp((double)z - top);
        }
        sum = sum_of_warp(sum);
    }
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        key[i] = 0;
        if (i < l.count) key[i] = to_key<double>(score_in_64_bits<kScored>(s, logit(row, l.first + i), top, sum, bias, l.first + i));
    }
    if (s.top_groups < s.groups) {
        U first = 0, second = 0;
        for (int i = 0; i < V; ++i) {
            const U k = key[i];
            second = k > first ? first : (k > second ? k : second);
            first = k > first ? k : first;
        }
        two_of_group(s, first, second);
        double value = -INFINITY;
        if (first) value = from_key<double>(first) + (s.group_top == 2 && second ? from_key<double>(second) : 0.0);
        value = __shfl_sync(kAll, value, (lane << s.lane_bits) & 31);   // lane g: group g's
        const unsigned kept = best_groups(s.groups == 32 ? kAll : (1u << s.groups) - 1, s.top_groups, lane, value);
        if (!(kept >> l.group & 1u))
            for (int i = 0; i < V; ++i) key[i] = 0;
    }
    int mine = -1;
#pragma unroll 1
    for (int r = 0; r < s.k; ++r) {
        U best = 0;
        int at = 0;
        for (int i = 0; i < V; ++i) {
            at = key[i] > best ? i : at;
            best = key[i] > best ? key[i] : best;
        }
        const U top_key = KeyOf<double>::max_of_warp(best);
        if (top_key == 0) break;
        const int winner = __ffs(__ballot_sync(kAll, best == top_key)) - 1;
        if (lane == winner) key[at] = 0;
        const int e = __shfl_sync(kAll, l.first + at, winner);
        if (lane == r) mine = e;
    }
    return mine;
}

// A lane's V neighbours: 16 bytes at a time where `wide`, closed ones behind `count`.
template <typename T, int V>
__device__ __forceinline__ void load_lane(const T* p, int count, bool wide, float none, float (&z)[V]) {
    constexpr int N = kVec<T>;
    if constexpr (V % N == 0) {
        if (wide) {
#pragma unroll
            for (int q = 0; q < V / N; ++q) {
                float f[N];
                unpack<T>(count > 0 ? __ldg(reinterpret_cast<const uint4*>(p) + q) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
                for (int i = 0; i < N; ++i) z[q * N + i] = count > 0 ? f[i] : none;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = i < count ? to_f32(__ldg(p + i)) : none;
}

// t / sum: exactly 1 for the only one, whose gradient then is 0.
__device__ __forceinline__ float share_of(float t, float sum) { return t == sum ? 1.f : __fdividef(t, sum); }

// Shares of the chosen logits z (lanes with `held`) among those of `width` lanes: softmax, or sigmoids over their sum.
__device__ __forceinline__ float renormalised(bool sigmoid, bool held, float z, int width) {
    float top = held ? z : -INFINITY;
    for (int o = width >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float t = 0.f;
    if (held) {
        if (sigmoid) t = __fdividef(expf(fminf(z, 0.f) - fminf(top, 0.f)), 1.f + expf(-fabsf(z)));
        else t = expf(z - top);
        if (z != z) t = z;
    }
    float sum = t;
    for (int o = width >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    return held ? share_of(t, sum) : 0.f;
}
__device__ __forceinline__ float sigmoid_of(float z) { return __fdividef(1.f, 1.f + expf(-z)); }

constexpr uint32_t kOpen = 0x00800000u;                   // the key of the lowest finite value: below are closed ones
template <int V> constexpr uint32_t kPlace = V - 1;       // a key's bits for the place in its lane, the last one 0
template <int V> constexpr float kRelative = V * 0x1p-23f + 0x1p-22f;   // what the place's bits and a sum's rounding take
// Keys of 16-bit logits are exact: they leave the place's bits clear.
template <typename T, bool kScored> constexpr bool kExact = !kScored && sizeof(T) == 2;

__device__ __forceinline__ uint32_t open_key(float v) {   // NaN apart
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// A warp's place in shared memory: its lanes' sorted keys (behind the first ones, and 0 behind the last), and what its
// rounds took (a key, and its lane).
template <int V>
struct RouteSpace {
    uint32_t list[V + 1][32];
    uint2 taken[kRouteMaxK + 1];
};
template <int V>
__device__ __forceinline__ int expert_of(const RouteShape& s, uint2 t) {
    return (int)((t.y >> s.lane_bits) * s.per + (t.y & (s.lanes - 1)) * s.each + (kPlace<V> - (t.x & kPlace<V>)));
}
// Whether the values of two keys, the second one behind the first, are closer than they are known.
template <int V>
__device__ __forceinline__ bool near_keys(uint32_t a, uint32_t b, float error) {
    const float p = from_key<float>(a & ~kPlace<V>), q = from_key<float>(b & ~kPlace<V>);
    return p - q <= 2.f * error + kRelative<V> * (fabsf(p) + fabsf(q)) + V * 0x1p-148f;
}

// Of the groups of the mask `border`, between which 32 bits do not tell, the `need` best as a mask: the elements of each
// that may be among its two largest, in 64 bits, a lane each; groups of nothing but one logit and bias (a router that has
// learnt nothing), and all of one or all of two terms, by their numbers.  0 where there are too many, or a softmax has a
// bias or scores so small that they may be alike.  `head` is a lane's first key, `row_top` the row's largest logit.
template <typename T, int V>
__device__ __noinline__ unsigned border_groups(const RouteShape& s, int lane, const T* __restrict__ row, const float* __restrict__ bias,
                                               RouteSpace<V>& space, uint32_t head, float error, float row_top, unsigned border, int need) {
    const Lane l(s, lane);
    uint32_t first = head & ~kPlace<V>, second = V > 1 ? space.list[1][lane] & ~kPlace<V> : 0;
    if (first < kOpen) first = 0;
    if (second < kOpen) second = 0;
    two_of_group(s, first, second);
    const uint32_t of = s.group_top == 2 ? second : first;   // what a group's candidates are near to, or above
    int n = 0, mine = 0;                                     // candidates, and how many are this lane's first keys
    for (int i = 0; i < V; ++i) {
        const uint32_t key = i == 0 ? head : space.list[i][lane];
        const bool in = (border >> l.group & 1u) && key >= kOpen && ((key & ~kPlace<V>) >= of || near_keys<V>(of, key, error));
        const unsigned all = __ballot_sync(kAll, in);
        if (!all) break;   // a lane's keys descend
        const int at = n + __popc(all & ((1u << lane) - 1));
        if (in && at < 32) space.taken[at] = make_uint2(key, lane);
        mine += in;
        n += __popc(all);
    }
    __syncwarp();
    if (n > 32 || (!s.sigmoid && bias)) {
        const int e = expert_of<V>(s, space.taken[0]);
        const float z = logit(row, e), b = bias ? __ldg(bias + e) : 0.f;
        // one term against two of the same score are not alike, and may be as near to each other as the score is to 0
        const bool in = border >> l.group & 1u, alone = s.group_top == 2 && second == 0;
        const unsigned of_one = __ballot_sync(kAll, in && alone), of_two = __ballot_sync(kAll, in && !alone);
        bool alike = !of_one || !of_two;
        for (int i = 0; i < mine; ++i) {
            const int f = expert_of<V>(s, make_uint2(i == 0 ? head : space.list[i][lane], lane));
            alike = alike && logit(row, f) == z && (!bias || __ldg(bias + f) == b);
        }
        __syncwarp();
        return __all_sync(kAll, alike) ? best_groups(border, need, lane, 0.0) : 0;
    }
    const int e = lane < n ? expert_of<V>(s, space.taken[lane]) : 0, group = lane < n ? e / s.per : -1;
    const double a = lane < n ? score_in_64_bits<true>(s, logit(row, e), row_top, 1.0, bias, e) : -INFINITY;
    if (!s.sigmoid && __any_sync(kAll, lane < n && a < kLeastExp)) return 0;
    double one = -INFINITY, two = -INFINITY;   // the two largest of group `lane`
    for (int j = 0; j < n; ++j) {
        const double other = __shfl_sync(kAll, a, j);
        if (__shfl_sync(kAll, group, j) != lane) continue;
        two = other > one ? one : fmax(two, other);
        one = fmax(one, other);
    }
    __syncwarp();
    return best_groups(border, need, lane, s.group_top == 2 && two != -INFINITY ? one + two : one);
}

// The order of the n candidates that the rounds took, by what the choice goes by in 64 bits (a softmax's scores, without a
// bias, by their exponentials): a lane each, by how many are ahead.  The expert of choice `lane` (or -1).
template <typename T, int V, bool kScored>
__device__ __noinline__ int order_in_64_bits(const RouteShape& s, int lane, const T* __restrict__ row, const float* __restrict__ bias,
                                             RouteSpace<V>& space, int n, float top) {
    const bool open = lane < n;
    const int e = open ? expert_of<V>(s, space.taken[lane]) : -1;
    const double a = open ? score_in_64_bits<kScored>(s, logit(row, e), top, 1.0, bias, e) : -INFINITY;
    if (kScored && !s.sigmoid && __any_sync(kAll, open && a < kLeastExp)) return choose_in_64_bits<T, V, kScored>(s, lane, row, bias);
    int ahead = 0;
    for (int j = 0; j < n; ++j) {
        const double other = __shfl_sync(kAll, a, j);
        const int f = __shfl_sync(kAll, e, j);
        ahead += other > a || (other == a && f < e);
    }
    __syncwarp();
    if (open) space.taken[ahead].x = e;
    __syncwarp();
    return lane < imin(n, s.k) ? (int)space.taken[lane].x : -1;
}

// Whether what is near the last choice behind those that the rounds took (a lane's first key `head`, the others from list[next]
// on) is all of the last choice's logit and bias.
template <typename T, int V>
__device__ __noinline__ bool alike_behind(const RouteShape& s, int lane, const T* __restrict__ row, const float* __restrict__ bias,
                                          RouteSpace<V>& space, uint32_t head, int next, uint32_t last, float error) {
    const int e = expert_of<V>(s, space.taken[s.k - 1]);
    const float z = logit(row, e), b = bias ? __ldg(bias + e) : 0.f;
    // A row of one logit and bias (a router that has learnt nothing) in the row's order, 32 neighbours at a time: a lane's own
    // experts are a cache line apart from the next one's (32768 rows of 1024 equal fp32 logits: 130 us, 212 without).
    bool same = true;
#pragma unroll 8
    for (int f = lane; f < s.E; f += 32) {
        const float v = logit(row, f), w = bias ? __ldg(bias + f) : b;
        same = same & ((v == z) | (v == -INFINITY)) & (w == b);
    }
    if (__all_sync(kAll, same)) return true;
    bool alike = true;
    for (uint32_t key = head; key >= kOpen && near_keys<V>(last, key, error); key = space.list[next++][lane]) {   // ends in 0
        const int f = expert_of<V>(s, make_uint2(key, lane));
        alike = alike && logit(row, f) == z && (!bias || __ldg(bias + f) == b);
    }
    return __all_sync(kAll, alike);
}

// A warp's row r0.
template <typename T, int V, bool kScored>
__device__ __forceinline__ void route_row(const RouteShape& s, int64_t r0, int lane, RouteSpace<V>& space, const T* __restrict__ logits,
                                          const float* __restrict__ bias, int32_t* __restrict__ ids, float* __restrict__ weights) {
    const T* row = logits + r0 * s.ld;
    const Lane l(s, lane);
    float a[V];
    load_lane<T, V>(row + l.first, l.count, s.wide, -INFINITY, a);

    const bool whole = !s.sigmoid && (kScored || !s.renormalise);   // a softmax's scores over all experts are wanted
    float top = 0.f, sum = 1.f, error = 0.f;                        // error: of a score, beside its rounding
    bool odd = false;
    uint32_t closed = 0;                                            // the lane's closed experts, by their bits
    if (kScored)
#pragma unroll
        for (int i = 0; i < V; ++i) closed |= (a[i] == -INFINITY ? 1u : 0u) << i;
    if (whole) {
        top = a[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, a[i]);
        top = max_of_warp(top);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float e = a[i] == -INFINITY ? 0.f : s.renormalise ? exp2_quick((a[i] - top) * kLog2e) : expf(a[i] - top);
            if (kScored) a[i] = e;
            sum += e;
        }
        sum = sum_of_warp(sum);
    }
    if (kScored) {
        // exp(x) is known to (4 + 2.5 |x|) 2^-24 of itself (2 ulps, and x log2(e) to 2.5 |x| 2^-24): 2^-22 of 1 whatever x,
        // times a sigmoid's slope 1.1 2^-24.  A sigmoid's sum and reciprocal add 3 2^-24 of it.  A sum of exponentials is up
        // to (V + 8) 2^-24 off, for all scores alike.
        const float inv = s.sigmoid ? 1.f : reciprocal_quick(fmaxf(sum, 1.f));   // 1 and more, but where all are closed
        error = s.sigmoid ? 0x1p-21f : 0x1p-18f * inv;
        float b[V];
        if (bias) load_lane<float, V>(bias + l.first, l.count, s.wide_bias, 0.f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = s.sigmoid ? reciprocal_quick(1.f + exp2_quick(a[i] * -kLog2e)) : a[i] * inv;
            if (bias) a[i] += b[i];
        }
    }
    // keys, sorted: the first one here, the others in shared memory
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        odd = odd || a[i] != a[i];
        if (kScored) a[i] = closed >> i & 1u ? -INFINITY : a[i];
        key[i] = (open_key(kScored ? a[i] : a[i] + 0.f) & ~kPlace<V>) | (kPlace<V> - i);   // -0 is 0
    }
    sort_keys(key);
    uint32_t head = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) space.list[i][lane] = key[i];
    space.list[V][lane] = 0;

    if (kScored && s.top_groups < s.groups) {
        uint32_t first = head & ~kPlace<V>, second = V > 1 ? key[V > 1] & ~kPlace<V> : 0;
        if (first < kOpen) first = 0;
        if (second < kOpen) second = 0;
        two_of_group(s, first, second);
        // a group's value, the last bits its number, so that no two are alike and the lower one of equal ones is ahead
        const uint32_t number = 32 / s.lanes - 1;
        const float p = from_key<float>(first), q = s.group_top == 2 && second ? from_key<float>(second) : 0.f;
        const uint32_t value = first && l.group < s.groups ? (open_key(p + q + 0.f) & ~number) | (number - l.group) : 0;
        const float sizes = __uint_as_float(__reduce_max_sync(kAll, value ? __float_as_uint(fabsf(p) + fabsf(q)) : 0));
        uint32_t left = value, last = 0;
        bool kept = false;
        for (int r = 0; r < s.top_groups; ++r) {
            last = __reduce_max_sync(kAll, left);
            kept = kept || left == last;
            left = left == last ? 0 : left;
        }
        const uint32_t out = __reduce_max_sync(kAll, left);
        const float in_value = from_key<float>(last & ~number), out_value = from_key<float>(out & ~number);
        const float known = 4.f * error + 2.f * (kRelative<V> + (number + 1) * 0x1p-23f) * sizes;
        if (out && in_value - out_value <= known) {
            // those that are above all that are out, or below all that are in, stay where they are
            const float v = from_key<float>(value & ~number);
            const bool speaks = value && lane == l.group << s.lane_bits;
            const bool at_border = speaks && !(v > out_value + known) && !(v < in_value - known);
            unsigned border = 0, sure = 0;   // by the groups' numbers
            for (int g = 0; g < s.groups; ++g) {
                border |= (unsigned)__shfl_sync(kAll, (int)at_border, g << s.lane_bits) << g;
                sure |= (unsigned)__shfl_sync(kAll, (int)(kept && speaks && !at_border), g << s.lane_bits) << g;
            }
            const unsigned mask = border_groups<T, V>(s, lane, row, bias, space, head, error, top, border, s.top_groups - __popc(sure));
            odd = odd || mask == 0;
            if (mask) kept = (mask | sure) >> l.group & 1u;
        }
        if (!kept) head = 0;
    }

    // Rounds: the lowest lane of the largest key notes it and moves on, at most V times (its list ends in 0, which no round
    // takes).  Closed keys are behind the open ones.  Then all that are near the last one may have to change places with it.
    const uint32_t below = (1u << lane) - 1;
    uint32_t last = 0, taken = (uint32_t)__cvta_generic_to_shared(space.taken), next = (uint32_t)__cvta_generic_to_shared(&space.list[1][lane]);
    int n = 0;
    auto round = [&](uint32_t best, uint32_t most) {   // predicated: a branch costs as much as the round
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b32 of;\n\t"
            "setp.eq.u32 p, %3, %4;\n\t"
            "vote.sync.ballot.b32 of, p, 0xffffffff;\n\t"
            "and.b32 of, of, %5;\n\t"
            "setp.eq.and.u32 p, of, 0, p;\n\t"
            "@p st.shared.v2.u32 [%2], {%0, %6};\n\t"
            "@p ld.shared.u32 %0, [%1];\n\t"
            "@p add.u32 %1, %1, 128;\n\t}"
            : "+r"(head), "+r"(next)
            : "r"(taken), "r"(best), "r"(most), "r"(below), "r"(lane)
            : "memory");
        taken += sizeof(uint2);
    };
#pragma unroll 1
    for (; n < s.k; ++n) {
        const uint32_t best = head & ~kPlace<V>, most = __reduce_max_sync(kAll, best);
        if (most < kOpen) break;
        last = most;
        round(best, most);
    }
    if (!kExact<T, kScored> && n == s.k)
        for (; n <= kRouteMaxK; ++n) {
            const uint32_t best = head & ~kPlace<V>, most = __reduce_max_sync(kAll, best);
            if (most < kOpen || !near_keys<V>(last, most, error)) break;
            round(best, most);
        }
    __syncwarp();
    int id = -1;
    bool near = false;
    if (lane < imin(n, s.k)) id = expert_of<V>(s, space.taken[lane]);
    if (!kExact<T, kScored> && lane + 1 < n) {
        const uint2 t = space.taken[lane], u = space.taken[lane + 1];
        if (near_keys<V>(t.x, u.x, error)) {
            const int e = expert_of<V>(s, t), f = expert_of<V>(s, u);   // two of one logit and bias are in their order
            near = !(logit(row, e) == logit(row, f) && (!bias || __ldg(bias + e) == __ldg(bias + f)));
        }
    }
    bool far = __any_sync(kAll, odd);
    if (!kExact<T, kScored> && !far) {
        if (__any_sync(kAll, near)) {
            far = n > kRouteMaxK || (kScored && !s.sigmoid && bias);
            if (!far) id = order_in_64_bits<T, V, kScored>(s, lane, row, bias, space, n, top);
        } else if (n > kRouteMaxK) {   // there may be more of them than were taken
            const int moved = (int)(next - (uint32_t)__cvta_generic_to_shared(&space.list[1][lane])) / 128;
            far = !alike_behind<T, V>(s, lane, row, bias, space, head, 1 + moved, last, error);
        }
    }
    if (far) id = choose_in_64_bits<T, V, kScored>(s, lane, row, bias);

    const bool held = id >= 0;
    const float zc = held ? logit(row, id) : -INFINITY;
    float w;
    if (s.renormalise) w = renormalised(s.sigmoid, held, zc, s.width);
    else w = !held ? 0.f : s.sigmoid ? sigmoid_of(zc) : __fdividef(expf(zc - top), sum);
    if (lane < s.k) {
        const int64_t to = r0 * s.k + lane;
        ids[to] = id;
        weights[to] = held ? w * s.scale : 0.f;
    }
}

template <typename T, int V, bool kScored>
__global__ void __launch_bounds__(kRouteWarps * 32, V <= 8 ? 12 : V <= 16 ? 8 : 4) route_rows(
    RouteShape s, const T* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ ids, float* __restrict__ weights) {
    __shared__ RouteSpace<V> spaces[kRouteWarps];
    const int64_t r0 = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (r0 < s.M) route_row<T, V, kScored>(s, r0, threadIdx.x & 31, spaces[threadIdx.x >> 5], logits, bias, ids, weights);
}

// Few experts (kRouteFew) without groups: a thread for a row, which looks through its V scores for each choice.  Rows where
// two neighbours of the choice are too near to be told apart, or with NaN, are left to their warp, one after another.  Below
// kRouteFewRows a warp for a row is as fast (2000 of 8: 2.6 us both, 4096 2.6 against 3.2, their gradients 3.0 and 2.5).
template <typename T, int V, bool kScored>
__global__ void __launch_bounds__(kRouteWarps * 32) route_rows_of_few(RouteShape s, const T* __restrict__ logits,
                                                                      const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                                      float* __restrict__ weights) {
    __shared__ RouteSpace<1> spaces[kRouteWarps];
    const int lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * (kRouteWarps * 32) + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    bool left = false;   // to the warp
    if (r0 < s.M) {
        const T* row = logits + r0 * s.ld;
        float a[V];
        load_lane<T, V>(row, s.E, s.wide, -INFINITY, a);
        uint32_t open = 0;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            left = left || a[i] != a[i];
            open |= (a[i] == -INFINITY ? 0u : 1u) << i;
            top = fmaxf(top, a[i]);
        }
        if (!s.sigmoid && (kScored || !s.renormalise)) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = open >> i & 1u ? expf(a[i] - top) : 0.f;
                if (kScored) a[i] = e;
                sum += e;
            }
        }
        float error = 0.f;
        if (kScored) {   // as above
            const float inv = s.sigmoid ? 1.f : reciprocal_quick(fmaxf(sum, 1.f));
            error = s.sigmoid ? 0x1p-21f : 0x1p-18f * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                a[i] = s.sigmoid ? reciprocal_quick(1.f + exp2_quick(a[i] * -kLog2e)) : a[i] * inv;
                if (bias && i < s.E) a[i] += __ldg(bias + i);
                left = left || (i < s.E && a[i] != a[i]);
                if (a[i] == -INFINITY) open &= ~(1u << i);
            }
        }
        uint64_t order = 0;   // four bits for a choice
        int n = 0, before = 0;
        float last = 0.f;
#pragma unroll 1
        for (;;) {   // scores are looked at behind the choice too, as long as they are near to its last one
            float best = -INFINITY;
            int at = -1;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((open >> i & 1u) && a[i] > best) best = a[i], at = i;
            if (at < 0) break;
            if (kScored && n > 0 && last - best <= 2.f * error + 0x1p-22f * (fabsf(last) + fabsf(best)))   // as near_keys
                left = left || !(logit(row, before) == logit(row, at) && (!bias || __ldg(bias + before) == __ldg(bias + at)));
            else if (n == s.k) break;
            if (n < s.k) {
                order |= (uint64_t)at << (4 * n);
                before = at;
                last = best;
                ++n;
            }
            if (left || (!kScored && n == s.k)) break;
            open &= ~(1u << at);
        }
        if (!left) {
            auto chosen = [&](int j) { return (int)(order >> (4 * j)) & 15; };
            float first = -INFINITY, all = 0.f;
            auto part = [&](float z) {
                return s.sigmoid ? __fdividef(expf(fminf(z, 0.f) - fminf(first, 0.f)), 1.f + expf(-fabsf(z))) : expf(z - first);
            };
            if (s.renormalise) {
#pragma unroll 1
                for (int j = 0; j < n; ++j) first = fmaxf(first, logit(row, chosen(j)));
#pragma unroll 1
                for (int j = 0; j < n; ++j) all += part(logit(row, chosen(j)));
            }
#pragma unroll 1
            for (int j = 0; j < s.k; ++j) {
                float w = 0.f;
                if (j < n) {
                    const float z = logit(row, chosen(j));
                    w = s.scale * (s.renormalise ? share_of(part(z), all) : s.sigmoid ? sigmoid_of(z) : __fdividef(expf(z - top), sum));
                }
                ids[r0 * s.k + j] = j < n ? chosen(j) : -1;
                weights[r0 * s.k + j] = w;
            }
        }
    }
    for (unsigned m = __ballot_sync(kAll, left); m; m &= m - 1) {
        route_row<T, 1, kScored>(s, r0 - lane + (__ffs(m) - 1), lane, spaces[threadIdx.x >> 5], logits, bias, ids, weights);
        __syncwarp();
    }
}

// Gradients by expert gather in shared memory; a lane writes every 32nd element, so that a warp's accesses are neighbours in
// global and in shared memory (65536 rows of 1024 fp32: 47 us, where 16-byte pieces of V neighbours a lane took 130; 45231 of
// 415 bf16: 14, and 86).  kWhole: softmax over all experts, whose every logit has a gradient.
template <typename T, int V, bool kWhole>
__global__ void __launch_bounds__(kBackWarps<V> * 32) route_rows_backward(RouteShape s, const float* __restrict__ dweights,
                                                                        const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                                        T* __restrict__ dlogits) {
    __shared__ __align__(16) float buffers[kBackWarps<V>][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * kBackWarps<V> + warp;
    float* g = buffers[warp];
    pdl_wait();
    pdl_trigger();
    if (r0 >= s.M) return;
    const T* row = logits + r0 * s.ld;
    float e[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (kWhole) e[i] = lane + 32 * i < s.E ? logit(row, lane + 32 * i) : -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) g[i * 32 + lane] = 0.f;
    const int id = lane < s.k ? __ldg(ids + r0 * s.k + lane) : -1;
    const bool held = (uint32_t)id < (uint32_t)s.E;
    const float z = held ? logit(row, id) : -INFINITY;
    const float d = held ? __fmul_rn(__ldg(dweights + r0 * s.k + lane), s.scale) : 0.f;   // rounded: the mean of one is itself
    float mean = 0.f, own = d;
    if (kWhole) {
        float top = e[0], sum = 0.f;
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, e[i]);
        top = max_of_warp(top);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = e[i] == -INFINITY ? 0.f : expf(e[i] - top);
            sum += e[i];
        }
        sum = sum_of_warp(sum);
        const float inv = 1.f / sum;   // no open expert: 0 times infinity is never asked for
        mean = sum_of_warp(held && z != -INFINITY ? d * (expf(z - top) * inv) : 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = e[i] == 0.f ? 0.f : e[i] * inv;
    } else if (s.renormalise) {
        const float share = renormalised(s.sigmoid, held, z, s.width);
        const float all = sum_of_warp(held ? share * d : 0.f);
        own = share * (d - all);
        if (s.sigmoid) own *= sigmoid_of(-z);
    } else {
        own = d * sigmoid_of(z) * sigmoid_of(-z);
    }
    __syncwarp();
    // an expert that is named twice: its lanes find another one's number there, and add one after another
    if (held) g[id] = __int_as_float(lane);
    __syncwarp();
    const bool twice = __any_sync(kAll, held && __float_as_int(g[id]) != lane);
    __syncwarp();
    if (held) g[id] = twice ? 0.f : own;
    __syncwarp();
    if (twice)
        for (int j = 0; j < s.k; ++j) {
            if (lane == j && held) g[id] += own;
            __syncwarp();
        }
    T* out = dlogits + r0 * s.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = lane + 32 * i;
        if (at >= s.E) break;
        float v = g[at];
        if (kWhole) v = e[i] == 0.f ? 0.f : e[i] * (v - mean);
        out[at] = from_f32<T>(v);
    }
}

// Of few experts by a thread for a row.
template <typename T, int V, bool kWhole>
__global__ void __launch_bounds__(kRouteWarps * 32) route_rows_backward_of_few(RouteShape s, const float* __restrict__ dweights,
                                                                               const T* __restrict__ logits,
                                                                               const int32_t* __restrict__ ids, T* __restrict__ dlogits) {
    const int64_t r0 = (int64_t)blockIdx.x * (kRouteWarps * 32) + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (r0 >= s.M) return;
    const T* row = logits + r0 * s.ld;
    float z[V], g[V] = {};
    load_lane<T, V>(row, s.E, s.wide, -INFINITY, z);
    auto of_choices = [&](auto f) {
#pragma unroll 1
        for (int j = 0; j < s.k; ++j) {
            const int id = __ldg(ids + r0 * s.k + j);
            if ((uint32_t)id < (uint32_t)s.E) f(id, logit(row, id), __fmul_rn(__ldg(dweights + r0 * s.k + j), s.scale));   // rounded: the mean of one is itself
        }
    };
    auto give = [&](int id, float v) {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += i == id ? v : 0.f;
    };
    if (kWhole) {
        float top = z[0], sum = 0.f, mean = 0.f;
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, z[i]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = z[i] == -INFINITY ? 0.f : expf(z[i] - top);
            sum += z[i];
        }
        const float inv = 1.f / sum;
        of_choices([&](int id, float at, float d) {
            if (at != -INFINITY) mean += d * (expf(at - top) * inv);
            give(id, d);
        });
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = z[i] == 0.f ? 0.f : z[i] * inv * (g[i] - mean);
    } else if (s.renormalise) {
        float first = -INFINITY, sum = 0.f, mean = 0.f;
        auto part = [&](float at) {
            return s.sigmoid ? __fdividef(expf(fminf(at, 0.f) - fminf(first, 0.f)), 1.f + expf(-fabsf(at))) : expf(at - first);
        };
        of_choices([&](int, float at, float) { first = fmaxf(first, at); });
        of_choices([&](int, float at, float) { sum += part(at); });
        of_choices([&](int, float at, float d) { mean += share_of(part(at), sum) * d; });
        of_choices([&](int id, float at, float d) {
            const float own = share_of(part(at), sum) * (d - mean);
            give(id, s.sigmoid ? own * sigmoid_of(-at) : own);
        });
    } else {
        of_choices([&](int id, float at, float d) { give(id, d * sigmoid_of(at) * sigmoid_of(-at)); });
    }
    T* out = dlogits + r0 * s.E;
    constexpr int N = kVec<T>;
    if constexpr (V % N == 0) {
        if (s.wide) {
#pragma unroll
            for (int q = 0; q < V; q += N) {
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = g[q + i];
                st_piece(out + q, pack<T>(f));
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < s.E) out[i] = from_f32<T>(g[i]);
}

// The least power of two of experts in a lane that holds `each`.
inline int lane_size(int each) {
    int v = 1;
    while (v < each) v *= 2;
    return v;
}
// Whether lanes that hold V experts (each, or none: `first` experts of a lane are multiples of V) read whole 16-byte pieces.
inline bool wide_lanes(const void* p, int64_t ld, int bytes, int V, int per, int each) {
    return each == V && per % V == 0 && V * bytes % 16 == 0 && aligned16(p) && ld * bytes % 16 == 0;
}

template <typename T, bool kScored>
zs_status route_launch(const RouteShape& s, const void* logits, const float* bias, int32_t* ids, float* weights, cudaStream_t stream) {
    const dim3 grid((unsigned)((s.M + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    const T* z = static_cast<const T*>(logits);
    if (s.groups == 1 && s.E <= kRouteFew && s.M >= kRouteFewRows) {   // 65536 rows of 8 bf16, 2 choices: 3.4 us by a thread each, 18.5 by a warp
        const dim3 rows((unsigned)((s.M + kRouteWarps * 32 - 1) / (kRouteWarps * 32)));
        RouteShape f = s;
        f.wide = wide_lanes(logits, s.M > 1 ? s.ld : s.E, sizeof(T), lane_size(s.E), s.E, s.E);
        switch (lane_size(s.E)) {
            case 1:
            case 2: launch(route_rows_of_few<T, 2, kScored>, rows, block, 0, stream, f, z, bias, ids, weights); break;
            case 4: launch(route_rows_of_few<T, 4, kScored>, rows, block, 0, stream, f, z, bias, ids, weights); break;
            case 8: launch(route_rows_of_few<T, 8, kScored>, rows, block, 0, stream, f, z, bias, ids, weights); break;
            default: launch(route_rows_of_few<T, 16, kScored>, rows, block, 0, stream, f, z, bias, ids, weights); break;
        }
        return check_launch("route");
    }
    switch (lane_size(s.each)) {
        case 1: launch(route_rows<T, 1, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
        case 2: launch(route_rows<T, 2, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
        case 4: launch(route_rows<T, 4, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
        case 8: launch(route_rows<T, 8, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
        case 16: launch(route_rows<T, 16, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
        default: launch(route_rows<T, 32, kScored>, grid, block, 0, stream, s, z, bias, ids, weights); break;
    }
    return check_launch("route");
}

template <typename T, bool kWhole>
zs_status route_backward_launch(const RouteShape& s, const float* dweights, const void* logits, const int32_t* ids, void* dlogits,
                                cudaStream_t stream) {
    const T* z = static_cast<const T*>(logits);
    T* dz = static_cast<T*>(dlogits);
    if (s.E <= kRouteFew && s.M >= kRouteFewRows) {
        const int V = lane_size(s.E);
        const dim3 rows((unsigned)((s.M + kRouteWarps * 32 - 1) / (kRouteWarps * 32))), block(kRouteWarps * 32);
        RouteShape f = s;
        f.wide = wide_lanes(logits, s.M > 1 ? s.ld : s.E, sizeof(T), V, s.E, s.E) && wide_lanes(dlogits, s.E, sizeof(T), V, s.E, s.E);
        switch (V) {
            case 1:
            case 2: launch(route_rows_backward_of_few<T, 2, kWhole>, rows, block, 0, stream, f, dweights, z, ids, dz); break;
            case 4: launch(route_rows_backward_of_few<T, 4, kWhole>, rows, block, 0, stream, f, dweights, z, ids, dz); break;
            case 8: launch(route_rows_backward_of_few<T, 8, kWhole>, rows, block, 0, stream, f, dweights, z, ids, dz); break;
            default: launch(route_rows_backward_of_few<T, 16, kWhole>, rows, block, 0, stream, f, dweights, z, ids, dz); break;
        }
        return check_launch("route gradient");
    }
    auto go = [&](auto size) {
        constexpr int V = decltype(size)::value, W = kBackWarps<V>;
        launch(route_rows_backward<T, V, kWhole>, dim3((unsigned)((s.M + W - 1) / W)), dim3(W * 32), 0, stream, s, dweights, z, ids, dz);
    };
    using std::integral_constant;
    switch (lane_size(s.each)) {
        case 1: go(integral_constant<int, 1>()); break;
        case 2: go(integral_constant<int, 2>()); break;
        case 4: go(integral_constant<int, 4>()); break;
        case 8: go(integral_constant<int, 8>()); break;
        case 16: go(integral_constant<int, 16>()); break;
        default: go(integral_constant<int, 32>()); break;
    }
    return check_launch("route gradient");
}

zs_status check(const char* fn, int32_t dtype, int32_t score, const void* logits, int64_t ld, int64_t M, int32_t E, int32_t k, float scale,
                RouteShape& s) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (score != ZS_SCORE_SOFTMAX && score != ZS_SCORE_SIGMOID)
        return fail(ZS_ERR_UNSUPPORTED, "%s: score %d is not a zs_score_kind", fn, score);
    if (M < 0 || M > ((int64_t)1 << 31) - (1 << 16) || E < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld E=%d", fn, (long long)M, E);
    if (k < 1 || k > E) return fail(ZS_ERR_INVALID_ARG, "%s: k=%d is outside [1, E=%d]", fn, k, E);
    if (E > kRouteMaxE || k > kRouteMaxK)
        return fail(ZS_ERR_UNSUPPORTED, "%s: E=%d is above %d or k=%d above %d", fn, E, kRouteMaxE, k, kRouteMaxK);
    if (!(scale - scale == 0.f)) return fail(ZS_ERR_INVALID_ARG, "%s: scale=%g", fn, (double)scale);
    if (M > 0 && !logits) return fail(ZS_ERR_INVALID_ARG, "%s: logits is NULL", fn);
    if (reinterpret_cast<uintptr_t>(logits) & (uintptr_t)(dtype_bytes(dtype) - 1))
        return fail(ZS_ERR_INVALID_ARG, "%s: logits is not aligned to its elements", fn);
    if (M > 1 && ld < E) return fail(ZS_ERR_INVALID_ARG, "%s: a row stride of logits, %lld, is below E=%d", fn, (long long)ld, E);
    s.M = M, s.ld = ld, s.E = E, s.k = k, s.scale = scale;
    s.width = 1;
    while (s.width < k) s.width *= 2;
    s.sigmoid = score == ZS_SCORE_SIGMOID;
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" {

zs_status zs_route(int32_t dtype, int32_t score, const void* logits, int64_t logits_ld, const float* bias, int64_t M, int32_t E,
                   int32_t k, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renormalise, float scale, int32_t* ids,
                   float* weights, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_route";
    RouteShape s = {};
    if (zs_status st = check(fn, dtype, score, logits, logits_ld, M, E, k, scale, s)) return st;
    if (groups < 1 || E % groups) return fail(ZS_ERR_INVALID_ARG, "%s: groups=%d does not divide E=%d", fn, groups, E);
    if (groups > kRouteMaxGroups) return fail(ZS_ERR_UNSUPPORTED, "%s: groups=%d is above %d", fn, groups, kRouteMaxGroups);
    if (top_groups < 1 || top_groups > groups)
        return fail(ZS_ERR_INVALID_ARG, "%s: top_groups=%d is outside [1, groups=%d]", fn, top_groups, groups);
    if (group_top != 1 && group_top != 2) return fail(ZS_ERR_INVALID_ARG, "%s: group_top=%d is neither 1 nor 2", fn, group_top);
    if ((int64_t)top_groups * (E / groups) < k)
        return fail(ZS_ERR_INVALID_ARG, "%s: k=%d experts are more than %d groups of %d hold", fn, k, top_groups, E / groups);
    if (M > 0 && (!ids || !weights)) return fail(ZS_ERR_INVALID_ARG, "%s: ids or weights is NULL", fn);
    for (const void* p : {(const void*)bias, (const void*)ids, (const void*)weights})
        if (reinterpret_cast<uintptr_t>(p) & 3) return fail(ZS_ERR_INVALID_ARG, "%s: bias, ids or weights is not aligned to its elements", fn);
    s.renormalise = renormalise != 0;
    s.groups = top_groups < groups ? groups : 1;   // where all are kept they make no difference
    s.top_groups = top_groups < groups ? top_groups : 1;
    s.per = E / s.groups;
    s.group_top = group_top;
    int slots = 1;
    while (slots < s.groups) slots *= 2;
    s.lanes = 32 / slots;
    while ((1 << s.lane_bits) < s.lanes) ++s.lane_bits;
    s.each = (s.per + s.lanes - 1) / s.lanes;
    if (s.each > kRouteMaxE / 32)
        return fail(ZS_ERR_UNSUPPORTED, "%s: %d groups of %d experts do not fit 32 lanes of %d", fn, s.groups, s.per, kRouteMaxE / 32);
    if (M == 0) return ZS_OK;
    const bool scored = bias || s.groups > 1;
    const int V = lane_size(s.each);
    s.wide = wide_lanes(logits, M > 1 ? logits_ld : E, dtype_bytes(dtype), V, s.per, s.each);
    s.wide_bias = wide_lanes(bias, 0, 4, V, s.per, s.each);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        return scored ? route_launch<T, true>(s, logits, bias, ids, weights, st) : route_launch<T, false>(s, logits, bias, ids, weights, st);
    };
    return dtype == ZS_F32 ? go(float()) : dtype == ZS_BF16 ? go(__nv_bfloat16()) : go(__half());
}

zs_status zs_route_backward(int32_t dtype, int32_t score, const float* dweights, const void* logits, int64_t logits_ld,
                            const int32_t* ids, int64_t M, int32_t E, int32_t k, int32_t renormalise, float scale, void* dlogits,
                            zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_route_backward";
    RouteShape s = {};
    if (zs_status st = check(fn, dtype, score, logits, logits_ld, M, E, k, scale, s)) return st;
    if (M > 0 && (!dweights || !ids || !dlogits)) return fail(ZS_ERR_INVALID_ARG, "%s: dweights, ids or dlogits is NULL", fn);
    if ((reinterpret_cast<uintptr_t>(dweights) | reinterpret_cast<uintptr_t>(ids)) & 3 ||
        reinterpret_cast<uintptr_t>(dlogits) & (uintptr_t)(dtype_bytes(dtype) - 1))
        return fail(ZS_ERR_INVALID_ARG, "%s: dweights, ids or dlogits is not aligned to its elements", fn);
    if (M == 0) return ZS_OK;
    s.renormalise = renormalise != 0;
    s.each = lane_size((E + 31) / 32);
    const bool whole = !s.sigmoid && !s.renormalise;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        using T = decltype(t);
        return whole ? route_backward_launch<T, true>(s, dweights, logits, ids, dlogits, st)
                     : route_backward_launch<T, false>(s, dweights, logits, ids, dlogits, st);
    };
    return dtype == ZS_F32 ? go(float()) : dtype == ZS_BF16 ? go(__nv_bfloat16()) : go(__half());
}

}  // extern "C"
