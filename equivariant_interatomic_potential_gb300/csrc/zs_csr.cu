// Stable destination CSR for the zonal scatter (row_ptr, perm).
//
// The forward of the deepmd-kit pull request "fused Triton zonal scatter for
// the GIE head" walks a destination CSR whose within-node order is the edge
// order ("stable-sort CSR order", section "What").  Two constructions, both
// integer-only in a fixed order, so perm is unique and bit-identical to a
// sequential counting sort; keys outside [0, N) count as key N, after all
// valid ones.
//
// Counting path (N + 1 <= kCntMaxKeys, every bench-sized graph but the
// largest): one pass, three launches with no inter-CTA waiting (one launch of
// one CTA, count_single, for up to kSingleMaxEdges edges; of up to kGroupMaxKeys
// keys one of a cluster, count_group, from 1025 to 16384 edges):
//   count_rank    -- per tile of edges, each edge's stable rank among the
//                    tile's edges of the same node (warp match + per-warp
//                    running counts in shared memory, then a prefix over
//                    warps), and the tile's per-node counts M[tile][n]
//   scan_cols     -- per node, exclusive scan of M[.][n] over tiles
//   count_scatter -- per tile, node bases from a block scan of the node
//                    totals; perm[base[n] + M[tile][n] + rank] = edge
// Radix path (larger N): LSD radix sort with 8-bit digits, each pass in
// three launches:
//   upsweep   -- per tile of keys, a 256-bin digit histogram (shared atomics)
//   scan      -- per digit, exclusive scan of its histogram row over tiles
//   downsweep -- per tile, stable rank of every key among equal digits
//                (warp ballots + per-warp running counts), staged in shared
//                memory in digit order and written out run by run
// and a final pass that reads the sorted keys to write row_ptr.  Up to a million
// keys a pass takes two launches (sort_few): the downsweep adds up the counts.
#include "zs_common.cuh"

namespace zs {
namespace {

constexpr int kCsrWarps = 8;
constexpr int kCsrThreads = kCsrWarps * 32;
#ifndef ZS_CSR_ITEMS
#define ZS_CSR_ITEMS 8
#endif
constexpr int kCsrItems = ZS_CSR_ITEMS;
constexpr int kTile = kCsrWarps * kCsrItems * 32;  // keys per tile
constexpr int kRadix = 256;

__device__ __forceinline__ int32_t key_of(const int32_t* keys_in, int64_t idx, int32_t N, bool first) {
    int32_t k = __ldg(keys_in + idx);
    if (first) k = (k >= 0 && k < N) ? k : N;
    return k;
}

// Lanes of the warp holding the same 8-bit digit as this lane (valid lanes
// only), from one ballot per digit bit (cheaper here than a match instruction).
__device__ __forceinline__ unsigned digit_peers(int dig, bool valid) {
    unsigned peers = __ballot_sync(0xffffffffu, valid);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool bit = (dig >> b) & 1;
        const unsigned bal = __ballot_sync(0xffffffffu, bit);
        peers &= bit ? bal : ~bal;
    }
    return peers;
}

__device__ __forceinline__ unsigned lanemask_lt() {
    unsigned m;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
    return m;
}

// kByTile: the counts of a tile together, for csr_downsweep<.., kScan>.
template <bool kFirst, int kItems, bool kByTile>
__global__ void __launch_bounds__(kCsrThreads)
csr_upsweep(const int32_t* __restrict__ keys_in, int64_t E, int32_t N, int shift,
            int32_t* __restrict__ hist, int T) {
    __shared__ int cnt[kRadix];
    const int tid = threadIdx.x;
    cnt[tid] = 0;   // kCsrThreads == kRadix
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    // counts do not depend on the order of the increments; the tile's keys
    // are all loaded before the first increment (one round trip, not eight)
    const int64_t base = (int64_t)blockIdx.x * (kItems * kCsrThreads);
    int dig[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const int64_t idx = base + u * kCsrThreads + tid;
        dig[u] = idx < E ? (key_of(keys_in, idx, N, kFirst) >> shift) & (kRadix - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u)
        if (dig[u] >= 0) atomicAdd(&cnt[dig[u]], 1);
    __syncthreads();
    hist[kByTile ? (int64_t)blockIdx.x * kRadix + tid : (int64_t)tid * T + blockIdx.x] = cnt[tid];
}

// The counts of kTileGroup tiles, a cluster's, in place of each tile's: those of the tiles before it in the group to `before`,
// a tile's together, and the group's to `groups`.  A CTA adds up 32 digits, which it reads from the others' shared memory.
constexpr int kTileGroup = 8;
template <bool kFirst, int kItems>
__global__ void __launch_bounds__(kCsrThreads)
csr_upsweep_group(const int32_t* __restrict__ keys_in, int64_t E, int32_t N, int shift, int32_t* __restrict__ before,
                  int32_t* __restrict__ groups) {
    __shared__ int cnt[kRadix];
    const int tid = threadIdx.x;
    cnt[tid] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * (kItems * kCsrThreads);
    int dig[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const int64_t idx = base + u * kCsrThreads + tid;
        dig[u] = idx < E ? (key_of(keys_in, idx, N, kFirst) >> shift) & (kRadix - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u)
        if (dig[u] >= 0) atomicAdd(&cnt[dig[u]], 1);
    cluster_barrier();
    if (tid < kRadix / kTileGroup) {
        const int group = blockIdx.x / kTileGroup, d = (blockIdx.x % kTileGroup) * (kRadix / kTileGroup) + tid;
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(cnt + d));
        int c[kTileGroup], run = 0;
#pragma unroll
        for (int r = 0; r < kTileGroup; ++r)
            asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
                         : "=r"(c[r]) : "r"(at), "r"(r) : "memory");
#pragma unroll
        for (int r = 0; r < kTileGroup; ++r) {
            before[(int64_t)(group * kTileGroup + r) * kRadix + d] = run;
            run += c[r];
        }
        groups[(int64_t)group * kRadix + d] = run;
    }
    cluster_barrier();   // no CTA ends before all have read
}

// One CTA per row: exclusive scan of hist[d, 0..T) in place, total to tot[d].
// Thread i takes the consecutive entries [i * per, (i + 1) * per), all loaded
// before they are added (a row is one round trip of loads, not one per
// 256 entries).
constexpr int kScanPer = 16;
__global__ void __launch_bounds__(kCsrThreads)
csr_scan(int32_t* __restrict__ hist, int T, int32_t* __restrict__ tot) {
    __shared__ int wsum[kCsrWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* row = hist + (int64_t)blockIdx.x * T;
    pdl_wait();
    pdl_trigger();
    int carry = 0;
    for (int c0 = 0; c0 < T; c0 += kScanPer * kCsrThreads) {
        const int per = imin(kScanPer, (imin(T - c0, kScanPer * kCsrThreads) + kCsrThreads - 1) / kCsrThreads);
        const int i0 = c0 + tid * per;
        int v[kScanPer];
        int own = 0;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) {
            v[k] = (k < per && i0 + k < T) ? row[i0 + k] : 0;
            own += v[k];
        }
        int incl = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int pre = carry;
        int all = carry;
#pragma unroll
        for (int w = 0; w < kCsrWarps; ++w) {
            if (w < warp) pre += wsum[w];
            all += wsum[w];
        }
        int run = pre + incl - own;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k)
            if (k < per && i0 + k < T) {
                row[i0 + k] = run;
                run += v[k];
            }
        carry = all;
        __syncthreads();
    }
    if (tid == 0) tot[blockIdx.x] = carry;
}

// kScan 0: hist and tot of csr_scan.  1: hist holds the T tiles' counts as
// csr_upsweep<.., kByTile> left them (few tiles), which every CTA adds up itself.
// 2: those of T groups of tiles, and tot what is before each tile in its group,
// as csr_upsweep_group left them.
template <bool kFirst, int kItems, int kScan>
__global__ void __launch_bounds__(kCsrThreads)
csr_downsweep(const int32_t* __restrict__ keys_in, const int32_t* __restrict__ vals_in,
              int64_t E, int32_t N, int shift,
              const int32_t* __restrict__ hist, const int32_t* __restrict__ tot, int T,
              int32_t* __restrict__ keys_out, int32_t* __restrict__ vals_out) {
    __shared__ int cnt[kCsrWarps][kRadix];
    __shared__ int wsum[kCsrWarps];
    __shared__ int dbase[kRadix];
    constexpr int kTileKeys = kItems * kCsrThreads;
    __shared__ int32_t skey[kTileKeys], sval[kTileKeys];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kCsrWarps * kRadix; i += kCsrThreads) (&cnt[0][0])[i] = 0;
    pdl_wait();
    pdl_trigger();

    const int64_t base = (int64_t)blockIdx.x * kTileKeys + (int64_t)warp * kItems * 32;
    int32_t key[kItems], val[kItems];
    int rank[kItems], dig[kItems];
    const unsigned lt = lanemask_lt();
    // every item's key and value are on their way before the digits' places are
    // added up and the ranking starts (whose synchronisations would hold them back)
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int64_t idx = base + i * 32 + lane;
        const bool valid = idx < E;
        key[i] = valid ? key_of(keys_in, idx, N, kFirst) : 0;
        val[i] = valid ? (kFirst ? (int32_t)idx : __ldg(vals_in + idx)) : 0;
        dig[i] = valid ? ((key[i] >> shift) & (kRadix - 1)) : kRadix;
    }
    // this tile's offset within each digit, loaded now beside the totals
    int hv = kScan == 2 ? tot[(int64_t)blockIdx.x * kRadix + tid] : 0, total = 0;
    if (kScan) {
        constexpr int kAtOnce = 16;   // loads in flight, the last ones too
        for (int t0 = 0; t0 < T; t0 += kAtOnce) {
            int c[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) c[u] = t0 + u < T ? hist[(int64_t)(t0 + u) * kRadix + tid] : 0;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                hv += t0 + u < (int)blockIdx.x / (kScan == 2 ? kTileGroup : 1) ? c[u] : 0;
                total += c[u];
            }
        }
    } else {
        hv = hist[(int64_t)tid * T + blockIdx.x];
        total = tot[tid];
    }
    // Exclusive scan of the 256 digit totals (kCsrThreads == kRadix).
    {
        const int v = total;
        int incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int pre = 0;
        for (int w = 0; w < warp; ++w) pre += wsum[w];
        dbase[tid] = pre + incl - v;
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const bool valid = dig[i] < kRadix;
        const unsigned peers = digit_peers(dig[i] & (kRadix - 1), valid);
        rank[i] = valid ? cnt[warp][dig[i]] + __popc(peers & lt) : 0;
        __syncwarp();
        if (valid && lane == __ffs(peers) - 1) cnt[warp][dig[i]] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    {
        // one thread per digit: per-warp offsets inside the tile, the tile's
        // count of the digit, and where the digit's run starts in the tile
        const int d = tid;
        int own = 0;
#pragma unroll
        for (int w = 0; w < kCsrWarps; ++w) {
            const int c = cnt[w][d];
            cnt[w][d] = own;
            own += c;
        }
        int incl = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        __syncthreads();                     // wsum is reused from the digit-total scan
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int pre = 0;
        for (int w = 0; w < warp; ++w) pre += wsum[w];
        const int local = pre + incl - own;  // first tile slot of digit d
        // global position of the tile's first key of digit d, minus its tile slot
        dbase[d] = dbase[d] + hv - local;
#pragma unroll
        for (int w = 0; w < kCsrWarps; ++w) cnt[w][d] += local;
    }
    __syncthreads();
    // stage the tile in digit order, then write each digit's run contiguously
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (dig[i] < kRadix) {
            const int slot = cnt[warp][dig[i]] + rank[i];
            skey[slot] = key[i];
            sval[slot] = val[i];
        }
    }
    __syncthreads();
    const int n_in_tile = (int)imin<int64_t>(kTileKeys, E - (int64_t)blockIdx.x * kTileKeys);
    for (int slot = tid; slot < n_in_tile; slot += kCsrThreads) {
        const int32_t k = skey[slot];
        const int pos = dbase[(k >> shift) & (kRadix - 1)] + slot;
        keys_out[pos] = k;
        vals_out[pos] = sval[slot];
    }
}

// row_ptr from sorted keys: position j is the first of every node in
// (key[j-1], key[j]]; the count of keys equal to N (invalid) is E - row_ptr[N].
// A thread looks at kRowPtrPer consecutive positions and writes the few nodes
// between two keys; where they are many, the lanes of its warp write them
// together (one key of 50021: 332 us by one thread).
constexpr int kRowPtrPer = 4, kRowPtrFew = 16;

__global__ void __launch_bounds__(256)
csr_row_ptr(const int32_t* __restrict__ sorted, int64_t E, int32_t N,
            int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    const int64_t j0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kRowPtrPer;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    int64_t kprev = j0 > 0 && j0 <= E ? (int64_t)__ldg(sorted + j0 - 1) : -1;
    int64_t kcur[kRowPtrPer];
#pragma unroll
    for (int i = 0; i < kRowPtrPer; ++i) kcur[i] = j0 + i < E ? (int64_t)__ldg(sorted + j0 + i) : (int64_t)N + 1;
#pragma unroll
    for (int i = 0; i < kRowPtrPer; ++i) {
        const int64_t j = j0 + i;
        const int64_t lo = kprev + 1, hi = j <= E ? imin(kcur[i], (int64_t)N) : -1;   // nodes [lo, hi]
        if (hi == N && lo <= hi && bad) *bad = (int32_t)(E - j);
        const bool many = hi - lo >= kRowPtrFew;
        if (!many)
            for (int64_t n = lo; n <= hi; ++n) row_ptr[n] = (int32_t)j;
        for (unsigned m = __ballot_sync(0xffffffffu, many); m; m &= m - 1) {
            const int src = __ffs(m) - 1;
            const int64_t from = __shfl_sync(0xffffffffu, lo, src), to = __shfl_sync(0xffffffffu, hi, src);
            const int at = __shfl_sync(0xffffffffu, (int)j, src);
            for (int64_t n = from + lane; n <= to; n += 32) row_ptr[n] = at;
        }
        kprev = kcur[i];
    }
}

// The same where nodes are many more than keys: for each node the first key that
// is not below it.  A CTA finds where the keys of its 256 nodes lie with as many
// probes at a time (two rounds for 65536 keys), then each thread its node's in
// there, three probes at a time.
struct Found {
    uint32_t lo, hi;   // the place is in [lo, hi]
    // after `below` of probes at lo + (i + 1) step - 1 were below the key
    __device__ __forceinline__ void narrow(uint32_t step, uint32_t below, uint32_t probes) {
        if (below < probes) hi = imin(hi, lo + (below + 1) * step - 1);
        lo += below * step;
    }
};
constexpr int kRowPtrNodes = 256;

__global__ void __launch_bounds__(kRowPtrNodes)
csr_row_ptr_of_few(const int32_t* __restrict__ sorted, int32_t E, int32_t N, int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    const int64_t v0 = (int64_t)blockIdx.x * kRowPtrNodes, v = v0 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    Found first = {0, (uint32_t)E}, last = first;
    while (first.lo < first.hi || last.lo < last.hi) {
        const uint32_t p = (first.hi - first.lo + kRowPtrNodes - 1) / kRowPtrNodes, q = (last.hi - last.lo + kRowPtrNodes - 1) / kRowPtrNodes;
        const uint32_t a = first.lo + (threadIdx.x + 1) * p - 1, b = last.lo + (threadIdx.x + 1) * q - 1;
        const int before = p && a < first.hi && __ldg(sorted + a) < v0;
        const int upto = q && b < last.hi && __ldg(sorted + b) < v0 + kRowPtrNodes;
        first.narrow(p, (uint32_t)__syncthreads_count(before), kRowPtrNodes);
        last.narrow(q, (uint32_t)__syncthreads_count(upto), kRowPtrNodes);
    }
    if (v > N) return;
    Found at = {first.lo, last.lo};
    while (at.lo < at.hi) {
        const uint32_t step = (at.hi - at.lo + 3) / 4;
        uint32_t below = 0;
#pragma unroll
        for (uint32_t i = 0; i < 3; ++i) {
            const uint32_t p = at.lo + (i + 1) * step - 1;
            below += p < at.hi && __ldg(sorted + p) < v;
        }
        at.narrow(step, below, 3);
    }
    row_ptr[v] = (int32_t)at.lo;
    if (v == N && bad) *bad = E - (int32_t)at.lo;
}

// ---------------------------------------------------------------------------
// Counting path.  A tile is kCntWarps warps x `rounds` rounds of 32 edges;
// warp w of tile t owns the edges [t*TS + w*TW, t*TS + (w+1)*TW), TW = 32*rounds.
constexpr int kCntWarps = 16;
constexpr int kCntThreads = kCntWarps * 32;
#ifndef ZS_CNT_MAX_KEYS
#define ZS_CNT_MAX_KEYS 5120
#endif
constexpr int kCntMaxKeys = ZS_CNT_MAX_KEYS;   // N + 1 up to this takes the counting path
constexpr int kCntMaxRounds = 16;       // tile of at most 8192 edges
constexpr int kCntTargetTiles = 152;    // tiles sized so one wave covers 152 SMs

constexpr int kCntMaxPer = (kCntMaxKeys + kCntThreads - 1) / kCntThreads;   // keys per thread in a block scan

// Keys rounded up to even, so two keys' 16-bit counters share a 32-bit word.
__host__ __device__ __forceinline__ int count_pairs(int nkeys) { return (nkeys + 1) >> 1; }

// Shared memory of csr_count_rank: 16-bit counters [kCntWarps][keys, padded
// to even], then one 32-bit word per edge of the tile.
inline int count_rank_smem(int nkeys, int rounds) { return count_pairs(nkeys) * 4 * kCntWarps + rounds * kCntThreads * 4; }

// 4-byte asynchronous copy global -> shared (cp.async): a CTA issues all of
// a tile's copies, then waits once (cp_async_wait_all + a barrier).
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(gmem) : "memory");
}

// 8- and 16-byte copies (both addresses aligned to the size).
__device__ __forceinline__ void cp_async8(void* smem, const void* gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async16b(void* smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(gmem) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// n int32 from global src to shared dst (16-byte aligned): 16-byte pieces
// when src is 16-byte aligned too, else 4-byte ones; CTA-cooperative.
__device__ __forceinline__ void copy_ints(int32_t* dst, const int32_t* src, int n, int tid, int nthreads) {
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        const int n4 = n >> 2;
        for (int j = tid; j < n4; j += nthreads) cp_async16b(dst + 4 * j, src + 4 * j);
        for (int i = 4 * n4 + tid; i < n; i += nthreads) cp_async4(dst + i, src + i);
    } else {
        for (int i = tid; i < n; i += nthreads) cp_async4(dst + i, src + i);
    }
}

__device__ __forceinline__ int32_t clamp_key(int32_t k, int32_t N) { return (uint32_t)k < (uint32_t)N ? k : N; }

// Ranks within each warp's run of a tile (warp w owns edges [w * 32 * rounds,
// (w + 1) * 32 * rounds) of the tile): packed[i] holds edge i's key on entry
// and key << 16 | (its rank among the warp's earlier edges of that key) on
// exit; wcnt (the warp's 16-bit counters, zeroed) ends with the warp's count
// of every key.  Per round of 32 edges, the lanes holding each key (peers)
// are found by claim and verify: every lane writes its lane id into bits
// 10..14 of its key's counter (count < 1024 stays in bits 0..9), reads the
// slot back, and lanes that lost the claim are grouped with the winner by
// one ballot per contested key.  Uncontested rounds cost no ballot loop.  Of
// few keys (species, experts) most lanes are contested: there the lanes of a key
// are found by one ballot for each of its bits instead (up to kFewKeyBits of
// them; 4096 edges, 89 skewed keys: the whole build 7.8 -> 6.4 us; with nine, 256
// keys, no gain).
constexpr int kFewKeyBits = 8;
__device__ __forceinline__ void rank_few_keys(uint32_t* packed, uint16_t* wcnt, int rounds, int n, int32_t N, int warp, int lane) {
    const unsigned lt = lanemask_lt();
    const int TW = rounds * 32, bits = 32 - __clz(N);
    for (int r = 0; r < rounds; ++r) {
        const int i = warp * TW + r * 32 + lane;
        const bool valid = i < n;
        const int key = valid ? clamp_key((int32_t)packed[i], N) : 0;
        unsigned peers = __ballot_sync(0xffffffffu, valid);
#pragma unroll
        for (int b = 0; b < kFewKeyBits; ++b) {
            if (b >= bits) break;
            const bool bit = (key >> b) & 1;
            const unsigned bal = __ballot_sync(0xffffffffu, bit);
            peers &= bit ? bal : ~bal;
        }
        const uint32_t before = valid ? wcnt[key] : 0u;
        __syncwarp();
        if (valid) {
            if ((peers & lt) == 0) wcnt[key] = (uint16_t)(before + __popc(peers));
            packed[i] = ((uint32_t)key << 16) | (before + __popc(peers & lt));
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void rank_in_warp(uint32_t* packed, uint16_t* wcnt, int rounds, int n, int32_t N, int warp,
                                             int lane) {
    if (N >> kFewKeyBits == 0) {
        rank_few_keys(packed, wcnt, rounds, n, N, warp, lane);
        return;
    }
    const unsigned lt = lanemask_lt();
    const int TW = rounds * 32;
    for (int r = 0; r < rounds; ++r) {
        const int i = warp * TW + r * 32 + lane;
        const bool valid = i < n;
        const int key = valid ? clamp_key((int32_t)packed[i], N) : 0;
        const uint32_t before = valid ? wcnt[key] : 0u;          // count so far, owner bits clear
        __syncwarp();
        if (valid) wcnt[key] = (uint16_t)(before | ((uint32_t)lane << 10));
        __syncwarp();
        const int owner = valid ? (int)(wcnt[key] >> 10) : lane;
        unsigned lost = __ballot_sync(0xffffffffu, valid && owner != lane);
        unsigned peers = 1u << lane;
        while (lost) {
            const int w = __shfl_sync(0xffffffffu, owner, __ffs(lost) - 1);
            const unsigned group = __ballot_sync(0xffffffffu, valid && owner == w);
            if (group & (1u << lane)) peers = group;
            lost &= ~group;
        }
        __syncwarp();
        if (valid) {
            if (lane == __ffs(peers) - 1) wcnt[key] = (uint16_t)(before + __popc(peers));
            packed[i] = ((uint32_t)key << 16) | (before + __popc(peers & lt));
        }
        __syncwarp();
    }
}

// Pair q of keys: the warps' counters turned into exclusive prefixes over the
// warps (both 16-bit halves at once: every partial sum is below 2^16); the
// tile's two counts are returned in the halves of the result.
__device__ __forceinline__ uint32_t prefix_over_warps(uint32_t* cnt_words, int npairs, int q) {
    uint32_t c[kCntWarps];
#pragma unroll
    for (int w = 0; w < kCntWarps; ++w) c[w] = cnt_words[w * npairs + q];
    uint32_t run = 0;
#pragma unroll
    for (int w = 0; w < kCntWarps; ++w) {
        cnt_words[w * npairs + q] = run;
        run += c[w];
    }
    return run;
}

// Node bases: an exclusive scan of the nkeys totals in tot (shared memory),
// thread tid taking keys [tid * per, (tid + 1) * per).  base[k] = first CSR
// position of key k plus off[k] (off may alias base; NULL: 0); with row_ptr,
// the positions go to row_ptr too and the total of key N (invalid keys) to
// *bad.  Every thread of the CTA must call it (it synchronises the CTA).
__device__ __forceinline__ void key_bases(const int32_t* tot, const int32_t* off, int32_t* base, int nkeys, int32_t N,
                                          int32_t* wsum, int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (nkeys + kCntThreads - 1) / kCntThreads;
    const int k0 = tid * per;
    int32_t v[kCntMaxPer], o[kCntMaxPer];
    int32_t own = 0;
#pragma unroll
    for (int j = 0; j < kCntMaxPer; ++j) {
        const bool in = j < per && k0 + j < nkeys;
        v[j] = in ? tot[k0 + j] : 0;
        o[j] = (in && off) ? off[k0 + j] : 0;
        own += v[j];
    }
    int32_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int32_t run = incl - own;
    for (int w = 0; w < warp; ++w) run += wsum[w];
#pragma unroll
    for (int j = 0; j < kCntMaxPer; ++j) {
        const int k = k0 + j;
        if (j < per && k < nkeys) {
            if (row_ptr) {
                row_ptr[k] = run;
                if (k == N && bad) *bad = v[j];
            }
            base[k] = run + o[j];
            run += v[j];
        }
    }
}

// Per tile: each edge's stable rank among the tile's edges of the same key
// (to rank[]), and the tile's count of every key (to row `tile` of M, whose
// rows hold 2 * count_pairs(N + 1) counts).
__global__ void __launch_bounds__(kCntThreads, 1)
csr_count_rank(const int32_t* __restrict__ dst, int64_t E, int32_t N, int rounds,
               int32_t* __restrict__ M, uint16_t* __restrict__ rank) {
    extern __shared__ uint32_t cnt_words[];
    const int nkeys = N + 1;
    const int npairs = count_pairs(nkeys);
    // warp w's counter of key k is the 16-bit half (k & 1) of word w * npairs + k / 2
    uint16_t* cnt = reinterpret_cast<uint16_t*>(cnt_words);
    uint32_t* packed = cnt_words + kCntWarps * npairs;      // [TS]: key << 16 | rank in warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TW = rounds * 32;
    const int64_t tbase = (int64_t)blockIdx.x * rounds * kCntThreads;
    const int n_in_tile = (int)imin<int64_t>((int64_t)rounds * kCntThreads, E - tbase);
    pdl_wait();
    pdl_trigger();
    // the tile's keys land in packed[] while the counters are cleared
    copy_ints(reinterpret_cast<int32_t*>(packed), dst + tbase, n_in_tile, tid, kCntThreads);
    // kCntWarps * npairs words, a multiple of four
    for (int i = tid; i < kCntWarps * npairs / 4; i += kCntThreads) reinterpret_cast<uint4*>(cnt_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    cp_async_wait_all();
    __syncthreads();

    rank_in_warp(packed, cnt + 2 * warp * npairs, rounds, n_in_tile, N, warp, lane);
    __syncthreads();
    // per pair of keys: prefixes over the warps, tile counts to M
    for (int q = tid; q < npairs; q += kCntThreads) {
        const uint32_t run = prefix_over_warps(cnt_words, npairs, q);
        reinterpret_cast<int2*>(M + (int64_t)blockIdx.x * 2 * npairs)[q] = make_int2((int)(run & 0xffffu), (int)(run >> 16));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCntMaxRounds; ++u) {
        const int i = tid + u * kCntThreads;
        if (i >= n_in_tile) break;
        const uint32_t p = packed[i];
        const int w = i / TW;
        rank[tbase + i] = (uint16_t)((p & 0xffffu) + cnt[2 * w * npairs + (p >> 16)]);
    }
}

// Per key: exclusive scan over the tiles of its column of M (rows of S
// counts) in place, total to tot[key].  A CTA takes 32 keys, one per lane;
// its warps split the tiles into chunks and combine through shared memory.
__global__ void __launch_bounds__(kCntThreads)
csr_scan_cols(int32_t* __restrict__ M, int T, int S, int nkeys, int32_t* __restrict__ tot) {
    __shared__ int32_t part[kCntWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int key = blockIdx.x * 32 + lane;
    const int chunk = (T + kCntWarps - 1) / kCntWarps;
    const int t0 = imin(T, warp * chunk), t1 = imin(T, t0 + chunk);
    pdl_wait();
    pdl_trigger();
    constexpr int kRegs = 16;
    __shared__ int32_t stage[kCntWarps][kRegs][32];
    int32_t c[kRegs];
    int32_t sum = 0;
    const bool in_regs = chunk <= kRegs;
    if (in_regs) {
        // one batch of copies per lane, then the lane's own values from shared memory
        if (key < nkeys)
            for (int j = 0; j < t1 - t0; ++j) cp_async4(&stage[warp][j][lane], M + (int64_t)(t0 + j) * S + key);
        cp_async_wait_all();
#pragma unroll
        for (int j = 0; j < kRegs; ++j) {
            c[j] = (key < nkeys && j < t1 - t0) ? stage[warp][j][lane] : 0;
            sum += c[j];
        }
    } else if (key < nkeys) {
#pragma unroll 8
        for (int t = t0; t < t1; ++t) sum += M[(int64_t)t * S + key];
    }
    part[warp][lane] = sum;
    __syncthreads();
    int32_t run = 0;
    for (int w = 0; w < warp; ++w) run += part[w][lane];
    if (key >= nkeys) return;
    if (warp == kCntWarps - 1) tot[key] = run + sum;
    if (in_regs) {
#pragma unroll
        for (int j = 0; j < kRegs; ++j) {
            if (t0 + j < t1) M[(int64_t)(t0 + j) * S + key] = run;
            run += c[j];
        }
        return;
    }
    for (int t = t0; t < t1; ++t) {
        const int64_t i = (int64_t)t * S + key;
        const int32_t v = M[i];
        M[i] = run;
        run += v;
    }
}

// Shared memory of csr_count_scatter (int32 words, each array starting on a
// 16-byte boundary): the node totals, the tile's row of M, kCntWarps warp
// sums, the tile's keys, its ranks (two per word).
__host__ __device__ __forceinline__ int align4(int n) { return (n + 3) & ~3; }
inline int count_scatter_smem(int nkeys, int rounds) {
    return (align4(nkeys) + align4(2 * count_pairs(nkeys)) + kCntWarps + rounds * kCntThreads + rounds * kCntThreads / 2) * 4;
}

// Dynamic shared memory requested so that no two CTAs of a kernel share an SM
// (a kernel launched early behind its predecessor otherwise lands two CTAs
// on one SM while others idle, doubling the slowest CTA's time).
constexpr int kOneCtaPerSmSmem = 120 * 1024;

// Per tile: node bases from an exclusive scan of the key totals plus the
// tile's offset within each key, then every edge to its CSR position.  Tile 0
// also writes row_ptr and the count of invalid keys.
__global__ void __launch_bounds__(kCntThreads)
csr_count_scatter(const int32_t* __restrict__ dst, const uint16_t* __restrict__ rank,
                  const int32_t* __restrict__ M, const int32_t* __restrict__ tot,
                  int64_t E, int32_t N, int rounds,
                  int32_t* __restrict__ perm, int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    extern __shared__ __align__(16) int32_t ktot[];
    const int nkeys = N + 1;
    const int S = 2 * count_pairs(nkeys);
    int32_t* kbase = ktot + align4(nkeys);
    int32_t* wsum = kbase + align4(S);
    int32_t* skey = wsum + kCntWarps;
    uint32_t* srank = reinterpret_cast<uint32_t*>(skey + rounds * kCntThreads);
    const int tid = threadIdx.x;
    const int64_t tbase = (int64_t)blockIdx.x * rounds * kCntThreads;
    const int n_in_tile = (int)imin<int64_t>((int64_t)rounds * kCntThreads, E - tbase);
    pdl_wait();
    pdl_trigger();
    // every input of the tile in one batch of asynchronous copies: the tile's
    // row of M, the node totals, the tile's keys and its ranks (in pairs; the
    // tile starts on an even edge, an odd last edge is read directly)
    // (rows of M are S = even counts long: 8-byte pieces; the rank array and
    // the tile start are 16-byte aligned: 16-byte pieces of eight ranks)
    const int32_t* mrow = M + (int64_t)blockIdx.x * S;
    for (int j = tid; j < S / 2; j += kCntThreads) cp_async8(kbase + 2 * j, mrow + 2 * j);
    copy_ints(ktot, tot, nkeys, tid, kCntThreads);
    copy_ints(skey, dst + tbase, n_in_tile, tid, kCntThreads);
    const int n8 = n_in_tile >> 3;
    for (int j = tid; j < n8; j += kCntThreads) cp_async16b(srank + 4 * j, rank + tbase + 8 * j);
    for (int j = 4 * n8 + tid; j < n_in_tile / 2; j += kCntThreads) cp_async4(srank + j, rank + tbase + 2 * j);
    if ((n_in_tile & 1) && tid == 0) srank[n_in_tile / 2] = __ldg(rank + tbase + n_in_tile - 1);
    cp_async_wait_all();
    __syncthreads();
    key_bases(ktot, kbase, kbase, nkeys, N, wsum, blockIdx.x == 0 ? row_ptr : nullptr, bad);
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n_in_tile; i += kCntThreads) {
        const uint32_t rk = (srank[i >> 1] >> (16 * (i & 1))) & 0xffffu;
        perm[kbase[clamp_key(skey[i], N)] + (int32_t)rk] = (int32_t)(tbase + i);
    }
}

// Small graphs (up to kSingleMaxEdges edges, where count_group does not take
// them): the whole counting path in one CTA and one launch -- csr_count_rank's
// ranking and counts, then csr_count_scatter's node bases and scatter, the
// counts staying in shared memory (with one tile, every edge's offset within its
// key is its rank).
constexpr int kSingleRounds = 8;
constexpr int kSingleMaxEdges = kSingleRounds * kCntThreads;   // 4096: 6.4 to 8.3 us; 8192 edges took 9.4 to 15, 6 in three launches
inline int count_single_smem(int nkeys, int rounds) {
    return count_rank_smem(nkeys, rounds) + 2 * count_pairs(nkeys) * 4;
}

__global__ void __launch_bounds__(kCntThreads, 1)
csr_count_single(const int32_t* __restrict__ dst, int64_t E, int32_t N, int rounds,
                 int32_t* __restrict__ perm, int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    extern __shared__ uint32_t cnt_words[];
    __shared__ int32_t wsum[kCntWarps];
    const int nkeys = N + 1;
    const int npairs = count_pairs(nkeys);
    uint16_t* cnt = reinterpret_cast<uint16_t*>(cnt_words);
    uint32_t* packed = cnt_words + kCntWarps * npairs;                          // [TS]: key << 16 | rank
    int32_t* ktot = reinterpret_cast<int32_t*>(packed + rounds * kCntThreads);   // [2 * npairs]: key totals, then bases
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TW = rounds * 32;
    const int n = (int)E;
    pdl_wait();
    pdl_trigger();
    copy_ints(reinterpret_cast<int32_t*>(packed), dst, n, tid, kCntThreads);
    for (int i = tid; i < kCntWarps * npairs / 4; i += kCntThreads) reinterpret_cast<uint4*>(cnt_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    cp_async_wait_all();
    __syncthreads();
    rank_in_warp(packed, cnt + 2 * warp * npairs, rounds, n, N, warp, lane);
    __syncthreads();
    // per pair of keys: exclusive prefix over the warps, and the key totals
    for (int q = tid; q < npairs; q += kCntThreads) {
        const uint32_t run = prefix_over_warps(cnt_words, npairs, q);
        ktot[2 * q] = (int32_t)(run & 0xffffu);
        ktot[2 * q + 1] = (int32_t)(run >> 16);
    }
    __syncthreads();
    for (int i = tid; i < n; i += kCntThreads) {
        const uint32_t p = packed[i];
        const int w = i / TW;
        packed[i] = (p & 0xffff0000u) | ((p & 0xffffu) + cnt[2 * w * npairs + (p >> 16)]);
    }
    // node bases (one tile: an edge's offset within its key is its rank)
    key_bases(ktot, nullptr, ktot, nkeys, N, wsum, row_ptr, bad);
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kCntThreads) {
        const uint32_t p = packed[i];
        perm[ktot[p >> 16] + (int32_t)(p & 0xffffu)] = i;
    }
}

// The same by a cluster of kGroupCtas CTAs, a tile each: what the others counted
// is read from their shared memory, so that no counts go through global memory
// and no second kernel waits for them (89 keys: 4096 edges 3.8 us, one CTA 7.1;
// 8192 4.2 and 12291 5.4, three launches 6.5 and 6.2; 1000 as long as one CTA).
constexpr int kGroupCtas = 8, kGroupMinEdges = 1024, kGroupMaxKeys = 1024, kGroupMaxRounds = 4;
inline int count_group_smem(int nkeys, int rounds) { return count_rank_smem(nkeys, rounds) + 6 * count_pairs(nkeys) * 4; }

__global__ void __launch_bounds__(kCntThreads, 1)
csr_count_group(const int32_t* __restrict__ dst, int64_t E, int32_t N, int rounds,
                int32_t* __restrict__ perm, int32_t* __restrict__ row_ptr, int32_t* __restrict__ bad) {
    extern __shared__ uint32_t cnt_words[];
    __shared__ int32_t wsum[kCntWarps];
    const int nkeys = N + 1;
    const int npairs = count_pairs(nkeys);
    uint16_t* cnt = reinterpret_cast<uint16_t*>(cnt_words);
    uint32_t* packed = cnt_words + kCntWarps * npairs;                           // [TS]: key << 16 | rank
    int32_t* mine = reinterpret_cast<int32_t*>(packed + rounds * kCntThreads);   // [2 * npairs]: this tile's counts
    int32_t* tot = mine + 2 * npairs;                                            // all tiles'
    int32_t* base = tot + 2 * npairs;                                            // those of the tiles before, then positions
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TW = rounds * 32;
    const int tbase = (int)blockIdx.x * rounds * kCntThreads;
    const int n = imax(imin(rounds * kCntThreads, (int)E - tbase), 0);
    pdl_wait();
    pdl_trigger();
    copy_ints(reinterpret_cast<int32_t*>(packed), dst + (n > 0 ? tbase : 0), n, tid, kCntThreads);
    for (int i = tid; i < kCntWarps * npairs / 4; i += kCntThreads) reinterpret_cast<uint4*>(cnt_words)[i] = make_uint4(0u, 0u, 0u, 0u);
    cp_async_wait_all();
    __syncthreads();
    rank_in_warp(packed, cnt + 2 * warp * npairs, rounds, n, N, warp, lane);
    __syncthreads();
    for (int q = tid; q < npairs; q += kCntThreads) {
        const uint32_t run = prefix_over_warps(cnt_words, npairs, q);
        mine[2 * q] = (int32_t)(run & 0xffffu);
        mine[2 * q + 1] = (int32_t)(run >> 16);
    }
    cluster_barrier();
    for (int k = tid; k < nkeys; k += kCntThreads) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine + k));
        int32_t c[kGroupCtas], all = 0, before = 0;
#pragma unroll
        for (int r = 0; r < kGroupCtas; ++r)
            asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
                         : "=r"(c[r]) : "r"(at), "r"(r) : "memory");
#pragma unroll
        for (int r = 0; r < kGroupCtas; ++r) {
            all += c[r];
            before += r < (int)blockIdx.x ? c[r] : 0;
        }
        tot[k] = all;
        base[k] = before;
    }
    cluster_arrive();   // no CTA ends before all have read
    __syncthreads();
    key_bases(tot, base, base, nkeys, N, wsum, blockIdx.x == 0 ? row_ptr : nullptr, bad);
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kCntThreads) {
        const uint32_t p = packed[i];
        perm[base[p >> 16] + (int32_t)((p & 0xffffu) + cnt[2 * (i / TW) * npairs + (p >> 16)])] = tbase + i;
    }
    cluster_wait();
}

// All passes over tiles of 256 * kItems keys, at most kFewTiles of them (so small that most SMs have one) or of groups of them
// (kGroups), and no kernel that scans their counts (262144 keys of 7921: 21 us, 30 with one).  These (1 KB a tile, at most 4
// bytes a key but for kItems = 1) lie in `hist` if they are one tile's, else where the pass leaves an array free: the last one
// that of the values it would write, of several the ones before it perm; of two both v[1], which has room behind it for the up
// to 1 KB that kItems = 1 takes more.  Returns the sorted keys.
constexpr int kFewTiles = 64;
template <int kItems, bool kGroups = false>
const int32_t* sort_few(int passes, const int32_t* dst, int64_t E, int32_t N, int32_t* const (&k)[2], int32_t* const (&v)[2], int32_t* perm,
                        int32_t* hist, cudaStream_t s) {
    const int T = (int)((E + kItems * kCsrThreads - 1) / (kItems * kCsrThreads)), G = (T + kTileGroup - 1) / kTileGroup;
    const int32_t* none = nullptr;
    auto pass_of = [&](auto first, int pass, const int32_t* kin, const int32_t* vin, int32_t* kout, int32_t* vout, int32_t* counted) {
        constexpr bool kFirst = decltype(first)::value;
        if constexpr (kGroups) {
            int32_t* groups = counted + (int64_t)G * kTileGroup * kRadix;
            launch_clusters(kTileGroup, csr_upsweep_group<kFirst, kItems>, G * kTileGroup, kCsrThreads, 0, s, kin, E, N, 8 * pass, counted, groups);
            launch(csr_downsweep<kFirst, kItems, 2>, T, kCsrThreads, 0, s, kin, vin, E, N, 8 * pass, (const int32_t*)groups,
                   (const int32_t*)counted, G, kout, vout);
        } else {
            launch(csr_upsweep<kFirst, kItems, true>, T, kCsrThreads, 0, s, kin, E, N, 8 * pass, counted, T);
            launch(csr_downsweep<kFirst, kItems, 1>, T, kCsrThreads, 0, s, kin, vin, E, N, 8 * pass, (const int32_t*)counted, none, T, kout,
                   vout);
        }
    };
    for (int pass = 0; pass < passes; ++pass) {
        int32_t* counted = T == 1 ? hist : passes == 2 ? v[1] : pass == passes - 1 ? v[pass & 1] : perm;
        int32_t *kout = k[pass & 1], *vout = pass == passes - 1 ? perm : v[pass & 1];
        if (pass == 0) pass_of(std::true_type(), 0, dst, none, kout, vout, counted);
        else pass_of(std::false_type(), pass, k[1 - (pass & 1)], v[1 - (pass & 1)], kout, vout, counted);
    }
    return k[(passes - 1) & 1];
}

struct CsrPlan {
    bool counting = false;
    int T = 0;
    int passes = 0;
    int rounds = 0;     // counting path: rounds of 32 edges per warp in a tile
    size_t off_k[2] = {0, 0}, off_v[2] = {0, 0}, off_hist = 0, off_tot = 0, off_rank = 0, bytes = 0;
};

CsrPlan csr_plan(int64_t E, int32_t N) {
    CsrPlan p;
    if (E <= 0) return p;
    const size_t ebytes = align_up((size_t)E * 4, 256);
    size_t off = 0;
    if ((int64_t)N + 1 <= kCntMaxKeys) {
        p.counting = true;
        const int64_t per_tile = (E + kCntTargetTiles - 1) / kCntTargetTiles;
        p.rounds = (int)imax<int64_t>(1, imin<int64_t>(kCntMaxRounds, (per_tile + kCntThreads - 1) / kCntThreads));
        const int64_t ts = (int64_t)p.rounds * kCntThreads;
        p.T = (int)((E + ts - 1) / ts);
        const int nkeys = N + 1;
        p.off_hist = off; off += align_up((size_t)2 * count_pairs(nkeys) * p.T * 4, 256);
        p.off_tot = off; off += align_up((size_t)nkeys * 4, 256);
        p.off_rank = off; off += align_up((size_t)E * 2, 256);
        p.bytes = off;
        return p;
    }
    p.T = (int)((E + kTile - 1) / kTile);
    const uint32_t maxkey = (uint32_t)N;
    const int bits = maxkey == 0 ? 1 : 32 - __builtin_clz(maxkey);
    p.passes = (bits + 7) / 8;
    p.off_k[0] = off; off += ebytes;
    p.off_v[0] = off; off += ebytes;
    p.off_k[1] = off; off += ebytes;
    p.off_v[1] = off; off += ebytes;
    p.off_hist = off; off += align_up((size_t)kRadix * p.T * 4, 256);
    p.off_tot = off; off += align_up((size_t)kRadix * 4, 256);
    p.bytes = off;
    return p;
}

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" size_t zs_build_csr_workspace_bytes(int64_t E, int32_t N) {
    if (E < 0 || N < 0) return 0;
    return csr_plan(E, N).bytes;
}

extern "C" zs_status zs_build_csr(const int32_t* dst, int64_t E, int32_t N,
                                  int32_t* row_ptr, int32_t* perm, int32_t* bad_dst_count,
                                  void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    if (E < 0 || N < 0) return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: negative size (E=%lld, N=%d)", (long long)E, N);
    if (E >= ((int64_t)1 << 31) - 1) return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: E=%lld exceeds the int32 index range", (long long)E);
    if (!row_ptr) return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: row_ptr is NULL");
    if (E > 0 && (!dst || !perm)) return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: dst or perm is NULL with E > 0");
    const CsrPlan p = csr_plan(E, N);
    if (workspace_bytes < p.bytes) return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
    if (p.bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(ZS_ERR_INVALID_ARG, "zs_build_csr: workspace NULL or not 256-byte aligned");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    if (p.counting) {
        static std::atomic<uint64_t> rank_smem_set[kMaxDevices];
        int32_t* M = reinterpret_cast<int32_t*>(ws + p.off_hist);
        int32_t* tot = reinterpret_cast<int32_t*>(ws + p.off_tot);
        uint16_t* rank = reinterpret_cast<uint16_t*>(ws + p.off_rank);
        if (E > kGroupMinEdges && E <= kGroupCtas * kGroupMaxRounds * kCntThreads && N < kGroupMaxKeys) {
            static std::atomic<uint64_t> group_smem_set[kMaxDevices];
            set_smem_limit_once(csr_count_group, count_group_smem(kGroupMaxKeys, kGroupMaxRounds), group_smem_set);
            const int rounds = (int)((E + kGroupCtas * kCntThreads - 1) / (kGroupCtas * kCntThreads));
            launch_clusters(kGroupCtas, csr_count_group, kGroupCtas, kCntThreads, count_group_smem(N + 1, rounds), s, dst, E, N, rounds, perm,
                            row_ptr, bad_dst_count);
            return check_launch("zs_build_csr");
        }
        if (E <= kSingleMaxEdges) {
            static std::atomic<uint64_t> single_smem_set[kMaxDevices];
            set_smem_limit_once(csr_count_single, count_single_smem(kCntMaxKeys, kSingleRounds), single_smem_set);
            const int rounds = (int)((E + kCntThreads - 1) / kCntThreads);
            launch(csr_count_single, 1, kCntThreads, count_single_smem(N + 1, rounds), s, dst, E, N, rounds, perm,
                   row_ptr, bad_dst_count);
            return check_launch("zs_build_csr");
        }
        const int smem = count_rank_smem(kCntMaxKeys, kCntMaxRounds);
        set_smem_limit_once(csr_count_rank, smem, rank_smem_set);
        const int S = 2 * count_pairs(N + 1);
        launch(csr_count_rank, p.T, kCntThreads, count_rank_smem(N + 1, p.rounds), s, dst, E, N, p.rounds, M, rank);
        static std::atomic<uint64_t> scan_smem_set[kMaxDevices];
        set_smem_limit_once(csr_scan_cols, kOneCtaPerSmSmem, scan_smem_set);
        launch(csr_scan_cols, (N + 1 + 31) / 32, kCntThreads, kOneCtaPerSmSmem, s, M, p.T, S, N + 1, tot);
        static std::atomic<uint64_t> scatter_smem_set[kMaxDevices];
        set_smem_limit_once(csr_count_scatter, imax(kOneCtaPerSmSmem, count_scatter_smem(kCntMaxKeys, kCntMaxRounds)), scatter_smem_set);
        launch(csr_count_scatter, p.T, kCntThreads, imax(kOneCtaPerSmSmem, count_scatter_smem(N + 1, p.rounds)), s, dst, (const uint16_t*)rank,
               (const int32_t*)M, (const int32_t*)tot, E, N, p.rounds, perm, row_ptr, bad_dst_count);
        return check_launch("zs_build_csr");
    }
    const int32_t* sorted = nullptr;
    if (E > 0) {
        int32_t* hist = reinterpret_cast<int32_t*>(ws + p.off_hist);
        int32_t* tot = reinterpret_cast<int32_t*>(ws + p.off_tot);
        int32_t* const k[2] = {reinterpret_cast<int32_t*>(ws + p.off_k[0]), reinterpret_cast<int32_t*>(ws + p.off_k[1])};
        int32_t* const v[2] = {reinterpret_cast<int32_t*>(ws + p.off_v[0]), reinterpret_cast<int32_t*>(ws + p.off_v[1])};
        if (p.passes > 1 && E <= (int64_t)kFewTiles * kTile) {
            if (E <= kFewTiles * 256 && p.passes == 2) sorted = sort_few<1>(p.passes, dst, E, N, k, v, perm, hist, s);
            else if (E <= kFewTiles * 512) sorted = sort_few<2>(p.passes, dst, E, N, k, v, perm, hist, s);
            else if (E <= kFewTiles * 1024) sorted = sort_few<4>(p.passes, dst, E, N, k, v, perm, hist, s);
            else sorted = sort_few<8>(p.passes, dst, E, N, k, v, perm, hist, s);
        } else if (p.passes > 1 && E <= (int64_t)kFewTiles * kTileGroup * kTile) {
            // Twice as large tiles where these are from 5/6 to 4/3 of the SMs (keys of 7921, us with 8 a thread against 16: 519000,
            // 127 tiles, 25.4 and 25.6; 560000 26.5 and 26.4; 647170 31.4 and 29.1; 829000, 203 tiles, 33.1 and 30.2; 900000 32.8
            // and 33.9).
            const int64_t tiles = (E + 2 * kTile - 1) / (2 * kTile);
            if (6 * tiles > 5 * num_sms() && 3 * tiles <= 4 * num_sms()) sorted = sort_few<2 * kCsrItems, true>(p.passes, dst, E, N, k, v, perm, hist, s);
            else sorted = sort_few<kCsrItems, true>(p.passes, dst, E, N, k, v, perm, hist, s);
        } else {
            const int32_t* kin = dst;
            const int32_t* vin = nullptr;
            for (int pass = 0; pass < p.passes; ++pass) {
                const bool first = pass == 0, last = pass == p.passes - 1;
                const int shift = 8 * pass;
                int32_t* kout = k[pass & 1];
                int32_t* vout = last ? perm : v[pass & 1];
                if (first) launch(csr_upsweep<true, kCsrItems, false>, p.T, kCsrThreads, 0, s, kin, E, N, shift, hist, p.T);
                else launch(csr_upsweep<false, kCsrItems, false>, p.T, kCsrThreads, 0, s, kin, E, N, shift, hist, p.T);
                launch(csr_scan, kRadix, kCsrThreads, 0, s, hist, p.T, tot);
                if (first) launch(csr_downsweep<true, kCsrItems, 0>, p.T, kCsrThreads, 0, s, kin, vin, E, N, shift, (const int32_t*)hist, (const int32_t*)tot, p.T, kout, vout);
                else launch(csr_downsweep<false, kCsrItems, 0>, p.T, kCsrThreads, 0, s, kin, vin, E, N, shift, (const int32_t*)hist, (const int32_t*)tot, p.T, kout, vout);
                kin = kout;
                vin = vout;
            }
            sorted = kin;
        }
    }
    // From two keys a node on by the keys' positions, else by the nodes (the whole build, positions against nodes: 647170 keys
    // of 7921 30 us and 31, 65536 of 50021 14.4 and 15.2; but 16384 skewed ones of 50021 24 and 13, 173 of 50021 33 and 7).
    if (E >= 2 * (int64_t)N) {
        const int64_t threads = (E + 1 + kRowPtrPer - 1) / kRowPtrPer;
        launch(csr_row_ptr, (unsigned)((threads + 255) / 256), 256, 0, s, sorted, E, N, row_ptr, bad_dst_count);
    } else {
        launch(csr_row_ptr_of_few, (unsigned)(((int64_t)N + kRowPtrNodes) / kRowPtrNodes), kRowPtrNodes, 0, s, sorted, (int32_t)E, N, row_ptr,
               bad_dst_count);
    }
    return check_launch("zs_build_csr");
}
