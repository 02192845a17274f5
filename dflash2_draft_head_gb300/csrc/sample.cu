// Sampling: one token of every logit row, by temperature, top-k, top-p and min-p,
// from a given uniform number.
//
//   w_j = 2^((x_j - max x) * (log2(e) / T))       (fp32; T <= 0: the largest entry alone)
//   W_j = round(w_j * 2^40)                       (a whole number, at most 2^40)
//   in order of falling x (equal values: lowest index first) entry j is kept while
//     fewer than top_k stand before it, the W before it are below
//     top_p * (sum of W over the top_k entries), and w_j >= min_p;
//   the token is the first, in order of index, at which the running sum of the
//   kept W passes floor(u * their sum).
//
// The weights are whole numbers so that their sums are exact in any order: the
// token does not depend on how a row is split.  A weight under 2^-41 of the
// largest one counts as 0: over 2^21 entries that is less than 2^-20 of the sum.
//
// The floor is HBM: a row is read once, by one CTA or by the CTAs of a cluster, and passed
// over two or more times on the chip.  What bounds the kernel is the instructions of
// those passes: exact weights take 7 an entry.  4096 x 151936 bf16 rows at a temperature
// take 298 us (4.2 TB/s), their bytes alone 183 us; 425 us for 512 x 262144 fp32 rows cut
// by top_p inside a flat distribution, which makes three passes and counts every entry.
//
// The largest entries of the row's groups (of 256 or 128) come first: the largest of them
// is the row's, and the n-th largest is a bound above which at least n entries lie.
//   - Neither top_k nor top_p: one pass of weights, summed by warp; one warp's part of
//     the row holds the token and is looked through.
//   - No more entries to keep than groups, or a top_p that the groups' largest entries
//     reach: the entries above such a bound (tens to hundreds) are listed, and one CTA
//     finishes the row from the list alone.
//   - Else counts over the distance from the maximum (with top_p alone taken in the pass
//     that sums all weights) tell which few bins hold the cut, by bounds of the weights in
//     each or, likely, by the weights of the bins' middles.  The next pass takes the exact
//     weight above them and lists their entries; a sorted list that does not hold the cut
//     narrows the bins.  More than 1024 entries in a bin (ties) are told apart by
//     histograms of their exact weights over their values, until the cut lies in one
//     value.  What is kept is summed by warp in the pass that lists, and looked through as
//     in the first case.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "dflash2.h"
#include "rows.cuh"

namespace df2 {
namespace {

using u32 = uint32_t;
using u64 = unsigned long long;

// Three CTAs of eight warps an SM: with two of sixteen the compiler has 64 registers a
// thread instead of 80 (4096 x 151936 bf16, all paths in one kernel: 332 us, 371).  Rows of
// up to kNarrowBytes take CTAs of four warps, of which an SM holds seven: such a row's time
// is the latency of the barriers, not of its bytes (4096 x 1000 bf16, temperature alone: 38
// us, 115 us with sixteen warps; 4096 x 32000, top-k: 97 us, 192).
using Wide = RowGeometry<256, 3, 6, 320>;
using Narrow = RowGeometry<128, 7, 4, 320>;
constexpr long long kNarrowBytes = 64 * 1024;
// Where top_p, or a top_k beyond the groups, may ask for all passes, the instructions bound
// them and a cluster's barriers stand between: slices of up to 640 KB (512 x 262144 fp32,
// top_p: 383 us, 428 with 320 KB).  A temperature or a short list is bound by what misses
// L2 (the same at a temperature: 158 us, 134).
constexpr long long kCutSliceBytes = 640 * 1024;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kOne = 1099511627776.f;  // 2^40, the largest entry's weight
constexpr float kDepth = 41.f;           // entries 2^-kDepth below the largest weigh nothing
constexpr int kDepthBins = 2048;         // of counts, over the depth
constexpr int kBins = 512;               // of counts, or of weights in four words, over keys
constexpr int kLimb = 11;                // bits of a weight in each word: 2^21 of them fit 32 bits
constexpr int kBinsLog = 9;
static_assert(kBins == 1 << kBinsLog && kDepthBins == 4 * kBins);

// An order-preserving whole number of a value (-0 like +0), and back.
template <typename T>
struct Key;
template <>
struct Key<float> {
    static __device__ __forceinline__ u32 of(float x) {
        const u32 b = __float_as_uint(x + 0.f);
        return b ^ ((u32)((int)b >> 31) | 0x80000000u);
    }
    static __device__ __forceinline__ float value(u32 k) {
        return __uint_as_float(k ^ ((u32)(~(int)k >> 31) | 0x80000000u));
    }
};
template <>
struct Key<__nv_bfloat16> {
    static __device__ __forceinline__ u32 of(float x) { return Key<float>::of(x) >> 16; }
    static __device__ __forceinline__ float value(u32 k) {
        return __uint_as_float(__float_as_uint(Key<float>::value(k << 16)) & 0xffff0000u);
    }
};

struct Weigh {
    float m, c;  // the row's largest entry, log2(e) / T
    __device__ __forceinline__ float depth(float x) const {
        return x == m ? 0.f : __fmul_rn(__fsub_rn(x, m), c);
    }
    // w of an entry at that depth; 0 for a NaN
    static __device__ __forceinline__ float w(float d) { return ex2(fmaxf(d, -200.f)); }
    static __device__ __forceinline__ u64 fixed(float w) { return __float2ull_rn(w * kOne); }
};

// The sum of the weights of many entries in two words, a pair of entries at a time:
// adding 12 to w rounds it to whole 2^-20 and leaves their number in the low bits of
// the fp32 value, adding 1.5 * 2^-17 to the (exact) rest does so for 2^-40.  Together
// that is w rounded to whole 2^-40, ties to even.  Good for 4095 entries.
struct WeightSum {
    u32 hi = 0, lo = 0;
    __device__ __forceinline__ void add(f32x2 w) {
        constexpr float kHi = 12.f, kLo = 1.5f / 131072;
        const f32x2 t = add2(w, pair(kHi, kHi));
        const f32x2 rest = fma2(add2(t, pair(-kHi, -kHi)), pair(-1.f, -1.f), w);
        const float2 h = halves(t), l = halves(add2(rest, pair(kLo, kLo)));
        hi += __float_as_uint(h.x) + __float_as_uint(h.y);
        lo += __float_as_uint(l.x) + __float_as_uint(l.y);
    }
    __device__ __forceinline__ u64 total(int entries) const {
        const u32 h = hi - (u32)entries * __float_as_uint(12.f);
        const int l = (int)(lo - (u32)entries * __float_as_uint(1.5f / 131072));
        return ((u64)h << 20) + (u64)(long long)l;
    }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the lanes before this one.
template <typename S>
__device__ __forceinline__ S warp_before(S v) {
    const int lane = threadIdx.x & 31;
    S s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const S t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    return s - v;
}

__device__ __forceinline__ u64 bin_weight(const uint4& b) {
    return (u64)b.x + ((u64)b.y << kLimb) + ((u64)b.z << (2 * kLimb)) + ((u64)b.w << (3 * kLimb));
}

// Where the kept entries end: those with a key above `key`, and the first `ties`
// (in order of index) of those with that key.
struct Cut {
    u32 key, ties;
    u64 weight;  // of one of those ties
};

// "The weight before an entry is below p * total", a comparison in fp64, as one of whole
// numbers: the least one that is not below the product.  One lane of each warp finds it
// (the SM's fp64 units are few).
__device__ __forceinline__ u64 limit_of(float p, u64 total) {
    u64 first = 0;
    if ((threadIdx.x & 31) == 0) {
        const double limit = (double)p * (double)total;
        first = __double2ull_ru(limit);
        if (limit >= 9007199254740992.) {  // 2^53: numbers just below it may round up to it
            u64 low = first - 512;         // spaced at most 2^9 apart below 2^62
            while (first - low > 1) {
                const u64 mid = low + (first - low) / 2;
                if ((double)mid >= limit)
                    first = mid;
                else
                    low = mid;
            }
        }
    }
    return __shfl_sync(0xffffffffu, first, 0);
}

// u * total as a whole number below total (u outside [0, 1): the nearer end).
__device__ __forceinline__ u64 target_of(float u, u64 total) {
    u64 t = 0;
    if ((threadIdx.x & 31) == 0)
        t = min((u64)__double2ull_rz((double)(u > 0.f ? u : 0.f) * (double)total), total - 1);
    return __shfl_sync(0xffffffffu, t, 0);
}

// groups of a row whose maxima are exchanged
template <typename G>
constexpr int kGroups = G::kThreads < 256 ? G::kThreads : 256;
constexpr int kMaxGroups = 256, kMaxWarps = 8;
constexpr int kListMax = 1024;  // entries of a row's list
constexpr int kParts = kRowMaxCluster * kMaxWarps;
constexpr int kMaxUnits = 256;  // of a warp: see the assertion beside the launch

struct Shared {
    union {
        u32 count[kDepthBins];
        uint4 bins[kBins];
        u64 own_list[kListMax];  // this CTA's listed entries
        u64 weight[kListMax];    // the weights of the row's, by place (rank 0)
    };
    union {
        uint4 total[kBins];  // the cluster's bins
        u64 list[kListMax];  // the row's listed entries (rank 0): key, then ~index
    };
    float group_max[kMaxGroups];
    float own_max[kMaxGroups];
    u64 told_n[kRowMaxCluster];  // every CTA's listed entries
    u64 told_w[kRowMaxCluster];  // and their weight
    u64 cta_w[kRowMaxCluster];   // sums over the row
    u64 answer[2];               // a cut's key and ties; the kept weight
    u64 part_w[kParts];          // kept weight of every warp of the row
    u32 part_t[kParts];          // and its ties at the cut
    u64 unit_w[kMaxUnits];       // the same of 32 vectors each of one warp
    u32 unit_t[kMaxUnits];
    u64 cta_span[kRowMaxCluster];  // largest and smallest key of a bracket, by CTA
    u32 own_n, list_n, base;
    float bound;
    u32 span_hi, span_lo;
    u32 scan_n[kMaxWarps];
    u64 scan_w[kMaxWarps];
    u64 scan_w3[3][kMaxWarps];
    // the bins that may hold the cut: what stands before them and with them; for one bin
    // the weights
    int at, at_hi;
    u32 before_n, upto_n;
    u64 before_w, in_w;
    // the bins of the likely cut, what stands before them and with them
    int likely, likely_hi;
    u32 likely_n, likely_upto, likely_at;
    // what find_cut found: the cut and the kept weight, every warp's part of that and its ties
    Cut found;
    u64 found_w;
    u64 found_warp_w[kMaxWarps];
    u32 found_warp_t[kMaxWarps];
};

// The CTA's, from any function (known to lie in shared memory, unlike an argument).
__device__ __forceinline__ Shared& shared_block() {
    __shared__ Shared sh;
    return sh;
}

__device__ __forceinline__ char* ring_block() {
    extern __shared__ __align__(16) char smem[];
    return smem;
}

// This CTA's row.
template <typename T, typename G>
struct Row {
    using Geo = G;
    static constexpr int E = VecOf<T>::kElems;
    int lg, cs, rank;
    RowView<T> r;
    RowSlice<G> sl;

    __device__ __forceinline__ explicit Row(const SampleArgs& a)
        : lg(a.lg), cs(1 << a.lg), rank(a.lg > 0 ? (int)cluster_ctarank() : 0),
          r(a.logits, a.ld, blockIdx.x >> a.lg, a.V),
          sl(r, a.per, a.ring, rank, threadIdx.x >> 5, ring_block(), l2_policy_evict_last()) {}

    template <typename F>
    __device__ __forceinline__ void each_vec(F f) {
        sl.pass(r, [&](int v, const uint4& vec, bool) { f(v, vec); });
    }
    // f(index, entries, their depths), two at a time.  `plain`: no NaN among them, a finite
    // maximum and a factor that is neither 0 nor infinite, so that no product is a NaN; else
    // a NaN has the depth of -inf
    template <typename F>
    __device__ __forceinline__ void each_pair(const Weigh& g, bool plain, F f) {
        const f32x2 nm = pair(-g.m, -g.m), c = pair(g.c, g.c);
        if (plain) {
            each_vec([&](int v, const uint4& vec) {
                f32x2 x[E / 2];
                unpack(vec, x);
#pragma unroll
                for (int j = 0; j < E / 2; ++j)
                    f(v * E - r.head + 2 * j, halves(x[j]), halves(mul2(add2(x[j], nm), c)));
            });
        } else {
            each_vec([&](int v, const uint4& vec) {
                float x[E];
                unpack(vec, x);
#pragma unroll 1
                for (int j = 0; j < E; j += 2)
                    f(v * E - r.head + j, make_float2(x[j], x[j + 1]),
                      make_float2(fmaxf(g.depth(x[j]), -200.f), fmaxf(g.depth(x[j + 1]), -200.f)));
            });
        }
    }
    __device__ __forceinline__ void sync() const {
        if (cs > 1) {
            __syncwarp();
            cluster_sync();
        } else {
            __syncthreads();
        }
    }
};

// Block-wide sums of a count and a weight; every thread gets both.
template <typename G>
__device__ __forceinline__ void block_sum(Shared& sh, u32& n, u64& w) {
    n = __reduce_add_sync(0xffffffffu, n);
    w = warp_sum(w);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sh.scan_n[threadIdx.x >> 5] = n;
        sh.scan_w[threadIdx.x >> 5] = w;
    }
    __syncthreads();
    n = 0;
    w = 0;
    for (int i = 0; i < G::kWarps; ++i) {
        n += sh.scan_n[i];
        w += sh.scan_w[i];
    }
}

// Sums of weights over the whole row; every thread gets them.  Between two calls a
// row.sync() has to stand, behind this one's reads: the next one's stores into the other
// CTAs' cta_w come before its own.
template <typename R>
__device__ __forceinline__ u64 row_weight(Shared& sh, const R& row, u64 w) {
    u32 none = 0;
    block_sum<typename R::Geo>(sh, none, w);
    if (row.cs == 1) return w;
    if ((int)threadIdx.x < row.cs)
        st_cluster_b64(map_cluster(smem_u32(&sh.cta_w[row.rank]), threadIdx.x), w);
    row.sync();
    w = 0;
    for (int i = 0; i < row.cs; ++i) w += sh.cta_w[i];
    return w;
}

// Running sums over the block's threads: what stands before this one.  Returns all.
template <typename G>
__device__ __forceinline__ u64 block_before(Shared& sh, u32& n, u64& w) {
    const u32 bn = warp_before(n);
    const u64 bw = warp_before(w);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) {
        sh.scan_n[threadIdx.x >> 5] = bn + n;
        sh.scan_w[threadIdx.x >> 5] = bw + w;
    }
    __syncthreads();
    n = bn;
    w = bw;
    u64 all = 0;
#pragma unroll
    for (int i = 0; i < G::kWarps; ++i) {
        if (i < (int)threadIdx.x >> 5) {
            n += sh.scan_n[i];
            w += sh.scan_w[i];
        }
        all += sh.scan_w[i];
    }
    return all;
}

// The same of a count and three weights; `all`: the sums of those.
template <typename G>
__device__ __forceinline__ void block_before(Shared& sh, u32& n, u64 (&w)[3], u64 (&all)[3]) {
    const int warp = (int)threadIdx.x >> 5;
    const u32 bn = warp_before(n);
    u64 bw[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) bw[q] = warp_before(w[q]);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) {
        sh.scan_n[warp] = bn + n;
#pragma unroll
        for (int q = 0; q < 3; ++q) sh.scan_w3[q][warp] = bw[q] + w[q];
    }
    __syncthreads();
    n = bn;
    for (int i = 0; i < warp; ++i) n += sh.scan_n[i];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        w[q] = bw[q];
        all[q] = 0;
        for (int i = 0; i < G::kWarps; ++i) {
            if (i == warp) w[q] += all[q];
            all[q] += sh.scan_w3[q][i];
        }
    }
}

// A thread's bins: kBinsOf<G> neighbours of the table.
template <typename G>
constexpr int kBinsOf = kBins / G::kThreads;
template <typename G>
struct Bins {
    uint4 b[kBinsOf<G>];
};

template <typename G>
__device__ __forceinline__ void clear_bins(Shared& sh) {
    for (int i = threadIdx.x; i < kBins; i += G::kThreads) sh.bins[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
}

// Adds up the cluster's bins (each CTA a share of them, which it then tells the others)
// and returns this thread's.  What stood in sh.bins may be overwritten afterwards.
template <typename R>
__device__ __forceinline__ Bins<typename R::Geo> merge_bins(Shared& sh, const R& row) {
    using G = typename R::Geo;
    const int tid = threadIdx.x;
    Bins<G> own;
    if (row.cs == 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBinsOf<G>; ++i) own.b[i] = sh.bins[tid * kBinsOf<G> + i];
        __syncthreads();
        return own;
    }
    const int log = kBinsLog - row.lg, share = 1 << log, first = row.rank * share;
    for (int i = tid; i < share; i += G::kThreads) sh.total[first + i] = make_uint4(0, 0, 0, 0);
    row.sync();  // every CTA's bins are filled
    for (int i = tid; i < kBins; i += G::kThreads) {
        const int mine = first + (i & (share - 1));
        const uint4 b = ld_cluster_v4(map_cluster(smem_u32(&sh.bins[mine]), i >> log));
        u32* sum = reinterpret_cast<u32*>(&sh.total[mine]);
        if (b.x != 0) atomicAdd(sum, b.x);
        if (b.y != 0) atomicAdd(sum + 1, b.y);
        if (b.z != 0) atomicAdd(sum + 2, b.z);
        if (b.w != 0) atomicAdd(sum + 3, b.w);
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += G::kThreads) {
        const int mine = first + (i & (share - 1)), to = i >> log;
        if (to != row.rank)
            st_cluster_v4(map_cluster(smem_u32(&sh.total[mine]), to),
                          *reinterpret_cast<const float4*>(&sh.total[mine]));
    }
    row.sync();
#pragma unroll
    for (int i = 0; i < kBinsOf<G>; ++i) own.b[i] = sh.total[tid * kBinsOf<G> + i];
    return own;
}

// Bins of equal width over the depths from 0 down to `deepest`.
struct DepthBins {
    float deepest, scale;
    __device__ __forceinline__ explicit DepthBins(float deepest)
        : deepest(deepest), scale((kDepthBins - 1) / fmaxf(-deepest, 1.f)) {}

    // The bin of a depth: d in bins, rounded by the addition of 2^23, which leaves it in
    // the low bits.
    static constexpr float kRound = 8388608.f;
    __device__ __forceinline__ u32 of(float d) const {
        return __float_as_uint(__fmaf_rn(d, -scale, kRound)) - __float_as_uint(kRound);
    }
    // Counts a pair of entries where `x`, `y`.
    __device__ __forceinline__ void count(u32* counts, float2 d, bool x, bool y) const {
        const float2 t =
            halves(fma2(pair(d.x, d.y), pair(-scale, -scale), pair(kRound, kRound)));
        if (x) atomicAdd(&counts[__float_as_uint(t.x) - __float_as_uint(kRound)], 1u);
        if (y) atomicAdd(&counts[__float_as_uint(t.y) - __float_as_uint(kRound)], 1u);
    }
    // The depth such that those above it, and no others, lie in bins before `bin`.
    __device__ __forceinline__ float edge(int bin) const {
        if (bin <= 0) return INFINITY;
        if (bin >= kDepthBins) return -INFINITY;
        const u32 near = __float_as_uint((bin - 0.5f) / scale);
        u32 lo = near - 64, hi = near + 64;  // the least number in (lo, hi] in that bin or behind
        while (hi - lo > 1) {
            const u32 mid = (lo + hi) >> 1;
            if (of(-__uint_as_float(mid)) >= (u32)bin)
                hi = mid;
            else
                lo = mid;
        }
        return -__uint_as_float(hi);
    }
};

// The depth below which no entry is before a cut by weight that leaves out `rest`: entries
// of less than an even share of that come behind it (less 1 for their rounding, and 7% for
// that of the depth).
__device__ __forceinline__ float deepest_cut(float rest, int V) {
    const float share = rest / (float)V - 1.f;
    return fmaxf(-kDepth, log2f(fmaxf(share, 0.f)) - 40.1f);
}

// This lane's part of its warp's weight: all entries.
template <typename T, typename G>
__device__ __forceinline__ u64 all_weight(Row<T, G>& row, const Weigh& g, bool plain) {
    WeightSum ws;
    int entries = 0;
    row.each_pair(g, plain, [&](int, float2, float2 d) {
        ws.add(pair(ex2(d.x), ex2(d.y)));
        entries += 2;
    });
    return ws.total(entries);
}

// This lane's part of its warp's kept weight, and its ties at the cut.
template <typename T, typename G>
__device__ __forceinline__ void kept_weight(Row<T, G>& row, const Weigh& g, bool plain,
                                            const Cut& cut, float min_p, u64& weight, u32& ties) {
    const float floor = cut.key != 0 ? Key<T>::value(cut.key) : neg_inf();
    const float least = min_p > 0.f ? min_p : 0.f;
    WeightSum ws;
    int entries = 0;
    u32 t = 0;
    row.each_pair(g, plain, [&](int, float2 x, float2 d) {
        const float wx = ex2(d.x), wy = ex2(d.y);
        const bool kx = wx >= least, ky = wy >= least;
        ws.add(pair(kx && x.x > floor ? wx : 0.f, ky && x.y > floor ? wy : 0.f));
        t += (kx && x.x == floor) + (ky && x.y == floor);
        entries += 2;
    });
    weight = ws.total(entries);
    ties = cut.ties != 0 ? t : 0;
}

// A listed entry: larger ones come first in the order of falling values.
template <typename T>
__device__ __forceinline__ u64 entry_of(float x, int index) {
    return (u64)Key<T>::of(x) << 32 | (u32)~index;
}

// Sorts the row's list of n entries, first ones first.  One CTA.  As many as it has
// threads, up to kCountSort: every entry counts those before it, n^2 steps on all
// threads.  More: a bitonic network over the next power of two, kPer neighbours a
// thread, through shuffles inside a warp and shared memory beyond (436 entries on 512
// threads: 1 us, against 4 us by counting).
constexpr int kCountSort = 128;
template <typename G>
__device__ __forceinline__ void sort_list(Shared& sh, int n) {
    constexpr int kPer = kListMax / G::kThreads;
    const int tid = threadIdx.x;
    if (n <= kCountSort) {
        static_assert(kCountSort <= G::kThreads);
        u64 e = 0;
        int before = 0;
        if (tid < n) {
            e = sh.list[tid];
#pragma unroll 8
            for (int j = 0; j < n; ++j) before += sh.list[j] > e;
        }
        __syncthreads();
        if (tid < n) sh.list[before] = e;
        __syncthreads();
        return;
    }
    const int size = 1 << (32 - __clz(n - 1)), base = tid * kPer;
    const bool live = base < size;
    u64 e[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = base + i < n ? sh.list[base + i] : 0;
    auto save = [&] {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) sh.list[base + i] = e[i];
    };
    for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j >= kPer; j >>= 1) {
            const bool larger = ((base & k) == 0) == ((base & j) == 0);  // which of two stays here
            u64 o[kPer];
            if (j < 32 * kPer) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) o[i] = __shfl_xor_sync(0xffffffffu, e[i], j / kPer);
            } else {
                __syncthreads();
                save();
                __syncthreads();
                if (live) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) o[i] = sh.list[(base ^ j) + i];
                }
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (live && (e[i] < o[i]) == larger) e[i] = o[i];
        }
#pragma unroll
        for (int j = kPer / 2; j > 0; j >>= 1) {
            if (j >= k) continue;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if ((i & j) != 0) continue;
                const bool falling = ((base + i) & k) == 0;
                if ((e[i] < e[i + j]) == falling) {
                    const u64 t = e[i];
                    e[i] = e[i + j];
                    e[i + j] = t;
                }
            }
        }
    }
    __syncthreads();
    save();
    __syncthreads();
}

// Sends this CTA's listed entries to rank 0's list, behind those that got there first.
// The caller's next row.sync() completes it.
template <typename R>
__device__ __forceinline__ void send_list(Shared& sh, const R& row, u32 n) {
    const int tid = threadIdx.x;
    if (row.cs == 1) {
        for (u32 i = tid; i < min(n, (u32)kListMax); i += R::Geo::kThreads)
            sh.list[i] = sh.own_list[i];
        return;
    }
    if (tid == 0)
        sh.base = n <= kListMax ? atom_add_cluster(map_cluster(smem_u32(&sh.list_n), 0), n)
                                : kListMax;
    __syncthreads();
    for (u32 i = tid; i < n && sh.base + i < kListMax; i += R::Geo::kThreads)
        st_cluster_b64(map_cluster(smem_u32(&sh.list[sh.base + i]), 0), sh.own_list[i]);
}

// Finds, from the largest entries down, the depth bins that may hold the cut: sh.at to
// sh.at_hi (one bin by count), with the counts before and up to them; sh.at is
// kDepthBins when there is no cut.  b: this thread's merged counts; the cut is known to
// lie in the bins from `from` to `to`, behind base_n entries; base_w: the weight before
// bin `from` or, with `at_end`, up to and with bin `to`.
// By weight and where those bins have more than kListSure entries: sh.likely to
// sh.likely_hi are the bins within kAside entries of the cut that the weights of the bins'
// middles give (of normal logits in fp32 and bf16 that held the cut in 97 of 100 rows, with
// 200 to 500 entries); sh.likely is kDepthBins when there are too many for a list.
constexpr u32 kListSure = 256;
constexpr u32 kAside = 64;
template <bool BY_COUNT, typename G>
__device__ __forceinline__ void find_bracket(Shared& sh, const DepthBins& depths,
                                             const Bins<G>& bins, int from, int to, u32 base_n,
                                             u64 base_w, bool at_end, u32 k, u64 limit) {
    using i64 = long long;
    constexpr int kPer = 4 * kBinsOf<G>;
    int first = (int)threadIdx.x * kPer;
    auto count = [&](int i) {
        const uint4& b = bins.b[i / 4];
        const u32 n = i % 4 == 0 ? b.x : i % 4 == 1 ? b.y : i % 4 == 2 ? b.z : b.w;
        return first + i < from || first + i > to ? 0 : n;
    };
    // the bounds of the bins' weights, in units of 2^-40 (the roundings of the depth, of 2^x
    // and of the weight are far inside 2^-16 of it and 1), and those of their middles
    const float width = 1.f / depths.scale;
    const float up = ex2(0.5f * width) * (1.f + 1.f / 65536);
    const float down = ex2(-0.5f * width) * (1.f - 1.f / 65536);
    auto bounds = [&](int i, u64 (&b)[3]) {
        const u32 n = count(i);
        const float w = ex2((float)(first + i) * -width) * kOne;
        const u64 l = __float2ull_rd(w * down);
        b[0] = first + i == kDepthBins - 1 || l == 0 ? 0 : n * (l - 1);
        b[1] = n * (__float2ull_ru(w * up) + 1);
        b[2] = n * __float2ull_rn(w);
    };
    u32 before_n = 0;
    u64 sum[3] = {}, all[3] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        before_n += count(i);
        if (!BY_COUNT) {
            u64 b[3];
            bounds(i, b);
#pragma unroll
            for (int q = 0; q < 3; ++q) sum[q] += b[q];
        }
    }
    // by weight: bounds of what stands before a bin, and an estimate of it
    if (BY_COUNT)
        block_before<G>(sh, before_n, sum[0]);
    else
        block_before<G>(sh, before_n, sum, all);
    i64 low = (i64)(sum[0] + base_w), high = (i64)(sum[1] + base_w), mid = (i64)(sum[2] + base_w);
    if (at_end) {
        low = (i64)(base_w - all[1] + sum[1]);
        high = (i64)(base_w - all[0] + sum[0]);
        mid -= (i64)all[2];
    }
    if (threadIdx.x == 0) {
        sh.at = at_end && high >= (i64)limit ? from : kDepthBins;
        sh.at_hi = to;
        sh.before_n = base_n;
        sh.upto_n = 0xffffffffu;
        sh.likely = kDepthBins;
    }
    __syncthreads();
    before_n += base_n;
    u32 bn = before_n;
    asm volatile("" : "+r"(first));  // the bins' weights again, rather than kept in registers
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const u32 n = count(i);
        u64 b[3] = {};
        if (!BY_COUNT) bounds(i, b);
        const i64 l = (i64)b[0], h = (i64)b[1], m = (i64)b[2], want = (i64)limit;
        const i64 to_low = low + (at_end ? h : l), to_high = high + (at_end ? l : h);
        const bool may = BY_COUNT ? bn < k && bn + n >= k : high < want && to_high >= want;
        const bool must = BY_COUNT ? may : low < want && to_low >= want;
        if (may) {
            sh.at = first + i;
            sh.before_n = bn;
        }
        if (must) {
            sh.at_hi = first + i;
            sh.upto_n = bn + n;
        }
        if (!BY_COUNT && mid < want && mid + m >= want && n <= kListMax) {
            sh.likely = sh.likely_hi = first + i;
            sh.likely_n = bn;
            sh.likely_upto = bn + n;
            sh.likely_at = bn + (u32)((float)n * __fdividef((float)(want - mid), (float)m));
        }
        bn += n;
        low = to_low;
        high = to_high;
        mid += m;
    }
    __syncthreads();
    const int bin = sh.likely, at = sh.at, at_hi = sh.at_hi;
    if (BY_COUNT || bin == kDepthBins || at == kDepthBins || sh.upto_n - sh.before_n <= kListSure)
        return;
    // and the bins with the entries next to that place
    const u32 likely_n = sh.likely_n, likely_upto = sh.likely_upto;
    const u32 lo = max(sh.likely_at - min(sh.likely_at, kAside), sh.before_n);
    const u32 hi = min(sh.likely_at + kAside, sh.upto_n - 1);
    const u32 spare = (kListMax - (likely_upto - likely_n)) / 2;
    __syncthreads();
    bn = before_n;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const u32 n = count(i);
        const int here = first + i;
        if (here >= at && here < bin && bn <= lo && lo < bn + n && likely_n - bn <= spare) {
            sh.likely = here;
            sh.likely_n = bn;
        }
        if (here > bin && here <= at_hi && bn <= hi && hi < bn + n &&
            bn + n - likely_upto <= spare) {
            sh.likely_hi = here;
            sh.likely_upto = bn + n;
        }
        bn += n;
    }
    __syncthreads();
}

// The same over the bins of keys: the one bin at which the running count reaches k or the
// running weight `limit`; sh.at is kBins when none does.
template <bool BY_COUNT, typename R>
__device__ __forceinline__ void find_bin(Shared& sh, const R& row, u32 base_n, u64 base_w, u32 k,
                                         u64 limit) {
    using G = typename R::Geo;
    const Bins<G> bins = merge_bins(sh, row);
    if (threadIdx.x == 0) sh.at = kBins;
    u32 bn = 0;
    u64 bw = 0;
#pragma unroll
    for (int i = 0; i < kBinsOf<G>; ++i) {
        bn += BY_COUNT ? bins.b[i].x : 0;
        bw += BY_COUNT ? 0 : bin_weight(bins.b[i]);
    }
    block_before<G>(sh, bn, bw);
    bn += base_n;
    bw += base_w;
#pragma unroll
    for (int i = 0; i < kBinsOf<G>; ++i) {
        const u32 n = BY_COUNT ? bins.b[i].x : 0;
        const u64 w = BY_COUNT ? 0 : bin_weight(bins.b[i]);
        if (BY_COUNT ? bn < k && bn + n >= k : bw < limit && bw + w >= limit) {
            sh.at = (int)threadIdx.x * kBinsOf<G> + i;
            sh.before_n = bn;
            sh.before_w = bw;
            sh.in_w = w;
        }
        bn += n;
        bw += w;
    }
    __syncthreads();
}

// The cut by count (the first k entries) or by weight (those with less than `limit`
// before them), among the entries inside `in`; `in` itself when that cuts nothing.
// `counted`: sh.count has the entries of the depths already.  `weigh`: the kept weight is
// asked for.  The results are left in sh.found and behind it, so that the call needs few
// registers; `in` is an earlier call's sh.found.
struct Flags {
    bool up;      // the direction of the row's next pass
    bool summed;  // the warps' kept weight and ties are known too
};
template <bool BY_COUNT, bool INSIDE, typename T, typename G>
__device__ __noinline__ Flags find_cut(const SampleArgs& a, const Weigh g, bool plain, bool up,
                                       u32 k, u64 limit, float deepest, bool counted,
                                       bool weigh) {
    constexpr int E = VecOf<T>::kElems;
    Shared& sh = shared_block();
    Row<T, G> row(a);
    row.sl.up = up;
    const DepthBins depths(deepest);
    const int tid = threadIdx.x, lane = tid & 31;
    const Cut in = INSIDE ? sh.found : Cut{0, 0, 0};
    auto leave = [&](const Cut& cut, u64 kept_w, bool summed) {
        if (tid == 0) {
            sh.found = cut;
            sh.found_w = kept_w;
        }
        __syncthreads();
        return Flags{row.sl.up, summed};
    };
    const float least = INSIDE ? Key<T>::value(in.key) : neg_inf();
    if (!counted) {
        clear_bins<G>(sh);
        row.each_pair(g, plain, [&](int, float2 x, float2 d) {
            depths.count(sh.count, d, d.x >= depths.deepest && (!INSIDE || x.x >= least),
                         d.y >= depths.deepest && (!INSIDE || x.y >= least));
        });
    }
    const Bins<G> counts = merge_bins(sh, row);
    if (tid == 0) {
        sh.span_hi = 0;
        sh.span_lo = 0xffffffffu;
    }
    // the cut is in the bins from `from` to `to`: behind base_n entries, and the weight w is
    // that before them or, with at_end, up to them
    int from = 0, to = kDepthBins - 1;
    u32 base_n = 0, n = 0;  // n: the entries before the bins that are looked at
    u64 w = 0;
    bool at_end = false;
    float hi_x = neg_inf(), lo_x = INFINITY;
    for (int turn = 0;; ++turn) {
        if (tid == 0) sh.own_n = sh.list_n = 0;
        find_bracket<BY_COUNT, G>(sh, depths, counts, from, to, base_n, w, at_end, k, limit);
        int at = sh.at, at_hi = sh.at_hi;
        n = sh.before_n;
        u32 inside = sh.upto_n - n;
        const bool sure = BY_COUNT || at == kDepthBins || inside <= kListSure || turn == 2 ||
                          sh.likely == kDepthBins;
        const bool listed = at < kDepthBins && (!sure || inside <= kListMax);
        if (!sure) {
            at = sh.likely;
            at_hi = sh.likely_hi;
            n = sh.likely_n;
            inside = sh.likely_upto - n;
        }
        // the weight before them, and their entries or the span of their keys
        const float edge = depths.edge(at), end = depths.edge(at_hi + 1);
        const float low = fmaxf(end, depths.deepest);
        WeightSum sum;
        int entries = 0;
        auto look = [&](int index, float x, float d) {
            if (d > edge || !(d > end) || (INSIDE && !(x >= least))) return;
            if (listed) {
                const u32 place = atomicAdd(&sh.own_n, 1u);  // below `inside`, by the counts
                if (place < kListMax) sh.own_list[place] = entry_of<T>(x, index);
            } else {
                hi_x = fmaxf(hi_x, x);
                lo_x = fminf(lo_x, x);
            }
        };
        // the row's last pass, most often (512 x 262144 fp32, top_p and min_p: 425 us, 432)
        row.sl.hint = l2_policy_evict_first();
        row.each_pair(g, plain, [&](int index, float2 x, float2 d) {
            const float wx = ex2(d.x), wy = ex2(d.y);
            const bool above_x = d.x > edge, above_y = d.y > edge;
            sum.add(pair(above_x && (!INSIDE || x.x >= least) ? wx : 0.f,
                         above_y && (!INSIDE || x.y >= least) ? wy : 0.f));
            entries += 2;
            if ((!above_x && d.x >= low) || (!above_y && d.y >= low)) {  // rare
                if (d.x >= low) look(index, x.x, d.x);
                if (d.y >= low) look(index + 1, x.y, d.y);
            }
        });
        const u64 lane_w = sum.total(entries);
        w = row_weight(sh, row, lane_w);
        if (at == kDepthBins) return leave(in, w, false);
        if (!listed) break;
        at_end = !sure && w >= limit;  // the cut comes before these bins
        if (!at_end) {
            const u32 own = min(sh.own_n, (u32)kListMax);
            send_list(sh, row, own);
            row.sync();
            if (row.rank == 0) {
                // the last kept entry's place in the sorted list; its ties before it are kept
                constexpr int kPer = kListMax / G::kThreads;
                sort_list<G>(sh, (int)inside);
                u64 W[kPer], upto = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const u32 q = (u32)(tid * kPer + i);
                    W[i] = q < inside ? Weigh::fixed(Weigh::w(
                                            g.depth(Key<T>::value((u32)(sh.list[q] >> 32)))))
                                      : 0;
                    upto += W[i];
                }
                u32 none = 0;
                block_before<G>(sh, none, upto);
                upto += w;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const u32 q = (u32)(tid * kPer + i);
                    if (q >= inside) break;
                    const bool last = BY_COUNT ? n + q + 1 == k
                                               : upto < limit && upto + W[i] >= limit;
                    upto += W[i];
                    const bool none_last = !sure && q + 1 == inside && upto < limit;
                    if (!last && !none_last) continue;
                    u64 answer = 0;
                    if (last) {
                        const u32 key = (u32)(sh.list[q] >> 32);
                        u32 ties = 1;
                        while (ties <= q && (u32)(sh.list[q - ties] >> 32) == key) ++ties;
                        answer = (u64)key << 32 | ties;
                    }
                    for (int cta = 0; cta < row.cs; ++cta) {
                        if (row.cs > 1) {
                            const u32 there = map_cluster(smem_u32(sh.answer), cta);
                            st_cluster_b64(there, answer);
                            st_cluster_b64(there + 8, upto);
                        } else {
                            sh.answer[0] = answer;
                            sh.answer[1] = upto;
                        }
                    }
                }
            }
            row.sync();
            Cut out{(u32)(sh.answer[0] >> 32), (u32)sh.answer[0], 0};
            w = sh.answer[1];
            if (sure || out.key != 0) {
                out.weight = Weigh::fixed(Weigh::w(g.depth(Key<T>::value(out.key))));
                if (out.key == in.key) out.ties = min(out.ties, in.ties);
                // this warp's entries of the list
                u64 warp_w = lane_w;
                u32 ties = 0;
                for (u32 i = lane; i < own; i += 32) {
                    const u64 e = sh.own_list[i];
                    const int v = ((int)~(u32)e + row.r.head) / E;
                    if (v < row.sl.wlo || v >= row.sl.whi) continue;
                    const u32 key = (u32)(e >> 32);
                    if (key > out.key)
                        warp_w += Weigh::fixed(Weigh::w(g.depth(Key<T>::value(key))));
                    ties += key == out.key;
                }
                warp_w = warp_sum(warp_w);
                ties = __reduce_add_sync(0xffffffffu, ties);
                if (lane == 0) {
                    sh.found_warp_w[tid >> 5] = warp_w;
                    sh.found_warp_t[tid >> 5] = ties;
                }
                return leave(out, w, true);
            }
        }
        // what was found narrows the bins
        from = at_end ? sh.at : at_hi + 1;
        to = at_end ? at - 1 : sh.at_hi;
        base_n = at_end ? sh.before_n : n + inside;
        if (at_end)
            row.sync();  // of this turn's sums: no list has been sent, whose syncs stand behind them
        else
            __syncthreads();
    }

    u32 hi = __reduce_max_sync(0xffffffffu, hi_x >= lo_x ? Key<T>::of(hi_x) : 0);
    u32 lo = __reduce_min_sync(0xffffffffu, hi_x >= lo_x ? Key<T>::of(lo_x) : 0xffffffffu);
    if (lane == 0) {
        atomicMax(&sh.span_hi, hi);
        atomicMin(&sh.span_lo, lo);
    }
    __syncthreads();
    const u64 span = (u64)sh.span_hi << 32 | sh.span_lo;
    if (row.cs > 1) {
        if (tid < row.cs) st_cluster_b64(map_cluster(smem_u32(&sh.cta_span[row.rank]), tid), span);
    } else if (tid == 0) {
        sh.cta_span[0] = span;
    }
    row.sync();
    hi = 0;
    lo = 0xffffffffu;
    for (int i = 0; i < row.cs; ++i) {
        hi = max(hi, (u32)(sh.cta_span[i] >> 32));
        lo = min(lo, (u32)sh.cta_span[i]);
    }
    u64 in_w = 0;
    bool more = true;
    while (more) {  // each turn leaves at most 1/256 of the span, rounded down
        more = hi != lo;
        const int shift = max(0, 32 - __clz((hi - lo) | 1) - 9);
        const float hi_v = Key<T>::value(hi), lo_v = Key<T>::value(lo);
        clear_bins<G>(sh);
        row.each_pair(g, plain, [&](int, float2 x, float2 d) {
            auto add = [&](float x, float d) {
                if (!(x >= lo_v && x <= hi_v)) return;
                u32* h = reinterpret_cast<u32*>(&sh.bins[(hi - Key<T>::of(x)) >> shift]);
                if (BY_COUNT) {
                    atomicAdd(h, 1u);
                    return;
                }
                const u64 W = Weigh::fixed(Weigh::w(d));
                constexpr u32 kMask = (1u << kLimb) - 1;
                atomicAdd(h, (u32)W & kMask);
                atomicAdd(h + 1, (u32)(W >> kLimb) & kMask);
                atomicAdd(h + 2, (u32)(W >> (2 * kLimb)) & kMask);
                atomicAdd(h + 3, (u32)(W >> (3 * kLimb)));
            };
            add(x.x, d.x);
            add(x.y, d.y);
        });
        find_bin<BY_COUNT>(sh, row, n, w, k, limit);
        if (sh.at == kBins) break;  // not reached: the bracket holds the cut
        n = sh.before_n;
        if (!BY_COUNT) {
            w = sh.before_w;
            in_w = sh.in_w;
        }
        hi -= (u32)sh.at << shift;
        lo = hi - min(hi - lo, (1u << shift) - 1);
        more = more && hi != lo;
    }
    Cut out{hi, 0, Weigh::fixed(Weigh::w(g.depth(Key<T>::value(hi))))};
    if (BY_COUNT) {
        out.ties = k - n;
    } else {  // those of the ties with less than `limit` before them
        const u64 W = max(out.weight, (u64)1);
        out.ties = (u32)min(in_w / W, (limit - w + W - 1) / W);
    }
    if (hi == in.key) out.ties = min(out.ties, in.ties);
    if (BY_COUNT && weigh) {
        u32 none;
        kept_weight(row, g, plain, out, 0.f, w, none);
        w = row_weight(sh, row, w);
    }
    return leave(out, w + out.ties * out.weight, false);
}

// Finishes a row from its list of n entries, which holds the first k (k > 0) or those
// that reach p of the row's weight `all` (k == 0).  One CTA.  What min_p keeps are the first
// of the sorted entries, as 2^x does not rise with the depth (its instruction was compared
// at every two neighbouring fp32 depths down to 42).
template <typename T, typename G>
__device__ __noinline__ void finish_list(const SampleArgs& a, const Weigh g, int rowi,
                                         int n, int k, float p, float min_p, u64 all) {
    constexpr int kPer = kListMax / G::kThreads;
    Shared& sh = shared_block();
    const int tid = threadIdx.x;
    sort_list<G>(sh, n);
    const int last = k > 0 ? min(k, n) : n;
    u64 W[kPer], before = 0;
    float w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        w[i] = at < last ? Weigh::w(g.depth(Key<T>::value((u32)(sh.list[at] >> 32)))) : 0.f;
        W[i] = Weigh::fixed(w[i]);
        sh.weight[at] = W[i];
        before += W[i];
    }
    u32 kept = 0;
    u64 kept_w = block_before<G>(sh, kept, before);
    const u64 limit = p < 1.f ? limit_of(p, k > 0 ? kept_w : all) : ~0ull;
    kept_w = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        if (at == 0 || (at < last && before < limit && !(w[i] < min_p))) {
            ++kept;
            kept_w += W[i];
        }
        before += W[i];
    }
    block_sum<G>(sh, kept, kept_w);
    const u64 target = target_of(a.uniform[rowi], kept_w);
    for (int i = tid; i < (int)kept; i += G::kThreads) {
        const u32 index = (u32)sh.list[i];  // ~index
        u64 cum = 0;
#pragma unroll 4
        for (int j = 0; j < (int)kept; ++j)
            if ((u32)sh.list[j] > index) cum += sh.weight[j];
        if (cum <= target && target < cum + sh.weight[i]) {
            a.tokens[rowi] = (int)~index;
            if (a.probs != nullptr) a.probs[rowi] = (float)((double)sh.weight[i] / (double)kept_w);
        }
    }
}

// The n-th largest of the row's group maxima, rounded down to the upper 16 bits of its
// key: at least n entries are not below it.  One warp.
template <typename G>
__device__ __forceinline__ float group_bound(const Shared& sh, int n) {
    constexpr int kPer = kGroups<G> / 32;
    const int lane = threadIdx.x & 31;
    u32 key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = Key<float>::of(sh.group_max[lane + 32 * i]) >> 16;
    u32 lo = key[0], hi = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) {
        lo = min(lo, key[i]);
        hi = max(hi, key[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);  // all keys reach it
    hi = __reduce_max_sync(0xffffffffu, hi);
    while (lo < hi) {  // the largest value that n keys reach
        const u32 mid = (lo + hi + 1) >> 1;
        u32 count = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += key[i] >= mid;
        if (__reduce_add_sync(0xffffffffu, count) >= (u32)n)
            lo = mid;
        else
            hi = mid - 1;
    }
    return Key<float>::value(lo << 16);
}

// Chooses the token among the entries inside the cut that min_p keeps.  `summed`: the
// warps' kept weight (without min_p) and their ties are left behind sh.found.
template <bool CUT, typename T, typename G>
__device__ __forceinline__ void choose(const SampleArgs& a, Row<T, G>& row, const Weigh& g,
                                       bool plain, const Cut cut, bool summed, float min_p) {
    constexpr int E = VecOf<T>::kElems;
    Shared& sh = shared_block();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const RowView<T>& r = row.r;
    const int cs = row.cs, rank = row.rank, rowi = blockIdx.x >> a.lg;
    const float uniform = a.uniform[rowi];

    // every warp's kept weight and its ties at the cut
    const bool everything = cut.key == 0 && !(min_p > 0.f);
    const float floor = cut.key != 0 ? Key<T>::value(cut.key) : neg_inf();
    const float least = min_p > 0.f ? min_p : 0.f;
    auto kept_of = [&](const uint4& vec, u64& w, u32& ties) {
        if (plain) {
            f32x2 x[E / 2];
            unpack(vec, x);
            const f32x2 nm = pair(-g.m, -g.m), c = pair(g.c, g.c);
            WeightSum ws;
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 h = halves(x[j]), d = halves(mul2(add2(x[j], nm), c));
                const float wx = ex2(d.x), wy = ex2(d.y);
                const bool kx = wx >= least, ky = wy >= least;
                ws.add(pair(kx && h.x > floor ? wx : 0.f, ky && h.y > floor ? wy : 0.f));
                ties += (kx && h.x == floor) + (ky && h.y == floor);
            }
            w += ws.total(E);
            return;
        }
        float x[E];
        unpack(vec, x);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const u32 key = Key<T>::of(x[j]);
            const float wj = Weigh::w(g.depth(x[j]));
            if (key < cut.key || wj < min_p) continue;
            if (key > cut.key)
                w += Weigh::fixed(wj);
            else
                ++ties;
        }
    };
    u64 sw = 0;
    u32 st = 0;
    // (the weights above the cut's are not below it by more than the rounding of 2^x)
    if (CUT && summed && Weigh::w(g.depth(floor)) >= min_p * (1.f + 1.f / 1048576)) {
        sw = sh.found_warp_w[warp];
        st = sh.found_warp_t[warp];
    } else {
        if (everything)
            sw = all_weight(row, g, plain);
        else
            kept_weight(row, g, plain, cut, min_p, sw, st);
        sw = warp_sum(sw);
        st = __reduce_add_sync(0xffffffffu, st);
    }
    const int me = rank * G::kWarps + warp;
    if (cs > 1) {
        if (lane < cs) {
            st_cluster_b64(map_cluster(smem_u32(&sh.part_w[me]), lane), sw);
            st_cluster_f32(map_cluster(smem_u32(&sh.part_t[me]), lane), __uint_as_float(st));
        }
    } else if (lane == 0) {
        sh.part_w[me] = sw;
        sh.part_t[me] = st;
    }
    row.sync();  // no CTA's shared memory is touched from outside after this

    // The part of the row that holds the token: of the warps' parts, then, by the warps of
    // that CTA, of their 32 vectors at a time, then of a warp's lanes and their entries.
    auto ties_weight = [&](u32 before, u32 n) {
        return cut.ties == 0
                   ? 0
                   : (u64)(min(cut.ties, before + n) - min(cut.ties, before)) * cut.weight;
    };
    struct Place {  // the parts of a lane, [lo, hi), and what stands before them
        int lo, hi;
        u64 sum, own;
        u32 ties;
    };
    auto scan = [&](const u64* w, const u32* t, int n, u64 sum, u32 ties) {
        const int per = (n + 31) >> 5;
        Place q;
        q.lo = min(lane * per, n);
        q.hi = min(q.lo + per, n);
        u32 own_t = 0;
        if (cut.ties != 0)
            for (int i = q.lo; i < q.hi; ++i) own_t += t[i];
        q.ties = ties + (cut.ties != 0 ? warp_before(own_t) : 0);
        q.own = 0;
        u32 tie = q.ties;
        for (int i = q.lo; i < q.hi; ++i) {
            q.own += w[i] + ties_weight(tie, t[i]);
            tie += t[i];
        }
        q.sum = sum + warp_before(q.own);
        return q;
    };
    // the part that holds `target`, for every lane; q: what stands before it
    auto pick = [&](const u64* w, const u32* t, Place& q, u64 target) {
        const int from =
            __ffs(__ballot_sync(0xffffffffu, q.sum <= target && target < q.sum + q.own)) - 1;
        int i = q.lo;
        for (; i < q.hi - 1; ++i) {
            const u64 one = w[i] + ties_weight(q.ties, t[i]);
            if (target < q.sum + one) break;
            q.sum += one;
            q.ties += t[i];
        }
        q.sum = __shfl_sync(0xffffffffu, q.sum, from);
        q.ties = __shfl_sync(0xffffffffu, q.ties, from);
        return __shfl_sync(0xffffffffu, i, from);
    };
    Place q = scan(sh.part_w, sh.part_t, cs * G::kWarps, 0, 0);
    const u64 total = __shfl_sync(0xffffffffu, q.sum + q.own, 31);
    const u64 target = target_of(uniform, total);
    const int holder = pick(sh.part_w, sh.part_t, q, target);
    if (holder / G::kWarps != rank) return;

    const RowSlice<G> own(r, a.per, a.ring, rank, holder % G::kWarps, ring_block(), 0);
    const int units = (own.whi - own.wlo + 31) >> 5;
    constexpr int kAhead = 3;  // units of a warp loaded together
    for (int u0 = warp; u0 < units; u0 += kAhead * G::kWarps) {
        uint4 vec[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = own.wlo + (u0 + i * G::kWarps) * 32 + lane;
            vec[i] = v < own.whi ? r.load(v) : r.nothing();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int unit = u0 + i * G::kWarps;
            if (unit >= units) break;
            u64 w = 0;
            u32 t = 0;
            kept_of(vec[i], w, t);
            w = warp_sum(w);
            t = __reduce_add_sync(0xffffffffu, t);
            if (lane == 0) {
                sh.unit_w[unit] = w;
                sh.unit_t[unit] = t;
            }
        }
    }
    __syncthreads();
    if (warp > 0) return;
    q = scan(sh.unit_w, sh.unit_t, units, q.sum, q.ties);
    const int v = own.wlo + pick(sh.unit_w, sh.unit_t, q, target) * 32 + lane;
    const uint4 vec = v < own.whi ? r.load(v) : r.nothing();
    u64 lw = 0;
    u32 lt = 0;
    kept_of(vec, lw, lt);
    u32 tie = q.ties + (cut.ties != 0 ? warp_before(lt) : 0);
    lw += ties_weight(tie, lt);
    u64 at = q.sum + warp_before(lw);
    if (at > target || target >= at + lw) return;
    float x[E];
    unpack(vec, x);
    int token = -1;
    u64 tw = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const u32 key = Key<T>::of(x[j]);
        const float wj = Weigh::w(g.depth(x[j]));
        u64 w = Weigh::fixed(wj);
        if (key < cut.key || wj < min_p) {
            w = 0;
        } else if (key == cut.key) {
            w = ties_weight(tie, 1);
            ++tie;
        }
        at += w;
        if (token < 0 && target < at) {
            token = v * E + j - r.head;
            tw = w;
        }
    }
    a.tokens[rowi] = token;
    if (a.probs != nullptr) a.probs[rowi] = (float)((double)tw / (double)total);
}

// Finds the cut by top_k, then that by top_p among what it keeps, and chooses.  all, limit:
// the row's weight and top_p's part of it, where there is no top_k.  A call of its own, the
// kernel's last: inside it its registers cost the passes before it (2048 x 151936 bf16,
// top_k 20: 149 us, 176).
template <typename T, typename G>
__device__ __noinline__ void choose_cut(const SampleArgs& a, const Weigh g, bool plain, bool up,
                                        int k, float p, float min_p, u64 all, u64 limit,
                                        float deepest, bool counted) {
    Shared& sh = shared_block();
    Flags f{up, false};
    const bool cuts = k > 0 || p < 1.f;
    if (k > 0) {
        f = find_cut<true, false, T, G>(a, g, plain, f.up, (u32)k, 0, -kDepth, false, p < 1.f);
        if (p < 1.f) {
            all = sh.found_w;
            limit = limit_of(p, all);
        }
    }
    if (p < 1.f) {
        if (!counted) deepest = deepest_cut((float)(all - min(all, limit)), a.V);
        if (k > 0 && sh.found.key != 0)
            f = find_cut<false, true, T, G>(a, g, plain, f.up, 0, limit, deepest, false, true);
        else
            f = find_cut<false, false, T, G>(a, g, plain, f.up, 0, limit, deepest, counted,
                                             true);
    }
    Row<T, G> row(a);
    row.sl.up = f.up;
    choose<true>(a, row, g, plain, cuts ? sh.found : Cut{0, 0, 0}, f.summed, min_p);
}

// CUTS: top_k or top_p may be set, or the largest entry may be all that is kept.  Without
// that code a temperature alone has more registers (4096 x 151936 bf16: 300 us, 360).
template <typename T, typename G, bool CUTS>
__global__ void __launch_bounds__(G::kThreads, G::kCtas)
    sample_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int E = VecOf<T>::kElems;
    Shared& sh = shared_block();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Row<T, G> row(a);
    const RowView<T>& r = row.r;
    const RowSlice<G>& sl = row.sl;
    const int cs = row.cs, rank = row.rank, rowi = blockIdx.x >> a.lg;
    if (cs > 1) cluster_arrive();  // met by cluster_wait below: every CTA has started
    row.sl.start(r);
    float T0 = a.temperature != nullptr ? a.temperature[rowi] : a.temperature0;
    int k = a.top_k != nullptr ? a.top_k[rowi] : a.top_k0;
    const float p = a.top_p != nullptr ? a.top_p[rowi] : a.top_p0;
    float min_p = a.min_p != nullptr ? a.min_p[rowi] : a.min_p0;
    if (!(T0 > 0.f)) T0 = 0.f;
    if (k < 0 || k >= a.V) k = 0;
    if (T0 == 0.f || p <= 0.f || min_p > 1.f) k = 1;  // the first entry is always kept
    if (k == 1) min_p = 0.f;
    if (tid == 0) sh.own_n = sh.list_n = 0;

    // the largest entries of the groups (kLanes * cs lanes each) and of the row
    constexpr int kLanes = G::kThreads / kGroups<G>;
    static_assert(kLanes >= 1 && kLanes * kRowMaxCluster <= 32);
    RunningMax<T> most;
    row.each_vec([&](int, const uint4& v) { most.add(v); });
    float m = most.value();
    const bool has_nan = __any_sync(0xffffffffu, m != m);
    if (has_nan) {
        m = neg_inf();
        row.each_vec([&](int, const uint4& v) { m = fmaxf(m, vec_max<T>(v)); });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, m, o);
        if (o < kLanes << a.lg) m = fmaxf(m, other);
    }
    if ((tid & ((kLanes << a.lg) - 1)) == 0)
        (cs > 1 ? sh.own_max : sh.group_max)[tid / kLanes >> a.lg] = m;
    __syncthreads();
    if (cs > 1) {
        cluster_wait();
        // kGroups / 4 of the threads send four maxima each to one of the CTAs
        constexpr int kLog = kGroups<G> == 256 ? 6 : 5;
        static_assert(kGroups<G> / 4 == 1 << kLog);
        const int lq = kLog - a.lg, quads = 1 << lq, to = tid >> lq, i = tid & (quads - 1);
        if (to < cs)
            st_cluster_v4(map_cluster(smem_u32(&sh.group_max[4 * (rank * quads + i)]), to),
                          reinterpret_cast<const float4*>(sh.own_max)[i]);
        row.sync();
    }
    m = neg_inf();
    for (int i = lane; i < kGroups<G>; i += 32) m = fmaxf(m, sh.group_max[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == neg_inf()) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            a.tokens[rowi] = -1;
            if (a.probs != nullptr) a.probs[rowi] = 0.f;
        }
        return;
    }
    // c is +inf below T = 4.3e-39, and 0 at T = +inf: there 0 stands for a finite maximum, so
    // that no x - m leaves fp32's range and all finite entries have the depth 0
    const float c = __fdiv_rn(kLog2e, T0 > 0.f ? T0 : 1.f);
    const Weigh g{c == 0.f && m < INFINITY ? 0.f : m, c};
    const bool plain = !has_nan && m < INFINITY && g.c > 0.f && g.c < INFINITY;

    u64 all = 0, limit = ~0ull;  // (without top_k) the row's weight and top_p's part of it
    float deepest = -kDepth;     // of the counts
    bool counted = false;
    if (CUTS && (k > 0 || p < 1.f)) {
        // Is a list short enough?  Without top_k: of about as many entries as half the
        // groups, unless the groups' maxima are far from what top_p asks for.  Where it is
        // not, all entries of a row of up to kListMax.
        const int want = k > 0 ? k : kGroups<G> / 2;
        const bool small = a.V <= kListMax;
        bool list = want <= kGroups<G>;
        if (k == 0) {
            clear_bins<G>(sh);
            u64 most = tid < kGroups<G> ? Weigh::fixed(Weigh::w(g.depth(sh.group_max[tid]))) : 0;
            u32 none = 0;
            block_sum<G>(sh, none, most);
            // (a part of the weight, whose rest is not above the row's)
            deepest = deepest_cut((1.f - p) * 0.999f * (float)most, a.V);
            const DepthBins depths(deepest);
            WeightSum ws;
            int entries = 0;
            row.each_pair(g, plain, [&](int, float2, float2 d) {
                ws.add(pair(ex2(d.x), ex2(d.y)));
                entries += 2;
                depths.count(sh.count, d, d.x >= deepest, d.y >= deepest);
            });
            all = row_weight(sh, row, ws.total(entries));
            limit = limit_of(p, all);
            list = most >= limit;
        }
        counted = k == 0;
        if (list || small) {
            counted = false;
            if (warp == 0) {
                const float b = list ? group_bound<G>(sh, want) : neg_inf();
                if (lane == 0) sh.bound = b > -3.402823466e38f ? b : -3.402823466e38f;
            }
            __syncthreads();
            const float bound = sh.bound;
            u64 listed_w = 0;
            row.each_vec([&](int v, const uint4& vec) {
                if (!(vec_max<T>(vec) >= bound)) return;
                float x[E];
                unpack(vec, x);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (!(x[j] >= bound)) continue;
                    const u32 at = atomicAdd(&sh.own_n, 1u);
                    if (at < kListMax) sh.own_list[at] = entry_of<T>(x[j], v * E + j - r.head);
                    if (k == 0) listed_w += Weigh::fixed(Weigh::w(g.depth(x[j])));
                }
            });
            u32 none = 0;
            if (k == 0) block_sum<G>(sh, none, listed_w);
            __syncthreads();
            const u32 own = sh.own_n;
            send_list(sh, row, own);
            if (cs > 1) {
                if (tid < cs) {
                    st_cluster_b64(map_cluster(smem_u32(&sh.told_n[rank]), tid), own);
                    st_cluster_b64(map_cluster(smem_u32(&sh.told_w[rank]), tid), listed_w);
                }
            } else if (tid == 0) {
                sh.told_n[0] = own;
                sh.told_w[0] = listed_w;
            }
            row.sync();
            u64 n = 0;
            listed_w = 0;
            for (int i = 0; i < cs; ++i) {
                n += sh.told_n[i];
                listed_w += sh.told_w[i];
            }
            if (n <= kListMax && (k > 0 || listed_w >= limit)) {
                // the other CTAs' shared memory is not touched any more
                if (rank == 0) finish_list<T, G>(a, g, rowi, (int)n, k, p, min_p, all);
                return;
            }
            __syncthreads();
        }
    }
    if (CUTS)
        choose_cut<T, G>(a, g, plain, row.sl.up, k, p, min_p, all, limit, deepest, counted);
    else
        choose<false>(a, row, g, plain, Cut{0, 0, 0}, false, min_p);
}

template <typename T, typename G>
cudaError_t launch_typed(SampleArgs a, cudaStream_t stream, int num_sms) {
    // the widest row: kSampleMaxV fp32 entries over the largest cluster
    static_assert(kSampleMaxV / 4 / kRowMaxCluster / Wide::kWarps / 32 < kMaxUnits);
    static_assert(kNarrowBytes / 16 / Narrow::kWarps / 32 < kMaxUnits);
    static_assert(kCutSliceBytes / 16 / Wide::kWarps / 32 < kMaxUnits);
    const bool top_k = a.top_k0 > 0 && a.top_k0 < a.V;
    const bool passes = a.top_k != nullptr || (top_k ? a.top_k0 > kGroups<G>
                                                     : a.top_p != nullptr || a.top_p0 < 1.f);
    const RowSplit p = split_rows<G>(a.rows, a.V, sizeof(T), num_sms,
                                     passes ? kCutSliceBytes : G::kSliceBytes);
    a.lg = p.lg;
    a.per = p.per;
    a.ring = p.ring;
    const bool cuts = passes || top_k || a.temperature != nullptr || !(a.temperature0 > 0.f) ||
                      a.min_p != nullptr || a.min_p0 > 1.f;
    return cuts ? launch_rows<G, sample_kernel<T, G, true>>(a, a.rows, a.lg, p.smem,
                                                            G::kRingBytes, stream)
                : launch_rows<G, sample_kernel<T, G, false>>(a, a.rows, a.lg, p.smem,
                                                             G::kRingBytes, stream);
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, int bf16, cudaStream_t stream, int num_sms) {
    const bool narrow = (long long)a.V * (bf16 ? 2 : 4) <= kNarrowBytes;
    if (bf16)
        return narrow ? launch_typed<__nv_bfloat16, Narrow>(a, stream, num_sms)
                      : launch_typed<__nv_bfloat16, Wide>(a, stream, num_sms);
    return narrow ? launch_typed<float, Narrow>(a, stream, num_sms)
                  : launch_typed<float, Wide>(a, stream, num_sms);
}

}  // namespace df2
