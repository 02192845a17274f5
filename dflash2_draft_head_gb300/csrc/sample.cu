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
// Bound by HBM: a row is read once.  It is split over the CTAs of a cluster, each
// holding its slice in shared memory for the passes over it.  The largest entries of
// 256 groups of the row come first: their maximum is the row's, and the n-th largest
// of them is a bound above which at least n entries lie.
//   - Neither top_k nor top_p: one pass of weights, summed by warp; one warp of the
//     row holds the token and looks it up.
//   - Up to 256 entries to keep, or a top_p that the entries above such a bound
//     reach: those entries (some hundreds) are listed, and one CTA finishes the row
//     from the list alone.
//   - Else the cut is found by histograms of the entries' weights (or counts), first
//     over their distance from the maximum, then over the values of the bin in which
//     the cut lies, until that is one value; ties there are kept by index.  The
//     weights of what is kept are then summed and looked up as in the first case.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "dflash2.h"
#include "rows.cuh"

namespace df2 {
namespace {

using u32 = uint32_t;
using u64 = unsigned long long;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kOne = 1099511627776.f;  // 2^40, the largest entry's weight
constexpr float kDepth = 41.f;           // entries 2^-kDepth below the largest weigh nothing
constexpr int kBins = 512;
constexpr int kLimb = 14;                // a weight in three words of a histogram: 14, 14, 13 bits

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
    return (u64)b.y + ((u64)b.z << kLimb) + ((u64)b.w << (2 * kLimb));
}

// Where the kept entries end: those with a key above `key`, and the first `ties`
// (in order of index) of those with that key.
struct Cut {
    u32 key, ties;
    u64 weight;  // of one of those ties
};

// How many of n equal entries of weight W, behind a sum of `before`, are kept:
// those with less than `limit` before them.
__device__ __forceinline__ u32 ties_below(u64 before, u64 W, u32 n, double limit) {
    u32 lo = 0, hi = n;  // the first i in [0, n) at which before + i * W reaches the limit
    while (lo < hi) {
        const u32 mid = (lo + hi) >> 1;
        if ((double)(before + (u64)mid * W) < limit)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

constexpr int kGroups = kRowThreads;  // groups of a row whose maxima are exchanged
constexpr int kListMax = 1024;        // entries of a row's list
constexpr int kParts = kRowMaxCluster * kRowWarps;

// What a CTA tells the others of its slice: listed entries, their weight, all weight.
struct Told {
    u64 listed, weight, all;
};

struct Shared {
    union {
        uint4 hist[kBins];       // count and the three words of the weight
        u64 own_list[kListMax];  // this CTA's listed entries
        u64 sorted[kListMax];    // the row's, in order (rank 0)
    };
    u64 list[kListMax];          // the row's listed entries (rank 0): key, then ~index
    float group_max[kGroups];
    float own_max[kGroups];
    Told told[kRowMaxCluster];
    u32 own_n, list_n, base;
    float bound;
    u64 part_w[kParts];          // kept weight of every warp of the row
    u64 part_t[kParts];          // and its ties at the cut
    u64 cta_span[kRowMaxCluster];  // largest and smallest key of a bin, by CTA
    u32 span_hi, span_lo;
    u32 scan_n[kRowWarps];
    u64 scan_w[kRowWarps];
    // the bin in which the cut lies, what stands before it and what it holds
    int at;
    u32 before_n;
    u64 before_w, in_w;
    u64 total_w;
};

template <typename T, bool STAGED>
struct Row {
    static constexpr int E = VecOf<T>::kElems;
    RowView<T> r;
    RowSlice sl;
    const uint4* staged;
    int cs, rank;

    __device__ __forceinline__ uint4 vec(int v) const { return STAGED ? staged[v] : r.load(v); }
    // f(vector's number, vector) for this lane's vectors
    template <typename F>
    __device__ __forceinline__ void each_vec(F f) const {
#pragma unroll 2
        for (int v = sl.wlo + (int)(threadIdx.x & 31); v < sl.whi; v += 32) f(v, vec(v));
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        for (int v = sl.wlo + (int)(threadIdx.x & 31); v < sl.whi; v += 32) {
            float x[E];
            unpack(vec(v), x);
#pragma unroll
            for (int j = 0; j < E; ++j) f(x[j]);
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

// Adds up the cluster's histograms and finds, from the largest entries down, the
// first bin at which the running count reaches k (BY_COUNT) or the running weight
// `limit`; sh.at is kBins when none does.  Leaves sh.before_*, in_n and total_w.
template <bool BY_COUNT, typename R>
__device__ void find_bin(Shared& sh, const R& row, u32 base_n, u64 base_w, u32 k, double p,
                         double limit, bool first_level) {
    constexpr int kPer = kBins / kRowThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    row.sync();  // every histogram is filled
    u32 n[kPer] = {};
    u64 w[kPer] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        for (int q = 0; q < row.cs; ++q) {
            const uint4 b = row.cs > 1
                                ? ld_cluster_v4(map_cluster(smem_u32(&sh.hist[tid * kPer + i]), q))
                                : sh.hist[tid * kPer + i];
            n[i] += b.x;
            w[i] += bin_weight(b);
        }
    }
    u32 tn = 0;
    u64 tw = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        tn += n[i];
        tw += w[i];
    }
    u32 bn = warp_before(tn);
    u64 bw = warp_before(tw);
    if (lane == 31) {
        sh.scan_n[warp] = bn + tn;
        sh.scan_w[warp] = bw + tw;
    }
    if (tid == 0) sh.at = kBins;
    row.sync();  // every histogram is read
    bn += base_n;
    bw += base_w;
    u64 total = base_w;
    for (int i = 0; i < kRowWarps; ++i) {
        if (i < warp) {
            bn += sh.scan_n[i];
            bw += sh.scan_w[i];
        }
        total += sh.scan_w[i];
    }
    if (!BY_COUNT && first_level && limit < 0) limit = p * (double)total;
    if (tid == 0) sh.total_w = total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool open = BY_COUNT ? bn < k : (double)bw < limit;
        const bool shut = BY_COUNT ? bn + n[i] >= k : (double)(bw + w[i]) >= limit;
        if (open && shut) {  // one bin of the row
            sh.at = tid * kPer + i;
            sh.before_n = bn;
            sh.before_w = bw;
            sh.in_w = w[i];
        }
        bn += n[i];
        bw += w[i];
    }
    __syncthreads();
}

// The cut by count (the first k entries) or by weight (those with less than
// p * total before them; total < 0: the row's own sum), among the entries inside
// `in`.  Returns false when nothing is cut.  *kept_w: the kept entries' weight (by
// count: where `weigh` asks for it).
template <bool BY_COUNT, typename T, bool STAGED>
__device__ bool find_cut(Shared& sh, const Row<T, STAGED>& row, const Weigh& g, const Cut& in,
                         u32 k, double p, double total, bool weigh, Cut* out, u64* kept_w) {
    const int tid = threadIdx.x, lane = tid & 31;
    auto clear = [&] {
        for (int i = tid; i < kBins; i += kRowThreads) sh.hist[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) {
            sh.span_hi = 0;
            sh.span_lo = 0xffffffffu;
        }
        __syncthreads();
    };
    auto add = [&](int b, u64 W) {
        u32* h = reinterpret_cast<u32*>(&sh.hist[b]);
        if (BY_COUNT) atomicAdd(h, 1u);
        if (BY_COUNT && !weigh) return;
        atomicAdd(h + 1, (u32)W & ((1u << kLimb) - 1));
        atomicAdd(h + 2, (u32)(W >> kLimb) & ((1u << kLimb) - 1));
        atomicAdd(h + 3, (u32)(W >> (2 * kLimb)));
    };
    auto bin_of = [&](float d) { return min(kBins - 1, (int)(d * -(kBins / kDepth))); };
    clear();
    row.each([&](float x) {
        const float d = g.depth(x);
        const u64 W = Weigh::fixed(Weigh::w(d));
        if (W != 0 && Key<T>::of(x) >= in.key) add(bin_of(d), W);
    });
    const double limit0 = total < 0 ? -1.0 : p * total;
    find_bin<BY_COUNT>(sh, row, 0, 0, k, p, limit0, true);
    *kept_w = sh.total_w;
    const double limit = total < 0 ? p * (double)sh.total_w : limit0;
    const int at = sh.at;
    if (at == kBins) return false;

    // the span of that bin's keys
    u32 hi = 0, lo = 0xffffffffu;
    row.each([&](float x) {
        const float d = g.depth(x);
        const u32 key = Key<T>::of(x);
        if (Weigh::fixed(Weigh::w(d)) != 0 && key >= in.key && bin_of(d) == at) {
            hi = max(hi, key);
            lo = min(lo, key);
        }
    });
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
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
    u32 n = sh.before_n;
    u64 w = sh.before_w;
    u64 in_w = sh.in_w;
    while (hi != lo) {  // each turn leaves at most 1/256 of the span, rounded down
        const int shift = max(0, 32 - __clz(hi - lo) - 9);
        __syncthreads();
        clear();
        row.each([&](float x) {
            const u32 key = Key<T>::of(x);
            if (key >= lo && key <= hi && x == x)
                add((hi - key) >> shift, Weigh::fixed(Weigh::w(g.depth(x))));
        });
        find_bin<BY_COUNT>(sh, row, n, w, k, p, limit, false);
        if (sh.at == kBins) break;  // not reached: the bin above holds the cut
        n = sh.before_n;
        w = sh.before_w;
        in_w = sh.in_w;
        hi -= (u32)sh.at << shift;
        lo = hi - min(hi - lo, (1u << shift) - 1);
    }
    out->key = hi;
    out->weight = Weigh::fixed(Weigh::w(g.depth(Key<T>::value(hi))));
    out->ties = BY_COUNT ? k - n : ties_below(w, out->weight, (u32)(in_w / out->weight), limit);
    if (hi == in.key) out->ties = min(out->ties, in.ties);
    *kept_w = w + out->ties * out->weight;
    __syncthreads();
    return true;
}

// This lane's part of its warp's kept weight: all entries (no cut, no min_p), two at a
// time.  `plain`: no NaN among them and a finite maximum.
template <typename T, bool STAGED>
__device__ __forceinline__ u64 all_weight(const Row<T, STAGED>& row, const Weigh& g, bool plain) {
    constexpr int E = VecOf<T>::kElems;
    u64 sum = 0;
    if (!plain) {
        row.each([&](float x) { sum += Weigh::fixed(Weigh::w(g.depth(x))); });
        return sum;
    }
    WeightSum ws;
    int vecs = 0;
    const f32x2 nm = pair(-g.m, -g.m), c = pair(g.c, g.c);
    row.each_vec([&](int, const uint4& vec) {
        f32x2 x[E / 2];
        unpack(vec, x);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 d = halves(mul2(add2(x[j], nm), c));
            ws.add(pair(ex2(d.x), ex2(d.y)));
        }
        ++vecs;
    });
    return ws.total(vecs * E);
}

// Block-wide sums of a count and a weight; every thread gets both.
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
    for (int i = 0; i < kRowWarps; ++i) {
        n += sh.scan_n[i];
        w += sh.scan_w[i];
    }
}

// u * total as a whole number below total (u outside [0, 1): the nearer end).
__device__ __forceinline__ u64 target_of(float u, u64 total) {
    return min((u64)__double2ull_rz((double)(u > 0.f ? u : 0.f) * (double)total), total - 1);
}

// A listed entry: larger ones come first in the order of falling values.
template <typename T>
__device__ __forceinline__ u64 entry_of(float x, int index) {
    return (u64)Key<T>::of(x) << 32 | (u32)~index;
}

// Finishes a row from its list of n entries, which holds the first k (k > 0) or those
// that reach p of the row's weight `all` (k == 0).  One CTA.
template <typename T>
__device__ void finish_list(const SampleArgs& a, Shared& sh, const Weigh& g, int rowi, int n, int k,
                            float p, float min_p, u64 all) {
    constexpr int kPer = kListMax / kRowThreads;
    const int tid = threadIdx.x;
    __syncthreads();  // `sorted` takes the place of this CTA's own list
    for (int i = tid; i < n; i += kRowThreads) {
        const u64 e = sh.list[i];
        int before = 0;
        for (int j = 0; j < n; ++j) before += sh.list[j] > e;
        sh.sorted[before] = e;
    }
    __syncthreads();
    const int last = k > 0 ? min(k, n) : n;
    u64 W[kPer], sum = 0;
    float w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        w[i] = at < last ? Weigh::w(g.depth(Key<T>::value((u32)(sh.sorted[at] >> 32)))) : 0.f;
        W[i] = Weigh::fixed(w[i]);
        sum += W[i];
    }
    u64 before = warp_before(sum);
    u32 none = 0;
    u64 total = sum;
    block_sum(sh, none, total);
    for (int i = 0; i < tid >> 5; ++i) before += sh.scan_w[i];
    const double limit = (double)p * (double)(k > 0 ? total : all);
    u32 kept = 0;
    u64 kept_w = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        if (at == 0 || (at < last && (!(p < 1.f) || (double)before < limit) && !(w[i] < min_p))) {
            ++kept;
            kept_w += W[i];
        }
        before += W[i];
        sh.list[at] = W[i];  // the list is read: weights by place now
    }
    block_sum(sh, kept, kept_w);
    const u64 target = target_of(a.uniform[rowi], kept_w);
    for (int i = tid; i < (int)kept; i += kRowThreads) {
        const u32 index = (u32)sh.sorted[i];  // ~index
        u64 cum = 0;
        for (int j = 0; j < (int)kept; ++j)
            if ((u32)sh.sorted[j] > index) cum += sh.list[j];
        if (cum <= target && target < cum + sh.list[i]) {
            a.tokens[rowi] = (int)~index;
            if (a.probs != nullptr) a.probs[rowi] = (float)((double)sh.list[i] / (double)kept_w);
        }
    }
}

// The n-th largest of the row's group maxima, rounded down to the upper 16 bits of its
// key: at least n entries are not below it.  One warp.
__device__ __forceinline__ float group_bound(const Shared& sh, int n) {
    constexpr int kPer = kGroups / 32;
    const int lane = threadIdx.x & 31;
    u32 key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = Key<float>::of(sh.group_max[lane + 32 * i]) >> 16;
    u32 lo = 0;  // the largest value that n keys reach, bit by bit
    for (u32 bit = 0x8000; bit != 0; bit >>= 1) {
        u32 count = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += key[i] >= (lo | bit);
        if (__reduce_add_sync(0xffffffffu, count) >= (u32)n) lo |= bit;
    }
    return Key<float>::value(lo << 16);
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kRowThreads) sample_kernel(SampleArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = 1 << a.lg, rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int rowi = blockIdx.x >> a.lg;
    const RowView<T> r(a.logits, a.ld, rowi, a.V);
    const RowSlice sl(r.nvec, a.per, rank, warp);
    const Row<T, STAGED> row{r, sl, reinterpret_cast<const uint4*>(smem) - sl.lo, cs, rank};
    if (cs > 1) cluster_arrive();  // met by cluster_wait below: every CTA has started
    if (STAGED) {
        for (int v = sl.wlo + lane; v < sl.whi; v += 32) r.stage(v, smem_u32(row.staged + v));
    }
    float T0 = a.temperature != nullptr ? a.temperature[rowi] : a.temperature0;
    int k = a.top_k != nullptr ? a.top_k[rowi] : a.top_k0;
    const float p = a.top_p != nullptr ? a.top_p[rowi] : a.top_p0;
    float min_p = a.min_p != nullptr ? a.min_p[rowi] : a.min_p0;
    if (!(T0 > 0.f)) T0 = 0.f;
    if (k < 0 || k >= a.V) k = 0;
    if (T0 == 0.f || p <= 0.f || min_p > 1.f) k = 1;  // the first entry is always kept
    if (k == 1) min_p = 0.f;
    if (tid == 0) sh.own_n = sh.list_n = 0;
    if (STAGED) cp_async_wait_all();

    // the largest entries of the groups (cs lanes each) and of the row
    float m = neg_inf();
    row.each_vec([&](int, const uint4& v) { m = max_or_nan(m, vec_max_or_nan<T>(v)); });
    const bool has_nan = __any_sync(0xffffffffu, m != m);
    if (has_nan) {
        m = neg_inf();
        row.each_vec([&](int, const uint4& v) { m = fmaxf(m, vec_max<T>(v)); });
    }
#pragma unroll
    for (int o = kRowMaxCluster / 2; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, m, o);
        if (o < cs) m = fmaxf(m, other);
    }
    if ((tid & (cs - 1)) == 0) (cs > 1 ? sh.own_max : sh.group_max)[tid >> a.lg] = m;
    __syncthreads();
    if (cs > 1) {
        cluster_wait();
        // kGroups / 4 of the threads send four maxima each to one of the CTAs
        const int lq = 6 - a.lg, quads = 1 << lq, to = tid >> lq, i = tid & (quads - 1);
        static_assert(kGroups / 4 == 1 << 6);
        if (to < cs)
            st_cluster_v4(map_cluster(smem_u32(&sh.group_max[4 * (rank * quads + i)]), to),
                          reinterpret_cast<const float4*>(sh.own_max)[i]);
        row.sync();
    }
    m = neg_inf();
    for (int i = lane; i < kGroups; i += 32) m = fmaxf(m, sh.group_max[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == neg_inf()) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            a.tokens[rowi] = -1;
            if (a.probs != nullptr) a.probs[rowi] = 0.f;
        }
        return;
    }
    const Weigh g{m, __fdiv_rn(kLog2e, T0 > 0.f ? T0 : 1.f)};
    const bool plain = !has_nan && m < INFINITY;

    Cut cut{0, 0, 0};
    if (k > 0 || p < 1.f) {
        // Is there a bound with a list short enough?  Without top_k: about as many entries
        // above it as half the groups; in a row of up to kListMax, all of them.
        const int want = k > 0 ? k : kGroups / 2;
        if (a.V <= kListMax || want <= kGroups) {
            if (warp == 0) {
                float b = a.V <= kListMax ? -3.402823466e38f : group_bound(sh, want);
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
            u64 all = k == 0 ? all_weight(row, g, plain) : 0;
            u32 none = 0;
            if (k == 0) {
                block_sum(sh, none, listed_w);
                block_sum(sh, none, all);
            } else {
                __syncthreads();
            }
            const u32 n = sh.own_n;
            if (cs > 1) {
                // to rank 0's list, behind those that got there first
                if (tid == 0)
                    sh.base = n <= kListMax
                                  ? atom_add_cluster(map_cluster(smem_u32(&sh.list_n), 0), n)
                                  : kListMax;
                __syncthreads();
                for (u32 i = tid; i < n && sh.base + i < kListMax; i += kRowThreads)
                    st_cluster_b64(map_cluster(smem_u32(&sh.list[sh.base + i]), 0),
                                   sh.own_list[i]);
                if (tid < cs) {
                    const u32 told = map_cluster(smem_u32(&sh.told[rank]), tid);
                    st_cluster_b64(told, n);
                    st_cluster_b64(told + 8, listed_w);
                    st_cluster_b64(told + 16, all);
                }
            } else {
                for (u32 i = tid; i < min(n, (u32)kListMax); i += kRowThreads)
                    sh.list[i] = sh.own_list[i];
                if (tid == 0) sh.told[0] = {n, listed_w, all};
            }
            row.sync();
            Told t{0, 0, 0};
            for (int i = 0; i < cs; ++i) {
                t.listed += sh.told[i].listed;
                t.weight += sh.told[i].weight;
                t.all += sh.told[i].all;
            }
            if (t.listed <= kListMax &&
                (k > 0 || (double)t.weight >= (double)p * (double)t.all)) {
                // the other CTAs' shared memory is not touched any more
                if (rank == 0)
                    finish_list<T>(a, sh, g, rowi, (int)t.listed, k, p, min_p, t.all);
                return;
            }
            __syncthreads();
        }
        double total = -1;
        u64 kept;
        if (k > 0) {
            find_cut<true>(sh, row, g, cut, (u32)k, 0, 0, p < 1.f, &cut, &kept);
            total = (double)kept;
        }
        if (p < 1.f) {
            const Cut in = cut;
            find_cut<false>(sh, row, g, in, 0, (double)p, total, true, &cut, &kept);
        }
    }

    // every warp's kept weight and its ties at the cut
    const bool everything = cut.key == 0 && !(min_p > 0.f);
    const float floor = cut.key != 0 ? Key<T>::value(cut.key) : neg_inf();
    const float min_d = min_p > 0.f ? log2f(min_p) - 0.02f : neg_inf();  // w < min_p below it
    auto kept_of = [&](const uint4& vec, u64& w, u32& ties) {
        if (everything && plain) {
            f32x2 x[E / 2];
            unpack(vec, x);
            WeightSum ws;
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 h = halves(x[j]);
                ws.add(pair(Weigh::w(g.depth(h.x)), Weigh::w(g.depth(h.y))));
            }
            w += ws.total(E);
            return;
        }
        const float most = vec_max<T>(vec);  // one of the kept entries is rare: look at it first
        if (!(most >= floor) || !(g.depth(most) >= min_d)) return;
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
                ties += Weigh::fixed(wj) != 0;
        }
    };
    u64 sw = 0;
    u32 st = 0;
    if (everything)
        sw = all_weight(row, g, plain);
    else
        row.each_vec([&](int, const uint4& vec) { kept_of(vec, sw, st); });
    sw = warp_sum(sw);
    st = __reduce_add_sync(0xffffffffu, st);
    const int me = rank * kRowWarps + warp;
    if (cs > 1) {
        if (lane < cs) {
            st_cluster_b64(map_cluster(smem_u32(&sh.part_w[me]), lane), sw);
            st_cluster_b64(map_cluster(smem_u32(&sh.part_t[me]), lane), st);
        }
    } else if (lane == 0) {
        sh.part_w[me] = sw;
        sh.part_t[me] = st;
    }
    row.sync();  // no CTA's shared memory is touched from outside after this

    // the warp that holds the token (every warp finds it: two parts a lane)
    auto ties_weight = [&](u32 before, u32 n) {
        return (u64)(min(cut.ties, before + n) - min(cut.ties, before)) * cut.weight;
    };
    const int parts = cs * kRowWarps;
    u64 pw[2];
    u32 pt[2], pb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int q = 2 * lane + i;
        pw[i] = q < parts ? sh.part_w[q] : 0;
        pt[i] = q < parts ? (u32)sh.part_t[q] : 0;
    }
    pb[0] = warp_before(pt[0] + pt[1]);
    pb[1] = pb[0] + pt[0];
#pragma unroll
    for (int i = 0; i < 2; ++i) pw[i] += ties_weight(pb[i], pt[i]);
    u64 base = warp_before(pw[0] + pw[1]);
    const u64 total = __shfl_sync(0xffffffffu, base + pw[0] + pw[1], 31);
    const u64 target = target_of(a.uniform[rowi], total);
    const bool second = base + pw[0] <= target;
    if (second) base += pw[0];
    const bool mine = base <= target && target < base + (second ? pw[1] : pw[0]);
    const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    const int holder = __shfl_sync(0xffffffffu, 2 * lane + (second ? 1 : 0), from);
    if (holder != me) return;
    u64 sum = __shfl_sync(0xffffffffu, base, from);  // kept weight and ties before this warp
    u32 ties = __shfl_sync(0xffffffffu, second ? pb[1] : pb[0], from);
    for (int v0 = sl.wlo; v0 < sl.whi; v0 += 32) {
        const int v = v0 + lane;
        u64 lw = 0;
        u32 lt = 0;
        if (v < sl.whi) kept_of(row.vec(v), lw, lt);
        const u32 all_t = __reduce_add_sync(0xffffffffu, lt);
        const u64 all_w = warp_sum(lw) + ties_weight(ties, all_t);
        if (sum + all_w <= target) {
            sum += all_w;
            ties += all_t;
            continue;
        }
        // these 32 vectors hold it: the lane, then the entry
        u32 tie = ties + warp_before(lt);
        lw += ties_weight(tie, lt);
        u64 at = sum + warp_before(lw);
        if (at > target || target >= at + lw) return;
        float x[E];
        unpack(row.vec(v), x);
        int token = -1;
        u64 tw = 0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const u32 key = Key<T>::of(x[j]);
            const float wj = Weigh::w(g.depth(x[j]));
            u64 w = wj < min_p ? 0 : Weigh::fixed(wj);
            if (key < cut.key) {
                w = 0;
            } else if (key == cut.key && w != 0) {
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
        return;
    }
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, int bf16, cudaStream_t stream, int num_sms,
                          size_t max_smem) {
    const RowSplit p = split_rows(a.rows, a.V, bf16 ? 2 : 4, num_sms, max_smem - sizeof(Shared) - 1024);
    a.lg = p.lg;
    a.per = p.per;
    if (bf16)
        return launch_rows(p.staged != 0 ? sample_kernel<__nv_bfloat16, true>
                                         : sample_kernel<__nv_bfloat16, false>,
                           a, a.rows, a.lg, p.staged, stream);
    return launch_rows(p.staged != 0 ? sample_kernel<float, true> : sample_kernel<float, false>, a,
                       a.rows, a.lg, p.staged, stream);
}

}  // namespace df2
