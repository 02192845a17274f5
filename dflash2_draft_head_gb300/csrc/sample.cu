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
// Bound by HBM: a row is read once, by one CTA or by the CTAs of a cluster, and passed
// over two or more times on the chip.  The largest entries of 256 groups of the row come first: their maximum is the row's, and the n-th largest
// of them is a bound above which at least n entries lie.
//   - Neither top_k nor top_p: one pass of weights, summed by warp; one warp of the
//     row holds the token and looks it up.
//   - Up to 256 entries to keep, or a top_p that the entries above such a bound
//     reach: those entries (some hundreds) are listed, and one CTA finishes the row
//     from the list alone.
//   - Else the cut is found by histograms: of counts over the distance from the maximum
//     first (a bin's weights differ by 1.4%, which leaves a few bins that may hold the
//     cut), then of the exact weights over the values of those bins, until that is one
//     value; ties there are kept by index.  The weights of what is kept are then
//     summed and looked up as in the first case.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "dflash2.h"
#include "rows.cuh"

namespace df2 {
namespace {

using u32 = uint32_t;
using u64 = unsigned long long;

using Geo = RowGeometry<512, 2, 5, 320>;
constexpr int kRowThreads = Geo::kThreads, kRowWarps = Geo::kWarps;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kOne = 1099511627776.f;  // 2^40, the largest entry's weight
constexpr float kDepth = 41.f;           // entries 2^-kDepth below the largest weigh nothing
constexpr int kDepthBins = 2048;         // of counts, over the depth
constexpr int kBins = 512;               // of counts and weights, over keys
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

constexpr int kGroups = 256;          // groups of a row whose maxima are exchanged
constexpr int kListMax = 1024;        // entries of a row's list
constexpr int kParts = kRowMaxCluster * kRowWarps;
constexpr int kMaxSteps = 64;         // of a warp: see the assertion beside the launch

// What a CTA tells the others of its slice: listed entries, their weight, all weight.
struct Told {
    u64 listed, weight, all;
};

struct Shared {
    union {
        u32 count[kDepthBins];
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
    u64 cta_span[kRowMaxCluster];  // largest and smallest key of a bracket, by CTA
    u64 cta_w[kRowMaxCluster];     // and the weight above it
    u64 step_w[kMaxSteps];       // kept weight of the steps of one warp
    u32 step_t[kMaxSteps];       // and their ties
    u32 span_hi, span_lo;
    u32 scan_n[kRowWarps];
    u64 scan_w[kRowWarps];
    // the bins that may hold the cut; for one bin, what stands before it and its weight
    int at, at_hi;
    u32 before_n;
    u64 before_w, in_w;
};

template <typename T>
struct Row {
    static constexpr int E = VecOf<T>::kElems;
    RowView<T> r;
    RowSlice<Geo> sl;
    int cs, rank;

    template <typename F>
    __device__ __forceinline__ void each_vec(F f) {
        sl.pass(r, [&](int v, const uint4& vec, bool) { f(v, vec); });
    }
    // f(entries, their depths), two at a time.  `plain`: no NaN among them and a finite
    // maximum; else a NaN has the depth of -inf
    template <typename F>
    __device__ __forceinline__ void each_pair(const Weigh& g, bool plain, F f) {
        const f32x2 nm = pair(-g.m, -g.m), c = pair(g.c, g.c);
        if (plain) {
            each_vec([&](int, const uint4& vec) {
                f32x2 x[E / 2];
                unpack(vec, x);
#pragma unroll
                for (int j = 0; j < E / 2; ++j)
                    f(halves(x[j]), halves(mul2(add2(x[j], nm), c)));
            });
        } else {
            each_vec([&](int, const uint4& vec) {
                float x[E];
                unpack(vec, x);
#pragma unroll 1
                for (int j = 0; j < E; j += 2)
                    f(make_float2(x[j], x[j + 1]),
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

// Sums of weights over the whole row; every thread gets them.
template <typename R>
__device__ __forceinline__ u64 row_weight(Shared& sh, const R& row, u64 w) {
    u32 none = 0;
    block_sum(sh, none, w);
    if (row.cs == 1) return w;
    if ((int)threadIdx.x < row.cs)
        st_cluster_b64(map_cluster(smem_u32(&sh.cta_w[row.rank]), threadIdx.x), w);
    row.sync();
    w = 0;
    for (int i = 0; i < row.cs; ++i) w += sh.cta_w[i];
    return w;
}

// Running sums over the block's threads: what stands before this one.
__device__ __forceinline__ void block_before(Shared& sh, u32& n, u64& w) {
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
    for (int i = 0; i < (int)threadIdx.x >> 5; ++i) {
        n += sh.scan_n[i];
        w += sh.scan_w[i];
    }
}

__device__ __forceinline__ int depth_bin(float d) {
    return min(kDepthBins - 1, (int)(d * -(kDepthBins / kDepth)));
}

// The bounds of a weight in that bin, in units of 2^-40: the roundings of the depth,
// of 2^x and of the weight are far inside 2^-16 of it and 1.
__device__ __forceinline__ u64 bin_most(int bin) {
    return __float2ull_ru(ex2(bin * -(kDepth / kDepthBins)) * (kOne * (1.f + 1.f / 65536))) + 1;
}
__device__ __forceinline__ u64 bin_least(int bin) {
    const u64 w = __float2ull_rd(ex2((bin + 1) * -(kDepth / kDepthBins)) *
                                 (kOne * (1.f - 1.f / 65536)));
    return bin == kDepthBins - 1 || w == 0 ? 0 : w - 1;
}

// Adds up the cluster's counts by depth and finds, from the largest entries down, the
// bins that may hold the cut: sh.at to sh.at_hi (one bin, with sh.before_n, by count);
// sh.at is kDepthBins when there is no cut.
template <bool BY_COUNT, typename R>
__device__ void find_bracket(Shared& sh, const R& row, u32 k, double limit) {
    constexpr int kPer = kDepthBins / kRowThreads;
    const int first = (int)threadIdx.x * kPer;
    if (threadIdx.x == 0) {
        sh.at = kDepthBins;
        sh.at_hi = kDepthBins - 1;
    }
    row.sync();  // every histogram is filled
    u32 n[kPer] = {};
    for (int q = 0; q < row.cs; ++q) {
#pragma unroll
        for (int i = 0; i < kPer; i += 4) {
            const uint4 b = row.cs > 1 ? ld_cluster_v4(map_cluster(smem_u32(&sh.count[first + i]), q))
                                       : *reinterpret_cast<const uint4*>(&sh.count[first + i]);
            n[i] += b.x;
            n[i + 1] += b.y;
            n[i + 2] += b.z;
            n[i + 3] += b.w;
        }
    }
    u32 bn = 0;
    u64 least = 0, most = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        bn += n[i];
        if (!BY_COUNT) {
            least += n[i] * bin_least(first + i);
            most += n[i] * bin_most(first + i);
        }
    }
    u32 none = 0;
    block_before(sh, bn, least);
    if (!BY_COUNT) block_before(sh, none, most);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const u64 l = BY_COUNT ? 0 : n[i] * bin_least(first + i);
        const u64 h = BY_COUNT ? 0 : n[i] * bin_most(first + i);
        if (BY_COUNT ? bn < k && bn + n[i] >= k
                     : (double)most < limit && (double)(most + h) >= limit) {
            sh.at = first + i;
            sh.before_n = bn;
            if (BY_COUNT) sh.at_hi = first + i;
        }
        if (!BY_COUNT && (double)least < limit && (double)(least + l) >= limit)
            sh.at_hi = first + i;
        bn += n[i];
        least += l;
        most += h;
    }
    row.sync();  // every histogram is read, and the bins are found
}

// Adds up the cluster's histograms and finds the first bin at which the running count
// reaches k or the running weight `limit`; sh.at is kBins when none does.
template <bool BY_COUNT, typename R>
__device__ void find_bin(Shared& sh, const R& row, u32 base_n, u64 base_w, u32 k, double limit) {
    constexpr int kPer = kBins / kRowThreads;
    const int first = (int)threadIdx.x * kPer;
    if (threadIdx.x == 0) sh.at = kBins;
    row.sync();  // every histogram is filled
    u32 n[kPer] = {}, bn = 0;
    u64 w[kPer] = {}, bw = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        for (int q = 0; q < row.cs; ++q) {
            const uint4 b = row.cs > 1 ? ld_cluster_v4(map_cluster(smem_u32(&sh.hist[first + i]), q))
                                       : sh.hist[first + i];
            n[i] += b.x;
            w[i] += bin_weight(b);
        }
        bn += n[i];
        bw += w[i];
    }
    block_before(sh, bn, bw);
    bn += base_n;
    bw += base_w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool open = BY_COUNT ? bn < k : (double)bw < limit;
        const bool shut = BY_COUNT ? bn + n[i] >= k : (double)(bw + w[i]) >= limit;
        if (open && shut) {  // one bin of the row
            sh.at = first + i;
            sh.before_n = bn;
            sh.before_w = bw;
            sh.in_w = w[i];
        }
        bn += n[i];
        bw += w[i];
    }
    row.sync();  // every histogram is read, and the bin is found
}

// The cut by count (the first k entries) or by weight (those with less than `limit`
// before them), among the entries inside `in`; `in` itself when that cuts nothing.
struct Found {
    Cut cut;
    u64 kept_w;  // the kept entries' weight (by count: where `weigh` asks for it)
    bool up;     // the direction of the row's next pass
};
template <bool BY_COUNT, typename T>
__device__ __noinline__ Found find_cut(Shared& sh, Row<T> row, const Weigh g, bool plain,
                                      const Cut in, u32 k, double limit, bool weigh) {
    const int tid = threadIdx.x, lane = tid & 31;
    auto clear = [&] {  // all of count and of hist
        for (int i = tid; i < kBins; i += kRowThreads) sh.hist[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) {
            sh.span_hi = 0;
            sh.span_lo = 0xffffffffu;
        }
        __syncthreads();
    };
    static_assert(sizeof(sh.count) == sizeof(sh.hist));
    const float least = in.key != 0 ? Key<T>::value(in.key) : neg_inf();
    clear();
    row.each_pair(g, plain, [&](float2 x, float2 d) {
        if (x.x >= least && d.x >= -kDepth) atomicAdd(&sh.count[depth_bin(d.x)], 1u);
        if (x.y >= least && d.y >= -kDepth) atomicAdd(&sh.count[depth_bin(d.y)], 1u);
    });
    find_bracket<BY_COUNT>(sh, row, k, limit);
    const int at = sh.at, at_hi = sh.at_hi;
    u32 n = sh.before_n;

    // the weight above the bracket, and the span of the keys in it
    WeightSum above;
    int entries = 0;
    float hi_x = neg_inf(), lo_x = INFINITY;
    row.each_pair(g, plain, [&](float2 x, float2 d) {
        const bool in_x = x.x >= least && d.x >= -kDepth, in_y = x.y >= least && d.y >= -kDepth;
        const int bx = depth_bin(d.x), by = depth_bin(d.y);
        above.add(pair(in_x && bx < at ? ex2(d.x) : 0.f, in_y && by < at ? ex2(d.y) : 0.f));
        entries += 2;
        if (in_x && bx >= at && bx <= at_hi) {
            hi_x = fmaxf(hi_x, x.x);
            lo_x = fminf(lo_x, x.x);
        }
        if (in_y && by >= at && by <= at_hi) {
            hi_x = fmaxf(hi_x, x.y);
            lo_x = fminf(lo_x, x.y);
        }
    });
    u64 w = BY_COUNT && !weigh ? 0 : row_weight(sh, row, above.total(entries));
    if (at == kDepthBins) return {in, w, row.sl.up};
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
        clear();
        row.each_pair(g, plain, [&](float2 x, float2 d) {
            auto add = [&](float x, float d) {
                if (!(x >= lo_v && x <= hi_v)) return;
                u32* h = reinterpret_cast<u32*>(&sh.hist[(hi - Key<T>::of(x)) >> shift]);
                const u64 W = Weigh::fixed(Weigh::w(d));
                if (BY_COUNT) atomicAdd(h, 1u);
                if (BY_COUNT && !weigh) return;
                atomicAdd(h + 1, (u32)W & ((1u << kLimb) - 1));
                atomicAdd(h + 2, (u32)(W >> kLimb) & ((1u << kLimb) - 1));
                atomicAdd(h + 3, (u32)(W >> (2 * kLimb)));
            };
            add(x.x, d.x);
            add(x.y, d.y);
        });
        find_bin<BY_COUNT>(sh, row, n, w, k, limit);
        if (sh.at == kBins) break;  // not reached: the bracket holds the cut
        n = sh.before_n;
        w = sh.before_w;
        in_w = sh.in_w;
        hi -= (u32)sh.at << shift;
        lo = hi - min(hi - lo, (1u << shift) - 1);
        more = more && hi != lo;
    }
    Cut out{hi, 0, Weigh::fixed(Weigh::w(g.depth(Key<T>::value(hi))))};
    out.ties = BY_COUNT ? k - n : ties_below(w, out.weight, (u32)(in_w / max(out.weight, (u64)1)), limit);
    if (hi == in.key) out.ties = min(out.ties, in.ties);
    __syncthreads();
    return {out, w + out.ties * out.weight, row.sl.up};
}

// This lane's part of its warp's weight: all entries.
template <typename T>
__device__ __forceinline__ u64 all_weight(Row<T>& row, const Weigh& g, bool plain) {
    WeightSum ws;
    int entries = 0;
    row.each_pair(g, plain, [&](float2, float2 d) {
        ws.add(pair(ex2(d.x), ex2(d.y)));
        entries += 2;
    });
    return ws.total(entries);
}

// This lane's part of its warp's kept weight, and its ties at the cut.
template <typename T>
__device__ __forceinline__ void kept_weight(Row<T>& row, const Weigh& g, bool plain,
                                            const Cut& cut, float min_p, u64& weight, u32& ties) {
    const float floor = cut.key != 0 ? Key<T>::value(cut.key) : neg_inf();
    const float least = min_p > 0.f ? min_p : 0.f;
    WeightSum ws;
    int entries = 0;
    u32 t = 0;
    row.each_pair(g, plain, [&](float2 x, float2 d) {
        const float wx = ex2(d.x), wy = ex2(d.y);
        const bool kx = wx >= least, ky = wy >= least;
        ws.add(pair(kx && x.x > floor ? wx : 0.f, ky && x.y > floor ? wy : 0.f));
        t += (kx && x.x == floor) + (ky && x.y == floor);
        entries += 2;
    });
    weight = ws.total(entries);
    ties = cut.ties != 0 ? t : 0;
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
__device__ __noinline__ void finish_list(const SampleArgs& a, Shared& sh, const Weigh g, int rowi, int n, int k,
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

template <typename T>
__global__ void __launch_bounds__(kRowThreads, Geo::kCtas) sample_kernel(SampleArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = 1 << a.lg, rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int rowi = blockIdx.x >> a.lg;
    const RowView<T> r(a.logits, a.ld, rowi, a.V);
    Row<T> row{r, RowSlice<Geo>(r, a.per, a.ring, rank, warp, smem, l2_policy_evict_last()), cs, rank};
    const RowSlice<Geo>& sl = row.sl;
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
    constexpr int kLanes = kRowThreads / kGroups;
    static_assert(kLanes >= 1 && kLanes * kRowMaxCluster <= 32);
    float m = neg_inf();
    row.each_vec([&](int, const uint4& v) { m = max_or_nan(m, vec_max_or_nan<T>(v)); });
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
        u64 listed_all = 0;  // the row's whole weight (without top_k)
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
            listed_all = t.all;
            __syncthreads();
        }
        u64 kept = listed_all;
        if (k > 0) {
            const Found f = find_cut<true>(sh, row, g, plain, cut, (u32)k, 0, p < 1.f);
            cut = f.cut;
            kept = f.kept_w;
            row.sl.up = f.up;
        }
        if (p < 1.f) {
            const Found f =
                find_cut<false>(sh, row, g, plain, cut, 0, (double)p * (double)kept, true);
            cut = f.cut;
            row.sl.up = f.up;
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
        kept_weight(row, g, plain, cut, min_p, sw, st);
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

    // the warp that holds the token (every warp finds it: `per` parts a lane)
    auto ties_weight = [&](u32 before, u32 n) {
        return (u64)(min(cut.ties, before + n) - min(cut.ties, before)) * cut.weight;
    };
    const int parts = cs * kRowWarps, per = max(1, parts >> 5);
    const int p_lo = min(lane * per, parts), p_hi = min(p_lo + per, parts);
    u32 ties = 0;  // before this lane's parts
    if (cut.ties != 0) {
        for (int i = p_lo; i < p_hi; ++i) ties += (u32)sh.part_t[i];
        ties = warp_before(ties);
    }
    u64 lane_w = 0;
    u32 tie = ties;
    for (int i = p_lo; i < p_hi; ++i) {
        lane_w += sh.part_w[i];
        if (cut.ties == 0) continue;
        lane_w += ties_weight(tie, (u32)sh.part_t[i]);
        tie += (u32)sh.part_t[i];
    }
    u64 sum = warp_before(lane_w);
    const u64 total = __shfl_sync(0xffffffffu, sum + lane_w, 31);
    const u64 target = target_of(a.uniform[rowi], total);
    const int from =
        __ffs(__ballot_sync(0xffffffffu, sum <= target && target < sum + lane_w)) - 1;
    int holder = p_lo;
    for (; holder < p_hi - 1; ++holder) {
        const u64 w = sh.part_w[holder] + ties_weight(ties, (u32)sh.part_t[holder]);
        if (target < sum + w) break;
        sum += w;
        ties += (u32)sh.part_t[holder];
    }
    holder = __shfl_sync(0xffffffffu, holder, from);
    if (holder / kRowWarps != rank) return;
    sum = __shfl_sync(0xffffffffu, sum, from);  // kept weight and ties before this warp
    ties = __shfl_sync(0xffffffffu, ties, from);

    // that warp's steps, by all warps of its CTA; then the warp of the step that holds it
    const RowSlice<Geo> own(r, a.per, a.ring, rank, holder % kRowWarps, smem, 0);
    for (int step = warp; step < own.steps; step += kRowWarps) {
        u64 w = 0;
        u32 t = 0;
#pragma unroll
        for (int i = 0; i < kStepVecs; i += 32) {
            const int v = own.wlo + step * kStepVecs + i + lane;
            if (v < own.whi) kept_of(r.load(v), w, t);
        }
        w = warp_sum(w);
        t = __reduce_add_sync(0xffffffffu, t);
        if (lane == 0) {
            sh.step_w[step] = w;
            sh.step_t[step] = t;
        }
    }
    __syncthreads();
    int step = 0;
    for (; step < own.steps - 1; ++step) {
        const u64 w = sh.step_w[step] + ties_weight(ties, sh.step_t[step]);
        if (target < sum + w) break;
        sum += w;
        ties += sh.step_t[step];
    }
    if (step % kRowWarps != warp) return;
    for (int i = 0; i < kStepVecs; i += 32) {  // its vectors 32 at a time: the lane, the entry
        const int v = own.wlo + step * kStepVecs + i + lane;
        u64 lw = 0;
        u32 lt = 0;
        if (v < own.whi) kept_of(r.load(v), lw, lt);
        u32 tie = ties + warp_before(lt);
        ties += __reduce_add_sync(0xffffffffu, lt);
        lw += ties_weight(tie, lt);
        u64 at = sum + warp_before(lw);
        sum = __shfl_sync(0xffffffffu, at + lw, 31);
        if (at > target || target >= at + lw) continue;
        float x[E];
        unpack(r.load(v), x);
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
    }
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, int bf16, cudaStream_t stream, int num_sms) {
    // the widest row: kSampleMaxV fp32 entries over the largest cluster
    static_assert(kSampleMaxV / 4 / kRowMaxCluster / kRowWarps / kStepVecs < kMaxSteps);
    const RowSplit p = split_rows<Geo>(a.rows, a.V, bf16 ? 2 : 4, num_sms);
    a.lg = p.lg;
    a.per = p.per;
    a.ring = p.ring;
    return launch_rows<Geo>(bf16 ? sample_kernel<__nv_bfloat16> : sample_kernel<float>, a, a.rows, a.lg,
                       p.smem, stream);
}

}  // namespace df2
