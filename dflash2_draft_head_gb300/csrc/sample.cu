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
// holding its slice in shared memory for the passes: the maximum, the cut (where
// top_k or top_p ask for one) and the sums by warp, of which one warp holds the
// token.  The cut is found by histograms of the entries' counts and weights, first
// over their distance from the maximum, then over the values of the bin in which
// the cut lies, until that is one value; ties there are kept by index.
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

struct Shared {
    uint4 hist[kBins];                        // count and the three words of the weight
    u64 part_w[kRowMaxCluster * kRowWarps];   // kept weight of every warp of the row
    u64 part_t[kRowMaxCluster * kRowWarps];   // and its ties at the cut
    float cta_max[kRowMaxCluster];
    u64 cta_span[kRowMaxCluster];             // largest and smallest key of a bin, by CTA
    float warp_max[kRowWarps];
    u32 span_hi, span_lo;
    u32 scan_n[kRowWarps];
    u64 scan_w[kRowWarps];
    // the bin in which the cut lies, what stands before it and what it holds
    int at;
    u32 before_n, in_n;
    u64 before_w;
    u64 total_w;
};

template <typename T, bool STAGED>
struct Row {
    static constexpr int E = VecOf<T>::kElems;
    RowView<T> r;
    RowSlice sl;
    u32 stage0;
    int cs, rank;

    __device__ __forceinline__ uint4 vec(int v) const {
        return STAGED ? lds_v4(stage0 + (u32)v * 16u) : r.load(v);
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
            sh.in_n = n[i];
        }
        bn += n[i];
        bw += w[i];
    }
    __syncthreads();
}

// The cut by count (the first k entries) or by weight (those with less than
// p * total before them; total < 0: the row's own sum), among the entries inside
// `in`.  Returns false when nothing is cut.  *kept_w: the kept entries' weight.
template <bool BY_COUNT, typename T, bool STAGED>
__device__ bool find_cut(Shared& sh, const Row<T, STAGED>& row, const Weigh& g, const Cut& in,
                         u32 k, double p, double total, Cut* out, u64* kept_w) {
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
        atomicAdd(h, 1u);
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
    u32 in_n = sh.in_n;
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
        in_n = sh.in_n;
        hi -= (u32)sh.at << shift;
        lo = hi - min(hi - lo, (1u << shift) - 1);
    }
    out->key = hi;
    out->weight = Weigh::fixed(Weigh::w(g.depth(Key<T>::value(hi))));
    out->ties = BY_COUNT ? k - n : ties_below(w, out->weight, in_n, limit);
    if (hi == in.key) out->ties = min(out->ties, in.ties);
    *kept_w = w + out->ties * out->weight;
    __syncthreads();
    return true;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kRowThreads) sample_kernel(SampleArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = a.cs, rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int rowi = blockIdx.x / cs;
    const RowView<T> r(a.logits, a.ld, rowi, a.V);
    const RowSlice sl(r.nvec, rank, cs, warp);
    const Row<T, STAGED> row{r, sl, smem_u32(smem) - (u32)sl.lo * 16u, cs, rank};
    if (cs > 1) cluster_arrive();  // met by cluster_wait below: every CTA has started
    if (STAGED) {
        for (int v = sl.wlo + lane; v < sl.whi; v += 32) r.stage(v, row.stage0 + (u32)v * 16u);
    }
    float T0 = a.temperature != nullptr ? a.temperature[rowi] : a.temperature0;
    int k = a.top_k != nullptr ? a.top_k[rowi] : a.top_k0;
    const float p = a.top_p != nullptr ? a.top_p[rowi] : a.top_p0;
    float min_p = a.min_p != nullptr ? a.min_p[rowi] : a.min_p0;
    if (!(T0 > 0.f)) T0 = 0.f;
    if (T0 == 0.f || p <= 0.f || min_p > 1.f) k = 1;  // the first entry is always kept
    if (k == 1) min_p = 0.f;
    if (STAGED) cp_async_wait_all();

    float m = neg_inf();
    for (int v = sl.wlo + lane; v < sl.whi; v += 32) m = fmaxf(m, vec_max<T>(row.vec(v)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sh.warp_max[warp] = m;
    __syncthreads();
    for (int i = 0; i < kRowWarps; ++i) m = fmaxf(m, sh.warp_max[i]);
    if (cs > 1) {
        cluster_wait();
        if (tid < cs) st_cluster_f32(map_cluster(smem_u32(&sh.cta_max[rank]), tid), m);
        row.sync();
        for (int i = 0; i < cs; ++i) m = fmaxf(m, sh.cta_max[i]);
    }
    if (m == neg_inf()) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            a.tokens[rowi] = -1;
            if (a.probs != nullptr) a.probs[rowi] = 0.f;
        }
        return;
    }
    const Weigh g{m, __fdiv_rn(kLog2e, T0 > 0.f ? T0 : 1.f)};

    Cut cut{0, 0, 0};
    if (k == 1) {
        cut = {Key<T>::of(m), 1, Weigh::fixed(1.f)};
    } else {
        double total = -1;
        u64 kept;
        if (k > 0 && k < a.V) {
            find_cut<true>(sh, row, g, cut, (u32)k, 0, 0, &cut, &kept);
            total = (double)kept;
        }
        if (p < 1.f) {
            const Cut in = cut;
            find_cut<false>(sh, row, g, in, 0, (double)p, total, &cut, &kept);
        }
    }

    // every warp's kept weight and its ties at the cut
    auto weight = [&](float x) {
        const float w = Weigh::w(g.depth(x));
        return w < min_p ? (u64)0 : Weigh::fixed(w);
    };
    u64 sw = 0;
    u32 st = 0;
    row.each([&](float x) {
        const u32 key = Key<T>::of(x);
        if (key > cut.key)
            sw += weight(x);
        else if (key == cut.key && weight(x) != 0)
            ++st;
    });
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
    const float u = a.uniform[rowi];
    const u64 target =
        min((u64)__double2ull_rz((double)(u > 0.f ? u : 0.f) * (double)total), total - 1);
    const bool second = base + pw[0] <= target;
    if (second) base += pw[0];
    const bool mine = base <= target && target < base + (second ? pw[1] : pw[0]);
    const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    const int holder = __shfl_sync(0xffffffffu, 2 * lane + (second ? 1 : 0), from);
    if (holder != me) return;
    u64 sum = __shfl_sync(0xffffffffu, base, from);                       // before this warp
    u32 ties = __shfl_sync(0xffffffffu, second ? pb[1] : pb[0], from);
    for (int v0 = sl.wlo; v0 < sl.whi; v0 += 32) {
        float x[E];
        u64 lw = 0;
        u32 lt = 0;
        const bool live = v0 + lane < sl.whi;
        if (live) {
            unpack(row.vec(v0 + lane), x);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const u32 key = Key<T>::of(x[j]);
                if (key > cut.key)
                    lw += weight(x[j]);
                else if (key == cut.key && weight(x[j]) != 0)
                    ++lt;
            }
        }
        const u32 tb = ties + warp_before(lt);
        lw += ties_weight(tb, lt);
        const u64 wb = sum + warp_before(lw);
        if (live && wb <= target && target < wb + lw) {
            // constant indices only: the vector stays in registers
            int token = -1;
            u64 tw = 0, at = wb;
            u32 tie = tb;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const u32 key = Key<T>::of(x[j]);
                u64 w = 0;
                if (key > cut.key) {
                    w = weight(x[j]);
                } else if (key == cut.key && weight(x[j]) != 0) {
                    w = ties_weight(tie, 1);
                    ++tie;
                }
                at += w;
                if (token < 0 && target < at) {
                    token = (v0 + lane) * E + j - r.head;
                    tw = w;
                }
            }
            a.tokens[rowi] = token;
            if (a.probs != nullptr) a.probs[rowi] = (float)((double)tw / (double)total);
        }
        sum = __shfl_sync(0xffffffffu, wb + lw, 31);
        ties = __shfl_sync(0xffffffffu, tb + lt, 31);
    }
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, int bf16, cudaStream_t stream, int num_sms,
                          size_t max_smem) {
    const RowPlan p = plan_rows(a.rows, a.V, bf16 ? 2 : 4, num_sms, max_smem - sizeof(Shared) - 1024);
    a.cs = p.cs;
    a.slice = (int)p.slice;
    if (bf16)
        return launch_rows(p.staged ? sample_kernel<__nv_bfloat16, true>
                                    : sample_kernel<__nv_bfloat16, false>,
                           a, a.rows, a.cs, p.slice, stream);
    return launch_rows(p.staged ? sample_kernel<float, true> : sample_kernel<float, false>, a,
                       a.rows, a.cs, p.slice, stream);
}

}  // namespace df2
