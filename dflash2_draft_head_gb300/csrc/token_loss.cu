// Losses of a token's log-probability on whole vocabulary rows, and their gradients: the
// clipped policy loss with a KL term, and the preference loss of pairs of sequences.
//
//   lse  = log sum_j exp(z_j / T),  logp = z_t / T - lse          (t the row's token)
//   dz_j = g * ((j == t) - exp(z_j / T - lse)) / T                (g = d loss / d logp)
//
// policy, by row:  rho = exp(logp - old),  d = ref - logp
//   loss = weight * (kl_coef * (exp(d) - d - 1) - min(rho * A, clamp(rho, lo, hi) * A))
// preference, by pair: S the sum (or mean) of logp over a sequence's rows with a token,
//   m = beta * ((S_c - R_c) - (S_r - R_r)) - margin
//   loss = weight * ((1 - e) * log(1 + exp(-m)) + e * log(1 + exp(m)))
//
// Bound by HBM.  The policy's g needs nothing but its own row: loss and gradient take the
// row through both uses of it while it is in L2, as distillation does.  A pair's g needs all
// rows of both sequences first: one pass over the rows for logp and lse, a kernel over
// the pairs, and a pass that writes the gradient from lse, each scheduled while the one before it
// ends.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "dflash2.h"
#include "softmax_rows.cuh"

namespace df2 {
namespace {

enum class Loss { kPolicy, kPreference };

// How a kernel takes wide rows.  Loss and gradient in one call read a row twice, the second time
// from the ring and L2: three CTAs an SM with slices of 200 KB keep about 70 MB of rows under way
// (4096 x 151936 bf16: 373 us; 408 with four CTAs, whose rows do not stay in L2, 438 with whole
// rows).  One reading wants few splits: slices of 640 KB (the loss of 1024 x 151936 bf16 45 us, of
// 512 x 262144 fp32 84 us; 47 and 88 with 160 KB, 59 and 132 with 80 KB).
using Twice = RowGeometry<256, 3, 9, 200>;
using Once = RowGeometry<256, 4, 6, 640>;

// Of the rows that a call reads twice in two passes, the last ones stay in L2 for the second pass,
// which goes backwards: 2048 x 151936 bf16, all with a token, with the gradient 282 us, 289 without;
// 400 rows 64 and 70 (with 96 MB 283 and 64).
constexpr long long kKeepBytes = 64ll << 20;

// As split_rows, but few rows are split only as far as their CTAs run all at once: the meetings of
// a cluster cost more than shorter slices bring where a second wave follows (64 x 151936 bf16 with
// the gradient 13.2 us, 20 without this; 100 rows 17.0 and 25).
template <typename G>
RowSplit split_fitting(int rows, int V, size_t es, int num_sms) {
    const long long vecs = row_max_vecs(V, es), bytes = vecs * 16;
    int lg = 0;
    while (lg < 3 && (long long)rows << (lg + 1) <= (long long)G::kCtas * num_sms &&
           bytes >> lg > kRowSliceMin)
        ++lg;
    while (1 << lg < kRowMaxCluster && bytes >> lg > G::kSliceBytes) ++lg;
    const int per = (int)((vecs + (1 << lg) - 1) >> lg), ring = G::ring_steps(per);
    return {lg, per, ring, ring * G::kStepBytes};
}

struct TokenGrad {
    float loss;  // without the row's weight
    float g;     // d loss / d logp, likewise
};

// The policy loss of one token.  A = 0 takes the ratio's term out, kl_coef = 0 the other,
// also where they are infinite; a NaN in logp stays visible.
__device__ __forceinline__ TokenGrad policy(const TokenLossArgs& a, int row, float logp) {
    const float A = a.advantage[row], rho = expf(logp - a.old_logp[row]);
    TokenGrad t = {0.f, 0.f};
    if (A != 0.f) {
        const bool inside = A > 0.f ? !(rho > a.ratio_hi) : !(rho < a.ratio_lo);
        t.loss = inside ? -rho * A : -(A > 0.f ? a.ratio_hi : a.ratio_lo) * A;
        t.g = inside ? t.loss : 0.f;
    }
    if (a.kl_coef != 0.f) {
        const float d = a.ref_logp[row] - logp, e = expm1f(d);
        // both infinite for a token of no share under the head, whose d - d is not a number
        t.loss += a.kl_coef * (e == INFINITY ? e : e - d);
        t.g -= a.kl_coef * e;
    }
    return t;
}

// The number of offsets[0..n) that are not above `row`, by a warp: a search that looks at 32 of
// them a turn.  Whatever they hold, it looks at none outside and ends.
__device__ __forceinline__ int offsets_upto(const int* offsets, int n, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 0) {
        const int step = (n + 31) / 32, at = (lane + 1) * step - 1;
        const unsigned up = __ballot_sync(0xffffffffu, at < n && offsets[lo + at] <= row);
        const int parts = up == 0xffffffffu ? 32 : __ffs(~up) - 1;
        lo += parts * step;
        n = min(step - 1, n - parts * step);
    }
    return lo;
}

__device__ __forceinline__ int clamp_row(int v, int rows) { return min(max(v, 0), rows); }

// A pair's m for the gradient: from the sums as they are returned, in fp32 (the loss takes those in
// 64 bits), so that the call with the loss and the gradient alone give the same bits.  Off by up to
// beta * 2^-22 of the sums' and references' magnitudes.
__device__ __forceinline__ float pair_margin(const TokenLossArgs& a, int i) {
    float c = a.seq_logp[i], r = a.seq_logp[a.pairs + i];
    if (a.ref_logp != nullptr) {
        c -= a.ref_logp[i];
        r -= a.ref_logp[a.pairs + i];
    }
    return fmaf(a.beta, c - r, -a.margin);
}
// d loss / d S of a pair's chosen sequence, without the weight (the rejected one's: minus that).
__device__ __forceinline__ float pair_slope(const TokenLossArgs& a, float m) {
    float s = (1.f - a.smoothing) / (1.f + expf(m));
    if (a.smoothing != 0.f) s -= a.smoothing / (1.f + expf(-m));
    return -a.beta * s;
}

// Rows of [lo, hi) with a token, by the whole block; every thread gets the number.  Every CTA of a
// row counts its sequence, a block's meeting for THREADS rows: with means the work grows with the
// square of a sequence's length (two sequences of 8192 rows x 32000 bf16 with the gradient 595 us,
// 469 with sums; four of 1000 rows 129 and 123).
template <int THREADS>
__device__ __forceinline__ int count_tokens(const TokenLossArgs& a, int lo, int hi) {
    int n = 0;
    for (int r = lo; r < hi; r += THREADS) {
        const int row = r + (int)threadIdx.x;
        const int t = row < hi ? a.tokens[row] : -1;
        n += __syncthreads_count(t >= 0 && t < a.V);
    }
    return n;
}

// What a row's or pair's gradient is multiplied by, its weight and the gradient by its loss: 0 where
// one of them is, whatever the other one is.
__device__ __forceinline__ float loss_factor(const TokenLossArgs& a, int i) {
    const float w = a.weight != nullptr ? a.weight[i] : 1.f;
    const float up = a.grad_loss != nullptr ? a.grad_loss[i] : 1.f;
    return w == 0.f || up == 0.f ? 0.f : w * up;
}

// g of a row of a sequence, by the whole block: the same in all CTAs of the row.
template <typename G>
__device__ __forceinline__ float sequence_slope(const TokenLossArgs& a, int row) {
    const int n = 2 * a.pairs, s = offsets_upto(a.offsets, n + 1, row) - 1;
    if (s < 0 || s >= n) return 0.f;
    const int start = clamp_row(a.offsets[s], a.rows), end = clamp_row(a.offsets[s + 1], a.rows);
    const int i = s < a.pairs ? s : s - a.pairs;
    const float m = pair_margin(a, i), w = loss_factor(a, i);
    if (w == 0.f || row < start || row >= end) return 0.f;
    float g = w * pair_slope(a, m);
    if (s >= a.pairs) g = -g;
    if (a.average) g /= (float)count_tokens<G::kThreads>(a, start, end);
    return g;
}

// The gradient at the row's token, behind the pass that wrote the shares.
template <typename T>
__device__ __forceinline__ void write_token(T* out, int token, int e_lo, int e_hi, float v) {
    if (threadIdx.x == 0 && token >= e_lo && token < e_hi) out[token] = from_f32<T>(v);
}

// A row's token; -1 where it has none (flagged, when it is not negative).
__device__ __forceinline__ int row_token(const TokenLossArgs& a, int row, bool flag) {
    const int t = a.tokens[row];
    if (t < a.V) return t;
    if (flag && a.err_flag != nullptr) atomicOr(a.err_flag, DF2_FLAG_BAD_ID);
    return -1;
}

template <typename T>
struct Out {  // a row of the gradient
    T* row;
    bool on_grid;  // its vectors lie as the logits'
    __device__ __forceinline__ Out(const TokenLossArgs& a, int r, const T* logits) {
        row = static_cast<T*>(a.grad) + (long long)r * a.grad_ld;
        on_grid =
            ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(logits)) & 15u) == 0;
    }
};

// The sum of a row's powers, by its cluster.  `inside` is called between the cluster's meetings.
template <typename T, typename G, typename F>
__device__ __forceinline__ MaxSum row_sum(const TokenLossArgs& a, const RowView<T>& r,
                                          RowSlice<G>& sl, int rank, F inside) {
    __shared__ MaxSum parts[kRowMaxCluster * G::kWarps];  // every warp of the row
    const int cs = 1 << a.lg, warp = threadIdx.x >> 5;
    if (cs > 1) cluster_arrive();  // met by cluster_wait below: every CTA has started
    sl.start(r);
    inside();
    const MaxSum mine = warp_part<T>(r, sl, a.c);
    if (cs > 1) cluster_wait();
    publish(parts, rank * G::kWarps + warp, mine, cs);
    if (cs > 1) cluster_wait();  // no CTA's shared memory is touched from outside after this
    __syncthreads();
    return join(parts, cs * G::kWarps, a.c);
}

// log of the share of a logit, ls = log2 of the powers' sum.  A token at the type's lowest value
// leaves fp32's range in powers of two before it does in those of e; ls is nothing beside it.
// Rounding does not take it above 0.
__device__ __forceinline__ float log_share(const TokenLossArgs& a, const Power& pg, float z,
                                           float ls) {
    const float depth = pg.fast ? fmaf(z, a.c, pg.nb) : (z - pg.m) * a.c;
    if (depth == neg_inf()) return (z - pg.m) * a.inv_t;
    return depth > ls ? 0.f : kLn2 * (depth - ls);
}

// logp and lse of every row, and for the policy its loss and, when GRAD, its gradient.
template <typename T, Loss L, bool GRAD, typename G>
__global__ void __launch_bounds__(G::kThreads, G::kCtas)
    token_loss_kernel(const __grid_constant__ TokenLossArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    if (L == Loss::kPreference) griddep_launch_dependents();
    const int tid = threadIdx.x, rank = a.lg > 0 ? (int)cluster_ctarank() : 0;
    const int row = blockIdx.x >> a.lg;
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, tid >> 5, smem,
                   GRAD || row >= a.rows - a.keep ? l2_policy_evict_last()
                                                  : l2_policy_evict_first());
    const Out<T> out(a, row, r.row);
    const int token = row_token(a, row, rank == 0 && tid == 0);
    const float weight = L == Loss::kPolicy && a.weight != nullptr ? a.weight[row] : 1.f;
    if (token < 0 || weight == 0.f) {  // the whole cluster leaves: the row's logits are not read
        if (GRAD) store_zeros<T>(r, out.row, out.on_grid, sl.wlo, sl.whi);
        if (rank == 0 && tid == 0) {
            if (L == Loss::kPolicy) a.loss[row] = 0.f;
            a.logp[row] = 0.f;
            a.lse[row] = 0.f;
        }
        return;
    }
    float z = 0.f;  // read ahead of the meeting that the first store waits for: in place works
    const MaxSum all = row_sum<T, G>(a, r, sl, rank, [&] { z = to_f32(r.row[token]); });
    const Power pg(all.max, a.c);
    const float S = all.sum, ls = log2f(S);
    // no logit above -inf: a softmax that is 0 everywhere
    const float logp = S == 0.f ? neg_inf() : log_share(a, pg, z, ls);
    TokenGrad t = {0.f, 0.f};
    if (L == Loss::kPolicy) t = policy(a, row, logp);
    if (rank == 0 && tid == 0) {
        if (L == Loss::kPolicy) a.loss[row] = weight * t.loss;
        a.logp[row] = logp;
        a.lse[row] = S == 0.f ? neg_inf() : (float)((double)kLn2 * (pg.base() + ls));
    }
    if (!GRAD) return;
    const float scale = weight * t.g * a.inv_t;
    if (scale == 0.f) {
        store_zeros<T>(r, out.row, out.on_grid, sl.wlo, sl.whi);
        return;
    }
    const float per_s = S == 0.f ? 0.f : 1.f / S;
    write_shares<T>(r, sl, pg, -scale * per_s, out.row, out.on_grid);
    __syncthreads();
    write_token(out.row, token, max(sl.lo * E - r.head, 0), min(sl.hi * E - r.head, a.V),
                (1.f - pg(z) * per_s) * scale);
}

// The row of a CTA of the gradient's pass.  Behind a pass for logp and lse in the same call it goes
// backwards: the last rows of that one are still in L2.
template <Loss L>
__device__ __forceinline__ int row_of(const TokenLossArgs& a) {
    const int row = blockIdx.x >> a.lg;
    return L == Loss::kPreference && a.grad_loss == nullptr ? a.rows - 1 - row : row;
}

// The gradient alone of a row whose lse is far from 0: its sum is taken again.  A call, so that
// other rows keep their registers.
template <typename T, Loss L, typename G>
__device__ __noinline__ void far_row(const TokenLossArgs& a, char* smem, int token, float scale) {
    constexpr int E = VecOf<T>::kElems;
    const int row = row_of<L>(a), rank = a.lg > 0 ? (int)cluster_ctarank() : 0;
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, threadIdx.x >> 5, smem, l2_policy_evict_last());
    const Out<T> out(a, row, r.row);
    float z = 0.f;
    const MaxSum all = row_sum<T, G>(a, r, sl, rank, [&] { z = to_f32(r.row[token]); });
    const Power pg(all.max, a.c);
    const float per_s = all.sum == 0.f ? 0.f : 1.f / all.sum;
    write_shares<T>(r, sl, pg, -scale * per_s, out.row, out.on_grid);
    __syncthreads();
    write_token(out.row, token, max(sl.lo * E - r.head, 0), min(sl.hi * E - r.head, a.V),
                (1.f - pg(z) * per_s) * scale);
}

// The gradient alone, from lse and g: the CTAs of a row do not wait on one another, unless
// |lse| is kFarLse or more.
template <typename T, Loss L, typename G>
__global__ void __launch_bounds__(G::kThreads, G::kCtas)
    token_grad_kernel(const __grid_constant__ TokenLossArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    if (L == Loss::kPreference) griddep_wait();
    const int tid = threadIdx.x;
    const int row = row_of<L>(a), rank = blockIdx.x & ((1 << a.lg) - 1);
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, tid >> 5, smem, l2_policy_evict_first());
    const Out<T> out(a, row, r.row);
    const int token = row_token(a, row, rank == 0 && tid == 0);
    const float w = L == Loss::kPolicy && token >= 0 ? loss_factor(a, row) : 1.f;
    if (token < 0 || w == 0.f) {  // the row's logits are not read
        store_zeros<T>(r, out.row, out.on_grid, sl.wlo, sl.whi);
        return;
    }
    sl.start(r);  // ahead of the slope, which takes several loads that wait for one another
    const float lse = a.lse[row];
    const float scale = (L == Loss::kPolicy ? w * policy(a, row, a.logp[row]).g
                                            : sequence_slope<G>(a, row)) * a.inv_t;
    if (scale == 0.f || fabsf(lse) >= kFarLse) {  // the same in all CTAs of the row
        cp_async_wait_all();
        if (scale == 0.f)
            store_zeros<T>(r, out.row, out.on_grid, sl.wlo, sl.whi);
        else
            far_row<T, L, G>(a, smem, token, scale);
        return;
    }
    const int e_lo = max(sl.lo * E - r.head, 0), e_hi = min(sl.hi * E - r.head, a.V);
    const bool mine = tid == 0 && token >= e_lo && token < e_hi;
    const float z = mine ? to_f32(r.row[token]) : 0.f;
    __syncthreads();  // z is read before the gradient may take its place
    write_shares_lse<T>(r, sl, a.inv_t, lse, -scale, out.row, out.on_grid);
    __syncthreads();
    write_token(out.row, token, e_lo, e_hi, (1.f - share_by_lse(z, a.inv_t, lse)) * scale);
}

// The sums of every sequence and the loss of every pair, one CTA a pair: in 64 bits and in an
// order of the sequence's own, the same every time.
constexpr int kPairThreads = 256, kSequenceThreads = kPairThreads / 2;
constexpr int kSequenceWarps = kSequenceThreads / 32;
__global__ void __launch_bounds__(kPairThreads)
    pair_loss_kernel(const __grid_constant__ TokenLossArgs a) {
    __shared__ double sums[2 * kSequenceWarps];
    __shared__ int counts[2 * kSequenceWarps];
    griddep_launch_dependents();
    // half of the threads to each sequence; what the pass over the rows does not write comes first
    const int i = blockIdx.x, tid = threadIdx.x, half = tid / kSequenceThreads;
    const int s = i + half * a.pairs, start = a.offsets[s], end = a.offsets[s + 1];
    const float weight = a.weight != nullptr ? a.weight[i] : 1.f;
    const float ref_c = a.ref_logp != nullptr ? a.ref_logp[i] : 0.f;
    const float ref_r = a.ref_logp != nullptr ? a.ref_logp[a.pairs + i] : 0.f;
    griddep_wait();
    if (tid % kSequenceThreads == 0 && a.err_flag != nullptr &&
        (start < 0 || end < start || end > a.rows))
        atomicOr(a.err_flag, DF2_FLAG_BAD_ID);
    const int lo = clamp_row(start, a.rows), hi = clamp_row(end, a.rows);
    double sum = 0;
    int n = 0;
    for (int row = lo + tid % kSequenceThreads; row < hi; row += kSequenceThreads) {
        sum += a.logp[row];
        if (a.average) {
            const int t = a.tokens[row];
            n += t >= 0 && t < a.V;
        }
    }
    sum = warp_sum(sum);
    n = warp_sum(n);
    if ((tid & 31) == 0) {
        sums[tid >> 5] = sum;
        counts[tid >> 5] = n;
    }
    __syncthreads();
    if (tid != 0) return;
    double d[2];  // the margin comes from the sums before they are rounded
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        double all = 0;
        int rows = 0;
        for (int w = k * kSequenceWarps; w < (k + 1) * kSequenceWarps; ++w) {
            all += sums[w];
            rows += counts[w];
        }
        if (a.average) all /= max(rows, 1);
        a.seq_logp[i + k * a.pairs] = (float)all;
        d[k] = all - (k == 0 ? ref_c : ref_r);
    }
    const float m = (float)(a.beta * (d[0] - d[1]) - a.margin);
    auto softplus = [](float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); };
    float loss = 0.f;  // a term with no weight is left out, also where it is infinite
    if (a.smoothing != 1.f) loss = (1.f - a.smoothing) * softplus(-m);
    if (a.smoothing != 0.f) loss += a.smoothing * softplus(m);
    a.loss[i] = weight == 0.f ? 0.f : weight * loss;
}

template <typename T, Loss L, typename ONCE, typename TWICE>
cudaError_t launch_typed(TokenLossArgs a, TokenLossPass pass, cudaStream_t stream, int num_sms) {
    const auto take = [&](const RowSplit& p) {
        a.lg = p.lg;
        a.per = p.per;
        a.ring = p.ring;
        return (size_t)p.smem;
    };
    if (pass == TokenLossPass::kGrad) {  // the CTAs of a row do not meet
        const size_t smem = take(split_rows<ONCE>(a.rows, a.V, sizeof(T), num_sms));
        return launch_rows<ONCE, token_grad_kernel<T, L, ONCE>>(
            a, a.rows, a.lg, smem, ONCE::kRingBytes, stream, a.grad_loss == nullptr);
    }
    if (L == Loss::kPolicy && a.grad != nullptr) {
        const size_t smem = take(split_fitting<TWICE>(a.rows, a.V, sizeof(T), num_sms));
        return launch_rows<TWICE, token_loss_kernel<T, Loss::kPolicy, true, TWICE>>(
            a, a.rows, a.lg, smem, TWICE::kRingBytes, stream);
    }
    const size_t smem = take(split_fitting<ONCE>(a.rows, a.V, sizeof(T), num_sms));
    return launch_rows<ONCE, token_loss_kernel<T, L, false, ONCE>>(a, a.rows, a.lg, smem,
                                                                   ONCE::kRingBytes, stream);
}

template <Loss L>
cudaError_t launch_pass(const TokenLossArgs& a, TokenLossPass pass, int bf16, cudaStream_t stream,
                        int num_sms) {
    const bool narrow = (long long)a.V * (bf16 ? 2 : 4) <= kNarrowBytes;
    if (bf16)
        return narrow ? launch_typed<__nv_bfloat16, L, Narrow, Narrow>(a, pass, stream, num_sms)
                      : launch_typed<__nv_bfloat16, L, Once, Twice>(a, pass, stream, num_sms);
    return narrow ? launch_typed<float, L, Narrow, Narrow>(a, pass, stream, num_sms)
                  : launch_typed<float, L, Once, Twice>(a, pass, stream, num_sms);
}

}  // namespace

cudaError_t launch_policy_loss(const TokenLossArgs& a, TokenLossPass pass, int bf16,
                               cudaStream_t stream, int num_sms) {
    return launch_pass<Loss::kPolicy>(a, pass, bf16, stream, num_sms);
}

cudaError_t launch_preference_loss(const TokenLossArgs& a, TokenLossPass pass, int bf16,
                                   cudaStream_t stream, int num_sms) {
    if (pass == TokenLossPass::kLoss) {
        if (a.rows > 0) {
            TokenLossArgs first = a;
            if (a.grad != nullptr)
                first.keep = (int)std::min<long long>(
                    a.rows, kKeepBytes / ((long long)a.V * (bf16 ? 2 : 4)));
            const cudaError_t e =
                launch_pass<Loss::kPreference>(first, pass, bf16, stream, num_sms);
            if (e != cudaSuccess) return e;
        }
        if (a.pairs > 0) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr = {};
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
            cfg.gridDim = dim3((unsigned)a.pairs);
            cfg.blockDim = dim3(kPairThreads);
            cfg.stream = stream;
            cfg.attrs = &attr;
            cfg.numAttrs = a.rows > 0 ? 1 : 0;  // ahead of the pass over the rows, of nothing else
            const cudaError_t e = cudaLaunchKernelEx(&cfg, pair_loss_kernel, a);
            if (e != cudaSuccess) return e;
        }
        if (a.grad == nullptr) return cudaSuccess;
    }
    if (a.rows == 0) return cudaSuccess;
    return launch_pass<Loss::kPreference>(a, TokenLossPass::kGrad, bf16, stream, num_sms);
}

}  // namespace df2
