// Distillation from a teacher's top-K logits: the loss of every row, its
// gradient, or both in one pass over the student's logits.
//
//   q_k   = softmax over the row's K teacher logits / T   (id < 0: an empty slot)
//   lse   = log sum_j exp(z_j / T)
//   loss  = weight * sum_k q_k (log q_k - z[id_k] / T + lse)
//   dz_j  = weight * g * (exp(z_j / T - lse) - sum_{k: id_k = j} q_k) / T
//
// Bound by HBM: the logits are read once and the gradient is written once.  A CTA,
// or the CTAs of a cluster, take a row through the two uses of it (the sum of
// exponentials, then the gradient), which only a (max, sum) pair per warp crosses.
// 4096 x 151936 bf16 with the gradient (one row in eight of weight 0): 412 us, 5.7 TB/s;
// the loss alone of 512 x 262144 fp32: 91 us, 5.9 TB/s; the gradient alone of 1024 x
// 151936 bf16: 99 us, 5.9 TB/s (a copy on the same card: 6.8 TB/s).
//
// All exponentials are powers of two with c = log2(e)/T folded in: a slice's
// sum is taken against its own rounded base b = c * max, 2^(c*z - b) being one
// fused multiply-add and one ex2, and the same b goes into lse, so the rounding
// of b cancels.  The loss takes c * z - b the same way (in 64 bits, K terms).
// Where c * max is 2^24 or more (a row masked by a large number or the type's lowest value
// all over) the power is 2^((z - max) * c).
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "dflash2.h"
#include "rows.cuh"

namespace df2 {
namespace {

// Four CTAs of eight warps an SM and at most 160 KB of a row each: 4096 x 151936 bf16 with
// the gradient takes 412 us; 500 us with whole rows, whose second reading misses L2, 445 us
// with 80 KB, where the clusters' barriers cost more.  Rows of up to kNarrowBytes take
// CTAs of four warps, of which an SM holds eight (4096 x 1000 bf16 with the gradient: 48
// us, against 78 us).
using Wide = RowGeometry<256, 4, 6, 160>;
using Narrow = RowGeometry<128, 8, 5, 160>;
constexpr long long kNarrowBytes = 64 * 1024;

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename S>
__device__ __forceinline__ S warp_sum(S v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row's teacher entries in shared memory.
struct Teacher {
    int* id;     // token, -1 for an empty slot
    float* q;    // its share
    float* lq;   // log of it
    float* z;    // the student's logit there (this CTA's tokens only)
    __device__ __forceinline__ Teacher(char* at, int K) {
        id = reinterpret_cast<int*>(at);
        q = reinterpret_cast<float*>(at) + K;
        lq = q + K;
        z = lq + K;
    }
};

// A row's tokens, teacher logits and, for the tokens among elements [e_lo, e_hi), the
// student's logits, by one warp.  A token outside [0, V) is an empty slot; one that
// is not negative is flagged too.
template <typename T>
__device__ __forceinline__ void teacher_load(const Teacher& t, const DistillArgs& a, int row,
                                             const T* z, int e_lo, int e_hi, bool flag) {
    const int lane = threadIdx.x & 31;
    for (int k = lane; k < a.K; k += 32) {
        int id = a.ids[(long long)row * a.K + k];
        t.lq[k] = a.teacher[(long long)row * a.K + k];
        if (id < 0 || id >= a.V) {
            if (id >= a.V && flag && a.err_flag != nullptr) atomicOr(a.err_flag, DF2_FLAG_BAD_ID);
            id = -1;
        }
        t.id[k] = id;
        if (id >= e_lo && id < e_hi) t.z[k] = to_f32(z[id]);
    }
}

// Softmax of the loaded teacher logits by the same warp; returns 1, or 0 when the row
// has no entry with a share.
__device__ __forceinline__ float teacher_softmax(const Teacher& t, int K, float inv_t) {
    const int lane = threadIdx.x & 31;
    float m = neg_inf();
    bool nan = false;  // fmaxf drops it
    for (int k = lane; k < K; k += 32) {
        if (t.id[k] < 0) t.lq[k] = neg_inf();
        m = fmaxf(m, t.lq[k]);
        nan = nan || t.lq[k] != t.lq[k];
    }
    m = __any_sync(0xffffffffu, nan) ? __int_as_float(0x7fffffff) : warp_max(m);
    if (m == neg_inf()) {
        for (int k = lane; k < K; k += 32) t.q[k] = 0.f;
        return 0.f;
    }
    float s = 0.f;
    for (int k = lane; k < K; k += 32) s += expf((t.lq[k] - m) * inv_t);
    s = warp_sum(s);
    const float ls = logf(s);
    for (int k = lane; k < K; k += 32) {
        const float y = (t.lq[k] - m) * inv_t;
        t.q[k] = t.id[k] < 0 ? 0.f : expf(y) / s;
        t.lq[k] = y - ls;
    }
    return 1.f;
}

// 2^(c * z - base), base = c * max: rounded to fp32 and by a fused multiply-add, or
// with the maximum taken off first where the base is too large for that: the multiply-add
// leaves the base's rounding error in all exponents, which is half at most below 2^24, but
// leaves fp32's range for bases from 2^31 on (a row masked by -1e10 all over).
constexpr float kFastBase = 16777216.f;
struct Power {
    bool fast;
    float c, m, nb;  // the maximum (0 for -inf: every z is), -base
    __device__ __forceinline__ Power(float m_, float c_) : c(c_), m(m_ == neg_inf() ? 0.f : m_) {
        nb = -__fmul_rn(m, c);
        fast = fabsf(nb) < kFastBase;
    }
    __device__ __forceinline__ float operator()(float z) const {
        return ex2(fast ? fmaf(z, c, nb) : (z - m) * c);
    }
    // the powers of a vector's logits, in their place (fast)
    template <int N>
    __device__ __forceinline__ void of(f32x2 (&z)[N]) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float2 d = halves(fma2(z[j], pair(c, c), pair(nb, nb)));
            z[j] = pair(ex2(d.x), ex2(d.y));
        }
    }
    // 2^(another's base - base); a base that is not fast is the product itself, not rounded
    __device__ __forceinline__ float against(const Power& o) const {
        if (fast) return ex2(o.fast ? nb - o.nb : fmaf(o.m, c, nb));
        return ex2(o.fast ? -fmaf(m, c, o.nb) : (o.m - m) * c);
    }
    __device__ __forceinline__ double base() const { return fast ? -(double)nb : (double)m * c; }
    // c * z - base in 64 bits
    __device__ __forceinline__ double depth(float z) const {
        return fast ? (double)z * c + nb : ((double)z - m) * c;
    }
};

// The powers of a vector's logits against any base: their sum, or themselves times k as
// a vector.  Calls, so that the fast path stays free of them.
template <typename T>
__device__ __noinline__ float slow_sum(uint4 v, const Power p) {
    constexpr int E = VecOf<T>::kElems;
    float f[E], s = 0.f;
    unpack(v, f);
#pragma unroll
    for (int j = 0; j < E; ++j) s += p(f[j]);
    return s;
}
template <typename T>
__device__ __noinline__ uint4 slow_grad(uint4 v, const Power p, float k) {
    constexpr int E = VecOf<T>::kElems;
    float f[E];
    unpack(v, f);
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = p(f[j]) * k;
    return pack(f);
}

// A part of a row: a logit as base (not far below the largest; -inf where nothing is
// above that) and the sum of the powers against it.
struct alignas(8) MaxSum {  // goes to other CTAs as one 64-bit store
    float max, sum;
};

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// Writes vector v of a gradient row: one 16-byte store where it is whole and the
// gradient's row lies on the logits' grid, else element by element.
template <typename T>
__device__ __noinline__ void store_edge(const RowView<T> r, T* out, int v, const uint4 vec) {
    constexpr int E = VecOf<T>::kElems;
    const T* f = reinterpret_cast<const T*>(&vec);
    for (int j = 0; j < E; ++j) {
        const int e = v * E - r.head + j;
        if (e >= 0 && e < r.V) out[e] = f[j];
    }
}
template <typename T>
__device__ __forceinline__ void store_vec(const RowView<T>& r, T* out, bool wide, int v, int v_hi,
                                          const uint4& vec) {
    if (wide)
        __stcs(reinterpret_cast<uint4*>(out - r.head) + v, vec);
    else if (v < v_hi)
        store_edge(r, out, v, vec);
}

// Zeros to a warp's vectors [wlo, whi) of a gradient row.
template <typename T>
__device__ __forceinline__ void store_zeros(const RowView<T>& r, T* out, bool on_grid, int wlo,
                                            int whi) {
    for (int v = wlo + (int)(threadIdx.x & 31); v < whi; v += 32)
        store_vec<T>(r, out, on_grid && r.inner(v), v, whi, make_uint4(0, 0, 0, 0));
}

// Rewrites the gradient at the teacher's tokens among elements [e_lo, e_hi):
// (share(z) - sum of q over the slots of that token) * scale, by the first slot of
// each token, whose warp adds up the others in a fixed order.  Call after a barrier
// behind the plain writes.
template <typename G, typename T, typename F>
__device__ __forceinline__ void fix_tokens(const Teacher& t, int K, T* out, int e_lo, int e_hi,
                                           float scale, F share) {
    const int lane = threadIdx.x & 31;
    for (int k0 = threadIdx.x - lane; k0 < K; k0 += G::kThreads) {
        const int mine = k0 + lane < K ? t.id[k0 + lane] : -1;
        unsigned left = __ballot_sync(0xffffffffu, mine >= e_lo && mine < e_hi);
        while (left != 0) {
            const int k = k0 + __ffs(left) - 1;
            left &= left - 1;
            const int id = t.id[k];
            int first = K;
            float q = 0.f;
            for (int j = lane; j < K; j += 32) {
                if (t.id[j] != id) continue;
                first = min(first, j);
                q += t.q[j];
            }
            first = __reduce_min_sync(0xffffffffu, first);
            q = warp_sum(q);
            if (lane == 0 && first == k) out[id] = from_f32<T>((share(t.z[k]) - q) * scale);
        }
    }
}

// Joins n slices' (maximum, sum); every lane gets the result.
__device__ __forceinline__ MaxSum join(const MaxSum* ms, int n, float c) {
    const int lane = threadIdx.x & 31;
    float m = neg_inf(), s = 0.f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, ms[i].max);
    m = warp_max(m);
    const Power p(m, c);
    for (int i = lane; i < n; i += 32)
        s += ms[i].max == neg_inf() ? ms[i].sum : ms[i].sum * p.against(Power(ms[i].max, c));
    return {m, warp_sum(s)};
}

// A row by its cluster: lse and loss when LOSS, and the gradient, times `up`, when GRAD.
template <typename T, bool LOSS, bool GRAD, typename G>
__device__ __forceinline__ void whole_row(const DistillArgs& a, const RowView<T>& r,
                                          RowSlice<G>& sl, char* smem, int row, int rank, T* out,
                                          bool on_grid, float weight, float up) {
    constexpr int E = VecOf<T>::kElems;
    __shared__ MaxSum parts[kRowMaxCluster * G::kWarps];  // every warp of the row
    __shared__ float has_teacher;                         // 1 or 0

    const int cs = 1 << a.lg, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int e_lo = max(sl.lo * E - r.head, 0), e_hi = min(sl.hi * E - r.head, a.V);
    if (cs > 1) cluster_arrive();  // met by cluster_wait below: every CTA has started

    sl.start(r);
    const Teacher t(smem, a.K);
    // rank 0, which makes the loss, needs z at all of the teacher's tokens
    if (warp == G::kWarps - 1)
        teacher_load(t, a, row, r.row, LOSS && rank == 0 ? 0 : e_lo,
                     LOSS && rank == 0 ? a.V : e_hi, rank == 0);
    // The warp's sum of powers against the largest logit of its first vectors: fp32 has
    // room for sums 2^66 times above that.  Where one was larger (or the base was -inf,
    // or a NaN is among them), once more against the largest of all.
    float m = neg_inf(), s;
    {
        bool first = true;
        Power pw(m, a.c);
        f32x2 sums[2] = {};
        sl.pass(r, [&](int, const uint4& v, bool) {
            if (first) {
                m = warp_max(vec_max<T>(v));
                pw = Power(m, a.c);
                first = false;
            }
            f32x2 f[E / 2];
            unpack(v, f);
            pw.of(f);
#pragma unroll
            for (int j = 0; j < E / 2; ++j) sums[j & 1] = add2(sums[j & 1], f[j]);
        });
        const float2 lanes = halves(add2(sums[0], sums[1]));
        s = warp_sum(lanes.x + lanes.y);
        if (!(m > neg_inf() && pw.fast && s < 1e20f) && sl.steps > 0) {
            m = neg_inf();
            sl.pass(r, [&](int, const uint4& v, bool) { m = fmaxf(m, vec_max<T>(v)); });
            m = warp_max(m);
            const Power slow(m, a.c);
            s = 0.f;
            sl.pass(r, [&](int, const uint4& v, bool) { s += slow_sum<T>(v, slow); });
            s = warp_sum(s);
        }
    }
    const int me = rank * G::kWarps + warp;
    if (cs > 1) {
        cluster_wait();
        if (lane < cs)
            st_cluster_b64(map_cluster(smem_u32(&parts[me]), lane),
                           __builtin_bit_cast(uint64_t, MaxSum{m, s}));
        __syncwarp();
        cluster_arrive();
    } else if (lane == 0) {
        parts[me] = {m, s};
    }
    if (warp == G::kWarps - 1) {
        const float q = teacher_softmax(t, a.K, a.inv_t);
        if (lane == 0) has_teacher = q;
    }
    if (cs > 1) {
        __syncwarp();
        cluster_wait();  // no CTA's shared memory is touched from outside after this
    }
    __syncthreads();
    const MaxSum all = join(parts, cs * G::kWarps, a.c);
    const Power pg(all.max, a.c);
    const float S = all.sum;
    if (LOSS && rank == 0 && warp == G::kWarps - 1) {
        const float ls = log2f(S);
        double loss = 0;
        for (int k = lane; k < a.K; k += 32)
            if (t.q[k] != 0.f)
                loss += (double)t.q[k] * (t.lq[k] - (double)kLn2 * (pg.depth(t.z[k]) - ls));
        loss = warp_sum(loss);
        if (lane == 0) {
            // no logit above -inf: the student gives the teacher's tokens no share
            if (S == 0.f) loss = has_teacher == 0.f ? 0.0 : (double)INFINITY;
            a.loss[row] = (float)(weight * loss);
            a.lse[row] = S == 0.f ? neg_inf() : (float)((double)kLn2 * (pg.base() + ls));
        }
    }
    if (GRAD) {
        if (has_teacher == 0.f) {  // whatever the logits are, a NaN too
            store_zeros<T>(r, out, on_grid, sl.wlo, sl.whi);
            return;
        }
        const float scale = up * weight * a.inv_t;
        const float per_s = S == 0.f ? 0.f : 1.f / S;
        const float k = scale * per_s;
        sl.hint = l2_policy_evict_first();
        if (pg.fast && on_grid) {
            uint4* const at = reinterpret_cast<uint4*>(out - r.head);
            sl.pass(r, [&](int v, const uint4& vec, bool whole) {
                f32x2 f[E / 2];
                unpack(vec, f);
                pg.of(f);
#pragma unroll
                for (int j = 0; j < E / 2; ++j) f[j] = mul2(f[j], pair(k, k));
                if (whole)
                    __stcs(at + v, pack_pairs(f));
                else if (v < sl.whi)
                    store_edge(r, out, v, pack_pairs(f));
            });
        } else {
            sl.pass(r, [&](int v, const uint4& vec, bool whole) {
                store_vec<T>(r, out, whole && on_grid, v, sl.whi, slow_grad<T>(vec, pg, k));
            });
        }
        __syncthreads();
        fix_tokens<G, T>(t, a.K, out, e_lo, e_hi, scale, [&](float z) { return pg(z) * per_s; });
    }
}

// One cluster per row: lse and loss, and the gradient when GRAD.
template <typename T, bool GRAD, typename G>
__global__ void __launch_bounds__(G::kThreads, G::kCtas) distill_kernel(DistillArgs a) {
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, rank = a.lg > 0 ? (int)cluster_ctarank() : 0;
    const int row = blockIdx.x >> a.lg;
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, tid >> 5, smem + (size_t)a.K * 16,
                   GRAD ? l2_policy_evict_last() : l2_policy_evict_first());
    T* out = GRAD ? static_cast<T*>(a.grad) + (long long)row * a.grad_ld : nullptr;
    const bool on_grid =
        GRAD &&
        ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.row)) & 15u) == 0;
    const float weight = a.weight != nullptr ? a.weight[row] : 1.f;
    if (weight == 0.f) {  // the whole cluster leaves: the row's logits are not read
        if (GRAD) store_zeros<T>(r, out, on_grid, sl.wlo, sl.whi);
        if (rank == 0 && tid == 0) {
            a.loss[row] = 0.f;
            a.lse[row] = 0.f;
        }
        return;
    }
    whole_row<T, true, GRAD, G>(a, r, sl, smem, row, rank, out, on_grid, weight, 1.f);
}

// The gradient alone of a row whose lse is far from 0: its sum is taken again (1024 x 151936
// bf16 from HBM, all rows so: 142 us, 108 with the given lse).  A call, so that other rows keep
// their registers.
template <typename T, typename G>
__device__ __noinline__ void far_row(const DistillArgs& a, char* smem, float weight, float up) {
    const int row = blockIdx.x >> a.lg, rank = a.lg > 0 ? (int)cluster_ctarank() : 0;
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, threadIdx.x >> 5, smem + (size_t)a.K * 16,
                   l2_policy_evict_last());
    T* out = static_cast<T*>(a.grad) + (long long)row * a.grad_ld;
    const bool on_grid =
        ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.row)) & 15u) == 0;
    whole_row<T, false, true, G>(a, r, sl, smem, row, rank, out, on_grid, weight, up);
}

// The gradient alone, from lse and the upstream gradient: the CTAs of a row do not
// wait on one another, unless |lse| is kFarLse or more.  exp(z / T - lse) is off by half a unit
// of lse, 2^-17 below 256, and by the rounding of log2(e) / T behind lse, 2^-16 there at most; at
// 1e4 the first is 5e-4, and a row masked by the type's lowest value all over has an lse that
// holds nothing of its sum (or none in fp32's range, with T < 1).
constexpr float kFarLse = 256.f;
template <typename T, typename G>
__global__ void __launch_bounds__(G::kThreads, G::kCtas)
    distill_grad_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int E = VecOf<T>::kElems;
    extern __shared__ __align__(16) char smem[];
    __shared__ float has_teacher;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x >> a.lg, rank = blockIdx.x & ((1 << a.lg) - 1);
    const RowView<T> r(a.logits, a.ld, row, a.V);
    RowSlice<G> sl(r, a.per, a.ring, rank, warp, smem + (size_t)a.K * 16,
                   l2_policy_evict_first());
    const int e_lo = max(sl.lo * E - r.head, 0), e_hi = min(sl.hi * E - r.head, a.V);
    T* out = static_cast<T*>(a.grad) + (long long)row * a.grad_ld;
    const bool on_grid =
        ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(r.row)) & 15u) == 0;
    const float weight = a.weight != nullptr ? a.weight[row] : 1.f;
    const float up = a.grad_loss[row];
    if (weight == 0.f || up == 0.f) {
        store_zeros<T>(r, out, on_grid, sl.wlo, sl.whi);
        return;
    }
    const float lse = a.lse[row];
    if (fabsf(lse) >= kFarLse) {  // the same in all CTAs of the row
        far_row<T, G>(a, smem, weight, up);
        return;
    }
    sl.start(r);
    const Teacher t(smem, a.K);
    if (warp == 0) {
        teacher_load(t, a, row, r.row, e_lo, e_hi, rank == 0);
        const float q = teacher_softmax(t, a.K, a.inv_t);
        if (lane == 0) has_teacher = q;
    }
    __syncthreads();  // also: z is read before the gradient may take its place
    const float scale = up * weight * a.inv_t;
    const bool none = has_teacher == 0.f;
    auto share = [&](float z) { return ex2(fmaf(z, a.inv_t, -lse) * kLog2e); };
    const float k = none ? 0.f : scale;
    const f32x2 it = pair(a.inv_t, a.inv_t), nl = pair(-lse, -lse), le = pair(kLog2e, kLog2e);
    sl.pass(r, [&](int v, const uint4& vec, bool whole) {
        f32x2 f[E / 2];
        unpack(vec, f);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 d = halves(mul2(fma2(f[j], it, nl), le));
            f[j] = mul2(pair(ex2(d.x), ex2(d.y)), pair(k, k));
        }
        store_vec<T>(r, out, whole && on_grid, v, sl.whi,
                     k == 0.f ? make_uint4(0, 0, 0, 0) : pack_pairs(f));
    });
    if (none) return;
    __syncthreads();
    fix_tokens<G, T>(t, a.K, out, e_lo, e_hi, scale, share);
}

template <typename T, typename G>
cudaError_t launch_typed(DistillArgs a, cudaStream_t stream, int num_sms) {
    const RowSplit p = split_rows<G>(a.rows, a.V, sizeof(T), num_sms);
    a.lg = p.lg;
    a.per = p.per;
    a.ring = p.ring;
    const size_t smem = p.smem + (size_t)a.K * 16;
    constexpr size_t kMost = G::kRingBytes + (size_t)kDistillMaxK * 16;
    if (a.grad_loss != nullptr)
        return launch_rows<G, distill_grad_kernel<T, G>>(a, a.rows, p.lg, smem, kMost, stream);
    if (a.grad != nullptr)
        return launch_rows<G, distill_kernel<T, true, G>>(a, a.rows, p.lg, smem, kMost, stream);
    return launch_rows<G, distill_kernel<T, false, G>>(a, a.rows, p.lg, smem, kMost, stream);
}

}  // namespace

cudaError_t launch_distill(DistillArgs a, int bf16, cudaStream_t stream, int num_sms) {
    const bool narrow = (long long)a.V * (bf16 ? 2 : 4) <= kNarrowBytes;
    if (bf16)
        return narrow ? launch_typed<__nv_bfloat16, Narrow>(a, stream, num_sms)
                      : launch_typed<__nv_bfloat16, Wide>(a, stream, num_sms);
    return narrow ? launch_typed<float, Narrow>(a, stream, num_sms)
                  : launch_typed<float, Wide>(a, stream, num_sms);
}

}  // namespace df2
