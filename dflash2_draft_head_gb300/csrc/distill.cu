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
#include "softmax_rows.cuh"

namespace df2 {
namespace {

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
    const MaxSum mine = warp_part<T>(r, sl, a.c);
    if (cs > 1) cluster_wait();
    publish(parts, rank * G::kWarps + warp, mine, cs);
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
        write_shares<T>(r, sl, pg, k, out, on_grid);
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
// wait on one another, unless |lse| is kFarLse or more.
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
    auto share = [&](float z) { return share_by_lse(z, a.inv_t, lse); };
    const float k = none ? 0.f : scale;
    write_shares_lse<T>(r, sl, a.inv_t, lse, k, out, on_grid);
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
