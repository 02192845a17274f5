// The softmax of a vocabulary row and its gradient, shared by the operators that need
// one (distillation, the policy and preference losses): the sum of exponentials of a row
// that is split over warps and CTAs, and the pass that writes shares of it.
//
// All exponentials are powers of two with c = log2(e)/T folded in, against a base near
// the largest logit of the part that a warp works on.
#pragma once

#include <cstdint>

#include "rows.cuh"

namespace df2 {

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

// The part of a row that a warp works on: its sum of powers against the largest logit of its
// first vectors: fp32 has room for sums 2^66 times above that.  Where one was larger (or the
// base was -inf, or a NaN is among them), once more against the largest of all.
template <typename T, typename G>
__device__ __forceinline__ MaxSum warp_part(const RowView<T>& r, RowSlice<G>& sl, float c) {
    constexpr int E = VecOf<T>::kElems;
    float m = neg_inf(), s;
    {
        bool first = true;
        Power pw(m, c);
        f32x2 sums[2] = {};
        sl.pass(r, [&](int, const uint4& v, bool) {
            if (first) {
                m = warp_max(vec_max<T>(v));
                pw = Power(m, c);
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
            const Power slow(m, c);
            s = 0.f;
            sl.pass(r, [&](int, const uint4& v, bool) { s += slow_sum<T>(v, slow); });
            s = warp_sum(s);
        }
    }
    return {m, s};
}

// Gives a warp's part (the me-th of its row) to all CTAs of the row.  In a cluster (cs > 1)
// call between the cluster's first meeting, after which every CTA has started, and the
// second, at which the parts are there; this arrives at the second.  Alone: a block barrier.
__device__ __forceinline__ void publish(MaxSum* parts, int me, const MaxSum& part, int cs) {
    const int lane = threadIdx.x & 31;
    if (cs > 1) {
        if (lane < cs)
            st_cluster_b64(map_cluster(smem_u32(&parts[me]), lane),
                           __builtin_bit_cast(uint64_t, part));
        __syncwarp();
        cluster_arrive();
    } else if (lane == 0) {
        parts[me] = part;
    }
}

// The gradient's pass over a warp's part: k times the powers against pg.
template <typename T, typename G>
__device__ __forceinline__ void write_shares(const RowView<T>& r, RowSlice<G>& sl, const Power& pg,
                                             float k, T* out, bool on_grid) {
    constexpr int E = VecOf<T>::kElems;
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
}

// From this |lse| on exp(z / T - lse) takes its row's sum again: it is off by half a unit of lse,
// 2^-17 below 256, and by the rounding of log2(e) / T behind lse, 2^-16 there at most; at
// 1e4 the first is 5e-4, and a row masked by the type's lowest value all over has an lse that
// holds nothing of its sum (or none in fp32's range, with T < 1).
constexpr float kFarLse = 256.f;

// The same with a given lse: k * exp(z / T - lse), zeros for k = 0.
__device__ __forceinline__ float share_by_lse(float z, float inv_t, float lse) {
    return ex2(fmaf(z, inv_t, -lse) * kLog2e);
}
template <typename T, typename G>
__device__ __forceinline__ void write_shares_lse(const RowView<T>& r, RowSlice<G>& sl, float inv_t,
                                                 float lse, float k, T* out, bool on_grid) {
    constexpr int E = VecOf<T>::kElems;
    const f32x2 it = pair(inv_t, inv_t), nl = pair(-lse, -lse), le = pair(kLog2e, kLog2e);
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
}

}  // namespace df2
