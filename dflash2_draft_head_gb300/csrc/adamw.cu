// Steps on the weights of many tensors at once: the 2-norm of their gradients, and AdamW
//
//   g' = g * grad_scale * min(1, max_norm / norm)
//   m  = beta1 * m + (1 - beta1) * g',   v = beta2 * v + (1 - beta2) * g'^2
//   p  = p - lr * weight_decay * p - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
//
// with the states m and v in fp32 or in 8 bits (state8.cuh).  Bound by HBM: every value is read
// and written once, 28 bytes a weight with everything in fp32, 10 with weights and
// gradients in bf16 and states in 8 bits.  The tensors' addresses are parameters of the
// launch; a CTA takes a chunk of one tensor, which it finds by a search among the chunks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "rows.cuh"
#include "state8.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                // neighbours that a thread works on
constexpr int kTurn = kThreads * kVec;

// Tensors of a launch: few with short parameters, or 27 KB of parameters (of the 32 KB that fit).
constexpr int kFew = 16, kMany = 384;

// Eight neighbours of a tensor as they lie in memory.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void store(float* p) const {
        __stcs(reinterpret_cast<float4*>(p), a);
        __stcs(reinterpret_cast<float4*>(p) + 1, b);
    }
    __device__ __forceinline__ void get(float (&x)[kVec]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[kVec]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        __stcs(reinterpret_cast<uint4*>(p), a);
    }
    __device__ __forceinline__ void get(float (&x)[kVec]) const { unpack(a, x); }
    __device__ __forceinline__ void set(const float (&x)[kVec]) { a = pack(x); }
    // Numbers whose upper halves are to be taken as they are.
    __device__ __forceinline__ void set_upper(const uint32_t (&x)[kVec]) {
        a = make_uint4(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632),
                       __byte_perm(x[4], x[5], 0x7632), __byte_perm(x[6], x[7], 0x7632));
    }
};
template <>
struct alignas(8) Vec<uint8_t> {
    uint32_t a[2];
    __device__ __forceinline__ void load(const uint8_t* p) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        a[0] = v.x;
        a[1] = v.y;
    }
    __device__ __forceinline__ void store(uint8_t* p) const {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(a[0], a[1]));
    }
    // Byte j in bits 24 to 31, something below it.
    __device__ __forceinline__ uint32_t high(int j) const { return a[j / 4] << (24 - 8 * (j & 3)); }
    // From bits 24 to 31 of numbers.
    __device__ __forceinline__ void set_high(const uint32_t (&x)[kVec]) {
#pragma unroll
        for (int q = 0; q < kVec / 4; ++q) {
            const uint32_t* y = x + 4 * q;
            a[q] = __byte_perm(__byte_perm(y[0], y[1], 0x0073), __byte_perm(y[2], y[3], 0x0073),
                               0x5410);
        }
    }
};

// Elements [i, i + 8) of n: at once where they are known to be there and aligned (FULL), else one
// by one, zeros beyond n.
template <bool FULL, typename T>
__device__ __forceinline__ Vec<T> load(const T* p, long long i, long long n) {
    Vec<T> o;
    if (FULL) {
        o.load(p + i);
    } else {
        alignas(16) T x[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[j] = i + j < n ? p[i + j] : T(0.f);
        o = *reinterpret_cast<const Vec<T>*>(x);
    }
    return o;
}
template <bool FULL, typename T>
__device__ __forceinline__ void store(T* p, long long i, long long n, const Vec<T>& o) {
    if (FULL) {
        o.store(p + i);
    } else {
        const T* x = reinterpret_cast<const T*>(&o);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (i + j < n) p[i + j] = x[j];
    }
}

// The tensor that chunk `c` belongs to: the last one whose first chunk is not above it.
template <typename Batch>
__device__ __forceinline__ int tensor_of(const Batch& b, int c) {
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.t[mid].first <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------------ the gradients' norm

constexpr int kNormTurns = 8;
constexpr long long kNormChunk = (long long)kNormTurns * kTurn;

struct NormTensor {
    const void* g;
    long long n;
    int first, wide;
};
template <int N>
struct NormBatch {
    NormTensor t[N];
    int count;
    double* sums;  // of this launch's chunks
};

// A chunk's sum of squares, by thread: 64 values in fp32.
template <bool FULL, typename T>
__device__ __forceinline__ float thread_squares(const T* g, long long i, long long n) {
    Vec<T> o[kNormTurns];
#pragma unroll
    for (int k = 0; k < kNormTurns; ++k) o[k] = load<FULL>(g, i + (long long)k * kTurn, n);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kNormTurns; ++k) {
        float x[kVec];
        o[k].get(x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[j & 1] = fmaf(x[j], x[j], s[j & 1]);
    }
    return s[0] + s[1];
}

// The sum of a chunk's squares where fp32's is not good: in 64 bits.  By the whole block.
template <typename T>
__device__ __noinline__ double far_squares(const T* g, long long i, long long n, double* part) {
    double s = 0;
    bool any = false;
    for (int turn = 0; turn < 2; ++turn) {
        for (int k = 0; k < kNormTurns; ++k) {
            float x[kVec];
            load<false>(g, i + (long long)k * kTurn, n).get(x);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (turn == 0)
                    any = any || x[j] != 0.f;
                else
                    s += (double)x[j] * x[j];
            }
        }
        if (turn == 0 && __syncthreads_or(any) == 0) return 0;
    }
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0;
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    return s;
}

// The sum of the squares of a chunk, for thread 0: 64 values a thread and 32 threads in fp32, the
// rest in 64 bits (by one thread: an SM adds two such numbers a cycle).  Squares leave fp32 from
// 1.8e19 on and lose bits below 1e-19: a chunk whose sum is outside [1e-24, 1e30] is taken again.
template <typename T, int N>
__device__ __forceinline__ double chunk_squares(const NormBatch<N>& b, int chunk, float* part,
                                                double* far_part) {
    const int tid = threadIdx.x;
    const NormTensor& t = b.t[tensor_of(b, chunk)];
    const T* g = static_cast<const T*>(t.g);
    const long long lo = (long long)(chunk - t.first) * kNormChunk, n = t.n;
    const long long i = lo + (long long)tid * kVec;
    const float sum = warp_sum(t.wide != 0 && lo + kNormChunk <= n
                                   ? thread_squares<true>(g, i, n)
                                   : thread_squares<false>(g, i, n));
    if ((tid & 31) == 0) part[tid >> 5] = sum;
    __syncthreads();
    float all = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) all += part[w];
    if (!(all >= 1e-24f && all <= 1e30f)) return far_squares(g, i, n, far_part);
    double exact = 0;
    if (tid == 0)
        for (int w = 0; w < kThreads / 32; ++w) exact += part[w];
    return exact;
}

// One CTA a chunk: 40.4 M bf16 gradients in 13 us, 136 M fp32 ones in 81 us (6.7 TB/s).
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4) norm_kernel(const __grid_constant__ NormBatch<N> b) {
    __shared__ float part[kThreads / 32];
    __shared__ double far_part[kThreads / 32];
    griddep_launch_dependents();
    const double s = chunk_squares<T>(b, blockIdx.x, part, far_part);
    if (threadIdx.x == 0) b.sums[blockIdx.x] = s;
}

// Few chunks: one cluster, whose first CTA adds up what the others have written to its shared
// memory; a launch and a workspace less (17 tensors of 100 elements: 19 us a call, 25 with both).
constexpr int kNormCluster = 8;
constexpr long long kNormFew = 4 * kNormCluster;
template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
    norm_few_kernel(const __grid_constant__ NormBatch<N> b, int chunks, float* norm) {
    __shared__ float part[kThreads / 32];
    __shared__ double far_part[kThreads / 32];
    __shared__ double sums[kNormCluster];
    const int rank = (int)cluster_ctarank();
    cluster_arrive();
    double s = 0;  // in thread 0
    for (int c = rank; c < chunks; c += kNormCluster) {
        s += chunk_squares<T>(b, c, part, far_part);
        __syncthreads();  // part is written again
    }
    cluster_wait();  // every CTA has started
    if (threadIdx.x == 0)
        st_cluster_b64(map_cluster(smem_u32(&sums[rank]), 0), __builtin_bit_cast(uint64_t, s));
    cluster_sync();
    if (rank != 0 || threadIdx.x != 0) return;
    double all = 0;
    for (int k = 0; k < kNormCluster; ++k) all += sums[k];
    *norm = (float)sqrt(all);
}

constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads)
    norm_join_kernel(const double* sums, long long n, float* norm) {
    __shared__ double part[kJoinThreads / 32];
    griddep_wait();
    double s = 0;
    for (long long i = threadIdx.x; i < n; i += kJoinThreads) s += sums[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    s = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) s += part[w];
    *norm = (float)sqrt(s);
}

// ------------------------------------------------------------------ AdamW

// How a launch takes its chunks.  The figures are those of bf16 weights and gradients, or of fp32
// ones; other types of weights and gradients take the same shapes.  With states in 8 bits
// instructions bound the step, 60 a weight, and warps to cover their latency count: 128 threads at
// 64 registers, 76 us for 40.4 M weights in bf16 (5.4 TB/s; 78 us with the states' sums one by
// one), against 81 us at 80 registers and 94 us with one vector a thread.  With states in fp32 HBM
// does: 535 to 550 us for 136 M fp32 weights (7.1 TB/s) in all of these shapes.
template <bool S8>
struct AdamShape {
    static constexpr int kThreads = S8 ? 128 : 256, kMinCtas = S8 ? 8 : 1;
    // vectors of a thread, all loads first, and how far apart they are
    static constexpr int kTurns = 2, kStride = kThreads * kVec;
    static constexpr long long kChunk = (long long)kTurns * kStride;
    static_assert(kChunk % kStateBlock == 0, "a block of 8-bit states lies in one chunk");
};

struct AdamTensor {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* master;
    uint8_t *m_scale, *v_scale;
    long long n;
    int first, wide;
};
template <int N>
struct AdamBatch {
    AdamTensor t[N];
    int count, ordinal;  // of the launch's first tensor among the call's
    const int32_t* step_at;
    const float* lr_at;
    const float* norm;
    float beta1, beta2, one_less1, one_less2, ln_beta1, ln_beta2;
    float lr, decay, rate, root, eps, weight_decay;  // decay = lr * weight_decay
    float max_norm, grad_scale;
    float one;  // 1, see sum_of
    int step, fine;
    uint32_t seed_lo, seed_hi;
};

// Pseudo-random bits of an element: two rounds of an odd product and a shift, with a key of
// the call (seed and step) in front of the first and one of the tensor behind it.  The two
// factors are the best of 1500 random pairs by how near to one half every output bit flips with
// each bit of the place.  The tensor's key passes one product alone: for one place in two tensors
// the bits of the states are correlated (over 65536 places and 200 seeds by 0.23 for m and 0.42 for
// v in the mean square, 0.004 for the weights' bits, as all are between steps and seeds).
constexpr uint32_t kMul1 = 0x927aa3cdu, kMul2 = 0x93e1aa55u;
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ x >> 16) * kMul1;
    x = (x ^ x >> 15) * kMul2;
    return x ^ x >> 16;
}
// Of element i with key1 already in it (the exclusive or of both) and times kMul1.
__device__ __forceinline__ uint32_t chance_bits(uint32_t first, uint32_t key2_mul2) {
    const uint32_t x = (first ^ first >> 16) * kMul2 + key2_mul2;
    return x ^ x >> 15;
}

// The root and the quotient of a step, within 2 units of the last place of fp32.  The quick ones
// take numbers below fp32's normal range as 0: a divisor moves by 1.1e-19 * root at most, which is
// nothing beside eps where it counts (`fine` says that it would be).
__device__ __forceinline__ float quick_root(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float quick_inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest magnitude of three, NaN where one is.
__device__ __forceinline__ float max_abs_or_nan(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ f32x2 twice(float x) { return pair(x, x); }
// The sum of two products, each rounded by itself: a packed addition behind a packed product is
// compiled into one multiply-add, whose product is not rounded, and so is a multiply-add with
// 1 unless the 1 comes from the launch's parameters.
__device__ __forceinline__ f32x2 sum_of(f32x2 a, f32x2 b, float one) {
    return fma2(a, twice(one), b);
}

// What a launch's threads take from the device, and the key of their chunk's chance.
struct Coefficients {
    float scale, rate, root, decay;
    uint32_t key1, key2;  // key1's exclusive or with an element's place; key2 * kMul2
};

// TURNS vectors of a thread, from element i on, a stride apart.
template <typename P, typename Gr, bool S8, bool MASTER, bool CHANCE, int TURNS, bool FULL,
          typename Batch>
__device__ __forceinline__ void adam_vectors(const Batch& b, const AdamTensor& t,
                                             const Coefficients& c, long long i) {
    using S = typename std::conditional<S8, uint8_t, float>::type;
    using W = typename std::conditional<MASTER, float, P>::type;
    constexpr int kStride = AdamShape<S8>::kStride;
    const long long n = t.n;
    W* const w_at = MASTER ? reinterpret_cast<W*>(t.master) : static_cast<W*>(t.p);
    S* const m_at = static_cast<S*>(t.m);
    S* const v_at = static_cast<S*>(t.v);
    Vec<W> wo[TURNS];
    Vec<Gr> go[TURNS];
    Vec<S> mo[TURNS], vo[TURNS];
    uint32_t ms[TURNS], vs[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
        const long long at = i + k * kStride;
        wo[k] = load<FULL>(w_at, at, n);
        go[k] = load<FULL>(static_cast<const Gr*>(t.g), at, n);
        mo[k] = load<FULL>(m_at, at, n);
        vo[k] = load<FULL>(v_at, at, n);
        if (S8) {
            ms[k] = FULL || at < n ? t.m_scale[at >> 5] : 0u;
            vs[k] = FULL || at < n ? t.v_scale[at >> 5] : 0u;
        }
    }
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
        const long long at = i + k * kStride;
        float w[kVec], g[kVec], m[kVec], v[kVec];
        wo[k].get(w);
        go[k].get(g);
        float mb = b.beta1, vb = b.beta2;
        if constexpr (S8) {
            // a product with a power of two is exact: where in the chain it stands does not show
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                m[j] = State8<false>::raw(mo[k].high(j));
                v[j] = State8<true>::raw(vo[k].high(j));
            }
            if (__any_sync(0xffffffffu,
                           ms[k] >= State8<false>::kFar || vs[k] >= State8<true>::kFar)) {
                const float mu = State8<false>::unit(ms[k]), vu = State8<true>::unit(vs[k]);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    m[j] *= mu;
                    v[j] *= vu;
                }
                mb *= State8<false>::far_unit(ms[k]);
                vb *= State8<true>::far_unit(vs[k]);
            } else {
                mb *= State8<false>::near_unit(ms[k]);
                vb *= State8<true>::near_unit(vs[k]);
            }
        } else {
            mo[k].get(m);
            vo[k].get(v);
        }
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            // products and sums rounded one by one: the states' last bits depend on nothing else
            const f32x2 gs = mul2(pair(g[j], g[j + 1]), twice(c.scale));
            const float2 mm = halves(sum_of(mul2(pair(m[j], m[j + 1]), twice(mb)),
                                            mul2(gs, twice(b.one_less1)), b.one));
            const float2 vv = halves(sum_of(mul2(pair(v[j], v[j + 1]), twice(vb)),
                                            mul2(mul2(gs, gs), twice(b.one_less2)), b.one));
            m[j] = mm.x;
            m[j + 1] = mm.y;
            v[j] = vv.x;
            v[j + 1] = vv.y;
        }
        if (b.fine) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) g[j] = m[j] / fmaf(sqrtf(v[j]), c.root, b.eps);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                g[j] = m[j] * quick_inverse(fmaf(quick_root(v[j]), c.root, b.eps));
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) w[j] -= fmaf(c.decay, w[j], c.rate * g[j]);
        uint32_t chance[kVec];
        if (CHANCE) {
            // the places of 8 neighbours differ in their lowest bits, and so do those in front of
            // the first product, by the same for all vectors
            const uint32_t low = c.key1 & (kVec - 1u), first = ((uint32_t)at ^ c.key1) * kMul1;
            const uint32_t key2 = c.key2 + (uint32_t)(at >> 32) * (kMul1 * kMul2);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                chance[j] = chance_bits(first + ((low ^ (uint32_t)j) - low) * kMul1, key2);
        }
        // the weights leave before the states are rounded, and with them their registers
        if constexpr (MASTER || sizeof(P) == 4 || !CHANCE) {
            wo[k].set(w);
        } else {
            // the upper half of a number and 16 bits of chance
            uint32_t up[kVec];
            float odd = 0.f;  // NaN with one among the numbers, or an infinity
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                odd = fmaf(w[j], 0.f, odd);
                up[j] = __float_as_uint(w[j]) + (chance[j] * kMul1 >> 16);
            }
            if (!(odd == 0.f)) {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (w[j] != w[j]) up[j] = 0x7fffffffu;
            }
            wo[k].set_upper(up);
        }
        store<FULL>(w_at, at, n, wo[k]);
        if constexpr (MASTER) {
            Vec<P> p;
            p.set(w);
            store<FULL>(static_cast<P*>(t.p), at, n, p);
        }
        if constexpr (S8) {
            if (!FULL) {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (at + j >= n) m[j] = v[j] = 0.f;
            }
            float mt = fabsf(m[0]), vt = v[0];
#pragma unroll
            for (int j = 1; j + 1 < kVec; j += 2) {
                mt = max_abs_or_nan(mt, m[j], m[j + 1]);
                vt = max_abs_or_nan(vt, v[j], v[j + 1]);
            }
            mt = max_or_nan(mt, fabsf(m[kVec - 1]));
            vt = max_or_nan(vt, v[kVec - 1]);
#pragma unroll
            for (int o = 1; o < kStateBlock / kVec; o *= 2) {
                mt = max_or_nan(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                vt = max_or_nan(vt, __shfl_xor_sync(0xffffffffu, vt, o));
            }
            uint32_t mn, vn, wm[kVec], wv[kVec];  // the scales; the magnitudes on their grids
            if (__all_sync(0xffffffffu, State8<false>::near(mt) && State8<true>::near(vt))) {
                mn = State8<false>::near_scale_of(mt);
                vn = State8<true>::near_scale_of(vt);
                const float md = State8<false>::near_down(mn), vd = State8<true>::near_down(vn);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    wm[j] = __float_as_uint(fabsf(m[j]) * md);
                    wv[j] = __float_as_uint(v[j] * vd);
                }
            } else {
                mn = State8<false>::scale_of(mt);
                vn = State8<true>::scale_of(vt);
                const float md = State8<false>::down(mn), vd = State8<true>::down(vn);
                const float mf = State8<false>::far_down(mn), vf = State8<true>::far_down(vn);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    wm[j] = mn == 255u ? 0u : __float_as_uint(fabsf(m[j]) * md * mf);
                    wv[j] = vn == 255u ? 0u : __float_as_uint(v[j] * vd * vf);
                    if (mn == 255u) m[j] = 0.f;
                    if (vn == 255u) v[j] = 0.f;
                }
            }
            uint32_t mc[kVec], vc[kVec], least = 0xffffffffu;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                // the lower and the upper 16 bits in bits 8 to 23, bit 7 set below them
                const uint32_t ml = CHANCE ? __byte_perm(chance[j], 0x80u, 0x5104) : 0u;
                const uint32_t vl = CHANCE ? __byte_perm(chance[j], 0x80u, 0x5324) : 0u;
                mc[j] = State8<false>::template encode<CHANCE>(m[j], wm[j], ml);
                vc[j] = State8<true>::template encode<CHANCE>(v[j], wv[j], vl);
                least = min(least, vc[j]);
            }
            if (least < State8<true>::kOne) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) vc[j] = State8<true>::above_zero(v[j], vc[j]);
            }
            mo[k].set_high(mc);
            vo[k].set_high(vc);
            if ((FULL || at < n) && (threadIdx.x & (kStateBlock / kVec - 1)) == 0) {
                t.m_scale[at >> 5] = (uint8_t)mn;
                t.v_scale[at >> 5] = (uint8_t)vn;
            }
        } else {
            mo[k].set(m);
            vo[k].set(v);
        }
        store<FULL>(m_at, at, n, mo[k]);
        store<FULL>(v_at, at, n, vo[k]);
    }
}

// The end of a tensor, or one whose vectors are not aligned.  A call, so that the others keep their
// registers.
template <typename P, typename Gr, bool S8, bool MASTER, bool CHANCE, typename Batch>
__device__ __noinline__ void adam_edge(const Batch& b, const AdamTensor& t, const Coefficients c,
                                       long long i) {
    adam_vectors<P, Gr, S8, MASTER, CHANCE, 1, false>(b, t, c, i);
}

template <typename P, typename Gr, bool S8, bool MASTER, bool CHANCE, int N>
__global__ void __launch_bounds__(AdamShape<S8>::kThreads, AdamShape<S8>::kMinCtas)
    adamw_kernel(const __grid_constant__ AdamBatch<N> b) {
    const int k = tensor_of(b, blockIdx.x);
    const AdamTensor& t = b.t[k];
    using Shape = AdamShape<S8>;
    const long long lo = (long long)((int)blockIdx.x - t.first) * Shape::kChunk;
    Coefficients c = {b.grad_scale, b.rate, b.root, b.decay, 0, 0};
    if (b.norm != nullptr) {
        const float norm = *b.norm;
        if (!(fabsf(norm) < INFINITY)) return;  // the step is left out
        if (b.max_norm > 0.f) {
            const float whole = norm * fabsf(b.grad_scale);
            if (whole < INFINITY)
                c.scale *= fminf(b.max_norm / whole, 1.f);
            else  // the product alone leaves fp32
                c.scale = copysignf(fminf(b.max_norm / norm, fabsf(c.scale)), c.scale);
        }
    }
    const int step = b.step_at != nullptr ? *b.step_at : b.step;
    if (b.step_at != nullptr || b.lr_at != nullptr) {
        const float lr = b.lr_at != nullptr ? *b.lr_at : b.lr;
        if (step < 1 || !(fabsf(lr) < INFINITY)) return;  // what a call refuses on the host
        c.decay = lr * b.weight_decay;
        c.rate = lr / -expm1f((float)step * b.ln_beta1);
        c.root = rsqrtf(-expm1f((float)step * b.ln_beta2));
    }
    if (CHANCE) {
        c.key1 = mix(b.seed_lo ^ mix(b.seed_hi ^ mix((uint32_t)step)));
        c.key2 = mix(c.key1 + (uint32_t)(b.ordinal + k) + 1u) * kMul2;
    }
    const long long i = lo + (long long)threadIdx.x * kVec;
    if (t.wide != 0 && lo + Shape::kChunk <= t.n)
        adam_vectors<P, Gr, S8, MASTER, CHANCE, Shape::kTurns, true>(b, t, c, i);
    else
#pragma unroll 1
        for (int turn = 0; turn < Shape::kTurns; ++turn) {
            // by warp, whose lanes share blocks of 8-bit states: the last one has less than a whole
            const long long at = i + turn * Shape::kStride;
            const long long warp_lo = at - (threadIdx.x & 31) * kVec;
            if (t.wide != 0 && warp_lo + 32 * kVec <= t.n)
                adam_vectors<P, Gr, S8, MASTER, CHANCE, 1, true>(b, t, c, at);
            else if (warp_lo < t.n)
                adam_edge<P, Gr, S8, MASTER, CHANCE>(b, t, c, at);
        }
}

// ------------------------------------------------------------------ states to values and back

template <typename T, bool SQUARES, bool FULL>
__device__ __forceinline__ void decode_vector(const uint8_t* codes, const uint8_t* scale,
                                             long long i, long long n, T* out) {
    const Vec<uint8_t> o = load<FULL>(codes, i, n);
    const uint32_t s = FULL || i < n ? scale[i >> 5] : 0u;
    const float unit = State8<SQUARES>::unit(s), far = State8<SQUARES>::far_unit(s);
    float x[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = State8<SQUARES>::raw(o.high(j)) * unit * far;
    Vec<T> y;
    y.set(x);
    store<FULL>(out, i, n, y);
}
template <typename T, bool SQUARES>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(const uint8_t* codes, const uint8_t* scale, long long n, bool wide, T* out) {
    const long long lo = (long long)blockIdx.x * kTurn, i = lo + (long long)threadIdx.x * kVec;
    if (wide && lo + kTurn <= n)
        decode_vector<T, SQUARES, true>(codes, scale, i, n, out);
    else
        decode_vector<T, SQUARES, false>(codes, scale, i, n, out);
}

template <typename T, bool SQUARES, bool FULL>
__device__ __forceinline__ void encode_vector(const T* in, long long i, long long n, uint8_t* codes,
                                             uint8_t* scale) {
    float x[kVec], top = 0.f;
    load<FULL>(in, i, n).get(x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        // a square is not negative: one that is reads as NaN, which a scale can say
        if (SQUARES && x[j] < 0.f) x[j] = NAN;
        top = max_or_nan(top, fabsf(x[j]));
    }
#pragma unroll
    for (int o = 1; o < kStateBlock / kVec; o *= 2)
        top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t s = State8<SQUARES>::scale_of(top);
    const float down = State8<SQUARES>::down(s), far = State8<SQUARES>::far_down(s);
    uint32_t c[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const uint32_t w = __float_as_uint(fabsf(x[j]) * down * far);
        c[j] = State8<SQUARES>::template encode<false>(x[j], w, 0);
        if (SQUARES) c[j] = State8<SQUARES>::above_zero(x[j], c[j]);
        if (s == 255u) c[j] = 0u;
    }
    Vec<uint8_t> o;
    o.set_high(c);
    store<FULL>(codes, i, n, o);
    if ((FULL || i < n) && (threadIdx.x & (kStateBlock / kVec - 1)) == 0)
        scale[i >> 5] = (uint8_t)s;
}
template <typename T, bool SQUARES>
__global__ void __launch_bounds__(kThreads)
    encode_kernel(const T* in, long long n, bool wide, uint8_t* codes, uint8_t* scale) {
    const long long lo = (long long)blockIdx.x * kTurn, i = lo + (long long)threadIdx.x * kVec;
    if (wide && lo + kTurn <= n)
        encode_vector<T, SQUARES, true>(in, i, n, codes, scale);
    else
        encode_vector<T, SQUARES, false>(in, i, n, codes, scale);
}

// ------------------------------------------------------------------ host

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
long long chunks_of(long long n, long long chunk) { return (n + chunk - 1) / chunk; }

// Chunks of one launch: a grid's limit, with room for a tensor's first chunk in 32 bits.
constexpr long long kMostChunks = 1 << 30;

template <typename T, int N>
cudaError_t norm_batches(const GradNormArgs& a, cudaStream_t stream) {
    NormBatch<N> b;
    double* sums = a.workspace;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    for (int k = 0; k < a.count;) {
        const bool from_first = sums == a.workspace;
        b.count = 0;
        b.sums = sums;
        long long first = 0;
        for (; k < a.count && b.count < N; ++k) {
            if (a.sizes[k] == 0) continue;
            const long long c = chunks_of(a.sizes[k], kNormChunk);
            if (first + c > kMostChunks) break;
            b.t[b.count++] = {a.grads[k], a.sizes[k], (int)first, aligned(a.grads[k], 16)};
            first += c;
        }
        if (b.count == 0) break;  // nothing but empty tensors left
        if (k == a.count && from_first && first <= kNormFew) {  // see grad_norm_chunks
            cfg.gridDim = dim3(kNormCluster);
            cfg.blockDim = dim3(kThreads);
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = kNormCluster;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            return cudaLaunchKernelEx(&cfg, norm_few_kernel<T, N>, b, (int)first, a.norm);
        }
        norm_kernel<T, N><<<(unsigned)first, kThreads, 0, stream>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        sums += first;
    }
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kJoinThreads);
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, norm_join_kernel, (const double*)a.workspace,
                              (long long)(sums - a.workspace), a.norm);
}

template <typename P, typename Gr, bool S8, bool MASTER, bool CHANCE, int N>
cudaError_t adam_batches(const AdamwArgs& a, AdamBatch<N>& b, cudaStream_t stream) {
    for (int k = 0; k < a.count;) {
        b.count = 0;
        b.ordinal = k;
        long long first = 0;
        for (; k < a.count && b.count < N; ++k) {
            const long long c = chunks_of(a.sizes[k], AdamShape<S8>::kChunk);
            if (first + c > kMostChunks) break;
            AdamTensor& t = b.t[b.count++];
            t = {a.params[k], a.grads[k], a.exp_avg[k], a.exp_avg_sq[k],
                 MASTER ? a.master[k] : nullptr, S8 ? a.exp_avg_scale[k] : nullptr,
                 S8 ? a.exp_avg_sq_scale[k] : nullptr, a.sizes[k], (int)first, 0};
            t.wide = aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.m, S8 ? kVec : 16) &&
                     aligned(t.v, S8 ? kVec : 16) && (!MASTER || aligned(t.master, 16));
            first += c;
        }
        if (first == 0) continue;  // a batch of empty tensors
        adamw_kernel<P, Gr, S8, MASTER, CHANCE, N>
            <<<(unsigned)first, AdamShape<S8>::kThreads, 0, stream>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename P, typename Gr, bool S8, bool MASTER, int N>
cudaError_t adam_rounding(const AdamwArgs& a, AdamBatch<N>& b, cudaStream_t stream) {
    // chance has a part where something is rounded to fewer bits
    constexpr bool kCan = S8 || (std::is_same<P, __nv_bfloat16>::value && !MASTER);
    if (kCan && a.by_chance) return adam_batches<P, Gr, S8, MASTER, kCan, N>(a, b, stream);
    return adam_batches<P, Gr, S8, MASTER, false, N>(a, b, stream);
}

template <typename P, typename Gr, int N>
cudaError_t adam_states(const AdamwArgs& a, AdamBatch<N>& b, cudaStream_t stream) {
    constexpr bool kCopies = std::is_same<P, __nv_bfloat16>::value;
    if (kCopies && a.master != nullptr)
        return a.exp_avg_scale != nullptr ? adam_rounding<P, Gr, true, kCopies, N>(a, b, stream)
                                          : adam_rounding<P, Gr, false, kCopies, N>(a, b, stream);
    return a.exp_avg_scale != nullptr ? adam_rounding<P, Gr, true, false, N>(a, b, stream)
                                      : adam_rounding<P, Gr, false, false, N>(a, b, stream);
}

template <int N>
cudaError_t adam_typed(const AdamwArgs& a, int param_bf16, int grad_bf16, cudaStream_t stream) {
    AdamBatch<N> b;
    b.step_at = a.step_at;
    b.lr_at = a.lr_at;
    b.norm = a.norm;
    b.beta1 = (float)a.beta1;
    b.beta2 = (float)a.beta2;
    b.one_less1 = (float)(1.0 - a.beta1);
    b.one_less2 = (float)(1.0 - a.beta2);
    b.ln_beta1 = (float)std::log(a.beta1);
    b.ln_beta2 = (float)std::log(a.beta2);
    b.lr = (float)a.lr;
    b.weight_decay = (float)a.weight_decay;
    b.decay = (float)(a.lr * a.weight_decay);
    b.rate = (float)(a.lr / (1.0 - std::pow(a.beta1, a.step)));
    b.root = (float)(1.0 / std::sqrt(1.0 - std::pow(a.beta2, a.step)));
    b.eps = (float)a.eps;
    b.max_norm = (float)a.max_norm;
    b.grad_scale = (float)a.grad_scale;
    b.one = 1.f;
    b.step = a.step;
    // see quick_root: its error, by the largest root a step can have, against 2^-24 of eps
    b.fine = 1.1e-19 / std::sqrt(1.0 - a.beta2) > a.eps * 0x1p-24;
    b.seed_lo = (uint32_t)a.seed;
    b.seed_hi = (uint32_t)(a.seed >> 32);
    using bf = __nv_bfloat16;
    if (param_bf16)
        return grad_bf16 ? adam_states<bf, bf, N>(a, b, stream)
                         : adam_states<bf, float, N>(a, b, stream);
    return grad_bf16 ? adam_states<float, bf, N>(a, b, stream)
                     : adam_states<float, float, N>(a, b, stream);
}

unsigned vec_grid(long long n) { return (unsigned)chunks_of(n, kTurn); }

}  // namespace

long long grad_norm_chunks(int count, const long long* sizes) {
    long long n = 0;
    for (int k = 0; k < count; ++k) n += chunks_of(sizes[k], kNormChunk);
    return n <= kNormFew ? 0 : n;
}

cudaError_t launch_grad_norm(const GradNormArgs& a, int grad_bf16, cudaStream_t stream) {
    if (grad_bf16)
        return a.count <= kFew ? norm_batches<__nv_bfloat16, kFew>(a, stream)
                               : norm_batches<__nv_bfloat16, kMany>(a, stream);
    return a.count <= kFew ? norm_batches<float, kFew>(a, stream)
                           : norm_batches<float, kMany>(a, stream);
}

cudaError_t launch_adamw(const AdamwArgs& a, int param_bf16, int grad_bf16, cudaStream_t stream) {
    return a.count <= kFew ? adam_typed<kFew>(a, param_bf16, grad_bf16, stream)
                           : adam_typed<kMany>(a, param_bf16, grad_bf16, stream);
}

cudaError_t launch_state_decode(const uint8_t* codes, const uint8_t* scale, long long n,
                                int squares, void* out, int out_bf16, cudaStream_t stream) {
    const bool wide = aligned(codes, 8) && aligned(out, 16);
    const unsigned grid = vec_grid(n);
    using bf = __nv_bfloat16;
    if (out_bf16) {
        bf* o = static_cast<bf*>(out);
        if (squares)
            decode_kernel<bf, true><<<grid, kThreads, 0, stream>>>(codes, scale, n, wide, o);
        else
            decode_kernel<bf, false><<<grid, kThreads, 0, stream>>>(codes, scale, n, wide, o);
    } else {
        float* o = static_cast<float*>(out);
        if (squares)
            decode_kernel<float, true><<<grid, kThreads, 0, stream>>>(codes, scale, n, wide, o);
        else
            decode_kernel<float, false><<<grid, kThreads, 0, stream>>>(codes, scale, n, wide, o);
    }
    return cudaGetLastError();
}

cudaError_t launch_state_encode(const void* values, int in_bf16, long long n, int squares,
                                uint8_t* codes, uint8_t* scale, cudaStream_t stream) {
    const bool wide = aligned(codes, 8) && aligned(values, 16);
    const unsigned grid = vec_grid(n);
    using bf = __nv_bfloat16;
    if (in_bf16) {
        const bf* in = static_cast<const bf*>(values);
        if (squares)
            encode_kernel<bf, true><<<grid, kThreads, 0, stream>>>(in, n, wide, codes, scale);
        else
            encode_kernel<bf, false><<<grid, kThreads, 0, stream>>>(in, n, wide, codes, scale);
    } else {
        const float* in = static_cast<const float*>(values);
        if (squares)
            encode_kernel<float, true><<<grid, kThreads, 0, stream>>>(in, n, wide, codes, scale);
        else
            encode_kernel<float, false><<<grid, kThreads, 0, stream>>>(in, n, wide, codes, scale);
    }
    return cudaGetLastError();
}

}  // namespace df2
