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

#include "common.cuh"
#include "state8.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                // neighbours that a thread works on
constexpr int kTurn = kThreads * kVec;

// Tensors of a launch: few with short parameters, or as many as 32 KB of parameters hold.
constexpr int kFew = 16, kMany = 384;

__device__ __forceinline__ void load_vec(const float* p, float (&x)[kVec]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[kVec]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load_vec(const uint8_t* p, uint32_t (&x)[kVec]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = v.x >> 8 * j & 0xffu;
        x[j + 4] = v.y >> 8 * j & 0xffu;
    }
}
__device__ __forceinline__ void store_vec(float* p, const float (&x)[kVec]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const __nv_bfloat16 (&x)[kVec]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __halves2bfloat162(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_vec(uint8_t* p, const uint32_t (&x)[kVec]) {
    uint2 v = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v.x |= x[j] << 8 * j;
        v.y |= x[j + 4] << 8 * j;
    }
    *reinterpret_cast<uint2*>(p) = v;
}
__device__ __forceinline__ float to_value(float x) { return x; }
__device__ __forceinline__ float to_value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ uint32_t to_value(uint8_t x) { return x; }

// Elements [i, i + 8) of n, zeros beyond; `wide`: the tensor's vectors are aligned.
template <typename T, typename X>
__device__ __forceinline__ void load(const T* p, long long i, long long n, bool wide, X (&x)[kVec]) {
    if (wide && i + kVec <= n) {
        load_vec(p + i, x);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[j] = i + j < n ? to_value(p[i + j]) : X(0);
    }
}
template <typename T, typename X>
__device__ __forceinline__ void store(T* p, long long i, long long n, bool wide, const X (&x)[kVec]) {
    if (wide && i + kVec <= n) {
        store_vec(p + i, x);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (i + j < n) p[i + j] = (T)x[j];
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

// The sum of a chunk's squares where fp32's is not good: in 64 bits.  By the whole block.
template <typename T>
__device__ __noinline__ double far_sum(const T* g, long long lo, long long n, bool wide,
                                       double* part) {
    double s = 0;
    bool any = false;
    for (int k = 0; k < kNormTurns; ++k) {
        float x[kVec];
        load(g, lo + (long long)k * kTurn + (long long)threadIdx.x * kVec, n, wide, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) any = any || x[j] != 0.f;
    }
    if (__syncthreads_or(any) == 0) return 0;
    for (int k = 0; k < kNormTurns; ++k) {
        float x[kVec];
        load(g, lo + (long long)k * kTurn + (long long)threadIdx.x * kVec, n, wide, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s += (double)x[j] * x[j];
    }
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0;
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    return s;
}

// The sum of the squares of a chunk: 64 values a thread and 32 threads in fp32, the rest in
// 64 bits.  Squares leave fp32 from 1.8e19 on and lose bits below 1e-19: a sum outside
// [1e-24, 1e30] is taken again.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormBatch<N> b) {
    __shared__ double part[kThreads / 32];
    const int tid = threadIdx.x;
    const NormTensor& t = b.t[tensor_of(b, blockIdx.x)];
    const T* g = static_cast<const T*>(t.g);
    const long long lo = (long long)((int)blockIdx.x - t.first) * kNormChunk, n = t.n;
    const bool wide = t.wide != 0;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kNormTurns; ++k) {
        float x[kVec];
        load(g, lo + (long long)k * kTurn + (long long)tid * kVec, n, wide, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[j & 1] = fmaf(x[j], x[j], s[j & 1]);
    }
    const float sum = warp_sum(s[0] + s[1]);
    if ((tid & 31) == 0) part[tid >> 5] = sum;
    __syncthreads();
    double all = 0;
    for (int w = 0; w < kThreads / 32; ++w) all += part[w];
    if (!(all >= 1e-24 && all <= 1e30)) {
        __syncthreads();
        all = far_sum(g, lo, n, wide, part);
    }
    if (tid == 0) b.sums[blockIdx.x] = all;
}

constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads)
    norm_join_kernel(const double* sums, long long n, float* norm) {
    __shared__ double part[kJoinThreads / 32];
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

constexpr int kAdamTurns = 2;
constexpr long long kAdamChunk = (long long)kAdamTurns * kTurn;
static_assert(kAdamChunk % kStateBlock == 0, "a block of 8-bit states lies in one chunk");

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
    int step, by_chance;
    uint32_t seed_lo, seed_hi;
};

// Pseudo-random bits of an element: two rounds of an odd product and a shift, with a key of
// the call (seed and step) in front of the first and one of the tensor behind it.  The two
// factors are the best of 1500 random pairs by how near to one half every output bit flips with
// each input bit.
constexpr uint32_t kMul1 = 0x927aa3cdu, kMul2 = 0x93e1aa55u;
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ x >> 16) * kMul1;
    x = (x ^ x >> 15) * kMul2;
    return x ^ x >> 16;
}
__device__ __forceinline__ uint32_t chance_bits(uint32_t i, uint32_t key1, uint32_t key2) {
    uint32_t x = (i ^ key1) * kMul1;
    x = ((x ^ x >> 16) + key2) * kMul2;
    return x ^ x >> 15;
}

// bf16 of x by 16 bits of chance; what is not finite stays so.
__device__ __forceinline__ __nv_bfloat16 round_by(float x, uint32_t chance) {
    const uint32_t w = __float_as_uint(x);
    if ((w & 0x7f800000u) == 0x7f800000u) return __float2bfloat16_rn(x);
    return __ushort_as_bfloat16((unsigned short)((w + chance) >> 16));
}

template <typename P, typename Gr, bool S8, bool MASTER, int N>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ AdamBatch<N> b) {
    using S = typename std::conditional<S8, uint8_t, float>::type;
    using X = typename std::conditional<S8, uint32_t, float>::type;
    const int k = tensor_of(b, blockIdx.x);
    const AdamTensor& t = b.t[k];
    const long long lo = (long long)((int)blockIdx.x - t.first) * kAdamChunk, n = t.n;
    const bool wide = t.wide != 0;
    P* const p = static_cast<P*>(t.p);
    const Gr* const g = static_cast<const Gr*>(t.g);
    S* const m = static_cast<S*>(t.m);
    S* const v = static_cast<S*>(t.v);

    float scale = b.grad_scale;
    if (b.norm != nullptr) {
        const float norm = *b.norm;
        if (!(fabsf(norm) < INFINITY)) return;  // the step is left out
        if (b.max_norm > 0.f) scale *= fminf(b.max_norm / (norm * fabsf(b.grad_scale)), 1.f);
    }
    const int step = b.step_at != nullptr ? *b.step_at : b.step;
    float rate = b.rate, root = b.root, decay = b.decay;
    if (b.step_at != nullptr || b.lr_at != nullptr) {
        const float lr = b.lr_at != nullptr ? *b.lr_at : b.lr;
        decay = lr * b.weight_decay;
        rate = lr / -expm1f((float)step * b.ln_beta1);
        root = rsqrtf(-expm1f((float)step * b.ln_beta2));
    }
    const uint32_t key1 = mix(b.seed_lo ^ mix(b.seed_hi ^ mix((uint32_t)step)));
    uint32_t key2 = mix(key1 + (uint32_t)(b.ordinal + k) + 1u);

#pragma unroll
    for (int turn = 0; turn < kAdamTurns; ++turn) {
        const long long i = lo + turn * kTurn + (long long)threadIdx.x * kVec;
        float w[kVec], x[kVec], m1[kVec], v1[kVec];
        X mc[kVec], vc[kVec];
        if (MASTER)
            load(t.master, i, n, wide, w);
        else
            load(p, i, n, wide, w);
        load(g, i, n, wide, x);
        load(m, i, n, wide, mc);
        load(v, i, n, wide, vc);
        float mu = 0.f, vu = 0.f;
        if constexpr (S8) {
            if (i < n) {
                mu = State8<false>::unit(t.m_scale[i / kStateBlock]);
                vu = State8<true>::unit(t.v_scale[i / kStateBlock]);
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if constexpr (S8) {
                m1[j] = State8<false>::decode(mc[j], mu);
                v1[j] = State8<true>::decode(vc[j], vu);
            } else {
                m1[j] = mc[j];
                v1[j] = vc[j];
            }
            // no contraction: the states' last bits do not depend on how the code is compiled
            const float gs = __fmul_rn(x[j], scale);
            m1[j] = __fadd_rn(__fmul_rn(m1[j], b.beta1), __fmul_rn(gs, b.one_less1));
            v1[j] = __fadd_rn(__fmul_rn(v1[j], b.beta2),
                              __fmul_rn(__fmul_rn(gs, gs), b.one_less2));
            const float by = m1[j] / fmaf(sqrtf(v1[j]), root, b.eps);
            w[j] -= fmaf(decay, w[j], rate * by);
        }
        uint32_t chance[kVec];
        const bool by_chance = b.by_chance != 0;
        if ((S8 || (!MASTER && sizeof(P) == 2)) && by_chance) {
            const uint32_t high = (uint32_t)(i >> 32) * kMul1;  // the same for all 8
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                chance[j] = chance_bits((uint32_t)i + j, key1, key2 + high);
        }
        if constexpr (S8) {
            uint32_t mt = 0, vt = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (i + j >= n) m1[j] = v1[j] = 0.f;
                mt = max(mt, __float_as_uint(m1[j]) & 0x7fffffffu);
                vt = max(vt, __float_as_uint(v1[j]) & 0x7fffffffu);
            }
#pragma unroll
            for (int o = 1; o < kStateBlock / kVec; o *= 2) {
                mt = max(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                vt = max(vt, __shfl_xor_sync(0xffffffffu, vt, o));
            }
            const uint32_t ms = State8<false>::scale_of(mt), vs = State8<true>::scale_of(vt);
            const float md = State8<false>::down(ms), vd = State8<true>::down(vs);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (by_chance) {
                    mc[j] = State8<false>::template encode<true>(m1[j], md, chance[j] & 0xffffu);
                    vc[j] = State8<true>::template encode<true>(v1[j], vd, chance[j] >> 16);
                } else {
                    mc[j] = State8<false>::template encode<false>(m1[j], md, 0);
                    vc[j] = State8<true>::template encode<false>(v1[j], vd, 0);
                }
                if (ms == 255u) mc[j] = 0;
                if (vs == 255u) vc[j] = 0;
            }
            store(m, i, n, wide, mc);
            store(v, i, n, wide, vc);
            if (i < n && i % kStateBlock == 0) {
                t.m_scale[i / kStateBlock] = (uint8_t)ms;
                t.v_scale[i / kStateBlock] = (uint8_t)vs;
            }
        } else {
            store(m, i, n, wide, m1);
            store(v, i, n, wide, v1);
        }
        if (MASTER) store(t.master, i, n, wide, w);
        if constexpr (sizeof(P) == 2) {
            __nv_bfloat16 h[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                h[j] = !MASTER && by_chance ? round_by(w[j], chance[j] * kMul1 >> 16)
                                            : __float2bfloat16_rn(w[j]);
            store(p, i, n, wide, h);
        } else {
            store(p, i, n, wide, w);
        }
    }
}

// ------------------------------------------------------------------ states to values and back

template <typename T, bool SQUARES>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(const uint8_t* codes, const uint8_t* scale, long long n, bool wide, T* out) {
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * kVec;
    if (i >= n) return;
    uint32_t c[kVec];
    load(codes, i, n, wide, c);
    const float unit = State8<SQUARES>::unit(scale[i / kStateBlock]);
    T x[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float f = State8<SQUARES>::decode(c[j], unit);
        if constexpr (sizeof(T) == 2)
            x[j] = __float2bfloat16_rn(f);
        else
            x[j] = f;
    }
    store(out, i, n, wide, x);
}

template <typename T, bool SQUARES>
__global__ void __launch_bounds__(kThreads)
    encode_kernel(const T* in, long long n, bool wide, uint8_t* codes, uint8_t* scale) {
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * kVec;
    float x[kVec];
    load(in, i, n, wide, x);  // zeros from n on
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        // a square is not negative: one that is reads as NaN, which a scale can say
        if (SQUARES && x[j] < 0.f) x[j] = NAN;
        top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < kStateBlock / kVec; o *= 2)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t s = State8<SQUARES>::scale_of(top);
    const float down = State8<SQUARES>::down(s);
    uint32_t c[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        c[j] = s == 255u ? 0u : State8<SQUARES>::template encode<false>(x[j], down, 0);
    if (i >= n) return;
    store(codes, i, n, wide, c);
    if (i % kStateBlock == 0) scale[i / kStateBlock] = (uint8_t)s;
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
    for (int k = 0; k < a.count;) {
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
        norm_kernel<T, N><<<(unsigned)first, kThreads, 0, stream>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        sums += first;
    }
    norm_join_kernel<<<1, kJoinThreads, 0, stream>>>(a.workspace, sums - a.workspace, a.norm);
    return cudaGetLastError();
}

template <typename P, typename Gr, bool S8, bool MASTER, int N>
cudaError_t adam_batches(const AdamwArgs& a, AdamBatch<N>& b, cudaStream_t stream) {
    for (int k = 0; k < a.count;) {
        b.count = 0;
        b.ordinal = k;
        long long first = 0;
        for (; k < a.count && b.count < N; ++k) {
            const long long c = chunks_of(a.sizes[k], kAdamChunk);
            if (first + c > kMostChunks) break;
            AdamTensor& t = b.t[b.count++];
            t = {a.params[k], a.grads[k], a.exp_avg[k], a.exp_avg_sq[k],
                 MASTER ? a.master[k] : nullptr, S8 ? a.exp_avg_scale[k] : nullptr,
                 S8 ? a.exp_avg_sq_scale[k] : nullptr, a.sizes[k], (int)first, 0};
            t.wide = aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.m, S8 ? 8 : 16) &&
                     aligned(t.v, S8 ? 8 : 16) && (!MASTER || aligned(t.master, 16));
            first += c;
        }
        if (first == 0) continue;  // a batch of empty tensors
        adamw_kernel<P, Gr, S8, MASTER, N><<<(unsigned)first, kThreads, 0, stream>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
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
    b.step = a.step;
    b.by_chance = a.by_chance;
    b.seed_lo = (uint32_t)a.seed;
    b.seed_hi = (uint32_t)(a.seed >> 32);
    const bool s8 = a.exp_avg_scale != nullptr, master = a.master != nullptr;
    using bf = __nv_bfloat16;
#define DF2_ADAM(P, GR)                                                                       \
    (s8 ? (master ? adam_batches<P, GR, true, sizeof(P) == 2, N>(a, b, stream)               \
                  : adam_batches<P, GR, true, false, N>(a, b, stream))                       \
        : (master ? adam_batches<P, GR, false, sizeof(P) == 2, N>(a, b, stream)              \
                  : adam_batches<P, GR, false, false, N>(a, b, stream)))
    if (param_bf16) return grad_bf16 ? DF2_ADAM(bf, bf) : DF2_ADAM(bf, float);
    return grad_bf16 ? DF2_ADAM(float, bf) : DF2_ADAM(float, float);
#undef DF2_ADAM
}

unsigned vec_grid(long long n) { return (unsigned)chunks_of(n, kTurn); }

}  // namespace

long long grad_norm_chunks(int count, const long long* sizes) {
    long long n = 0;
    for (int k = 0; k < count; ++k) n += chunks_of(sizes[k], kNormChunk);
    return n;
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

cudaError_t launch_state_decode(const uint8_t* codes, const uint8_t* scale, long long n, int squares,
                                void* out, int out_bf16, cudaStream_t stream) {
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
