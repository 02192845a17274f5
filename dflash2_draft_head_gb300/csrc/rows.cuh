// Shared by the operators that work on whole vocabulary rows (sampling and
// distillation): a row of V elements as 16-byte vectors, held by one CTA or split over
// the CTAs of a thread-block cluster and, inside a CTA, over its warps in index order.
//
// A row may start at any element: the vectors lie on the 16-byte grid of memory,
// so the first and the last one may hold places that are not the row's.  Those
// are never read; they get the fill value -inf, which no operator counts.
//
// A row is passed over one or more times and read from HBM once: every warp streams its
// part through a ring in shared memory (cp.async, each lane the vectors that it works on
// itself, so there is no barrier), and every other pass runs backwards, so that it
// starts on what the ring still holds; the rest comes again from L2.  Several CTAs share
// an SM, so that one's loads run under another's arithmetic and barriers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "ptx.cuh"

namespace df2 {

constexpr int kRowMaxCluster = 16;
constexpr int kStepVecs = 64;  // vectors that a warp handles between two waits

// How a kernel takes rows: threads of a CTA, CTAs that share an SM, steps that a warp's
// ring holds, and the largest part of a row that a CTA takes.
template <int THREADS, int CTAS, int RING, int SLICE_KB>
struct RowGeometry {
    static constexpr int kThreads = THREADS, kWarps = THREADS / 32, kCtas = CTAS, kRing = RING;
    static constexpr long long kSliceBytes = SLICE_KB * 1024;
    static constexpr int kStepBytes = kWarps * kStepVecs * 16;  // a CTA's part of the ring, a step
    static constexpr int kRingBytes = kRing * kStepBytes;
    // A warp's part of n vectors: whole steps where it has several (a short one costs as
    // much as a whole one), else lines of 128 bytes.
    static __host__ __device__ constexpr int warp_vecs(int n) {
        const int even = (n + kWarps - 1) / kWarps;
        return even > 4 * kStepVecs ? (even + kStepVecs - 1) / kStepVecs * kStepVecs
                                    : (even + 7) & ~7;
    }
    static int ring_steps(int n) {
        return std::min(kRing, (warp_vecs(n) + kStepVecs - 1) / kStepVecs);
    }
};

template <typename T>
struct VecOf;
template <>
struct VecOf<float> {
    static constexpr int kElems = 4;
};
template <>
struct VecOf<__nv_bfloat16> {
    static constexpr int kElems = 8;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Two fp32 values in a register pair: one instruction works on both, which
// leaves the issue slots that these kernels run out of first.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 halves(f32x2 p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// One vector's elements in fp32, in index order.
__device__ __forceinline__ void unpack(const uint4& v, f32x2 (&f)[2]) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unpack(const uint4& v, f32x2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <int E>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[E]) {
    f32x2 p[E / 2];
    unpack(v, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 h = halves(p[i]);
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
    }
}

// One vector's largest element; a NaN is passed over.
template <typename T>
__device__ __forceinline__ float vec_max(const uint4& v);
template <>
__device__ __forceinline__ float vec_max<float>(const uint4& v) {
    float f[4];
    unpack(v, f);
    return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
}
template <>
__device__ __forceinline__ float vec_max<__nv_bfloat16>(const uint4& v) {
    const __nv_bfloat162 a = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&v.x),
                                     *reinterpret_cast<const __nv_bfloat162*>(&v.y));
    const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&v.z),
                                     *reinterpret_cast<const __nv_bfloat162*>(&v.w));
    const __nv_bfloat162 c = __hmax2(a, b);
    return fmaxf(__low2float(c), __high2float(c));
}

// The largest element of vectors, NaN where one of them is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
template <typename T>
struct RunningMax;
template <>
struct RunningMax<float> {
    float m;
    __device__ __forceinline__ RunningMax() : m(neg_inf()) {}
    __device__ __forceinline__ void add(const uint4& v) {
        m = max_or_nan(m, max_or_nan(max_or_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                                     max_or_nan(__uint_as_float(v.z), __uint_as_float(v.w))));
    }
    __device__ __forceinline__ float value() const { return m; }
};
template <>
struct RunningMax<__nv_bfloat16> {
    __nv_bfloat162 m;
    __device__ __forceinline__ RunningMax() : m(__float2bfloat162_rn(neg_inf())) {}
    __device__ __forceinline__ void add(const uint4& v) {
        const __nv_bfloat162 a = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&v.x),
                                             *reinterpret_cast<const __nv_bfloat162*>(&v.y));
        const __nv_bfloat162 b = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&v.z),
                                             *reinterpret_cast<const __nv_bfloat162*>(&v.w));
        m = __hmax2_nan(m, __hmax2_nan(a, b));
    }
    __device__ __forceinline__ float value() const {
        return max_or_nan(__low2float(m), __high2float(m));
    }
};

// Four or eight fp32 values as one vector, rounded to the row's type.
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int N>
__device__ __forceinline__ uint4 pack_pairs(const f32x2 (&p)[N]) {
    float f[2 * N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float2 h = halves(p[j]);
        f[2 * j] = h.x;
        f[2 * j + 1] = h.y;
    }
    return pack(f);
}

// 2^x, flushing results below 2^-126 to 0 (relative error about 2^-22).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Row `r` of a [rows, V] array whose rows are `ld` elements apart.
template <typename T>
struct RowView {
    static constexpr int E = VecOf<T>::kElems;
    const T* row;   // element 0
    const T* grid;  // start of the vector that holds element 0 (16-byte aligned)
    int head;       // places before element 0 in that vector
    int V;
    int nvec;
    int ilo, ihi;   // the vectors that hold nothing else than the row's elements

    __device__ __forceinline__ RowView(const void* base, long long ld, int r, int V_) : V(V_) {
        row = static_cast<const T*>(base) + (long long)r * ld;
        head = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        grid = row - head;
        nvec = (head + V + E - 1) / E;
        ilo = head > 0 ? 1 : 0;
        ihi = (head + V) / E;
    }
    __device__ __forceinline__ bool inner(int v) const { return v >= ilo && v < ihi; }
    // Vector v by guarded loads of single elements, -inf in the places outside the row.
    __device__ __forceinline__ uint4 edge(int v) const {
        float f[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int e = v * E + j - head;
            f[j] = e >= 0 && e < V ? to_f32(row[e]) : neg_inf();
        }
        return pack(f);
    }
    // A vector of -inf alone.
    __device__ __forceinline__ uint4 nothing() const {
        const uint32_t w = E == 8 ? 0xff80ff80u : 0xff800000u;
        return make_uint4(w, w, w, w);
    }
    __device__ __forceinline__ uint4 load(int v) const {
        return inner(v) ? *reinterpret_cast<const uint4*>(grid + (long long)v * E) : edge(v);
    }
};

// Which vectors of a row a CTA (the rank-th, `per` vectors each) and one of its warps
// work on, and the warp's ring of `ring` steps in shared memory.  Both splits are in
// index order, warps' parts start on 128-byte lines.
template <typename G>
struct RowSlice {
    static constexpr uint32_t kStepBytes = kStepVecs * 16;
    int lo, hi;      // the CTA's vectors
    int wlo, whi;    // this warp's
    int steps;       // the last one may be short
    int clean_lo, clean_hi;  // steps of nothing but whole vectors of the row
    uint32_t slots;  // this lane's place in the ring
    bool up = true;  // the direction of the next pass
    uint64_t hint;   // L2 policy of the loads

    template <typename T>
    __device__ __forceinline__ RowSlice(const RowView<T>& r, int per, int ring, int rank, int warp,
                                        const char* smem, uint64_t hint_)
        : hint(hint_) {
        lo = min(rank * per, r.nvec);
        hi = min(lo + per, r.nvec);
        const int pw = G::warp_vecs(hi - lo);
        wlo = min(lo + warp * pw, hi);
        whi = min(wlo + pw, hi);
        steps = (whi - wlo + kStepVecs - 1) / kStepVecs;
        clean_lo = wlo < r.ilo ? 1 : 0;
        clean_hi = max(min(whi, r.ihi) - wlo, 0) / kStepVecs;
        slots = smem_u32(smem) + (uint32_t)(warp * ring * kStepVecs + (threadIdx.x & 31)) * 16u;
    }
    __device__ __forceinline__ bool clean(int step) const {
        return step >= clean_lo && step < clean_hi;
    }
    // A step that is not clean, from vector v on: -inf in the places beyond the warp's.
    template <typename T>
    static __device__ __noinline__ void load_edge(const RowView<T> r, int v, int whi, uint32_t at) {
        for (int i = 0; i < kStepVecs; i += 32, v += 32) {
            if (v < whi && r.inner(v))
                cp_async16(at + 16u * i, r.grid + (long long)v * RowView<T>::E);
            else if (v < whi)
                st_shared_v4(at + 16u * i, r.edge(v));
            else
                st_shared_v4(at + 16u * i, r.nothing());
        }
    }
    template <typename T>
    __device__ __forceinline__ void load(const RowView<T>& r, int step, const char* src,
                                         uint32_t at) const {
        if (clean(step)) {
#pragma unroll
            for (int i = 0; i < kStepVecs; i += 32)
                cp_async16_hint(at + 16u * i, src + 16 * i, hint);
        } else if ((unsigned)step < (unsigned)steps) {
            load_edge(r, wlo + step * kStepVecs + (int)(threadIdx.x & 31), whi, at);
        }
    }
    // This lane's first vector of a step.
    template <typename T>
    __device__ __forceinline__ const char* source(const RowView<T>& r, int step) const {
        return reinterpret_cast<const char*>(r.grid) +
               ((long long)wlo + (long long)step * kStepVecs + (threadIdx.x & 31)) * 16;
    }
    // Fills the ring for a first pass.  A step's copies are a group of their own, and
    // G::kRing groups are always under way or done.
    template <typename T>
    __device__ __forceinline__ void start(const RowView<T>& r) const {
        const char* src = source(r, 0);
#pragma unroll 1
        for (int i = 0; i < G::kRing; ++i) {
            load(r, i, src, slots + i * kStepBytes);
            cp_async_commit();
            src += kStepBytes;
        }
    }
    // f(vector's number, vector, whether it is whole) for this lane's vectors, and for
    // some of nothing but -inf beyond the warp's
    template <typename T, typename F>
    __device__ __forceinline__ void pass(const RowView<T>& r, F f) {
        const int by = up ? 1 : -1;
        int i = up ? 0 : steps - 1;
        uint32_t at = slots + (up ? 0 : max(i, 0) % G::kRing) * kStepBytes;
        const char* src = source(r, i + by * G::kRing);
        const uint32_t end = slots + G::kRing * kStepBytes;
#pragma unroll 1
        for (int n = steps; n > 0; --n) {
            cp_async_wait_group<G::kRing - 1>();
            const int v = wlo + i * kStepVecs + (int)(threadIdx.x & 31);
            const bool whole = clean(i);
            uint4 now[kStepVecs / 32];
#pragma unroll
            for (int h = 0; h < kStepVecs / 32; ++h) now[h] = lds_v4(at + h * 512);
#pragma unroll
            for (int h = 0; h < kStepVecs / 32; ++h) f(v + 32 * h, now[h], whole);
            load(r, i + by * G::kRing, src, at);
            cp_async_commit();
            i += by;
            src += by * (int)kStepBytes;
            at += by * (int)kStepBytes;
            if (at == end) at = slots;
            if (at < slots) at = end - kStepBytes;
        }
        up = !up;
    }
};

// How a [rows, V] array is split over clusters.
struct RowSplit {
    int lg;    // log2 of the CTAs per row (the cluster's size)
    int per;   // vectors of a row per CTA
    int ring;  // steps of a warp's ring
    int smem;  // bytes of a CTA's rings
};

// 16-byte vectors of a row of V elements of `es` bytes, wherever it starts.
inline long long row_max_vecs(long long V, size_t es) {
    const long long E = 16 / (long long)es;
    return (V + 2 * (E - 1)) / E;
}

// Slices of at most `slice` bytes; with few rows smaller ones, so that more SMs take
// part, but in clusters of 8 at most (16 x 151936 bf16, top-k: 12 us with 8 CTAs a row,
// 19 us with 16, whose barriers cost more than the shorter passes save).
constexpr long long kRowSliceMin = 16 * 1024;
template <typename G>
RowSplit split_rows(int rows, int V, size_t es, int num_sms,
                    long long slice = G::kSliceBytes) {
    const long long vecs = row_max_vecs(V, es), bytes = vecs * 16;
    int lg = 0;
    while (lg < 3 && (long long)rows << lg < (long long)G::kCtas * num_sms &&
           bytes >> lg > kRowSliceMin)
        ++lg;
    while (1 << lg < kRowMaxCluster && bytes >> lg > slice) ++lg;
    const int per = (int)((vecs + (1 << lg) - 1) >> lg), ring = G::ring_steps(per);
    return {lg, per, ring, ring * G::kStepBytes};
}

// Launches a kernel over `rows` clusters of 2^lg CTAs.  Its shared memory and cluster
// size go beyond the defaults: the attributes that allow this are set on the first
// launch on a device, and again where they turn out to be gone (a device reset).
template <typename G, auto KERNEL, typename Args>
cudaError_t launch_rows(const Args& a, int rows, int lg, size_t smem, size_t most_smem,
                        cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};  // a bit for each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)rows << lg));
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << lg;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = lg > 0 ? 1 : 0;
    const bool known = dev < 64 && (allowed.load(std::memory_order_relaxed) & bit) != 0;
    if (known) {
        e = cudaLaunchKernelEx(&cfg, KERNEL, a);
        if (e == cudaSuccess) return e;
        cudaGetLastError();
    }
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, KERNEL, a);
}

}  // namespace df2
