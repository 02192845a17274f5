// Optimizer states in 8 bits: 32 neighbours share a power of two, and each has the bits of a
// short float.
//
//   exp_avg     sign, 4 bits of exponent, 3 of mantissa (values 2^-9 to 480)
//   exp_avg_sq  5 bits of exponent, 3 of mantissa (values 2^-17 to 122880; no sign)
//
// value = short float * 2^(scale - 127); the block's largest lies in the second highest power
// of two (below 256 and 65536), so that rounding up, to these at most, cannot overflow.  Both
// short floats are the top of an fp32 number's bits at the bottom of its exponents: codes << 20 is
// the value times 2^-120 (2^-112), subnormal ones included, and back is an integer addition (the
// rounding) and a shift.
// Each product is by a power of two, so a value has at most 4 significant bits and is
// exact in bf16.  scale 255 stands for a block with an infinite or NaN value, which reads as NaN.
#pragma once

#include <cstdint>

namespace df2 {

constexpr int kStateBlock = 32;  // elements that share a scale

template <bool SQUARES>
struct State8 {
    // from the short float's exponents to the lowest of fp32's, and the highest that is used
    static constexpr uint32_t kField = SQUARES ? 112u : 120u;
    static constexpr int kTop = SQUARES ? 15 : 7;
    // Scales from here on take their power of two in two factors.
    static constexpr uint32_t kFar = 254u - kField;

    // 2^(scale - 127) * 2^kField as two factors, the first of which is all of it below kFar.  The
    // second says what scale 255 does.
    static __device__ __forceinline__ float unit(uint32_t scale) {
        return __uint_as_float(min(scale + kField, 254u) << 23);
    }
    static __device__ __forceinline__ float far_unit(uint32_t scale) {
        if (scale == 255u) return __uint_as_float(0x7f800000u);
        return __uint_as_float((127u + max((int)(scale + kField) - 254, 0)) << 23);
    }
    // The short float of the code in bits 24 to 31 (anything below), times 2^-kField.
    static __device__ __forceinline__ float raw(uint32_t high) {
        return __uint_as_float(SQUARES ? high >> 4 & 0x0ff00000u
                                       : (uint32_t)((int32_t)high >> 4) & 0x87f00000u);
    }

    // The scale of a block whose largest magnitude is `top` (NaN where one value is).
    static __device__ __forceinline__ uint32_t scale_of(float top) {
        const int field = (int)(__float_as_uint(top) >> 23);
        return field >= 255 ? 255u : (uint32_t)max(field - kTop, 1);
    }
    // Whether that is below kFar, and then by fewer operations.
    static __device__ __forceinline__ bool near(float top) {
        return __float_as_uint(top) < (kFar + kTop) << 23;
    }
    static __device__ __forceinline__ uint32_t near_scale_of(float top) {
        return (uint32_t)max((int)(__float_as_uint(top) >> 23) - kTop, 1);
    }
    static __device__ __forceinline__ float near_unit(uint32_t scale) {
        return __uint_as_float((scale + kField) << 23);
    }
    static __device__ __forceinline__ float near_down(uint32_t scale) {
        return __uint_as_float((254u - kField - scale) << 23);
    }
    // 2^(127 - scale) * 2^-kField, all of it below kFar, else without the second.
    static __device__ __forceinline__ float down(uint32_t scale) {
        return __uint_as_float(scale < kFar ? (254u - kField - scale) << 23
                                            : (254u - min(scale, 254u)) << 23);
    }
    static __device__ __forceinline__ float far_down(uint32_t scale) {
        return scale < kFar ? 1.f : SQUARES ? 0x1p-112f : 0x1p-120f;
    }
    // The code, in bits 24 to 31 over others, of a value x whose magnitude has the bits w after
    // down (and far_down).  chance: bits 8 to 23 say which way it goes, bit 7 is set, nothing
    // else; the nearest without CHANCE.
    template <bool CHANCE>
    static __device__ __forceinline__ uint32_t encode(float x, uint32_t w, uint32_t chance) {
        const uint32_t high =
            CHANCE ? w * 16u + chance : (w + 0x7ffffu + (w >> 20 & 1u)) * 16u;
        return SQUARES ? high : high | (__float_as_uint(x) & 0x80000000u);
    }
    // A square above 0 keeps a code above 0: at 0 the step would be divided by eps alone.
    static constexpr uint32_t kOne = 1u << 24;
    static __device__ __forceinline__ uint32_t above_zero(float x, uint32_t high) {
        return x > 0.f ? max(high, kOne) : high;
    }
};

}  // namespace df2
