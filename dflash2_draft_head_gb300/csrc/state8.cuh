// Optimizer states in 8 bits: 32 neighbours share a power of two, and each has the bits of a
// short float.
//
//   exp_avg     sign, 4 bits of exponent, 3 of mantissa (values 2^-9 to 240)
//   exp_avg_sq  5 bits of exponent, 3 of mantissa (values 2^-17 to 61440; no sign)
//
// value = short float * 2^(scale - 127); the block's largest lies in the second highest power
// of two, so that rounding up cannot overflow.  Both short floats are the top of an fp32
// number's bits at the bottom of its exponents: codes << 20 is the value times 2^-120 (2^-112),
// subnormal ones included, and back is an integer addition (the rounding) and a shift.
// Each product is by a power of two, so a value has at most 4 significant bits and is
// exact in bf16.  scale 255 stands for a block with an infinite or NaN value, which reads as NaN.
#pragma once

#include <cstdint>

namespace df2 {

constexpr int kStateBlock = 32;  // elements that share a scale

template <bool SQUARES>
struct State8 {
    // of the short float's smallest exponent to fp32's, and the highest one that is used
    static constexpr float kUp = SQUARES ? 0x1p112f : 0x1p120f;
    static constexpr float kDown = SQUARES ? 0x1p-112f : 0x1p-120f;
    static constexpr int kTop = SQUARES ? 15 : 7;

    static __device__ __forceinline__ float unit(uint32_t scale) {
        return __uint_as_float(scale << 23);
    }
    static __device__ __forceinline__ float decode(uint32_t code, float unit) {
        const uint32_t bits =
            SQUARES ? code << 20 : (code & 0x80u) << 24 | (code & 0x7fu) << 20;
        return __uint_as_float(bits) * kUp * unit;
    }
    // The scale of a block whose largest magnitude has these bits.
    static __device__ __forceinline__ uint32_t scale_of(uint32_t top) {
        const int field = (int)(top >> 23);
        return field == 255 ? 255u : (uint32_t)max(field - kTop, 1);
    }
    static __device__ __forceinline__ float down(uint32_t scale) {
        return __uint_as_float((254u - min(scale, 254u)) << 23);
    }
    // The code of x; `chance`: 16 bits that say which way it goes, or ~0 for the nearest.
    // A square above 0 keeps a code above 0: at 0 the step would be divided by eps alone.
    template <bool CHANCE>
    static __device__ __forceinline__ uint32_t encode(float x, float down, uint32_t chance) {
        const uint32_t w = __float_as_uint(fabsf(x) * down * kDown);
        uint32_t code = (w + (CHANCE ? chance << 4 | 8u : 0x7ffffu + (w >> 20 & 1u))) >> 20;
        if (SQUARES) return x > 0.f && code == 0u ? 1u : code;
        return code | (__float_as_uint(x) >> 24 & 0x80u);
    }
};

}  // namespace df2
