// Codes of the 8-bit caches: what a code stands for, in the 16-bit operand types
// of the tensor cores and in f32.
//
// int8: two's complement.  Spread to the low bytes of 16-bit halves, a code's
// low seven bits over the exponent of 128 are the bf16 number 128 + low, its top
// bit over the same exponent gives 128 or 256: the difference is the code,
// exact.  In fp16 a byte over the exponent of 1024 is 1024 + (code + 128).
// e4m3: sign and magnitude moved to where the 16-bit type has them, times two to
// the difference of the exponents' biases; subnormal codes come out right since
// the product of a subnormal and a power of two is exact.  0x7f and 0xff, which
// stand for no number, become +-480 like any other code.
#pragma once

#include "common.cuh"

namespace w4a16 {

W4A16_DEVICE uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
W4A16_DEVICE uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes LO and HI of the eight of x (0 .. 3) and y (4 .. 7) as a pair, LO in the low half.
template <bool E4M3, bool BF, int LO, int HI>
W4A16_DEVICE uint32_t code_pair(uint32_t x, uint32_t y) {
    if constexpr (E4M3) {
        const uint32_t v = __byte_perm(x, y, (LO << 4) | LO | (HI << 12) | (HI << 8));  // each code in both bytes of its half
        if constexpr (BF) return bf16x2_mul(((v >> 4) & 0x07f007f0u) | (v & 0x80008000u), 0x7b807b80u);  // 2^120
        return f16x2_mul(((v >> 1) & 0x3f803f80u) | (v & 0x80008000u), 0x5c005c00u);                     // 2^8
    } else if constexpr (BF) {
        const uint32_t v = __byte_perm(x, y, (LO << 4) | LO | (HI << 12) | (HI << 8));
        return bf16x2_sub((v & 0x007f007fu) | 0x43004300u, (v & 0x00800080u) | 0x43004300u);
    } else {
        const uint32_t v = __byte_perm(x, y, (LO << 4) | LO | (HI << 12) | (HI << 8));
        return f16x2_sub(((v & 0x00ff00ffu) ^ 0x00800080u) | 0x64006400u, 0x64806480u);  // 1024 + 128
    }
}

// One code in f32.
template <bool E4M3>
W4A16_DEVICE float code_value(uint32_t c) {
    if constexpr (E4M3)  // exponent bias 7 -> 127
        return __uint_as_float(((c & 0x7fu) << 20) | ((c & 0x80u) << 24)) * __uint_as_float(247u << 23);
    else
        return (float)(int8_t)c;
}

// A scale that is not finite stands for NaN.
W4A16_DEVICE float finite_or_nan(float s) {
    return (__float_as_uint(s) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : s;
}

}  // namespace w4a16
