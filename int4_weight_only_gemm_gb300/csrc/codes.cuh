// Codes of the 8-bit caches: what a code stands for, in the 16-bit operand types
// of the tensor cores and in f32.
//
// int8: two's complement.  In the low byte of a 16-bit half, a code's low seven
// bits over the exponent of 128 are the bf16 number 128 + low, its top bit over
// the same exponent gives 128 or 256: the difference is the code, exact.  In fp16
// a byte over the exponent of 1024 is 1024 + (code + 128).
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

// (a & b) | c and (a & b) ^ c in one instruction each.  Written out, since of the plain expressions the compiler makes
// two, and unpacking is what the kernels over 8-bit caches spend their time on (64 requests: 150 us with two, 121 with one).
W4A16_DEVICE uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
W4A16_DEVICE uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// The number that int8 codes are laid over, kept in a register: an instruction takes one constant operand, the mask.
template <bool BF>
W4A16_DEVICE uint32_t code_base() {
    uint32_t x;
    if constexpr (BF) asm volatile("mov.b32 %0, 0x43004300;" : "=r"(x));
    else asm volatile("mov.b32 %0, 0x64806480;" : "=r"(x));
    return x;
}
// The codes in bytes 0 and 2 of w (ODD: 1 and 3) as a pair, the lower byte's in the low half; base: code_base<BF>().
template <bool E4M3, bool BF, bool ODD>
W4A16_DEVICE uint32_t code_pair(uint32_t w, uint32_t base) {
    if constexpr (E4M3) {
        const uint32_t sign = (ODD ? w : w << 8) & 0x80008000u;
        if constexpr (BF) return bf16x2_mul(and_or(ODD ? w >> 4 : w << 4, 0x07f007f0u, sign), 0x7b807b80u);  // 2^120
        return f16x2_mul(and_or(ODD ? w >> 1 : w << 7, 0x3f803f80u, sign), 0x5c005c00u);                    // 2^8
    } else {
        const uint32_t v = ODD ? w >> 8 : w;
        if constexpr (BF) return bf16x2_sub(and_or(v, 0x007f007fu, base), and_or(v, 0x00800080u, base));
        return f16x2_sub(and_xor(v, 0x00ff00ffu, base), base);  // (the top bit flipped: + 128)
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

// A scale that is not finite stands for NaN (infinity times 0 is one).
W4A16_DEVICE float finite_or_nan(float s) { return __fmaf_rn(s, 0.f, s); }

}  // namespace w4a16
