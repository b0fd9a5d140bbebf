// tq_decode.cuh -- packed codes to fp16 operands in registers.
//
// Codes are turned to fp16 by byte permutation: a register whose nibbles are codes is the selector
// that picks the high, then the low bytes of four table entries (two permutations a four codes
// each), and two more interleave them to fp16 pairs.  With the selectors, which come from the bit
// planes by shifts and masks, that is about 1.5 to 2 instructions a value, against 6 and more for
// shifting each code out.  4-bit value codes use the codebook's antisymmetry: a table of 8
// magnitudes, the top bit as the sign.
#pragma once

#include <stdint.h>

namespace tq {
namespace decode {

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// Selectors of N bits: nibble n of x[i] = bits 4 n + i of the planes w[0 .. N-1].
template <int N>
__device__ __forceinline__ void selectors(const uint32_t *w, uint32_t (&x)[4]) {
    if constexpr (N == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (w[0] >> i) & 0x11111111u;
    } else {
        const uint32_t a = pick(w[0], w[1] << 1, 0x55555555u);  // nibble: w0.0 w1.0 w0.2 w1.2
        const uint32_t b = pick(w[0] >> 1, w[1], 0x55555555u);  // nibble: w0.1 w1.1 w0.3 w1.3
        if constexpr (N == 2) {
            x[0] = a & 0x33333333u;
            x[1] = b & 0x33333333u;
            x[2] = (a >> 2) & 0x33333333u;
            x[3] = (b >> 2) & 0x33333333u;
        } else {
            x[0] = pick(a, w[2] << 2, 0x33333333u) & 0x77777777u;
            x[1] = pick(b, w[2] << 1, 0x33333333u) & 0x77777777u;
            x[2] = pick(a >> 2, w[2], 0x33333333u) & 0x77777777u;
            x[3] = pick(b >> 2, w[2] >> 1, 0x33333333u) & 0x77777777u;
        }
    }
}

// A table of up to 8 fp16 numbers, its high and its low bytes.
struct Lut {
    uint32_t h0, h1, l0, l1;
};

template <int N>
__device__ __forceinline__ Lut load_lut(const uint16_t *t) {
    Lut u = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t v = t[k];
        (k < 4 ? u.h0 : u.h1) |= (v >> 8) << (8 * (k & 3));
        (k < 4 ? u.l0 : u.l1) |= (v & 255u) << (8 * (k & 3));
    }
    return u;
}

// Bytes of (a, b) by the nibbles of `sel`, each 0..7.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// The four numbers that the low 16 bits of the selector pick, as two pairs.  `flip`: bytes to xor
// into the high bytes.
__device__ __forceinline__ void look_up(const Lut &t, uint32_t sel, uint32_t flip, uint32_t &p0, uint32_t &p1) {
    const uint32_t h = prmt(t.h0, t.h1, sel) ^ flip, l = prmt(t.l0, t.l1, sel);
    p0 = prmt(l, h, 0x5140);
    p1 = prmt(l, h, 0x7362);
}

// x >> 16 on the multiplier (two16 is 2^16, from where the compiler cannot see it): decoding is bound
// by the pipe that shifts, masks and permutes.
__device__ __forceinline__ uint32_t half_up(uint32_t x, uint32_t two16) {
    uint32_t r;
    asm("mul.hi.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(two16));
    return r;
}

// 2-bit codes straight to pairs of fp16 numbers: with a table of four numbers in two registers, code
// c is its bytes 2 c and 2 c + 1, so the selector of a code is the byte 0x22 c + 0x10, a product.
// selector(i) has the codes of bits i, i + 8, i + 16 and i + 24.
struct Pairs2 {
    uint32_t a, b;  // even and odd bits: fields of two, (w0, w1) of one bit
    __device__ __forceinline__ Pairs2(uint32_t w0, uint32_t w1)
        : a(pick(w0, w1 << 1, 0x55555555u)), b(pick(w0 >> 1, w1, 0x55555555u)) {}
    __device__ __forceinline__ uint32_t selector(int i) const {
        return (((i & 1 ? b : a) >> (i & 6)) & 0x03030303u) * 0x22u + 0x10101010u;
    }
};

}  // namespace decode
}  // namespace tq
