// The 8-bit checkpoint format (liger_train.h): groups of 32 columns of a row
// share a power-of-two step, E = floor(log2 max |x|), step = 2^(E - 6), int8
// codes.  A power of two needs one byte a group, makes the division and the
// reading back exact, and comes straight from the exponent bits of the group's
// largest magnitude.
#pragma once

#include "common.cuh"

namespace liger {

constexpr int kCkptGroup = 32;          // LIGER_CKPT8_GROUP
constexpr uint32_t kCkptMinExp = 16;    // biased exponents below this (magnitudes under 2^-111): zeros

// magnitude bits of x: ordered as the magnitudes are, infinities and NaN above all finite values
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// scale byte of a group from its largest magnitude bits
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t top) {
    const uint32_t e = top >> 23;   // biased exponent: E + 127, 255 with an infinity or NaN
    return e < kCkptMinExp ? 0u : e;
}
// 1 / step (exact; 0 for a group stored as zeros or as NaN)
__device__ __forceinline__ float ckpt_inv(uint32_t scale) {
    return scale == 0u || scale == 255u ? 0.f : __uint_as_float((260u - scale) << 23);   // 2^(133 - scale)
}
// step: 2^(scale - 133); 0 for zeros, NaN for 255
__device__ __forceinline__ float ckpt_step(uint32_t scale) {
    return scale == 0u ? 0.f : scale == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((scale - 6u) << 23);
}
// code of x as a signed byte in the low bits of the result (the others are not zero): adding
// 1.5 * 2^23 rounds to an integer, halves to even, and leaves it in the low mantissa bits
__device__ __forceinline__ uint32_t ckpt_code(float x, float inv) {
    float v = x * inv;                                   // exact, |v| < 128
    v = fminf(fmaxf(v, -127.f), 127.f);                  // a NaN (infinity times 0) becomes -127: its group reads back NaN
    return __float_as_uint(v + 12582912.f);
}
// four codes in a word, first in the low byte
__device__ __forceinline__ uint32_t ckpt_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// the four codes of a word as floats: byte + 128 in the mantissa of 2^23, less 2^23 + 128
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, float (&f)[4]) {
    const uint32_t x = w ^ 0x80808080u;
    f[0] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7650)) - 8388736.f;
    f[1] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7651)) - 8388736.f;
    f[2] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7652)) - 8388736.f;
    f[3] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7653)) - 8388736.f;
}

}  // namespace liger
