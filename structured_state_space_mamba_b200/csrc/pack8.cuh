// pack8.cuh -- the 8-bit activation checkpoint: blocks of 64 values along a row
// share one power-of-two step 2^(e - 127), e the block's exponent byte, and each
// value is a signed byte of steps.
//
// With a power of two, value / step and code * step are exact, so a value read
// back depends on nothing but the block's largest magnitude and the rounding
// to the nearest code (ties to even), and is a bf16 number (7 bits and a sign).
// A step of max / 127 would use up to one more bit of the code, for a division
// a value and four bytes a block in place of one.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

constexpr int kPackBlock = 64;

// Exponent byte of a block from the bits of its largest magnitude (sign
// cleared; a NaN's bits are above infinity's): the smallest e >= 1 with
// max < 127.5 * 2^(e - 127), so that the largest code rounds to at most 127.
// 127.5 = 1.9921875 * 2^6, so e is the exponent less 6, after a carry out of
// mantissas from .9921875 (0x7f0000) up.  At most 248 (64 steps of the next one
// are past the largest float): there alone codes saturate.  255 for a block with
// an infinity or a NaN.
__device__ __forceinline__ uint32_t pack8_exp(uint32_t maxbits) {
    const int e = min(max(int((maxbits + 0x10000u) >> 23) - 6, 1), 248);
    return maxbits >= 0x7f800000u ? 255u : uint32_t(e);
}
// Blocks from this byte on need pack8_code(); the others may take pack8_fast().
constexpr uint32_t kPackEdge = 248;
// 1 / step as a float (0 for the byte 255: every code of such a block is 0)
__device__ __forceinline__ float pack8_inv(uint32_t e) {
    return __uint_as_float(e == 255u ? 0u : (254u - e) << 23);
}
// step as a float; infinity for the byte 255, so that its codes, all 0, read
// back as NaN
__device__ __forceinline__ float pack8_step(uint32_t e) { return __uint_as_float(e << 23); }
// The code of v, -127 .. 127.  v * inv is exact, but for values far below the
// smallest step.  An infinity or NaN times 0 is NaN, which converts to 0.
__device__ __forceinline__ int pack8_code(float v, float inv) {
    return min(max(__float2int_rn(v * inv), -127), 127);
}
// The same in the low byte, below kPackEdge: adding 1.5 * 2^23 rounds to a whole
// number, ties to even, and leaves it in the low bits.  The conversion to an
// integer runs at a quarter of the rate, on the unit that the exponentials need.
__device__ __forceinline__ uint32_t pack8_fast(float v, float inv) {
    return __float_as_uint(fmaf(v, inv, 12582912.f));
}
// Four, and eight, values of a block as codes.
__device__ __forceinline__ uint32_t pack8_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t pack8_four(const float (&v)[4], uint32_t ex) {
    const float inv = pack8_inv(ex);
    if (ex < kPackEdge)
        return pack8_bytes(pack8_fast(v[0], inv), pack8_fast(v[1], inv), pack8_fast(v[2], inv), pack8_fast(v[3], inv));
    return pack8_bytes(pack8_code(v[0], inv), pack8_code(v[1], inv), pack8_code(v[2], inv), pack8_code(v[3], inv));
}
__device__ __forceinline__ uint2 pack8_eight(const float (&v)[8], uint32_t ex) {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    return make_uint2(pack8_four(lo, ex), pack8_four(hi, ex));
}
// Two codes (the low bytes of a word) as numbers: a byte with its sign bit flipped,
// in the mantissa of 2^23, is 8388736 + code.  Without conversions for the same
// reason.
__device__ __forceinline__ float2 unpack8_two(uint32_t w, float step) {
    const uint32_t u = w ^ 0x8080u;
    return make_float2((__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f) * step,
                       (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f) * step);
}

}  // namespace ssd
