// The 8-bit row cache ("fp8row"): each row -- one token of one KV head -- is D
// E4M3 codes with one power-of-two scale of its own.
//
// A (block, KV head) tile is bs * (D + 1) contiguous bytes: the bs rows of D
// codes, then the bs scale bytes, so one bulk copy brings a tile with its
// scales and a block copy or swap moves both.  A scale byte b stands for
// 2^(b - 127); an element is code * 2^(b - 127).  A power of two costs E4M3
// nothing (its own exponent absorbs the up to one binade the scale rounds up
// by), makes x / scale and code * scale exact, and lets the attention kernels
// carry scales as exponents.
//
// Quantising a row x: e is the smallest exponent in [-60, 60] with max|x| <=
// 448 * 2^e; codes are x * 2^-e rounded once, to nearest even, saturating at
// +-448; b = e + 127.  The clamp keeps every product of scales and softmax
// weights below fp32's largest; a weight below 2^-126 beside the largest
// contribution counts as none, also in the sum (that takes V scales 2^100 apart in
// one context).  A row that holds a NaN gets b = 255 and NaN codes: it reads as NaN
// throughout.
#pragma once

#include "common.cuh"

namespace pkv {

struct fp8row {
    uint8_t bits;
};

template <> struct Elem<fp8row> : Elem<fp8e4m3> {};

// An E4M3 cache of either kind.
template <typename TC> constexpr bool kIsFp8 = false;
template <> inline constexpr bool kIsFp8<fp8e4m3> = true;
template <> inline constexpr bool kIsFp8<fp8row> = true;
template <typename TC> constexpr bool kRowScaled = false;
template <> inline constexpr bool kRowScaled<fp8row> = true;

constexpr int kRowScaleMin = 127 - 60, kRowScaleMax = 127 + 60, kRowScaleNan = 255;

// Bytes of one (block, KV head) tile.
template <typename TC>
__host__ __device__ constexpr int cache_tile_bytes(int D, int bs) {
    return bs * (D * (int)sizeof(TC) + (kRowScaled<TC> ? 1 : 0));
}

// Scale byte of a row whose largest |x| has these fp32 bits (the maximum taken
// on the bits, so that a NaN is above every number).  amax = 1.m * 2^x <= 1.75
// * 2^(8 + e): e = x - 8, one more if 1.m > 1.75 (m above 0x600000: the
// addition then carries into the exponent).
__device__ __forceinline__ int row_scale_byte(uint32_t amax_bits) {
    if (amax_bits > 0x7f800000u) return kRowScaleNan;
    const int b = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
    return min(max(b, kRowScaleMin), kRowScaleMax);
}

// 2^(b - 127), and its inverse; NaN for the byte of a NaN row.
__device__ __forceinline__ float row_scale(int b) {
    return __uint_as_float(b == kRowScaleNan ? 0x7fffffffu : (uint32_t)b << 23);
}
__device__ __forceinline__ float row_scale_inv(int b) {
    return __uint_as_float(b == kRowScaleNan ? 0x7fffffffu : (uint32_t)(254 - b) << 23);
}
// b - 127 as a float; NaN for the byte of a NaN row.
__device__ __forceinline__ float row_exponent(int b) {
    return b == kRowScaleNan ? __uint_as_float(0x7fffffffu) : (float)(b - 127);
}

}  // namespace pkv
