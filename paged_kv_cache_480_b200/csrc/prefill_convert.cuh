// K and V tiles of the prefill kernel from an E4M3 cache: the tensor core takes
// both operands of a product in q's 16-bit type, so four warps turn the codes
// of each 128-key tile into that type on their way to shared memory, in the
// 128-byte-swizzled layout that TMA gives the 16-bit caches.
//
// A code has four significant bits, so code * 2^e is exact in 16 bits but at
// the ends of fp16's range.  Codes come straight from global memory into
// registers, a whole tile ahead of their conversion (16 KB in flight a stream
// and SM), so they need no staging in shared memory.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "fp8row.cuh"

namespace pkv {

// Two E4M3 codes (in the high bytes of x's halves) as two bf16 values times
// 2^-120: the code's exponent and fraction moved to the low end of bf16's
// exponent and the top of its fraction.
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2_raw(uint32_t x) {
    return ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t twice16(uint32_t h) { return h | (h << 16); }

// 16 codes of one row with scale byte b, as 16-bit values: lo holds codes 0-7.
template <typename T, bool ROW>
__device__ __forceinline__ void convert16(const uint4& c, int b, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
    if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu));
            o[2 * i + 1] = e4m3x2_to_f16x2((uint16_t)(w[i] >> 16));
        }
        if constexpr (ROW) {
            // 2^e as an fp16 multiplier: one rounding.  Outside fp16's powers
            // of two, two steps of which the first is exact (down: codes are
            // multiples of 2^-9, times 2^-12 still of 2^-21) or overflows (up).
            const int e = b - 127;
            uint32_t m = e >= -14 ? (uint32_t)(e + 15) << 10 : 1u << (max(e, -24) + 24);
            if (e < -24 || e > 15) {
                const uint32_t first = twice16(b == kRowScaleNan ? 0x7fffu : e < 0 ? 3u << 10 : 30u << 10);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = mul_f16x2(o[i], first);
                const int r = e < 0 ? e + 12 : min(e - 15, 15);
                m = r >= -14 ? (uint32_t)(r + 15) << 10 : 1u << (max(r, -24) + 24);
            }
            m = twice16(m);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = mul_f16x2(o[i], m);
        }
    } else {
        const int e = ROW ? b - 127 : 0;
        // 2^(120 + e): one exact product; two where that is above bf16's largest
        uint32_t m = 0x7b80u;
        if constexpr (ROW) m = b == kRowScaleNan ? 0x7fffu : e <= 7 ? (uint32_t)(b + 120) << 7 : 0x7b80u;
        m = twice16(m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = mul_bf16x2(e4m3_hi_to_bf16x2_raw(__byte_perm(w[i], 0, 0x1404)), m);
            o[2 * i + 1] = mul_bf16x2(e4m3_hi_to_bf16x2_raw(__byte_perm(w[i], 0, 0x3424)), m);
        }
        if (ROW && e > 7 && b != kRowScaleNan) {
            const uint32_t up = twice16((uint32_t)b << 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], up);
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One thread's share of a 128-key tile: NJ pieces of 16 codes.  A warp step
// covers 512 contiguous bytes of codes; within it the lanes are ordered so
// that the eight lanes of a shared-memory phase write eight different 16-byte
// columns of the swizzled rows (even columns from one row, odd from the next).
template <typename T, typename TC, int D, int BS>
struct TileCodes {
    static constexpr int RPW = 512 / D;          // rows a warp step covers
    static constexpr int RPS = 4 * RPW;          // rows the four warps cover
    static constexpr int NJ = 128 / RPS;
    static constexpr bool kRow = kRowScaled<TC>;
    static constexpr int TILE = cache_tile_bytes<TC>(D, BS);

    uint4 c[NJ];
    int b[kRow ? NJ : 1];

    __device__ __forceinline__ static int dim0(int lane) { return (lane & 3) * 16 + (D == 128 ? ((lane >> 3) & 1) * 64 : 0); }
    __device__ __forceinline__ static int row0(int w, int lane) {
        return w * RPW + (D == 128 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2);
    }

    // tbl: lane j holds the tile's j-th physical block id (negative: none);
    // rows past nrows of the tile and rows of no block read as zeros
    __device__ __forceinline__ void load(const unsigned char* cache, int tbl, int Hkv, int g, int nrows, int w, int lane) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int t = j * RPS + row0(w, lane);
            const int phys = __shfl_sync(0xffffffffu, tbl, t / BS);
            c[j] = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kRow) b[j] = 127;
            if (t < nrows && phys >= 0) {
                const unsigned char* tile = cache + ((int64_t)phys * Hkv + g) * TILE;
                c[j] = __ldg(reinterpret_cast<const uint4*>(tile + (t % BS) * D + dim0(lane)));
                if constexpr (kRow) b[j] = __ldg(tile + BS * D + t % BS);
            }
        }
    }

    // into the swizzled tile at shared address dst (64-dim halves of 16 KB)
    __device__ __forceinline__ void store(uint32_t dst, int w, int lane) const {
        const int d = dim0(lane), ch = (d & 63) / 8;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int t = j * RPS + row0(w, lane);
            uint4 lo, hi;
            convert16<T, kRow>(c[j], kRow ? b[j] : 127, lo, hi);
            const uint32_t row = dst + (uint32_t)((d >> 6) * 16384 + t * 128);
            sts128(row + (((uint32_t)ch ^ (t & 7)) << 4), lo);
            sts128(row + (((uint32_t)(ch + 1) ^ (t & 7)) << 4), hi);
        }
    }
};

}  // namespace pkv
