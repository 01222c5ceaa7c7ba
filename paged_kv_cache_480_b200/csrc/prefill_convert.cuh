// K and V tiles of the prefill kernel from an E4M3 cache: the tensor core takes
// both operands of a product in q's 16-bit type, so converting warps turn the
// codes of each 128-key tile into that type on their way to shared memory, in
// the 128-byte-swizzled layout that TMA gives the 16-bit caches.
//
// A code has four significant bits, so code * 2^e is exact in 16 bits but at
// the ends of fp16's range.  The codes come through bulk copies, not loads
// into registers: the proxy fence after each converted tile would wait for
// outstanding loads, and with them for a memory latency a tile (measured).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "fp8row.cuh"

namespace pkv {

// Two E4M3 codes, y = b0 | b1 << 16, as two bf16 values times 2^-120: the code's
// exponent and fraction moved to the low end of bf16's exponent and the top of
// its fraction, m << 4 with m = y & 0x7f, its sign (y - m) << 8: 256 y - 240 m.
// Multiply-adds with the factors in registers, because shifts and masks share
// the half-rate integer pipe with most of the softmax and would bind it.
struct Bf16Factors {
    uint32_t up = 256u, down = (uint32_t)-240;
    __device__ __forceinline__ Bf16Factors() { asm volatile("" : "+r"(up), "+r"(down)); }
};
__device__ __forceinline__ uint32_t e4m3_to_bf16x2_raw(uint32_t y, const Bf16Factors& f) {
    return (y & 0x007f007fu) * f.down + y * f.up;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
// Finite and infinite halves to +-65504 at most; NaN stays.
__device__ __forceinline__ uint32_t clamp_f16x2(uint32_t a) {
    const uint32_t most = 0x7bff7bffu, least = 0xfbfffbffu;
    __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<const __half2*>(&most));
    r = __hmax2_nan(r, *reinterpret_cast<const __half2*>(&least));
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t twice16(uint32_t h) { return h | (h << 16); }

// 16 codes as 16-bit values, lo the codes 0-7; of a row cache times the pair
// multiplier m, 2^e in both halves for fp16 and 2^(120 + e) for bf16 (rows with
// NaN codes have a NaN multiplier, so the codes' own NaN need no care there).
template <typename T, bool ROW>
__device__ __forceinline__ void convert16(const uint4& c, uint32_t m, const Bf16Factors& f, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
            o[2 * i] = e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu));
            o[2 * i + 1] = e4m3x2_to_f16x2((uint16_t)(w[i] >> 16));
            if constexpr (ROW) {
                o[2 * i] = mul_f16x2(o[2 * i], m);
                o[2 * i + 1] = mul_f16x2(o[2 * i + 1], m);
            }
        } else if constexpr (!ROW) {
            // through fp16 and fp32: no scale to apply, and NaN codes stay NaN
            float a0, a1, b0, b1;
            Elem<__half>::widen2(e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu)), a0, a1);
            Elem<__half>::widen2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)), b0, b1);
            o[2 * i] = Elem<__nv_bfloat16>::pack2(a0, a1);
            o[2 * i + 1] = Elem<__nv_bfloat16>::pack2(b0, b1);
        } else {
            o[2 * i] = mul_bf16x2(e4m3_to_bf16x2_raw(__byte_perm(w[i], 0, 0x4140), f), m);
            o[2 * i + 1] = mul_bf16x2(e4m3_to_bf16x2_raw(__byte_perm(w[i], 0, 0x4342), f), m);
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Pair multipliers of scale bytes: one multiply-add for the exponents whose
// multiplier is a normal number of the type, fp16: -14 .. 15, bf16: up to 7
// (down to the -60 of the format).  For any other byte two products: the first
// exact (down: codes are multiples of 2^-9,
// times 2^-12 still of 2^-21) or an overflow (up).
template <typename T>
struct PairScale {
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    static constexpr int LO = kHalf ? 127 - 14 : 1, HI = kHalf ? 127 + 15 : 127 + 7;
    // up to it no element overflows (448 * 2^7 < 65504), and slices take the short way
    static constexpr int FAST = 127 + 7;
    __device__ __forceinline__ static uint32_t of(int b) {
        return kHalf ? (uint32_t)(b - 112) * 0x04000400u : (uint32_t)(b + 120) * 0x00800080u;
    }
    // m for the byte, and a second multiplier
    __device__ __forceinline__ static uint32_t first(int b) {
        if (b == kRowScaleNan) return 0x7fff7fffu;
        return kHalf ? of(b < LO ? 127 - 12 : HI) : of(127);
    }
    __device__ __forceinline__ static uint32_t second(int b) {
        if (b == kRowScaleNan) return of(127);
        if constexpr (kHalf) {
            const int r = b < LO ? b + 12 : min(b - 15, HI);          // byte of the rest
            return twice16(r >= LO ? (uint32_t)(r - 112) << 10 : 1u << (max(r, 127 - 24) - 103));
        }
        return twice16((uint32_t)b << 7);                             // 2^e as bf16
    }
};

// Elements of V that are no finite numbers of q's type (NaN, and beyond fp16's
// range infinities) cannot stay in a tile of which some query sees only a part:
// a hidden key's weight is 0, and 0 * NaN is NaN.  The converting warps take
// them out and note where they begin: for each dim the first position of an
// element that is +inf or NaN, and of one that is -inf or NaN.  The output takes
// them from there (both: NaN).  An entry is the item's tag in its high and ~position
// in its low half, so the largest of a slot is its newest item's first position,
// and no slot is ever cleared.
struct Aside {
    unsigned long long* at = nullptr;   // [2][D] entries of the item's slot; null: elements stay in the tile
    uint32_t* any = nullptr;            // the tag, once there is an entry
    uint32_t tag = 0;
    int t0 = 0;                         // position of the slice's first row
    bool scan = false;                  // per-tensor caches: the slice has keys that some query of the item does not see
};

__device__ __forceinline__ unsigned long long aside_entry(uint32_t tag, int position) {
    return (unsigned long long)tag << 32 | (0xffffffffu - (uint32_t)position);
}
// Whether a query at pos sees the entry's element.
__device__ __forceinline__ bool aside_seen(unsigned long long entry, uint32_t tag, int pos) {
    return (uint32_t)(entry >> 32) == tag && (int)(0xffffffffu - (uint32_t)entry) <= pos;
}

// 16 codes of the row with scale byte b (per-tensor caches: 127) at position t, dims d
// .. d + 15: those that are not finite in T become zeros and entries.  A loop, and
// nothing unrolled: it hardly ever runs, and the code around it has to stay in the
// instruction caches.  (In place: a role of a kernel that shares its registers out
// calls no functions.)
template <typename T, int D>
__device__ __forceinline__ void take_out(uint4& c, int& b, const Aside& aside, int t, int d) {
    const unsigned long long entry = aside_entry(aside.tag, t);
    const float most = (std::is_same<T, __half>::value ? 65504.f : INFINITY), scale = row_scale(b);
#pragma unroll 1
    for (int k = 0; k < 16; ++k) {
        const uint32_t code = c.x & 0xffu;
        const uint32_t h = e4m3x2_to_f16x2((uint16_t)code);
        const float x = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu))) * scale;
        const bool fine = fabsf(x) <= most;
        if (!fine) {
            if (!(x < 0.f)) atomicMax(aside.at + d + k, entry);
            if (!(x > 0.f)) atomicMax(aside.at + D + d + k, entry);
            *aside.any = aside.tag;
        }
        // the next code to the front, this one (or zero) to the end
        const uint32_t last = fine ? code : 0u;
        c.x = __funnelshift_r(c.x, c.y, 8);
        c.y = __funnelshift_r(c.y, c.z, 8);
        c.z = __funnelshift_r(c.z, c.w, 8);
        c.w = __funnelshift_r(c.w, last, 8);
    }
    if (b == kRowScaleNan) b = 127;
}
// Whether one of 16 codes is 0x7f or 0xff.
__device__ __forceinline__ bool has_nan_code(const uint4& c) {
    auto carry = [](uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; };     // into bit 7 of the byte
    return ((carry(c.x) | carry(c.y) | carry(c.z) | carry(c.w)) & 0x80808080u) != 0;
}

// One warp's 32 rows of a 128-key tile: bulk copies bring them from their
// blocks into the warp's own staging slot (each block's rows, then its scale
// bytes); the warp converts them piece by piece (16 codes of a row) into the
// swizzled tile.  A lane takes NJ pieces of neighbouring rows, dealt so that
// the eight lanes of a shared-memory phase touch eight different 16-byte
// columns, both reading the slot (two rows of opposite halves, or of opposite
// parity for 64 dims) and writing the tile (rows of opposite parity).
//
// What bounds the chunk kernel is the issue slots these instructions take from
// the softmax (its time grows in step with the share of the slices converted),
// so their number counts: an address is one xor, a scale one multiply-add.
template <typename T, typename TC, int D, int BS>
struct SliceConverter {
    static constexpr int ROWS = 32;
    static constexpr int BLOCKS = ROWS / BS;            // blocks of a slice
    static constexpr int TILE = cache_tile_bytes<TC>(D, BS);
    static constexpr int SLOT = BLOCKS * TILE;          // staging bytes
    static constexpr int NJ = D / 16;                   // pieces (rows) a lane takes
    static constexpr bool kRow = kRowScaled<TC>;
    using P = PairScale<T>;
    static constexpr int kPairsUnrolled = 2;
    static_assert(D == 64 || D == 128, "head size");
    static_assert(BLOCKS * BS == ROWS && BS % NJ == 0, "a lane's rows lie in one block");

    int odd;            // piece j is row r0 + (j ^ odd) of the slice
    int r0;
    uint32_t src;       // codes of row r0 from the slot's start
    uint32_t sca;       // scale byte of row r0 from the slot's start
    // First column of piece 0 from the slice's first row in the tile; its second
    // column is at ^ 16, piece j at ^ (j * 128 | j * 16): the slice starts at a
    // multiple of 1 KB, a row is 128 bytes, its 16-byte columns are permuted by
    // the row's number mod 8.
    uint32_t dst;
    Bf16Factors factors;

    __device__ __forceinline__ explicit SliceConverter(int lane) {
        odd = (lane >> 2) & 1;
        r0 = NJ * (D == 128 ? odd | ((lane >> 4) << 1) : lane >> 2);
        const int d = (lane & 3) * 16 + (D == 128 ? 64 * (((lane >> 3) & 1) ^ odd) : 0);
        src = (r0 / BS) * TILE + (r0 % BS) * D + d;
        sca = (r0 / BS) * TILE + BS * D + r0 % BS;
        const int r = r0 + odd;         // the row of piece 0
        dst = (uint32_t)(d >> 6) * 16384u + r * 128 + (((uint32_t)(d & 63) / 8 ^ (r & 7)) << 4);
    }

    __device__ __forceinline__ static void put(uint32_t at, const uint4& lo, const uint4& hi) {
        sts128(at, lo);
        sts128(at ^ 16u, hi);
    }

    // The slot at shared address `slot` into a tile, its rows from address `tile`
    // on; rows at or past n, and rows of the blocks in `missing`, become zeros.  In
    // fp16 elements of K beyond its range are +-65504: an infinity would leave nothing
    // of a logit.
    __device__ __forceinline__ void run(uint32_t slot, uint32_t tile, int n, uint32_t missing, int lane, bool is_k,
                                        const Aside& aside = Aside()) const {
        bool plain = n >= ROWS && missing == 0;
        if constexpr (kRow) {
            // lane r looks at row r's scale
            const uint32_t far = (uint32_t)(lds8(slot + (lane / BS) * TILE + BS * D + lane % BS) - P::LO);
            plain = __all_sync(0xffffffffu, far <= (uint32_t)(P::FAST - P::LO)) && plain;
        } else if (aside.scan && plain) {
            bool nan = false;
#pragma unroll 4
            for (int j = 0; j < NJ; ++j) nan |= has_nan_code(lds128(slot + src + j * D));
            plain = !__any_sync(0xffffffffu, nan);
        }
        const uint32_t to = tile + dst;
        if (plain) {
            // (rows of even and of odd pieces)
            uint32_t even = slot + src + odd * D, other = slot + src + (1 ^ odd) * D;
            uint4 a = lds128(even), b = lds128(other);
            uint32_t sb[NJ / 4];        // the scale bytes, those of a pair in the order of its pieces
            if constexpr (kRow) {
#pragma unroll
                for (int k = 0; k < NJ / 4; ++k)
                    sb[k] = __byte_perm((uint32_t)lds32(slot + sca + 4 * k), 0, odd ? 0x2301 : 0x3210);
            }
#pragma unroll kPairsUnrolled
            for (int j = 0; j < NJ; j += 2) {
                const uint4 ca = a, cb = b;
                uint32_t ma = P::of(127), mb = ma;
                if constexpr (kRow) {
                    const uint32_t w = (NJ == 4 || j < 4 ? sb[0] : sb[NJ / 4 - 1]) >> (8 * (j & 2));
                    ma = P::of((int)(w & 0xffu));
                    mb = P::of((int)((w >> 8) & 0xffu));
                }
                if (j + 2 < NJ) {
                    a = lds128(even + (j + 2) * D);
                    b = lds128(other + (j + 2) * D);
                }
                uint4 lo, hi;
                convert16<T, kRow>(ca, ma, factors, lo, hi);
                put(to ^ (uint32_t)(j * 144), lo, hi);
                convert16<T, kRow>(cb, mb, factors, lo, hi);
                put(to ^ (uint32_t)((j + 1) * 144), lo, hi);
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < NJ; ++j) {
                const int u = j ^ odd;
                uint4 c = lds128(slot + src + u * D);
                int b = kRow ? lds8(slot + sca + u) : 127;
                if (r0 + u >= n || ((missing >> ((r0 + u) / BS)) & 1u)) {
                    c = make_uint4(0u, 0u, 0u, 0u);
                    b = 127;
                }
                if (aside.at && (kRow ? b > (P::kHalf ? P::FAST : kRowScaleMax) : has_nan_code(c)))
                    take_out<T, D>(c, b, aside, aside.t0 + r0 + u, (int)(src - (r0 / BS) * TILE) % D);
                const bool in = b >= P::LO && b <= P::HI;
                uint4 lo, hi;
                convert16<T, kRow>(c, in ? P::of(b) : P::first(b), factors, lo, hi);
                if constexpr (kRow) {
                    const uint32_t m2 = in ? P::kHalf ? 0x3c003c00u : 0x3f803f80u : P::second(b);
                    uint32_t* o[8] = {&lo.x, &lo.y, &lo.z, &lo.w, &hi.x, &hi.y, &hi.z, &hi.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) *o[k] = P::kHalf ? mul_f16x2(*o[k], m2) : mul_bf16x2(*o[k], m2);
                    if (P::kHalf && is_k && b > P::FAST) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) *o[k] = clamp_f16x2(*o[k]);
                    }
                }
                put(to ^ (uint32_t)(j * 144), lo, hi);
            }
        }
    }
};

}  // namespace pkv
