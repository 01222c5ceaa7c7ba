// Row kernels around the paged cache: rotary positions of q and k (alone, or
// fused with the cache write), the quantising cache write, and the read-back
// of whole sequences.  All are bound by HBM (each element is read and written
// once) for many tokens and by latency for a few.
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "fp8row.cuh"
#include "pagedkv.h"
#include "row_ops.cuh"

namespace pkv {
namespace {

// packed fp32 pairs
__device__ __forceinline__ uint64_t f2pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2unpack(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2sub(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

constexpr int kThreads = 128;       // about that many a CTA (run_rotary); up to 32 more
constexpr int kMostThreads = kThreads + 32;

// Row lengths are multiples of 2 * kPerChunk elements, and a thread takes
// kPerChunk pairs of one row: rotary pairs (2i, 2i + 1) or (i, i + rot / 2),
// and beyond the rotated part neighbours.  A unit's elements are loaded and
// stored in runs of W: whole 16-byte chunks unless the half layout's offset
// rot / 2 is not a whole number of those, then as many elements as divide it
// (12,968 tokens of 39 + 39 heads of 80, 40 rotated: 63 us with runs of 4, 358
// one by one).  A pair lives in one thread, so q_out may be q and k_out may be k.
template <int N> struct Run;
template <> struct Run<1> { using type = unsigned char; };
template <> struct Run<2> { using type = uint16_t; };
template <> struct Run<4> { using type = uint32_t; };
template <> struct Run<8> { using type = uint2; };
template <> struct Run<16> { using type = uint4; };

template <typename T, bool INTERLEAVED, int W>
struct Unit {
    static constexpr int E = Elem<T>::kPerChunk;
    using Elements = typename Run<W * sizeof(T)>::type;
    using Codes = typename Run<W>::type;
    static_assert(W <= E && (W == E || !INTERLEAVED), "runs of a unit");

    // First elements of the two runs that hold W pairs from pair i on.
    __device__ __forceinline__ static int2 runs(int i, int rot) {
        if (!INTERLEAVED && i < rot / 2) return make_int2(i, i + rot / 2);
        return make_int2(2 * i, 2 * i + W);
    }

    // A unit's elements as they are in memory: the first and the second runs.
    struct Raw {
        uint4 a, b;
    };
    __device__ __forceinline__ static Raw fetch(const T* row, int u, int rot) {
        Raw x;
#pragma unroll
        for (int k = 0; k < E / W; ++k) {
            const int2 c = runs(u * E + k * W, rot);
            reinterpret_cast<Elements*>(&x.a)[k] = *reinterpret_cast<const Elements*>(row + c.x);
            reinterpret_cast<Elements*>(&x.b)[k] = *reinterpret_cast<const Elements*>(row + c.y);
        }
        return x;
    }
    __device__ __forceinline__ static void widen(const Raw& r, float (&x)[2 * E]) {
        Elem<T>::widen(r.a, x);
        Elem<T>::widen(r.b, x + E);
    }
    __device__ __forceinline__ static Raw narrow(const float (&x)[2 * E]) {
        return Raw{Elem<T>::narrow(x), Elem<T>::narrow(x + E)};
    }

    // Where a token's pair i keeps cos (sin two floats further): pairs i and i + 1
    // of a unit share four floats, and those of neighbouring units are
    // neighbours (span = ceil(rot / 2 / E) units), so that the lanes of a read
    // touch different banks.
    __device__ __forceinline__ static int angle(int i, int span) {
        return ((i % E) / 2 * span + i / E) * 4 + (i & 1);
    }

    // The unit's pairs by their angles, two at a time in packed fp32.
    __device__ __forceinline__ static void rotate(const float4* cs, int span, int u, int rot, float (&x)[2 * E]) {
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            float& a0 = x[INTERLEAVED ? 2 * j : j];
            float& b0 = x[INTERLEAVED ? 2 * j + 1 : E + j];
            float& a1 = x[INTERLEAVED ? 2 * j + 2 : j + 1];
            float& b1 = x[INTERLEAVED ? 2 * j + 3 : E + j + 1];
            const float4 w = cs[j / 2 * span + u];
            const uint64_t c = f2pack(w.x, w.y), s = f2pack(w.z, w.w), a = f2pack(a0, a1), b = f2pack(b0, b1);
            const uint64_t ya = f2sub(f2mul(a, c), f2mul(b, s)), yb = f2fma(a, s, f2mul(b, c));
            if (W == E && !INTERLEAVED) {           // whole units are rotated or none of it
                f2unpack(ya, a0, a1);
                f2unpack(yb, b0, b1);
            } else {
                float p0, p1, q0, q1;
                f2unpack(ya, p0, p1);
                f2unpack(yb, q0, q1);
                if (u * E + j < rot / 2) { a0 = p0; b0 = q0; }
                if (u * E + j + 1 < rot / 2) { a1 = p1; b1 = q1; }
            }
        }
    }

    __device__ __forceinline__ static void put(T* row, int u, int rot, const Raw& r) {
#pragma unroll
        for (int k = 0; k < E / W; ++k) {
            const int2 c = runs(u * E + k * W, rot);
            *reinterpret_cast<Elements*>(row + c.x) = reinterpret_cast<const Elements*>(&r.a)[k];
            *reinterpret_cast<Elements*>(row + c.y) = reinterpret_cast<const Elements*>(&r.b)[k];
        }
    }

    // E codes of one chunk as bytes, E = 4 or 8
    __device__ __forceinline__ static void codes(const float* x, float mult, uint32_t (&w)[E / 4]) {
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
            const uint32_t lo = f32x2_to_e4m3x2(x[4 * j] * mult, x[4 * j + 1] * mult);
            const uint32_t hi = f32x2_to_e4m3x2(x[4 * j + 2] * mult, x[4 * j + 3] * mult);
            w[j] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ static void store_codes(unsigned char* row, int u, int rot, const float (&x)[2 * E],
                                                       float mult) {
        __align__(8) uint32_t a[E / 4], b[E / 4];
        codes(x, mult, a);
        codes(x + E, mult, b);
#pragma unroll
        for (int k = 0; k < E / W; ++k) {
            const int2 c = runs(u * E + k * W, rot);
            *reinterpret_cast<Codes*>(row + c.x) = reinterpret_cast<const Codes*>(a)[k];
            *reinterpret_cast<Codes*>(row + c.y) = reinterpret_cast<const Codes*>(b)[k];
        }
    }
};

// n / d for small numbers (n * d below 2^32), from the launcher's inverse of d.
__device__ __forceinline__ int divide(int n, uint32_t inverse) {
    return inverse ? (int)__umulhi((uint32_t)n, inverse) : n;
}
uint32_t inverse_of(int d) { return d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d); }

// cos and sin of position * inv_freq.  The product and its reduction to a
// fraction of a turn are in fp64 (an fp32 angle of a far position is off by
// whole radians).  sincospif takes the fraction as fp32; what that leaves off, up
// to 2^-26 of a turn, goes into the first-order terms: without them cosines are
// off by 3.3e-8 rms, with them by about what rounding them twice costs.
__device__ __forceinline__ float2 turn(int64_t position, float inv_freq, float mscale) {
    const double t = (double)position * (double)inv_freq * 0.15915494309189535;   // 1 / (2 pi)
    const double r = t - rint(t);
    const float f = (float)r, rest = (float)(r - (double)f) * 6.2831855f;
    float s, c;
    sincospif(2.f * f, &s, &c);
    return make_float2(fmaf(-s, rest, c) * mscale, fmaf(c, rest, s) * mscale);
}

// grid.x takes tokens (tokens_cta a CTA), grid.y parts of a token's units (a
// few tokens are spread over the SMs that way).  A thread takes kDepth units
// at a time and has all their loads in flight before it works on the first;
// those of the first round are requested before the CTA takes cos and sin of
// its tokens' positions, one thread a frequency, into shared memory where every
// head of the token reads them.
constexpr int kDepth = 2;
constexpr int kMaxTokens = 8;   // of a CTA

template <typename T, RowSink SINK, bool INTERLEAVED, int W>
__global__ void __launch_bounds__(kMostThreads) rotary_kernel(const RotaryParams p) {
    using U = Unit<T, INTERLEAVED, W>;
    using UV = Unit<T, true, U::E>;        // rows that are not rotated: plain chunks
    constexpr int E = U::E;
    constexpr bool kCached = SINK != RowSink::kRows;
    extern __shared__ __align__(16) float angles[];
    __shared__ int64_t slots[kMaxTokens];
    griddep_wait();
    griddep_launch();
    const int half = p.rot / 2, span = (half + E - 1) / E;
    const int64_t token0 = (int64_t)blockIdx.x * p.tokens_cta;
    const int tokens = (int)min((int64_t)p.tokens_cta, p.num_tokens - token0);
    const int first = blockIdx.y * p.units_cta;
    const int last = min(first + p.units_cta, p.units_token * tokens);
    const int D = p.head_size, H = p.num_heads, Hkv = p.num_kv_heads;

    // Unit w of the CTA: token t, row (q rows, then k, then v), part u of the row.
    struct Where {
        int t, row, u;
    };
    auto where = [&](int w) {
        Where x{-1, 0, 0};
        if (w < last) {
            x.t = tokens == 1 ? 0 : divide(w, p.token_inverse);
            const int rem = w - x.t * p.units_token;
            x.row = divide(rem, p.row_inverse);
            x.u = rem - x.row * p.units_row;
        }
        return x;
    };
    auto fetch = [&](const Where& x) {
        typename U::Raw r;
        r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
        if (x.t >= 0) {
            const int64_t token = token0 + x.t;
            if (x.row < H) {
                r = U::fetch(static_cast<const T*>(p.q) + token * p.q_stride + (int64_t)x.row * D, x.u, p.rot);
            } else if (!kCached || x.row < H + Hkv) {
                r = U::fetch(static_cast<const T*>(p.k) + token * p.k_stride + (int64_t)(x.row - H) * D, x.u, p.rot);
            } else {
                const typename UV::Raw v =
                    UV::fetch(static_cast<const T*>(p.v) + token * p.v_stride + (int64_t)(x.row - H - Hkv) * D, x.u, 0);
                r.a = v.a;
                r.b = v.b;
            }
        }
        return r;
    };
    const float4* cs = reinterpret_cast<const float4*>(angles);
    const int cs_token = span * E / 2;     // float4s of a token's angles
    auto finish = [&](const Where& w, typename U::Raw raw) {
        const bool is_v = kCached && w.row >= H + Hkv;
        const bool turned = w.t >= 0 && !is_v && w.u * E < half;
        const int64_t token = token0 + w.t;
        float x[2 * E];
        // (a unit that is neither rotated nor quantised goes on as it came)
        if (SINK == RowSink::kCacheFp8Row || turned) {
            U::widen(raw, x);
            if (turned) U::rotate(cs + w.t * cs_token, span, w.u, p.rot, x);
            if (SINK != RowSink::kCacheFp8Row || w.row < H) raw = U::narrow(x);
        }
        if (w.t >= 0 && w.row < H)
            U::put(static_cast<T*>(p.q_out) + token * p.q_out_stride + (int64_t)w.row * D, w.u, p.rot, raw);
        if constexpr (!kCached) {
            if (w.t >= 0 && w.row >= H)
                U::put(static_cast<T*>(p.k_out) + token * p.k_out_stride + (int64_t)(w.row - H) * D, w.u, p.rot, raw);
        } else {
            const int g = w.row - H - (is_v ? Hkv : 0);
            int64_t slot = -1;
            if (w.t >= 0 && w.row >= H) {
                slot = slots[w.t];
                if (slot >= p.pool_slots) {
                    if (w.u == 0 && g == 0 && !is_v) flag_error(p.errors, PKV_DEVERR_SLOT);
                    slot = -1;
                }
            }
            const bool put = slot >= 0;
            const int64_t blk = slot >> p.block_shift;
            const int bs = 1 << p.block_shift;
            const int off = (int)(slot & (bs - 1));
            unsigned char* cache = is_v ? p.v_cache : p.k_cache;
            if constexpr (SINK == RowSink::kCache) {
                if (put) {
                    T* dst = reinterpret_cast<T*>(cache) + ((blk * Hkv + g) * bs + off) * D;
                    if (is_v) UV::put(dst, w.u, 0, typename UV::Raw{raw.a, raw.b});
                    else U::put(dst, w.u, p.rot, raw);
                }
            } else if (__any_sync(0xffffffffu, put)) {
                // the row's largest magnitude over its D / (2 E) lanes
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 2 * E; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
                for (int o = 1; o < p.units_row; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (put) {
                    const int b = row_scale_byte(top);
                    unsigned char* tile = cache + (blk * Hkv + g) * (int64_t)(bs * (D + 1));
                    if (is_v) UV::store_codes(tile + off * D, w.u, 0, x, row_scale_inv(b));
                    else U::store_codes(tile + off * D, w.u, p.rot, x, row_scale_inv(b));
                    if (w.u == 0) tile[bs * D + off] = (unsigned char)b;
                }
            }
        }
    };

    // (whole warps stay in the loop: quantised rows shuffle over their lanes)
    const int step = blockDim.x * kDepth;
    Where at[kDepth];
    typename U::Raw raw[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
        at[k] = where(first + k * (int)blockDim.x + (int)threadIdx.x);
        raw[k] = fetch(at[k]);
    }
    if constexpr (kCached)
        if ((int)threadIdx.x < tokens) slots[threadIdx.x] = p.slot_mapping[token0 + threadIdx.x];
    for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
        const int t = i / half;
        const int k = i - t * half;
        const float2 w = turn(p.positions[token0 + t], p.inv_freq[k], p.mscale);
        float* at = angles + t * (span * E * 2) + U::angle(k, span);
        at[0] = w.x;
        at[2] = w.y;
    }
    __syncthreads();
    for (int base = first; base < last; base += step) {
        if (base != first) {
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                at[k] = where(base + k * (int)blockDim.x + (int)threadIdx.x);
                raw[k] = fetch(at[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kDepth; ++k) finish(at[k], raw[k]);
    }
}

template <typename T, RowSink SINK>
cudaError_t run_rotary(RotaryParams& p, bool interleaved, int num_sms, cudaStream_t stream) {
    constexpr int E = Elem<T>::kPerChunk;
    p.units_row = p.head_size / (2 * E);
    const int rows = p.num_heads + p.num_kv_heads * (SINK == RowSink::kRows ? 1 : 2);
    p.units_token = rows * p.units_row;
    if (p.num_tokens == 0 || p.units_token == 0) return cudaSuccess;
    // A CTA takes whole tokens, enough of them for kDepth units a thread (at most
    // kMaxTokens: their angles stay within 16 KB); with too few such CTAs for the
    // SMs a token's units are split into parts of one unit a thread.
    // About 128 threads a CTA, or 64 for many 16-bit tokens of the quantising write:
    // 16384 of 32 + 32 heads take 121 us with 64 and 126 with 128, but the plain
    // write 125 and 122, the same in 32 bits 209 and 207 (16384 of 8 + 1 heads of 64:
    // 25 and 18), and 1500 tokens, whose CTAs are on the SMs all at once, 21 and 16.
    int about = SINK == RowSink::kCacheFp8Row && sizeof(T) == 2 && p.num_tokens >= 16 * num_sms ? kThreads / 2
                                                                                               : kThreads;
    int tpc = kDepth * about / p.units_token;
    tpc = tpc < 1 ? 1 : tpc > kMaxTokens ? kMaxTokens : tpc;
    while (tpc > 1 && (p.num_tokens + tpc - 1) / tpc < 4 * num_sms) tpc >>= 1;
    const int groups = (p.num_tokens + tpc - 1) / tpc;
    p.tokens_cta = tpc;
    p.units_cta = p.units_token * tpc;
    int parts = 1, depth = kDepth;
    if (tpc == 1 && groups < 4 * num_sms) {
        const int most = (p.units_token + about - 1) / about;
        parts = (4 * num_sms + groups - 1) / groups;
        if (parts > most) parts = most;
        p.units_cta = ((p.units_token + parts - 1) / parts + 31) / 32 * 32;
        parts = (p.units_token + p.units_cta - 1) / p.units_cta;
        depth = 1;
    }
    // near that, the count that leaves the fewest without a unit in the last round
    int threads = about, idle = INT_MAX;
    for (int t = about + 32; t >= about - 32; t -= 32) {
        const int round = t * depth, over = (p.units_cta + round - 1) / round * round - p.units_cta;
        if (over < idle || (over == idle && t == about)) {
            threads = t;
            idle = over;
        }
    }
    if (p.units_cta < threads) threads = (p.units_cta + 31) / 32 * 32;
    p.row_inverse = inverse_of(p.units_row);
    p.token_inverse = inverse_of(p.units_token);
    const size_t smem = sizeof(float2) * (size_t)tpc * ((p.rot / 2 + E - 1) / E * E);
    const dim3 grid((unsigned)groups, (unsigned)parts), block((unsigned)threads);
    const int half = p.rot / 2;
    if (interleaved) return launch_pdl(rotary_kernel<T, SINK, true, E>, grid, block, smem, stream, p);
    if (half % E == 0) return launch_pdl(rotary_kernel<T, SINK, false, E>, grid, block, smem, stream, p);
    if (E == 8 && half % 4 == 0) return launch_pdl(rotary_kernel<T, SINK, false, 4>, grid, block, smem, stream, p);
    if (half % 2 == 0) return launch_pdl(rotary_kernel<T, SINK, false, 2>, grid, block, smem, stream, p);
    return launch_pdl(rotary_kernel<T, SINK, false, 1>, grid, block, smem, stream, p);
}

template <typename T>
cudaError_t by_sink(RotaryParams& p, RowSink sink, bool interleaved, int num_sms, cudaStream_t stream) {
    switch (sink) {
        case RowSink::kRows: return run_rotary<T, RowSink::kRows>(p, interleaved, num_sms, stream);
        case RowSink::kCache: return run_rotary<T, RowSink::kCache>(p, interleaved, num_sms, stream);
        default: return run_rotary<T, RowSink::kCacheFp8Row>(p, interleaved, num_sms, stream);
    }
}

// ---------------------------------------------------------------------------
// Read-back: rows of the sequences' tokens from the pages to packed [N][Hkv][D].
// A CTA takes a run of tokens; a thread finds each token's sequence (the last
// one that starts at or before it) and block once, then the threads copy or
// convert 16 bytes of K and of V at a time.  The CTA's part of the output is
// contiguous, so a unit's number is its place there.
// ---------------------------------------------------------------------------
constexpr int kGatherTokens = 32, kGatherThreads = 128;

// The codes of 16 output bytes (4 for fp32, 8 for 16 bits), rounded once from the
// exact product.
template <typename T> struct CodeWord { using type = uint2; };
template <> struct CodeWord<float> { using type = uint32_t; };
__device__ __forceinline__ void widen_codes(uint32_t c, float* f) { Elem<fp8e4m3>::widen4(c, f); }
__device__ __forceinline__ void widen_codes(const uint2& c, float* f) {
    Elem<fp8e4m3>::widen4(c.x, f);
    Elem<fp8e4m3>::widen4(c.y, f + 4);
}

template <typename T, CacheKind KIND>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
    constexpr int ES = KIND == CacheKind::kSame ? (int)sizeof(T) : 1;   // bytes of a cache element
    constexpr int EPU = Elem<T>::kPerChunk;                             // elements of a unit: 16 output bytes
    using Word = typename std::conditional<KIND == CacheKind::kSame, uint4, typename CodeWord<T>::type>::type;
    __shared__ int64_t s_base[kGatherTokens];   // row of KV head 0 in its cache; -1: zeros (a bad id); -2: no row
    __shared__ int s_scale[kGatherTokens];      // its scale byte, from there
    griddep_wait();
    griddep_launch();
    const int64_t n0 = (int64_t)blockIdx.x * p.tokens_cta;
    const int tokens = (int)min((int64_t)p.tokens_cta, p.num_tokens - n0);
    const int D = p.head_size, bs = 1 << p.block_shift;
    const int tile = KIND == CacheKind::kFp8Row ? bs * (D + 1) : bs * D * ES;
    if ((int)threadIdx.x < tokens) {
        const int64_t n = n0 + threadIdx.x;
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.start_loc[mid] <= n) lo = mid; else hi = mid - 1;
        }
        const int64_t t = n - p.start_loc[lo];
        int64_t base = -2;
        const int off = (int)(t & (bs - 1));
        if (t >= 0 && n < p.start_loc[lo + 1]) {
            const int64_t j = t >> p.block_shift;
            if (j < p.max_blocks_per_seq) {
                const int phys = p.block_tables[(int64_t)lo * p.max_blocks_per_seq + j];
                if (phys < 0 || phys >= p.num_blocks) {
                    flag_error(p.errors, PKV_DEVERR_BLOCK_ID);
                    base = -1;
                } else {
                    base = (int64_t)phys * p.num_kv_heads * tile + off * D * ES;
                }
            } else {
                flag_error(p.errors, PKV_DEVERR_CONTEXT);
            }
        }
        s_base[threadIdx.x] = base;
        s_scale[threadIdx.x] = bs * D + off - off * D;
    }
    __syncthreads();
    const int upr = D / EPU, row_shift = 31 - __clz(upr);      // units of a row, a power of two
    const int per_token = p.num_kv_heads * upr;
    T* k_out = static_cast<T*>(p.k_out) + n0 * p.num_kv_heads * D;
    T* v_out = static_cast<T*>(p.v_out) + n0 * p.num_kv_heads * D;
    constexpr int kUnits = 4;                                  // in flight a thread
    for (int w0 = threadIdx.x; w0 < tokens * per_token; w0 += kUnits * blockDim.x) {
        Word ck[kUnits] = {}, cv[kUnits] = {};
        int bk[kUnits], bv[kUnits];
        bool on[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int w = w0 + k * blockDim.x;
            bk[k] = bv[k] = 127;
            on[k] = false;
            if (w >= tokens * per_token) continue;
            const int i = tokens == 1 ? 0 : divide(w, p.token_inverse);   // (a row of many heads is past divide's range)
            const int rem = w - i * per_token;
            const int64_t base = s_base[i];
            on[k] = base != -2;
            if (base < 0) continue;
            const int64_t at = base + (rem >> row_shift) * tile, codes = at + (rem & (upr - 1)) * (int)sizeof(Word);
            ck[k] = *reinterpret_cast<const Word*>(p.k_cache + codes);
            cv[k] = *reinterpret_cast<const Word*>(p.v_cache + codes);
            if constexpr (KIND == CacheKind::kFp8Row) {
                bk[k] = p.k_cache[at + s_scale[i]];
                bv[k] = p.v_cache[at + s_scale[i]];
            }
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            if (!on[k]) continue;
            const int64_t to = (int64_t)(w0 + k * (int)blockDim.x) * EPU;
            if constexpr (KIND == CacheKind::kSame) {
                *reinterpret_cast<uint4*>(k_out + to) = ck[k];
                *reinterpret_cast<uint4*>(v_out + to) = cv[k];
            } else {
                auto put = [&](T* dst, const Word& c, int b, float scale) {
                    const float sc = KIND == CacheKind::kFp8Row ? row_scale(b) : scale;
                    float f[EPU];
                    widen_codes(c, f);
#pragma unroll
                    for (int j = 0; j < EPU; ++j) f[j] *= sc;
                    *reinterpret_cast<uint4*>(dst) = Elem<T>::narrow(f);
                };
                put(k_out + to, ck[k], bk[k], p.k_scale);
                put(v_out + to, cv[k], bv[k], p.v_scale);
            }
        }
    }
}

template <typename T, CacheKind KIND>
cudaError_t run_gather(GatherParams& p, int num_sms, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    // enough tokens for four units (K and V) a thread, fewer while the SMs are not filled
    const int per_token = p.num_kv_heads * p.head_size / Elem<T>::kPerChunk;
    int tpc = 4 * kGatherThreads / per_token;
    tpc = tpc < 1 ? 1 : tpc > kGatherTokens ? kGatherTokens : tpc;
    while (tpc > 1 && (p.num_tokens + tpc - 1) / tpc < 4 * num_sms) tpc >>= 1;
    p.token_inverse = inverse_of(per_token);
    p.tokens_cta = tpc;
    const dim3 grid((unsigned)((p.num_tokens + tpc - 1) / tpc));
    return launch_pdl(gather_kernel<T, KIND>, grid, dim3(kGatherThreads), 0, stream, p);
}

template <typename T>
cudaError_t by_kind(GatherParams& p, CacheKind kind, int num_sms, cudaStream_t stream) {
    switch (kind) {
        case CacheKind::kSame: return run_gather<T, CacheKind::kSame>(p, num_sms, stream);
        case CacheKind::kFp8: return run_gather<T, CacheKind::kFp8>(p, num_sms, stream);
        default: return run_gather<T, CacheKind::kFp8Row>(p, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, RowSink sink, bool interleaved, int dtype, int num_sms, cudaStream_t stream) {
    switch (dtype) {
        case PKV_F32: return by_sink<float>(p, sink, interleaved, num_sms, stream);
        case PKV_F16: return by_sink<__half>(p, sink, interleaved, num_sms, stream);
        default: return by_sink<__nv_bfloat16>(p, sink, interleaved, num_sms, stream);
    }
}

cudaError_t launch_gather(GatherParams p, CacheKind kind, int dtype, int num_sms, cudaStream_t stream) {
    switch (dtype) {
        case PKV_F32: return by_kind<float>(p, kind, num_sms, stream);
        case PKV_F16: return by_kind<__half>(p, kind, num_sms, stream);
        default: return by_kind<__nv_bfloat16>(p, kind, num_sms, stream);
    }
}

}  // namespace pkv
