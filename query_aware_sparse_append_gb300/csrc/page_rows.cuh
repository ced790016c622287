// page_rows.cuh -- what the kernels that write rows into pages share: the fold of a
// page's box and the E4M3 codes of values under a page's scale.
#pragma once

#include "qasa_device.cuh"

namespace qasa {

// Minima and maxima of the stored keys of a lane's chunk pair, in the pool's own
// type (exact, and half the registers of fp32 for 16-bit pools; E4M3 codes go as
// halves).  A number wins over a NaN, as in the other box code.
template <typename T> struct Box {
    static constexpr int N = 8;                  // words of a chunk pair
    uint32_t lo[N], hi[N];
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (sizeof(T) == 4) r = __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
        else if constexpr (elem<T>::id == QASA_DTYPE_BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (sizeof(T) == 4) r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        else if constexpr (elem<T>::id == QASA_DTYPE_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ void clear() {
        const uint32_t inf = sizeof(T) == 4 ? 0x7f800000u : elem<T>::id == QASA_DTYPE_BF16 ? 0x7f807f80u : 0x7c007c00u;
        const uint32_t minus = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
#pragma unroll
        for (int i = 0; i < N; ++i) { lo[i] = inf; hi[i] = inf | minus; }
    }
    __device__ __forceinline__ void fold(const uint4 &a, const uint4 &b) {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < N; ++i) { lo[i] = least(lo[i], w[i]); hi[i] = most(hi[i], w[i]); }
    }
    template <int LPR> __device__ __forceinline__ void join() {      // the warp's lane groups
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                lo[i] = least(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
                hi[i] = most(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
            }
    }
};

// Eight floats from eight codes.
__device__ __forceinline__ void codes_to_f(const uint2 &w, float *f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e4m3_to_f(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu);
}
// Two codes (low byte first), ties to even, saturating.
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(lo), "f"(hi));
    return c;
}
// Codes of y / s, the quotient rounded to fp32 as everywhere, eight at a time.
static __device__ __noinline__ uint2 quantise8_exact(float4 a, float4 b, float s) {
    const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[2] = {0u, 0u};
    if (s > 0.f)
#pragma unroll
        for (int e = 0; e < 8; e += 2) w[e >> 2] |= code2(__fdiv_rn(y[e], s), __fdiv_rn(y[e + 1], s)) << (8 * (e & 2));
    return make_uint2(w[0], w[1]);
}
// The division is needed only where a code border lies near: the product with the
// reciprocal `inv` is within 2^-22 of the quotient (half a step each for the
// reciprocal, the product and the quotient), so where products scaled by 1 - 2^-21
// and 1 + 2^-21 have the same code, the quotient has it too.  The exact way is out
// of line: the kernel's rows run into the instruction cache's size otherwise.
__device__ __forceinline__ uint2 quantise8(const float *y, float s, float inv) {
    uint32_t w[2] = {0u, 0u};
    bool same = inv < INFINITY;                // a scale of 0, or one whose reciprocal is too large
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float a = y[e] * inv, b = y[e + 1] * inv;
        const uint32_t in = code2(a * (1.f - 0x1p-21f), b * (1.f - 0x1p-21f));
        const uint32_t out = code2(a * (1.f + 0x1p-21f), b * (1.f + 0x1p-21f));
        same = same && in == out;
        w[e >> 2] |= out << (8 * (e & 2));
    }
    if (!same) {
        const uint2 x = quantise8_exact(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), s);
        w[0] = x.x;
        w[1] = x.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] &= ((w[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // zero is +0
    return make_uint2(w[0], w[1]);
}

// Codes under a page's scale of values that are codes under another one's: c a / a_new of
// code values c and the two pages' amax (the 448 of both scales cancels), eight at a time.
// Such quotients often lie on the border of two codes exactly, as a_new is itself some
// code times a scale; its two fp32 roundings, 2^-23 of it, must not decide there, so within
// 2^-22 of a border the even code is taken.  Out of line: only quotients that are near a
// border in fp32 come here.  On which side of the border B one lies is told by
// c amax - B a_new, whose second product is split into its fp32 rounding and the rest, so
// that only the difference is rounded, once (in 64 bits, which this device has few units
// for, 64 sequences' accepted paths took 13 us, not 6).
static __device__ __noinline__ uint2 recode8_near(float4 a, float4 b, float by, float amax, float amax_new) {
    const float c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const float far = amax_new < 0x1p-60f ? 0x1p80f : amax_new > 0x1p60f ? 0x1p-80f : 1.f;   // no product leaves the normal range
    const float x = amax * far, y = amax_new * far;
    if (!(amax_new > 0.f)) by = 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = c[e] == 0.f ? 0.f : c[e] * by;
        const uint32_t in = code2(q * (1.f - 0x1p-21f), 0.f) & 0xffu, out = code2(q * (1.f + 0x1p-21f), 0.f) & 0xffu;
        const float border = 0.5f * fabsf(e4m3_to_f(in) + e4m3_to_f(out));                   // of neighbours: exact
        const float near = border * y;
        const float past = __fmaf_rn(fabsf(c[e]), x, -near) - __fmaf_rn(border, y, -near);   // |c| amax - B a_new
        const uint32_t even = out & 1u ? in : out;
        w[e >> 2] |= (in == out || fabsf(past) <= 0x1p-22f * near ? even : past > 0.f ? out : in) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
}
// `by` = amax / amax_new in fp32, or infinite or NaN where that is no number.  Its product with a
// code value is within 2^-23 of the quotient: where products scaled by 1 - 2^-21 and 1 + 2^-21
// have the same code, no border is within 2^-22 of it.
__device__ __forceinline__ uint2 recode8(const uint2 &codes, float by, float amax, float amax_new) {
    float c[8];
    codes_to_f(codes, c);
    uint32_t w[2] = {0u, 0u};
    bool same = by < INFINITY;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float a = c[e] * by, b = c[e + 1] * by;
        const uint32_t in = code2(a * (1.f - 0x1p-21f), b * (1.f - 0x1p-21f));
        const uint32_t out = code2(a * (1.f + 0x1p-21f), b * (1.f + 0x1p-21f));
        same = same && in == out;
        w[e >> 2] |= out << (8 * (e & 2));
    }
    if (!same) {
        const uint2 x = recode8_near(make_float4(c[0], c[1], c[2], c[3]), make_float4(c[4], c[5], c[6], c[7]), by, amax, amax_new);
        w[0] = x.x;
        w[1] = x.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] &= ((w[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // zero is +0
    return make_uint2(w[0], w[1]);
}

// Eight codes as halves, exactly, and back (halves that are codes' values).
__device__ __forceinline__ uint4 codes_to_halves(const uint2 &w) {
    return make_uint4(e4m3x2_to_h2(w.x), e4m3x2_to_h2(w.x >> 16), e4m3x2_to_h2(w.y), e4m3x2_to_h2(w.y >> 16));
}
__device__ __forceinline__ uint2 halves_to_codes(const uint32_t *h) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h[i]));
        w[i >> 1] |= (uint32_t)c << (16 * (i & 1));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] &= ((w[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // zero is +0
    return make_uint2(w[0], w[1]);
}

}  // namespace qasa
