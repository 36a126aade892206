// The FP4 format of the caches on the device: E2M1 codes, two to a byte (channel
// 2i in the low nibble), one E4M3 scale per 16 channels.
#pragma once

#include "common.cuh"

namespace csa2 {

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two E4M3 bytes (the low one in the low half) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// Eight codes -> f16, each byte's low and high nibble in the halves of a word, times
// the scales of the halves: exact, 6 significant bits between 2^-10 and 2688.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t scale, uint32_t (&r)[4]) {
    uint32_t h0, h1, h2, h3;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
        : "r"(w));
    r[0] = mul_f16x2(h0, scale), r[1] = mul_f16x2(h1, scale), r[2] = mul_f16x2(h2, scale), r[3] = mul_f16x2(h3, scale);
}

// Eight fp32 -> eight codes, nearest even, saturating (x[0] in the lowest nibble).
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// 16-bit values of either type: a word's two as fp32, two fp32 as a word.
template <bool HALF>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if (HALF) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (HALF) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The rotation of a pair: every product and sum rounded, so that the bits do not
// depend on which kernel rotates.
__device__ __forceinline__ float2 rotate(float a, float b, float c, float s) {
    return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c)));
}

// ---- host side: where rows of 16-bit elements [T, H, D] lie
struct Rows {
    const void *p;
    int64_t T, H, D, token, head;    // strides in elements
    int64_t bytes() const { return T && H ? 2 * ((T - 1) * token + (H - 1) * head + D) : 0; }
    bool apart() const {             // no two rows share an element
        if (T <= 1) return H <= 1 || head >= D;
        if (H <= 1) return token >= D;
        return token >= head ? head >= D && token >= (H - 1) * head + D : token >= D && head >= (T - 1) * token + D;
    }
};
// Whether n bytes at p and m bytes at q meet.
static inline bool meet(const void *p, int64_t n, const void *q, int64_t m) {
    return n > 0 && m > 0 && (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n;
}
// Whether two tensors' rows may share elements.  They do not if one lies behind the other, nor if they are different
// parts of the same tokens (slices of one projection's output), of the same heads (the same with heads first) or of the
// same rows (projections side by side in each head): modulo strides that both have, their elements are in intervals
// that do not meet.
static inline bool share(const Rows &x, const Rows &y) {
    if (!meet(x.p, x.bytes(), y.p, y.bytes())) return false;
    const int64_t gap = (int64_t)(uintptr_t)y.p - (int64_t)(uintptr_t)x.p;
    if (gap % 2) return true;
    auto common = [](int64_t a, int64_t b) {
        while (b) {
            const int64_t r = a % b;
            a = b, b = r;
        }
        return a;
    };
    auto apart = [&](int64_t m, int64_t nx, int64_t ny) {            // x in [0, nx), y in [d, d + ny) modulo m
        if (m <= 0) return false;
        const int64_t d = ((gap / 2) % m + m) % m;
        return nx <= d && d + ny <= m;
    };
    auto across = [](int64_t n, int64_t stride) { return n > 1 ? stride : 0; };      // a stride of an extent of one says nothing
    const int64_t token = common(across(x.T, x.token), across(y.T, y.token)), head = common(across(x.H, x.head), across(y.H, y.head));
    return !apart(token, (x.H - 1) * x.head + x.D, (y.H - 1) * y.head + y.D) &&
           !apart(head, (x.T - 1) * x.token + x.D, (y.T - 1) * y.token + y.D) && !apart(common(token, head), x.D, y.D);
}

}  // namespace csa2
