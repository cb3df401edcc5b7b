// quant.cuh -- the formats' quantisation of 8-element chunks held by neighbouring lanes
// (4 lanes make a 32-element block, 2 lanes a 16-element one), as used by the norm and the
// linear product. The recipe and its rounding are the dispatch quantiser's; values that are
// not finite give a NaN scale instead of a saturated code.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8_rn(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// largest magnitude, NaN if one of the values is
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax_or_nan(const float (&f)[8]) {
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_or_nan(m, fabsf(f[i]));
    return m;
}

__device__ __forceinline__ uint32_t max2_or_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// largest magnitude of the 16 bf16 in two pieces, NaN if one of them is
__device__ __forceinline__ float unit_amax(const uint4& p, const uint4& q) {
    constexpr uint32_t M = 0x7FFF7FFFu;
    const uint32_t m = max2_or_nan(max2_or_nan(max2_or_nan(p.x & M, p.y & M), max2_or_nan(p.z & M, p.w & M)),
                                   max2_or_nan(max2_or_nan(q.x & M, q.y & M), max2_or_nan(q.z & M, q.w & M)));
    return max_or_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

// 2^n exactly for -127 <= n <= 127
__device__ __forceinline__ float exp2_exact(int n) {
    return n >= -126 ? __int_as_float((n + 127) << 23) : __int_as_float(1 << 22);
}

// E4M3 codes of f * 2^-e (the product is exact up to one correct rounding), -127 <= e <= 127
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ uint2 e4m3_codes(const float (&f)[8], int e) {
    const float sc = exp2_exact(-e);
    return make_uint2(e4m3x4(f[0] * sc, f[1] * sc, f[2] * sc, f[3] * sc),
                      e4m3x4(f[4] * sc, f[5] * sc, f[6] * sc, f[7] * sc));
}

// E2M1 codes, the first value in the lowest nibble
__device__ __forceinline__ uint32_t e2m1_codes(const float (&f)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

constexpr uint32_t UE8M0_NAN = 0xFF;
constexpr uint32_t E4M3_NAN = 0x7F;

// The smallest e with amax <= TOP * 2^e, clamped to -127, and 0 for amax = 0; TOP = 448 = 1.75 * 2^8
// (FP8) or 6 = 1.5 * 2^2. For amax = (1 + f) 2^p: e = p - 8 while 1 + f <= 1.75, else p - 7 (FP4:
// p - 2, 1.5, p - 1). A subnormal amax (biased exponent 0) lies below every clamped e.
template <bool FP8>
__device__ __forceinline__ int mx_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - (FP8 ? 8 : 2) + ((b & 0x7FFFFFu) > (FP8 ? 0x600000u : 0x400000u));
    return b == 0 ? 0 : max(e, -127);
}

// exponent and scale byte of a block of this magnitude
template <bool FP8>
__device__ __forceinline__ int mx_scale(float amax, uint32_t& sb) {
    const bool finite = amax < __uint_as_float(0x7F800000u);
    const int e = finite ? mx_exponent<FP8>(amax) : 0;
    sb = finite ? (uint32_t)(e + 127) : UE8M0_NAN;
    return e;
}
// the magnitude of the block that 4 neighbouring lanes hold
__device__ __forceinline__ float block_amax4(const float (&f)[8]) {
    float amax = amax_or_nan(f);
    amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    return max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
}

__device__ __forceinline__ uint32_t mxfp4_codes(const float (&f)[8], int e) {
    const float sc = exp2_exact(-e);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j] * sc;
    return e2m1_codes(v);
}
__device__ __forceinline__ uint2 quant_mxfp8(const float (&f)[8], uint32_t& sb) {
    return e4m3_codes(f, mx_scale<true>(block_amax4(f), sb));
}
__device__ __forceinline__ uint32_t quant_mxfp4(const float (&f)[8], uint32_t& sb) {
    return mxfp4_codes(f, mx_scale<false>(block_amax4(f), sb));
}

// the row scale from the row's magnitude (not finite: the row holds such a value)
__device__ __forceinline__ float nvfp4_row_scale(float amax) {
    if (!(amax < __uint_as_float(0x7F800000u))) return __uint_as_float(0x7FC00000u);
    const float gs = __fdiv_rn(amax, 2688.0f);
    return gs > 0.0f ? gs : 1.0f;  // a row of zeros, or too small for any scale: all codes are zero
}

// Correctly rounded quotients without a division for each element (Markstein, 1990): y is the
// correctly rounded 1 / b, q = a y, and one correction by the exact remainder rounds a / b
// correctly. One Newton step on an approximation within an ulp gives that y unless b's
// significand is all ones. No step may leave the normal range: b lies between 2^-100 and 2^100
// and |a| within 2^10 b, or a is zero; an a so small that its remainder underflows rounds to
// code 0 either way.
__device__ __forceinline__ float reciprocal(float b) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
    return __fmaf_rn(__fmaf_rn(-b, y, 1.0f), y, y);
}
__device__ __forceinline__ bool all_ones(float b) { return (__float_as_uint(b) & 0x7FFFFFu) == 0x7FFFFFu; }
__device__ __forceinline__ float div_by_reciprocal(float a, float b, float y) {
    const float q = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
}

// Two of them at once, in the packed instructions: v[0] / b and v[1] / b. The remainder is exact in any
// rounding mode; rounding it down makes a zero remainder -0, which leaves the quotient -0 of a -0
// as it is (a remainder of +0 would turn it into +0, another code).
__device__ __forceinline__ float2 div2_by_reciprocal(float v0, float v1, float b, float y) {
    float2 r;
    asm("{\n\t.reg .b64 v, b, y, q, e;\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 b, {%4, %4};\n\t"
        "mov.b64 y, {%5, %5};\n\t"
        "mul.rn.f32x2 q, v, y;\n\t"
        "fma.rm.f32x2 e, q, b, v;\n\t"
        "fma.rn.f32x2 q, e, y, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(v0), "f"(v1), "f"(-b), "f"(y));
    return r;
}

// What a row's NVFP4 blocks share.
struct Nvfp4Row {
    float gs, gs6, inv6;
    bool finite, ordinary;  // ordinary: the row's divisors are within the range above
    __device__ __forceinline__ explicit Nvfp4Row(float row_scale) : gs(row_scale) {
        finite = gs == gs;
        gs6 = __fmul_rn(gs, 6.0f);
        inv6 = reciprocal(gs6);
        ordinary = gs > 0x1p-90f && gs < 0x1p90f && !all_ones(gs6);  // times 2^-9 .. 448
    }
    // scale byte of a block of this magnitude, and the value it stands for times the row's scale
    __device__ __forceinline__ float block_scale(float amax, uint32_t& sb) const {
        const float r = ordinary ? div_by_reciprocal(amax, gs6, inv6) : __fdiv_rn(amax, gs6);
        sb = finite ? cvt_e4m3x2(r, 0.0f) & 0xFF : E4M3_NAN;
        return __fmul_rn(e4m3_to_f32(sb), gs);
    }
    // codes of N 8-element pieces of a block with this scale
    template <int N>
    __device__ __forceinline__ void codes(const float (&f)[N][8], float eff, uint32_t (&q)[N]) const {
        if (ordinary && !all_ones(eff)) {
            const float y = reciprocal(eff);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 r = div2_by_reciprocal(f[n][j], f[n][j + 1], eff, y);
                    v[j] = r.x, v[j + 1] = r.y;
                }
                q[n] = eff > 0.0f ? e2m1_codes(v) : 0u;  // a zero scale: the code zero, without a sign
            }
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = eff > 0.0f ? __fdiv_rn(f[n][j], eff) : 0.0f;
                q[n] = e2m1_codes(v);
            }
        }
    }
};
__device__ __forceinline__ uint32_t quant_nvfp4(const float (&f)[8], const Nvfp4Row& row, uint32_t& sb) {
    float amax = amax_or_nan(f);
    amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const float eff = row.block_scale(amax, sb);
    uint32_t q[1];
    row.codes<1>(reinterpret_cast<const float (&)[1][8]>(f), eff, q);
    return q[0];
}

}  // namespace moe
