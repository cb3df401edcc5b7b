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

// largest magnitude; a NaN counts as infinity, so that both mark the block
__device__ __forceinline__ float amax_or_inf(const float (&f)[8]) {
    // the bit patterns of magnitudes order like the magnitudes, with NaN above infinity
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m > 0x7F800000u ? __uint_as_float(0x7F800000u) : __uint_as_float(m);
}

// 2^n exactly for -127 <= n <= 127
__device__ __forceinline__ float exp2_exact(int n) {
    return n >= -126 ? __int_as_float((n + 127) << 23) : __int_as_float(1 << 22);
}

// x * 2^-e, the correctly rounded product, for -127 <= e <= 127
__device__ __forceinline__ uint2 e4m3_codes(const float (&f)[8], int e) {
    const float sc = exp2_exact(-e);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = cvt_e4m3x2(f[4 * i] * sc, f[4 * i + 1] * sc);
        const uint32_t hi = cvt_e4m3x2(f[4 * i + 2] * sc, f[4 * i + 3] * sc);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t e2m1_codes(const float (&f)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= cvt_e2m1x2(f[2 * j], f[2 * j + 1]) << (8 * j);
    return w;
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

template <bool FP8>
__device__ __forceinline__ int mx_block(const float (&f)[8], uint32_t& sb) {
    float amax = amax_or_inf(f);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool finite = amax < __uint_as_float(0x7F800000u);
    const int e = finite ? mx_exponent<FP8>(amax) : 0;
    sb = finite ? (uint32_t)(e + 127) : UE8M0_NAN;
    return e;
}

__device__ __forceinline__ uint2 quant_mxfp8(const float (&f)[8], uint32_t& sb) {
    const int e = mx_block<true>(f, sb);
    return e4m3_codes(f, e);
}

__device__ __forceinline__ uint32_t quant_mxfp4(const float (&f)[8], uint32_t& sb) {
    const float sc = exp2_exact(-mx_block<false>(f, sb));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j] * sc;
    return e2m1_codes(v);
}

// the row scale from the row's magnitude (infinite: the row holds a value that is not finite)
__device__ __forceinline__ float nvfp4_row_scale(float amax) {
    if (!(amax < __uint_as_float(0x7F800000u))) return __uint_as_float(0x7FC00000u);
    const float gs = __fdiv_rn(amax, 2688.0f);
    return gs > 0.0f ? gs : 1.0f;  // a row of zeros, or too small for any scale: all codes are zero
}

__device__ __forceinline__ uint32_t quant_nvfp4(const float (&f)[8], float gs, uint32_t& sb) {
    float amax = amax_or_inf(f);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const bool finite = gs == gs;
    sb = finite ? cvt_e4m3x2(__fdiv_rn(amax, __fmul_rn(gs, 6.0f)), 0.0f) & 0xFF : E4M3_NAN;
    const float eff = __fmul_rn(e4m3_to_f32(sb), gs);
    if (!(eff > 0.0f)) return 0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(f[j], eff);
    return e2m1_codes(v);
}

}  // namespace moe
