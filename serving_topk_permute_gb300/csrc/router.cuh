// router.cuh -- what the routers share: ordered keys of floats, logits of either type, the
// approximate exponential and quotient, warp sums.
#pragma once

#include "common.cuh"

namespace moe {

// SMs of the GPU this is built for. The number of CTAs is part of the sums' order and of the workspace's
// size, which a caller may ask for without a GPU: a constant, not the device's answer.
constexpr int SMS = 152;

// Unsigned keys in the order of the floats: -inf < ... < +inf < NaN. The addition makes -0 a +0
// and any NaN the canonical, positive one (0x7FFFFFFF), whose key is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // order_key(-inf): the lowest key of a logit
constexpr uint32_t KEY_NAN = 0xFFFFFFFFu;
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == KEY_NAN) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
    if constexpr (BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    else
        return reinterpret_cast<const float*>(p)[i];
}

// 2^x and a / b to 2 ulp, e^x to some (2 + |x|) ulp, as the product x log2(e) is rounded; results below
// 2^-126 are flushed to zero
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_exp(float x) { return fast_exp2(x * LOG2E); }
__device__ __forceinline__ float fast_div(float a, float b) { return __fdividef(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace moe
