// rows.cuh -- rows of bf16 held by the threads of a CTA (the norms): loads and stores at any alignment, sums
// over a row, and the quantised output.
#pragma once

#include "block.h"
#include "common.cuh"
#include "quant.cuh"

namespace moe {

// The 16 bytes that start `bytes` (even, below 16) into the pair (lo, hi). `bytes` is the same for
// a whole row: the branch is uniform.
__device__ __forceinline__ uint4 cut(const uint4& lo, const uint4& hi, int bytes) {
    const int sh = (bytes & 2) * 8;
    auto four = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e) {
        return make_uint4(__funnelshift_r(a, b, sh), __funnelshift_r(b, c, sh), __funnelshift_r(c, d, sh),
                          __funnelshift_r(d, e, sh));
    };
    switch (bytes >> 2) {
        case 0: return four(lo.x, lo.y, lo.z, lo.w, hi.x);
        case 1: return four(lo.y, lo.z, lo.w, hi.x, hi.y);
        case 2: return four(lo.z, lo.w, hi.x, hi.y, hi.z);
        default: return four(lo.w, hi.x, hi.y, hi.z, hi.w);
    }
}

// The chunks tid, tid + NT, ... of one row of a bf16 matrix as they lie in memory, 8 elements
// each, zeros past the row.
template <int MAXC, bool RAGGED>
struct RowLoad {
    uint4 lo[MAXC], hi[RAGGED ? MAXC : 1];
    // Issues the loads: nothing here depends on a loaded value. RAGGED: chunk c lies in two aligned
    // pieces, the first starting m bytes before it. A piece may hold bytes of the neighbouring
    // rows, which are cut off, but none before the matrix's first or past its last element.
    __device__ __forceinline__ void issue(const __nv_bfloat16* mat, int64_t ld, int64_t t, int T, int H, int nchunks,
                                          int tid, int NT) {
        const __nv_bfloat16* row = mat + t * ld;
        if constexpr (!RAGGED) {
#pragma unroll
            for (int i = 0; i < MAXC; ++i) {
                const int c = tid + i * NT;
                lo[i] = make_uint4(0, 0, 0, 0);
                if (c < nchunks) lo[i] = reinterpret_cast<const uint4*>(row)[c];
            }
        } else {
            const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15);
            const uint8_t* base = reinterpret_cast<const uint8_t*>(row) - m;
            // bytes of the matrix before the row (16 are enough) and from its start on
            const int first = -(int)min((int64_t)16, 2 * t * ld);
            const int last = 2 * H + (int)min((int64_t)16, 2 * (T - 1 - t) * ld);
#pragma unroll
            for (int i = 0; i < MAXC; ++i) {
                const int c = tid + i * NT, b = 16 * c - m;  // the first piece's first byte, in the row
                lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
                if (c < nchunks && b >= first && b + 16 <= last) lo[i] = *reinterpret_cast<const uint4*>(base + 16 * c);
                if (c < nchunks && b + 16 < 2 * H && b + 32 <= last)
                    hi[i] = *reinterpret_cast<const uint4*>(base + 16 * c + 16);
            }
            if (first > -16 || last < 2 * H + 16) {
#pragma unroll
                for (int i = 0; i < MAXC; ++i) {  // pieces that reach over an end of the matrix
                    const int c = tid + i * NT, b = 16 * c - m;
                    if (c < nchunks && (b < first || b + 16 > last)) lo[i] = edge(row, b / 2, H);
                    if (c < nchunks && b + 16 < 2 * H && b + 32 > last) hi[i] = edge(row, b / 2 + 8, H);
                }
            }
        }
    }
    // elements [e, e + 8) of which only some lie in the row
    static __device__ __noinline__ uint4 edge(const __nv_bfloat16* row, int e, int H) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = e + 2 * j;
            const uint32_t a = k >= 0 && k < H ? h[k] : 0u, b = k + 1 >= 0 && k + 1 < H ? h[k + 1] : 0u;
            w[j] = a | b << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // chunk c = tid + i NT of the row
    __device__ __forceinline__ uint4 chunk(int i, const __nv_bfloat16* row, int c, int H) const {
        if constexpr (!RAGGED) {
            return lo[i];
        } else {
            uint4 v = cut(lo[i], hi[i], (int)(reinterpret_cast<uintptr_t>(row) & 15));
            const int left = H - 8 * c;  // elements of the row from here on
            if (left < 8) {
                v.x &= left <= 0 ? 0u : left == 1 ? 0xFFFFu : ~0u;
                v.y &= left <= 2 ? 0u : left == 3 ? 0xFFFFu : ~0u;
                v.z &= left <= 4 ? 0u : left == 5 ? 0xFFFFu : ~0u;
                v.w &= left <= 6 ? 0u : 0xFFFFu;
            }
            return v;
        }
    }
};

// Writes a row of H bf16 that lies as 8-element chunks in shared memory: thread tid of NT takes
// the aligned 16-byte pieces tid, tid + NT, ... of the destination.
__device__ __forceinline__ void store_ragged(const uint4* s, __nv_bfloat16* row, int H, int tid, int NT) {
    const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    uint8_t* base = reinterpret_cast<uint8_t*>(row) - m;
    const int pieces = (m + 2 * H + 15) / 16;
    for (int g = tid; g < pieces; g += NT) {
        const int b0 = 16 * g - m;  // the piece's first byte, in the row
        if (b0 >= 0 && b0 + 16 <= 2 * H) {
            const uint4 hi = s[g];  // with m > 0 a whole piece has g >= 1 and ends in chunk g
            *reinterpret_cast<uint4*>(base + 16 * g) = m == 0 ? hi : cut(s[g - 1], hi, 16 - m);
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(s);
            uint16_t* o = reinterpret_cast<uint16_t*>(row);
            const int e0 = b0 / 2;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j >= 0 && e0 + j < H) o[e0 + j] = h[e0 + j];
        }
    }
}

// A plain load, as everywhere here: the kernel may be resident while its predecessor still writes gamma,
// and the read-only path (__ldg) is for data that no one writes during the kernel's whole life.
__device__ __forceinline__ void load_gamma(float (&g)[8], const float* gamma, int c, int H, bool aligned) {
    const float* p = gamma + 8 * c;
    if (aligned && 8 * c + 8 <= H) {
        const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
        g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w;
        g[4] = v.x, g[5] = v.y, g[6] = v.z, g[7] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 8 * c + j < H ? p[j] : 0.0f;
    }
}

constexpr int NORM_MAX_WARPS = 32;

// Joins the row's warps (32 at most), in a fixed order: one value for each row of the CTA.
template <bool MAX>
__device__ __forceinline__ float row_join(float v, float* s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_or_nan(v, u) : v + u;
    }
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    float* s = s_red + threadIdx.y * warps;
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    float t = (int)threadIdx.x % 32 < warps ? s[threadIdx.x % 32] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, t, o);
        t = MAX ? max_or_nan(t, u) : t + u;
    }
    return t;
}

// 1 / sqrt(ss / H + eps) as an unevaluated sum hi + lo, good to some 2^-40 of it: an approximation
// and its Newton correction, whose residual 1 - v hi^2 is taken exactly by FMAs.
struct Scale {
    float hi, lo;
    __device__ __forceinline__ Scale(float ss, float h, float inv_h, float eps) {
        const float q = ss * inv_h, q_lo = __fmaf_rn(-q, h, ss) * inv_h;  // ss / h = q + q_lo
        const float v = q + eps, b = v - q;
        const float v_lo = ((q - (v - b)) + (eps - b)) + q_lo;  // the exact rest of the sum (Knuth's two-sum)
        hi = rsqrtf(v);
        const float t = v * hi, e = __fmaf_rn(v, hi, -t);  // v hi = t + e
        const float r = __fmaf_rn(v_lo * hi, hi, __fmaf_rn(e, hi, __fmaf_rn(t, hi, -1.0f)));
        lo = v < __uint_as_float(0x7F800000u) && v > 0.0f ? -0.5f * hi * r : 0.0f;
    }
    // z (hi + lo) g with one rounding that matters
    __device__ __forceinline__ float apply(float z, float g) const {
        const float t = z * hi;
        const float e = __fmaf_rn(z, lo, __fmaf_rn(z, hi, -t));
        return __fmaf_rn(t, g, e * g);
    }
};

__device__ __forceinline__ void row_barrier() {
    if (blockDim.x == 32)
        __syncwarp();
    else
        __syncthreads();
}

// The row's chunks z in the quantised format: codes, block scales, row scale. s_red: one value a warp.
template <int FMT, int MAXC>
__device__ __forceinline__ void quantize_row(const NormArgs& a, const float (&z)[MAXC][8], int64_t t, bool live,
                                             int nchunks, float* s_red) {
    const int tid = threadIdx.x, NT = blockDim.x, H = a.H;
    constexpr int S = fmt_sf_atoms(FMT), G = fmt_sf_block(FMT);
    float gs = 1.0f;
    if constexpr (FMT == MOE_FMT_NVFP4) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < MAXC; ++i) m = max_or_nan(m, amax_or_nan(z[i]));
        gs = nvfp4_row_scale(row_join<true>(m, s_red));
        if (tid == 0 && live) a.row_scale[t] = gs;
    }
    if (!live) return;
    const Nvfp4Row nv(gs);
    const int nkb = H / G;
    uint8_t* sf = a.atoms ? a.sf + act_sf_offset(t, 0, S, a.nks) : a.sf + t * nkb;
    auto put_sf = [&](int kb, uint32_t b) { sf[a.atoms ? (kb / 4) * ATOM_BYTES + kb % 4 : kb] = (uint8_t)b; };
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        if (i * NT >= nchunks) break;  // uniform across the row
        const bool in = c < nchunks;
        uint32_t sb;
        if constexpr (FMT == MOE_FMT_MXFP8) {
            const uint2 q = quant_mxfp8(z[i], sb);
            if (in) *reinterpret_cast<uint2*>(a.codes + t * H + c * 8) = q;
        } else {
            const uint32_t q = FMT == MOE_FMT_MXFP4 ? quant_mxfp4(z[i], sb) : quant_nvfp4(z[i], nv, sb);
            if (in) *reinterpret_cast<uint32_t*>(a.codes + t * (H / 2) + c * 4) = q;
        }
        if (in && c % (G / 8) == 0) put_sf(c / (G / 8), sb);
    }
    // scale bytes past K inside the last K stage: zero, so that they cannot turn the zero
    // codes there into NaN
    if (a.atoms)
        for (int kb = nkb + tid; kb < a.nks * 4 * S; kb += NT) put_sf(kb, 0);
}

}  // namespace moe
