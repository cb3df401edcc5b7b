// norm.cu -- residual add, RMSNorm and quantisation of rows (moe_add_rmsnorm, moe_quantize).
//
//   z = x + r,  s = bf16(z),  y = gamma z / sqrt(mean(z^2) + eps),  out = bf16(y),  q = Q(y)
//
// One CTA per row, the row in registers between its one read and its writes: x, r in, s,
// out or codes out, nothing else. Thread t owns the V-element chunks t, t + NT, ...; V is 8
// (16-byte accesses) where H and every stride and address allow it, else 2 or 1. A 32-element
// scale block is then 4 neighbouring lanes (V = 8 is the only width that quantises; rows whose
// addresses are not 16-byte aligned are read element by element there).
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace moe {

template <int V>
__device__ __forceinline__ void load_chunk(float (&f)[V], const __nv_bfloat16* p, bool aligned) {
    if constexpr (V == 8) {
        if (aligned) {
            unpack_bf16x8(*reinterpret_cast<const uint4*>(p), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __bfloat162float(p[j]);
        }
    } else if constexpr (V == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xFFFF0000u);
    } else {
        f[0] = __bfloat162float(p[0]);
    }
}

template <int V>
__device__ __forceinline__ void store_chunk(const float (&f)[V], __nv_bfloat16* p, bool aligned) {
    if constexpr (V == 8) {
        if (aligned) {
            *reinterpret_cast<uint4*>(p) = pack_bf16x8_rn(f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = __float2bfloat16_rn(f[j]);
        }
    } else if constexpr (V == 2) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
    } else {
        p[0] = __float2bfloat16_rn(f[0]);
    }
}

template <int NT>
__device__ __forceinline__ float cta_sum(float v, float* s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += s_red[w];
    return t;
}
template <int NT>
__device__ __forceinline__ float cta_max(float v, float* s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t = fmaxf(t, s_red[w]);
    return t;
}

// FMT: -1 (bf16 output only) or the quantised format; V elements per chunk, up to MAXC chunks
// per thread, NT threads
template <int FMT, int V, int MAXC, int NT>
__global__ void __launch_bounds__(NT) norm_kernel(const NormArgs a, const bool aligned) {
    const int tid = threadIdx.x, t = blockIdx.x;
    const int nchunks = a.H / V;
    __shared__ float s_red[NT / 32], s_red2[NT / 32];
    float z[MAXC][V];
    const __nv_bfloat16* x = a.x + (int64_t)t * a.ldx;
    const __nv_bfloat16* r = a.res ? a.res + (int64_t)t * a.ldr : nullptr;
    grid_dep_wait();
    grid_dep_launch();
    if (t == 0)
        for (int i = tid; i < a.n_zero; i += NT) a.zero[i] = 0;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        if (c < nchunks) {
            load_chunk<V>(z[i], x + (int64_t)c * V, aligned);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) z[i][j] = 0.0f;
        }
    }
    if (r) {
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) {
                float f[V];
                load_chunk<V>(f, r + (int64_t)c * V, aligned);
#pragma unroll
                for (int j = 0; j < V; ++j) z[i][j] += f[j];
            }
        }
    }
    if (a.sum) {
        __nv_bfloat16* s = a.sum + (int64_t)t * a.lds;
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) store_chunk<V>(z[i], s + (int64_t)c * V, aligned);
        }
    }
    if (a.gamma) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < MAXC; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(z[i][j], z[i][j], ss);
        const float scale = 1.0f / sqrtf(cta_sum<NT>(ss, s_red) / (float)a.H + a.eps);
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) {
#pragma unroll
                for (int j = 0; j < V; ++j) z[i][j] = z[i][j] * scale * a.gamma[(int64_t)c * V + j];
            }
        }
    }
    if (a.out) {
        __nv_bfloat16* o = a.out + (int64_t)t * a.ldo;
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) store_chunk<V>(z[i], o + (int64_t)c * V, aligned);
        }
    }
    if constexpr (FMT >= 0) {
        static_assert(V == 8, "scale blocks are made of 8-element chunks");
        constexpr int S = fmt_sf_atoms(FMT), G = fmt_sf_block(FMT);
        float gs = 1.0f;
        if constexpr (FMT == MOE_FMT_NVFP4) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < MAXC; ++i) m = fmaxf(m, amax_or_inf(z[i]));
            gs = nvfp4_row_scale(cta_max<NT>(m, s_red2));
            if (tid == 0) a.row_scale[t] = gs;
        }
        const int nkb = a.H / G;
        uint8_t* sf = a.atoms ? a.sf + act_sf_offset(t, 0, S, a.nks) : a.sf + (int64_t)t * nkb;
        auto put_sf = [&](int kb, uint32_t b) { sf[a.atoms ? (int64_t)(kb / 4) * ATOM_BYTES + kb % 4 : kb] = (uint8_t)b; };
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (i * NT >= nchunks) break;  // uniform across the CTA
            const bool in = c < nchunks;
            uint32_t sb;
            if constexpr (FMT == MOE_FMT_MXFP8) {
                const uint2 q = quant_mxfp8(z[i], sb);
                if (in) *reinterpret_cast<uint2*>(a.codes + (int64_t)t * a.H + c * 8) = q;
            } else {
                const uint32_t q = FMT == MOE_FMT_MXFP4 ? quant_mxfp4(z[i], sb) : quant_nvfp4(z[i], gs, sb);
                if (in) *reinterpret_cast<uint32_t*>(a.codes + (int64_t)t * (a.H / 2) + c * 4) = q;
            }
            if (in && c % (G / 8) == 0) put_sf(c / (G / 8), sb);
        }
        // scale bytes past K inside the last K stage: zero, so that they cannot turn the zero
        // codes there into NaN
        if (a.atoms)
            for (int kb = nkb + tid; kb < a.nks * 4 * S; kb += NT) put_sf(kb, 0);
    }
}

template <int FMT, int V, int MAXC, int NT>
static cudaError_t norm_t(const NormArgs& a, bool aligned, cudaStream_t st, bool pdl) {
    LaunchAttrs at(pdl);
    cudaLaunchConfig_t cfg = at.config(dim3(a.T), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&cfg, norm_kernel<FMT, V, MAXC, NT>, a, aligned);
}

template <int FMT>
static cudaError_t norm_v8(const NormArgs& a, bool aligned, cudaStream_t st, bool pdl) {
    if (a.H <= 8 * 256 * 4) return norm_t<FMT, 8, 4, 256>(a, aligned, st, pdl);
    return norm_t<FMT, 8, 8, 256>(a, aligned, st, pdl);  // H <= 16384
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st, bool pdl) {
    // the widest access that the sizes, strides and addresses of every row allow
    uintptr_t bits = (uintptr_t)a.x | (uintptr_t)(2 * a.ldx);
    if (a.res) bits |= (uintptr_t)a.res | (uintptr_t)(2 * a.ldr);
    if (a.sum) bits |= (uintptr_t)a.sum | (uintptr_t)(2 * a.lds);
    if (a.out) bits |= (uintptr_t)a.out | (uintptr_t)(2 * a.ldo);
    const bool aligned = bits % 16 == 0;
    switch (a.fmt) {
        case MOE_FMT_MXFP8: return norm_v8<MOE_FMT_MXFP8>(a, aligned, st, pdl);
        case MOE_FMT_NVFP4: return norm_v8<MOE_FMT_NVFP4>(a, aligned, st, pdl);
        case MOE_FMT_MXFP4: return norm_v8<MOE_FMT_MXFP4>(a, aligned, st, pdl);
        default: break;
    }
    if (aligned && a.H % 8 == 0) return norm_v8<-1>(a, true, st, pdl);
    if (bits % 4 == 0 && a.H % 2 == 0) {
        if (a.H <= 2 * 256 * 8) return norm_t<-1, 2, 8, 256>(a, false, st, pdl);
        return norm_t<-1, 2, 8, 1024>(a, false, st, pdl);  // H <= 16384
    }
    if (a.H <= 256 * 16) return norm_t<-1, 1, 16, 256>(a, false, st, pdl);
    return norm_t<-1, 1, 16, 1024>(a, false, st, pdl);
}

}  // namespace moe
