// sandwich.cu -- the norm after a block, its gate, the scaled residual and the norm before the next block in
// one pass over the rows (moe_sandwich_norm), and its gradient (moe_sandwich_norm_backward).
//
//   fh = f / rms(f),  u = post fh,  z = alpha r + g u,  zh = z / rms(z),  h = pre zh
//   g: 1, one for each token, or one for each channel
//
// Gradient, with w = post (times the channel's g), gt the token's g or 1, e = pre dh:
//   dz = ds + (e - zh mean(e zh)) / rms(z),  dr = alpha dz,
//   df = (gt w dz - fh mean(gt w dz fh)) / rms(f),
//   dpre = sum_t dh zh,  C = sum_t gt fh dz:  dpost = C (channel gates: g C),  dg = post C,
//   token gates: dg = sum_h w fh dz
// The second mean needs dz, which needs the first one; but sum(w fh dz) = sum(w fh ds) +
// (sum(w fh e) - mean(e zh) sum(w fh zh)) / rms(z), so that one round of sums over a row is enough.
//
// Forward: a row lives in the registers of its threads between its one read and its writes, as in the
// norm. Gradient: a thread keeps the same columns for every row of its CTA and sums C and dpre for them in
// registers; each CTA leaves one row of sums to a second kernel, which adds them in a fixed order.
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "rows.cuh"

namespace moe {

// FMT, MAXC, MAXT, MIN_CTAS, RAGGED: as in the norm. a.n: x is f, gamma the second norm's.
template <int FMT, int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
__global__ void __launch_bounds__(MAXT, MIN_CTAS) sandwich_kernel(const SandwichArgs a, const bool vectors_aligned) {
    const NormArgs& n = a.n;
    const int tid = threadIdx.x, NT = blockDim.x, H = n.H;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < n.T;  // uniform in a warp; other rows only take part in the barriers
    const int nchunks = live ? (H + 7) / 8 : 0;
    __shared__ float s_red[NORM_MAX_WARPS], s_red2[NORM_MAX_WARPS], s_red3[NORM_MAX_WARPS];
    const __nv_bfloat16* x = n.x + t * n.ldx;
    const __nv_bfloat16* r = n.res + t * n.ldr;
    grid_dep_wait();
    grid_dep_launch();
    RowLoad<MAXC, RAGGED> xv, rv;
    xv.issue(n.x, n.ldx, t, n.T, H, nchunks, tid, NT);
    rv.issue(n.res, n.ldr, t, n.T, H, nchunks, tid, NT);
    const float gate = live && a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
    float z[MAXC][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        unpack_bf16x8(xv.chunk(i, x, tid + i * NT, H), z[i]);
        float sq = 0.0f;  // by chunks: the rounding errors of many short sums average out
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(z[i][j], z[i][j], sq);
        ss += sq;
    }
    const Scale first(row_join<false>(ss, s_red), (float)H, n.inv_h, n.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        float w[8], f[8];
        if (c < nchunks) {
            load_gamma(w, a.post, c, H, vectors_aligned);
            if (a.gate_kind == MOE_GATE_CHANNEL) {
                load_gamma(f, a.gate, c, H, vectors_aligned);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= f[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.0f;
        }
        unpack_bf16x8(rv.chunk(i, r, c, H), f);
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[i][j] = fmaf(z[i][j] * first.hi, w[j] * gate, a.alpha * f[j]);
            sq = fmaf(z[i][j], z[i][j], sq);
        }
        ss += sq;
    }
    extern __shared__ uint4 s_rows[];  // RAGGED: [rows][chunks]
    uint4* s_row = s_rows + threadIdx.y * ((H + 7) / 8);
    auto store = [&](__nv_bfloat16* dst) {
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) (RAGGED ? s_row : reinterpret_cast<uint4*>(dst))[c] = pack_bf16x8_rn(z[i]);
        }
        if constexpr (RAGGED) {
            row_barrier();
            if (live) store_ragged(s_row, dst, H, tid, NT);
        }
    };
    if (n.sum) store(n.sum + t * n.lds);
    // quantised rows get h to about its last bit, as in the norm
    const Scale second(row_join<false>(ss, s_red2), (float)H, n.inv_h, n.eps);
    if (a.stats && live && tid == 0) {
        a.stats[2 * t] = first.hi;
        a.stats[2 * t + 1] = second.hi;
    }
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        if (c < nchunks) {
            float g[8];
            load_gamma(g, n.gamma, c, H, vectors_aligned);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = FMT < 0 ? z[i][j] * second.hi * g[j] : second.apply(z[i][j], g[j]);
        }
    }
    if (n.out) {
        if (RAGGED && n.sum) row_barrier();  // the sum has left shared memory
        store(n.out + t * n.ldo);
    }
    if constexpr (FMT >= 0) quantize_row<FMT, MAXC>(n, z, t, live, nchunks, s_red3);
}

constexpr int SANDWICH_CTA = 128;  // rows of fewer threads share a CTA of about this many

template <int FMT, int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
static cudaError_t sandwich_t(const SandwichArgs& a, cudaStream_t st) {
    const int64_t chunks = ceil_div(a.n.H, 8), threads = align_up(ceil_div(chunks, MAXC), 32);
    const int64_t rows = threads >= SANDWICH_CTA ? 1 : SANDWICH_CTA / threads;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg =
        at.config(dim3((unsigned)ceil_div(a.n.T, rows)), dim3((unsigned)threads, (unsigned)rows),
                  RAGGED && (a.n.sum || a.n.out) ? (size_t)(rows * chunks * 16) : 0, st);
    const uintptr_t v = (uintptr_t)a.post | (uintptr_t)a.n.gamma |
                        (a.gate_kind == MOE_GATE_CHANNEL ? (uintptr_t)a.gate : 0);
    return cudaLaunchKernelEx(&cfg, sandwich_kernel<FMT, MAXC, MAXT, MIN_CTAS, RAGGED>, a, v % 16 == 0);
}

template <int FMT, bool RAGGED>
static cudaError_t sandwich_f(const SandwichArgs& a, cudaStream_t st) {
    if (a.n.T <= 152 && a.n.H <= 8192) return sandwich_t<FMT, 1, 1024, 1, RAGGED>(a, st);
    if (a.n.H <= 4096) return sandwich_t<FMT, 2, 256, RAGGED ? 4 : 5, RAGGED>(a, st);
    if constexpr (RAGGED) {
        return sandwich_t<FMT, 2, 1024, 1, true>(a, st);
    } else {
        if (a.n.H <= 7168) return sandwich_t<FMT, 4, 224, 5, false>(a, st);
        return sandwich_t<FMT, 4, 512, 2, false>(a, st);
    }
}

cudaError_t launch_sandwich(const SandwichArgs& args, cudaStream_t st) {
    SandwichArgs a = args;
    NormArgs& n = a.n;
    n.inv_h = 1.0f / (float)n.H;
    // whether the sizes, strides and addresses give every row whole, aligned 16-byte pieces
    uintptr_t bits = (uintptr_t)n.x | (uintptr_t)(2 * n.ldx) | (uintptr_t)(2 * n.H) | (uintptr_t)n.res |
                     (uintptr_t)(2 * n.ldr);
    if (n.sum) bits |= (uintptr_t)n.sum | (uintptr_t)(2 * n.lds);
    if (n.out) bits |= (uintptr_t)n.out | (uintptr_t)(2 * n.ldo);
    const bool ragged = bits % 16 != 0;
    switch (n.fmt) {
        case MOE_FMT_MXFP8:
            return ragged ? sandwich_f<MOE_FMT_MXFP8, true>(a, st) : sandwich_f<MOE_FMT_MXFP8, false>(a, st);
        case MOE_FMT_NVFP4:
            return ragged ? sandwich_f<MOE_FMT_NVFP4, true>(a, st) : sandwich_f<MOE_FMT_NVFP4, false>(a, st);
        case MOE_FMT_MXFP4:
            return ragged ? sandwich_f<MOE_FMT_MXFP4, true>(a, st) : sandwich_f<MOE_FMT_MXFP4, false>(a, st);
        default: return ragged ? sandwich_f<-1, true>(a, st) : sandwich_f<-1, false>(a, st);
    }
}

// ------------------------------------------------------------------ gradient
// SMs of the GPU this is built for: how many CTAs share the column sums is part of their order and of the
// workspace's size, which a caller may ask for without a GPU.
constexpr int SANDWICH_SMS = 152;

// The sums of four values over a row's threads, in every thread. s: four values for each warp of the CTA.
__device__ __forceinline__ float4 four_sums(float4 v, float4* s) {
    const int lane = threadIdx.x % 32;
    auto warp4 = [&](float4 u) {  // lanes 0, 8, 16, 24 end with the sums of x, z, y, w
        const bool up = lane & 16, odd = lane & 8;
        float a = (up ? u.y : u.x) + __shfl_xor_sync(0xffffffffu, up ? u.x : u.y, 16);
        float b = (up ? u.w : u.z) + __shfl_xor_sync(0xffffffffu, up ? u.z : u.w, 16);
        a = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        return a;
    };
    float a = warp4(v);
    const int warps = blockDim.x / 32;
    if (warps > 1) {
        float* mine = reinterpret_cast<float*>(s + threadIdx.y * warps + threadIdx.x / 32);
        if (lane % 8 == 0) mine[(lane & 16 ? 1 : 0) + (lane & 8 ? 2 : 0)] = a;
        __syncthreads();
        a = warp4(lane < warps ? s[threadIdx.y * warps + lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    }
    return make_float4(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, a, 16),
                       __shfl_sync(0xffffffffu, a, 8), __shfl_sync(0xffffffffu, a, 24));
}

template <int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
__global__ void __launch_bounds__(MAXT, MIN_CTAS)
    sandwich_grad_kernel(const SandwichGradArgs a, const bool vectors_aligned) {
    const int tid = threadIdx.x, NT = blockDim.x, H = a.H, chunks = (H + 7) / 8;
    __shared__ float4 s_sums[2][NORM_MAX_WARPS];
    extern __shared__ uint4 s_rows[];  // RAGGED: [rows][chunks]
    uint4* s_row = s_rows + threadIdx.y * chunks;
    grid_dep_wait();
    grid_dep_launch();
    const bool columns = a.part != nullptr;
    float w[MAXC][8], pre[MAXC][8], c_sum[MAXC][8], p_sum[MAXC][8];
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = pre[i][j] = c_sum[i][j] = p_sum[i][j] = 0.0f;
        if (c < chunks) {
            load_gamma(w[i], a.post, c, H, vectors_aligned);
            load_gamma(pre[i], a.pre, c, H, vectors_aligned);
            if (a.gate_kind == MOE_GATE_CHANNEL) {
                float g[8];
                load_gamma(g, a.gate, c, H, vectors_aligned);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[i][j] *= g[j];
            }
        }
    }
    int round = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < a.T; t0 += (int64_t)gridDim.x * blockDim.y, round ^= 1) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        const int nchunks = live ? chunks : 0;
        RowLoad<MAXC, RAGGED> fv, rv, sv, ov;
        fv.issue(a.f, a.ldf, t, a.T, H, nchunks, tid, NT);
        rv.issue(a.res, a.ldr, t, a.T, H, nchunks, tid, NT);
        if (a.d_sum) sv.issue(a.d_sum, a.lds, t, a.T, H, nchunks, tid, NT);
        if (a.d_out) ov.issue(a.d_out, a.ldo, t, a.T, H, nchunks, tid, NT);
        const float rf = live ? a.stats[2 * t] : 0.0f, rz = live ? a.stats[2 * t + 1] : 0.0f;
        const float gt = live && a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
        float fh[MAXC][8], zh[MAXC][8], e[MAXC][8], ds[MAXC][8];
        float4 sums = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // e zh, w fh ds, w fh e, w fh zh
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            unpack_bf16x8(fv.chunk(i, a.f + t * a.ldf, c, H), fh[i]);
            unpack_bf16x8(rv.chunk(i, a.res + t * a.ldr, c, H), zh[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ds[i][j] = e[i][j] = 0.0f;
            if (a.d_sum) unpack_bf16x8(sv.chunk(i, a.d_sum + t * a.lds, c, H), ds[i]);
            if (a.d_out) unpack_bf16x8(ov.chunk(i, a.d_out + t * a.ldo, c, H), e[i]);
            float4 part = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // by chunks, as in the norm
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                fh[i][j] *= rf;
                const float u = w[i][j] * fh[i][j];
                zh[i][j] = fmaf(gt, u, a.alpha * zh[i][j]) * rz;
                if (columns) p_sum[i][j] = fmaf(e[i][j], zh[i][j], p_sum[i][j]);
                e[i][j] *= pre[i][j];
                part.x = fmaf(e[i][j], zh[i][j], part.x);
                part.y = fmaf(u, ds[i][j], part.y);
                part.z = fmaf(u, e[i][j], part.z);
                part.w = fmaf(u, zh[i][j], part.w);
            }
            sums.x += part.x, sums.y += part.y, sums.z += part.z, sums.w += part.w;
        }
        const float4 s = four_sums(sums, s_sums[round]);  // two places: the last row's may still be read
        const float m1 = s.x * a.inv_h, total = fmaf(rz, fmaf(-m1, s.w, s.z), s.y), m2 = gt * total * a.inv_h;
        if (a.gate_kind == MOE_GATE_TOKEN && a.d_gate && live && tid == 0) a.d_gate[t] = total;
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dz = fmaf(rz, fmaf(-m1, zh[i][j], e[i][j]), ds[i][j]);
                if (columns) c_sum[i][j] = fmaf(gt * fh[i][j], dz, c_sum[i][j]);
                fh[i][j] = rf * fmaf(-m2, fh[i][j], gt * w[i][j] * dz);  // df
                ds[i][j] = a.alpha * dz;                                 // dr
            }
        }
        auto store = [&](const float (&v)[MAXC][8], __nv_bfloat16* dst) {
#pragma unroll
            for (int i = 0; i < MAXC; ++i) {
                const int c = tid + i * NT;
                if (c < nchunks) (RAGGED ? s_row : reinterpret_cast<uint4*>(dst))[c] = pack_bf16x8_rn(v[i]);
            }
            if constexpr (RAGGED) {
                row_barrier();
                if (live) store_ragged(s_row, dst, H, tid, NT);
                row_barrier();  // shared memory is written again
            }
        };
        store(fh, a.d_f + t * a.ldd);
        store(ds, a.d_res + t * a.ldg);
    }
    if (columns) {
        const int64_t rows = (int64_t)gridDim.x * blockDim.y, at = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
        const int64_t ld = 8 * (int64_t)chunks;
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < chunks) {
                float4* p = reinterpret_cast<float4*>(a.part + at * ld) + 2 * c;
                float4* q = reinterpret_cast<float4*>(a.part + (rows + at) * ld) + 2 * c;
                p[0] = make_float4(p_sum[i][0], p_sum[i][1], p_sum[i][2], p_sum[i][3]);
                p[1] = make_float4(p_sum[i][4], p_sum[i][5], p_sum[i][6], p_sum[i][7]);
                q[0] = make_float4(c_sum[i][0], c_sum[i][1], c_sum[i][2], c_sum[i][3]);
                q[1] = make_float4(c_sum[i][4], c_sum[i][5], c_sum[i][6], c_sum[i][7]);
            }
        }
    }
}

constexpr int COLUMN_THREADS = 1024;
// The column sums: CTA c the columns 32 c .. 32 c + 31, one in each lane; warp w adds the parts w, w + 32, ...,
// then the warps in order.
__global__ void __launch_bounds__(COLUMN_THREADS) sandwich_columns_kernel(const SandwichGradArgs a, int parts) {
    constexpr int WARPS = COLUMN_THREADS / 32;
    __shared__ float s_p[WARPS][32], s_c[WARPS][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, h = 32 * (int)blockIdx.x + lane;
    const int64_t ld = (int64_t)((a.H + 7) / 8) * 8;
    grid_dep_wait();
    grid_dep_launch();
    float p = 0.0f, c = 0.0f;
    if (h < a.H) {
#pragma unroll 5
        for (int i = warp; i < parts; i += WARPS) {
            p += __ldcg(a.part + i * ld + h);
            c += __ldcg(a.part + (parts + i) * ld + h);
        }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    if (warp != 0 || h >= a.H) return;
    p = c = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) p += s_p[w][lane], c += s_c[w][lane];
    const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
    if (a.d_pre) a.d_pre[h] = p;
    if (a.d_post) a.d_post[h] = channel ? c * a.gate[h] : c;
    if (channel && a.d_gate) a.d_gate[h] = c * a.post[h];
}

namespace {
struct GradShape {
    int maxc, threads, rows, grid;  // chunks a thread, threads a row, rows of a CTA, CTAs
};
GradShape grad_shape(int T, int H) {
    const int64_t chunks = ceil_div(H, 8);
    GradShape s;
    s.maxc = chunks <= 1024 ? 1 : 2;
    s.threads = (int)align_up(ceil_div(chunks, s.maxc), 32);
    s.rows = s.threads >= SANDWICH_CTA ? 1 : SANDWICH_CTA / s.threads;
    const int resident = s.threads <= 256 ? 3 : s.threads <= 512 ? 2 : 1;
    const int64_t want = ceil_div(T, s.rows), most = (int64_t)SANDWICH_SMS * resident;
    s.grid = (int)(want < most ? want : most);
    return s;
}

template <int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
cudaError_t grad_t(const SandwichGradArgs& a, const GradShape& s, cudaStream_t st) {
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)s.grid), dim3((unsigned)s.threads, (unsigned)s.rows),
                                       RAGGED ? (size_t)s.rows * ceil_div(a.H, 8) * 16 : 0, st);
    const uintptr_t v = (uintptr_t)a.post | (uintptr_t)a.pre | (a.gate_kind == MOE_GATE_CHANNEL ? (uintptr_t)a.gate : 0);
    return cudaLaunchKernelEx(&cfg, sandwich_grad_kernel<MAXC, MAXT, MIN_CTAS, RAGGED>, a, v % 16 == 0);
}
template <bool RAGGED>
cudaError_t grad_r(const SandwichGradArgs& a, const GradShape& s, cudaStream_t st) {
    if (s.maxc == 2) return grad_t<2, 1024, 1, RAGGED>(a, s, st);
    if (s.threads * s.rows <= 256) return grad_t<1, 256, 3, RAGGED>(a, s, st);
    if (s.threads <= 512) return grad_t<1, 512, 2, RAGGED>(a, s, st);
    return grad_t<1, 1024, 1, RAGGED>(a, s, st);
}
}  // namespace

int64_t sandwich_grad_floats(int T, int H) {
    const GradShape s = grad_shape(T, H);
    return 2 * (int64_t)s.grid * s.rows * align_up(H, 8);
}

cudaError_t launch_sandwich_grad(const SandwichGradArgs& args, cudaStream_t st) {
    SandwichGradArgs a = args;
    a.inv_h = 1.0f / (float)a.H;
    if (!a.d_pre && !a.d_post && !(a.gate_kind == MOE_GATE_CHANNEL && a.d_gate)) a.part = nullptr;
    const GradShape s = grad_shape(a.T, a.H);
    uintptr_t bits = (uintptr_t)(2 * a.H);
    auto rows = [&](const void* p, int64_t ld) { bits |= p ? (uintptr_t)p | (uintptr_t)(2 * ld) : 0; };
    rows(a.f, a.ldf);
    rows(a.res, a.ldr);
    rows(a.d_sum, a.lds);
    rows(a.d_out, a.ldo);
    rows(a.d_f, a.ldd);
    rows(a.d_res, a.ldg);
    const cudaError_t e = bits % 16 ? grad_r<true>(a, s, st) : grad_r<false>(a, s, st);
    if (e != cudaSuccess || !a.part) return e;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)ceil_div(a.H, 32)), dim3(COLUMN_THREADS), 0, st);
    return cudaLaunchKernelEx(&cfg, sandwich_columns_kernel, a, s.grid * s.rows);
}

}  // namespace moe
