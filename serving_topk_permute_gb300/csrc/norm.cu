// norm.cu -- residual add, RMSNorm and quantisation of rows (moe_add_rmsnorm, moe_quantize).
//
//   z = x + r,  s = bf16(z),  y = gamma z / sqrt(mean(z^2) + eps),  out = bf16(y),  q = Q(y)
//
// A row lives in the registers of 1 to 32 warps between its one read and its writes: x and r in,
// s and out or codes out, nothing else. Thread t owns the 8-element chunks t, t + NT, ..., so a
// 32-element scale block is 4 neighbouring lanes. All loads of a row are issued before the first
// value is used; CTAs of other rows cover the reduction's latency. Short rows share a CTA.
//
// Rows whose starts are not 16-byte aligned (odd widths, sliced tensors) go through the RAGGED
// variant: a chunk is cut out of the two aligned 16-byte pieces that hold it (the second one is
// the neighbour's, so it comes from L1), and results go through shared memory, from where
// aligned 16-byte pieces are cut and stored; only a row's two ends use 2-byte accesses. Nothing
// outside a row is written, nothing outside the matrix read.
//
// Memory bounds all of them once there are rows enough. Measured on GB300: 8192 x 7168 with a residual
// to the sum and MXFP8 64.0 us (6.45 TB/s, 95% of the copy rate), MXFP4 59.4 and NVFP4 68.5 (their bytes
// 56.6 and 57.2); 16 x 7168 2.7 us, the launch and one trip to memory; 2999 x 2050 rows of 4-byte alignment
// 7.3 us (3.4 TB/s: a CTA loads a row, waits for it, reduces and stores, and the CTAs that fit make two to
// three waves). Quantisation alone of 8192 x 7168: MXFP8 26.8, MXFP4 23.1, NVFP4 27.8 us (6.6, 6.5 and 5.4
// TB/s).
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "rows.cuh"

namespace moe {

// FMT: -1 (bf16 output only) or the quantised format; at most MAXC chunks for each thread, at
// most MAXT threads. blockDim: threads of a row, rows of a CTA.
template <int FMT, int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
__global__ void __launch_bounds__(MAXT, MIN_CTAS) norm_kernel(const NormArgs a, const bool gamma_aligned) {
    const int tid = threadIdx.x, NT = blockDim.x, H = a.H;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.T;  // uniform in a warp; other rows only take part in the barriers
    const int nchunks = live ? (H + 7) / 8 : 0;
    __shared__ float s_red[NORM_MAX_WARPS], s_red2[NORM_MAX_WARPS];
    const __nv_bfloat16* x = a.x + t * a.ldx;
    const __nv_bfloat16* r = a.res + t * a.ldr;
    grid_dep_wait();
    grid_dep_launch();
    // every load of the row is under way before the first value is used
    RowLoad<MAXC, RAGGED> xv, rv;
    xv.issue(a.x, a.ldx, t, a.T, H, nchunks, tid, NT);
    if (a.res) rv.issue(a.res, a.ldr, t, a.T, H, nchunks, tid, NT);
    float z[MAXC][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        unpack_bf16x8(xv.chunk(i, x, tid + i * NT, H), z[i]);
        if (a.res) {
            float f[8];
            unpack_bf16x8(rv.chunk(i, r, tid + i * NT, H), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] += f[j];
        }
        float sq = 0.0f;  // by chunks: the rounding errors of many short sums average out
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(z[i][j], z[i][j], sq);
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
    if (a.sum) store(a.sum + t * a.lds);
    if (a.gamma) {
        // Quantised rows get y to about its last bit: where a block's magnitude lies at the edge between
        // two exponents, an error of a few bits would change all of its codes.
        const float total = row_join<false>(ss, s_red);
        const float scale = FMT < 0 ? 1.0f / sqrtf(total / (float)H + a.eps) : 0.0f;
        const Scale fine(total, (float)H, a.inv_h, a.eps);
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < nchunks) {
                float g[8];
                load_gamma(g, a.gamma, c, H, gamma_aligned);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[i][j] = FMT < 0 ? z[i][j] * scale * g[j] : fine.apply(z[i][j], g[j]);
            }
        }
    }
    if (a.out) {
        if (RAGGED && a.sum) row_barrier();  // the sum has left shared memory
        store(a.out + t * a.ldo);
    }
    if constexpr (FMT >= 0) quantize_row<FMT, MAXC>(a, z, t, live, nchunks, s_red2);
}

// Quantisation alone, of aligned rows: thread t owns the 16-element units t, t + NT, ... (an NVFP4
// block; two lanes make an MX block), and the magnitudes are taken on the packed bf16 pairs. This
// takes fewer instructions than the norm's path, which would otherwise bound it: 8192 x 7168 to NVFP4,
// MXFP4 and MXFP8 38.9, 29.6 and 31.2 us through the norm's path, 27.8, 23.1 and 26.8 so.
template <int FMT, int MAXU, int MAXT, int MIN_CTAS>
__global__ void __launch_bounds__(MAXT, MIN_CTAS) quant_kernel(const NormArgs a) {
    constexpr int S = fmt_sf_atoms(FMT), G = fmt_sf_block(FMT);
    const int tid = threadIdx.x, NT = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.T;  // uniform in a warp; other rows only take part in the barriers
    const int units = live ? a.H / 16 : 0;
    __shared__ float s_red[NORM_MAX_WARPS];
    const uint4* x = reinterpret_cast<const uint4*>(a.x + t * a.ldx);
    grid_dep_wait();
    grid_dep_launch();
    uint4 v[MAXU][2];
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int u = tid + i * NT;
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (u < units) {
            v[i][0] = x[2 * u];
            v[i][1] = x[2 * u + 1];
        }
    }
    float amax[MAXU], row = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        amax[i] = unit_amax(v[i][0], v[i][1]);
        row = max_or_nan(row, amax[i]);
    }
    float gs = 1.0f;
    if constexpr (FMT == MOE_FMT_NVFP4) {
        gs = nvfp4_row_scale(row_join<true>(row, s_red));
        if (tid == 0 && live) a.row_scale[t] = gs;
    }
    if (!live) return;
    const Nvfp4Row nv(gs);
    const int nkb = a.H / G;
    uint8_t* sf = a.atoms ? a.sf + act_sf_offset(t, 0, S, a.nks) : a.sf + t * nkb;
    auto put_sf = [&](int kb, uint32_t b) { sf[a.atoms ? (kb / 4) * ATOM_BYTES + kb % 4 : kb] = (uint8_t)b; };
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int u = tid + i * NT;
        if (i * NT >= units) break;  // uniform across the row
        const bool in = u < units;
        float f[2][8];
        unpack_bf16x8(v[i][0], f[0]);
        unpack_bf16x8(v[i][1], f[1]);
        uint32_t sb;
        if constexpr (FMT == MOE_FMT_NVFP4) {
            const float eff = nv.block_scale(amax[i], sb);
            uint32_t q[2];
            nv.codes<2>(f, eff, q);
            if (in) {
                *reinterpret_cast<uint2*>(a.codes + t * (a.H / 2) + u * 8) = make_uint2(q[0], q[1]);
                put_sf(u, sb);
            }
        } else {
            const float m = max_or_nan(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
            const int e = mx_scale<FMT == MOE_FMT_MXFP8>(m, sb);
            if constexpr (FMT == MOE_FMT_MXFP8) {
                const uint2 lo = e4m3_codes(f[0], e), hi = e4m3_codes(f[1], e);
                if (in) *reinterpret_cast<uint4*>(a.codes + t * a.H + u * 16) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                const uint2 q = make_uint2(mxfp4_codes(f[0], e), mxfp4_codes(f[1], e));
                if (in) *reinterpret_cast<uint2*>(a.codes + t * (a.H / 2) + u * 8) = q;
            }
            if (in && u % 2 == 0) put_sf(u / 2, sb);
        }
    }
    if (a.atoms)
        for (int kb = nkb + tid; kb < a.nks * 4 * S; kb += NT) put_sf(kb, 0);
}

constexpr int NORM_CTA = 128;  // rows of fewer threads share a CTA of about this many

template <int FMT, int MAXC, int MAXT, int MIN_CTAS, bool RAGGED>
static cudaError_t norm_t(const NormArgs& a, cudaStream_t st) {
    const int64_t chunks = ceil_div(a.H, 8), threads = align_up(ceil_div(chunks, MAXC), 32);
    const int64_t rows = threads >= NORM_CTA ? 1 : NORM_CTA / threads;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)ceil_div(a.T, rows)), dim3((unsigned)threads, (unsigned)rows),
                                       RAGGED && (a.sum || a.out) ? (size_t)(rows * chunks * 16) : 0, st);
    return cudaLaunchKernelEx(&cfg, norm_kernel<FMT, MAXC, MAXT, MIN_CTAS, RAGGED>, a, (uintptr_t)a.gamma % 16 == 0);
}

// Chunks per thread, measured on GB300 (MXFP8, residual): few rows, up to one for each of the 152 SMs,
// finish soonest with one (16 x 7168: 2.5 against 3.3 us without this rule, 152 x 7168 2.7 and 3.5, but
// 304 x 7168 4.8 and 4.1, 608 x 7168 10.0 and 6.5); otherwise two up to 4096 elements (4096 x 4096 bf16:
// 22.3 against 23.6 us with four) and four above (8192 x 7168: 69.5 against 79.6 us with two),
// where more would leave too few rows in flight.
template <int FMT, bool RAGGED>
static cudaError_t norm_f(const NormArgs& a, cudaStream_t st) {
    if (a.T <= 152 && a.H <= 8192) return norm_t<FMT, 1, 1024, 1, RAGGED>(a, st);
    if (a.H <= 4096) return norm_t<FMT, 2, 256, RAGGED ? 4 : 5, RAGGED>(a, st);
    if constexpr (RAGGED) {
        return norm_t<FMT, 2, 1024, 1, true>(a, st);
    } else {
        if (a.H <= 7168) return norm_t<FMT, 4, 224, 5, false>(a, st);
        return norm_t<FMT, 4, 512, 2, false>(a, st);
    }
}

// bf16 output of even rows whose starts are only 4-byte aligned: coalesced 4-byte accesses, thread t
// owns the pairs t, t + NT, ...
template <int MAXC, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_pairs_kernel(const NormArgs a, const bool gamma_aligned) {
    const int tid = threadIdx.x, NT = blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int pairs = t < a.T ? a.H / 2 : 0;
    __shared__ float s_red[NORM_MAX_WARPS];
    const uint32_t* x = reinterpret_cast<const uint32_t*>(a.x + t * a.ldx);
    const uint32_t* r = reinterpret_cast<const uint32_t*>(a.res + t * a.ldr);
    grid_dep_wait();
    grid_dep_launch();
    uint32_t xv[MAXC], rv[MAXC];
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        xv[i] = rv[i] = 0;
        if (c < pairs) {
            xv[i] = x[c];
            if (a.res) rv[i] = r[c];
        }
    }
    float z[MAXC][2];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        z[i][0] = __uint_as_float(xv[i] << 16) + __uint_as_float(rv[i] << 16);
        z[i][1] = __uint_as_float(xv[i] & 0xFFFF0000u) + __uint_as_float(rv[i] & 0xFFFF0000u);
        ss = fmaf(z[i][0], z[i][0], fmaf(z[i][1], z[i][1], ss));
    }
    if (a.sum) {
        __nv_bfloat162* s = reinterpret_cast<__nv_bfloat162*>(a.sum + t * a.lds);
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
            const int c = tid + i * NT;
            if (c < pairs) s[c] = __floats2bfloat162_rn(z[i][0], z[i][1]);
        }
    }
    const float scale = 1.0f / sqrtf(row_join<false>(ss, s_red) / (float)a.H + a.eps);
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(a.out + t * a.ldo);
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
        const int c = tid + i * NT;
        if (c < pairs) {
            float g0, g1;
            if (gamma_aligned) {
                const float2 g = reinterpret_cast<const float2*>(a.gamma)[c];
                g0 = g.x, g1 = g.y;
            } else {
                g0 = a.gamma[2 * c], g1 = a.gamma[2 * c + 1];
            }
            o[c] = __floats2bfloat162_rn(z[i][0] * scale * g0, z[i][1] * scale * g1);
        }
    }
}

template <int MAXC, int MAXT>
static cudaError_t norm_pairs(const NormArgs& a, cudaStream_t st) {
    const int64_t threads = align_up(ceil_div(a.H / 2, MAXC), 32), rows = threads >= NORM_CTA ? 1 : NORM_CTA / threads;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg =
        at.config(dim3((unsigned)ceil_div(a.T, rows)), dim3((unsigned)threads, (unsigned)rows), 0, st);
    return cudaLaunchKernelEx(&cfg, norm_pairs_kernel<MAXC, MAXT>, a, (uintptr_t)a.gamma % 16 == 0);
}

template <int FMT, int MAXU, int MAXT, int MIN_CTAS>
static cudaError_t quant_t(const NormArgs& a, cudaStream_t st) {
    const int64_t threads = align_up(ceil_div(a.H / 16, MAXU), 32), rows = threads >= NORM_CTA ? 1 : NORM_CTA / threads;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg =
        at.config(dim3((unsigned)ceil_div(a.T, rows)), dim3((unsigned)threads, (unsigned)rows), 0, st);
    return cudaLaunchKernelEx(&cfg, quant_kernel<FMT, MAXU, MAXT, MIN_CTAS>, a);
}
// Units per thread: one for few rows, as in the norm (152 x 7168 NVFP4 2.0 us against 2.2, 304 x 7168 2.7
// and 2.5). MX formats: two up to 6144 elements (8192 x 2048
// MXFP8 9.1 us, 9.9 with four), four above (8192 x 7168 27.2 and 27.3, MXFP4 24.0 and 24.6). NVFP4, whose
// rows wait for their magnitude: four, so that there are fewer warps to join (8192 x 7168 28.5 us, 32.3
// with two), but two where four would not fill a warp (16384 x 1024 9.8, 11.2 with four); seven CTAs
// on an SM, as eight of 64 registers spill (29.6).
template <int FMT>
static cudaError_t quant_f(const NormArgs& a, cudaStream_t st) {
    constexpr bool NV = FMT == MOE_FMT_NVFP4;
    if (a.T <= 152 && a.H <= 8192) return quant_t<FMT, 1, 512, 1>(a, st);
    if (a.H <= (NV ? 1024 : 6144)) return quant_t<FMT, 2, 256, 5>(a, st);
    if (a.H <= 8192) return quant_t<FMT, 4, 128, NV ? 7 : 8>(a, st);
    return quant_t<FMT, 4, 256, NV ? 3 : 4>(a, st);  // H <= 16384
}

cudaError_t launch_norm(const NormArgs& args, cudaStream_t st) {
    NormArgs a = args;
    a.inv_h = 1.0f / (float)a.H;
    // whether the sizes, strides and addresses give every row whole, aligned 16-byte pieces
    uintptr_t bits = (uintptr_t)a.x | (uintptr_t)(2 * a.ldx) | (uintptr_t)(2 * a.H);
    if (a.res) bits |= (uintptr_t)a.res | (uintptr_t)(2 * a.ldr);
    if (a.sum) bits |= (uintptr_t)a.sum | (uintptr_t)(2 * a.lds);
    if (a.out) bits |= (uintptr_t)a.out | (uintptr_t)(2 * a.ldo);
    const bool ragged = bits % 16 != 0;
    if (!a.gamma && !ragged) {
        switch (a.fmt) {
            case MOE_FMT_MXFP8: return quant_f<MOE_FMT_MXFP8>(a, st);
            case MOE_FMT_NVFP4: return quant_f<MOE_FMT_NVFP4>(a, st);
            default: return quant_f<MOE_FMT_MXFP4>(a, st);
        }
    }
    switch (a.fmt) {
        case MOE_FMT_MXFP8: return ragged ? norm_f<MOE_FMT_MXFP8, true>(a, st) : norm_f<MOE_FMT_MXFP8, false>(a, st);
        case MOE_FMT_NVFP4: return ragged ? norm_f<MOE_FMT_NVFP4, true>(a, st) : norm_f<MOE_FMT_NVFP4, false>(a, st);
        case MOE_FMT_MXFP4: return ragged ? norm_f<MOE_FMT_MXFP4, true>(a, st) : norm_f<MOE_FMT_MXFP4, false>(a, st);
        default:
            // 4-byte pieces where they are whole: 4096 x 4098 with residual 27.8 us against 39.2 through
            // the ragged variant (4096 x 4097: 39.6), 22.3 for aligned 4096 x 4096. Five pairs a thread where
            // 256 threads hold the row so: without a residual 2999 x 2050 7.3 us, with eight 9.4; 3000 x
            // 2558 8.1 and 10.2; 3000 x 1026 4.9 and 5.6.
            if (ragged && bits % 4 == 0)
                return a.H <= 2 * 5 * 256 ? norm_pairs<5, 256>(a, st) : norm_pairs<8, 1024>(a, st);
            return ragged ? norm_f<-1, true>(a, st) : norm_f<-1, false>(a, st);
    }
}

}  // namespace moe
