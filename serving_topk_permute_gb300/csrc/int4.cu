// int4.cu -- product of bf16 activations with 4-bit integer weights that have a scale, and optionally a zero
// point, for each group of K (moe_int4_forward):
//   out[t, n] = bf16(sum_k x[t, k] (q[n, k] - z[n, k / g]) s[n, k / g]),  z = 8 without zero points
//
// Weights are laid out once in units of 16 features x 64 k, 512 bytes: lane i of a warp owns 16 bytes, in 4
// words the 16 k steps; word s holds, for the features i / 4 and i / 4 + 8, the four k from 16 s + 4 (i % 4) on.
// That is what lane i feeds to the tensor cores for its rows, from registers (mma.sync) as well as through
// tensor memory (16 lanes x 256 bits), so one layout serves every batch size. Inside a word the nibbles lie so
// that (w >> 4 i) & 0x000F000F is a pair of neighbouring k.
//
// A code becomes a bf16 without a conversion: 0x4300 | q is 128 + q, and 128 + q - (128 + z) is exact.
//
// int4_few_kernel: up to 16 tokens a tile. The codes go from global memory straight into the registers of the
// warps that multiply them; a CTA's warps share out K, and the CTAs of a cluster where there are few features.
// Products of whole numbers times activations are summed for each group in fp32 and scaled there: the only
// roundings are fp32's.
#include <cuda_fp16.h>

#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "pipeline.cuh"
#include "quant.cuh"

namespace moe {

// ------------------------------------------------------------------ layout
// where nibble i of a word comes from: feature + 8 row(i), k offset(i)
__host__ __device__ constexpr int nibble_row(int i) { return i & 1; }
__host__ __device__ constexpr int nibble_k(int i) { return (i >> 2 & 1) + (i & 2); }

// one thread for each word of the codes
__global__ void __launch_bounds__(256) int4_codes_kernel(const uint8_t* src, uint32_t* dst, int N, int K, int64_t words) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    if (at >= words) return;
    const int units = int4_units(K);
    const int s = (int)(at % 4), lane = (int)(at / 4 % 32);
    const int64_t unit = at / 128;
    const int u = (int)(unit % units), tile = (int)(unit / units);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = 16 * tile + lane / 4 + 8 * nibble_row(i), k = 64 * u + 16 * s + 4 * (lane % 4) + nibble_k(i);
        if (n < N && k < K) w |= (uint32_t)(src[((int64_t)n * K + k) / 2] >> (4 * (k % 2)) & 15) << (4 * i);
    }
    dst[at] = w;
}
// Scales: for each 16 features and group, 8 words of the scales of the features i and i + 8; zero points
// behind them: 8 bytes of the two nibbles. One thread for each word. Features past N have the scale 0.
__global__ void __launch_bounds__(256)
    int4_scales_kernel(const uint16_t* scales, const uint8_t* zeros, uint32_t* dst, uint8_t* dst_zeros, int N, int groups,
                       int slots, int64_t words) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    if (at >= words) return;
    const int i = (int)(at % 8), g = (int)(at / 8 % slots);
    const int64_t n = 16 * (at / 8 / slots) + i;
    auto scale = [&](int64_t row) { return row < N && g < groups ? (uint32_t)scales[row * groups + g] : 0u; };
    dst[at] = scale(n) | scale(n + 8) << 16;
    if (zeros) {
        auto zero = [&](int64_t row) { return row < N && g < groups ? (uint32_t)zeros[row * groups + g] & 15u : 0u; };
        dst_zeros[at] = (uint8_t)(zero(n) | zero(n + 8) << 4);
    }
}

// rows that are not 16-byte aligned, into the workspace
__global__ void __launch_bounds__(256) int4_rows_kernel(const uint16_t* x, int64_t ldx, uint4* dst, int K, int64_t pieces) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    if (at >= pieces) return;
    const int per_row = K / 8;
    const uint16_t* p = x + at / per_row * ldx + at % per_row * 8;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (uint32_t)p[2 * j] | (uint32_t)p[2 * j + 1] << 16;
    dst[at] = make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ codes to bf16
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// A word's fragment: (k, k + 1) of the features i and i + 8, then (k + 2, k + 3), as whole numbers q - z.
// low, high: 128 + z of the two features, twice each.
__device__ __forceinline__ void whole_numbers(uint32_t w, uint32_t low, uint32_t high, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t q = (w >> (4 * i) & 0x000F000Fu) | 0x43004300u;
        a[i] = sub_bf16x2(q, i & 1 ? high : low);
    }
}
// 128 + z twice, of the byte of two zero points
__device__ __forceinline__ void zero_points(uint32_t byte, uint32_t& low, uint32_t& high) {
    low = 0x43004300u | (byte & 15u) * 0x00010001u;
    high = 0x43004300u | (byte >> 4 & 15u) * 0x00010001u;
}
// the scales of two features from their word
template <bool HALF>
__device__ __forceinline__ float2 two_scales(uint32_t w) {
    if constexpr (HALF) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// ------------------------------------------------------------------ few tokens
constexpr int FEW_WARPS = 8, FEW_THREADS = 32 * FEW_WARPS;
constexpr int few_max_splits(int RT, int MT) { return RT * MT >= 8 ? 2 : 8; }  // by shared memory

// RT: 16-feature tiles of a CTA, MT: 8-token tiles, DEPTH: units in flight in a warp. SPAN: groups of a unit (2: of
// 32 k, 1: of 64 or 128).
template <int RT, int MT, int DEPTH, int SPAN, bool ZEROS, bool HALF>
__global__ void __launch_bounds__(FEW_THREADS, 2) int4_few_kernel(const Int4Args p) {
    constexpr int F = 16 * RT, TOKENS = 8 * MT;
    __shared__ float s_part[FEW_WARPS][TOKENS][F];
    __shared__ float s_sum[few_max_splits(RT, MT)][TOKENS * F];  // rank 0: the CTAs' sums
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane % 4;
    const int rank = blockIdx.x, splits = gridDim.x, tile0 = blockIdx.y * RT, t0 = blockIdx.z * TOKENS;
    const int units = int4_units(p.K);
    const int u1 = (int)((int64_t)units * (rank + 1) / splits);
    // matched just before the first store into another CTA's shared memory: by then it has started
    if (splits > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    grid_dep_wait();
    grid_dep_launch();
    float acc[RT][MT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][m][j] = 0.0f;
    const int tiles = (p.N + 15) / 16;
    const __nv_bfloat16* x[MT];
    bool token[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int t = t0 + 8 * m + lane / 4;
        token[m] = t < p.M;
        x[m] = p.x + (token[m] ? t : 0) * p.ldx + 4 * q;
    }
    for (int u0 = (int)((int64_t)units * rank / splits) + warp; u0 < u1; u0 += FEW_WARPS * DEPTH) {
        uint4 codes[DEPTH][RT];
        uint2 xs[DEPTH][MT][4];
        uint32_t sc[DEPTH][RT][SPAN], zp[DEPTH][RT][SPAN];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int u = u0 + d * FEW_WARPS;
            const bool in = u < u1;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                codes[d][r] = make_uint4(0, 0, 0, 0);
                const bool there = in && tile0 + r < tiles;
                if (there) codes[d][r] = p.codes[((int64_t)(tile0 + r) * units + u) * 32 + lane];
#pragma unroll
                for (int g = 0; g < SPAN; ++g) {
                    sc[d][r][g] = zp[d][r][g] = 0;
                    if (there) {
                        const int64_t at = ((int64_t)(tile0 + r) * p.slots + (SPAN == 2 ? 2 * u + g : u >> p.unit_shift)) * 8 + lane / 4;
                        sc[d][r][g] = p.scales[at];
                        if (ZEROS) zp[d][r][g] = p.zeros[at];
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    xs[d][m][s] = make_uint2(0, 0);
                    if (in && token[m] && 64 * u + 16 * s < p.K)
                        xs[d][m][s] = *reinterpret_cast<const uint2*>(x[m] + 64 * u + 16 * s);
                }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t w[4] = {codes[d][r].x, codes[d][r].y, codes[d][r].z, codes[d][r].w};
#pragma unroll
                for (int g = 0; g < SPAN; ++g) {
                    uint32_t low = 0x43084308u, high = low;  // 136: the zero point is 8
                    if (ZEROS) zero_points(zp[d][r][g], low, high);
                    float part[MT][4];
#pragma unroll
                    for (int m = 0; m < MT; ++m) part[m][0] = part[m][1] = part[m][2] = part[m][3] = 0.0f;
#pragma unroll
                    for (int s = 4 / SPAN * g; s < 4 / SPAN * (g + 1); ++s) {
                        uint32_t a[4];
                        whole_numbers(w[s], low, high, a);
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma_16x8x16(part[m], a, xs[d][m][s]);
                    }
                    const float2 f = two_scales<HALF>(sc[d][r][g]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        acc[r][m][0] = fmaf(f.x, part[m][0], acc[r][m][0]);
                        acc[r][m][1] = fmaf(f.x, part[m][1], acc[r][m][1]);
                        acc[r][m][2] = fmaf(f.y, part[m][2], acc[r][m][2]);
                        acc[r][m][3] = fmaf(f.y, part[m][3], acc[r][m][3]);
                    }
                }
            }
    }
    // the warps in order, then the CTAs
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s_part[warp][8 * m + 2 * q + (j & 1)][16 * r + lane / 4 + 8 * (j >> 1)] = acc[r][m][j];
    __syncthreads();
    if (splits > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    const int tokens = min(TOKENS, p.M - t0);
    const uint32_t sums = splits > 1 ? mapa_shared(smem_u32(s_sum[rank]), 0) : 0;
    __nv_bfloat16* out = p.out + t0 * p.ldo + tile0 * 16;
    for (int i = threadIdx.x; i < tokens * F; i += FEW_THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < FEW_WARPS; ++w) v += s_part[w][i / F][i % F];
        if (splits > 1)
            st_cluster_u32(sums + 4 * i, __float_as_uint(v));
        else if (tile0 * 16 + i % F < p.N)
            out[i / F * p.ldo + i % F] = __float2bfloat16_rn(v);
    }
    if (splits > 1) {
        cluster_sync();
        if (rank > 0) return;
        for (int i = threadIdx.x; i < tokens * F; i += FEW_THREADS) {
            float v = 0.0f;
            for (int r = 0; r < splits; ++r) v += s_sum[r][i];
            if (tile0 * 16 + i % F < p.N) out[i / F * p.ldo + i % F] = __float2bfloat16_rn(v);
        }
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) p.status[0] = 0;  // no CTA of this kernel waits
}

// ------------------------------------------------------------------ host side
cudaError_t launch_int4_layout(const Int4Layout& a, cudaStream_t st) {
    const int64_t tiles = int4_tiles(a.N), words = tiles * int4_units(a.K) * 128;
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)ceil_div(words, 256)), dim3(256), 0, st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, int4_codes_kernel, a.src_codes, a.codes, a.N, a.K, words);
    if (e != cudaSuccess) return e;
    const int slots = int4_slots(a.K, a.group);
    const int64_t swords = tiles * slots * 8;
    LaunchAttrs at2(true);
    cfg = at2.config(dim3((unsigned)ceil_div(swords, 256)), dim3(256), 0, st);
    return cudaLaunchKernelEx(&cfg, int4_scales_kernel, a.src_scales, a.src_zeros, a.scales, a.zeros, a.N,
                              (int)ceil_div(a.K, a.group), slots, swords);
}

cudaError_t launch_int4_rows(const void* x, int64_t ldx, void* dst, int M, int K, cudaStream_t st) {
    const int64_t pieces = (int64_t)M * (K / 8);
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)ceil_div(pieces, 256)), dim3(256), 0, st);
    return cudaLaunchKernelEx(&cfg, int4_rows_kernel, (const uint16_t*)x, ldx, (uint4*)dst, K, pieces);
}

template <int RT, int MT, int DEPTH, int SPAN, bool ZEROS, bool HALF>
static cudaError_t few_t(const Int4Args& p, int splits, cudaStream_t st) {
    LaunchAttrs at(true, splits);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)splits, (unsigned)ceil_div(p.N, 16 * RT), (unsigned)ceil_div(p.M, 8 * MT)),
                                       dim3(FEW_THREADS), 0, st);
    return cudaLaunchKernelEx(&cfg, int4_few_kernel<RT, MT, DEPTH, SPAN, ZEROS, HALF>, p);
}
template <int RT, int MT, int DEPTH>
static cudaError_t few_g(const Int4Args& p, int splits, cudaStream_t st) {
    const bool z = p.zeros != nullptr;
    if (p.group == 32) {
        if (z) return p.half ? few_t<RT, MT, DEPTH, 2, true, true>(p, splits, st) : few_t<RT, MT, DEPTH, 2, true, false>(p, splits, st);
        return p.half ? few_t<RT, MT, DEPTH, 2, false, true>(p, splits, st) : few_t<RT, MT, DEPTH, 2, false, false>(p, splits, st);
    }
    if (z) return p.half ? few_t<RT, MT, DEPTH, 1, true, true>(p, splits, st) : few_t<RT, MT, DEPTH, 1, true, false>(p, splits, st);
    return p.half ? few_t<RT, MT, DEPTH, 1, false, true>(p, splits, st) : few_t<RT, MT, DEPTH, 1, false, false>(p, splits, st);
}

static int few_splits(int64_t ctas, int units, int num_sms, int most) {
    int s = 1;
    while (2 * s <= most && ctas * 2 * s <= 4 * num_sms && units >= 2 * s * FEW_WARPS) s *= 2;
    return s;
}

cudaError_t launch_int4(const Int4Args& args, int num_sms, cudaStream_t st) {
    Int4Args p = args;
    p.slots = int4_slots(p.K, p.group);
    p.unit_shift = p.group == 128 ? 1 : 0;
    const int units = int4_units(p.K);
    auto few = [&](int RT, int MT) {
        return few_splits(ceil_div(p.N, 16 * RT) * ceil_div(p.M, 8 * MT), units, num_sms, few_max_splits(RT, MT));
    };
    if (p.M <= 2) return few_g<1, 1, 4>(p, few(1, 1), st);
    if (p.M <= 8) return few_g<2, 1, 4>(p, few(2, 1), st);
    return few_g<4, 2, 2>(p, few(4, 2), st);
}

int int4_max_ctas(int N, int num_sms) { return 0; }
cudaError_t int4_prepare() { return cudaSuccess; }

}  // namespace moe
