// int4.cu -- product of bf16 activations with 4-bit integer weights that have a scale, and optionally a zero
// point, for each group of K (moe_int4_forward):
//   out[t, n] = bf16(sum_k x[t, k] (q[n, k] - z[n, k / g]) s[n, k / g]),  z = 8 without zero points
//
// Weights are laid out once in blocks of 16 features x 128 k, two units of 64 k and 512 bytes each: lane i of a
// warp owns 16 bytes of a unit, in 4 words its 16 k steps; word s holds, for the features i / 4 and i / 4 + 8, the
// four k from 16 s + 4 (i % 4) on.
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
    const int units = 2 * int4_blocks(K);
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
// low, high: 128 + z of the two features, twice each. The shifts are the upper halves of products with 2^28 and so
// on, which p brings along so that they stay products: shifts and masks share a pipe of half the rate, which
// would bound the kernel.
__device__ __forceinline__ uint32_t upper(uint32_t w, uint32_t by) {
    unsigned long long r;
    asm("mul.wide.u32 %0, %1, %2;" : "=l"(r) : "r"(w), "r"(by));
    return (uint32_t)(r >> 32);
}
__device__ __forceinline__ void whole_numbers(const Int4Args& p, uint32_t w, uint32_t low, uint32_t high, uint32_t (&a)[4]) {
    const uint32_t v[4] = {w, upper(w, p.by4), upper(w, p.by8), upper(w, p.by12)};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = sub_bf16x2((v[i] & 0x000F000Fu) | 0x43004300u, i & 1 ? high : low);
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

// d = a b, or d += a b
__device__ __forceinline__ void mma_16x8x16_first(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.0f));
}
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// ------------------------------------------------------------------ few tokens
constexpr int few_max_splits(int RT, int MT) { return RT * MT >= 8 ? 2 : 8; }  // by shared memory

// RT: 16-feature tiles of a CTA, MT: 8-token tiles, SPAN: groups of a block. A warp takes every WARPS-th block of
// its CTA's, and fetches one block's codes, activations and scales while it multiplies another's.
template <int RT, int MT, int WARPS, int CTAS, int SPAN, bool ZEROS, bool HALF>
__global__ void __launch_bounds__(32 * WARPS, CTAS) int4_few_kernel(const __grid_constant__ Int4Args p) {
    constexpr int THREADS = 32 * WARPS;
    constexpr int F = 16 * RT, TOKENS = 8 * MT;
    __shared__ float s_part[WARPS][TOKENS][F];
    __shared__ float s_sum[few_max_splits(RT, MT)][TOKENS * F];  // rank 0: the CTAs' sums
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane % 4;
    const int rank = blockIdx.x, splits = gridDim.x, tile0 = blockIdx.y * RT, t0 = blockIdx.z * TOKENS;
    const int blocks = int4_blocks(p.K), whole = p.K / 128;
    const int first = (int)((int64_t)blocks * rank / splits) + warp, last = (int)((int64_t)blocks * (rank + 1) / splits);
    const int end = min(last, whole);
    // matched just before the first store into another CTA's shared memory: by then it has started
    if (splits > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    // Tiles past the last feature's are those of the padding, or the last one again, and tokens past the last one
    // are the first one again: their sums are not stored.
    const int last_tile = (int)int4_tiles(p.N) - 1;
    const uint4* codes[RT];
    const uint32_t* scales[RT];
    const uint8_t* zeros[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int tile = min(tile0 + r, last_tile);
        codes[r] = p.codes + ((int64_t)tile * blocks + first) * 64 + lane;
        const int64_t at = ((int64_t)tile * p.slots + SPAN * first) * 8 + lane / 4;
        scales[r] = p.scales + at;
        zeros[r] = p.zeros + at;
    }
    const __nv_bfloat16* x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int t = t0 + 8 * m + lane / 4;
        x[m] = p.x + (t < p.M ? t : 0) * p.ldx + 128 * first + 4 * q;
    }
    grid_dep_wait();
    grid_dep_launch();
    float acc[RT][MT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][m][j] = 0.0f;
    struct Block {
        uint4 codes[RT][2];
        uint2 x[MT][8];
        uint32_t scale[RT][SPAN], zero[RT][SPAN];
    };
    auto fetch = [&](Block& a, int steps) {  // the block that the addresses stand at, which has so many steps of 16 k
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            a.codes[r][0] = codes[r][0];
            a.codes[r][1] = codes[r][32];
            codes[r] += 64 * WARPS;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (steps == 8)
                    a.x[m][s] = *reinterpret_cast<const uint2*>(x[m] + 16 * s);
                else
                    a.x[m][s] = s < steps ? *reinterpret_cast<const uint2*>(x[m] + 16 * s) : make_uint2(0, 0);
            }
            x[m] += 128 * WARPS;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int g = 0; g < SPAN; ++g) {
                a.scale[r][g] = scales[r][8 * g];
                if (ZEROS) a.zero[r][g] = zeros[r][8 * g];
            }
            scales[r] += 8 * SPAN * WARPS;
            if (ZEROS) zeros[r] += 8 * SPAN * WARPS;
        }
    };
    auto multiply = [&](const Block& h) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint32_t w[8] = {h.codes[r][0].x, h.codes[r][0].y, h.codes[r][0].z, h.codes[r][0].w,
                                   h.codes[r][1].x, h.codes[r][1].y, h.codes[r][1].z, h.codes[r][1].w};
#pragma unroll
            for (int g = 0; g < SPAN; ++g) {
                uint32_t low = 0x43084308u, high = low;  // 136: the zero point is 8
                if (ZEROS) zero_points(h.zero[r][g], low, high);
                float part[MT][4];
#pragma unroll
                for (int s = 0; s < 8 / SPAN; ++s) {
                    uint32_t a[4];
                    whole_numbers(p, w[8 / SPAN * g + s], low, high, a);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (s == 0)
                            mma_16x8x16_first(part[m], a, h.x[m][8 / SPAN * g]);
                        else
                            mma_16x8x16(part[m], a, h.x[m][8 / SPAN * g + s]);
                    }
                }
                const float2 f = two_scales<HALF>(h.scale[r][g]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    acc[r][m][0] = fmaf(f.x, part[m][0], acc[r][m][0]);
                    acc[r][m][1] = fmaf(f.x, part[m][1], acc[r][m][1]);
                    acc[r][m][2] = fmaf(f.y, part[m][2], acc[r][m][2]);
                    acc[r][m][3] = fmaf(f.y, part[m][3], acc[r][m][3]);
                }
            }
        }
    };
    Block one, two;
    int b = first;
    if (b < end) fetch(one, 8);
#pragma unroll 1
    for (; b < end; b += 2 * WARPS) {
        if (b + WARPS < end) fetch(two, 8);
        multiply(one);
        if (b + WARPS >= end) {
            b += WARPS;
            break;
        }
        if (b + 2 * WARPS < end) fetch(one, 8);
        multiply(two);
    }
    if (b < last) {  // the block inside which K ends: the addresses stand at it
        fetch(one, (p.K - 128 * b) / 16);
        multiply(one);
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
    for (int i = threadIdx.x; i < tokens * F; i += THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += s_part[w][i / F][i % F];
        if (splits > 1)
            st_cluster_u32(sums + 4 * i, __float_as_uint(v));
        else if (tile0 * 16 + i % F < p.N)
            out[i / F * p.ldo + i % F] = __float2bfloat16_rn(v);
    }
    if (splits > 1) {
        cluster_sync();
        if (rank > 0) return;
        for (int i = threadIdx.x; i < tokens * F; i += THREADS) {
            float v = 0.0f;
            for (int r = 0; r < splits; ++r) v += s_sum[r][i];
            if (tile0 * 16 + i % F < p.N) out[i / F * p.ldo + i % F] = __float2bfloat16_rn(v);
        }
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) p.status[0] = 0;  // no CTA of this kernel waits
}

// ------------------------------------------------------------------ more tokens
// bf16 pairs q s of whole numbers: the nearest ones. An fp16 scale is two bf16, the second the exact rest of the
// first, its product with q exact: one FMA rounds their sum.
template <bool HALF>
struct Scaled {
    uint32_t hi[2], lo[2];  // of the two features, twice each
    __device__ __forceinline__ explicit Scaled(uint32_t w) {
        if constexpr (HALF) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
            const float v[2] = {f.x, f.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
                // an infinite or NaN scale has no rest
                const float rest = isfinite(v[i]) ? v[i] - __bfloat162float(h) : 0.0f;
                const __nv_bfloat162 a = __bfloat162bfloat162(h), b = __float2bfloat162_rn(rest);
                hi[i] = *reinterpret_cast<const uint32_t*>(&a);
                lo[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        } else {
            hi[0] = __byte_perm(w, 0, 0x1010);
            hi[1] = __byte_perm(w, 0, 0x3232);
        }
    }
    __device__ __forceinline__ uint32_t times(uint32_t q, int feature) const {
        const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&q);
        const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&hi[feature]);
        __nv_bfloat162 r;
        if constexpr (HALF)
            r = __hfma2(a, s, __hmul2(a, *reinterpret_cast<const __nv_bfloat162*>(&lo[feature])));
        else
            r = __hmul2(a, s);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
};

// 16 lanes x 32 columns of tensor memory: registers 4 i .. 4 i + 3 are columns 8 i + 2 (lane % 4) and the next one,
// of the tensor-memory lane lane / 4, then of lane / 4 + 8
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// A (128 rows x 16 k) from tensor memory
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

constexpr int MANY_WARPS = 8;                        // that make bf16 weights of the codes, and store the tile
constexpr int MANY_THREADS = 64 + 32 * MANY_WARPS;   // warp 0: copies, warp 1: MMAs
constexpr int MANY_MAX_SPLITS = 8;

template <int BT>
struct ManyCfg {
    static constexpr int X_BYTES = BT * 256, CODE_BYTES = 8192;  // a stage of 128 k: tokens in two swizzled halves, codes
    static constexpr int STAGE = X_BYTES + CODE_BYTES;
    static constexpr int BAR_BYTES = 256;
    static constexpr int CTAS = BT <= 128 ? 2 : 1;
    static constexpr int BUDGET = (CTAS == 2 ? 233472 / 2 - 1024 : 232448) - BAR_BYTES - 1024;
    static constexpr int STAGES = BUDGET / STAGE < 6 ? BUDGET / STAGE : 6;
    static constexpr int SMEM = STAGES * STAGE + BAR_BYTES + 1024;
    static constexpr int BUFS = BT == 256 ? 4 : 2;   // weights of a stage in tensor memory: 64 columns each
    static constexpr int TMEM = BT == 256 ? 512 : 256;
    static constexpr int SUM_BYTES = (BT + MANY_MAX_SPLITS) * 128 * 4;
    static_assert(BT + 64 * BUFS <= TMEM && (2 * STAGES + 2 * BUFS + 2) * 8 + 16 <= BAR_BYTES, "budgets");
    static_assert(BT == 256 || STAGES * STAGE >= SUM_BYTES, "the ring holds the sums");
    static_assert(STAGES >= 2, "stages");
};

// 128 features x BT tokens a CTA, K split over the CTAs of a cluster where there are few tiles. Each stage of 128 k:
// the tokens come by TMA, the codes by bulk copies; eight warps turn the codes into bf16 weights and store
// them to tensor memory, from where the MMAs take them as their row side, with the tokens in shared memory as
// columns. So weights never pass through shared memory as bf16, and a tile's features are the accumulator's lanes.
template <int BT, int SPAN, bool ZEROS, bool HALF>
__global__ void __launch_bounds__(MANY_THREADS, ManyCfg<BT>::CTAS)
    int4_many_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ Int4Args p) {
    using C = ManyCfg<BT>;
    constexpr int STAGES = C::STAGES, BUFS = C::BUFS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2 * BUFS + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* never = reinterpret_cast<int*>(tmem_slot + 2);
    float* sums = reinterpret_cast<float*>(smem);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, made0 = empty0 + 8 * STAGES,
                   used0 = made0 + 8 * BUFS, done_bar = used0 + 8 * BUFS, free_bar = done_bar + 8;
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t tmo = p.timeout_ns;
    const uint32_t splits = gridDim.x, rank = blockIdx.x;
    const int blocks = int4_blocks(p.K), n_tiles = (p.N + 127) / 128, tiles = n_tiles * ((p.M + BT - 1) / BT);
    const int k0 = (int)((int64_t)blocks * rank / splits), steps = (int)((int64_t)blocks * (rank + 1) / splits) - k0;
    // a CTA's tiles, one after the other: a split tile's cluster has one alone
    const int tile0 = blockIdx.y, tile_step = gridDim.y;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1 + MANY_WARPS);  // the MMAs' commit, and each warp that has read its codes
        }
        for (int b = 0; b < BUFS; ++b) {
            mbar_init(made0 + 8 * b, MANY_WARPS);
            mbar_init(used0 + 8 * b, 1);
        }
        mbar_init(done_bar, 1);
        mbar_init(free_bar, MANY_WARPS);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot, weights0 = tmem_base + BT;
    auto give_up = [&]() { *abort_flag = 1; };
    grid_dep_wait();
    grid_dep_launch();

    bool complete = true;  // meaningful in the warps that store
    if (warp == 0) {
        const bool elected = elect_one();
        int issued = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < tiles; tile += tile_step) {
            const int nt = tile % n_tiles, tt = tile / n_tiles;
            for (int i = 0; i < steps; ++i, ++issued) {
                const int stage = issued % STAGES;
                if (!warp_wait(empty0 + 8 * stage, ((issued / STAGES) & 1) ^ 1, tmo, abort_flag)) {
                    give_up();
                    ok = false;
                    break;
                }
                if (elected) {
                    const uint32_t st = smem0 + stage * C::STAGE, full = full0 + 8 * stage;
                    const int ks = k0 + i;
                    mbar_arrive_expect_tx(full, C::STAGE);
                    tma_load_2d(st, &tmX, full, 128 * ks, tt * BT);
                    tma_load_2d(st + C::X_BYTES / 2, &tmX, full, 128 * ks + 64, tt * BT);
                    const uint4* codes = p.codes + ((int64_t)nt * 8 * blocks + ks) * 64;
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        bulk_load(st + C::X_BYTES + 1024 * r, codes + (int64_t)r * blocks * 64, 1024, full);
                }
                __syncwarp();
            }
        }
        // every load issued lands before the CTA may exit or reuse the ring
        for (int s = 0; s < STAGES && s < issued; ++s) {
            const int last = s + (issued - 1 - s) / STAGES * STAGES;
            mbar_wait(full0 + 8 * s, (last / STAGES) & 1, DRAIN_TIMEOUT_NS, never);
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool elected = elect_one();
        int at = 0, round = 0;  // stages, tiles so far
        bool ok = true;
        for (int tile = tile0; ok && tile < tiles; tile += tile_step, ++round) {
            if (round > 0 && !warp_wait(free_bar, (round - 1) & 1, tmo, abort_flag)) {  // the accumulators
                give_up();
                break;
            }
            for (int i = 0; i < steps; ++i, ++at) {
                const int stage = at % STAGES, buf = at % BUFS;
                if (!warp_wait(full0 + 8 * stage, (at / STAGES) & 1, tmo, abort_flag) ||
                    !warp_wait(made0 + 8 * buf, (at / BUFS) & 1, tmo, abort_flag)) {
                    give_up();
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elected) {
                    const uint32_t x = (smem0 + stage * C::STAGE) / 16, w = weights0 + 64 * buf;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mma_bf16_ta(tmem_base, w + 8 * j, row_desc(x + j / 4 * (C::X_BYTES / 32) + 2 * (j % 4)),
                                    idesc_bf16(BT), i > 0 || j > 0);
                    tc_commit(empty0 + 8 * stage);
                    tc_commit(used0 + 8 * buf);
                }
                __syncwarp();
            }
            // every MMA issued has completed; also the signal to store
            if (elected) tc_commit(done_bar);
            __syncwarp();
        }
        if (round > 0) mbar_wait(done_bar, (round - 1) & 1, DRAIN_TIMEOUT_NS, never);
        __syncwarp();
    } else {
        // a quarter of the tensor memory's lanes, two tiles of 16 features, and one of the stage's units
        const int quarter = warp % 4, half = (warp - 2) / 4;
        const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16);
        constexpr int OWN = SPAN == 4 ? 2 : 1;  // groups of a unit
        uint32_t sc[2][OWN], zp[2][OWN];
        auto fetch = [&](int tile, int i) {  // the scales of a tile's stage, or of the next tile's first one
            if (i == steps) i = 0, tile += tile_step;
            if (tile >= tiles) return;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < OWN; ++g) {
                    const int slot = SPAN * (k0 + i) + (SPAN == 1 ? 0 : OWN * half) + g;
                    const int64_t from = ((int64_t)(tile % n_tiles * 8 + 2 * quarter + j) * p.slots + slot) * 8 + lane / 4;
                    sc[j][g] = p.scales[from];
                    if (ZEROS) zp[j][g] = p.zeros[from];
                }
        };
        int at = 0, round = 0;
        fetch(tile0, 0);
        for (int tile = tile0; complete && tile < tiles; tile += tile_step, ++round) {
            for (int i = 0; i < steps; ++i, ++at) {
                const int stage = at % STAGES, buf = at % BUFS;
                uint32_t scale[2][OWN], zero[2][OWN];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int g = 0; g < OWN; ++g) scale[j][g] = sc[j][g], zero[j][g] = ZEROS ? zp[j][g] : 0;
                fetch(tile, i + 1);
                if (!warp_wait(full0 + 8 * stage, (at / STAGES) & 1, tmo, abort_flag)) {
                    complete = false;
                    break;
                }
                uint4 codes[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    codes[j] = *reinterpret_cast<const uint4*>(smem + stage * C::STAGE + C::X_BYTES +
                                                               (2 * quarter + j) * 1024 + half * 512 + lane * 16);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * stage);
                if (!warp_wait(used0 + 8 * buf, ((at / BUFS) & 1) ^ 1, tmo, abort_flag)) {
                    complete = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
                    uint32_t r[16];
#pragma unroll
                    for (int g = 0; g < OWN; ++g) {
                        uint32_t low = 0x43084308u, high = low;  // 136: the zero point is 8
                        if (ZEROS) zero_points(zero[j][g], low, high);
                        const Scaled<HALF> scaled(scale[j][g]);
#pragma unroll
                        for (int s = 4 / OWN * g; s < 4 / OWN * (g + 1); ++s) {
                            uint32_t a[4];
                            whole_numbers(p, w[s], low, high, a);
                            r[4 * s] = scaled.times(a[0], 0);
                            r[4 * s + 1] = scaled.times(a[2], 0);
                            r[4 * s + 2] = scaled.times(a[1], 1);
                            r[4 * s + 3] = scaled.times(a[3], 1);
                        }
                    }
                    tmem_st_16x32(weights0 + 64 * buf + 32 * half + ((uint32_t)(32 * quarter + 16 * j) << 16), r);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(made0 + 8 * buf);
            }
            if (complete) complete = warp_wait(done_bar, round & 1, tmo, abort_flag);
            if (!complete) {
                give_up();
                break;
            }
            tc_fence_after();
            if (splits > 1) continue;
            const int n = tile % n_tiles * 128 + quarter * 32 + lane, t0 = tile / n_tiles * BT;
            const int tokens = min(BT, p.M - t0);
#pragma unroll 1
            for (int c0 = half * 32; c0 < tokens; c0 += 64) {
                float v[32];
                tmem_ld32(tacc + c0, v);
                tmem_ld_wait();
                if (n < p.N) {
                    __nv_bfloat16* o = p.out + (int64_t)(t0 + c0) * p.ldo + n;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c0 + j < tokens) *o = __float2bfloat16_rn(v[j]);
                        o += p.ldo;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(free_bar);
        }
    }
    // Sums of a split tile: its tokens are shared out in runs of per_rank, and every CTA sends its accumulators of a
    // token to its owner. The ring, which serves as that area, is free in all CTAs after the first barrier.
    if (splits > 1) {
        const int nt = tile0 % n_tiles, t0 = tile0 / n_tiles * BT, tokens = min(BT, p.M - t0);
        const int per_rank = (tokens + (int)splits - 1) / (int)splits;
        cluster_sync();
        if (warp >= 2) {
            const int quarter = warp % 4;
            const uint32_t mine = smem_u32(sums + (int)rank * per_rank * 128 + quarter * 32 + lane);
#pragma unroll 1
            for (int c0 = (warp - 2) / 4 * 32; c0 < tokens; c0 += 64) {
                float v[32];
                tmem_ld32(tmem_base + ((uint32_t)(quarter * 32) << 16) + c0, v);
                tmem_ld_wait();
                int owner = c0 / per_rank, left = (owner + 1) * per_rank - c0;  // tokens until the next owner
                uint32_t at = mapa_shared(mine + (c0 - owner * per_rank) * 512, owner);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j < tokens) st_cluster_u32(at, __float_as_uint(v[j]));
                    at += 512;
                    if (--left == 0 && c0 + j + 1 < tokens) {
                        at = mapa_shared(mine, ++owner);
                        left = per_rank;
                    }
                }
            }
            tc_fence_before();
        }
        cluster_sync();
        // this CTA's tokens: a warp takes a token, a lane 4 features, the ranks added in order
        if (warp >= 2 && complete) {
            const int first = (int)rank * per_rank, count = min(per_rank, tokens - first);
            for (int i = warp - 2; i < count; i += MANY_WARPS) {
                const float4* u = reinterpret_cast<const float4*>(sums + i * 128) + lane;
                float4 y = u[0];
                for (uint32_t r = 1; r < splits; ++r) {
                    const float4 v = u[r * per_rank * 32];
                    y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
                }
                const int n = nt * 128 + 4 * lane;
                __nv_bfloat16* o = p.out + (int64_t)(t0 + first + i) * p.ldo + n;
                if (n < p.N) o[0] = __float2bfloat16_rn(y.x);
                if (n + 1 < p.N) o[1] = __float2bfloat16_rn(y.y);
                if (n + 2 < p.N) o[2] = __float2bfloat16_rn(y.z);
                if (n + 3 < p.N) o[3] = __float2bfloat16_rn(y.w);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {  // after every warp's last wait
        const uint32_t cta = blockIdx.x + gridDim.x * blockIdx.y;
        if (cta == 0) p.status[0] = (int)(gridDim.x * gridDim.y);
        p.status[1 + cta] = *abort_flag != 0 ? MOE_ERR_TIMEOUT : MOE_OK;
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM);
    }
}

// ------------------------------------------------------------------ host side
cudaError_t launch_int4_layout(const Int4Layout& a, cudaStream_t st) {
    const int64_t tiles = int4_tiles(a.N), words = tiles * int4_blocks(a.K) * 256;
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

template <int RT, int MT, int WARPS, int CTAS, int SPAN, bool ZEROS, bool HALF>
static cudaError_t few_t(const Int4Args& p, int splits, cudaStream_t st) {
    LaunchAttrs at(true, splits);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)splits, (unsigned)ceil_div(p.N, 16 * RT), (unsigned)ceil_div(p.M, 8 * MT)),
                                       dim3(32 * WARPS), 0, st);
    return cudaLaunchKernelEx(&cfg, int4_few_kernel<RT, MT, WARPS, CTAS, SPAN, ZEROS, HALF>, p);
}
template <int RT, int MT, int WARPS, int CTAS, int SPAN>
static cudaError_t few_s(const Int4Args& p, int splits, cudaStream_t st) {
    if (p.zeros) return p.half ? few_t<RT, MT, WARPS, CTAS, SPAN, true, true>(p, splits, st) : few_t<RT, MT, WARPS, CTAS, SPAN, true, false>(p, splits, st);
    return p.half ? few_t<RT, MT, WARPS, CTAS, SPAN, false, true>(p, splits, st) : few_t<RT, MT, WARPS, CTAS, SPAN, false, false>(p, splits, st);
}
template <int RT, int MT, int WARPS, int CTAS>
static cudaError_t few_g(const Int4Args& p, int num_sms, cudaStream_t st) {
    // K over the CTAs of a cluster, as long as all CTAs fit and a warp has two blocks or more
    const int64_t ctas = ceil_div(p.N, 16 * RT) * ceil_div(p.M, 8 * MT);
    int s = 1;
    while (2 * s <= few_max_splits(RT, MT) && ctas * 2 * s <= CTAS * num_sms && int4_blocks(p.K) >= 4 * s * WARPS) s *= 2;
    return p.group == 32   ? few_s<RT, MT, WARPS, CTAS, 4>(p, s, st)
           : p.group == 64 ? few_s<RT, MT, WARPS, CTAS, 2>(p, s, st)
                           : few_s<RT, MT, WARPS, CTAS, 1>(p, s, st);
}

template <int BT, int SPAN, bool ZEROS, bool HALF>
static cudaError_t many_t(const CUtensorMap& x, const Int4Args& p, int splits, int num_sms, cudaStream_t st) {
    using C = ManyCfg<BT>;
    const auto kernel = int4_many_kernel<BT, SPAN, ZEROS, HALF>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ceil_div(p.N, 128) * ceil_div(p.M, BT), most = (int64_t)C::CTAS * num_sms;
    LaunchAttrs at(true, splits);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)splits, (unsigned)(splits > 1 || tiles < most ? tiles : most)),
                                       dim3(MANY_THREADS), C::SMEM, st);
    return cudaLaunchKernelEx(&cfg, kernel, x, p);
}
template <int BT, int SPAN>
static cudaError_t many_s(const CUtensorMap& x, const Int4Args& p, int s, int sms, cudaStream_t st) {
    if (p.zeros) return p.half ? many_t<BT, SPAN, true, true>(x, p, s, sms, st) : many_t<BT, SPAN, true, false>(x, p, s, sms, st);
    return p.half ? many_t<BT, SPAN, false, true>(x, p, s, sms, st) : many_t<BT, SPAN, false, false>(x, p, s, sms, st);
}
template <int BT>
static cudaError_t many_g(const CUtensorMap& x, const Int4Args& p, int num_sms, cudaStream_t st) {
    // K over the CTAs of a cluster, as long as all CTAs fit and each has four stages or more
    const int64_t tiles = ceil_div(p.N, 128) * ceil_div(p.M, BT);
    int s = 1;
    while (BT < 256 && 2 * s <= MANY_MAX_SPLITS && tiles * 2 * s <= ManyCfg<BT>::CTAS * num_sms && int4_blocks(p.K) >= 8 * s) s *= 2;
    return p.group == 32   ? many_s<BT, 4>(x, p, s, num_sms, st)
           : p.group == 64 ? many_s<BT, 2>(x, p, s, num_sms, st)
                           : many_s<BT, 1>(x, p, s, num_sms, st);
}

static int many_tokens(int M) { return M <= 32 ? 32 : M <= 64 ? 64 : M <= 512 ? 128 : 256; }
bool int4_few(int M) { return M <= 16; }
int int4_box(int M) { return many_tokens(M); }

cudaError_t launch_int4(const CUtensorMap& x, const Int4Args& args, int num_sms, cudaStream_t st) {
    Int4Args p = args;
    p.slots = int4_slots(p.K, p.group);
    p.by4 = 1u << 28;
    p.by8 = 1u << 24;
    p.by12 = 1u << 20;
    if (p.M <= 8) return few_g<2, 1, 8, 2>(p, num_sms, st);
    if (int4_few(p.M)) return few_g<2, 2, 4, 3>(p, num_sms, st);
    switch (many_tokens(p.M)) {
        case 32: return many_g<32>(x, p, num_sms, st);
        case 64: return many_g<64>(x, p, num_sms, st);
        case 128: return many_g<128>(x, p, num_sms, st);
        default: return many_g<256>(x, p, num_sms, st);
    }
}

// CTAs that report: as many as there are places at most
int int4_max_ctas(int num_sms) { return 2 * num_sms; }

}  // namespace moe
