// linear.cu -- dense product of quantised activations and weights (moe_linear_forward):
//   out[m, n] = bf16(xs[m] ws sum_k x[m, k] W[n, k]),  xs, ws only for NVFP4
// with the block scales applied by the block-scaled tcgen05 MMAs and fp32 accumulators in
// tensor memory. A persistent CTA per SM computes 128 x 256 tiles: warp 0 feeds a ring of
// K stages (128 bytes of codes of each row, and their scale atoms) by TMA, one thread of warp 1
// issues the scale copies and MMAs, 16 warps store the accumulators. Every wait is bounded.
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace moe {

template <int FMT>
struct LinCfg {
    static constexpr int S = fmt_sf_atoms(FMT);
    static constexpr int BN = 256;
    static constexpr int NB = BN / NBLK;
    static constexpr int STAGES = 4;
    static constexpr int A_BYTES = BM * BK_BYTES;
    static constexpr int B_BYTES = BN * BK_BYTES;
    static constexpr int SFA_BYTES = S * ATOM_BYTES;
    static constexpr int SFB_BYTES = S * NB * ATOM_BYTES;
    static constexpr uint32_t TX_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGE_BYTES = (TX_BYTES + 1023) / 1024 * 1024;
    static constexpr int ACC_COLS = BN;
    static constexpr int SF_COLS = 4 * S * (1 + NB);
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM = STAGES * STAGE_BYTES + BAR_BYTES + 1024;
    static_assert(ACC_COLS + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int FMT>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const LinearArgs p) {
    using C = LinCfg<FMT>;
    constexpr int S = C::S, NB = C::NB, STAGES = C::STAGES, BN = C::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* never = reinterpret_cast<int*>(tmem_slot + 2);  // stays 0: drains ignore the abort flag

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t tfull_bar = bar0 + 8 * (2 * STAGES);
    const uint32_t tempty_bar = tfull_bar + 8;
    const uint32_t drain_bar = tfull_bar + 16;
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * STAGES; ++s) mbar_init(bar0 + 8 * s, 1);
        mbar_init(tfull_bar, 1);
        mbar_init(tempty_bar, EPI_WARPS);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_wait();
    grid_dep_launch();

    const int m_tiles = (p.M + BM - 1) / BM, n_tiles = (p.N + BN - 1) / BN;
    const int total = m_tiles * n_tiles;
    auto give_up = [&]() {
        set_error(p.err, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int last_parity[STAGES];
#pragma unroll
            for (int s = 0; s < STAGES; ++s) last_parity[s] = -1;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const int mt = tile % m_tiles, nt = tile / m_tiles;
                for (int ks = 0; ks < p.nks; ++ks) {
                    const uint32_t full = bar0 + 8 * stage, empty = bar0 + 8 * (STAGES + stage);
                    if (!mbar_wait(empty, phase ^ 1, tmo, abort_flag)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem_u32(smem + stage * C::STAGE_BYTES);
                    mbar_arrive_expect_tx(full, C::TX_BYTES);
                    tma_load_2d(st, &tmA, full, ks * BK_BYTES, mt * BM);
                    tma_load_2d(st + C::A_BYTES, &tmB, full, ks * BK_BYTES, nt * BN);
                    bulk_load(st + C::A_BYTES + C::B_BYTES, p.sfa + ((int64_t)mt * p.nks + ks) * C::SFA_BYTES,
                              C::SFA_BYTES, full);
                    bulk_load(st + C::A_BYTES + C::B_BYTES + C::SFA_BYTES,
                              p.sfb + ((int64_t)ks * p.sf_blocks + (int64_t)nt * NB) * S * ATOM_BYTES, C::SFB_BYTES,
                              full);
                    last_parity[stage] = (int)phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // every load this thread issued lands before the CTA may exit
            for (int s = 0; s < STAGES; ++s)
                if (last_parity[s] >= 0) mbar_wait(bar0 + 8 * s, (uint32_t)last_parity[s], DRAIN_TIMEOUT_NS, never);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                if (!mbar_wait(tempty_bar, acc_phase ^ 1, tmo, abort_flag)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                for (int ks = 0; ks < p.nks; ++ks) {
                    const uint32_t full = bar0 + 8 * stage, empty = bar0 + 8 * (STAGES + stage);
                    if (!mbar_wait(full, phase, tmo, abort_flag)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + stage * C::STAGE_BYTES);
                    const uint32_t sfa_col = tmem_base + C::ACC_COLS + stage * C::SF_COLS;
                    const uint32_t sfb_col = sfa_col + 4 * S;
                    const uint32_t sfa_smem = st + C::A_BYTES + C::B_BYTES;
#pragma unroll
                    for (int a = 0; a < S; ++a) tc_cp_sf_atom(sfa_col + 4 * a, sf_atom_desc(sfa_smem + a * ATOM_BYTES));
                    // smem holds the weight atoms as [block][s]; tensor memory wants [s][block]
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int a = 0; a < S; ++a)
                            tc_cp_sf_atom(sfb_col + 4 * (a * NB + nb),
                                          sf_atom_desc(sfa_smem + C::SFA_BYTES + (nb * S + a) * ATOM_BYTES));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t ad = kmajor_sw128_desc(st + j * 32);
                        const uint64_t bd = kmajor_sw128_desc(st + C::A_BYTES + j * 32);
                        const uint32_t accumulate = (ks > 0 || j > 0) ? 1u : 0u;
                        if constexpr (FMT == MOE_FMT_MXFP4)
                            mma_mxf4(tmem_base, ad, bd, idesc_mxf4(BN, 2u * (j & 1)), sfa_col + 4 * (j >> 1),
                                     sfb_col + 4 * NB * (j >> 1), accumulate);
                        else if constexpr (FMT == MOE_FMT_MXFP8)
                            mma_mxf8(tmem_base, ad, bd, idesc_mxf8(BN, j), sfa_col, sfb_col, accumulate);
                        else
                            mma_nvf4(tmem_base, ad, bd, idesc_nvf4(BN), sfa_col + 4 * j, sfb_col + 4 * NB * j,
                                     accumulate);
                    }
                    tc_commit(empty);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit(tfull_bar);
                acc_phase ^= 1;
            }
            // every MMA and copy this thread issued completes before tensor memory is freed
            tc_commit(drain_bar);
            mbar_wait(drain_bar, 0, DRAIN_TIMEOUT_NS, never);
        }
    } else {
        const int q = warp % 4;           // the lane quarter of tensor memory this warp may read
        const int cg = (warp - 2) / 4;    // its 64 columns of the tile
        uint32_t acc_phase = 0;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
            const int mt = tile % m_tiles, nt = tile / m_tiles;
            // warp-uniform: every lane leaves together (a lane left behind would block in __syncwarp)
            if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar, acc_phase, tmo, abort_flag))) {
                give_up();
                break;
            }
            tc_fence_after();
            const int row = mt * BM + q * 32 + lane, col = nt * BN + cg * 64;
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + cg * 64;
            float v[2][32];
            tmem_ld32(tacc, v[0]);
            tmem_ld32(tacc + 32, v[1]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar);  // the accumulator sits in registers
            if (row < p.M) {
                float alpha = 1.0f;
                if constexpr (FMT == MOE_FMT_NVFP4) alpha = p.x_scale[row] * *p.w_scale;
                __nv_bfloat16* o = p.out + (int64_t)row * p.ldo + col;
                const bool vec = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c0 = col + 32 * h + 8 * g;
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = v[h][8 * g + j] * alpha;
                        if (vec && c0 + 8 <= p.N) {
                            *reinterpret_cast<uint4*>(o + 32 * h + 8 * g) = pack_bf16x8_rn(f);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (c0 + j < p.N) o[32 * h + 8 * g + j] = __float2bfloat16_rn(f[j]);
                        }
                    }
            }
            acc_phase ^= 1;
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// weight scales into atoms: one thread per destination byte
__global__ void pack_linear_sf_kernel(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int64_t total, int S,
                                      int64_t blocks, int N, int nkb) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= total) return;
    const int in_atom = (int)(idx % ATOM_BYTES);
    const int64_t atom = idx / ATOM_BYTES;
    const int s = (int)(atom % S);
    const int64_t nb = atom / S % blocks, ks = atom / S / blocks;
    const int64_t n = nb * NBLK + (in_atom % 16) / 4 * 32 + in_atom / 16;
    const int64_t kb = ks * 4 * S + s * 4 + in_atom % 4;
    dst[idx] = n < N && kb < nkb ? src[n * nkb + kb] : 0;
}

cudaError_t launch_pack_linear_sf(const uint8_t* src, uint8_t* dst, int fmt, int N, int K, cudaStream_t st) {
    const int S = fmt_sf_atoms(fmt);
    const int64_t blocks = wt_sf_blocks(N), nks = ceil_div(fmt_row_bytes(fmt, K), BK_BYTES);
    const int64_t total = nks * blocks * S * ATOM_BYTES;
    pack_linear_sf_kernel<<<(unsigned)ceil_div(total, 256), 256, 0, st>>>(src, dst, total, S, blocks, N,
                                                                         K / fmt_sf_block(fmt));
    return cudaGetLastError();
}

// ------------------------------------------------------------------ host side
template <int FMT>
static cudaError_t lin_attr() {
    return cudaFuncSetAttribute(linear_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, LinCfg<FMT>::SMEM);
}
cudaError_t linear_prepare(int fmt) {
    switch (fmt) {
        case MOE_FMT_MXFP8: return lin_attr<MOE_FMT_MXFP8>();
        case MOE_FMT_MXFP4: return lin_attr<MOE_FMT_MXFP4>();
        default: return lin_attr<MOE_FMT_NVFP4>();
    }
}

template <int FMT>
static cudaError_t lin_t(const CUtensorMap& a, const CUtensorMap& b, const LinearArgs& p, int num_sms,
                         cudaStream_t st, bool pdl) {
    LaunchAttrs at(pdl);
    const int64_t tiles = ceil_div(p.M, BM) * ceil_div(p.N, LinCfg<FMT>::BN);
    const int grid = (int)(tiles < num_sms ? tiles : num_sms);
    cudaLaunchConfig_t cfg = at.config(dim3(grid), dim3(GEMM_THREADS), LinCfg<FMT>::SMEM, st);
    return cudaLaunchKernelEx(&cfg, linear_kernel<FMT>, a, b, p);
}
cudaError_t launch_linear(int fmt, const CUtensorMap& a, const CUtensorMap& b, const LinearArgs& p, int num_sms,
                          cudaStream_t st, bool pdl) {
    switch (fmt) {
        case MOE_FMT_MXFP8: return lin_t<MOE_FMT_MXFP8>(a, b, p, num_sms, st, pdl);
        case MOE_FMT_MXFP4: return lin_t<MOE_FMT_MXFP4>(a, b, p, num_sms, st, pdl);
        default: return lin_t<MOE_FMT_NVFP4>(a, b, p, num_sms, st, pdl);
    }
}

}  // namespace moe
