// linear.cu -- dense product of quantised activations and weights (moe_linear_forward):
//   out[m, n] = bf16(xs[m] ws sum_k x[m, k] W[n, k]),  xs, ws only for NVFP4
// with the block scales applied by the block-scaled tcgen05 MMAs and fp32 accumulators in
// tensor memory. Both kernels put the weights on the MMA's row side and the tokens on its
// column side, so an accumulator lane is an output feature and a column a token: a warp's 32
// lanes store 32 neighbouring features of one token, coalesced whatever N and the stride are.
//
//   linear_pair_kernel   many tiles: persistent CTA pairs (cta_group::2), 256 features x 256
//                        tokens a tile, each CTA staging its 128 weight rows and half of the
//                        tokens
//   linear_split_kernel  few tiles (decode, small layers): 128 features x 16 .. 128 tokens a tile,
//                        K split over the CTAs of a cluster, which add their accumulators
//                        through distributed shared memory in rank order
//
// A K stage is 128 bytes of codes of each row with their scale atoms. Every wait is bounded;
// a CTA that gives up reports MOE_ERR_TIMEOUT and still waits for its own copies and MMAs.
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace moe {

// ------------------------------------------------------------------ shared pieces
// The bounded waits. Short limits are counted in polls of some 16 ns each, so that a limit of a
// nanosecond is one poll.
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int* abort) {
    if (timeout_ns >= SHORT_WAIT_NS) return mbar_wait(bar, parity, timeout_ns, abort);
    for (uint64_t i = 0; i <= timeout_ns / 16; ++i)
        if (mbar_test_wait(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ bool lin_wait_cl(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                            const volatile int* abort) {
    if (timeout_ns >= SHORT_WAIT_NS) return mbar_wait_cl(bar, parity, timeout_ns, abort);
    for (uint64_t i = 0; i <= timeout_ns / 16; ++i)
        if (mbar_test_wait_cl(bar, parity)) return true;
    return false;
}

// One lane of the warp, always the same. The producer and MMA warps run their loops with all
// lanes and predicate only the copies and MMAs with this: the loop's addresses and descriptors
// then stay in uniform registers. (A loop that one thread runs alone moves every operand there
// for each instruction: measured, 4 MMAs and 12 scale copies took 1085 cycles to issue that way
// and 408 this way, against 512 that the MMAs need.)
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// a wait of the whole warp: every lane returns the same
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int* abort) {
    return __all_sync(0xffffffffu, lin_wait(bar, parity, timeout_ns, abort));
}
__device__ __forceinline__ bool warp_wait_cl(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                             const volatile int* abort) {
    return __all_sync(0xffffffffu, lin_wait_cl(bar, parity, timeout_ns, abort));
}

// One 32-byte K step of a stage: j-th of 4.
template <int FMT, int GROUP>
__device__ __forceinline__ void lin_mma(uint32_t d, uint64_t ad, uint64_t bd, int n, int j, uint32_t sfa, uint32_t sfb,
                                        int sfb_blocks, uint32_t accumulate) {
    uint32_t id, ca, cb;
    if constexpr (FMT == MOE_FMT_MXFP4) {
        id = idesc_mxf4(n, 2u * (j & 1)), ca = sfa + 4 * (j >> 1), cb = sfb + 4 * sfb_blocks * (j >> 1);
    } else if constexpr (FMT == MOE_FMT_MXFP8) {
        id = idesc_mxf8(n, j), ca = sfa, cb = sfb;
    } else {
        id = idesc_nvf4(n), ca = sfa + 4 * j, cb = sfb + 4 * sfb_blocks * j;
    }
    if constexpr (GROUP == 2) {
        id = idesc_m(id, 2 * BM);
        if constexpr (FMT == MOE_FMT_MXFP4)
            mma2_mxf4(d, ad, bd, id, ca, cb, accumulate);
        else if constexpr (FMT == MOE_FMT_MXFP8)
            mma2_mxf8(d, ad, bd, id, ca, cb, accumulate);
        else
            mma2_nvf4(d, ad, bd, id, ca, cb, accumulate);
    } else {
        if constexpr (FMT == MOE_FMT_MXFP4)
            mma_mxf4(d, ad, bd, id, ca, cb, accumulate);
        else if constexpr (FMT == MOE_FMT_MXFP8)
            mma_mxf8(d, ad, bd, id, ca, cb, accumulate);
        else
            mma_nvf4(d, ad, bd, id, ca, cb, accumulate);
    }
}

// ------------------------------------------------------------------ CTA pairs
template <int FMT>
struct PairCfg {
    static constexpr int S = fmt_sf_atoms(FMT);
    static constexpr int BT = 256;                         // tokens of a tile
    static constexpr int NB = BT / NBLK;
    static constexpr int THREADS = GEMM_THREADS;
    static constexpr int STAGES = FMT == MOE_FMT_NVFP4 ? 5 : 6;
    static constexpr int A_BYTES = BM * BK_BYTES;         // this CTA's 128 weight rows
    static constexpr int B_BYTES = NBLK * BK_BYTES;       // this CTA's half of the tokens
    static constexpr int SFA_BYTES = S * ATOM_BYTES;
    static constexpr int SFB_BYTES = S * NB * ATOM_BYTES;  // both halves: each CTA's MMA half needs them
    static constexpr uint32_t TX_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGE_BYTES = (TX_BYTES + 1023) / 1024 * 1024;
    static constexpr int ACC_COLS = BT;
    static constexpr int SF_COLS = 4 * S * (1 + NB);
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM = STAGES * STAGE_BYTES + BAR_BYTES + 1024;
    // barriers: full, empty [STAGES]; tfull, tempty, drain, teardown
    static constexpr int NUM_BARS = 2 * STAGES + 4;
    static_assert(NUM_BARS * 8 + 16 <= BAR_BYTES, "barrier area");
    static_assert(ACC_COLS + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

// Tiles in groups of GROUP weight tiles, the tokens inside a group: the clusters that run at the
// same time share few weight and token tiles.
constexpr int RASTER_GROUP = 8;
__device__ __forceinline__ void raster(int tile, int n_tiles, int t_tiles, int& nt, int& tt) {
    const int per = RASTER_GROUP * t_tiles, g = tile / per, rest = tile - g * per;
    const int width = min(RASTER_GROUP, n_tiles - g * RASTER_GROUP);
    nt = g * RASTER_GROUP + rest % width;
    tt = rest / width;
}

template <int FMT>
__global__ void __launch_bounds__(PairCfg<FMT>::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmSFW, const __grid_constant__ CUtensorMap tmSFX,
                       const LinearArgs p) {
    using C = PairCfg<FMT>;
    constexpr int S = C::S, NB = C::NB, STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* never = reinterpret_cast<int*>(tmem_slot + 2);
    volatile uint32_t* peer_issued = tmem_slot + 3;  // leader: stages the follower's producer issued

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, tfull_bar = empty0 + 8 * STAGES,
                   tempty_bar = tfull_bar + 8, drain_bar = tfull_bar + 16, teardown_bar = tfull_bar + 24;
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, leader ? 2 : 1);  // full (the leader's counts): both producers arrive
            mbar_init(empty0 + 8 * s, 1);              // empty: the leader's commit
        }
        mbar_init(tfull_bar, 1);
        mbar_init(tempty_bar, leader ? 2 * EPI_WARPS : EPI_WARPS);
        mbar_init(drain_bar, 1);
        mbar_init(teardown_bar, 1);
        *abort_flag = 0;
        *peer_issued = 0;
        *never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmSFW);
        prefetch_tmap(&tmSFX);
    }
    if (warp == 1) {
        tmem_alloc2(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before anyone arrives on them
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_wait();  // the set-up above overlaps the previous kernel; everything below reads its output
    grid_dep_launch();

    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int n_tiles = (p.N + 255) / 256, t_tiles = (p.M + C::BT - 1) / C::BT;
    const int total = n_tiles * t_tiles;

    auto give_up = [&]() {
        set_error(p.err, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // Both CTAs count their bytes on the leader's full barrier: each arrives on it with its own
        // transaction count (the follower remotely), and its loads complete on it (cta_group::2).
        const bool elected = elect_one();
        const uint32_t full_cl0 = mapa_shared(full0, 0);
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        for (int tile = pair; ok && tile < total; tile += npairs) {
            int nt, tt;
            raster(tile, n_tiles, t_tiles, nt, tt);
            const int w_blk = 2 * nt + (int)rank, x_blk = 2 * tt + (int)rank;  // this CTA's 128-row blocks
            for (int ks = 0; ks < p.nks; ++ks) {
                if (!warp_wait(empty0 + 8 * stage, phase ^ 1, tmo, abort_flag)) {
                    give_up();
                    ok = false;
                    break;
                }
                const uint32_t st = smem0 + stage * C::STAGE_BYTES, sf = st + C::A_BYTES + C::B_BYTES;
                const uint32_t full_cl = full_cl0 + 8 * stage;
                if (elected) {
                    if (leader)
                        mbar_arrive_expect_tx(full0 + 8 * stage, C::TX_BYTES);
                    else
                        mbar_arrive_expect_tx_cluster(full_cl, C::TX_BYTES);
                    tma_load_2d_cg2(st, &tmW, full_cl, ks * BK_BYTES, w_blk * BM);
                    tma_load_2d_cg2(st + C::A_BYTES, &tmX, full_cl, ks * BK_BYTES, x_blk * NBLK);
                    tma_load_2d_cg2(sf, &tmSFW, full_cl, 0, (ks * p.sf_blocks + w_blk) * S);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        tma_load_2d_cg2(sf + (1 + b) * C::SFA_BYTES, &tmSFX, full_cl, 0,
                                        ((NB * tt + b) * p.nks + ks) * S);
                }
                __syncwarp();
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // Every load either CTA issued lands before the pair may exit. The follower reports its
        // count to the leader; for a stage only one CTA issued (one of them gave up), the
        // leader supplies the missing arrival, so that the stage's phase completes once the
        // issued bytes have landed. A producer can run at most STAGES stages ahead of the other
        // one (a slot is reused only after the MMA consumed it, which needs both arrivals), so
        // each slot is touched once.
        if (elected) {
            if (!leader) {
                st_cluster_u32(mapa_shared(smem_u32((const void*)peer_issued), 0), issued);
                mbar_arrive_release_cluster(mapa_shared(teardown_bar, 0));
            } else {
                uint32_t other = issued;
                if (mbar_wait_cl(teardown_bar, 0, DRAIN_TIMEOUT_NS, never)) other = *peer_issued;
                const uint32_t lo = min(issued, other), hi = max(issued, other);
                for (uint32_t n = lo; n < hi; ++n) mbar_arrive(full0 + 8 * (n % STAGES));
                for (uint32_t s = 0; s < (uint32_t)STAGES && s < hi; ++s) {
                    const uint32_t last = s + (hi - 1 - s) / STAGES * STAGES;  // last stage n < hi in slot s
                    mbar_wait(full0 + 8 * s, (last / STAGES) & 1u, DRAIN_TIMEOUT_NS, never);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const bool elected = elect_one();
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued = false;
            for (int tile = pair; ok && tile < total; tile += npairs) {
                if (!warp_wait_cl(tempty_bar, acc_phase ^ 1, tmo, abort_flag)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                for (int ks = 0; ks < p.nks; ++ks) {
                    if (!warp_wait_cl(full0 + 8 * stage, phase, tmo, abort_flag)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem0 + stage * C::STAGE_BYTES, sf = st + C::A_BYTES + C::B_BYTES;
                    const uint32_t sfa_col = tmem_base + C::ACC_COLS + stage * C::SF_COLS;
                    const uint32_t sfb_col = sfa_col + 4 * S;
                    if (elected) {
#pragma unroll
                        for (int a = 0; a < S; ++a) tc_cp2_sf_atom(sfa_col + 4 * a, sf_atom_desc(sf + a * ATOM_BYTES));
                        // shared memory holds the token atoms as [block][s]; tensor memory wants [s][block]
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int a = 0; a < S; ++a)
                                tc_cp2_sf_atom(sfb_col + 4 * (a * NB + b),
                                               sf_atom_desc(sf + C::SFA_BYTES + (b * S + a) * ATOM_BYTES));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            lin_mma<FMT, 2>(tmem_base, kmajor_sw128_desc(st + j * 32),
                                            kmajor_sw128_desc(st + C::A_BYTES + j * 32), C::BT, j, sfa_col, sfb_col, NB,
                                            (ks > 0 || j > 0) ? 1u : 0u);
                        tc_commit2_mc(empty0 + 8 * stage, 0x3);
                    }
                    __syncwarp();
                    issued = true;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elected) tc_commit2_mc(tfull_bar, 0x3);
                __syncwarp();
                acc_phase ^= 1;
            }
            // every MMA and copy issued completes before either CTA frees its tensor memory
            if (issued) {
                if (elected) tc_commit2_mc(drain_bar, 0x1);
                __syncwarp();
                mbar_wait(drain_bar, 0, DRAIN_TIMEOUT_NS, never);
            }
        }
    } else {
        const int q = warp % 4;         // the lane quarter of tensor memory this warp may read
        const int cg = (warp - 2) / 4;  // its 64 tokens of the tile
        const uint32_t leader_tempty = mapa_shared(tempty_bar, 0);
        uint32_t acc_phase = 0;
        for (int tile = pair; tile < total; tile += npairs) {
            // warp-uniform: every lane leaves together (a lane left behind would block in __syncwarp)
            if (!__all_sync(0xffffffffu, lin_wait(tfull_bar, acc_phase, tmo, abort_flag))) {
                give_up();
                break;
            }
            tc_fence_after();
            int nt, tt;
            raster(tile, n_tiles, t_tiles, nt, tt);
            const int n = nt * 256 + (int)rank * BM + q * 32 + lane, t0 = tt * C::BT + cg * 64;
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + cg * 64;
            float v[2][32];
            tmem_ld32(tacc, v[0]);
            tmem_ld32(tacc + 32, v[1]);
            tmem_ld_wait();
            // hand the accumulator back as soon as it sits in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    mbar_arrive(tempty_bar);
                else
                    mbar_arrive_cluster(leader_tempty);
            }
            acc_phase ^= 1;
            if (n < p.N) {
                float ws = 1.0f;
                if constexpr (FMT == MOE_FMT_NVFP4) ws = __ldg(p.w_scale);
                __nv_bfloat16* o = p.out + (int64_t)t0 * p.ldo + n;
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    if (t0 + j < p.M) {
                        float y = v[j / 32][j % 32];
                        if constexpr (FMT == MOE_FMT_NVFP4) y *= __ldg(p.x_scale + t0 + j) * ws;
                        *o = __float2bfloat16_rn(y);
                    }
                    o += p.ldo;
                }
            }
        }
    }
    __syncthreads();
    cluster_sync();  // both CTAs are done with each other's barriers and the MMAs have drained
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ clusters that split K
constexpr int MAX_SPLITS = 8;  // the portable cluster size

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int FMT, int BT>
struct SplitCfg {
    static constexpr int S = fmt_sf_atoms(FMT);
    static constexpr int STAGES = BT <= 32 || (BT <= 64 && S < 4) ? 4 : 3;  // two CTAs fit on an SM
    static constexpr int EPI = 4;                     // epilogue warps, one for each lane quarter
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int A_BYTES = BM * BK_BYTES;
    static constexpr int B_BYTES = BT * BK_BYTES;
    static constexpr int SF_BYTES = S * ATOM_BYTES;    // of either side
    static constexpr uint32_t TX_BYTES = A_BYTES + B_BYTES + 2 * SF_BYTES;
    static constexpr int STAGE_BYTES = (TX_BYTES + 1023) / 1024 * 1024;
    static constexpr int SF_COLS = 8 * S;
    static constexpr int COLS = BT + STAGES * SF_COLS;
    static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM = STAGES * STAGE_BYTES + BAR_BYTES + 1024;
    static_assert(COLS <= 256, "tensor memory budget of two CTAs");
    static_assert(2 * (SMEM + 1024) <= 233472, "shared memory budget of two CTAs");
    static_assert(STAGES * STAGE_BYTES >= BT * BM * 4, "the ring holds the partial sums");
};

template <int FMT, int BT>
__global__ void __launch_bounds__(SplitCfg<FMT, BT>::THREADS, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const LinearArgs p) {
    using C = SplitCfg<FMT, BT>;
    constexpr int S = C::S, STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* never = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, done_bar = empty0 + 8 * STAGES;
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t tmo = p.timeout_ns;
    // grid.x = splits (one cluster), grid.y = weight tiles, grid.z = token tiles
    const uint32_t splits = gridDim.x, rank = blockIdx.x;
    const int nt = blockIdx.y, tt = blockIdx.z;
    const int k0 = (int)((int64_t)p.nks * rank / splits), k1 = (int)((int64_t)p.nks * (rank + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * STAGES; ++s) mbar_init(full0 + 8 * s, 1);
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    auto give_up = [&]() {
        set_error(p.err, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
    };

    bool complete = true;  // meaningful in the epilogue's warps
    if (warp == 0) {
        const bool elected = elect_one();
        auto load_w = [&](int ks, int stage) {
            const uint32_t st = smem0 + stage * C::STAGE_BYTES, full = full0 + 8 * stage;
            mbar_arrive_expect_tx(full, C::TX_BYTES);
            tma_load_2d(st, &tmW, full, ks * BK_BYTES, nt * BM);
            bulk_load(st + C::A_BYTES + C::B_BYTES, p.sfb + ((int64_t)ks * p.sf_blocks + nt) * C::SF_BYTES, C::SF_BYTES,
                      full);
        };
        auto load_x = [&](int ks, int stage) {
            const uint32_t st = smem0 + stage * C::STAGE_BYTES, full = full0 + 8 * stage;
            tma_load_2d(st + C::A_BYTES, &tmX, full, ks * BK_BYTES, tt * BT);
            // token tiles start at multiples of 128 rows, or there is only one
            bulk_load(st + C::A_BYTES + C::B_BYTES + C::SF_BYTES,
                      p.sfa + ((int64_t)(tt * BT / BM) * p.nks + ks) * C::SF_BYTES, C::SF_BYTES, full);
        };
        // The weights do not depend on the previous kernel (the quantisation of x): the first
        // stages' weights are on their way before the wait for it.
        const int ahead = min(k1 - k0, STAGES);
        if (elected)
            for (int i = 0; i < ahead; ++i) load_w(k0 + i, i);
        grid_dep_wait();
        grid_dep_launch();
        if (elected)
            for (int i = 0; i < ahead; ++i) load_x(k0 + i, i);
        __syncwarp();
        int issued = ahead;
        for (; issued < k1 - k0; ++issued) {
            const int stage = issued % STAGES;
            if (!warp_wait(empty0 + 8 * stage, ((issued / STAGES) & 1) ^ 1, tmo, abort_flag)) {
                give_up();
                break;
            }
            if (elected) {
                load_w(k0 + issued, stage);
                load_x(k0 + issued, stage);
            }
            __syncwarp();
        }
        // every load issued lands before the CTA may exit or reuse the ring
        for (int s = 0; s < STAGES && s < issued; ++s) {
            const int last = s + (issued - 1 - s) / STAGES * STAGES;
            mbar_wait(full0 + 8 * s, (last / STAGES) & 1, DRAIN_TIMEOUT_NS, never);
        }
    } else if (warp == 1) {
        const bool elected = elect_one();
        grid_dep_wait();
        for (int i = 0; i < k1 - k0; ++i) {
            const int stage = i % STAGES;
            if (!warp_wait(full0 + 8 * stage, (i / STAGES) & 1, tmo, abort_flag)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t st = smem0 + stage * C::STAGE_BYTES, sf = st + C::A_BYTES + C::B_BYTES;
            const uint32_t sfa_col = tmem_base + BT + stage * C::SF_COLS, sfb_col = sfa_col + 4 * S;
            if (elected) {
#pragma unroll
                for (int a = 0; a < 2 * S; ++a) tc_cp_sf_atom(sfa_col + 4 * a, sf_atom_desc(sf + a * ATOM_BYTES));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    lin_mma<FMT, 1>(tmem_base, kmajor_sw128_desc(st + j * 32),
                                    kmajor_sw128_desc(st + C::A_BYTES + j * 32), BT, j, sfa_col, sfb_col, 1,
                                    (i > 0 || j > 0) ? 1u : 0u);
                tc_commit(empty0 + 8 * stage);
            }
            __syncwarp();
        }
        // every MMA and copy issued has completed; also the epilogue's signal
        if (elected) tc_commit(done_bar);
        __syncwarp();
        mbar_wait(done_bar, 0, DRAIN_TIMEOUT_NS, never);
    } else {
        grid_dep_wait();
        complete = __all_sync(0xffffffffu, lin_wait(done_bar, 0, tmo, abort_flag));
        if (!complete) give_up();
        tc_fence_after();
    }
    // partial sums [token][128 features] into the ring, which no copy or MMA uses any more
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
    const int tokens = min(BT, p.M - tt * BT);
    if (warp >= 2) {
        const int q = warp % 4;
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
        for (int c0 = 0; c0 < tokens; c0 += 32) {
            float v[32];
            tmem_ld32(tacc + c0, v);  // for BT = 16 the upper columns hold scales: not kept
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c0 + j < BT) part[(c0 + j) * BM + q * 32 + lane] = v[j];
        }
        tc_fence_before();
    }
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    // The CTA of rank r adds the tokens r, r + splits, ... in rank order: a warp takes a token, a
    // lane 4 features, with the loads of all ranks in flight.
    if (warp >= 2 && complete) {
        const int n = nt * BM + 4 * lane;
        float ws = 1.0f;
        if constexpr (FMT == MOE_FMT_NVFP4) ws = __ldg(p.w_scale);
        for (int c = (int)(rank + splits * (warp - 2)); c < tokens; c += (int)splits * C::EPI) {
            const uint32_t at = smem_u32(part + c * BM + 4 * lane);
            float4 u[MAX_SPLITS];
#pragma unroll
            for (int r = 0; r < MAX_SPLITS; ++r) {
                u[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (r < (int)splits) u[r] = ld_cluster_f32x4(mapa_shared(at, r));
            }
            float4 y = u[0];
#pragma unroll
            for (int r = 1; r < MAX_SPLITS; ++r) y.x += u[r].x, y.y += u[r].y, y.z += u[r].z, y.w += u[r].w;
            const int t = tt * BT + c;
            if constexpr (FMT == MOE_FMT_NVFP4) {
                const float alpha = p.x_scale[t] * ws;
                y.x *= alpha, y.y *= alpha, y.z *= alpha, y.w *= alpha;
            }
            __nv_bfloat16* o = p.out + (int64_t)t * p.ldo + n;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
            if (n + 4 <= p.N && (reinterpret_cast<uintptr_t>(o) & 7) == 0) {
                *reinterpret_cast<uint2*>(o) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
                if (n < p.N) o[0] = lo.x;
                if (n + 1 < p.N) o[1] = lo.y;
                if (n + 2 < p.N) o[2] = hi.x;
                if (n + 3 < p.N) o[3] = hi.y;
            }
        }
    }
    if (splits > 1)
        cluster_sync();  // no CTA leaves while its sums are read
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM);
    }
}

// ------------------------------------------------------------------ weight scales
// one thread per destination byte
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
#ifndef LIN_PAIR_TILES
#define LIN_PAIR_TILES 76
#endif
#ifndef LIN_CTAS
#define LIN_CTAS 304
#endif
LinearShape linear_shape(int M, int N, int nks) {
    LinearShape s{};
    const int64_t pair_tiles = ceil_div(M, 256) * ceil_div(N, 256);
    if (M > 128 && pair_tiles >= LIN_PAIR_TILES) return s;
    s.bt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t tiles = ceil_div(M, s.bt) * ceil_div(N, BM);
    s.splits = 1;
    while (s.splits < MAX_SPLITS && tiles * s.splits * 2 <= LIN_CTAS && nks >= s.splits * 2) s.splits *= 2;
    return s;
}

template <int FMT, int BT>
static cudaError_t split_attr() {
    return cudaFuncSetAttribute(linear_split_kernel<FMT, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SplitCfg<FMT, BT>::SMEM);
}
template <int FMT>
static cudaError_t lin_attr() {
    cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PairCfg<FMT>::SMEM);
    if (e == cudaSuccess) e = split_attr<FMT, 16>();
    if (e == cudaSuccess) e = split_attr<FMT, 32>();
    if (e == cudaSuccess) e = split_attr<FMT, 64>();
    if (e == cudaSuccess) e = split_attr<FMT, 128>();
    return e;
}
cudaError_t linear_prepare(int fmt) {
    switch (fmt) {
        case MOE_FMT_MXFP8: return lin_attr<MOE_FMT_MXFP8>();
        case MOE_FMT_MXFP4: return lin_attr<MOE_FMT_MXFP4>();
        default: return lin_attr<MOE_FMT_NVFP4>();
    }
}

template <int FMT, int BT>
static cudaError_t split_t(const LinearMaps& m, const LinearArgs& p, int splits, cudaStream_t st) {
    using C = SplitCfg<FMT, BT>;
    LaunchAttrs at(true, splits);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)splits, (unsigned)ceil_div(p.N, BM), (unsigned)ceil_div(p.M, BT)),
                                       dim3(C::THREADS), C::SMEM, st);
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<FMT, BT>, m.w, m.x, p);
}

template <int FMT>
static cudaError_t lin_t(const LinearMaps& m, const LinearArgs& p, const LinearShape& s, int num_sms, cudaStream_t st) {
    switch (s.bt) {
        case 16: return split_t<FMT, 16>(m, p, s.splits, st);
        case 32: return split_t<FMT, 32>(m, p, s.splits, st);
        case 64: return split_t<FMT, 64>(m, p, s.splits, st);
        case 128: return split_t<FMT, 128>(m, p, s.splits, st);
        default: break;
    }
    LaunchAttrs at(true, 2);
    const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256), pairs = num_sms / 2;
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))),
                                       dim3(PairCfg<FMT>::THREADS), PairCfg<FMT>::SMEM, st);
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<FMT>, m.w, m.x, m.sfw, m.sfx, p);
}
cudaError_t launch_linear(int fmt, const LinearMaps& m, const LinearArgs& p, const LinearShape& s, int num_sms,
                          cudaStream_t st) {
    switch (fmt) {
        case MOE_FMT_MXFP8: return lin_t<MOE_FMT_MXFP8>(m, p, s, num_sms, st);
        case MOE_FMT_MXFP4: return lin_t<MOE_FMT_MXFP4>(m, p, s, num_sms, st);
        default: return lin_t<MOE_FMT_NVFP4>(m, p, s, num_sms, st);
    }
}

}  // namespace moe
