// linear.cu -- dense product of quantised activations and weights (moe_linear_forward):
//   out[m, n] = bf16(xs[m] ws sum_k x[m, k] W[n, k]),  xs, ws only for NVFP4
// with the block scales applied by the block-scaled tcgen05 MMAs and fp32 accumulators in
// tensor memory. Both kernels put the weights on the MMA's row side and the tokens on its
// column side, so an accumulator lane is an output feature and a column a token: a warp's 32
// lanes store 32 neighbouring features of one token, coalesced whatever N and the stride are.
//
//   linear_pair_kernel   many tiles: persistent CTA pairs (cta_group::2), 256 features x 256
//                        tokens a tile, each CTA staging its 128 weight rows and half of the
//                        tokens: a third less operand traffic for each SM than single CTAs with
//                        128 x 256 tiles, which L2 could not feed
//   linear_split_kernel  few tiles (decode, small layers): 128 features x 16 .. 128 tokens a tile,
//                        K split over the CTAs of a cluster, which add their accumulators
//                        through distributed shared memory in rank order
//
// A K stage is 128 bytes of codes of each row with their scale atoms: 4 MMAs, 512 cycles of the
// tensor pipe in every format. Every wait is bounded; a CTA that gives up reports
// MOE_ERR_TIMEOUT and still waits for its own copies and MMAs. Each CTA has a status word of its own,
// which it writes whatever happened, so that no word depends on the order in which CTAs run and the
// workspace needs no clearing before the launch.
//
// Measured on GB300: 4096 x 8192 x 4096 MXFP8 in 78 us (3.5 PFLOP/s, twice the chip's sustained bf16
// rate: power-bound; 2.2 PFLOP/s before the issuing loops ran converged), 8192 x 7168 x 7168 NVFP4 in
// 121 us (7.0 PFLOP/s) after 28 us of quantisation; with every operand load taken out it takes 113, the rate
// of the K = 64 MMAs that it issues.
// Where one wave of tiles does it, the fixed steps count: 1024 x 4096 x 4096 NVFP4 9.9 us, of which 0.8
// until the first stage has landed, 0.3 for each of 16 stages (the MMAs alone 0.27), 0.6 until the
// last one is through, 1.6 to store a tile and 0.7 to leave.
// One token through 4096 x 7168 NVFP4: 5.6 us (16.5 MB of weights, 2.4 us at the copy rate), 128
// tokens through 7168 x 4096: 8.8 us, 7.2 from quantised rows. There 1 us goes to set up, 1 us until the
// first stage has landed, 0.24 us to each stage (36 KB, 80 bytes a clock), 1.7 to 2.7 us to the sums of
// split tiles.
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
// One thread of each CTA, after every warp's last wait: status[0] is the number of CTAs, the words
// after it are theirs.
__device__ __forceinline__ void write_status(const LinearArgs& p, uint32_t cta, uint32_t ctas, bool gave_up) {
    if (cta == 0) p.status[0] = (int)ctas;
    p.status[1 + cta] = gave_up ? MOE_ERR_TIMEOUT : MOE_OK;
}
// a wait of the whole warp: every lane returns the same
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int* abort) {
    return __all_sync(0xffffffffu, lin_wait(bar, parity, timeout_ns, abort));
}
__device__ __forceinline__ bool warp_wait_cl(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                             const volatile int* abort) {
    return __all_sync(0xffffffffu, lin_wait_cl(bar, parity, timeout_ns, abort));
}

// What an NVFP4 token's sums are multiplied by, one factor after the other: its scale times the weight's
// and 1. Where that product leaves the normal range though an output need not (rows or weights around
// 2^-100), the significands' product with an exponent that keeps every sum (2^-20 .. 2^40, or zero) in
// range, and the power of two that is left.
__device__ __forceinline__ float2 token_scale(float xs, float ws) {
    const float a = xs * ws;
    if (a >= 0x1p-126f && a <= 0x1.fffffep127f) return make_float2(a, 1.0f);
    if (!(xs > 0.0f && ws > 0.0f) || isinf(xs) || isinf(ws)) return make_float2(a, 1.0f);  // NaN, zero, infinity
    int ex, ew;
    const float m = frexpf(xs, &ex) * frexpf(ws, &ew);
    const int e = ex + ew, first = min(max(e, -100), 80);
    return make_float2(ldexpf(m, first), ldexpf(1.0f, min(e - first, 127)));
}

// Shared-memory descriptors differ only in their low word: the address / 16 (and, for operand rows,
// a leading offset of 1 in bits 16 ..). The high words are those of kmajor_sw128_desc and
// sf_atom_desc.
__device__ __forceinline__ uint64_t row_desc(uint32_t addr16) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | 0x10000u), "n"(0x40004040));
    return d;
}
__device__ __forceinline__ uint64_t atom_desc(uint32_t addr16) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16), "n"(0x4008));
    return d;
}

// The 4 K steps of a stage: rows at a and b (addresses / 16), N columns, scale factors in tensor
// memory at sfa and sfb (of sfb_blocks 128-row blocks). fresh: the first stage of an accumulator.
template <int FMT, int GROUP, int N>
__device__ __forceinline__ void lin_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t sfa, uint32_t sfb,
                                          int sfb_blocks, bool fresh) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t id, ca, cb;
        if constexpr (FMT == MOE_FMT_MXFP4) {
            id = idesc_mxf4(N, 2u * (j & 1)), ca = sfa + 4 * (j >> 1), cb = sfb + 4 * sfb_blocks * (j >> 1);
        } else if constexpr (FMT == MOE_FMT_MXFP8) {
            id = idesc_mxf8(N, j), ca = sfa, cb = sfb;
        } else {
            id = idesc_nvf4(N), ca = sfa + 4 * j, cb = sfb + 4 * sfb_blocks * j;
        }
        const uint64_t ad = row_desc(a + 2 * j), bd = row_desc(b + 2 * j);
        const uint32_t accumulate = j > 0 ? 1u : (fresh ? 0u : 1u);
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
}

// ------------------------------------------------------------------ CTA pairs
template <int FMT>
struct PairCfg {
    static constexpr int S = fmt_sf_atoms(FMT);
    static constexpr int BT = 256;                         // tokens of a tile
    static constexpr int NB = BT / NBLK;                   // 128-token blocks of scale atoms
    static constexpr int THREADS = GEMM_THREADS;
    static constexpr int A_BYTES = BM * BK_BYTES;          // this CTA's 128 weight rows
    static constexpr int B_BYTES = NBLK * BK_BYTES;        // this CTA's half of the tokens
    static constexpr int SFA_BYTES = S * ATOM_BYTES;
    static constexpr int SFB_BYTES = S * NB * ATOM_BYTES;  // both halves: each CTA's MMA half needs them
    static constexpr uint32_t TX_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGE_BYTES = (TX_BYTES + 1023) / 1024 * 1024;
    static constexpr int STAGES = FMT == MOE_FMT_NVFP4 ? 5 : 6;
    static constexpr int BAR_BYTES = 256;
    static constexpr int SF_COLS = 4 * S * (1 + NB);
    static constexpr int SMEM = STAGES * STAGE_BYTES + BAR_BYTES + 1024;
    // barriers: full, empty [STAGES]; tfull, tempty, drain, teardown
    static constexpr int NUM_BARS = 2 * STAGES + 4;
    static_assert(NUM_BARS * 8 + 16 <= BAR_BYTES, "barrier area");
    static_assert(BT + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

// Tiles in groups of 8 weight tiles, the tokens inside a group, so that the clusters that run at
// the same time share few weight and token tiles.
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
    constexpr int S = C::S, NB = C::NB, STAGES = C::STAGES, BT = C::BT;
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

    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int n_tiles = (p.N + 255) / 256, t_tiles = (p.M + BT - 1) / BT;
    const int total = n_tiles * t_tiles;  // at least one for each pair

    // Both CTAs count their bytes on the leader's full barrier: each arrives on it with its own
    // transaction count (the follower remotely), and its loads complete on it (cta_group::2).
    const uint32_t full_cl0 = mapa_shared(full0, 0);
    auto load_w = [&](int nt, int ks, int stage) {
        const uint32_t st = smem0 + stage * C::STAGE_BYTES, full_cl = full_cl0 + 8 * stage;
        const int w_blk = 2 * nt + (int)rank;  // this CTA's 128 weight rows
        if (leader)
            mbar_arrive_expect_tx(full0 + 8 * stage, C::TX_BYTES);
        else
            mbar_arrive_expect_tx_cluster(full_cl, C::TX_BYTES);
        tma_load_2d_cg2(st, &tmW, full_cl, ks * BK_BYTES, w_blk * BM);
        tma_load_2d_cg2(st + C::A_BYTES + C::B_BYTES, &tmSFW, full_cl, 0, (ks * p.sf_blocks + w_blk) * S);
    };
    auto load_x = [&](int tt, int ks, int stage) {
        const uint32_t st = smem0 + stage * C::STAGE_BYTES + C::A_BYTES, sf = st + C::B_BYTES + C::SFA_BYTES;
        const uint32_t full_cl = full_cl0 + 8 * stage;
        tma_load_2d_cg2(st, &tmX, full_cl, ks * BK_BYTES, (2 * tt + (int)rank) * NBLK);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            tma_load_2d_cg2(sf + b * C::SFA_BYTES, &tmSFX, full_cl, 0, ((NB * tt + b) * p.nks + ks) * S);
    };
    // Behind this call's own quantiser, which has waited for whatever came before it, the weights
    // may be read while it runs: the first ring of them. All else reads its output.
    const int ahead = min(p.nks, STAGES);
    int nt0, tt0;
    raster(pair, n_tiles, t_tiles, nt0, tt0);
    if (warp == 0 && !p.first) {
        if (elect_one())
            for (int i = 0; i < ahead; ++i) load_w(nt0, i, i);
        __syncwarp();
    }
    grid_dep_wait();
    grid_dep_launch();

    auto give_up = [&]() { *abort_flag = 1; };

    if (warp == 0) {
        const bool elected = elect_one();
        if (elected)
            for (int i = 0; i < ahead; ++i) {
                if (p.first) load_w(nt0, i, i);
                load_x(tt0, i, i);
            }
        __syncwarp();
        int stage = ahead % STAGES;
        uint32_t phase = ahead / STAGES, issued = ahead;
        bool ok = true;
        for (int tile = pair; ok && tile < total; tile += npairs) {
            int nt, tt;
            raster(tile, n_tiles, t_tiles, nt, tt);
            for (int ks = tile == pair ? ahead : 0; ks < p.nks; ++ks) {
                if (!warp_wait(empty0 + 8 * stage, phase ^ 1, tmo, abort_flag)) {
                    give_up();
                    ok = false;
                    break;
                }
                if (elected) {
                    load_w(nt, ks, stage);
                    load_x(tt, ks, stage);
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
                    const uint32_t st = (smem0 + stage * C::STAGE_BYTES) / 16, sf = st + (C::A_BYTES + C::B_BYTES) / 16;
                    const uint32_t sfa_col = tmem_base + BT + stage * C::SF_COLS;
                    const uint32_t sfb_col = sfa_col + 4 * S;
                    if (elected) {
#pragma unroll
                        for (int a = 0; a < S; ++a) tc_cp2_sf_atom(sfa_col + 4 * a, atom_desc(sf + a * ATOM_BYTES / 16));
                        // shared memory holds the token atoms as [block][s]; tensor memory wants [s][block]
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int a = 0; a < S; ++a)
                                tc_cp2_sf_atom(sfb_col + 4 * (a * NB + b),
                                               atom_desc(sf + (C::SFA_BYTES + (b * S + a) * ATOM_BYTES) / 16));
                        lin_stage<FMT, 2, BT>(tmem_base, st, st + C::A_BYTES / 16, sfa_col, sfb_col, NB, ks == 0);
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
        constexpr int COLS = BT / 4;    // tokens of a warp
        const int q = warp % 4;         // the lane quarter of tensor memory this warp may read
        const int cg = (warp - 2) / 4;  // its tokens of the tile
        const uint32_t leader_tempty = mapa_shared(tempty_bar, 0);
        uint32_t acc_phase = 0;
        for (int tile = pair; tile < total; tile += npairs) {
            int nt, tt;
            raster(tile, n_tiles, t_tiles, nt, tt);
            const int n = nt * 256 + (int)rank * BM + q * 32 + lane, t0 = tt * BT + cg * COLS;
            // Of token t0 + 32 c + lane, on its way while the MMAs run, and handed round by shuffles: 256
            // loads of one word each in the epilogue made it 1 us longer (2048 x 4096 x 4096 23.9 us, 22.2
            // so). Through shared memory they take less, but 4 KB more of it delay the quantiser of a
            // call that follows (23.2).
            // Plain loads: the quantiser writes the scales while this kernel is resident already, which the
            // read-only path does not allow.
            float2 scale[COLS / 32];
            if constexpr (FMT == MOE_FMT_NVFP4) {
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c)
                    scale[c] = t0 + 32 * c + lane < p.M ? token_scale(p.x_scale[t0 + 32 * c + lane], *p.w_scale)
                                                        : make_float2(0.0f, 1.0f);
            }
            // warp-uniform: every lane leaves together (a lane left behind would block in __syncwarp)
            if (!warp_wait(tfull_bar, acc_phase, tmo, abort_flag)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + cg * COLS;
            // into registers, then the accumulator is handed back, and only then scaled and stored
            float v[COLS / 32][32];
#pragma unroll
            for (int c = 0; c < COLS / 32; ++c) tmem_ld32(tacc + 32 * c, v[c]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    mbar_arrive(tempty_bar);
                else
                    mbar_arrive_cluster(leader_tempty);
            }
            acc_phase ^= 1;
            if constexpr (FMT == MOE_FMT_NVFP4) {
#pragma unroll
                for (int j = 0; j < COLS; ++j) v[j / 32][j % 32] *= __shfl_sync(0xffffffffu, scale[j / 32].x, j % 32);
                bool rest = false;
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) rest |= scale[c].y != 1.0f;
                if (__any_sync(0xffffffffu, rest)) {
#pragma unroll
                    for (int j = 0; j < COLS; ++j) v[j / 32][j % 32] *= __shfl_sync(0xffffffffu, scale[j / 32].y, j % 32);
                }
            }
            if (n < p.N) {
                __nv_bfloat16* o = p.out + (int64_t)t0 * p.ldo + n;
#pragma unroll
                for (int j = 0; j < COLS; ++j) {
                    float y = v[j / 32][j % 32];
                    if (t0 + j < p.M) *o = __float2bfloat16_rn(y);
                    o += p.ldo;
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) write_status(p, blockIdx.x, gridDim.x, *abort_flag != 0);
    cluster_sync();  // both CTAs are done with each other's barriers and the MMAs have drained
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ clusters that split K
constexpr int MAX_SPLITS = 8;  // the portable cluster size

// QUANT: the kernel quantises its slice of x itself, straight into the operand layout in shared
// memory (all its K stages at once), instead of loading quantised rows.
// DEEP: one CTA on an SM with a ring as deep as fits (grids of at most one CTA for each SM); else
// two CTAs share an SM.
template <int FMT, int BT, bool QUANT, bool DEEP>
struct SplitCfg {
    static constexpr int S = fmt_sf_atoms(FMT);
    static constexpr int EPI = 8;                       // epilogue warps, two for each lane quarter
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int A_BYTES = BM * BK_BYTES;
    static constexpr int B_BYTES = BT * BK_BYTES;
    static constexpr int SF_BYTES = S * ATOM_BYTES;      // of either side
    static constexpr int X_STAGE = B_BYTES + SF_BYTES;   // a stage of x
    static constexpr int X_STAGES = QUANT ? (FMT == MOE_FMT_MXFP8 ? 16 : 8) : 0;
    // QUANT: x's code rows of every stage (multiples of 1024 bytes), then their atoms
    static constexpr int X_CODES = X_STAGES * B_BYTES;
    static constexpr int X_AREA = (X_STAGES * X_STAGE + 1023) / 1024 * 1024;
    static constexpr uint32_t TX_BYTES = A_BYTES + SF_BYTES + (QUANT ? 0 : X_STAGE);
    // a stage: weight rows, their atoms, x's atoms, then x's rows at a multiple of 1024 bytes
    static constexpr int X_PAD = (2 * SF_BYTES + 1023) / 1024 * 1024 - SF_BYTES;
    static constexpr int STAGE_BYTES =
        QUANT ? (A_BYTES + SF_BYTES + 1023) / 1024 * 1024 : A_BYTES + SF_BYTES + X_PAD + B_BYTES;
    // the sums of a tile: an area of their own where they are small, else the ring
    static constexpr int SUM_BYTES = (BT + MAX_SPLITS) * BM * 4;  // splits * ceil(BT / splits) rows at most
    static constexpr bool OWN_SUMS = BT <= 16;
    static constexpr int BAR_BYTES = 256;
    static constexpr int FIXED = X_AREA + (OWN_SUMS ? SUM_BYTES : 0) + BAR_BYTES + 1024;
    static constexpr int BUDGET = DEEP ? 232448 : 233472 / 2 - 1024 - 512;
    static constexpr int STAGES_MAX = (BUDGET - FIXED) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_MAX < 8 ? STAGES_MAX : 8;
    static constexpr int SMEM = FIXED + STAGES * STAGE_BYTES;
    static constexpr int SF_COLS = 8 * S;
    static constexpr int COLS = BT + STAGES * SF_COLS;
    static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(COLS <= (DEEP ? 512 : 256), "tensor memory budget");
    static_assert(STAGES >= 3 && (!DEEP || SMEM + 8 * BT <= 232448), "shared memory budget");
    static_assert(OWN_SUMS || STAGES * STAGE_BYTES >= SUM_BYTES, "the ring holds the sums");
};

// The codes of 16 elements, unit u of row r of a K stage, where the MMA reads them: a row has 128
// bytes, its 16-byte pieces numbered XOR r % 8 (the 128-byte swizzle that TMA applies).
template <int FMT>
__device__ __forceinline__ void put_unit(uint8_t* s, int r, int u, const uint32_t (&q)[4]) {
    if constexpr (FMT == MOE_FMT_MXFP8)
        *reinterpret_cast<uint4*>(s + r * BK_BYTES + ((u ^ (r & 7)) * 16)) = make_uint4(q[0], q[1], q[2], q[3]);
    else
        *reinterpret_cast<uint2*>(s + r * BK_BYTES + (((u >> 1) ^ (r & 7)) * 16) + (u & 1) * 8) = make_uint2(q[0], q[1]);
}

template <int FMT, int BT, bool QUANT, bool DEEP>
__global__ void __launch_bounds__(SplitCfg<FMT, BT, QUANT, DEEP>::THREADS, DEEP ? 1 : 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const LinearArgs p) {
    using C = SplitCfg<FMT, BT, QUANT, DEEP>;
    constexpr int S = C::S, STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xs = smem + STAGES * C::STAGE_BYTES;  // QUANT: x's codes and atoms
    float* sums = reinterpret_cast<float*>(C::OWN_SUMS ? xs + C::X_AREA : smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(xs + C::X_AREA + (C::OWN_SUMS ? C::SUM_BYTES : 0));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* never = reinterpret_cast<int*>(tmem_slot + 2);
    __shared__ uint32_t s_amax[QUANT ? BT : 1];  // NVFP4: the tokens' magnitudes (bit patterns)
    // NVFP4: what a token's sums are multiplied by (token_scale), and whether any second factor is not 1
    __shared__ float s_alpha[FMT == MOE_FMT_NVFP4 ? BT : 1], s_rest[FMT == MOE_FMT_NVFP4 ? BT : 1];
    __shared__ int s_any_rest;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, done_bar = empty0 + 8 * STAGES,
                   x_bar = done_bar + 8;
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t tmo = p.timeout_ns;
    // grid.x = splits (one cluster), grid.y = weight tiles, grid.z = token tiles
    const uint32_t splits = gridDim.x, rank = blockIdx.x;
    const int nt = blockIdx.y, tt = blockIdx.z;
    const int k0 = (int)((int64_t)p.nks * rank / splits), k1 = (int)((int64_t)p.nks * (rank + 1) / splits);
    const int tokens = min(BT, p.M - tt * BT);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * STAGES; ++s) mbar_init(full0 + 8 * s, 1);
        mbar_init(done_bar, 1);
        mbar_init(x_bar, C::EPI);
        *abort_flag = 0;
        *never = 0;
        if constexpr (FMT == MOE_FMT_NVFP4) s_any_rest = 0;
        fence_mbar_init();
        prefetch_tmap(&tmW);
        if constexpr (!QUANT) prefetch_tmap(&tmX);
    }
    if (QUANT && threadIdx.x < BT) s_amax[threadIdx.x] = 0;
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // matched just before the first store into another CTA's shared memory: by then it has started
    if (C::OWN_SUMS && splits > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    auto give_up = [&]() { *abort_flag = 1; };
    if (QUANT || p.first) {
        // the predecessor may be any kernel: not even the weights are read before the wait
        grid_dep_wait();
        grid_dep_launch();
    }

    bool complete = true;  // meaningful in the epilogue's warps
    if (warp == 0) {
        const bool elected = elect_one();
        auto load_w = [&](int ks, int stage) {
            const uint32_t st = smem0 + stage * C::STAGE_BYTES, full = full0 + 8 * stage;
            mbar_arrive_expect_tx(full, C::TX_BYTES);
            tma_load_2d(st, &tmW, full, ks * BK_BYTES, nt * BM);
            bulk_load(st + C::A_BYTES, p.sfb + ((int64_t)ks * p.sf_blocks + nt) * C::SF_BYTES, C::SF_BYTES, full);
        };
        auto load_x = [&](int ks, int stage) {
            if constexpr (!QUANT) {
                const uint32_t st = smem0 + stage * C::STAGE_BYTES + C::A_BYTES + C::SF_BYTES, full = full0 + 8 * stage;
                // token tiles start at multiples of 128 rows, or there is only one
                bulk_load(st, p.sfa + ((int64_t)(tt * BT / BM) * p.nks + ks) * C::SF_BYTES, C::SF_BYTES, full);
                tma_load_2d(st + C::X_PAD, &tmX, full, ks * BK_BYTES, tt * BT);
            }
        };
        // Behind this call's own quantiser, which has waited for whatever came before it, the weights
        // may be read while it runs.
        const int ahead = min(k1 - k0, STAGES);
        if (elected)
            for (int i = 0; i < ahead; ++i) load_w(k0 + i, i);
        if constexpr (!QUANT) {
            grid_dep_wait();
            grid_dep_launch();
        }
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
        __syncwarp();
    } else if (warp == 1) {
        const bool elected = elect_one();
        bool ok = true;
        if constexpr (QUANT) {
            ok = warp_wait(x_bar, 0, tmo, abort_flag);  // x is in shared memory
            if (!ok) give_up();
        } else {
            grid_dep_wait();
        }
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; ok && i < k1 - k0; ++i) {
            if (!warp_wait(full0 + 8 * stage, phase, tmo, abort_flag)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t st = (smem0 + stage * C::STAGE_BYTES) / 16, sfw = st + C::A_BYTES / 16;
            const uint32_t x = QUANT ? smem_u32(xs) / 16 + i * (C::B_BYTES / 16) : sfw + (C::SF_BYTES + C::X_PAD) / 16;
            const uint32_t sfx = QUANT ? smem_u32(xs) / 16 + (C::X_CODES + i * C::SF_BYTES) / 16 : sfw + C::SF_BYTES / 16;
            const uint32_t sfa_col = tmem_base + BT + stage * C::SF_COLS, sfb_col = sfa_col + 4 * S;
            if (elected) {
#pragma unroll
                for (int a = 0; a < S; ++a) tc_cp_sf_atom(sfa_col + 4 * a, atom_desc(sfw + a * ATOM_BYTES / 16));
#pragma unroll
                for (int a = 0; a < S; ++a) tc_cp_sf_atom(sfb_col + 4 * a, atom_desc(sfx + a * ATOM_BYTES / 16));
                lin_stage<FMT, 1, BT>(tmem_base, st, x, sfa_col, sfb_col, 1, i == 0);
                tc_commit(empty0 + 8 * stage);
            }
            __syncwarp();
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
        // every MMA and copy issued has completed; also the epilogue's signal
        if (elected) tc_commit(done_bar);
        __syncwarp();
        mbar_wait(done_bar, 0, DRAIN_TIMEOUT_NS, never);
        __syncwarp();
    } else {
        if constexpr (QUANT) {
            // Units of 16 elements, one thread each, a token after the other. NVFP4's row scale needs
            // the whole row's magnitude: every CTA reads the whole rows for it (a few tokens from
            // L2), which takes less than an exchange between the CTAs.
            constexpr int UNITS = FMT == MOE_FMT_MXFP8 ? 8 : 16;  // of a stage and token
            constexpr int NT = 32 * C::EPI;
            const int tid = threadIdx.x - 64, u0 = k0 * UNITS, per_token = (k1 - k0) * UNITS, uk = p.K / 16;
            const uint4* x = reinterpret_cast<const uint4*>(p.x);
            const int64_t row = p.ldx / 8;  // 16-byte pieces between rows
            if constexpr (FMT == MOE_FMT_NVFP4) {
                for (int r = 0; r < tokens; ++r) {
                    float m = 0.0f;
#pragma unroll 4
                    for (int u = tid; u < uk; u += NT) m = max_or_nan(m, unit_amax(x[r * row + 2 * u], x[r * row + 2 * u + 1]));
                    // magnitudes order like their bits, a NaN above infinity
                    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7FFFFFFFu);
                    if (lane == 0) atomicMax(&s_amax[r], top);
                }
                asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
            }
            // every lane of a warp takes part in the shuffles: whole warps of units
            const int total = tokens * per_token;
            for (int i = tid; i - lane < total; i += NT) {
                const int at = min(i, total - 1), r = at / per_token, u = at - r * per_token;
                const bool past = u0 + u >= uk;  // past K: zeros, so that a scale cannot make a NaN of them
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (!past) {
                    a = x[r * row + 2 * (u0 + u)];
                    b = x[r * row + 2 * (u0 + u) + 1];
                }
                float f[2][8];
                unpack_bf16x8(a, f[0]);
                unpack_bf16x8(b, f[1]);
                const float amax = unit_amax(a, b);
                uint8_t* codes = xs + (u / UNITS) * C::B_BYTES;
                uint8_t* atoms = xs + C::X_CODES + (u / UNITS) * C::SF_BYTES;
                const int us = u % UNITS;
                uint32_t q[4] = {0, 0, 0, 0}, sb;
                if constexpr (FMT == MOE_FMT_NVFP4) {
                    const Nvfp4Row nv(nvfp4_row_scale(__uint_as_float(s_amax[r])));
                    const float eff = nv.block_scale(amax, sb);
                    uint32_t c[2];
                    nv.codes<2>(f, eff, c);
                    q[0] = c[0], q[1] = c[1];
                } else {
                    const float m = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    const int e = mx_scale<FMT == MOE_FMT_MXFP8>(m, sb);
                    if constexpr (FMT == MOE_FMT_MXFP8) {
                        const uint2 lo = e4m3_codes(f[0], e), hi = e4m3_codes(f[1], e);
                        q[0] = lo.x, q[1] = lo.y, q[2] = hi.x, q[3] = hi.y;
                    } else {
                        q[0] = mxfp4_codes(f[0], e), q[1] = mxfp4_codes(f[1], e);
                    }
                }
                if (i >= total) continue;
                put_unit<FMT>(codes, r, us, q);
                const int kb = FMT == MOE_FMT_NVFP4 ? us : us / 2;
                if (FMT == MOE_FMT_NVFP4 || us % 2 == 0)
                    atoms[(kb / 4) * ATOM_BYTES + (r % 32) * 16 + (r / 32) * 4 + kb % 4] = past ? 0 : (uint8_t)sb;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(x_bar);
        } else {
            grid_dep_wait();
        }
        if constexpr (FMT == MOE_FMT_NVFP4) {
            const int c = (int)threadIdx.x - 64;
            if (c < tokens) {
                const float2 f = token_scale(QUANT ? nvfp4_row_scale(__uint_as_float(s_amax[c])) : p.x_scale[tt * BT + c],
                                             *p.w_scale);
                s_alpha[c] = f.x;
                s_rest[c] = f.y;
                if (f.y != 1.0f) s_any_rest = 1;
            }
        }
        complete = warp_wait(done_bar, 0, tmo, abort_flag);
        if (!complete) give_up();
        tc_fence_after();
    }
    // Sums: the tile's tokens are shared out in runs of per_rank, and every CTA sends its
    // accumulators of a token to its owner (rows of 128 features, one for each rank and token).
    // The ring, where it serves as that area, is free in all CTAs after the first barrier.
    const int per_rank = (tokens + (int)splits - 1) / (int)splits;
    if (splits == 1) {
        __syncthreads();
    } else if (C::OWN_SUMS) {
        __syncthreads();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    } else {
        cluster_sync();
    }
    // Without a split the accumulators are stored from the registers, a lane its feature of each token
    // (600 x 2048 x 2048 NVFP4 7.8 us, through shared memory 9.3).
    if (warp >= 2 && splits == 1) {
        const int q = warp % 4, n = nt * BM + q * 32 + lane;
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16);
        constexpr int STEP = BT >= 32 ? 32 : 16;
#pragma unroll 1
        for (int c0 = (warp - 2) / 4 * STEP; c0 < tokens; c0 += 2 * STEP) {
            float v[32];
            tmem_ld32(tacc + c0, v);  // for BT = 16 the upper columns hold scales: not kept
            tmem_ld_wait();
            const float* last = s_alpha + c0;  // the factor that is applied where a value is stored
            if (FMT == MOE_FMT_NVFP4 && s_any_rest) {
#pragma unroll
                for (int j = 0; j < STEP; ++j) v[j] *= last[j];  // past the tokens: not kept
                last = s_rest + c0;
            }
            if (n < p.N && complete) {
                __nv_bfloat16* o = p.out + (int64_t)(tt * BT + c0) * p.ldo + n;
#pragma unroll
                for (int j = 0; j < STEP; ++j) {
                    if (c0 + j < tokens) *o = __float2bfloat16_rn(FMT == MOE_FMT_NVFP4 ? v[j] * last[j] : v[j]);
                    o += p.ldo;
                }
            }
        }
        tc_fence_before();
    } else if (warp >= 2) {
        const int q = warp % 4;
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16);
        const uint32_t mine = smem_u32(sums + (int)rank * per_rank * BM + q * 32 + lane);
        constexpr int STEP = BT >= 32 ? 32 : 16;
#pragma unroll 1
        for (int c0 = (warp - 2) / 4 * STEP; c0 < tokens; c0 += 2 * STEP) {
            float v[32];
            tmem_ld32(tacc + c0, v);  // for BT = 16 the upper columns hold scales: not kept
            tmem_ld_wait();
            int owner = c0 / per_rank, left = (owner + 1) * per_rank - c0;  // tokens until the next owner
            uint32_t at = mapa_shared(mine + (c0 - owner * per_rank) * (BM * 4), owner);
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                if (c0 + j < tokens) st_cluster_u32(at, __float_as_uint(v[j]));
                at += BM * 4;
                if (--left == 0 && c0 + j + 1 < tokens) {
                    at = mapa_shared(mine, ++owner);
                    left = per_rank;
                }
            }
        }
        tc_fence_before();
    }
    if (splits > 1) cluster_sync();
    // This CTA's tokens: a warp takes a token, a lane 4 features, the ranks added in order.
    if (warp >= 2 && complete && splits > 1) {
        const int n = nt * BM + 4 * lane, first = (int)rank * per_rank, count = min(per_rank, tokens - first);
        __nv_bfloat16* out = p.out + (int64_t)(tt * BT + first) * p.ldo + n;
        const bool whole = n + 4 <= p.N && ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(2 * p.ldo)) & 7) == 0;
#pragma unroll 4
        for (int i = warp - 2; i < count; i += C::EPI) {
            const float4* u = reinterpret_cast<const float4*>(sums + i * BM) + lane;
            float4 y = u[0];
            for (uint32_t r = 1; r < splits; ++r) {
                const float4 v = u[r * per_rank * (BM / 4)];
                y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
            }
            if constexpr (FMT == MOE_FMT_NVFP4) {
                const float alpha = s_alpha[first + i], rest = s_rest[first + i];
                y.x = y.x * alpha * rest, y.y = y.y * alpha * rest, y.z = y.z * alpha * rest, y.w = y.w * alpha * rest;
            }
            __nv_bfloat16* o = out + i * p.ldo;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
            if (whole) {
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
    __syncthreads();
    if (threadIdx.x == 0)
        write_status(p, blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z),
                     gridDim.x * gridDim.y * gridDim.z, *abort_flag != 0);
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
// Pairs once there are more tiles of 128 x 128 than SMs (1024 x 4096 x 4096 MXFP8, 256 of them: 21.2
// us, split kernel 24.3; 384 x 6400 x 4096, 150: 16.4 and 14.8, NVFP4 12.2 and 11.5). Below, K is
// split in powers of two (clusters of 3 or 5 find fewer places: 300 x 2048 x 4096 NVFP4 13.5 us in
// threes, 12.0 in fours) over at most one CTA for each SM (128 x 7168 x 4096 NVFP4 in four parts 11.6 us,
// in one 8.8).
// A stage takes 0.24 us, the sums of a split tile some 2.7 us with 128 tokens and 1.7 with 64: a split has
// to save more stages than that (128 x 4096 x 4096: NVFP4, 16 stages, 8.6 us in one part, 9.6 in two,
// 8.6 in four; MXFP8, 32 stages, 12.1, 10.8 and 9.6). Eight parts pay with 16 tokens alone (128 x 2048 x
// 7168 NVFP4 11.3 us in eight, 9.1 in four). With few tokens and long slices the MMA warp's issue bounds a
// CTA, and two on an SM are faster: 1 x 7168 x 7168 MXFP8 11.8 us against 13.9.
LinearShape linear_shape(int M, int N, int nks, int num_sms) {
    LinearShape s{};
    if (M > 128 && ceil_div(M, 128) * ceil_div(N, BM) > num_sms) {
        s.bt = 256;  // splits = 0
        return s;
    }
    s.bt = M <= 16 ? 16 : M <= 64 ? 64 : 128;
    const int max_splits = s.bt == 16 ? MAX_SPLITS : 4, sum_stages = s.bt == 16 ? 0 : s.bt == 64 ? 7 : 11;
    const int64_t tiles = ceil_div(M, s.bt) * ceil_div(N, BM);
    auto most = [&](int64_t slots) {
        int k = 1;
        while (2 * k <= max_splits && tiles * 2 * k <= slots && 4 * k <= nks) k *= 2;
        return nks - nks / k > sum_stages ? k : 1;
    };
    s.splits = most(num_sms);
    s.deep = tiles * s.splits <= num_sms && s.splits <= 4;  // clusters of 8 with an SM for each CTA find few places
    if (s.bt == 16 && nks > 10 * s.splits) {
        s.splits = most(2 * num_sms);
        s.deep = false;
    }
    return s;
}

// Most CTAs of a product with N outputs on any number of tokens: pairs fill the SMs once, and tiles of 128
// features are only multiplied (by K splits or further token tiles) up to two CTAs for each SM.
int linear_max_ctas(int N, int num_sms) {
    const int64_t n_tiles = ceil_div(N, BM);
    return (int)(n_tiles > 2 * num_sms ? n_tiles : 2 * num_sms);
}

// Whether the product quantises x itself: few tokens, x's stages within the kernel's area, aligned
// rows. It saves a launch, but every CTA then quantises its slice, and for NVFP4 reads the whole
// rows for their scales. Measured with N = 4096, in the product against separately: MXFP4 8 x 4096
// 4.7 and 5.4 us, 8 x 7168 both 6.35, 12 x 7168 7.2 and 6.4; MXFP8 8 x 7168 7.7 and 8.5, 16 x 7168 9.0 and
// 8.7; NVFP4 2 x 7168 6.3 and 6.6, 3 x 7168 7.5 and 6.6, 3 x 2048 5.0 and 4.8.
bool linear_quantises(int fmt, const LinearShape& s, int M, int nks, const void* x, int64_t ldx) {
    return M <= (fmt == MOE_FMT_NVFP4 ? 2 : 8) && s.bt == 16 &&
           ceil_div(nks, s.splits) <= (fmt == MOE_FMT_MXFP8 ? 16 : 8) &&
           ((uintptr_t)x | (uintptr_t)(2 * ldx)) % 16 == 0;
}

template <int FMT, int BT, bool QUANT, bool DEEP>
static cudaError_t split_attr() {
    return cudaFuncSetAttribute(linear_split_kernel<FMT, BT, QUANT, DEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SplitCfg<FMT, BT, QUANT, DEEP>::SMEM);
}
template <int FMT>
static cudaError_t lin_attr() {
    cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PairCfg<FMT>::SMEM);
    if (e == cudaSuccess) e = split_attr<FMT, 16, true, false>();
    if (e == cudaSuccess) e = split_attr<FMT, 16, false, false>();
    if (e == cudaSuccess) e = split_attr<FMT, 16, false, true>();
    if (e == cudaSuccess) e = split_attr<FMT, 64, false, false>();
    if (e == cudaSuccess) e = split_attr<FMT, 64, false, true>();
    if (e == cudaSuccess) e = split_attr<FMT, 128, false, false>();
    if (e == cudaSuccess) e = split_attr<FMT, 128, false, true>();
    return e;
}
cudaError_t linear_prepare(int fmt) {
    switch (fmt) {
        case MOE_FMT_MXFP8: return lin_attr<MOE_FMT_MXFP8>();
        case MOE_FMT_MXFP4: return lin_attr<MOE_FMT_MXFP4>();
        default: return lin_attr<MOE_FMT_NVFP4>();
    }
}

template <int FMT, int BT, bool QUANT, bool DEEP>
static cudaError_t split_d(const LinearMaps& m, const LinearArgs& p, int splits, cudaStream_t st) {
    using C = SplitCfg<FMT, BT, QUANT, DEEP>;
    LaunchAttrs at(true, splits);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)splits, (unsigned)ceil_div(p.N, BM), (unsigned)ceil_div(p.M, BT)),
                                       dim3(C::THREADS), C::SMEM, st);
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<FMT, BT, QUANT, DEEP>, m.w, m.x, p);
}
template <int FMT, int BT>
static cudaError_t split_t(const LinearMaps& m, const LinearArgs& p, const LinearShape& s, cudaStream_t st) {
    return s.deep ? split_d<FMT, BT, false, true>(m, p, s.splits, st) : split_d<FMT, BT, false, false>(m, p, s.splits, st);
}

template <int FMT>
static cudaError_t pair_t(const LinearMaps& m, const LinearArgs& p, int num_sms, cudaStream_t st) {
    LaunchAttrs at(true, 2);
    const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256), pairs = num_sms / 2;
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))),
                                       dim3(PairCfg<FMT>::THREADS), PairCfg<FMT>::SMEM, st);
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<FMT>, m.w, m.x, m.sfw, m.sfx, p);
}

template <int FMT>
static cudaError_t lin_t(const LinearMaps& m, const LinearArgs& p, const LinearShape& s, int num_sms, cudaStream_t st) {
    if (s.splits == 0)
        return pair_t<FMT>(m, p, num_sms, st);
    switch (s.bt) {
        case 16: return p.x ? split_d<FMT, 16, true, false>(m, p, s.splits, st) : split_t<FMT, 16>(m, p, s, st);
        case 64: return split_t<FMT, 64>(m, p, s, st);
        default: return split_t<FMT, 128>(m, p, s, st);
    }
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
