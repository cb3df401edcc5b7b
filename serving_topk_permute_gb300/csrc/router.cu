// router.cu -- softmax router with top-k selection, per-expert counts and the balance loss
// (moe_router_forward), and its gradient (moe_router_backward).
//
//   p = softmax(l),  ids = the k largest logits (ties to the lowest id),  w = p[ids] (/ their sum)
//   counts_e = #{id = e},  P_e = sum_t p[t,e] / n,  loss = coef E sum_e counts_e / (k n) P_e
//   dl = p (g - sum_e p g),  g[t,e] = d_loss coef E counts_e / (k n^2) + [e = id_j] dw'_j,
//   dw'_j = dw_j, or (dw_j - sum_m w_m dw_m) / sum_m p[id_m] with renormalised weights
//
// One warp per token row, C experts in each lane.
//
// Selection: a logit becomes an order-preserving 32-bit key whose low 9 bits hold 511 - id, so
// that keys are unique and the larger key is the larger logit, then the lower id. Each lane
// finds the two largest of its C keys; a pick is the warp's maximum of the lanes' largest, and
// the lane that held it moves its second one up. Only a lane that is picked from a third time
// looks through its keys again, for the largest below the pick m: max over (key - m) mod 2^32,
// because keys below m wrap to values above all others. bf16 logits fit the upper 23 bits. fp32
// logits lose their last 9 bits there: one pick more is made, and neighbours in the order that
// agree in the upper 23 bits are put in order by their full logits, or, if they are the k-th
// and the next, the row takes the exact way, as one with a NaN or +inf does: k rounds on
// full 32-bit keys.
//
// Column sums: each warp sums its rows' probabilities in registers, the warps of a CTA join in a
// fixed order, then the CTAs: small batches run as one cluster, which joins through distributed
// shared memory, larger ones leave partial sums to a second kernel of one cluster. No floating
// atomics: every sum has a fixed order.
//
// Measured on GB300, 256 experts, fp32, the 8 largest. 32,768 tokens with the loss: 23.4 us, of which 2.5 are the
// sums' (loss and counts left out: 21.9 with 34,048 tokens, 24.5 with). The bytes would take 5.3 us, the some 410
// instructions a row at full issue about 11; they fill 63% of the slots. A warp has one row at a time, whose
// k + 1 picks are a chain of dependent warp reductions, and 32 warps on an SM do not cover it. Neither a
// row's loads one row ahead (23.5 us) nor three CTAs of 40 registers on an SM (28.9) help. 128 tokens:
// 4.4 us, a cluster's launch and one row's chain of picks. The gradient of 32,768 tokens: 15.0 us,
// 4.6 TB/s, 68% of the copy rate: loads that wait for the row before (one row ahead 15.3 to 16.6 us),
// and issue, 65% of the slots.
#include "block.h"
#include "common.cuh"
#include "kernels.h"
#include "router.cuh"

namespace moe {

constexpr int ROUTER_WARPS = 16;
constexpr int ROUTER_THREADS = 32 * ROUTER_WARPS;
// CTAs on an SM, the whole grid resident at once. 16 experts a lane: one CTA's registers fill the SM
// (two of 64 registers, 32,768 x 512 bf16: 33.7 us against 34.2, but 4096 x 512 fp32 11.9 against
// 10.3).
constexpr int router_ctas(int E) { return E > 256 ? 1 : 2; }
constexpr int GRAD_WARPS = 8;
constexpr int GRAD_THREADS = 32 * GRAD_WARPS;
// The gradient's: 32,768 x 256 fp32 15.0 us with five, 17.1 with four, 15.1 with six; 32,768 x 512
// bf16 20.6 with four, 22.2 with five, 22.5 with three, 29.1 with two.
constexpr int grad_ctas(int C) { return C > 8 ? 4 : 5; }
constexpr int JOIN_CTAS = 8;
constexpr int JOIN_THREADS = 1024;
// Up to this many tokens run as one cluster of at most 8 CTAs of 16 warps, joined in place.
constexpr int CLUSTER_WARPS = 16;
constexpr int CLUSTER_TOKENS = 512;

constexpr uint32_t ID_BITS = 511u;              // E <= 512
constexpr uint32_t PACKED_FINITE = 0x00800000u;  // packed keys below hold -inf, or no expert

// Experts of a lane: W consecutive ones (one vector access) every 32 W. MODE 0: W = 1, where rows
// are not aligned for more; 1: vector accesses; 2: vector accesses and E = 32 C, no bounds.
template <bool BF16, int C, int MODE>
struct Lanes {
    static constexpr int WMAX = BF16 ? 8 : 4;
    static constexpr int W = MODE ? (C < WMAX ? C : WMAX) : 1;
    static constexpr bool FULL = MODE == 2;
    static __device__ __forceinline__ int expert(int lane, int i) { return (i / W) * 32 * W + lane * W + i % W; }
    // the row's logits, -inf past E (E is a multiple of W)
    static __device__ __forceinline__ void load(const void* logits, int64_t row, int E, int lane, float (&v)[C]) {
#pragma unroll
        for (int g = 0; g < C / W; ++g) {
            const int e = expert(lane, g * W);
            if (FULL || e < E) {
                if constexpr (W == 1) {
                    v[g] = logit_at<BF16>(logits, row + e);
                } else if constexpr (BF16) {
                    uint32_t w[W / 2];
                    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(logits) + row + e;
                    if constexpr (W == 8) {
                        const uint4 q = *reinterpret_cast<const uint4*>(p);
                        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
                    } else if constexpr (W == 4) {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        w[0] = q.x, w[1] = q.y;
                    } else {
                        w[0] = *reinterpret_cast<const uint32_t*>(p);
                    }
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) {
                        v[g * W + 2 * j] = __uint_as_float(w[j] << 16);
                        v[g * W + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                } else if constexpr (W == 4) {
                    const float4 q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(logits) + row + e);
                    v[g * 4] = q.x, v[g * 4 + 1] = q.y, v[g * 4 + 2] = q.z, v[g * 4 + 3] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(logits) + row + e);
                    v[g * 2] = q.x, v[g * 2 + 1] = q.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[g * W + j] = -__int_as_float(0x7F800000);
            }
        }
    }
    static __device__ __forceinline__ void store(void* out, int64_t row, int E, int lane, const float (&v)[C]) {
#pragma unroll
        for (int g = 0; g < C / W; ++g) {
            const int e = expert(lane, g * W);
            if (!FULL && e >= E) continue;
            if constexpr (BF16) {
                __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(out) + row + e;
                if constexpr (W == 1) {
                    *p = __float2bfloat16_rn(v[g]);
                } else {
                    uint32_t w[W / 2];
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[g * W + 2 * j], v[g * W + 2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    if constexpr (W == 8)
                        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
                    else if constexpr (W == 4)
                        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t*>(p) = w[0];
                }
            } else {
                float* p = reinterpret_cast<float*>(out) + row + e;
                if constexpr (W == 4)
                    *reinterpret_cast<float4*>(p) = make_float4(v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]);
                else if constexpr (W == 2)
                    *reinterpret_cast<float2*>(p) = make_float2(v[g * 2], v[g * 2 + 1]);
                else
                    *p = v[g];
            }
        }
    }
};

// both sums: the lower 16 lanes add the first one up, the upper ones the second
__device__ __forceinline__ void warp_sums(float& a, float& b, int lane) {
    const bool upper = lane >= 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// The row's largest logit; NaN when the row holds a NaN.
template <int C>
__device__ __forceinline__ float row_max(const float (&v)[C]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < C; ++i) m = max_nan(m, v[i]);
    const uint32_t key = order_key(m);
    return key_value(__reduce_max_sync(0xffffffffu, key));
}

// exact selection on full keys: lane j gets the j-th expert (-1: only -inf left) and its logit
template <bool BF16, int C, int MODE>
__device__ __noinline__ void select_exact(const void* logits, int64_t row, int E, int k, int lane, int& id, float& l) {
    using L = Lanes<BF16, C, MODE>;
    float v[C];
    L::load(logits, row, E, lane, v);
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; ++i) key[i] = L::FULL || L::expert(lane, i) < E ? order_key(v[i]) : 0u;
    for (int j = 0; j < k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (m <= KEY_NEG_INF) break;
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
            if (key[i] == m) at = min(at, (uint32_t)L::expert(lane, i));
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (at == (uint32_t)L::expert(lane, i)) key[i] = 0;
        if (lane == j) {
            id = (int)at;
            l = key_value(m);
        }
    }
}

constexpr uint32_t PACKED_INF = 0xFF800000u & ~ID_BITS;  // packed keys from here on: +inf or NaN

// The row's packed keys, and the largest two of the lane's (0: none).
template <bool BF16, int C, int MODE>
__device__ __forceinline__ void pack_keys(const float (&v)[C], int E, int lane, uint32_t (&key)[C], uint32_t& h1,
                                          uint32_t& h2) {
    using L = Lanes<BF16, C, MODE>;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = L::expert(lane, i);
        key[i] = L::FULL || e < E ? (order_key(v[i]) & ~ID_BITS) | (ID_BITS - (uint32_t)e) : 0u;
    }
    h1 = max(key[0], key[1]);
    h2 = min(key[0], key[1]);
#pragma unroll
    for (int i = 2; i < C; i += 2) {
        const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
        h2 = __vimax3_u32(min(h1, hi), h2, lo);
        h1 = max(h1, hi);
    }
}

// Ids and logits of the row's top k, slot j in lane j (id -1: none), from its packed keys, the
// lanes' largest two and the largest of all, m.
template <bool BF16, int C, int MODE>
__device__ __forceinline__ void select(const RouterArgs& a, int64_t row, const uint32_t (&key)[C], uint32_t h1,
                                       uint32_t h2, uint32_t m, int lane, int& id, float& l) {
    id = -1;
    l = 0.0f;
    if (m >= PACKED_INF) {
        select_exact<BF16, C, MODE>(a.logits, row, a.E, a.k, lane, id, l);
        return;
    }
    uint32_t mine = 0;
    const int last = BF16 ? a.k - 1 : a.k;  // fp32: one pick more
#pragma unroll 4
    for (int j = 0;; ++j) {
        mine = lane == j ? m : mine;
        if (j == last) break;
        const bool held = h1 == m;
        h1 = held ? h2 : h1;
        h2 = held ? 0 : h2;
        if constexpr (C > 2) {
            if (__any_sync(0xffffffffu, held && h1 == 0)) {  // its third, or it has no more
                uint32_t d = 0;
#pragma unroll
                for (int i = 0; i < C; ++i) d = __viaddmax_u32(key[i], 0u - m, d);
                d = m + d < m ? m + d : 0;
                h1 = held ? d : h1;
            }
        }
        m = __reduce_max_sync(0xffffffffu, h1);
    }
    const bool got = lane < a.k && mine >= PACKED_FINITE;
    id = got ? (int)(ID_BITS - (mine & ID_BITS)) : -1;
    if (got) l = logit_at<BF16>(a.logits, row + id);
    if constexpr (!BF16) {
        uint32_t after = __shfl_down_sync(0xffffffffu, mine, 1);
        if (lane == 31) after = m;  // k = 32: the pick past the last lane's
        const uint32_t equal =
            __ballot_sync(0xffffffffu, id >= 0 && after >= PACKED_FINITE && ((after ^ mine) & ~ID_BITS) == 0);
        if (equal >> (a.k - 1)) {  // warp-uniform
            id = -1;
            select_exact<BF16, C, MODE>(a.logits, row, a.E, a.k, lane, id, l);
        } else if (equal) {
            const uint32_t full = id >= 0 ? order_key(l) : 0u;
            int rank = 0;  // slots that come before mine
            for (int j = 0; j < a.k; ++j) {
                const uint32_t f = __shfl_sync(0xffffffffu, full, j);
                const int i = __shfl_sync(0xffffffffu, id, j);
                rank += f > full || (f == full && (i < id && i >= 0));
            }
            if (id < 0) rank = lane;  // empty slots stay behind the others
            int from = lane;
            for (int j = 0; j < a.k; ++j)
                if (__shfl_sync(0xffffffffu, rank, j) == lane) from = j;
            const int nid = __shfl_sync(0xffffffffu, id, from);
            const float nl = __shfl_sync(0xffffffffu, l, from);
            id = nid;
            l = nl;
        }
    }
}

// This CTA's rows: ids and weights to memory, counts to s_counts, probability sums to s_probs
// (one row of [E] for each warp), the number of valid rows returned per warp.
template <bool BF16, int C, int MODE, int WARPS>
__device__ __forceinline__ void route_rows(const RouterArgs& a, int* s_counts, float* s_probs, int* s_valid) {
    using L = Lanes<BF16, C, MODE>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float psum[C];
#pragma unroll
    for (int i = 0; i < C; ++i) psum[i] = 0.0f;
    int valid_rows = 0;
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
        float v[C];
        L::load(a.logits, t * a.ld, a.E, lane, v);
        const bool masked = a.mask && a.mask[t] == 0;
        uint32_t key[C];
        uint32_t h1, h2;
        pack_keys<BF16, C, MODE>(v, a.E, lane, key, h1, h2);
        const uint32_t m = __reduce_max_sync(0xffffffffu, h1);
        int id = -1;
        float w = 0.0f;
        if (!masked && m >= PACKED_FINITE) {  // warp-uniform
            ++valid_rows;
            // Any value near the largest logit serves as the exponent's offset. The largest key's
            // upper bits are within 2^-14 of it; only for huge logits is that not near enough.
            // These are subtracted first; the others' offset enters with the factor log2(e), its
            // rounding the same for the whole row.
            float top = key_value(m & ~ID_BITS), huge = 0.0f;
            if (!(fabsf(top) < 4096.0f)) {
                huge = row_max<C>(v);
                top = 0.0f;
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] -= huge;
            }
            const float offset = -LOG2E * top;
            float l;
            select<BF16, C, MODE>(a, t * a.ld, key, h1, h2, m, lane, id, l);
            w = id >= 0 ? fast_exp2(fmaf(l - huge, LOG2E, offset)) : 0.0f;
            float sum = 0.0f, picked = w;
            if (a.want_probs || !a.renorm) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    v[i] = fast_exp2(fmaf(v[i], LOG2E, offset));  // 0 for -inf
                    sum += v[i];
                }
            }
            warp_sums(sum, picked, lane);
            if (a.want_probs) {
                const float inv = fast_div(1.0f, sum);
#pragma unroll
                for (int i = 0; i < C; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
            }
            w = id >= 0 ? fast_div(w, a.renorm ? picked : sum) : 0.0f;
            if (id >= 0) atomicAdd(&s_counts[id], 1);
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.w[t * a.k + lane] = w;
        }
    }
    if (lane == 0) s_valid[warp] = valid_rows;
    if (a.want_probs) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = L::expert(lane, i);
            if (e < a.E) s_probs[warp * a.E + e] = psum[i];
        }
    }
}

// The CTA's sums: the warps in order. s_counts[E] is complete; probabilities end in s_probs[0..E).
template <int WARPS>
__device__ __forceinline__ void join_warps(const RouterArgs& a, float* s_probs) {
    __syncthreads();
    if (!a.want_probs) return;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += s_probs[w * a.E + e];
        s_probs[e] = s;
    }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// One expert's results from its totals; returns its term of the loss's sum.
__device__ __forceinline__ float expert_totals(const RouterArgs& a, int e, int c, float p, float n) {
    p /= n;
    if (a.counts) a.counts[e] = c;
    if (a.prob_mean) a.prob_mean[e] = p;
    return (float)c / ((float)a.k * n) * p;
}

// sum of the threads' terms over the CTA (NT threads), in every thread
template <int NT>
__device__ __forceinline__ float cta_total(float v, float* s_red) {
    v = warp_sum(v);
    if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += s_red[w];
    return t;
}

// CTA rank 0 of the cluster adds the CTAs' terms of the loss in order and writes the scalars.
template <int NT>
__device__ __forceinline__ void cluster_loss(const RouterArgs& a, float term, int n, float* s_term, float* s_red,
                                             uint32_t rank, uint32_t ctas) {
    if (rank == 0 && threadIdx.x == 0 && a.num_valid) *a.num_valid = n;
    if (a.loss) {  // the same for every CTA
        const float t = cta_total<NT>(term, s_red);
        if (threadIdx.x == 0) *s_term = t;
        cluster_sync();
        if (rank == 0 && threadIdx.x == 0) {
            float s = 0.0f;
            for (uint32_t c = 0; c < ctas; ++c) s += ld_cluster_f32(mapa_shared(smem_u32(s_term), c));
            *a.loss = a.coef * (float)a.E * s;
        }
    }
    cluster_sync();  // no CTA leaves while its shared memory is read
}

// Larger batches: partial sums of each CTA to memory, joined by router_join_kernel.
template <bool BF16, int C, int MODE>
__global__ void __launch_bounds__(ROUTER_THREADS, router_ctas(32 * C)) router_kernel(const RouterArgs a) {
    extern __shared__ int s_dyn[];
    int* s_counts = s_dyn;                                   // [E]
    float* s_probs = reinterpret_cast<float*>(s_dyn + a.E);  // [warps][E] when probabilities are summed
    __shared__ int s_valid[ROUTER_WARPS];
    for (int e = threadIdx.x; e < a.E; e += ROUTER_THREADS) s_counts[e] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    route_rows<BF16, C, MODE, ROUTER_WARPS>(a, s_counts, s_probs, s_valid);
    if (!a.part_counts) return;
    join_warps<ROUTER_WARPS>(a, s_probs);
    for (int e = threadIdx.x; e < a.E; e += ROUTER_THREADS) {
        a.part_counts[(int64_t)blockIdx.x * a.E + e] = s_counts[e];
        if (a.want_probs) a.part_probs[(int64_t)blockIdx.x * a.E + e] = s_probs[e];
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < ROUTER_WARPS; ++w) n += s_valid[w];
        a.part_valid[blockIdx.x] = n;
    }
}

// One cluster of JOIN_CTAS CTAs; CTA c takes every JOIN_CTAS-th group of 32 experts. Warp w of a
// CTA adds the parts w, w + 32, ... of 32 experts (one in each lane), then the warps in order.
__global__ void __launch_bounds__(JOIN_THREADS) router_join_kernel(const RouterArgs a, int parts) {
    constexpr int WARPS = JOIN_THREADS / 32;
    __shared__ int s_n[WARPS], s_c[WARPS][32];
    __shared__ float s_p[WARPS][32], s_red[WARPS], s_term;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t rank = cluster_ctarank();
    grid_dep_wait();
    grid_dep_launch();
    int n = 0;
    for (int i = threadIdx.x; i < parts; i += JOIN_THREADS) n += __ldcg(a.part_valid + i);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_n[warp] = n;
    float term = 0.0f;
    for (int e0 = 32 * (int)rank; e0 < a.E; e0 += 32 * JOIN_CTAS) {
        const int e = e0 + lane;
        int c = 0;
        float p = 0.0f;
        if (e < a.E) {
            if (a.want_probs) {
#pragma unroll 5
                for (int i = warp; i < parts; i += WARPS) {
                    c += __ldcg(a.part_counts + (int64_t)i * a.E + e);
                    p += __ldcg(a.part_probs + (int64_t)i * a.E + e);
                }
            } else {
#pragma unroll 5
                for (int i = warp; i < parts; i += WARPS) c += __ldcg(a.part_counts + (int64_t)i * a.E + e);
            }
        }
        __syncthreads();  // the previous group's sums have been read
        s_c[warp][lane] = c;
        s_p[warp][lane] = p;
        __syncthreads();
        if (warp == 0 && e < a.E) {
            n = 0;
            c = 0;
            p = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                n += s_n[w];
                c += s_c[w][lane];
                p += s_p[w][lane];
            }
            term += expert_totals(a, e, c, p, (float)max(n, 1));
        }
    }
    __syncthreads();
    n = 0;
    for (int w = 0; w < WARPS; ++w) n += s_n[w];
    cluster_loss<JOIN_THREADS>(a, term, n, &s_term, s_red, rank, JOIN_CTAS);
}

// Small batches: one cluster, the CTAs' sums joined through distributed shared memory; CTA c
// takes the experts c, c + ctas, ... of each CTA-wide group.
template <bool BF16, int C, int MODE>
__global__ void __launch_bounds__(32 * CLUSTER_WARPS) router_cluster_kernel(const RouterArgs a) {
    constexpr int NT = 32 * CLUSTER_WARPS;
    extern __shared__ int s_dyn[];
    int* s_counts = s_dyn;
    float* s_probs = reinterpret_cast<float*>(s_dyn + a.E);
    __shared__ int s_valid[CLUSTER_WARPS], s_n;
    __shared__ float s_red[CLUSTER_WARPS], s_term;
    const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
    for (int e = threadIdx.x; e < a.E; e += NT) s_counts[e] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    route_rows<BF16, C, MODE, CLUSTER_WARPS>(a, s_counts, s_probs, s_valid);
    if (!a.counts && !a.num_valid && !a.want_probs) return;  // the same for every CTA of the cluster
    join_warps<CLUSTER_WARPS>(a, s_probs);
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < CLUSTER_WARPS; ++w) n += s_valid[w];
        s_n = n;
    }
    cluster_sync();
    int n = 0;
    for (uint32_t c = 0; c < ctas; ++c) n += ld_cluster_s32(mapa_shared(smem_u32(&s_n), c));
    float term = 0.0f;
    const int e = (int)(threadIdx.x * ctas + rank);  // E <= 512 <= NT
    if (e < a.E) {
        int c = 0;
        float p = 0.0f;
        for (uint32_t r = 0; r < ctas; ++r) {
            c += ld_cluster_s32(mapa_shared(smem_u32(s_counts + e), r));
            if (a.want_probs) p += ld_cluster_f32(mapa_shared(smem_u32(s_probs + e), r));
        }
        term = expert_totals(a, e, c, p, (float)max(n, 1));
    }
    cluster_loss<NT>(a, term, n, &s_term, s_red, rank, ctas);
}

// The gradient: dense part p_e (base_e - dot) for every expert, then the selected experts, whose
// g holds dw' too, written over it by the lanes that hold the slots.
template <bool BF16, int C, int MODE>
__global__ void __launch_bounds__(GRAD_THREADS, grad_ctas(C)) router_grad_kernel(const RouterGradArgs a) {
    using L = Lanes<BF16, C, MODE>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const float inf = __int_as_float(0x7F800000);
    grid_dep_wait();
    grid_dep_launch();
    float c0 = 0.0f;
    if (a.dloss) {
        const float n = (float)max(*a.num_valid, 1);
        c0 = *a.dloss * a.coef * (float)a.E / ((float)a.k * n * n);
    }
    // The softmax's gradient does not change when every g shifts by the same amount, so counts
    // enter as differences from their mean: under balanced routing g - p.g would otherwise be
    // the difference of two nearly equal numbers.
    float base[C];
    int cnt[C], mean = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = L::expert(lane, i);
        cnt[i] = a.dloss && e < a.E ? a.counts[e] : 0;
        mean += cnt[i];
    }
    mean = __reduce_add_sync(0xffffffffu, mean) / a.E;
#pragma unroll
    for (int i = 0; i < C; ++i) base[i] = L::expert(lane, i) < a.E ? c0 * (float)(cnt[i] - mean) : 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * GRAD_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * GRAD_WARPS) {
        float v[C];
        L::load(a.logits, t * a.ld, a.E, lane, v);
        int id = -1;
        float dw = 0.0f, l = 0.0f, own = 0.0f;
        if (a.dw && lane < a.k) {
            id = a.ids[t * a.k + lane];
            dw = a.dw[t * a.k + lane];
            if ((unsigned)id >= (unsigned)a.E) id = -1;
            dw *= a.dw_scale;
            if (id >= 0) {
                l = logit_at<BF16>(a.logits, t * a.ld + id);
                own = a.dloss ? c0 * (float)(a.counts[id] - mean) : 0.0f;
            }
        }
        const bool masked = a.mask && a.mask[t] == 0;
        const float top = row_max<C>(v);
        bool valid = !masked && top != -inf;  // warp-uniform
        if (a.empty_zero) valid = valid && __any_sync(0xffffffffu, id >= 0);
        float sel = 0.0f;
        if (valid) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[i] = fast_exp(v[i] - top);
                sum += v[i];
            }
            const float inv = fast_div(1.0f, warp_sum(sum));
            const float pk = id >= 0 ? fast_exp(l - top) * inv : 0.0f;
            if (id < 0) dw = 0.0f;
            if (a.dw && a.renorm) {
                const float ps = warp_sum(pk), pd = warp_sum(pk * dw);
                dw = id >= 0 && ps != 0.0f ? fast_div(dw - fast_div(pd, ps), ps) : 0.0f;
            }
            float dot = pk * dw;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[i] *= inv;  // p
                dot = fmaf(v[i], base[i], dot);
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] *= base[i] - dot;
            sel = pk * (own + dw - dot);
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = 0.0f;
        }
        L::store(a.dlogits, t * a.ldd, a.E, lane, v);
        if (a.dw && valid) {
            __syncwarp();  // the dense part is written before the selected experts' values
            if (id >= 0) {
                if constexpr (BF16)
                    reinterpret_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + id] = __float2bfloat16_rn(sel);
                else
                    reinterpret_cast<float*>(a.dlogits)[t * a.ldd + id] = sel;
            }
        }
    }
}

// ------------------------------------------------------------------ host side
static bool router_joins(const RouterArgs& a) { return a.counts || a.num_valid || a.want_probs; }

// CTAs that leave partial sums (0: one cluster does everything). A fixed function of the
// sizes, so that sums keep their order.
int router_grid(int T, int E) {
    if (T <= CLUSTER_TOKENS) return 0;
    const int64_t g = ceil_div(T, ROUTER_WARPS), most = SMS * router_ctas(E);
    return (int)(g < most ? g : most);
}

template <bool BF16, int C, int MODE>
static cudaError_t router_t(const RouterArgs& a, cudaStream_t st) {
    const int grid = router_grid(a.T, a.E);
    if (grid == 0) {
        const int64_t want = ceil_div(a.T, CLUSTER_WARPS);
        const int ctas = want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
        const size_t smem = 4 * (size_t)a.E * (1 + (a.want_probs ? CLUSTER_WARPS : 0));
        LaunchAttrs at(true, ctas);
        cudaLaunchConfig_t cfg = at.config(dim3(ctas), dim3(32 * CLUSTER_WARPS), smem, st);
        return cudaLaunchKernelEx(&cfg, router_cluster_kernel<BF16, C, MODE>, a);
    }
    {
        const size_t smem = 4 * (size_t)a.E * (1 + (a.want_probs ? ROUTER_WARPS : 0));
        LaunchAttrs at(true);
        cudaLaunchConfig_t cfg = at.config(dim3(grid), dim3(ROUTER_THREADS), smem, st);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, router_kernel<BF16, C, MODE>, a);
        if (e != cudaSuccess || !router_joins(a)) return e;
    }
    LaunchAttrs at(true, JOIN_CTAS);
    cudaLaunchConfig_t cfg = at.config(dim3(JOIN_CTAS), dim3(JOIN_THREADS), 0, st);
    return cudaLaunchKernelEx(&cfg, router_join_kernel, a, grid);
}

template <bool BF16, int C, int MODE>
static cudaError_t router_grad_t(const RouterGradArgs& a, cudaStream_t st) {
    const int64_t g = ceil_div(a.T, GRAD_WARPS), most = SMS * grad_ctas(C);
    LaunchAttrs at(true);
    cudaLaunchConfig_t cfg = at.config(dim3((unsigned)(g < most ? g : most)), dim3(GRAD_THREADS), 0, st);
    return cudaLaunchKernelEx(&cfg, router_grad_kernel<BF16, C, MODE>, a);
}

// rows that vector accesses of W elements may read: aligned starts, whole vectors
static bool vector_rows(const void* p, int64_t ld, int E, int el, int C) {
    const int wmax = el == 2 ? 8 : 4, W = C < wmax ? C : wmax;
    return reinterpret_cast<uintptr_t>(p) % (W * el) == 0 && ld % W == 0 && E % W == 0;
}

template <int C>
static cudaError_t router_c(const RouterArgs& a, cudaStream_t st) {
    const bool vec = vector_rows(a.logits, a.ld, a.E, a.bf16 ? 2 : 4, C), full = a.E == 32 * C;
    if (!vec) return a.bf16 ? router_t<true, C, 0>(a, st) : router_t<false, C, 0>(a, st);
    if (!full) return a.bf16 ? router_t<true, C, 1>(a, st) : router_t<false, C, 1>(a, st);
    return a.bf16 ? router_t<true, C, 2>(a, st) : router_t<false, C, 2>(a, st);
}
template <int C>
static cudaError_t router_grad_c(const RouterGradArgs& a, cudaStream_t st) {
    const int el = a.bf16 ? 2 : 4;
    const bool vec = vector_rows(a.logits, a.ld, a.E, el, C) && vector_rows(a.dlogits, a.ldd, a.E, el, C);
    const bool full = a.E == 32 * C;
    if (!vec) return a.bf16 ? router_grad_t<true, C, 0>(a, st) : router_grad_t<false, C, 0>(a, st);
    if (!full) return a.bf16 ? router_grad_t<true, C, 1>(a, st) : router_grad_t<false, C, 1>(a, st);
    return a.bf16 ? router_grad_t<true, C, 2>(a, st) : router_grad_t<false, C, 2>(a, st);
}

cudaError_t launch_router(const RouterArgs& a, cudaStream_t st) {
    if (a.E <= 64) return router_c<2>(a, st);
    if (a.E <= 128) return router_c<4>(a, st);
    if (a.E <= 256) return router_c<8>(a, st);
    return router_c<16>(a, st);
}

cudaError_t launch_router_grad(const RouterGradArgs& a, cudaStream_t st) {
    if (a.E <= 64) return router_grad_c<2>(a, st);
    if (a.E <= 128) return router_grad_c<4>(a, st);
    if (a.E <= 256) return router_grad_c<8>(a, st);
    return router_grad_c<16>(a, st);
}

}  // namespace moe
