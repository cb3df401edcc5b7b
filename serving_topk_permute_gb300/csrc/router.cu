// router.cu -- softmax router with top-k selection, per-expert counts and the balance loss
// (moe_router_forward), and its gradient (moe_router_backward).
//
//   p = softmax(l),  ids = the k largest logits (ties to the lowest id),  w = p[ids] (/ their sum)
//   counts_e = #{id = e},  P_e = sum_t p[t,e] / n,  loss = coef E sum_e counts_e / (k n) P_e
//   dl = p (g - sum_e p g),  g[t,e] = d_loss coef E counts_e / (k n^2) + [e = id_j] dw'_j,
//   dw'_j = dw_j, or (dw_j - sum_m w_m dw_m) / sum_m p[id_m] with renormalised weights
//
// One warp per token row, expert e in lane e % 32. Selection works on the logits' order-
// preserving integer keys. Column sums: each warp sums its rows' probabilities in registers,
// the warps of a CTA join in a fixed order, and a second small kernel joins the CTAs'
// partial sums, again in a fixed order; no floating atomics.
#include "block.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int ROUTER_WARPS_PER_CTA = 8;
constexpr int ROUTER_THREADS = 32 * ROUTER_WARPS_PER_CTA;
constexpr int ROUTER_MAX_GRID = 152 * 4;

// unsigned keys in the order of the floats: -inf < ... < +inf < NaN (either sign); -0 as +0
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // order_key(-inf): the lowest key of a logit
constexpr uint32_t KEY_NAN = 0xFFFFFFFFu;
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == KEY_NAN) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
    if constexpr (BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    else
        return reinterpret_cast<const float*>(p)[i];
}

// C: experts per lane, 32 C >= E
template <bool BF16, int C>
__global__ void __launch_bounds__(ROUTER_THREADS) router_kernel(const RouterArgs a) {
    extern __shared__ int s_dyn[];
    int* s_counts = s_dyn;                                    // [E]
    float* s_probs = reinterpret_cast<float*>(s_dyn + a.E);   // [warps][E] when probabilities are summed
    __shared__ int s_valid[ROUTER_WARPS_PER_CTA];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    for (int e = tid; e < a.E; e += ROUTER_THREADS) s_counts[e] = 0;
    __syncthreads();
    float psum[C];
#pragma unroll
    for (int i = 0; i < C; ++i) psum[i] = 0.0f;
    int valid_rows = 0;
    for (int64_t t = (int64_t)blockIdx.x * ROUTER_WARPS_PER_CTA + warp; t < a.T;
         t += (int64_t)gridDim.x * ROUTER_WARPS_PER_CTA) {
        uint32_t key[C];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = lane + 32 * i;
            key[i] = e < a.E ? order_key(logit_at<BF16>(a.logits, t * a.ld + e)) : 0u;
            best = max(best, key[i]);
        }
        best = __reduce_max_sync(0xffffffffu, best);
        const bool valid = best > KEY_NEG_INF && (!a.mask || a.mask[t] != 0);
        int32_t my_id = -1;      // of slot `lane`
        float my_e = 0.0f;
        if (valid) {  // warp-uniform
            ++valid_rows;
            const float top = key_value(best);
            float ex[C], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                ex[i] = key[i] ? expf(key_value(key[i]) - top) : 0.0f;
                sum += ex[i];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = 1.0f / sum;
            if (a.want_probs) {
#pragma unroll
                for (int i = 0; i < C; ++i) psum[i] += ex[i] * inv;
            }
            uint32_t m = best;
            float ksum = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                if (j > 0) {
                    m = 0;
#pragma unroll
                    for (int i = 0; i < C; ++i) m = max(m, key[i]);
                    m = __reduce_max_sync(0xffffffffu, m);
                }
                if (m <= KEY_NEG_INF) break;  // only -inf experts are left
                uint32_t at = 0xFFFFFFFFu;
#pragma unroll
                for (int i = C - 1; i >= 0; --i)
                    if (key[i] == m) at = lane + 32 * i;
                at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
                for (int i = 0; i < C; ++i)
                    if (at == (uint32_t)(lane + 32 * i)) key[i] = 0;
                const float v = expf(key_value(m) - top);
                ksum += v;
                if (lane == j) {
                    my_id = (int32_t)at;
                    my_e = v;
                }
            }
            if (lane < a.k) {
                my_e = my_id >= 0 ? my_e / (a.renorm ? ksum : sum) : 0.0f;
                if (my_id >= 0) atomicAdd(&s_counts[my_id], 1);
            }
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = my_id;
            a.w[t * a.k + lane] = my_e;
        }
    }
    if (lane == 0) s_valid[warp] = valid_rows;
    if (a.want_probs) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) s_probs[warp * a.E + e] = psum[i];
        }
    }
    __syncthreads();
    if (!a.part_counts) return;
    for (int e = tid; e < a.E; e += ROUTER_THREADS) {
        a.part_counts[(int64_t)blockIdx.x * a.E + e] = s_counts[e];
        if (a.want_probs) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < ROUTER_WARPS_PER_CTA; ++w) s += s_probs[w * a.E + e];
            a.part_probs[(int64_t)blockIdx.x * a.E + e] = s;
        }
    }
    if (tid == 0) {
        int n = 0;
        for (int w = 0; w < ROUTER_WARPS_PER_CTA; ++w) n += s_valid[w];
        a.part_valid[blockIdx.x] = n;
    }
}

// joins the CTAs' partial counts and sums: thread e takes expert e
__global__ void __launch_bounds__(512) router_join_kernel(const RouterArgs a, int parts) {
    __shared__ float s_red[16];
    __shared__ int s_n[16];
    const int e = threadIdx.x, lane = e % 32, warp = e / 32;
    grid_dep_wait();
    int n = 0;
    for (int i = e; i < parts; i += 512) n += a.part_valid[i];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < 16; ++w) n += s_n[w];
    const float nf = (float)max(n, 1);
    float term = 0.0f;
    if (e < a.E) {
        int c = 0;
        float p = 0.0f;
        for (int i = 0; i < parts; ++i) {
            c += a.part_counts[(int64_t)i * a.E + e];
            if (a.want_probs) p += a.part_probs[(int64_t)i * a.E + e];
        }
        p /= nf;
        if (a.counts) a.counts[e] = c;
        if (a.prob_mean) a.prob_mean[e] = p;
        term = (float)c / ((float)a.k * nf) * p;
    }
    if (e == 0 && a.num_valid) *a.num_valid = n;
    if (!a.loss) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
    if (lane == 0) s_red[warp] = term;
    __syncthreads();
    if (e == 0) {
        float s = 0.0f;
        for (int w = 0; w < 16; ++w) s += s_red[w];
        *a.loss = a.coef * (float)a.E * s;
    }
}

template <bool BF16, int C>
__global__ void __launch_bounds__(ROUTER_THREADS) router_grad_kernel(const RouterGradArgs a) {
    extern __shared__ float s_grad[];  // [warps][E]: the selected slots' part of g
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    float* sg = s_grad + warp * a.E;
    float base[C];
    float c0 = 0.0f;
    if (a.dloss) {
        const float n = (float)max(*a.num_valid, 1);
        c0 = *a.dloss * a.coef * (float)a.E / ((float)a.k * n * n);
    }
    // The softmax's gradient does not change when every g shifts by the same amount, so counts
    // enter as differences from their mean: under balanced routing g - p.g would otherwise be
    // the difference of two nearly equal numbers.
    int cnt[C], mean = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = lane + 32 * i;
        cnt[i] = a.dloss && e < a.E ? a.counts[e] : 0;
        mean += cnt[i];
    }
    mean = __reduce_add_sync(0xffffffffu, mean) / a.E;
#pragma unroll
    for (int i = 0; i < C; ++i) base[i] = lane + 32 * i < a.E ? c0 * (float)(cnt[i] - mean) : 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * ROUTER_WARPS_PER_CTA + warp; t < a.T;
         t += (int64_t)gridDim.x * ROUTER_WARPS_PER_CTA) {
        float v[C];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = lane + 32 * i;
            v[i] = 0.0f;
            if (e < a.E) {
                v[i] = logit_at<BF16>(a.logits, t * a.ld + e);
                best = max(best, order_key(v[i]));
            }
        }
        best = __reduce_max_sync(0xffffffffu, best);
        const bool valid = best > KEY_NEG_INF && (!a.mask || a.mask[t] != 0);
        float d[C];
#pragma unroll
        for (int i = 0; i < C; ++i) d[i] = 0.0f;
        if (valid) {  // warp-uniform
            const float top = key_value(best);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[i] = lane + 32 * i < a.E ? expf(v[i] - top) : 0.0f;
                sum += v[i];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] *= inv;  // p
            float g[C];
#pragma unroll
            for (int i = 0; i < C; ++i) g[i] = base[i];
            if (a.dw) {
                int id = -1;
                float dw = 0.0f;
                if (lane < a.k) {
                    id = a.ids[t * a.k + lane];
                    if ((unsigned)id >= (unsigned)a.E) id = -1;
                    if (id >= 0) dw = a.dw[t * a.k + lane];
                }
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.E) sg[e] = v[i];
                }
                __syncwarp();
                float pk = id >= 0 ? sg[id] : 0.0f;
                __syncwarp();
                if (a.renorm) {
                    float ps = pk, pd = pk * dw;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        ps += __shfl_xor_sync(0xffffffffu, ps, o);
                        pd += __shfl_xor_sync(0xffffffffu, pd, o);
                    }
                    dw = ps != 0.0f ? (dw - pd / ps) / ps : 0.0f;
                    if (id < 0) dw = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.E) sg[e] = 0.0f;
                }
                __syncwarp();
                for (int j = 0; j < a.k; ++j) {  // in slot order: a repeated id adds up in a fixed order
                    const int ij = __shfl_sync(0xffffffffu, id, j);
                    const float dj = __shfl_sync(0xffffffffu, dw, j);
                    if (ij >= 0 && (ij & 31) == lane) sg[ij] += dj;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.E) g[i] += sg[e];
                }
                __syncwarp();
            }
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) dot = fmaf(v[i], g[i], dot);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
#pragma unroll
            for (int i = 0; i < C; ++i) d[i] = v[i] * (g[i] - dot);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) {
                if constexpr (BF16)
                    reinterpret_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + e] = __float2bfloat16_rn(d[i]);
                else
                    reinterpret_cast<float*>(a.dlogits)[t * a.ldd + e] = d[i];
            }
        }
    }
}

// CTAs of the forward pass: a fixed function of the sizes, so that sums keep their order
int router_grid(int T, int E) {
    (void)E;
    const int64_t g = ceil_div(T, ROUTER_WARPS_PER_CTA);
    return (int)(g < ROUTER_MAX_GRID ? g : ROUTER_MAX_GRID);
}

template <bool BF16, int C>
static cudaError_t router_t(const RouterArgs& a, cudaStream_t st) {
    const int grid = router_grid(a.T, a.E);
    if (grid > 0) {
        const size_t smem = 4 * (size_t)a.E * (1 + (a.want_probs ? ROUTER_WARPS_PER_CTA : 0));
        router_kernel<BF16, C><<<grid, ROUTER_THREADS, smem, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!a.part_counts) return cudaSuccess;
    LaunchAttrs at(false);
    cudaLaunchConfig_t cfg = at.config(dim3(1), dim3(512), 0, st);
    return cudaLaunchKernelEx(&cfg, router_join_kernel, a, grid);
}

template <bool BF16, int C>
static cudaError_t router_grad_t(const RouterGradArgs& a, cudaStream_t st) {
    const int grid = router_grid(a.T, a.E);
    if (grid == 0) return cudaSuccess;
    router_grad_kernel<BF16, C><<<grid, ROUTER_THREADS, 4 * (size_t)a.E * ROUTER_WARPS_PER_CTA, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_router(const RouterArgs& a, cudaStream_t st) {
    if (a.E <= 64) return a.bf16 ? router_t<true, 2>(a, st) : router_t<false, 2>(a, st);
    if (a.E <= 128) return a.bf16 ? router_t<true, 4>(a, st) : router_t<false, 4>(a, st);
    if (a.E <= 256) return a.bf16 ? router_t<true, 8>(a, st) : router_t<false, 8>(a, st);
    return a.bf16 ? router_t<true, 16>(a, st) : router_t<false, 16>(a, st);
}

cudaError_t launch_router_grad(const RouterGradArgs& a, cudaStream_t st) {
    if (a.E <= 64) return a.bf16 ? router_grad_t<true, 2>(a, st) : router_grad_t<false, 2>(a, st);
    if (a.E <= 128) return a.bf16 ? router_grad_t<true, 4>(a, st) : router_grad_t<false, 4>(a, st);
    if (a.E <= 256) return a.bf16 ? router_grad_t<true, 8>(a, st) : router_grad_t<false, 8>(a, st);
    return a.bf16 ? router_grad_t<true, 16>(a, st) : router_grad_t<false, 16>(a, st);
}

}  // namespace moe
