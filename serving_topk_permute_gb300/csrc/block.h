// block.h -- internal host-side launchers of the operators around the experts (norm and
// quantisation, router, linear product).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// ------------------------------------------------------------------ residual add, RMSNorm, quantisation
struct NormArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* res;    // or null
    const float* gamma;          // null: no norm (quantise x itself)
    __nv_bfloat16* sum;          // or null
    __nv_bfloat16* out;          // or null
    int64_t ldx, ldr, lds, ldo;  // row strides in elements
    int T, H;
    float eps;
    float inv_h;                 // 1 / H (set by launch_norm)
    int fmt;                     // -1: no quantised output
    int atoms;                   // 1: scales in atoms, 0: row-major
    int64_t nks;                 // K stages of the atom layout
    uint8_t* codes;
    uint8_t* sf;
    float* row_scale;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);

// ------------------------------------------------------------------ router
struct RouterArgs {
    const void* logits;
    int64_t ld;
    int bf16;
    const uint8_t* mask;
    int T, E, k, renorm;
    float coef;
    int32_t* ids;
    float* w;
    int32_t* counts;
    int32_t* num_valid;
    float* prob_mean;
    float* loss;
    int want_probs;              // sum the probabilities
    int32_t* part_counts;        // [grid][E]
    int32_t* part_valid;         // [grid]
    float* part_probs;           // [grid][E]
};
struct RouterGradArgs {
    const void* logits;
    int64_t ld;
    int bf16;
    const uint8_t* mask;
    int T, E, k, renorm;
    float coef;
    const int32_t* ids;
    const int32_t* counts;
    const int32_t* num_valid;
    const float* dw;
    const float* dloss;
    void* dlogits;
    int64_t ldd;
};
int router_grid(int T, int E);  // CTAs that leave partial sums in the workspace
cudaError_t launch_router(const RouterArgs& a, cudaStream_t st);
cudaError_t launch_router_grad(const RouterGradArgs& a, cudaStream_t st);

// ------------------------------------------------------------------ linear product
struct LinearArgs {
    const uint8_t* sfa;          // activation scale atoms [row tiles][nks][S][512]
    const uint8_t* sfb;          // weight scale atoms [nks][sf_blocks][S][512]
    int M, N, K, nks, sf_blocks;
    const __nv_bfloat16* x;      // quantised by the kernel when set (linear_quantises), rows ldx apart
    int64_t ldx;
    const float* x_scale;        // NVFP4: fp32 [M]
    const float* w_scale;        // NVFP4: fp32 [1]
    __nv_bfloat16* out;
    int64_t ldo;
    int* status;  // number of CTAs, then a word of each (linear_max_ctas at most)
    int first;    // no other kernel of this call came before: read nothing before the wait
    unsigned long long timeout_ns;
};
// weight scale atoms [nks][sf_blocks][S][512] from row-major [N, K/g] bytes, zeros past N and K
cudaError_t launch_pack_linear_sf(const uint8_t* src, uint8_t* dst, int fmt, int N, int K, cudaStream_t st);
cudaError_t linear_prepare(int fmt);
// The kernel for a product of these sizes: bt tokens a tile, K split over `splits` CTAs; splits 0
// means CTA pairs.
struct LinearShape {
    int bt, splits;
    bool deep;  // at most one CTA for each SM: the ring takes all of its shared memory
    // rows of the token map's box
    int x_box() const { return splits ? bt : 128; }
};
LinearShape linear_shape(int M, int N, int nks, int num_sms);
int linear_max_ctas(int N, int num_sms);
bool linear_quantises(int fmt, const LinearShape& s, int M, int nks, const void* x, int64_t ldx);
struct LinearMaps {
    CUtensorMap w, x;      // code rows, boxes of 128 weight rows and of x_box() tokens
    CUtensorMap sfw, sfx;  // scale atoms as uint32 [atoms][128], boxes of S atoms (pairs only)
};
cudaError_t launch_linear(int fmt, const LinearMaps& m, const LinearArgs& p, const LinearShape& s, int num_sms,
                          cudaStream_t st);

}  // namespace moe
