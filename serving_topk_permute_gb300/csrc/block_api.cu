// block_api.cu -- the C ABI of the operators around the experts (include/moe.h, "around the
// experts"): argument checks, workspace layout, tensor maps and launches.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>
#include <new>

#include "block.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int MAX_ROW = 16384;          // widest row of the norm, the quantiser and the product's K
constexpr int MAX_EXPERTS = 512;
constexpr int MAX_TOP_K = 32;
constexpr int MAX_OUT = 1 << 20;
constexpr int64_t REGION_ALIGN = 1024;
constexpr unsigned long long DEFAULT_TIMEOUT_NS = 2000000000ull;  // 2 s per bounded wait

#define CUDA_TRY(x)                      \
    do {                                 \
        if ((x) != cudaSuccess) {        \
            (void)cudaGetLastError();    \
            return MOE_ERR_CUDA;         \
        }                                \
    } while (0)

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool quant_format(int f) { return f == MOE_FMT_MXFP8 || f == MOE_FMT_NVFP4 || f == MOE_FMT_MXFP4; }
// K stages of a row of K codes, the last one possibly part full
int64_t stages_of(int fmt, int64_t K) { return ceil_div(fmt_row_bytes(fmt, K), BK_BYTES); }

int check_quant(const moe_quant_t* q) {
    if (!quant_format(q->format)) return MOE_ERR_UNSUPPORTED;
    if (q->sf_layout != MOE_SF_ROWS && q->sf_layout != MOE_SF_ATOMS) return MOE_ERR_INVALID_ARG;
    if (!q->codes || !q->sf || !aligned_to(q->codes, 16) || (q->format == MOE_FMT_NVFP4) != (q->row_scale != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (q->row_scale && !aligned_to(q->row_scale, 4)) return MOE_ERR_INVALID_ARG;
    if (q->sf_layout == MOE_SF_ATOMS && !aligned_to(q->sf, 16)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// a bf16 matrix of rows at least H wide, ld elements apart (one row may have any stride)
bool rows_ok(const void* p, int64_t ld, int rows, int H) { return aligned_to(p, 2) && (rows <= 1 || ld >= H); }

// ------------------------------------------------------------------ tensor maps
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
bool get_encode() {
    std::call_once(g_encode_once, [] {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}
// rows of row_bytes code bytes, loaded as 128-byte x box_rows tiles with 128-byte swizzle;
// bytes past the row and rows past the last one are filled with zeros
bool map_rows(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows) {
    cuuint64_t dims[2] = {row_bytes, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {(cuuint32_t)BK_BYTES, box_rows};
    cuuint32_t es[2] = {1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// an array of 512-byte scale atoms as a 2-D uint32 tensor [atoms][128], loaded box_atoms at a time;
// atoms past the last one are filled with zeros
bool map_atoms(CUtensorMap* m, const void* base, uint64_t atoms, uint32_t box_atoms) {
    cuuint64_t dims[2] = {ATOM_BYTES / 4, atoms};
    cuuint64_t strides[1] = {ATOM_BYTES};
    cuuint32_t box[2] = {ATOM_BYTES / 4, box_atoms};
    cuuint32_t es[2] = {1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

struct moe_linear_plan_s {
    moe_linear_config_t cfg;
    int num_sms;
    unsigned long long timeout_ns;
};

namespace {

int check_linear(const moe_linear_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (!quant_format(c->format)) return MOE_ERR_UNSUPPORTED;
    if (c->out_features < 1 || c->out_features > MAX_OUT) return MOE_ERR_INVALID_ARG;
    if (c->in_features < 32 || c->in_features % 32 || c->in_features > MAX_ROW) return MOE_ERR_INVALID_ARG;
    if (c->max_tokens < 1 || c->max_tokens > (1 << 28)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_router(const moe_router_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->num_experts < 1 || c->num_experts > MAX_EXPERTS) return MOE_ERR_INVALID_ARG;
    if (c->top_k < 1 || c->top_k > c->num_experts || c->top_k > MAX_TOP_K) return MOE_ERR_INVALID_ARG;
    if (c->renormalize != 0 && c->renormalize != 1) return MOE_ERR_INVALID_ARG;
    if (c->logits_type != MOE_LOGITS_F32 && c->logits_type != MOE_LOGITS_BF16) return MOE_ERR_UNSUPPORTED;
    if (!isfinite(c->balance_coef)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// workspace of the product: the CTAs' status words at its start (as many for every T), then the
// quantised activations
struct LinLayout {
    int64_t codes, sf, scale, total;
};
LinLayout lin_layout(const moe_linear_plan_s* plan, int T) {
    const moe_linear_config_t& c = plan->cfg;
    LinLayout L{};
    const int S = fmt_sf_atoms(c.format);
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += align_up(bytes, REGION_ALIGN);
        return at;
    };
    take(4 * (1 + (int64_t)linear_max_ctas(c.out_features, plan->num_sms)));
    L.codes = take((int64_t)T * fmt_row_bytes(c.format, c.in_features));
    L.sf = take(ceil_div(T, BM) * stages_of(c.format, c.in_features) * S * ATOM_BYTES);
    L.scale = take(c.format == MOE_FMT_NVFP4 ? 4 * (int64_t)T : 0);
    L.total = o;
    return L;
}

// x: quantised rows, or (codes null) bf16 rows xb that the product quantises itself; first: no other
// kernel of the call comes before
int run_linear(moe_linear_plan_t plan, int T, const moe_quant_t& x, bool first, const void* xb, int64_t x_stride,
               const moe_linear_weight_t* w, void* out, int64_t out_stride, void* workspace, cudaStream_t st) {
    const moe_linear_config_t& c = plan->cfg;
    const uint64_t row_bytes = (uint64_t)fmt_row_bytes(c.format, c.in_features);
    const int nks = (int)stages_of(c.format, c.in_features), S = fmt_sf_atoms(c.format);
    const LinearShape shape = linear_shape(T, c.out_features, nks, plan->num_sms);
    const int64_t sf_blocks = wt_sf_blocks(c.out_features);
    LinearMaps m{};
    if (!map_rows(&m.w, w->codes, row_bytes, (uint64_t)c.out_features, BM) ||
        (x.codes && !map_rows(&m.x, x.codes, row_bytes, (uint64_t)T, shape.x_box())))
        return MOE_ERR_CUDA;
    if (!shape.splits && (!map_atoms(&m.sfw, w->sf, (uint64_t)(nks * sf_blocks * S), S) ||
                      !map_atoms(&m.sfx, x.sf, (uint64_t)(ceil_div(T, BM) * nks * S), S)))
        return MOE_ERR_CUDA;
    LinearArgs p{};
    p.sfa = (const uint8_t*)x.sf;
    p.sfb = (const uint8_t*)w->sf;
    p.M = T;
    p.N = c.out_features;
    p.K = c.in_features;
    p.nks = nks;
    p.x = x.codes ? nullptr : (const __nv_bfloat16*)xb;
    p.ldx = x_stride;
    p.sf_blocks = (int)sf_blocks;
    p.x_scale = x.row_scale;
    p.w_scale = w->global_scale;
    p.out = (__nv_bfloat16*)out;
    p.ldo = out_stride;
    p.status = (int*)workspace;
    p.first = first;
    p.timeout_ns = plan->timeout_ns;
    CUDA_TRY(launch_linear(c.format, m, p, shape, plan->num_sms, st));
    return MOE_OK;
}

int check_forward(moe_linear_plan_t plan, int T, const moe_linear_weight_t* w, const void* out, int64_t out_stride,
                  const void* workspace, size_t workspace_bytes) {
    if (!plan || T < 0) return MOE_ERR_INVALID_ARG;
    const moe_linear_config_t& c = plan->cfg;
    if (T > c.max_tokens) return MOE_ERR_CAPACITY;
    if (T == 0) return MOE_OK;
    if (!w || !w->codes || !w->sf || !out || !workspace) return MOE_ERR_INVALID_ARG;
    if ((c.format == MOE_FMT_NVFP4) != (w->global_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(w->codes, 256) || !aligned_to(w->sf, 256) || !aligned_to(workspace, 256) ||
        !aligned_to(w->global_scale, 4))
        return MOE_ERR_INVALID_ARG;
    if (!rows_ok(out, out_stride, T, c.out_features)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < (size_t)lin_layout(plan, T).total) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_quant_sf_size(int32_t format, int32_t sf_layout, int64_t rows, int64_t K, size_t* bytes) {
    if (!bytes || rows < 0 || K < 32 || K % 32 || K > MAX_ROW) return MOE_ERR_INVALID_ARG;
    if (!quant_format(format)) return MOE_ERR_UNSUPPORTED;
    if (sf_layout == MOE_SF_ROWS)
        *bytes = (size_t)(rows * (K / fmt_sf_block(format)));
    else if (sf_layout == MOE_SF_ATOMS)
        *bytes = (size_t)(ceil_div(rows, BM) * stages_of(format, K) * fmt_sf_atoms(format) * ATOM_BYTES);
    else
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int moe_quantize(int32_t rows, int32_t K, const void* x, int64_t x_stride, const moe_quant_t* q, void* stream) {
    if (rows < 0 || K < 32 || K % 32 || K > MAX_ROW || !q) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    const int v = check_quant(q);
    if (v != MOE_OK) return v;
    if (!x || !rows_ok(x, x_stride, rows, K)) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = (const __nv_bfloat16*)x;
    a.ldx = x_stride;
    a.T = rows;
    a.H = K;
    a.fmt = q->format;
    a.atoms = q->sf_layout == MOE_SF_ATOMS;
    a.nks = stages_of(q->format, K);
    a.codes = (uint8_t*)q->codes;
    a.sf = (uint8_t*)q->sf;
    a.row_scale = q->row_scale;
    CUDA_TRY(launch_norm(a, (cudaStream_t)stream));
    return MOE_OK;
}

int moe_add_rmsnorm(int32_t rows, int32_t hidden, const void* x, int64_t x_stride, const void* residual,
                    int64_t residual_stride, const float* gamma, float eps, void* sum_out, int64_t sum_stride,
                    void* out, int64_t out_stride, const moe_quant_t* q, void* stream) {
    if (rows < 0 || hidden < 1 || hidden > MAX_ROW || !(eps >= 0.0f) || !isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (q && hidden % 32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!out && !q) return MOE_ERR_INVALID_ARG;
    if (q) {
        const int v = check_quant(q);
        if (v != MOE_OK) return v;
    }
    if (!x || !gamma || !aligned_to(gamma, 4)) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(x, x_stride, rows, hidden) || (residual && !rows_ok(residual, residual_stride, rows, hidden)) ||
        (sum_out && !rows_ok(sum_out, sum_stride, rows, hidden)) || (out && !rows_ok(out, out_stride, rows, hidden)))
        return MOE_ERR_INVALID_ARG;
    if (sum_out && sum_out == out) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = (const __nv_bfloat16*)x;
    a.ldx = x_stride;
    a.res = (const __nv_bfloat16*)residual;
    a.ldr = residual_stride;
    a.gamma = gamma;
    a.eps = eps;
    a.sum = (__nv_bfloat16*)sum_out;
    a.lds = sum_stride;
    a.out = (__nv_bfloat16*)out;
    a.ldo = out_stride;
    a.T = rows;
    a.H = hidden;
    a.fmt = -1;
    if (q) {
        a.fmt = q->format;
        a.atoms = q->sf_layout == MOE_SF_ATOMS;
        a.nks = stages_of(q->format, hidden);
        a.codes = (uint8_t*)q->codes;
        a.sf = (uint8_t*)q->sf;
        a.row_scale = q->row_scale;
    }
    CUDA_TRY(launch_norm(a, (cudaStream_t)stream));
    return MOE_OK;
}

// ------------------------------------------------------------------ router
int moe_router_workspace_size(const moe_router_config_t* cfg, int32_t num_tokens, size_t* bytes) {
    const int v = check_router(cfg);
    if (v != MOE_OK) return v;
    if (!bytes || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const int64_t g = router_grid(num_tokens, cfg->num_experts);
    const int64_t need = 2 * align_up(4 * g * cfg->num_experts, 256) + align_up(4 * g, 256);
    *bytes = (size_t)(need > 256 ? need : 256);  // never none: one rule for every size
    return MOE_OK;
}

int moe_router_forward(const moe_router_config_t* cfg, int32_t num_tokens, const void* logits, int64_t logits_stride,
                       const uint8_t* token_mask, int32_t* topk_ids, float* topk_weights, int32_t* counts,
                       int32_t* num_valid, float* prob_mean, float* loss, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const int v = check_router(cfg);
    if (v != MOE_OK) return v;
    if (num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const int T = num_tokens, E = cfg->num_experts;
    const uintptr_t el = cfg->logits_type == MOE_LOGITS_BF16 ? 2 : 4;
    if (T > 0 && (!logits || !topk_ids || !topk_weights)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, el) || (T > 1 && logits_stride < E)) return MOE_ERR_INVALID_ARG;
    for (const void* q : {(const void*)topk_ids, (const void*)topk_weights, (const void*)counts, (const void*)num_valid,
                          (const void*)prob_mean, (const void*)loss})
        if (!aligned_to(q, 4)) return MOE_ERR_INVALID_ARG;
    RouterArgs a{};
    a.logits = logits;
    a.ld = logits_stride;
    a.bf16 = cfg->logits_type == MOE_LOGITS_BF16;
    a.mask = token_mask;
    a.T = T;
    a.E = E;
    a.k = cfg->top_k;
    a.renorm = cfg->renormalize;
    a.coef = cfg->balance_coef;
    a.ids = topk_ids;
    a.w = topk_weights;
    a.counts = counts;
    a.num_valid = num_valid;
    a.prob_mean = prob_mean;
    a.loss = loss;
    a.want_probs = prob_mean || loss;
    if (counts || num_valid || a.want_probs) {
        size_t need = 0;
        moe_router_workspace_size(cfg, T, &need);
        if (workspace && workspace_bytes < need) return MOE_ERR_WORKSPACE;
        if (!workspace || !aligned_to(workspace, 256)) return MOE_ERR_INVALID_ARG;
        const int64_t part = align_up(4 * (int64_t)router_grid(T, E) * E, 256);
        uint8_t* ws = (uint8_t*)workspace;
        a.part_counts = (int32_t*)ws;
        a.part_probs = (float*)(ws + part);
        a.part_valid = (int32_t*)(ws + 2 * part);
    }
    CUDA_TRY(launch_router(a, (cudaStream_t)stream));
    return MOE_OK;
}

int moe_router_backward(const moe_router_config_t* cfg, int32_t num_tokens, const void* logits, int64_t logits_stride,
                        const uint8_t* token_mask, const int32_t* topk_ids, const int32_t* counts,
                        const int32_t* num_valid, const float* d_weights, const float* d_loss, void* d_logits,
                        int64_t d_logits_stride, void* stream) {
    const int v = check_router(cfg);
    if (v != MOE_OK) return v;
    if (num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    const int T = num_tokens, E = cfg->num_experts;
    const uintptr_t el = cfg->logits_type == MOE_LOGITS_BF16 ? 2 : 4;
    if (!logits || !d_logits || !aligned_to(logits, el) || !aligned_to(d_logits, el)) return MOE_ERR_INVALID_ARG;
    if (T > 1 && (logits_stride < E || d_logits_stride < E)) return MOE_ERR_INVALID_ARG;
    if ((d_weights && !topk_ids) || (d_loss && (!counts || !num_valid))) return MOE_ERR_INVALID_ARG;
    for (const void* q : {(const void*)topk_ids, (const void*)counts, (const void*)num_valid, (const void*)d_weights,
                          (const void*)d_loss})
        if (!aligned_to(q, 4)) return MOE_ERR_INVALID_ARG;
    RouterGradArgs a{};
    a.logits = logits;
    a.ld = logits_stride;
    a.bf16 = cfg->logits_type == MOE_LOGITS_BF16;
    a.mask = token_mask;
    a.T = T;
    a.E = E;
    a.k = cfg->top_k;
    a.renorm = cfg->renormalize;
    a.coef = cfg->balance_coef;
    a.ids = topk_ids;
    a.counts = counts;
    a.num_valid = num_valid;
    a.dw = d_weights;
    a.dloss = d_loss;
    a.dlogits = d_logits;
    a.ldd = d_logits_stride;
    CUDA_TRY(launch_router_grad(a, (cudaStream_t)stream));
    return MOE_OK;
}

// ------------------------------------------------------------------ linear product
int moe_linear_config_validate(const moe_linear_config_t* cfg) { return check_linear(cfg); }

int moe_linear_plan(const moe_linear_config_t* cfg, moe_linear_plan_t* out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    const int v = check_linear(cfg);
    if (v != MOE_OK) return v;
    int dev = 0, major = 0, sms = 0;
    CUDA_TRY(cudaGetDevice(&dev));
    CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10) return MOE_ERR_UNSUPPORTED;
    if (!get_encode()) return MOE_ERR_CUDA;
    CUDA_TRY(linear_prepare(cfg->format));
    moe_linear_plan_s* p = new (std::nothrow) moe_linear_plan_s{*cfg, sms, DEFAULT_TIMEOUT_NS};
    if (!p) return MOE_ERR_CUDA;
    *out = p;
    return MOE_OK;
}

int moe_linear_plan_destroy(moe_linear_plan_t plan) {
    delete plan;
    return MOE_OK;
}

int moe_linear_set_wait_timeout(moe_linear_plan_t plan, uint64_t timeout_ns) {
    if (!plan) return MOE_ERR_INVALID_ARG;
    plan->timeout_ns = timeout_ns ? timeout_ns : DEFAULT_TIMEOUT_NS;
    return MOE_OK;
}

int moe_linear_weight_sf_size(moe_linear_plan_t plan, size_t* bytes) {
    if (!plan || !bytes) return MOE_ERR_INVALID_ARG;
    const moe_linear_config_t& c = plan->cfg;
    *bytes = (size_t)(stages_of(c.format, c.in_features) * wt_sf_blocks(c.out_features) * fmt_sf_atoms(c.format) *
                      ATOM_BYTES);
    return MOE_OK;
}

int moe_linear_transform_weight(moe_linear_plan_t plan, const moe_linear_weight_t* src, moe_linear_weight_t* dst,
                                void* stream) {
    if (!plan || !src || !dst || !src->codes || !src->sf || !dst->codes || !dst->sf || src->sf == dst->sf)
        return MOE_ERR_INVALID_ARG;
    const moe_linear_config_t& c = plan->cfg;
    const bool nv = c.format == MOE_FMT_NVFP4;
    if (nv != (src->global_scale != nullptr) || nv != (dst->global_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(dst->codes, 256) || !aligned_to(dst->sf, 256) || !aligned_to(src->global_scale, 4) ||
        !aligned_to(dst->global_scale, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (src->codes != dst->codes)
        CUDA_TRY(cudaMemcpyAsync(dst->codes, src->codes,
                                 (size_t)(c.out_features * fmt_row_bytes(c.format, c.in_features)),
                                 cudaMemcpyDeviceToDevice, st));
    if (nv && src->global_scale != dst->global_scale)
        CUDA_TRY(cudaMemcpyAsync(dst->global_scale, src->global_scale, 4, cudaMemcpyDeviceToDevice, st));
    CUDA_TRY(launch_pack_linear_sf((const uint8_t*)src->sf, (uint8_t*)dst->sf, c.format, c.out_features,
                                   c.in_features, st));
    return MOE_OK;
}

int moe_linear_workspace_size(moe_linear_plan_t plan, int32_t num_tokens, size_t* bytes) {
    if (!plan || !bytes || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens > plan->cfg.max_tokens) return MOE_ERR_CAPACITY;
    *bytes = (size_t)lin_layout(plan, num_tokens).total;
    return MOE_OK;
}

int moe_linear_forward(moe_linear_plan_t plan, int32_t num_tokens, const void* x, int64_t x_stride,
                       const moe_linear_weight_t* weight, void* out, int64_t out_stride, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const int v = check_forward(plan, num_tokens, weight, out, out_stride, workspace, workspace_bytes);
    if (v != MOE_OK || num_tokens == 0) return v;
    const moe_linear_config_t& c = plan->cfg;
    if (!x || !rows_ok(x, x_stride, num_tokens, c.in_features) || x == out) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* ws = (uint8_t*)workspace;
    const int64_t nks = stages_of(c.format, c.in_features);
    if (linear_quantises(c.format, linear_shape(num_tokens, c.out_features, (int)nks, plan->num_sms),
                         num_tokens, (int)nks, x, x_stride))
        return run_linear(plan, num_tokens, moe_quant_t{}, true, x, x_stride, weight, out, out_stride, workspace, st);
    const LinLayout L = lin_layout(plan, num_tokens);
    NormArgs a{};
    a.x = (const __nv_bfloat16*)x;
    a.ldx = x_stride;
    a.T = num_tokens;
    a.H = c.in_features;
    a.fmt = c.format;
    a.atoms = 1;
    a.nks = nks;
    a.codes = ws + L.codes;
    a.sf = ws + L.sf;
    a.row_scale = c.format == MOE_FMT_NVFP4 ? (float*)(ws + L.scale) : nullptr;
    CUDA_TRY(launch_norm(a, st));
    const moe_quant_t q{c.format, MOE_SF_ATOMS, a.codes, a.sf, a.row_scale};
    return run_linear(plan, num_tokens, q, false, nullptr, 0, weight, out, out_stride, workspace, st);
}

int moe_linear_forward_quantized(moe_linear_plan_t plan, int32_t num_tokens, const moe_quant_t* x,
                                 const moe_linear_weight_t* weight, void* out, int64_t out_stride, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    int v = check_forward(plan, num_tokens, weight, out, out_stride, workspace, workspace_bytes);
    if (v != MOE_OK || num_tokens == 0) return v;
    if (!x) return MOE_ERR_INVALID_ARG;
    if ((v = check_quant(x)) != MOE_OK) return v;
    if (x->format != plan->cfg.format || x->sf_layout != MOE_SF_ATOMS) return MOE_ERR_INVALID_ARG;
    return run_linear(plan, num_tokens, *x, true, nullptr, 0, weight, out, out_stride, workspace, (cudaStream_t)stream);
}

int moe_linear_last_status(moe_linear_plan_t plan, void* workspace, void* stream, int32_t* status) {
    if (!plan || !workspace || !status) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    // words[0]: how many CTAs the last product had (bounded: before the first one it may be anything)
    const int most = linear_max_ctas(plan->cfg.out_features, plan->num_sms);
    const int* words = (const int*)workspace;
    int ctas = 0, v = MOE_OK;
    CUDA_TRY(cudaMemcpyAsync(&ctas, words, sizeof(int), cudaMemcpyDeviceToHost, st));
    CUDA_TRY(cudaStreamSynchronize(st));
    ctas = ctas < 0 || ctas > most ? most : ctas;
    int part[512];
    for (int i = 0; i < ctas && v == MOE_OK; i += 512) {
        const int n = ctas - i < 512 ? ctas - i : 512;
        CUDA_TRY(cudaMemcpyAsync(part, words + 1 + i, n * sizeof(int), cudaMemcpyDeviceToHost, st));
        CUDA_TRY(cudaStreamSynchronize(st));
        for (int j = 0; j < n && v == MOE_OK; ++j) v = part[j];
    }
    CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), st));
    CUDA_TRY(cudaStreamSynchronize(st));
    *status = v;
    return MOE_OK;
}

}  // extern "C"
