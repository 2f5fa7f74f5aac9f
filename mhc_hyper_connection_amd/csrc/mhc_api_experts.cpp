// mhc_api_experts.cpp -- the exported C entry points of the routing to experts, the microscaled 4-bit
// floats and the products with 4-bit weights: validation and dispatch, on the host before the
// first HIP call (no HIP header here, as in mhc_api.cpp).
#include <cstdint>

#include "../../include/mhc.h"
#include "mhc_experts_plan.h"
#include "mhc_mxfp4_plan.h"
#include "mhc_route_plan.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mhc_status status_of(int hip) { return hip == 0 ? MHC_OK : MHC_ERR_RUNTIME; }

bool is_x_dtype(int32_t d) { return d == MHC_DTYPE_BF16 || d == MHC_DTYPE_F16; }

mhc_status check_route(const mhc_route_params* p, mhc::route::Geometry* g)
{
    static_assert(MHC_DTYPE_BF16 == mhc::route::kBf16 && MHC_DTYPE_F16 == mhc::route::kF16 &&
                  MHC_DTYPE_F32 == mhc::route::kF32, "formats");
    if (!p) return MHC_ERR_NULLPTR;
    return mhc::route::make_geometry(p->T, p->E, p->top_k, p->groups, p->top_groups, p->group_top, p->score,
                                     p->renormalise, p->logits_dtype, p->scale, g)
               ? MHC_OK : MHC_ERR_PARAM_INVALID;
}

uintptr_t logit_bytes(const mhc::route::Geometry& g) { return g.dtype == mhc::route::kF32 ? 4 : 2; }

mhc_status check_mxfp4(const mhc_mxfp4_params* p, const void* x, const void* codes, const void* scales)
{
    if (!p) return MHC_ERR_NULLPTR;
    if (!is_x_dtype(p->x_dtype) || p->D < 1 || p->D > mhc::mx::kMaxD || p->rows < 0) return MHC_ERR_PARAM_INVALID;
    if (mhc::mx::octet_blocks(p->rows, p->D) < 0) return MHC_ERR_PARAM_INVALID;
    if (p->rows == 0) return MHC_OK;
    if (!x || !codes || !scales) return MHC_ERR_NULLPTR;
    return aligned(x, 16) && aligned(codes, 16) && aligned(scales, 4) ? MHC_OK : MHC_ERR_PARAM_INVALID;
}

using mhc::experts::Geometry;

mhc_status geometry_of(const mhc_mxfp4_product_params* p, Geometry* g)
{
    if (!p) return MHC_ERR_NULLPTR;
    if (!is_x_dtype(p->x_dtype) || p->reserved != 0) return MHC_ERR_PARAM_INVALID;
    g->op = mhc::experts::kProduct;
    g->P = g->X = p->T;
    g->K = p->K;
    g->R = p->N;
    g->f16 = p->x_dtype == MHC_DTYPE_F16;
    return mhc::experts::valid(*g) ? MHC_OK : MHC_ERR_PARAM_INVALID;
}
mhc_status geometry_of(const mhc_experts_params* p, bool down, Geometry* g)
{
    if (!p) return MHC_ERR_NULLPTR;
    const int32_t dtype = down ? p->x_dtype & ~MHC_SHORT_TERMS : p->x_dtype;
    if (!is_x_dtype(dtype) || p->T < 0 || p->T > 0x7fffffff || p->top_k < 1 || p->top_k > mhc::experts::kMaxTopK)
        return MHC_ERR_PARAM_INVALID;
    // both widths are rows of results of one of the two products
    if (p->D < 8 || p->D % 8 != 0 || p->F < 8 || p->F % 8 != 0) return MHC_ERR_PARAM_INVALID;
    g->op = down ? mhc::experts::kDown : mhc::experts::kGlu;
    g->P = p->T * p->top_k;
    g->X = down ? g->P : p->T;
    g->E = p->E;
    g->share = down ? 1 : p->top_k;
    g->K = down ? p->F : p->D;
    g->R = down ? p->D : p->F;
    g->act = p->act;
    g->f16 = dtype == MHC_DTYPE_F16;
    g->short_terms = dtype != p->x_dtype;
    return mhc::experts::valid(*g) ? MHC_OK : MHC_ERR_PARAM_INVALID;
}

mhc_status workspace_of(mhc_status st, const Geometry& g, int32_t in_4_bits, size_t* bytes)
{
    if (st != MHC_OK) return st;
    if (!bytes) return MHC_ERR_NULLPTR;
    if (in_4_bits != 0 && in_4_bits != 1) return MHC_ERR_PARAM_INVALID;
    *bytes = mhc::experts::make_workspace(g, in_4_bits == 0).bytes;
    return MHC_OK;
}

// The left operand in 16 bits (rounded to 4 into the workspace here) or in 4, and the launch.
struct Operand {
    const uint16_t* x;
    const uint8_t* codes;
    const uint8_t* scales;
};
mhc_status check_operand(const Operand& o, const void* out)
{
    if (o.x && (o.codes || o.scales)) return MHC_ERR_PARAM_INVALID;
    if (!o.x && (!o.codes || !o.scales)) return MHC_ERR_NULLPTR;
    if (!out) return MHC_ERR_NULLPTR;
    return aligned(o.x, 16) && aligned(o.codes, 16) && aligned(o.scales, 4) && aligned(out, 16) ? MHC_OK : MHC_ERR_PARAM_INVALID;
}
mhc_status run(const Geometry& g, const Operand& o, mhc::experts::Args a, void* workspace, size_t workspace_bytes, void* stream)
{
    const mhc::experts::Workspace w = mhc::experts::make_workspace(g, o.x != nullptr);
    if (w.bytes > 0) {
        if (!workspace) return MHC_ERR_NULLPTR;
        if (!aligned(workspace, 256) || workspace_bytes < w.bytes) return MHC_ERR_PARAM_INVALID;
    }
    char* const ws = static_cast<char*>(workspace);
    const mhc::experts::Tiling t = mhc::experts::make_tiling(g, o.x != nullptr);
    a.x_codes = o.codes;
    a.x_scales = o.scales;
    if (t.rounds_x) a.x = o.x;
    else if (o.x) {
        uint8_t* const codes = reinterpret_cast<uint8_t*>(ws + w.off_codes);
        uint8_t* const scales = reinterpret_cast<uint8_t*>(ws + w.off_scales);
        if (mhc::mx::launch_quantise(g.X, g.K, o.x, codes, scales, g.f16, stream) != 0) return MHC_ERR_RUNTIME;
        a.x_codes = codes;
        a.x_scales = scales;
    }
    if (g.op == mhc::experts::kDown) {
        a.part = ws + w.off_part;
        a.part_scales = reinterpret_cast<uint8_t*>(ws + w.off_part_scales);
    }
    return status_of(mhc::experts::launch_products(g, t, a, stream));
}

}  // namespace

extern "C" {

mhc_status mhc_route(const mhc_route_params* params, const void* logits, const float* bias, float* weights,
                     int32_t* experts, void* stream)
{
    mhc::route::Geometry g;
    const mhc_status st = check_route(params, &g);
    if (st != MHC_OK || g.T == 0) return st;
    if (!logits || !weights || !experts) return MHC_ERR_NULLPTR;
    if (!aligned(logits, logit_bytes(g)) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(experts, 4)) return MHC_ERR_PARAM_INVALID;
    mhc::route::Args a = {};
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.experts = experts;
    return status_of(mhc::route::launch_route(g, a, stream));
}

mhc_status mhc_route_backward(const mhc_route_params* params, const float* grad_weights, const void* logits,
                              const float* weights, const int32_t* experts, void* grad_logits, void* stream)
{
    mhc::route::Geometry g;
    const mhc_status st = check_route(params, &g);
    if (st != MHC_OK || g.T == 0) return st;
    if (!grad_weights || !logits || !weights || !experts || !grad_logits) return MHC_ERR_NULLPTR;
    if (!aligned(grad_weights, 4) || !aligned(weights, 4) || !aligned(experts, 4) || !aligned(logits, logit_bytes(g)) ||
        !aligned(grad_logits, logit_bytes(g)))
        return MHC_ERR_PARAM_INVALID;
    mhc::route::Args a = {};
    a.logits = logits;
    a.weights = const_cast<float*>(weights);
    a.experts = const_cast<int32_t*>(experts);
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    return status_of(mhc::route::launch_route_backward(g, a, stream));
}

mhc_status mhc_experts_plan_workspace_size(int64_t P, int32_t E, size_t* bytes)
{
    if (!bytes) return MHC_ERR_NULLPTR;
    mhc::route::Plan p;
    if (!mhc::route::make_plan(P, E, &p)) return MHC_ERR_PARAM_INVALID;
    *bytes = p.ws_bytes;
    return MHC_OK;
}

mhc_status mhc_experts_plan(int64_t P, int32_t E, const int32_t* experts, int32_t* offsets, int32_t* pairs,
                            void* workspace, size_t workspace_bytes, void* stream)
{
    mhc::route::Plan p;
    if (!mhc::route::make_plan(P, E, &p)) return MHC_ERR_PARAM_INVALID;
    if (!offsets || (P > 0 && (!experts || !pairs)) || (p.ws_bytes > 0 && !workspace)) return MHC_ERR_NULLPTR;
    if (!aligned(experts, 4) || !aligned(offsets, 4) || !aligned(pairs, 4)) return MHC_ERR_PARAM_INVALID;
    if (p.ws_bytes > 0 && (!aligned(workspace, 256) || workspace_bytes < p.ws_bytes)) return MHC_ERR_PARAM_INVALID;
    return status_of(mhc::route::launch_plan(p, experts, offsets, pairs, static_cast<int32_t*>(workspace), stream));
}

mhc_status mhc_mxfp4(const mhc_mxfp4_params* params, const uint16_t* x, uint8_t* codes, uint8_t* scales, void* stream)
{
    const mhc_status st = check_mxfp4(params, x, codes, scales);
    if (st != MHC_OK || params->rows == 0) return st;
    return status_of(mhc::mx::launch_quantise(params->rows, params->D, x, codes, scales, params->x_dtype == MHC_DTYPE_F16, stream));
}

mhc_status mhc_mxfp4_restore(const mhc_mxfp4_params* params, const uint8_t* codes, const uint8_t* scales, uint16_t* x,
                             void* stream)
{
    const mhc_status st = check_mxfp4(params, x, codes, scales);
    if (st != MHC_OK || params->rows == 0) return st;
    return status_of(mhc::mx::launch_restore(params->rows, params->D, codes, scales, x, params->x_dtype == MHC_DTYPE_F16, stream));
}

mhc_status mhc_mxfp4_product_workspace_size(const mhc_mxfp4_product_params* params, int32_t x_mxfp4, size_t* bytes)
{
    Geometry g;
    const mhc_status st = geometry_of(params, &g);
    return workspace_of(st, g, x_mxfp4, bytes);
}

mhc_status mhc_mxfp4_product(const mhc_mxfp4_product_params* params, const mhc_mxfp4_product_tensors* t, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    Geometry g;
    mhc_status st = geometry_of(params, &g);
    if (st != MHC_OK) return st;
    if (!t->w_codes || !t->w_scales) return MHC_ERR_NULLPTR;
    if (!aligned(t->w_codes, 16) || !aligned(t->w_scales, 4)) return MHC_ERR_PARAM_INVALID;
    if (g.P == 0) return MHC_OK;
    const Operand o = {t->x, t->x_codes, t->x_scales};
    st = check_operand(o, t->y);
    if (st != MHC_OK) return st;
    mhc::experts::Args a = {};
    a.w_codes[0] = t->w_codes;
    a.w_scales[0] = t->w_scales;
    a.out = t->y;
    return run(g, o, a, workspace, workspace_bytes, stream);
}

mhc_status mhc_experts_glu_workspace_size(const mhc_experts_params* params, int32_t x_mxfp4, size_t* bytes)
{
    Geometry g;
    const mhc_status st = geometry_of(params, false, &g);
    return workspace_of(st, g, x_mxfp4, bytes);
}

mhc_status mhc_experts_glu(const mhc_experts_params* params, const mhc_experts_glu_tensors* t, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    Geometry g;
    mhc_status st = geometry_of(params, false, &g);
    if (st != MHC_OK) return st;
    if (!t->w_gate_codes || !t->w_gate_scales || !t->w_up_codes || !t->w_up_scales) return MHC_ERR_NULLPTR;
    if (!aligned(t->w_gate_codes, 16) || !aligned(t->w_up_codes, 16) || !aligned(t->w_gate_scales, 4) ||
        !aligned(t->w_up_scales, 4))
        return MHC_ERR_PARAM_INVALID;
    if (g.P == 0) return MHC_OK;
    if (!t->offsets || !t->pairs) return MHC_ERR_NULLPTR;
    if (!aligned(t->offsets, 4) || !aligned(t->pairs, 4)) return MHC_ERR_PARAM_INVALID;
    const Operand o = {t->x, t->x_codes, t->x_scales};
    st = check_operand(o, t->h);
    if (st != MHC_OK) return st;
    mhc::experts::Args a = {};
    a.w_codes[0] = t->w_gate_codes;
    a.w_codes[1] = t->w_up_codes;
    a.w_scales[0] = t->w_gate_scales;
    a.w_scales[1] = t->w_up_scales;
    a.offsets = t->offsets;
    a.pairs = t->pairs;
    a.out = t->h;
    return run(g, o, a, workspace, workspace_bytes, stream);
}

mhc_status mhc_experts_down_workspace_size(const mhc_experts_params* params, int32_t h_mxfp4, size_t* bytes)
{
    Geometry g;
    const mhc_status st = geometry_of(params, true, &g);
    return workspace_of(st, g, h_mxfp4, bytes);
}

mhc_status mhc_experts_down(const mhc_experts_params* params, const mhc_experts_down_tensors* t, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    Geometry g;
    mhc_status st = geometry_of(params, true, &g);
    if (st != MHC_OK) return st;
    if (!t->w_down_codes || !t->w_down_scales) return MHC_ERR_NULLPTR;
    if (!aligned(t->w_down_codes, 16) || !aligned(t->w_down_scales, 4)) return MHC_ERR_PARAM_INVALID;
    if (g.P == 0) return MHC_OK;
    if (!t->offsets || !t->pairs || !t->weights) return MHC_ERR_NULLPTR;
    if (!aligned(t->offsets, 4) || !aligned(t->pairs, 4) || !aligned(t->weights, 4)) return MHC_ERR_PARAM_INVALID;
    const Operand o = {t->h, t->h_codes, t->h_scales};
    st = check_operand(o, t->y);
    if (st != MHC_OK) return st;
    mhc::experts::Args a = {};
    a.w_codes[0] = t->w_down_codes;
    a.w_scales[0] = t->w_down_scales;
    a.offsets = t->offsets;
    a.pairs = t->pairs;
    a.weights = t->weights;
    a.out = t->y;
    a.top_k = params->top_k;
    return run(g, o, a, workspace, workspace_bytes, stream);
}

}  // extern "C"
