// mhc_api_train.cpp -- the exported C entry points of the sub-layer's training operators:
// validation and dispatch, on the host before the first HIP call (no HIP header here, as in
// mhc_api.cpp).
#include <cstdint>

#include "../../include/mhc.h"
#include "mhc_glu_plan.h"
#include "mhc_plan.h"
#include "mhc_train_plan.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mhc_status status_of(int hip) { return hip == 0 ? MHC_OK : MHC_ERR_RUNTIME; }

bool is_x_dtype(int32_t d) { return d == MHC_DTYPE_BF16 || d == MHC_DTYPE_F16; }
bool is_row(int32_t D) { return D >= 8 && D % 8 == 0 && D <= mhc::kMaxD; }

mhc_status check_checkpoint(const mhc_checkpoint_params* p, const void* x, const void* codes, const void* scales)
{
    if (!p) return MHC_ERR_NULLPTR;
    if (!is_x_dtype(p->x_dtype) || !is_row(p->D) || p->rows < 0) return MHC_ERR_PARAM_INVALID;
    if (mhc::octet_blocks(p->rows, p->D) < 0) return MHC_ERR_PARAM_INVALID;
    if (p->rows == 0) return MHC_OK;
    if (!x || !codes || !scales) return MHC_ERR_NULLPTR;
    return aligned(x, 16) && aligned(codes, 16) ? MHC_OK : MHC_ERR_PARAM_INVALID;
}

mhc_status check_post(const mhc_post_params* p)
{
    if (p->T < 0 || (p->n != 4 && p->n != 6 && p->n != 8) || !is_row(p->D)) return MHC_ERR_PARAM_INVALID;
    if (!is_x_dtype(p->x_dtype) || p->reserved != 0) return MHC_ERR_PARAM_INVALID;
    return mhc::octet_blocks(p->T, p->D) < 0 ? MHC_ERR_PARAM_INVALID : MHC_OK;
}

mhc_status check_glu(const mhc_glu_params* p, mhc::glu::Geometry* g)
{
    if (!p) return MHC_ERR_NULLPTR;
    if (!is_x_dtype(p->x_dtype)) return MHC_ERR_PARAM_INVALID;
    if (!mhc::glu::make_geometry(p->T, p->D, p->F, p->act, p->x_dtype == MHC_DTYPE_F16, g)) return MHC_ERR_PARAM_INVALID;
    return MHC_OK;
}

}  // namespace

extern "C" {

mhc_status mhc_checkpoint(const mhc_checkpoint_params* params, const uint16_t* x, int8_t* codes, uint8_t* scales,
                          void* stream)
{
    const mhc_status st = check_checkpoint(params, x, codes, scales);
    if (st != MHC_OK || params->rows == 0) return st;
    return status_of(mhc::launch_checkpoint(params->rows, params->D, x, codes, scales,
                                            params->x_dtype == MHC_DTYPE_F16, stream));
}

mhc_status mhc_checkpoint_restore(const mhc_checkpoint_params* params, const int8_t* codes, const uint8_t* scales,
                                  uint16_t* x, void* stream)
{
    const mhc_status st = check_checkpoint(params, x, codes, scales);
    if (st != MHC_OK || params->rows == 0) return st;
    return status_of(mhc::launch_checkpoint_restore(params->rows, params->D, codes, scales, x,
                                                    params->x_dtype == MHC_DTYPE_F16, stream));
}

mhc_status mhc_post_checkpoint(const mhc_post_params* params, const mhc_post_tensors* t, int8_t* codes,
                               uint8_t* scales, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    const mhc_status st = check_post(params);
    if (st != MHC_OK || params->T == 0) return st;
    if (!t->x || !t->residual || !t->post || !t->comb || !t->out || !codes || !scales) return MHC_ERR_NULLPTR;
    if (!aligned(t->x, 16) || !aligned(t->residual, 16) || !aligned(t->out, 16) || !aligned(t->post, 4) ||
        !aligned(t->comb, 4) || !aligned(codes, 16))
        return MHC_ERR_PARAM_INVALID;
    return status_of(mhc::launch_post_checkpoint(params->T, params->n, params->D, t->x, t->residual, t->post, t->comb,
                                                 t->out, codes, scales, params->x_dtype == MHC_DTYPE_F16, stream));
}

mhc_status mhc_post_backward(const mhc_post_params* params, const mhc_post_bwd_tensors* t, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    const mhc_status st = check_post(params);
    if (st != MHC_OK || params->T == 0) return st;
    if (!t->grad_out || !t->post || !t->comb || !t->grad_x || !t->grad_residual || !t->grad_post || !t->grad_comb)
        return MHC_ERR_NULLPTR;
    if (t->x && (t->x_codes || t->x_scales)) return MHC_ERR_PARAM_INVALID;
    if (t->residual && (t->residual_codes || t->residual_scales)) return MHC_ERR_PARAM_INVALID;
    if (!t->x && (!t->x_codes || !t->x_scales)) return MHC_ERR_NULLPTR;
    if (!t->residual && (!t->residual_codes || !t->residual_scales)) return MHC_ERR_NULLPTR;
    const void* wide[] = {t->grad_out, t->x, t->residual, t->x_codes, t->residual_codes, t->grad_x, t->grad_residual};
    for (const void* q : wide)
        if (!aligned(q, 16)) return MHC_ERR_PARAM_INVALID;
    const void* f32s[] = {t->post, t->comb, t->grad_post, t->grad_comb};
    for (const void* q : f32s)
        if (!aligned(q, 4)) return MHC_ERR_PARAM_INVALID;
    const mhc::PostBwdArgs a = {t->grad_out, t->x, t->x_codes, t->x_scales, t->residual, t->residual_codes,
                                t->residual_scales, t->post, t->comb, t->grad_x, t->grad_residual, t->grad_post,
                                t->grad_comb};
    return status_of(mhc::launch_post_backward(params->T, params->n, params->D, a, params->x_dtype == MHC_DTYPE_F16,
                                               stream));
}

mhc_status mhc_glu(const mhc_glu_params* params, const mhc_glu_tensors* t, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    mhc::glu::Geometry g;
    const mhc_status st = check_glu(params, &g);
    if (st != MHC_OK) return st;
    if (!t->w_gate || !t->w_up || (g.T > 0 && (!t->x || !t->h))) return MHC_ERR_NULLPTR;
    if (!aligned(t->x, 16) || !aligned(t->w_gate, 16) || !aligned(t->w_up, 16) || !aligned(t->h, 16))
        return MHC_ERR_PARAM_INVALID;
    if (g.T == 0) return MHC_OK;
    mhc::glu::Args a = {};
    a.x = t->x;
    a.w_gate = t->w_gate;
    a.w_up = t->w_up;
    a.h = t->h;
    return status_of(mhc::glu::launch_glu(g, a, stream));
}

mhc_status mhc_glu_backward_workspace_size(const mhc_glu_params* params, int32_t from_checkpoint, size_t* bytes)
{
    if (!params || !bytes) return MHC_ERR_NULLPTR;
    mhc::glu::Geometry g;
    const mhc_status st = check_glu(params, &g);
    if (st != MHC_OK) return st;
    if (from_checkpoint != 0 && from_checkpoint != 1) return MHC_ERR_PARAM_INVALID;
    *bytes = mhc::glu::make_backward_plan(g, from_checkpoint == 1).ws_bytes;
    return MHC_OK;
}

mhc_status mhc_glu_backward(const mhc_glu_params* params, const mhc_glu_bwd_tensors* t, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    if (!params || !t) return MHC_ERR_NULLPTR;
    mhc::glu::Geometry g;
    const mhc_status st = check_glu(params, &g);
    if (st != MHC_OK) return st;
    if (!t->w_gate || !t->w_up || !t->grad_w_gate || !t->grad_w_up) return MHC_ERR_NULLPTR;
    const bool tok = g.T > 0, ck = t->x_codes || t->x_scales;
    if (tok && (!workspace || !t->grad_h || !t->grad_x)) return MHC_ERR_NULLPTR;
    if (t->x && ck) return MHC_ERR_PARAM_INVALID;
    if (tok && !t->x && (!t->x_codes || !t->x_scales)) return MHC_ERR_NULLPTR;
    const void* wide[] = {t->grad_h, t->x, t->x_codes, t->w_gate, t->w_up, t->grad_x, t->grad_w_gate, t->grad_w_up, t->h};
    for (const void* q : wide)
        if (!aligned(q, 16)) return MHC_ERR_PARAM_INVALID;
    const mhc::glu::BackwardPlan p = mhc::glu::make_backward_plan(g, ck);
    if (tok && (!aligned(workspace, 256) || workspace_bytes < p.ws_bytes)) return MHC_ERR_PARAM_INVALID;
    if (ck && mhc::octet_blocks(g.T, g.D) < 0) return MHC_ERR_PARAM_INVALID;
    char* const ws = static_cast<char*>(workspace);
    mhc::glu::Args a = {};
    a.x = t->x;
    a.w_gate = t->w_gate;
    a.w_up = t->w_up;
    a.h = t->h;
    a.grad_h = t->grad_h;
    a.grad_x = t->grad_x;
    a.grad_w_gate = t->grad_w_gate;
    a.grad_w_up = t->grad_w_up;
    if (tok) {
        a.dgu = reinterpret_cast<uint16_t*>(ws + p.off_dgu);
        a.part = reinterpret_cast<float*>(ws + p.off_part);
        if (ck) {
            uint16_t* const x = reinterpret_cast<uint16_t*>(ws + p.off_x);
            const int e = mhc::launch_checkpoint_restore(g.T, g.D, t->x_codes, t->x_scales, x, g.f16, stream);
            if (e != 0) return MHC_ERR_RUNTIME;
            a.x = x;
        }
    }
    return status_of(mhc::glu::launch_glu_backward(g, p, a, stream));
}

}  // extern "C"
