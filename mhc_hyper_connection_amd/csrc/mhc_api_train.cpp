// mhc_api_train.cpp -- the exported C entry points of the sub-layer's training operators:
// validation and dispatch, on the host before the first HIP call (no HIP header here, as in
// mhc_api.cpp).
#include <cstdint>

#include "../../include/mhc.h"
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

}  // extern "C"
