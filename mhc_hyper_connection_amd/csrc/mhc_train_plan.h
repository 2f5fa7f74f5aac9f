// mhc_train_plan.h -- geometry and launch interface of the sub-layer's training operators:
// the 8-bit checkpoints, hc_post with a checkpoint, and hc_post's backward.
//
// Host-side and plain C++ (no HIP headers), like mhc_plan.h.
#pragma once

#include <cstddef>
#include <cstdint>

namespace mhc {

constexpr int kCkptBlock = 32;       // values per scale

// Scale bytes of a row of D values.
inline int ckpt_blocks(int D) { return (D + kCkptBlock - 1) / kCkptBlock; }
// Octets of a row with its last block padded to a whole one: what the kernels that work on
// quads of lanes per block count in.
inline int ckpt_octets(int D) { return 4 * ckpt_blocks(D); }

// Workgroups of 256 threads over rows x padded octets, or -1 where that passes a grid's
// 2^32 - 1 threads.
inline int64_t octet_blocks(int64_t rows, int D)
{
    const int64_t P = ckpt_octets(D);
    if (rows > (int64_t)0xffffff * 256 / P) return -1;
    return (rows * P + 255) / 256;
}

// hc_post's backward: waves per token (4 or 1; mhc_post_bwd.hip has the rule's measurements),
// and the tokens of one launch, whose workgroups of 256 threads (a token, or four of one wave
// each) stay within a grid's 2^32 - 1 threads. More tokens go in several launches.
constexpr int64_t kPostBwdFewTokens = 512;
inline int post_bwd_waves(int64_t T, int n, int D) { return D >= 512 * n || T < kPostBwdFewTokens ? 4 : 1; }
inline int64_t post_bwd_launch_tokens(int waves) { return (int64_t)0xffffff * (4 / waves); }
inline int64_t post_bwd_blocks(int64_t tokens, int waves) { return waves == 1 ? (tokens + 3) / 4 : tokens; }

struct PostBwdArgs {
    const uint16_t* grad_out;      // [T, n, D]
    const uint16_t* x;             // [T, D], or NULL: x_codes, x_scales
    const int8_t* x_codes;
    const uint8_t* x_scales;
    const uint16_t* residual;      // [T, n, D], or NULL: r_codes, r_scales
    const int8_t* r_codes;
    const uint8_t* r_scales;
    const float* post;             // [T, n]
    const float* comb;             // [T, n, n]
    uint16_t* grad_x;              // [T, D]
    uint16_t* grad_residual;       // [T, n, D]
    float* grad_post;              // [T, n]
    float* grad_comb;              // [T, n, n]
};

// The arguments of the tokens behind the first t.
inline PostBwdArgs post_bwd_after(PostBwdArgs a, int64_t t, int n, int D)
{
    const int64_t row = t * D, rows = row * n, nb = t * ckpt_blocks(D);
    a.grad_out += rows;
    if (a.x) a.x += row;
    else {
        a.x_codes += row;
        a.x_scales += nb;
    }
    if (a.residual) a.residual += rows;
    else {
        a.r_codes += rows;
        a.r_scales += nb * n;
    }
    a.post += t * n;
    a.comb += t * n * n;
    a.grad_x += row;
    a.grad_residual += rows;
    a.grad_post += t * n;
    a.grad_comb += t * n * n;
    return a;
}

// Implemented in mhc_ckpt.hip and mhc_post_bwd.hip. Each returns 0 or the HIP error code.
int launch_checkpoint(int64_t rows, int D, const uint16_t* x, int8_t* codes, uint8_t* scales, int x_f16, void* stream);
int launch_checkpoint_restore(int64_t rows, int D, const int8_t* codes, const uint8_t* scales, uint16_t* x, int x_f16,
                              void* stream);
int launch_post_checkpoint(int64_t T, int n, int D, const uint16_t* x, const uint16_t* residual, const float* post,
                           const float* comb, uint16_t* out, int8_t* codes, uint8_t* scales, int x_f16, void* stream);
int launch_post_backward(int64_t T, int n, int D, const PostBwdArgs& a, int x_f16, void* stream);

}  // namespace mhc
