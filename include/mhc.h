/*
 * mhc.h -- C ABI of the fused mHC pre-mapping forward, of the MhcPre backward, of hc_post
 * and its backward, of 8-bit activation checkpoints for the two backward passes, and of the
 * gated projection of the sub-layer in between, for AMD Instinct MI355X (gfx950).
 *
 * What one call computes, per token t (x viewed as xFlat of length K = n*D):
 *   invRms = (mean(xFlat^2) + normEps)^(-1/2)
 *   hMix   = (xFlat (.) gammaFlat) . phi^T            (gamma optional)
 *   w      = hMix * invRms, split [n, n, n*n] (alpha has 3 entries) or [n, n] (2 entries)
 *   hPre   = sigmoid(alpha0 * wPre + biasPre) + hcEps
 *   hPost  = 2 sigmoid(alpha1 * wPost + biasPost)   (+ hcEps when alpha has 2 entries)
 *   hRes   = Sinkhorn(alpha2 * wRes + biasRes)       (0 when alpha has 2 entries)
 *   hIn[d] = sum_i weight_i * x[i][d], weight = pre_mix[t] if given, else hPre
 * Sources:
 *   - aclnnMhcPreV2 guide (kwkr.cn/news/422178), section 3 (math semantics) and
 *     section 5 (inputs/outputs, optional outputs, shapes);
 *   - aclnnMhcPreSinkhorn guide (m.mzlw.cn/news/197063), section 3.2 (Sinkhorn steps:
 *     a row softmax + hcEps, then alternating column/row normalisations with + hcEps on
 *     every sum, 2*numIters steps, hRes = normOut[2*numIters-1]), section 4 (two-phase
 *     call), section 5.1 (needBackward outputs and their shapes), section 6 (error codes);
 *   - HcPre guide (mhpn.cn/news/2282827), function prototype (pre_mix, hc_pre output)
 *     and parameter defaults (numIters 20, normEps = hcEps = 1e-6).
 *
 * Layout and ownership. Every tensor is a caller-owned, contiguous, row-major device
 * buffer in the TND layout (a [B, S, n, D] input is the same bytes as [B*S, n, D]).
 * bf16 and fp16 tensors are passed as raw 16-bit patterns. The library allocates nothing
 * (the no-allocation entry point's array is static), never synchronises the stream except
 * where an entry point says so (mhc_pre_wait_status), and keeps between calls only what a
 * caller's workspace holds (call counters, which mhc_pre_workspace_size's buffer carries)
 * and, per device, facts it queries once (compute units, which kernels fit).
 *
 * Errors. Every entry point validates on the host before any HIP call and returns:
 *   MHC_OK                 success (also for T == 0: nothing is launched);
 *   MHC_ERR_NULLPTR        a required pointer is NULL;
 *   MHC_ERR_PARAM_INVALID  unsupported size or attribute, inconsistent output set,
 *                          misaligned pointer, or a buffer smaller than required;
 *   MHC_ERR_RUNTIME        a HIP call (kernel launch) failed.
 * The three codes have the values the aclnnMhcPreSinkhorn guide (section 6) lists for
 * the same three classes. Kernel faults surface at the caller's next synchronisation.
 */
#ifndef MHC_H
#define MHC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t mhc_status;

#define MHC_OK 0
#define MHC_ERR_NULLPTR 161001
#define MHC_ERR_PARAM_INVALID 161002
#define MHC_ERR_RUNTIME 361001

/* Problem description (host memory; read during the call only).
 *   T              tokens, >= 0
 *   n              hyper-streams (hcMult): 4, 6 or 8 (the aclnnMhcPreV2 guide, section 7.3,
 *                  allows these three; the MhcPreBackward guide, section 5, the same
 *                  three for the backward)
 *   D              hidden size per stream: a multiple of 8 in [8, 16384]; with n == 8 and
 *                  n_alpha == 3 at most 8192
 *   n_alpha        3 (pre/post/res branches, phi has n*n+2n rows) or
 *                  2 (pre/post only, phi has 2n rows, hRes = 0)
 *   num_iters      Sinkhorn iterations, >= 1 (ignored when n_alpha == 2)
 *   norm_eps       > 0 (RMS guard);  hc_eps >= 0 (gate / Sinkhorn guard)
 *   need_backward  0 or 1; with 1 the backward intermediates are mandatory outputs
 *   x_dtype        MHC_DTYPE_BF16 (0) or MHC_DTYPE_F16 (1): the 16-bit format of x and hIn
 *                  (the aclnnMhcPreSinkhorn and aclnnMhcPreV2 guides, section 5.1, list
 *                  BF16 and FLOAT16). With fp16 the weights are packed as three fp16 terms
 *                  scaled by 1, 2^11, 2^22 (phi * gamma must stay within 65504 in
 *                  magnitude); every forward path takes it, and the standalone stages
 *                  read and write fp16 too. hc_post takes either format (its own
 *                  x_dtype), and so does the backward (mhc_pre_bwd_params.x_f16). */
typedef struct mhc_pre_params {
    int64_t T;
    int32_t n;
    int32_t D;
    int32_t n_alpha;
    int32_t num_iters;
    double norm_eps;
    double hc_eps;
    int32_t need_backward;
    int32_t x_dtype;
} mhc_pre_params;

#define MHC_DTYPE_BF16 0
#define MHC_DTYPE_F16 1

/* Device pointers. M = n*n + 2n (n_alpha == 3) or 2n (n_alpha == 2); it = num_iters.
 * Inputs:
 *   x          x_dtype [T, n, D], 16-byte aligned                        required
 *   phi        f32  [M, n*D]                          required unless phi_packed is given
 *   alpha      f32  [n_alpha]                                            required
 *   bias       f32  [M]                                                  required
 *   gamma      f32  [n, D]          scales the projection input only     optional
 *   pre_mix    f32  [T, n]          hIn weights instead of hPre          optional
 *   phi_packed from mhc_pre_prepack for these (n, D, n_alpha, gamma)     optional; when
 *              given, phi and gamma are not read
 * Outputs (must not alias inputs or each other):
 *   h_in       x_dtype [T, D], 16-byte aligned                           required
 *   h_post     f32  [T, n]                                               required
 *   h_res      f32  [T, n, n]    required when n_alpha == 3; with n_alpha == 2 it may be
 *                                NULL, else it is filled with zeros
 *   inv_rms    f32  [T]          optional (required with need_backward)
 *   h_mix      f32  [T, M]       un-normalised projection; optional (required with need_backward)
 *   h_pre      f32  [T, n]       optional (required with need_backward)
 *   sum_out    f32  [2*it, T, n]       step-major Sinkhorn sums; only with n_alpha == 3;
 *                                optional (required with need_backward and n_alpha == 3);
 *                                plane 0 holds the row softmax denominators
 *   norm_out   f32  [2*it, T, n, n]    step-major Sinkhorn matrices; same rules as sum_out */
typedef struct mhc_pre_tensors {
    const uint16_t* x;
    const float* phi;
    const float* alpha;
    const float* bias;
    const float* gamma;
    const float* pre_mix;
    const void* phi_packed;
    uint16_t* h_in;
    float* h_post;
    float* h_res;
    float* inv_rms;
    float* h_mix;
    float* h_pre;
    float* sum_out;
    float* norm_out;
} mhc_pre_tensors;

/* Library version as major*10000 + minor*100 + patch. */
int mhc_version(void);

/* Static, human-readable text for a status code (never NULL). */
const char* mhc_status_string(mhc_status status);

/* Bytes of the packed projection weights for this problem (phi with gamma folded in,
 * split into three bf16 terms and ordered for the matrix cores). Host only; T is
 * ignored. Errors: NULLPTR, PARAM_INVALID. */
mhc_status mhc_pre_packed_size(const mhc_pre_params* params, size_t* bytes);

/* Bytes of device workspace mhc_pre_forward needs for this problem. Host only.
 * The workspace holds per-call intermediate results (partial sums, the hIn weights, the
 * values workgroups of the single-read kernel exchange) and, in its first 256 bytes, a
 * call counter that tags those exchanged values with the call that wrote them. Zero-fill
 * it once after allocating it and then leave it to the library; it may serve calls of
 * any size that fit it, one at a time. Concurrent calls need distinct workspaces.
 * Errors: NULLPTR, PARAM_INVALID. */
mhc_status mhc_pre_workspace_size(const mhc_pre_params* params, size_t* bytes);

/* Packs phi (f32 [M, n*D]) and the optional gamma (f32 [n, D]) into phi_packed
 * (device, >= mhc_pre_packed_size bytes, 16-byte aligned) asynchronously on `stream`
 * (a hipStream_t; NULL = the default stream). Weights are static across calls, so a
 * caller can pack once and pass phi_packed to every forward. T is ignored.
 * Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
mhc_status mhc_pre_prepack(const mhc_pre_params* params, const float* phi, const float* gamma,
                           void* phi_packed, size_t packed_bytes, void* stream);

/* The forward, asynchronous on `stream` (a hipStream_t; NULL = default stream). Emits
 * every non-NULL output listed in mhc_pre_tensors. `workspace` is device memory of at
 * least mhc_pre_workspace_size bytes, 256-byte aligned, zero-filled before its first use.
 * When tensors->phi_packed is NULL the weights are packed from phi (and gamma): by a pack
 * kernel into the workspace on the classic path, inside the kernel on the streaming,
 * single-read and one-launch paths. Then one of four kernel sequences
 * (mhc_pre_forward_path tells which):
 *   classic path: a projection kernel (which with pre_mix also writes hIn) and a
 *     per-token epilogue, which without pre_mix also writes hIn (x is read twice);
 *   streaming path (no pre_mix, D a multiple of 32, n == 4 with either alpha length or
 *     n == 6 or 8 with n_alpha == 2, where neither kernel below serves): the same
 *     epilogue (writing hIn) after a projection by persistent workgroups (one per
 *     compute unit) that keep their slice of the packed weights in LDS, read x in
 *     contiguous 1 KB runs of each token's row and load the next task's x while the
 *     current one is on the matrix cores;
 *   single-read path (n == 4, n_alpha == 3, no pre_mix, 992 < D <= 7168 (32 to 224
 *     blocks of 32 positions), T >= 8192, a device of 8 XCDs with 32 compute units each):
 *     one kernel computes the projection, hPre and hIn, x read once, then the per-token
 *     epilogue. Its workgroups (one per compute unit, in one group of 32 per XCD) wait on
 *     each other, each wait bounded: it needs every compute unit of an XCD at once, as an
 *     otherwise idle device gives; a wait that times out (other work holding compute
 *     units that long) leaves NaN in hIn for the tokens concerned, which
 *     mhc_pre_wait_status reports;
 *   one-launch path (n == 4, n_alpha == 3, no pre_mix, T <= 64, the device able to hold
 *     ceil(D / 32) workgroups of 256 threads at once): the whole forward in one kernel,
 *     one workgroup per block of 32 positions, which exchange their partial sums and hPre
 *     through the workspace (bounded waits, as above: a time-out leaves the token's
 *     outputs NaN, or only hIn when it comes at hPre, and mhc_pre_wait_status reports it).
 *   Every path takes bf16 or fp16 x.
 * Every path can be captured into a HIP graph.
 * The paths sum the projection's partial products in different groupings, so their
 * outputs may differ in the last bits; each meets the same accuracy. Within a call, hIn
 * uses exactly the hPre it emits. Results are bitwise reproducible for the same inputs,
 * parameters and path. The environment variable MHC_FORWARD_PATH = "classic" or
 * "fused" (for tests) overrides the choice: "classic" the classic path, "fused" the
 * single-read kernel where its geometry allows it (neither then takes the one-launch path;
 * "fused" falls back to the streaming or classic path elsewhere).
 * Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
mhc_status mhc_pre_forward(const mhc_pre_params* params, const mhc_pre_tensors* tensors,
                           void* workspace, size_t workspace_bytes, void* stream);

/* mhc_pre_forward for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same computation,
 * outputs and errors, without a workspace argument. The workspace is a device array of
 * 64 MiB that the library holds on every GPU it runs on, from the first such call on that
 * GPU (whose device must be current) to the end of the process; it is zero-filled when the
 * library is loaded and keeps the last call's contents. The call itself allocates nothing.
 * Every call on one GPU shares that GPU's array: calls that overlap on one GPU (different
 * streams, other host threads) race and must not be made. A problem whose
 * mhc_pre_workspace_size exceeds 64 MiB is rejected with MHC_ERR_PARAM_INVALID (it fits
 * up to 7808 tokens at n = 4, D = 7168; 12544 at D = 4096; 25216 at n = 8, D = 2048). The
 * wait-time-out flag of this workspace is not readable through mhc_pre_wait_status.
 * Errors: NULLPTR, PARAM_INVALID, RUNTIME (also when the array's address cannot be
 * obtained on the current device). */
mhc_status mhc_pre_forward_noalloc(const mhc_pre_params* params, const mhc_pre_tensors* tensors,
                                   void* stream);

/* Whether a single-read or one-launch forward that used `workspace` has given up one of
 * its waits since the last report. The single-read kernel's workgroups wait for values
 * other workgroups of their group publish, the one-launch kernel's for every workgroup at
 * its two barriers; each wait is bounded (about 0.3 s of polling), and one that gives up
 * leaves NaN in outputs of the tokens concerned (mhc_pre_forward has already
 * returned MHC_OK by then: it is asynchronous). This call synchronises `stream` (the stream
 * those forwards ran on; NULL = the default stream), then sets *timed_out to 1 if the
 * workspace's time-out flag is set, else 0, and clears the flag. In normal operation the
 * waits end by construction and the flag stays 0; it can be set when the workgroups that
 * wait for each other cannot all run at once (another workload holding compute units for
 * that long).
 *   workspace        the forward's workspace (>= 256 bytes, 256-byte aligned)
 *   workspace_bytes  its size
 * Errors: NULLPTR (workspace or timed_out), PARAM_INVALID (workspace too small or
 * misaligned), RUNTIME (a HIP call failed). */
mhc_status mhc_pre_wait_status(void* workspace, size_t workspace_bytes, void* stream, int32_t* timed_out);

/* Which path mhc_pre_forward would take for these parameters on the current device:
 * *path = 3 the streaming projection, 2 the one-launch kernel, 1 the single-read kernel,
 * 0 the classic path
 * (has_pre_mix: whether pre_mix
 * will be given). Errors: NULLPTR, PARAM_INVALID. */
mhc_status mhc_pre_forward_path(const mhc_pre_params* params, int32_t has_pre_mix, int32_t* path);

/* Events mhc_pre_forward_timed records: one before the first kernel and one after each
 * of the forward's four stages (weight pack, projection, epilogue, hIn). */
#define MHC_FORWARD_EVENTS 5

/* mhc_pre_forward, plus per-kernel timing: also records the caller's events (hipEvent_t
 * handles, created by the caller, who keeps ownership) on `stream`, in this order:
 *   events[0] before the weight-pack kernel,
 *   events[1] after it, before the projection kernel,
 *   events[2] after the projection kernel,
 *   events[3] after the per-token epilogue kernel,
 *   events[4] after the hIn stage, which launches no kernel on any forward path (the
 *     projection writes hIn with pre_mix and on the single-read path, the epilogue
 *     otherwise).
 * A stage the call does not launch a kernel for (the pack when phi_packed is given or on
 * the streaming, single-read and one-launch paths, which pack inside their kernel; the
 * epilogue on the one-launch path; the hIn stage always) has its two events recorded
 * back to back, so elapsed time between events[i] and events[i+1] is kernel i's duration
 * (plus the launch gap) whatever the inputs; with T == 0 all five are recorded back to
 * back. A NULL entry is not recorded: a caller that only wants some boundaries (each
 * record costs a few microseconds on the stream) passes NULL for the others. Computes
 * exactly what mhc_pre_forward computes.
 * Errors: as mhc_pre_forward; NULLPTR also for a NULL events array; PARAM_INVALID when
 * num_events != MHC_FORWARD_EVENTS. */
mhc_status mhc_pre_forward_timed(const mhc_pre_params* params, const mhc_pre_tensors* tensors,
                                 void* workspace, size_t workspace_bytes, void* stream,
                                 void* const* events, int32_t num_events);

/* ------------------------------------------------------------------ MhcPre backward
 *
 * The gradient of the MhcPre forward (aclnnMhcPreV2 guide, section 3: the same invRms,
 * hMix, gates and hIn as above, with hRes = alpha2 * wRes + biasRes, no Sinkhorn) with
 * respect to x, phi, alpha, bias and gamma, for the scalar whose gradients with respect to
 * hIn, hPost and hRes are given. Source: MhcPreBackward guide (0539edu.com/news/4871844),
 * section 3 (stages 3.1-3.8), section 6.1 (inputs and outputs), section 8.2 (shapes and
 * types: gradX takes gradHIn's type, the other gradients are float32, gradAlpha has 3
 * entries). Per token t, with s = hPre - hcEps and w = hMix * invRms:
 *   gHPre_i = sum_d gradHIn[d] x[i][d]
 *   gW      = [gHPre s(1-s) alpha0 | gradHPost hPost(1-hPost/2) alpha1 | gradHRes alpha2]
 *   gMix    = gW invRms;  gInv = sum_m gW[m] hMix[m]
 *   gradX   = gradHIn[d] hPre_i + (gMix . phi)[k] gamma[k] - gInv invRms^3 x[k] / (n D)
 *             + gradXPost[k]                                   (k = i D + d)
 *   gradPhi[m][k] = sum_t gMix[t][m] x[t][k] gamma[k];  gradGamma[k] = sum_t x[t][k] (gMix[t] . phi)[k]
 *   gradAlpha = sums over t of (gate term * w) per branch;  gradBias = sums of the gate terms
 * The RMS term uses raw x (invRms is defined on raw x); the guide writes x_rs there,
 * which is the same value when gamma is absent. Only the three-entry alpha (n*n + 2n phi
 * rows) has a backward (section 5 of the guide).
 *
 * With num_iters >= 1 the same call is the MhcPreSinkhorn backward: the forward's hRes
 * is then Sinkhorn(alpha2 * wRes + biasRes) (2 num_iters steps, as mhc_pre_forward
 * computes it), and the residual logits' gradient comes back through the forward's saved
 * sum_out / norm_out planes (the aclnnMhcPreSinkhorn guide, section 1, names that
 * backward and those inputs; it gives no formula). With G = gradHRes, for k = 2 it - 1
 * down to 1: a column step (k odd) passes back (G[r][c] - sum_r' G[r'][c] A_k[r'][c]) /
 * s_k[c], a row step (k even) the same along rows, with A_k = norm_out[k] and s_k =
 * sum_out[k]; the first step (row softmax + hcEps) passes back P (G - rowsum(G P)),
 * P = norm_out[0] - hcEps. That logit gradient takes gradHRes's place above.
 *
 * Problem description (host memory):
 *   T          tokens, 0 .. 67108860 (a wave of 64 threads each, in one grid)
 *   n          4, 6 or 8;  D  a multiple of 8 in [8, 16384]
 *   hc_eps     >= 0: the hcEps the forward used (hPre = sigmoid(...) + hcEps)
 *   num_iters  0: MhcPre backward (affine hRes); 1 .. 1000: MhcPreSinkhorn backward with
 *              that many Sinkhorn iterations
 *   x_f16      0: x, grad_h_in, grad_x_post and grad_x hold bf16; 1: all four hold fp16
 *              (IEEE binary16). The guide's section 8.2 gives gradX gradHIn's type, BF16
 *              or FP16. Other values: PARAM_INVALID. */
typedef struct mhc_pre_bwd_params {
    int64_t T;
    int32_t n;
    int32_t D;
    double hc_eps;
    int32_t num_iters;
    int32_t x_f16;
} mhc_pre_bwd_params;

/* Device pointers, M = n*n + 2n, K = n*D. Inputs (x, grad_h_in and grad_x_post 16-bit
 * values in the format x_f16 names, the rest float32):
 *   x            [T, n, D], 16-byte aligned                            required
 *   phi          [M, K]                                                required
 *   alpha        [3]                                                   required
 *   grad_h_in    [T, D], 16-byte aligned                               required
 *   grad_h_post  [T, n]                                                required
 *   grad_h_res   [T, n, n]                                             required
 *   inv_rms      [T]        the forward's saved invRms                  required
 *   h_mix        [T, M]     the forward's saved (un-normalised) hMix    required
 *   h_pre        [T, n]     the forward's saved hPre                    required
 *   h_post       [T, n]     the forward's saved hPost                   required
 *   gamma        [n, D]                                                optional
 *   grad_x_post  [T, n, D], 16-byte aligned: added to gradX            optional
 * Outputs (must not alias inputs or each other):
 *   grad_x       [T, n, D] in x's format, 16-byte aligned              required
 *   grad_phi     [M, K]                                                required
 *   grad_alpha   [3]                                                   required
 *   grad_bias    [M]                                                   required
 *   grad_gamma   [n, D]     required when gamma is given, else ignored
 * Saved Sinkhorn planes (inputs; required when num_iters >= 1, else ignored):
 *   sum_out      [2 it, T, n]       the forward's sum_out (step-major)
 *   norm_out     [2 it, T, n, n]    the forward's norm_out (step-major)
 * With T == 0 the per-token tensors (x, grad_h_in, grad_h_post, grad_h_res, inv_rms,
 * h_mix, h_pre, h_post, grad_x_post, grad_x, sum_out, norm_out) are empty and may be
 * NULL. */
typedef struct mhc_pre_bwd_tensors {
    const uint16_t* x;
    const float* phi;
    const float* alpha;
    const uint16_t* grad_h_in;
    const float* grad_h_post;
    const float* grad_h_res;
    const float* inv_rms;
    const float* h_mix;
    const float* h_pre;
    const float* h_post;
    const float* gamma;
    const uint16_t* grad_x_post;
    uint16_t* grad_x;
    float* grad_phi;
    float* grad_alpha;
    float* grad_bias;
    float* grad_gamma;
    const float* sum_out;
    const float* norm_out;
} mhc_pre_bwd_tensors;

/* Bytes of device workspace mhc_pre_backward needs. Host only. The workspace holds
 * per-call intermediates only (packed phi, per-token gradients, per-group partial sums)
 * and needs no initialisation. Errors: NULLPTR, PARAM_INVALID. */
mhc_status mhc_pre_backward_workspace_size(const mhc_pre_bwd_params* params, size_t* bytes);

/* The backward, asynchronous on `stream` (a hipStream_t; NULL = default stream).
 * `workspace`: device memory of at least mhc_pre_backward_workspace_size bytes, 256-byte
 * aligned. Every cross-token sum runs in a fixed order, so results are bitwise
 * reproducible for the same inputs. With T == 0, gradPhi, gradAlpha, gradBias and
 * gradGamma are set to zero. Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
mhc_status mhc_pre_backward(const mhc_pre_bwd_params* params, const mhc_pre_bwd_tensors* tensors,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ standalone stages
 *
 * The HcPre guide (mhpn.cn/news/2282827, "功能说明") splits the pre-mapping into
 * invRms, the mixing projection and the Sinkhorn stage, and names invRms and the Sinkhorn
 * stage as operators of their own; the Sinkhorn operator takes the mixes and the rsqrt as
 * inputs instead of computing them. These two entry points run those stages alone, on
 * the same per-token arithmetic as mhc_pre_forward; they serve callers that already hold
 * the mixes (a projection of their own) and tests that check one stage at a time.
 *
 * mhc_pre_inv_rms: inv_rms[t] = 1 / sqrt(mean over the n*D entries of x[t]^2 + norm_eps)
 * (the same reading of the mean as mhc_pre_forward; aclnnMhcPreV2 guide, section 3).
 * Squares and sums in fp64, one rounding to f32.
 *   params     validated as for mhc_pre_forward (T, n, D and norm_eps are used)
 *   x          x_dtype [T, n, D], 16-byte aligned
 *   inv_rms    f32  [T]
 * Pointers may be NULL only when T == 0. Asynchronous on `stream`, no workspace, no
 * allocation. Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
mhc_status mhc_pre_inv_rms(const mhc_pre_params* params, const uint16_t* x, float* inv_rms,
                           void* stream);

/* mhc_pre_sinkhorn: from the mixes hMix (the un-normalised projection, mhc_pre_forward's
 * h_mix) and invRms, everything the forward derives from them: hPre, hPost, the Sinkhorn
 * of the res logits with its planes, and hIn (aclnnMhcPreSinkhorn guide, m.mzlw.cn/news/
 * 197063, sections 3.1 and 3.2; aclnnMhcPreV2 guide, section 3). Outputs follow the rules
 * of mhc_pre_tensors, except that h_pre is always required (it carries the hIn weights
 * when pre_mix is not given).
 *   params     as for mhc_pre_forward; need_backward makes sum_out / norm_out mandatory
 *              (n_alpha == 3)
 * Inputs:  x x_dtype [T, n, D] (16-byte aligned), h_mix f32 [T, M], inv_rms f32 [T],
 *          alpha f32 [n_alpha], bias f32 [M], pre_mix f32 [T, n] (optional)
 * Outputs: h_in x_dtype [T, D] (16-byte aligned), h_pre, h_post f32 [T, n], h_res f32 [T, n, n]
 *          (required when n_alpha == 3), sum_out / norm_out as in mhc_pre_tensors
 * Pointers may be NULL only when T == 0. Asynchronous on `stream`, no workspace, no
 * allocation. Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
typedef struct mhc_pre_sinkhorn_tensors {
    const uint16_t* x;
    const float* h_mix;
    const float* inv_rms;
    const float* alpha;
    const float* bias;
    const float* pre_mix;
    uint16_t* h_in;
    float* h_pre;
    float* h_post;
    float* h_res;
    float* sum_out;
    float* norm_out;
} mhc_pre_sinkhorn_tensors;

mhc_status mhc_pre_sinkhorn(const mhc_pre_params* params, const mhc_pre_sinkhorn_tensors* tensors,
                            void* stream);

/* ------------------------------------------------------------------ hc_post
 *
 * The mHC post-mapping (HcPre guide, mhpn.cn/news/2282827, section "mHC 架构与 HcPre 的
 * 定位"): the layer output x is expanded back into the n streams by post (the forward's
 * hPost) and added to the streams fused across streams by comb (the forward's hRes):
 *     out[t][j][d] = post[t][j] x[t][d] + sum_i comb[t][i][j] residual[t][i][d]
 * This is the guide's printed broadcast expression evaluated on the [b, s, n, n] comb_frag
 * its section "返回值说明" documents: the sum runs over comb's first index, so output
 * stream j takes column j of comb (comb transposed times the residual streams). fp32 fused
 * multiply-adds (post term first, then i in order), one rounding to the 16-bit format.
 *   T >= 0; n: 4, 6 or 8; D: a multiple of 8 in [8, 16384]
 *   x        x_dtype [T, D]       16-byte aligned    (the attention / MLP output)
 *   residual x_dtype [T, n, D]    16-byte aligned    (the n streams)
 *   post     f32     [T, n]
 *   comb     f32     [T, n, n]
 *   out      x_dtype [T, n, D]    16-byte aligned; must not alias the inputs
 * Pointers may be NULL only when T == 0 (nothing is launched). Asynchronous on `stream`,
 * no workspace, no allocation. Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
typedef struct mhc_post_params {
    int64_t T;
    int32_t n;
    int32_t D;
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16: the format of x, residual and out */
    int32_t reserved;   /* must be 0 */
} mhc_post_params;

typedef struct mhc_post_tensors {
    const uint16_t* x;
    const uint16_t* residual;
    const float* post;
    const float* comb;
    uint16_t* out;
} mhc_post_tensors;

mhc_status mhc_post(const mhc_post_params* params, const mhc_post_tensors* tensors, void* stream);

/* ------------------------------------------------------------------ 8-bit checkpoints
 *
 * Activations kept from the forward to the backward pass in 8 bits: the n streams are the
 * largest tensors that an mHC layer keeps, n times a plain residual network's. A row of D
 * values is cut into blocks of 32 along D (the last may be shorter). With a = the largest
 * magnitude in a block, its step is 2^e, e = floor(log2 a) - 6, but not below -24 for fp16
 * (its least value) nor -126 for bf16 (its least normal value); a value's code is its
 * nearest multiple of the step (ties to even) within +-127, as a signed byte; the block's
 * scale byte is e + 127. A value is off by at most half a step (those above 127.5 steps by
 * less than a step): in all by at most a/128, or 2^-127 where that is more, as in bf16
 * blocks of a < 2^-120. code * step is exact in the 16-bit format it came from. A block
 * that holds a NaN or an infinity has the scale byte 255, and all its values come back
 * NaN. Scale bytes are 1 .. 248 and 255; a byte that the library did not write scales by
 * 2^(byte - 127) too (0 by zero), never out of bounds.
 *   rows      >= 0; D: a multiple of 8 in [8, 16384]
 *   x         x_dtype [rows, D], 16-byte aligned
 *   codes     int8    [rows, D], 16-byte aligned
 *   scales    uint8   [rows, ceil(D / 32)]
 * Pointers may be NULL only when rows == 0 (nothing is launched). Asynchronous on `stream`,
 * no workspace, no allocation; outputs must not alias inputs. Errors: NULLPTR,
 * PARAM_INVALID (also where rows hold more than 2^32 - 256 octets of values, each row
 * counted with its last block whole), RUNTIME. */
typedef struct mhc_checkpoint_params {
    int64_t rows;       /* T * n for the streams, T for a [T, D] tensor */
    int32_t D;
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16 */
} mhc_checkpoint_params;

/* x to codes and scales. */
mhc_status mhc_checkpoint(const mhc_checkpoint_params* params, const uint16_t* x, int8_t* codes, uint8_t* scales,
                          void* stream);

/* Codes and scales back to x_dtype values. */
mhc_status mhc_checkpoint_restore(const mhc_checkpoint_params* params, const int8_t* codes, const uint8_t* scales,
                                  uint16_t* x, void* stream);

/* mhc_post, bit for bit, and the checkpoint of its out (codes int8 [T, n, D], 16-byte
 * aligned; scales uint8 [T, n, ceil(D / 32)]) written from the same registers: what
 * mhc_checkpoint of out gives, without reading out again. Rules and errors as mhc_post's,
 * and PARAM_INVALID where a stream's T rows hold more than 2^32 - 256 octets, each row counted
 * with its last block whole (T = 2^30 - 64 is the most at D = 8). */
mhc_status mhc_post_checkpoint(const mhc_post_params* params, const mhc_post_tensors* tensors, int8_t* codes,
                               uint8_t* scales, void* stream);

/* mhc_pre_backward with x as its checkpoint (x_codes int8 [T, n, D], 16-byte aligned;
 * x_scales uint8 [T, n, ceil(D / 32)], of the format params->x_f16 names): bit for bit what
 * mhc_pre_backward gives for the restored x, without restoring it to memory. tensors->x
 * must be NULL. The same workspace; rules and errors otherwise as mhc_pre_backward's
 * (x_codes and x_scales may be NULL with T == 0). */
mhc_status mhc_pre_backward_checkpoint(const mhc_pre_bwd_params* params, const mhc_pre_bwd_tensors* tensors,
                                       const int8_t* x_codes, const uint8_t* x_scales, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ hc_post backward
 *
 * The gradients of mhc_post (out[t][j][d] = post[t][j] x[t][d] + sum_i comb[t][i][j]
 * residual[t][i][d]) for the scalar whose gradient with respect to out is grad_out:
 *   grad_x[t][d]           = sum_j post[t][j] grad_out[t][j][d]
 *   grad_residual[t][i][d] = sum_j comb[t][i][j] grad_out[t][j][d]
 *   grad_post[t][j]        = sum_d grad_out[t][j][d] x[t][d]
 *   grad_comb[t][i][j]     = sum_d residual[t][i][d] grad_out[t][j][d]
 * fp32 fused multiply-adds and sums in a fixed order (results are bitwise reproducible),
 * one rounding to the 16-bit format. grad_residual is what mhc_pre_backward takes as
 * grad_x_post, grad_post and grad_comb what it takes as grad_h_post and grad_h_res. x and
 * residual, each by itself, come as 16-bit tensors or as 8-bit checkpoints (the pointers of
 * the other form NULL).
 *   params as for mhc_post
 *   grad_out x_dtype [T, n, D]  16-byte aligned
 *   x        x_dtype [T, D]     16-byte aligned, or x_codes [T, D] (16-byte aligned) and
 *                               x_scales [T, ceil(D / 32)]
 *   residual x_dtype [T, n, D]  16-byte aligned, or residual_codes [T, n, D] (16-byte
 *                               aligned) and residual_scales [T, n, ceil(D / 32)]
 *   post f32 [T, n], comb f32 [T, n, n]
 *   grad_x x_dtype [T, D], grad_residual x_dtype [T, n, D] (16-byte aligned),
 *   grad_post f32 [T, n], grad_comb f32 [T, n, n]: outputs, which must not alias inputs or
 *   each other
 * Pointers may be NULL only when T == 0 (nothing is launched). Asynchronous on `stream`, no
 * workspace, no allocation. Errors: NULLPTR (neither form of x or of residual given, or a
 * checkpoint without its scales), PARAM_INVALID (both forms given, or more tokens than
 * mhc_post_checkpoint takes), RUNTIME. */
typedef struct mhc_post_bwd_tensors {
    const uint16_t* grad_out;
    const uint16_t* x;
    const uint16_t* residual;
    const int8_t* x_codes;
    const uint8_t* x_scales;
    const int8_t* residual_codes;
    const uint8_t* residual_scales;
    const float* post;
    const float* comb;
    uint16_t* grad_x;
    uint16_t* grad_residual;
    float* grad_post;
    float* grad_comb;
} mhc_post_bwd_tensors;

mhc_status mhc_post_backward(const mhc_post_params* params, const mhc_post_bwd_tensors* tensors, void* stream);

/* ------------------------------------------------------------------ gated projection
 *
 * The gated projection of a sub-layer's feed-forward block, between mhc_pre_forward (whose
 * hIn it takes) and mhc_post (which takes the block's result, after the projection back to
 * D, a plain matrix product of the caller's):
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) (.) u
 *   act(g) = g sigmoid(g)                                          (MHC_ACT_SILU)
 *            g sigmoid(2 sqrt(2/pi) (g + 0.044715 g^3))            (MHC_ACT_GELU_TANH: GELU's
 *                                                                   tanh form)
 * in one kernel: g and u stay in registers (fp32 sums of exact 16-bit products), one
 * rounding to h's format. Few tokens are bound by reading the weights, many by the matrix cores.
 *   T >= 0 tokens; D a multiple of 8 in [8, 16384]; F a multiple of 8 in [8, 65536];
 *   ceil(T / 128) * ceil(F / 64) < 2^23
 *   x      x_dtype [T, D]    w_gate, w_up x_dtype [F, D] (a row per result, as a linear
 *   layer keeps its weight)  h x_dtype [T, F]            all 16-byte aligned
 * With T == 0 nothing is launched, and x and h may be NULL. Asynchronous on `stream`, no
 * workspace, no allocation; results are bitwise reproducible for the same sizes. h must not
 * alias the inputs. Errors: NULLPTR, PARAM_INVALID, RUNTIME. */
#define MHC_ACT_SILU 0
#define MHC_ACT_GELU_TANH 1

typedef struct mhc_glu_params {
    int64_t T;
    int32_t D;
    int32_t F;
    int32_t act;        /* MHC_ACT_SILU or MHC_ACT_GELU_TANH */
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16: every tensor's format */
} mhc_glu_params;

typedef struct mhc_glu_tensors {
    const uint16_t* x;
    const uint16_t* w_gate;
    const uint16_t* w_up;
    uint16_t* h;
} mhc_glu_tensors;

mhc_status mhc_glu(const mhc_glu_params* params, const mhc_glu_tensors* tensors, void* stream);

/* Its backward, from x (or x's 8-bit checkpoint) and the weights alone: g and u are computed
 * again and never stored. With dh = grad_h,
 *   dg = dh (.) u (.) act'(g),  du = dh (.) act(g)         rounded once to x_dtype
 *   grad_x = dg Wg + du Wu,  grad_w_gate = dg^T x,  grad_w_up = du^T x
 * (fp32 sums, one rounding to x_dtype), and h again where asked for: the gradient of the
 * projection behind it needs it, so a caller need not keep it.
 * dg and du are operands of the matrix products and have x_dtype's precision and range, as
 * the gradient of a layer kept in that format has. The gradients carry two roundings, not
 * one: 2.3e-3 of their norm in bf16 and 2.9e-4 in fp16, where one is 1.7e-3 and 2.1e-4. In
 * fp16 a value of dg or du from 65520 on becomes infinite (then that token's grad_x, and
 * that f's rows of the weights' gradients, are infinite or NaN), below 6e-5 values are
 * multiples of 6e-8, and under 3e-8 they are zero: the loss scale that keeps grad_h in
 * fp16's range has to keep dh u act'(g) and dh act(g) there too. bf16 has fp32's range.
 *   grad_h x_dtype [T, F]; x x_dtype [T, D], or x_codes int8 [T, D] and x_scales uint8
 *   [T, ceil(D / 32)] (then x NULL; the values are restored into the workspace);
 *   w_gate, w_up x_dtype [F, D]; grad_x x_dtype [T, D]; grad_w_gate, grad_w_up x_dtype
 *   [F, D] (overwritten, not added to); h x_dtype [T, F] or NULL. All but x_scales 16-byte
 *   aligned; outputs must not alias inputs or each other.
 * With T == 0 the weights' gradients are set to zero, and the per-token tensors may be NULL.
 * The workspace (of mhc_glu_backward_workspace_size bytes, 256-byte aligned; from_checkpoint
 * 1 where x comes as its checkpoint, else 0) holds [dg | du], the restored x and partial
 * sums; it needs no initialisation, and calls that may overlap need distinct ones.
 * Asynchronous on `stream`; every sum in a fixed order. Errors: NULLPTR, PARAM_INVALID,
 * RUNTIME. */
typedef struct mhc_glu_bwd_tensors {
    const uint16_t* grad_h;
    const uint16_t* x;
    const int8_t* x_codes;
    const uint8_t* x_scales;
    const uint16_t* w_gate;
    const uint16_t* w_up;
    uint16_t* grad_x;
    uint16_t* grad_w_gate;
    uint16_t* grad_w_up;
    uint16_t* h;
} mhc_glu_bwd_tensors;

mhc_status mhc_glu_backward_workspace_size(const mhc_glu_params* params, int32_t from_checkpoint, size_t* bytes);

mhc_status mhc_glu_backward(const mhc_glu_params* params, const mhc_glu_bwd_tensors* tensors, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ routing to experts
 *
 * A sub-layer whose feed-forward block is a mixture of experts: each token goes to top_k of E
 * experts (gated projections of their own), whose results are added up by the token's weights.
 * mhc_route chooses them from the router's logits l (hIn times the router's weight, a plain
 * matrix product of the caller's):
 *   s = softmax(l) over the E logits (MHC_SCORE_SOFTMAX) or sigmoid(l) (MHC_SCORE_SIGMOID)
 *   c = s + bias                                  the choice; bias (optional) balances the load
 *   groups > 1: the experts are `groups` equal runs; a group's value is the sum of its
 *     group_top (1 or 2) largest c, and the top_groups groups of the largest values stay
 *   the top_k experts with the largest c of what stays, in descending order
 *   weights[j] = scale s_j, or with renormalise scale s_j / (the sum of the chosen s)
 * Ties go to the lowest index. Scores, choices and sums are fp64 (without a bias the logits, whose
 * order is that of the scores, are compared themselves), and each weight is rounded once.
 * An expert whose logit or bias is -inf is masked: it is never chosen (a masked logit has the score
 * 0; an expert masked by its bias still counts in the softmax). Where fewer than top_k experts
 * are left (none, say, for a padded token whose logits are all -inf), the remaining slots hold expert
 * -1 and weight 0; weights of scores that are all 0 are 0. A NaN among a token's logits
 * or the biases, or with softmax a logit of +inf, makes all its weights NaN and its experts -1.
 *   0 <= T <= 2^26 (2^26 - 4 for E > 256), T * top_k < 2^31; 1 <= E <= 1024; 1 <= groups <= 16, a divisor of E;
 *   1 <= top_groups <= groups; 1 <= top_k <= min(32, E / groups * top_groups); 0 < scale <= 1e30
 *   logits  logits_dtype [T, E]     bias f32 [E] or NULL     weights f32 [T, top_k]
 *   experts int32 [T, top_k]
 * Pointers may be NULL only when T == 0 (nothing is launched). Asynchronous on `stream`, no
 * workspace, no allocation; results are bitwise reproducible. Errors: NULLPTR, PARAM_INVALID,
 * RUNTIME. */
#define MHC_SCORE_SOFTMAX 0
#define MHC_SCORE_SIGMOID 1
#define MHC_DTYPE_F32 2

typedef struct mhc_route_params {
    int64_t T;
    int32_t E;
    int32_t top_k;
    int32_t groups;
    int32_t top_groups;
    int32_t group_top;
    int32_t score;          /* MHC_SCORE_SOFTMAX or MHC_SCORE_SIGMOID */
    int32_t renormalise;    /* 0 or 1 */
    int32_t logits_dtype;   /* MHC_DTYPE_BF16, MHC_DTYPE_F16 or MHC_DTYPE_F32 */
    double scale;
} mhc_route_params;

mhc_status mhc_route(const mhc_route_params* params, const void* logits, const float* bias, float* weights,
                     int32_t* experts, void* stream);

/* Its backward: the logits' gradient from the weights' (the choice itself has none, and nor
 * has the bias). With g = grad_weights, p_j = weights_j / scale and S = sum_j g_j p_j:
 *   softmax, renormalise   dl_j = weights_j (g_j - S)                 at the chosen experts
 *   sigmoid, renormalise   dl_j = weights_j (1 - s_j) (g_j - S)       at the chosen experts
 *   sigmoid                dl_j = weights_j (1 - s_j) g_j             at the chosen experts
 *   softmax                dl_e = [e chosen] weights_e g_e - s_e sum_j weights_j g_j
 * and zero elsewhere. Slots with an expert that is not in [0, E) count for nothing; a token
 * with a NaN weight gets NaN. Both terms of a token's slots are fp64, the scores of its other
 * experts and their part of the softmax's sum fp32, with one rounding to logits_dtype. An expert in two slots of a token gets their sum.
 *   params as in the forward (groups, top_groups and group_top are checked and not used)
 *   grad_weights f32 [T, top_k]; logits, weights, experts as in the forward;
 *   grad_logits logits_dtype [T, E]: overwritten, must not alias the inputs
 * Rules and errors as mhc_route's. */
mhc_status mhc_route_backward(const mhc_route_params* params, const float* grad_weights, const void* logits,
                              const float* weights, const int32_t* experts, void* grad_logits, void* stream);

/* What the experts' products read of a routing: the P = T * top_k pairs (token, slot), numbered
 * t * top_k + j, sorted by expert, each expert's in their order, the pairs without an expert (-1, or
 * any number outside [0, E)) last.
 *   0 <= P < 2^31; 1 <= E <= 1024
 *   experts int32 [P]
 *   offsets int32 [E + 1]: expert e has the sorted pairs [offsets[e], offsets[e + 1]); offsets[E] is
 *           where those without an expert begin
 *   pairs   int32 [P]
 * experts and pairs may be NULL when P == 0 (the offsets are then zeros). The workspace (of
 * mhc_experts_plan_workspace_size bytes, 0 for few pairs, 256-byte aligned) needs no
 * initialisation, and calls that may overlap need distinct ones. Asynchronous on `stream`, no
 * allocation; the result does not depend on the order of execution. Errors: NULLPTR,
 * PARAM_INVALID, RUNTIME. */
mhc_status mhc_experts_plan_workspace_size(int64_t P, int32_t E, size_t* bytes);

mhc_status mhc_experts_plan(int64_t P, int32_t E, const int32_t* experts, int32_t* offsets, int32_t* pairs,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ microscaled 4-bit floats
 *
 * Rows of D values in 4 bits each with one power of two for each block of 32 along D (the last may be
 * shorter). A code is e2m1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 for 0 .. 7, their negatives for 8 .. 15. With
 * a = the largest magnitude in a block, its step is 2^e with e the least exponent for which a is
 * under 7 steps (not below -127, nor above what keeps 6 steps finite: 13 for fp16, 125 for bf16); a
 * value's code is its nearest multiple's, ties to the even code, within +-6. Every value is off by at
 * most a / 5, or by 2^-129 where that is more (by a / 4 where a passes 7 steps of the largest e).
 * code * step is exact in the 16-bit format it came from. The scale byte is e + 127; 255 marks a
 * block that held a NaN or an infinity, whose values come back NaN and whose products are NaN.
 *   codes    uint8 [rows, 16 * ceil(D / 32)]: two to a byte, the even value's in the low half
 *   scales   uint8 [rows, 4 * ceil(D / 128)]: a row's in whole 32-bit words
 * Codes behind D and scale bytes behind the last block are written as zeros; the products take them for that
 * (a scale byte of 255 there would spoil its row).
 *   rows >= 0; 1 <= D <= 65536;  x x_dtype [rows, D], 16-byte aligned; codes 16-byte, scales
 *   4-byte aligned; rows * ceil(D / 128) * 16 <= 2^32 - 256
 * Pointers may be NULL only when rows == 0 (nothing is launched). Asynchronous on `stream`,
 * no workspace, no allocation; outputs must not alias inputs. Errors: NULLPTR,
 * PARAM_INVALID, RUNTIME. */
typedef struct mhc_mxfp4_params {
    int64_t rows;
    int32_t D;
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16 */
} mhc_mxfp4_params;

mhc_status mhc_mxfp4(const mhc_mxfp4_params* params, const uint16_t* x, uint8_t* codes, uint8_t* scales, void* stream);

mhc_status mhc_mxfp4_restore(const mhc_mxfp4_params* params, const uint8_t* codes, const uint8_t* scales, uint16_t* x,
                             void* stream);

/* ------------------------------------------------------------------ products with 4-bit weights
 *
 * y = x w^T, both in microscaled 4-bit floats on the matrix cores: sums in fp32 of products that are exact, one
 * rounding to x_dtype. For serving: there is no gradient of a rounding to 4 bits. x comes in 16
 * bits and is rounded to 4 as mhc_mxfp4 does, into the workspace or (few rows) within the product, or in 4 bits.
 *   T >= 0; 1 <= K <= 65536; N a multiple of 8 in [8, 65536]; T * 16 ceil(K / 32) < 2^31
 *   x x_dtype [T, K] (16-byte aligned), or x_codes and x_scales (as mhc_mxfp4 lays them out);
 *   w_codes [N, 16 ceil(K / 32)], w_scales [N, 4 ceil(K / 128)];
 *   y x_dtype [T, N], 16-byte aligned
 * With T == 0 nothing is launched, and x and y may be NULL. The workspace (256-byte aligned, of
 * mhc_mxfp4_product_workspace_size bytes, NULL if that is 0; x_mxfp4 1 where x comes in 4 bits, which needs
 * none, else 0) needs no initialisation, and calls that may overlap need distinct ones. Asynchronous on
 * `stream`, no allocation; every sum in a fixed order. y must not alias the inputs. Errors: NULLPTR
 * (neither form of x given, or codes without scales), PARAM_INVALID (both forms given), RUNTIME. */
typedef struct mhc_mxfp4_product_params {
    int64_t T;
    int32_t K;
    int32_t N;
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16: x's (where it is in 16 bits) and y's */
    int32_t reserved;   /* must be 0 */
} mhc_mxfp4_product_params;

typedef struct mhc_mxfp4_product_tensors {
    const uint16_t* x;
    const uint8_t* x_codes;
    const uint8_t* x_scales;
    const uint8_t* w_codes;
    const uint8_t* w_scales;
    uint16_t* y;
} mhc_mxfp4_product_tensors;

mhc_status mhc_mxfp4_product_workspace_size(const mhc_mxfp4_product_params* params, int32_t x_mxfp4, size_t* bytes);

mhc_status mhc_mxfp4_product(const mhc_mxfp4_product_params* params, const mhc_mxfp4_product_tensors* tensors,
                             void* workspace, size_t workspace_bytes, void* stream);

/* The experts' products, over the pairs of mhc_experts_plan:
 *   mhc_experts_glu    h[t, j] = act(x[t] Wg[e]^T) (.) (x[t] Wu[e]^T),  e = experts[t, j]
 *   mhc_experts_down   y[t] = sum_j weights[t, j] (h[t, j] Wd[e]^T)
 * with the weights of E experts in 4 bits, x and h in 16 bits (rounded to 4, as there) or in 4. act as
 * mhc_glu's. h is zero, and adds weights times zero, for pairs without an expert. Sums, activations and
 * the weighted sum (in the order of the slots) are fp32, with one rounding to x_dtype. With MHC_SHORT_TERMS added to
 * x_dtype mhc_experts_down may round the terms of a bf16 result before it adds them up, to 11 significant bits (bf16 has 8; from
 * 2^128 - 2^116 on they become infinite), or to 2^-39 of the largest finite one of 32 neighbours where that is more: less
 * time and workspace where there are many tokens. A NaN or an infinite term is that of its own column alone. A token's result does not
 * depend on the other tokens but through the sizes T, E and top_k, which choose the order of the sums.
 *   T >= 0, T * top_k < 2^31; 1 <= E <= 1024; 1 <= top_k <= 32; D, F multiples of 8 in [8, 65536];
 *   of x (T rows of D values) and h (T * top_k rows of F): rows * 16 ceil(width / 32) < 2^31;
 *   of mhc_experts_down: T * top_k * D < 2^35
 *   x x_dtype [T, D], or codes and scales      h x_dtype [T, top_k, F], or (down) codes and scales
 *   offsets int32 [E + 1], pairs int32 [T * top_k]   mhc_experts_plan's (pairs and offsets outside
 *   [0, T * top_k] are taken for none, never read through)
 *   w_gate, w_up [E, F, D], w_down [E, D, F]: codes [.., 16 ceil(width / 32)] and scales [.., 4
 *   ceil(width / 128)] along their last dimension
 *   weights f32 [T, top_k]      y x_dtype [T, D]
 * 16-bit tensors and codes 16-byte, the others 4-byte aligned. With T == 0 nothing is launched, and
 * the tensors of tokens and pairs may be NULL. Workspace, order and errors as mhc_mxfp4_product's (the
 * workspace of mhc_experts_down holds T * top_k results of D values in 32 bits, or 16 with MHC_SHORT_TERMS, too). */
#define MHC_SHORT_TERMS 0x100

typedef struct mhc_experts_params {
    int64_t T;
    int32_t E;
    int32_t top_k;
    int32_t D;
    int32_t F;
    int32_t act;        /* MHC_ACT_SILU or MHC_ACT_GELU_TANH (mhc_experts_down: not used, but checked) */
    int32_t x_dtype;    /* MHC_DTYPE_BF16 or MHC_DTYPE_F16 (mhc_experts_down: plus MHC_SHORT_TERMS or not) */
} mhc_experts_params;

typedef struct mhc_experts_glu_tensors {
    const uint16_t* x;
    const uint8_t* x_codes;
    const uint8_t* x_scales;
    const int32_t* offsets;
    const int32_t* pairs;
    const uint8_t* w_gate_codes;
    const uint8_t* w_gate_scales;
    const uint8_t* w_up_codes;
    const uint8_t* w_up_scales;
    uint16_t* h;
} mhc_experts_glu_tensors;

typedef struct mhc_experts_down_tensors {
    const uint16_t* h;
    const uint8_t* h_codes;
    const uint8_t* h_scales;
    const int32_t* offsets;
    const int32_t* pairs;
    const float* weights;
    const uint8_t* w_down_codes;
    const uint8_t* w_down_scales;
    uint16_t* y;
} mhc_experts_down_tensors;

mhc_status mhc_experts_glu_workspace_size(const mhc_experts_params* params, int32_t x_mxfp4, size_t* bytes);

mhc_status mhc_experts_glu(const mhc_experts_params* params, const mhc_experts_glu_tensors* tensors, void* workspace,
                           size_t workspace_bytes, void* stream);

mhc_status mhc_experts_down_workspace_size(const mhc_experts_params* params, int32_t h_mxfp4, size_t* bytes);

mhc_status mhc_experts_down(const mhc_experts_params* params, const mhc_experts_down_tensors* tensors, void* workspace,
                            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_H */
