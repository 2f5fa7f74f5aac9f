// mhc_route.hip -- gfx950 kernels of the routing to experts.
//
//   s = softmax(l) or sigmoid(l) over a token's E logits; choice c = s + bias
//   the k experts with the largest choice (with groups: of the top_groups groups whose group_top
//   largest choices have the largest sums), weights w_j = scale s_j (/ the sum of the chosen s)
//
// Two experts may be nearer to each other than fp32 tells, and the order of a choice is an exact
// result: scores, choices and their sums are fp64. Without a bias the scores are ordered as
// the logits are, which are then compared themselves. Ties go to the lowest index.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_device.h"
#include "mhc_route_plan.h"

namespace mhc {
namespace route {
namespace {

constexpr int kThr = 256;
constexpr int kRowMirror = 0x140;

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i)
{
    if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
    else if constexpr (DT == kF16) return f16_lo(static_cast<const uint16_t*>(p)[i]);
    else return bf16_lo(static_cast<const uint16_t*>(p)[i]);
}

// A token belongs to L = 16 or 64 lanes. Lane exchanges among them: xor 1, 2, mirrored halves
// (4), mirrored rows (8) by DPP, 16 and 32 through the LDS crossbar.
template <int S>
__device__ __forceinline__ int other(int v)
{
    if constexpr (S == 0) return __builtin_amdgcn_update_dpp(0, v, kQuadXor1, 0xF, 0xF, true);
    else if constexpr (S == 1) return __builtin_amdgcn_update_dpp(0, v, kQuadXor2, 0xF, 0xF, true);
    else if constexpr (S == 2) return __builtin_amdgcn_update_dpp(0, v, kRowHalfMirror, 0xF, 0xF, true);
    else if constexpr (S == 3) return __builtin_amdgcn_update_dpp(0, v, kRowMirror, 0xF, 0xF, true);
    else return __shfl_xor(v, S == 4 ? 16 : 32);
}
template <int S>
__device__ __forceinline__ double other(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)other<S>((int)(uint32_t)u), hi = (uint32_t)other<S>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int S>
__device__ __forceinline__ float other(float v) { return __int_as_float(other<S>(__float_as_int(v))); }

// f(a, b) over the L lanes of a token, the same in each of them.
template <int L, typename V, typename F>
__device__ __forceinline__ V reduce(V v, F f)
{
    v = f(v, other<0>(v));
    v = f(v, other<1>(v));
    v = f(v, other<2>(v));
    v = f(v, other<3>(v));
    if constexpr (L == 64) {
        v = f(v, other<4>(v));
        v = f(v, other<5>(v));
    }
    return v;
}
template <int L, typename V>
__device__ __forceinline__ V sum_of(V v) { return reduce<L>(v, [](V a, V b) { return a + b; }); }

// The largest key and, among equal ones, the lowest index.
struct Best {
    double key;
    int at;
};
__device__ __forceinline__ void better(Best& b, double key, int at)
{
    const bool take = key > b.key || (key == b.key && at < b.at);
    b.key = take ? key : b.key;
    b.at = take ? at : b.at;
}
template <int L>
__device__ __forceinline__ Best best_of(Best b)
{
    better(b, other<0>(b.key), other<0>(b.at));
    better(b, other<1>(b.key), other<1>(b.at));
    better(b, other<2>(b.key), other<2>(b.at));
    better(b, other<3>(b.key), other<3>(b.at));
    if constexpr (L == 64) {
        better(b, other<4>(b.key), other<4>(b.at));
        better(b, other<5>(b.key), other<5>(b.at));
    }
    return b;
}
template <int L>
__device__ __forceinline__ bool any_of(bool v)
{
    const uint64_t m = __ballot(v);
    if constexpr (L == 64) return m != 0;
    else return ((m >> (threadIdx.x & 48)) & 0xffff) != 0;
}

struct RouteArgs {
    Args t;
    int64_t T;
    int E, k, groups, top_groups, group_top, score, renormalise;
    uint32_t per, magic;     // experts of a group; e / per = e magic >> 20
    double scale;
};

constexpr double kInf = __builtin_huge_val();

// L lanes a token, V experts a lane (lane + L v): E <= L V.
template <int DT, int L, int V, bool GROUPS>
__global__ void __launch_bounds__(kThr)
route_kernel(RouteArgs p)
{
    constexpr int TOK = kThr / L;
    __shared__ double shared_c[GROUPS ? TOK * L * V : 1];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t t0 = (int64_t)blockIdx.x * TOK + slot;
    const bool live = t0 < p.T;
    const int64_t t = live ? t0 : p.T - 1;      // the lanes past the last token compute it again and store nothing
    const int E = p.E;
    const bool softmax = p.score == kSoftmax, biased = p.t.bias != nullptr;

    float l[V];
    double c[V];
    bool bad = false;
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + L * v;
        l[v] = e < E ? load_logit<DT>(p.t.logits, t * E + e) : -__builtin_huge_valf();
        bad |= l[v] != l[v];
        top = fmaxf(top, l[v]);
    }
    double most = 0, total = 1;
    if (softmax) {
        top = reduce<L>(top, [](float a, float b) { return fmaxf(a, b); });
        bad |= top == __builtin_huge_valf();
        most = top > -__builtin_huge_valf() ? (double)top : 0.0;
    }
    auto raw = [&](float x) { return softmax ? exp((double)x - most) : 1.0 / (1.0 + exp(-(double)x)); };
    if (softmax || biased || GROUPS) {
        double sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = lane + L * v < E ? raw(l[v]) : 0.0;
            sum += c[v];
        }
        if (softmax) {
            total = sum_of<L>(sum);
            total = total > 0 ? total : 1.0;
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] /= total;
        }
    }
    // the choice; masked experts at -inf
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + L * v;
        bool masked = !(l[v] > -__builtin_huge_valf());
        if (biased && e < E) {
            const float b = p.t.bias[e];
            bad |= b != b;
            masked |= b == -__builtin_huge_valf();
            c[v] += (double)b;
        }
        if (GROUPS) shared_c[slot * (L * V) + e] = masked ? -kInf : c[v];
        if (!biased) c[v] = l[v];
        if (masked) c[v] = -kInf;
    }
    bad = any_of<L>(bad);

    if constexpr (GROUPS) {
        __syncthreads();
        // a lane to a group: its largest, or the sum of its two largest
        double value = -kInf;
        if (lane < p.groups) {
            const double* const row = shared_c + slot * (L * V) + lane * p.per;
            double a = -kInf, b = -kInf;
            for (uint32_t i = 0; i < p.per; ++i) {
                const double x = row[i];
                b = fmax(b, fmin(a, x));
                a = fmax(a, x);
            }
            value = p.group_top == 2 && b > -kInf ? a + b : a;
        }
        uint32_t open = 0;
        for (int i = 0; i < p.top_groups; ++i) {
            const Best g = best_of<L>({value, lane});
            if (g.key > -kInf) open |= 1u << g.at;
            if (lane == g.at) value = -kInf;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t g = ((uint32_t)(lane + L * v) * p.magic) >> 20;
            if (!((open >> (g & 31)) & 1)) c[v] = -kInf;
        }
    }

    // lane j keeps the experts j and, past L lanes of 16, j + 16
    constexpr int H = L == 16 ? 2 : 1;
    int mine[H];
#pragma unroll
    for (int h = 0; h < H; ++h) mine[h] = -1;
    for (int j = 0; j < p.k; ++j) {
        Best b = {-kInf, kMaxE};
#pragma unroll
        for (int v = 0; v < V; ++v) better(b, c[v], lane + L * v);
        b = best_of<L>(b);
        if (b.key == -kInf) break;       // none left, for every lane of the token
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + L * v == b.at) c[v] = -kInf;
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (j == lane + L * h) mine[h] = b.at;
    }
    double w[H], chosen = 0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        w[h] = mine[h] < 0 ? 0.0 : raw(load_logit<DT>(p.t.logits, t * E + mine[h])) / total;
        chosen += w[h];
    }
    if (p.renormalise) {
        chosen = sum_of<L>(chosen);
        chosen = chosen > 0 ? chosen : 1.0;
    } else chosen = 1.0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int j = lane + L * h;
        if (live && j < p.k) {
            p.t.weights[t * p.k + j] = bad ? __builtin_nanf("") : (float)(w[h] / chosen * p.scale);
            p.t.experts[t * p.k + j] = bad ? -1 : mine[h];
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_grad(void* out, int64_t i, float v)
{
    if constexpr (DT == kF32) static_cast<float*>(out)[i] = v;
    else static_cast<uint16_t*>(out)[i] = (uint16_t)(DT == kF16 ? pack_f16x2(v, 0.f) : f32_to_bf16_bits(v));
}

// With g = the weights' gradient, p_j = w_j / scale and S = sum_j g_j p_j:
//   softmax, renormalised   dl_j = w_j (g_j - S)
//   sigmoid, renormalised   dl_j = w_j (1 - s_j) (g_j - S)
//   sigmoid                 dl_j = w_j (1 - s_j) g_j
//   softmax                 dl_e = [e chosen] w_j g_j - s_e sum_j w_j g_j
// at the chosen experts, and zero elsewhere but in the last. The k terms are fp64, the rest of a
// softmax's row fp32.
template <int DT, int L, int V>
__global__ void __launch_bounds__(kThr)
backward_kernel(RouteArgs p)
{
    constexpr int TOK = kThr / L, H = L == 16 ? 2 : 1;
    __shared__ float row[TOK][L * V];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t t0 = (int64_t)blockIdx.x * TOK + slot;
    const bool live = t0 < p.T;
    const int64_t t = live ? t0 : p.T - 1;
    const int E = p.E, k = p.k;
    const bool softmax = p.score == kSoftmax;
#pragma unroll
    for (int v = 0; v < V; ++v) row[slot][lane + L * v] = 0.f;
    int e[H];
    double g[H], w[H], S = 0;
    bool bad = false;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int j = lane + L * h;
        e[h] = j < k ? p.t.experts[t * k + j] : -1;
        w[h] = j < k ? (double)p.t.weights[t * k + j] : 0.0;
        bad |= w[h] != w[h];             // a row that the forward found a NaN in
        if (e[h] < 0 || e[h] >= E) e[h] = -1, w[h] = 0.0;
        g[h] = e[h] < 0 ? 0.0 : (double)p.t.grad_weights[t * k + j];
        S += g[h] * (w[h] / p.scale);
    }
    bad = any_of<L>(bad);
    S = sum_of<L>(S);
    double d[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        d[h] = w[h] * (p.renormalise ? g[h] - S : g[h]);
        if (!softmax && e[h] >= 0) d[h] /= 1.0 + exp((double)load_logit<DT>(p.t.logits, t * E + e[h]));
    }
    // an expert that a token has more than once: its first slot adds up the later ones
    bool first[H];
    double all[H];
#pragma unroll
    for (int h = 0; h < H; ++h) first[h] = e[h] >= 0, all[h] = d[h];
    for (int j = 0; j < k; ++j) {
        const int src = (threadIdx.x & 63) - lane + j % L;
        const int ej = __shfl(H == 2 && j >= L ? e[H - 1] : e[0], src);
        const double dj = __shfl(H == 2 && j >= L ? d[H - 1] : d[0], src);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int i = lane + L * h;
            if (ej == e[h] && j < i) first[h] = false;
            if (ej == e[h] && j > i) all[h] += dj;
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h)
        if (first[h]) row[slot][e[h]] = (float)all[h];
    __syncthreads();
    float s[V], sub = 0.f;
    const bool every = softmax && !p.renormalise;
    if (every) {
        float top = -__builtin_huge_valf(), total = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = lane + L * v;
            s[v] = i < E ? load_logit<DT>(p.t.logits, t * E + i) : -__builtin_huge_valf();
            top = fmaxf(top, s[v]);
        }
        top = reduce<L>(top, [](float a, float b) { return fmaxf(a, b); });
        if (!(top > -__builtin_huge_valf())) top = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = expf(s[v] - top);
            total += s[v];
        }
        total = sum_of<L>(total);
        sub = total > 0.f ? (float)(S * p.scale) / total : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = lane + L * v;
        if (live && i < E) {
            const float r = every ? row[slot][i] - s[v] * sub : row[slot][i];
            store_grad<DT>(p.t.grad_logits, t * E + i, bad ? __builtin_nanf("") : r);
        }
    }
}

// --- the plan. Wave w of a workgroup takes a contiguous part of its chunk, 64 pairs at a time in
// order: the pairs of an expert keep their order, whatever runs when.

// Which lanes have this lane's value (of kBits bits).
constexpr int kBits = 11;                 // experts 0 .. 1023, and 1024 at most for "none"
__device__ __forceinline__ uint64_t same_as_mine(int v)
{
    uint64_t m = ~0ull;
#pragma unroll
    for (int b = 0; b < kBits; ++b) {
        const bool bit = (v >> b) & 1;
        const uint64_t on = __ballot(bit);
        m &= bit ? on : ~on;
    }
    return m;
}
// The expert of pair i, E for none (and for what is no expert).
__device__ __forceinline__ int expert_of(const int32_t* experts, int64_t i, int E)
{
    const int e = experts[i];
    return e < 0 || e >= E ? E : e;
}

__global__ void __launch_bounds__(kPlanThreads)
count_kernel(const int32_t* __restrict__ experts, int32_t* __restrict__ counts, int64_t P, int64_t chunk, int E)
{
    __shared__ int n[kMaxE + 1];
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) n[e] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < P ? i0 + chunk : P;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kPlanThreads) atomicAdd(&n[expert_of(experts, i, E)], 1);   // whole numbers: any order
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) counts[(int64_t)blockIdx.x * (E + 1) + e] = n[e];
}

// counts NULL: the only workgroup.
__global__ void __launch_bounds__(kPlanThreads)
place_kernel(const int32_t* __restrict__ experts, const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
             int32_t* __restrict__ pairs, int64_t P, int64_t chunk, int E)
{
    constexpr int W = kPlanThreads / 64;
    __shared__ int n[W][kMaxE + 1];       // a wave's counts, then where its next pair of an expert goes
    __shared__ int part[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < W * (kMaxE + 1); i += kPlanThreads) (&n[0][0])[i] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < P ? i0 + chunk : P;
    const int64_t run = ((i1 - i0 + W - 1) / W + 63) / 64 * 64;
    const int64_t w0 = i0 + wave * run, w1 = w0 + run < i1 ? w0 + run : i1;
    for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&n[wave][expert_of(experts, i, E)], 1);
    __syncthreads();
    // thread e (and e + threads, ..): pairs of expert e before this chunk and in all; their sums in the order of experts
    constexpr int M = (kMaxE + 1 + kPlanThreads - 1) / kPlanThreads;
    int carried = 0;                      // pairs of the experts before this round's
    for (int m = 0; m < M && m * kPlanThreads <= E; ++m) {
        const int e = m * kPlanThreads + tid;
        int before = 0, all = 0;
        if (e <= E) {
            if (counts) {
                for (int64_t b = 0; b < (int64_t)gridDim.x; ++b) {
                    const int c = counts[b * (E + 1) + e];
                    before += b < (int64_t)blockIdx.x ? c : 0;
                    all += c;
                }
            } else {
                for (int w = 0; w < W; ++w) all += n[w][e];
            }
        }
        int scan = all;                   // inclusive over the wave's lanes
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 63) part[wave] = scan;
        __syncthreads();
        int base = carried, round = 0;
        for (int w = 0; w < W; ++w) {
            if (w < wave) base += part[w];
            round += part[w];
        }
        const int begin = base + scan - all;
        if (e <= E) {
            if (blockIdx.x == 0) offsets[e] = begin;
            int at = begin + before;
            for (int w = 0; w < W; ++w) {
                const int c = n[w][e];
                n[w][e] = at;
                at += c;
            }
        }
        carried += round;
        __syncthreads();
    }
    for (int64_t g = w0; g < w1; g += 64) {
        const int64_t i = g + lane;
        const bool live = i < w1;
        const int e = live ? expert_of(experts, i, E) : 2047;
        const uint64_t same = same_as_mine(e);
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int at = 0;
        if (live) at = n[wave][e];
        // the wave's LDS accesses keep their order: all have read before the first of each expert adds
        __builtin_amdgcn_wave_barrier();
        if (live && rank == 0) n[wave][e] = at + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (live) pairs[at + rank] = (int32_t)i;
    }
}

template <int DT, int L, int V>
hipError_t route_shape(const RouteArgs& p, bool groups, bool backward, hipStream_t st)
{
    const dim3 grid((unsigned)((p.T + kThr / L - 1) / (kThr / L))), block(kThr);
    if (backward) hipLaunchKernelGGL((backward_kernel<DT, L, V>), grid, block, 0, st, p);
    else if (groups) hipLaunchKernelGGL((route_kernel<DT, L, V, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((route_kernel<DT, L, V, false>), grid, block, 0, st, p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch(const Geometry& g, const Args& a, bool backward, hipStream_t st)
{
    const uint32_t per = (uint32_t)(g.E / g.groups);
    const RouteArgs p = {a, g.T, g.E, g.k, g.groups, g.top_groups, g.group_top, g.score, g.renormalise,
                         per, ((1u << 20) + per - 1) / per, g.scale};
    const bool groups = g.groups > 1;
    if (g.E <= 64) return route_shape<DT, 16, 4>(p, groups, backward, st);
    if (g.E <= 128) return route_shape<DT, 16, 8>(p, groups, backward, st);
    if (g.E <= 256) return route_shape<DT, 16, 16>(p, groups, backward, st);
    if (g.E <= 512) return route_shape<DT, 64, 8>(p, groups, backward, st);
    return route_shape<DT, 64, 16>(p, groups, backward, st);
}

int launch_any(const Geometry& g, const Args& a, bool backward, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (g.dtype == kF32) return (int)launch<kF32>(g, a, backward, st);
    if (g.dtype == kF16) return (int)launch<kF16>(g, a, backward, st);
    return (int)launch<kBf16>(g, a, backward, st);
}

}  // namespace

int launch_route(const Geometry& g, const Args& a, void* stream) { return launch_any(g, a, false, stream); }
int launch_route_backward(const Geometry& g, const Args& a, void* stream) { return launch_any(g, a, true, stream); }

int launch_plan(const Plan& p, const int32_t* experts, int32_t* offsets, int32_t* pairs, int32_t* counts, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (p.chunks > 1) {
        hipLaunchKernelGGL(count_kernel, dim3((unsigned)p.chunks), dim3(kPlanThreads), 0, st, experts, counts, p.pairs, p.chunk, p.E);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
    }
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)p.chunks), dim3(kPlanThreads), 0, st, experts,
                       p.chunks > 1 ? counts : (const int32_t*)nullptr, offsets, pairs, p.pairs, p.chunk, p.E);
    return (int)hipGetLastError();
}

}  // namespace route
}  // namespace mhc
