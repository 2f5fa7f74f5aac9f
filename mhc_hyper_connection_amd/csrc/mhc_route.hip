// mhc_route.hip -- gfx950 kernels of the routing to experts.
//
//   s = softmax(l) or sigmoid(l) over a token's E logits; choice c = s + bias
//   the k experts with the largest choice (with groups: of the top_groups groups whose group_top
//   largest choices have the largest sums), weights w_j = scale s_j (/ the sum of the chosen s)
//
// Two experts may be nearer to each other than fp32 tells, and the order of a choice is an exact
// result: that of fp64 scores, choices and sums. Without a bias the scores are ordered as
// the logits are, which are then compared themselves. Ties go to the lowest index.
// The choice is first made in fp32, with a bound on its error. Where two neighbours in the order are nearer than that,
// experts are taken on until one is surely the last, and those few are put in order by their fp64 values; where
// the last group in and the first one out are, or no expert is surely the last in time, the token's choice is made again
// in fp64. T = 16384, E = 256, top 8, 4 of 8 groups, sigmoid and bias: 20 us (all in fp64 35). Instructions bound it, not the 19 MB
// (3.7 us at a copy's rate): some 1700 vector instructions of a wave, four waves to a SIMD, which issues them 58 % of the time.
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
__device__ __forceinline__ uint32_t other(uint32_t v) { return (uint32_t)other<S>((int)v); }
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
constexpr float kInfF = __builtin_huge_valf();
constexpr float kU = 5.9604645e-8f;       // 2^-24

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v)
{
    return reduce<L>(v, [](uint32_t a, uint32_t b) { return max_u32(a, b); });
}
template <int L>
__device__ __forceinline__ float max_of(float v)
{
    return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
// What a wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void lds_of_the_wave() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Whole numbers that are ordered as floats are, and back.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k)
{
    return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// Largest first: Batcher's network over a power of two of registers.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&s)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = s[i + j], b = s[i + j + k];
                        s[i + j] = max_u32(a, b);
                        s[i + j + k] = a < b ? a : b;
                    }
}

// A token's logits in L lanes, V a lane (expert lane + L v), and what of them both choices need.
template <int L, int V>
struct Token {
    float l[V], b[V];       // -inf past E; the biases
    uint32_t off;           // masked experts, a bit for each v
    float top;              // the largest logit (0 where none is finite)
    int lane, slot;
};

// The choice in fp64. Lane j gets expert j of the order (and, with 16 lanes, j + 16); -1 where none is left.
template <int L, int V, bool GROUPS, int H>
__device__ __forceinline__ void choose_exactly(const RouteArgs& p, const Token<L, V>& k, double* row, int (&mine)[H])
{
    const bool softmax = p.score == kSoftmax, biased = p.t.bias != nullptr;
    double c[V];
    if (biased || GROUPS) {
        double sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double x = (double)k.l[v];
            c[v] = k.lane + L * v < p.E ? (softmax ? exp(x - (double)k.top) : 1.0 / (1.0 + exp(-x))) : 0.0;
            sum += c[v];
        }
        if (softmax) {
            sum = sum_of<L>(sum);
            sum = sum > 0 ? sum : 1.0;
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] /= sum;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool masked = (k.off >> v) & 1;
        if (biased) c[v] += (double)k.b[v];
        if (GROUPS) row[k.lane + L * v] = masked ? -kInf : c[v];
        if (!biased) c[v] = (double)k.l[v];
        if (masked) c[v] = -kInf;
    }
    if constexpr (GROUPS) {
        lds_of_the_wave();
        // a lane to a group: its largest, or the sum of its two largest
        double value = -kInf;
        if (k.lane < p.groups) {
            const double* const g = row + k.lane * p.per;
            double a = -kInf, b = -kInf;
            for (uint32_t i = 0; i < p.per; ++i) {
                const double x = g[i];
                b = fmax(b, fmin(a, x));
                a = fmax(a, x);
            }
            value = p.group_top == 2 && b > -kInf ? a + b : a;
        }
        uint32_t open = 0;
        for (int i = 0; i < p.top_groups; ++i) {
            const Best g = best_of<L>({value, k.lane});
            if (g.key > -kInf) open |= 1u << g.at;
            if (k.lane == g.at) value = -kInf;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t g = ((uint32_t)(k.lane + L * v) * p.magic) >> 20;
            if (!((open >> (g & 31)) & 1)) c[v] = -kInf;
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) mine[h] = -1;
    for (int j = 0; j < p.k; ++j) {
        Best b = {-kInf, kMaxE};
#pragma unroll
        for (int v = 0; v < V; ++v) better(b, c[v], k.lane + L * v);
        b = best_of<L>(b);
        if (b.key == -kInf) break;       // none left, for every lane of the token
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (k.lane + L * v == b.at) c[v] = -kInf;
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (j == k.lane + L * h) mine[h] = b.at;
    }
}

enum Found { kSure, kNear, kUnknown };   // in order; a set whose order fp64 has to say; neither

// The choice in fp32: the first n experts of its order, n >= p.k (or all that there are). A score is off by at most A 2^-24 (softmax: the exponentials'
// arguments, their sum of E terms and the division, 2 + 64 times the largest score; sigmoid: 8) and a choice by 2^-24 of
// itself more. A lane sorts its experts by one word each: the choice as an ordered whole number, whose last four bits (32
// 2^-24 of it) are the expert's place in the lane; of 16-bit logits alone all bits and the expert's number, so
// that their many ties are in order too. Then the lanes' first ones are compared, and the winning lane's list moves up.
template <int DT, int L, int V, bool GROUPS, int H>
__device__ __forceinline__ Found choose(const RouteArgs& p, const Token<L, V>& k, float* row, int (&mine)[H], int* n)
{
    const bool softmax = p.score == kSoftmax, biased = p.t.bias != nullptr, numbered = DT != kF32 && !biased;
    float c[V], A = 0.f;
    bool sure = true;
    if (biased || GROUPS) {
        A = 8.f;
        if (softmax) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                c[v] = __expf(k.l[v] - k.top);
                sum += c[v];
            }
            sum = sum_of<L>(sum);
            const float r = sum > 0.f ? 1.f / sum : 0.f;
            A = 2.f + 64.f * r;
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] *= r;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = __builtin_amdgcn_rcpf(1.f + __expf(-k.l[v]));
        }
    }
    uint32_t open = ~0u;
    if (biased)
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] += k.b[v];
    if constexpr (GROUPS) {
        const uint32_t wide = p.per + 4;      // groups four words apart, so that their lanes read different banks
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t e = (uint32_t)(k.lane + L * v), g = (e * p.magic) >> 20;
            if (e < (uint32_t)p.E) row[e + 4 * g] = (k.off >> v) & 1 ? -kInfF : c[v];
        }
        lds_of_the_wave();
        float value = -kInfF, size = 0.f;
        if (k.lane < p.groups) {
            const float* const g = row + k.lane * wide;
            float a = -kInfF, b = -kInfF;
            auto take = [&](float x) { b = __builtin_amdgcn_fmed3f(a, b, x), a = fmaxf(a, x); };   // b <= a
            uint32_t i = 0;
            if (p.per % 4 == 0)
                for (; i < p.per; i += 4) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(g + i);
                    take(x[0]), take(x[1]), take(x[2]), take(x[3]);
                }
            else
                for (; i < p.per; ++i) take(g[i]);
            const bool two = p.group_top == 2 && b > -kInfF;
            value = two ? a + b : a;
            size = value > -kInfF ? fabsf(a) + (two ? fabsf(b) : 0.f) : 0.f;
        }
        size = max_of<L>(size);
        open = 0;
        float least = kInfF;
        for (int i = 0; i <= p.top_groups; ++i) {
            const float m = max_of<L>(value);
            if (i == p.top_groups) {      // the first one out
                sure = m == -kInfF || least - m > kU * (4.f * A + 8.f * size);
                break;
            }
            if (m == -kInfF) break;
            least = m;
            const uint64_t who = __ballot(value == m) >> (threadIdx.x & (64 - L));
            const int at = __builtin_ctzll(who);   // of equal ones the first; another one, left out, is no surer than the bound
            open |= 1u << at;
            if (k.lane == at) value = -kInfF;
        }
    }
    uint32_t s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t e = (uint32_t)(k.lane + L * v);
        bool out = (k.off >> v) & 1;
        if (GROUPS) out |= !((open >> (((e * p.magic) >> 20) & 31)) & 1);
        if (numbered) {
            const float x = k.l[v] + 0.f;     // not -0
            const uint32_t u = DT == kF16 ? pack_f16x2(0.f, x) : __float_as_uint(x);
            s[v] = ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & 0xffff0000u) | (0xffffu - e);
        } else s[v] = (ordered(biased ? c[v] : k.l[v]) & ~15u) | (15u - v);
        s[v] = out ? 0u : s[v];
    }
    sort_down(s);
#pragma unroll
    for (int h = 0; h < H; ++h) mine[h] = -1;
    Found found = sure ? kSure : kUnknown;
    float last = 0.f;
    int j = 0;
    for (;; ++j) {
        const uint32_t m = max_of<L>(s[0]);
        if (m == 0 || (numbered && j == p.k)) break;
        bool won = s[0] == m;
        int e;
        if (numbered) e = (int)(0xffffu - (m & 0xffffu));
        else {
            const uint64_t who = (__ballot(won) >> (threadIdx.x & (64 - L))) & (L == 64 ? ~0ull : 0xffffull);
            const float now = from_ordered(m & ~15u);
            // surely behind the one before (1e-36: what the factors lose where they are subnormal)
            const bool apart = j == 0 || last - now > kU * (2.f * A + 40.f * fmaxf(fabsf(last), fabsf(now))) + 1e-36f;
            if (j >= p.k && apart) break;
            if (!apart && found == kSure) found = kNear;
            if (j == L * H) {
                found = kUnknown;
                break;
            }
            last = now;
            e = __builtin_ctzll(who);
            won = k.lane == e;               // of lanes with the same word the first; the next one is not apart from it
            e += L * (int)(15u - (m & 15u));
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (j == k.lane + L * h) mine[h] = e;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t up = v + 1 < V ? s[v + 1 < V ? v + 1 : 0] : 0u;
            asm("" : "+v"(up));              // a value: not a choice between two places of the array
            s[v] = won ? up : s[v];
        }
    }
    *n = j;
    return found;
}

// The n experts of `mine` in the order of their fp64 values. Each lane counts those before its own.
template <int L, int V, int H>
__device__ __forceinline__ void put_in_order(const RouteArgs& p, const Token<L, V>& k, const void* logits, int64_t row, float (*load)(const void*, int64_t), int n,
                                             int (&mine)[H])
{
    const bool softmax = p.score == kSoftmax, biased = p.t.bias != nullptr;
    double sum = 1;
    if (softmax && biased) {
        sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += k.lane + L * v < p.E ? exp((double)k.l[v] - (double)k.top) : 0.0;
        sum = sum_of<L>(sum);
    }
    double key[H];
    int before[H], at[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int e = mine[h];
        key[h] = -kInf;
        before[h] = 0;
        at[h] = -1;
        if (e >= 0) {
            key[h] = (double)load(logits, row + e);
            if (biased) key[h] = (softmax ? exp(key[h] - (double)k.top) / sum : 1.0 / (1.0 + exp(-key[h]))) + (double)p.t.bias[e];
        }
    }
    const int lane0 = (threadIdx.x & 63) - k.lane;
    for (int i = 0; i < n; ++i) {
        const int src = lane0 + i % L;
        const bool upper = H == 2 && i >= L;
        const double x = __shfl(upper ? key[H - 1] : key[0], src);
        const int e = __shfl(upper ? mine[H - 1] : mine[0], src);
#pragma unroll
        for (int h = 0; h < H; ++h) before[h] += x > key[h] || (x == key[h] && e < mine[h]) ? 1 : 0;
    }
    for (int i = 0; i < n; ++i) {
        const int src = lane0 + i % L;
        const bool upper = H == 2 && i >= L;
        const int place = __shfl(upper ? before[H - 1] : before[0], src), e = __shfl(upper ? mine[H - 1] : mine[0], src);
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (place == k.lane + L * h) at[h] = e;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) mine[h] = at[h];
}

// L lanes a token, V experts a lane (lane + L v): E <= L V.
template <int DT, int L, int V, bool GROUPS>
__global__ void __launch_bounds__(kThr)
route_kernel(RouteArgs p)
{
    constexpr int TOK = kThr / L, ROW = L * V + 4 * kMaxGroups;     // floats, or doubles, of a token's row
    __shared__ __attribute__((aligned(16))) double shared_c[GROUPS ? TOK * ROW : 1];
    Token<L, V> k;
    k.lane = threadIdx.x % L;
    k.slot = threadIdx.x / L;
    const int64_t t0 = (int64_t)blockIdx.x * TOK + k.slot;
    const bool live = t0 < p.T;
    const int64_t t = live ? t0 : p.T - 1;      // the lanes past the last token compute it again and store nothing
    const int E = p.E;
    const bool softmax = p.score == kSoftmax, biased = p.t.bias != nullptr;

    bool bad = false;
    k.top = -kInfF;
    k.off = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = k.lane + L * v;
        k.l[v] = e < E ? load_logit<DT>(p.t.logits, t * E + e) : -kInfF;
        k.b[v] = biased && e < E ? p.t.bias[e] : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bad |= k.l[v] != k.l[v] || k.b[v] != k.b[v];
        k.top = fmaxf(k.top, k.l[v]);
        if (!(k.l[v] > -kInfF) || k.b[v] == -kInfF) k.off |= 1u << v;
    }
    if (softmax) {
        k.top = max_of<L>(k.top);
        bad |= k.top == kInfF;
        if (!(k.top > -kInfF)) k.top = 0.f;
    }
    bad = any_of<L>(bad);

    // lane j keeps the experts j and, past L lanes of 16, j + 16
    constexpr int H = L == 16 ? 2 : 1;
    int mine[H];
    double* const row = shared_c + (GROUPS ? k.slot * ROW : 0);
    int n;
    Found found = choose<DT, L, V, GROUPS>(p, k, reinterpret_cast<float*>(row), mine, &n);
    if (bad) found = kSure;
    if (__ballot(found == kNear)) {
        int other[H];
#pragma unroll
        for (int h = 0; h < H; ++h) other[h] = mine[h];
        int most = found == kNear ? n : 0;       // tokens of a wave go through together
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_xor(most, d);
            most = most > o ? most : o;
        }
        put_in_order<L, V>(p, k, p.t.logits, t * E, load_logit<DT>, most, other);
#pragma unroll
        for (int h = 0; h < H; ++h) mine[h] = found == kNear ? other[h] : mine[h];
    }
    if (__ballot(found == kUnknown)) {
        int exact[H];
        choose_exactly<L, V, GROUPS>(p, k, row, exact);
#pragma unroll
        for (int h = 0; h < H; ++h) mine[h] = found == kUnknown ? exact[h] : mine[h];
    }
    // a set in order is as long as it had to be for that
#pragma unroll
    for (int h = 0; h < H; ++h)
        if (k.lane + L * h >= p.k) mine[h] = -1;

    // the weights, in fp64
    auto score = [&](float x) { return softmax ? exp((double)x - (double)k.top) : 1.0 / (1.0 + exp(-(double)x)); };
    double w[H], sum = 0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        w[h] = 0;
        if (h == 0 || p.k > L) {
            if (mine[h] >= 0) w[h] = score(load_logit<DT>(p.t.logits, t * E + mine[h]));
            sum += w[h];
        }
    }
    if (softmax && !p.renormalise) {
        sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += k.lane + L * v < E ? score(k.l[v]) : 0.0;
    }
    if (softmax || p.renormalise) {
        sum = sum_of<L>(sum);
        sum = sum > 0 ? sum : 1.0;
    } else sum = 1.0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int j = k.lane + L * h;
        if (live && j < p.k) {
            p.t.weights[t * p.k + j] = bad ? __builtin_nanf("") : (float)(w[h] / sum * p.scale);
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
// at the chosen experts, and zero elsewhere but in the last. The k terms are fp64, the other experts' scores of a
// softmax fp32. T = 16384, E = 256, top 8: 9.1 us, of which the 19 MB would take 3.6: the chosen experts' logits are
// read one by one before the row is written.
// EVERY: softmax without renormalisation.
template <int DT, int L, int V, bool EVERY>
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
    uint32_t chosen = 0;                 // of this lane's V experts
    double all[H];
#pragma unroll
    for (int h = 0; h < H; ++h) first[h] = e[h] >= 0, all[h] = d[h];
    for (int j = 0; j < k; ++j) {
        const int src = (threadIdx.x & 63) - lane + j % L;
        const int ej = __shfl(H == 2 && j >= L ? e[H - 1] : e[0], src);
        const double dj = __shfl(H == 2 && j >= L ? d[H - 1] : d[0], src);
        if (EVERY && ej >= 0 && ej % L == lane) chosen |= 1u << (ej / L);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int i = lane + L * h;
            if (ej == e[h] && j < i) first[h] = false;
            if (ej == e[h] && j > i) all[h] += dj;
        }
    }
    float s[V], sub = 0.f;
    if constexpr (EVERY) {
        float top = -__builtin_huge_valf(), rest = 0.f;
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
            rest += (chosen >> v) & 1 ? 0.f : s[v];
        }
        // A chosen expert's two terms nearly cancel where the router is sure of it: what is left is the other experts' part of the sum,
        // so the chosen ones' exponentials are fp64 in it and the others' fp32. (In fp32 throughout, with k = 1 and 1 - s = 5e-7, the
        // gradient was off by a tenth; T = 16384, E = 256, top 8: 11.0 us then, 12.2 now.)
        double x[H], total = 0;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            x[h] = first[h] ? exp((double)load_logit<DT>(p.t.logits, t * E + e[h]) - (double)top) : 0.0;
            total += x[h];
        }
        total = sum_of<L>(total) + (double)sum_of<L>(rest);
        const double each = total > 0 ? S * p.scale / total : 0.0;
#pragma unroll
        for (int h = 0; h < H; ++h) all[h] -= x[h] * each;
        sub = (float)each;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h)
        if (first[h]) row[slot][e[h]] = (float)all[h];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = lane + L * v;
        if (live && i < E) {
            const float r = EVERY && !((chosen >> v) & 1) ? 0.f - s[v] * sub : row[slot][i];
            store_grad<DT>(p.t.grad_logits, t * E + i, bad ? __builtin_nanf("") : r);
        }
    }
}

// --- the plan: 3.4 us to count and 8.4 to place 131072 pairs of 256 experts (1 MB), latency: a workgroup adds up the
// chunks' counts, 64 here, 16 loads at a time, and then places 64 pairs of each wave after the other. 8 pairs in one workgroup: 2.6 us. Wave w of a workgroup takes a contiguous part of its chunk, 64 pairs at a time in
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
    for (int w = 0; w < W; ++w)
        for (int e = tid; e <= E; e += kPlanThreads) n[w][e] = 0;
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
#pragma unroll 16
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int c = counts[(int64_t)b * (E + 1) + e];
                    before += b < (int)blockIdx.x ? c : 0;
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
    static_assert(kThr == 256 && (L == 16 || L == 64), "what the plan's bound on T assumes");
    const dim3 grid((unsigned)((p.T + kThr / L - 1) / (kThr / L))), block(kThr);
    if (backward && p.score == kSoftmax && !p.renormalise) hipLaunchKernelGGL((backward_kernel<DT, L, V, true>), grid, block, 0, st, p);
    else if (backward) hipLaunchKernelGGL((backward_kernel<DT, L, V, false>), grid, block, 0, st, p);
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
    if (g.E <= kFewExperts) return route_shape<DT, 16, 16>(p, groups, backward, st);
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
