// mhc_route_plan.h -- geometry and launch interface of the routing to experts: the choice of each
// token's experts with its backward, and the plan (the pairs sorted by expert).
//
// Host-side and plain C++ (no HIP headers), like mhc_plan.h.
#pragma once

#include <cstddef>
#include <cstdint>

namespace mhc {
namespace route {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kMaxGroups = 16;
constexpr int64_t kMaxT = (int64_t)1 << 26;
constexpr int64_t kMaxGrid = 0xffffff;            // workgroups of 256 threads within a grid's 2^32 - 1
constexpr int kFewExperts = 256;                  // up to here 16 lanes take a token, above 64
inline int64_t tokens_of_a_workgroup(int E) { return E <= kFewExperts ? 16 : 4; }
constexpr int64_t kMaxPairs = 0x7fffffff;         // pairs are numbered in 32 bits

enum Dtype { kBf16 = 0, kF16 = 1, kF32 = 2 };
enum Score { kSoftmax = 0, kSigmoid = 1 };

struct Geometry {
    int64_t T = 0;
    int E = 0, k = 0, groups = 1, top_groups = 1, group_top = 1;
    int score = 0, renormalise = 0, dtype = 0;
    double scale = 1;
};

inline bool make_geometry(int64_t T, int E, int k, int groups, int top_groups, int group_top, int score, int renormalise,
                          int dtype, double scale, Geometry* g)
{
    if (T < 0 || T > kMaxT || E < 1 || E > kMaxE || k < 1 || k > kMaxK || T * k > kMaxPairs) return false;
    if (T > kMaxGrid * tokens_of_a_workgroup(E)) return false;
    if (groups < 1 || groups > kMaxGroups || E % groups != 0 || top_groups < 1 || top_groups > groups) return false;
    if (k > E / groups * top_groups) return false;
    if (group_top != 1 && group_top != 2) return false;
    if (score != kSoftmax && score != kSigmoid) return false;
    if (renormalise != 0 && renormalise != 1) return false;
    if (dtype != kBf16 && dtype != kF16 && dtype != kF32) return false;
    if (!(scale > 0) || scale > 1e30) return false;
    *g = {T, E, k, groups, top_groups, group_top, score, renormalise, dtype, scale};
    return true;
}

struct Args {
    const void* logits;           // [T, E]
    const float* bias;            // [E] or NULL
    float* weights;               // [T, k]
    int32_t* experts;             // [T, k]
    // backward
    const float* grad_weights;    // [T, k]
    void* grad_logits;            // [T, E]
};

// The plan: a stable counting sort of P pairs by expert. One workgroup up to kPlanSmall pairs;
// above, one workgroup counts each chunk's experts, and one per chunk then adds up the chunks
// before it and places its pairs.
constexpr int kPlanThreads = 512;
constexpr int64_t kPlanSmall = 4096;
constexpr int64_t kPlanChunk = 2048;
constexpr int64_t kPlanChunks = 256;              // at most
struct Plan {
    int64_t pairs = 0, chunk = 0, chunks = 1;
    int E = 0;
    size_t ws_bytes = 0;                          // counts [chunks][E + 1]
};
inline bool make_plan(int64_t pairs, int E, Plan* p)
{
    if (pairs < 0 || pairs > kMaxPairs || E < 1 || E > kMaxE) return false;
    p->pairs = pairs;
    p->E = E;
    p->chunk = pairs;
    p->chunks = 1;
    p->ws_bytes = 0;
    if (pairs > kPlanSmall) {
        p->chunk = (pairs + kPlanChunks - 1) / kPlanChunks;
        if (p->chunk < kPlanChunk) p->chunk = kPlanChunk;
        p->chunks = (pairs + p->chunk - 1) / p->chunk;
        p->ws_bytes = (size_t)p->chunks * (size_t)(E + 1) * 4;
    }
    return true;
}

// Implemented in mhc_route.hip. Each returns 0 or the HIP error code.
int launch_route(const Geometry& g, const Args& a, void* stream);
int launch_route_backward(const Geometry& g, const Args& a, void* stream);
int launch_plan(const Plan& p, const int32_t* experts, int32_t* offsets, int32_t* pairs, int32_t* counts, void* stream);

}  // namespace route
}  // namespace mhc
