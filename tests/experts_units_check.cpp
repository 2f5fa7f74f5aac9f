// Replays on the host how the products' kernels find their units from a plan's offsets, for offsets of any content: a unit is of
// rows that are there, its pairs are of its bucket, and units come in the order of their buckets; a plan's own units are all found, once.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "mhc_experts_plan.h"

using namespace mhc::experts;

static uint64_t state = 88172645463325252ull;
static uint64_t rnd(uint64_t n)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state % n;
}
static int fail(const char* what, long long a, long long b)
{
    printf("FAIL %s %lld %lld\n", what, a, b);
    return 1;
}

// `plan`: the offsets are a plan's
static int check(const std::vector<int32_t>& offsets, int64_t P, int BC, uint32_t na, bool plan)
{
    const int E = (int)offsets.size() - 1, most = most_units(P, BC, E);
    std::vector<int> before(E + 2), begin(E + 2), end(E + 2), units(E + 2);
    int at = 0;
    for (int e0 = 0; e0 <= E; e0 += 64) {                    // a wave's 64 buckets at a time
        int64_t scan = 0;
        for (int l = 0; l < 64; ++l) {
            int b, n;
            bucket_pairs(offsets.data(), E, (int)P, e0 + l, &b, &n);
            if (b < 0 || b > n || n > P) return fail("bucket", b, n);
            const int64_t tiles = ((int64_t)n - b + BC - 1) / BC;
            if (e0 + l <= E) {
                if (scan > 0x7fffffff - most) return fail("64 buckets past 32 bits", scan, most);
                before[e0 + l] = units_sum(at, (int)scan, most);
                begin[e0 + l] = b;
                end[e0 + l] = n;
                units[e0 + l] = (int)tiles;
            }
            scan += tiles;
        }
        if (scan > 0x7fffffff - most) return fail("64 buckets past 32 bits", scan, most);
        at = units_sum(at, (int)scan, most);
    }
    before[E + 1] = at;
    for (int e = 0; e <= E; ++e)
        if (before[e + 1] < before[e] || before[e + 1] - before[e] > units[e]) return fail("buckets' units", before[e], before[e + 1]);
    const int64_t total = (int64_t)at * na;
    if (total > 0x7fffffff) return fail("units past 32 bits", total, at);
    if (plan)
        for (int e = 0; e <= E; ++e)
            if (before[e + 1] - before[e] != units[e]) return fail("a plan's units", e, units[e]);
    const bool all = total < 20000;
    std::vector<char> seen(all ? (size_t)total : 0, 0);
    int last = 0;
    for (int64_t i = 0; i < (all ? total : 4000); ++i) {
        const uint32_t unit = (uint32_t)(all ? i : total * i / 4000 + (int64_t)rnd((uint64_t)(total / 4000)));
        int e;
        uint32_t a;
        int64_t first;
        find_unit(before.data(), begin.data(), E, na, BC, unit, &e, &a, &first);
        if (e < last || e > E) return fail("order of buckets", last, e);
        last = e;
        if (a >= na) return fail("rows", a, na);
        if (first < begin[e] || first >= end[e] || (first - begin[e]) % BC) return fail("pairs", first, e);
        if (all) {
            char& s = seen[(size_t)((before[e] + (first - begin[e]) / BC) * na + a)];
            if (s) return fail("twice", e, unit);
            s = 1;
        }
    }
    return 0;
}

int main()
{
    long long n = 0;
    for (int it = 0; it < 3000; ++it) {
        const int E = it % 50 == 0 ? 1024 : 1 + (int)rnd(it % 3 ? 20 : 300), BC = it % 2 ? 256 : 128;
        // up to 2^23 units in all, as the plan's check keeps them
        const uint32_t na = 1 + (uint32_t)rnd(it % 4 ? 40 : 1024);
        int64_t most = ((1 << 23) / na - E - 10) * (int64_t)BC;
        if (most > 0x7fffffff) most = 0x7fffffff;
        if (most < 1) continue;
        const int64_t P = 1 + (int64_t)rnd(it % 5 ? (most < 5000 ? most : 5000) : most);
        for (int kind = 0; kind < 5; ++kind) {
            std::vector<int32_t> o(E + 1);
            int64_t sum = 0;
            for (int e = 0; e <= E; ++e) {
                if (kind == 0) o[e] = (int32_t)sum, sum += (int64_t)rnd((uint64_t)(2 * P / E + 1)), sum = sum > P ? P : sum;      // a plan's
                else if (kind == 1) o[e] = e % 2 ? (int32_t)P : 0;                 // every pair in every other bucket
                else if (kind == 2) o[e] = (int32_t)rnd(0xffffffff);
                else if (kind == 3) o[e] = (int32_t)(P - P * e / E);               // descending
                else o[e] = (int32_t)rnd((uint64_t)P + 1);
            }
            if (check(o, P, BC, na, kind == 0)) return 1;
            ++n;
        }
    }
    // the most that valid() allows: every pair named 512 times over passes 32 bits
    for (int BC : {128, 256}) {
        const int64_t P = 0x7fffffff / 256 * BC < 0x7fffffff ? 0x7fffffff / 256 * (int64_t)BC : 0x7fffffff;
        std::vector<int32_t> o(1025);
        for (int e = 0; e <= 1024; ++e) o[e] = e % 2 ? (int32_t)P : 0;
        if (check(o, P, BC, 1, false)) return 1;
        ++n;
    }
    printf("ok %lld\n", n);
    return 0;
}
