// How the SMs are split between the own lists and the prefixes, how the lists,
// laid end to end, are split over the warps of k_own, and where k_finish finds a
// list's partials.
#pragma once

#include "moira_device.cuh"
#include "moira_launch.h"

namespace moira {

constexpr int kOwnMinPages = 2;                     // fewest pages a warp takes (fewer, longer partials to join)

// k_own and k_prefix run side by side, k_own on x of the SMs (its other blocks
// end at once, and k_prefix starts where they were), so that the call pays one
// start-up and one tail, and the bytes of one overlap the arithmetic of the
// other.  x is where the later of the two ends first, by their measured times:
// a start-up, then per SM 0.085 us a list page (100 GB/s, what an SM draws while
// k_prefix leaves it the memory) and 1.75 us a prefix tile of 128 keys, 3.1 us
// with more than 128 query rows.
// (32 requests behind 8k: 50 us one after the other, 45 us side by side; 256
// requests behind 32k: 263 us, 230 us.)
constexpr float kOwnStart = 14.f, kOwnPageTime = 0.085f;
constexpr float kPrefixStart = 13.f, kNarrowTime = 1.75f, kWideTime = 3.1f;

// The prefix work of one group in key tiles, of row tiles with at most and with
// more than 128 rows.
__device__ __forceinline__ int2 prefix_work(int requests, int len, int hkv)
{
    const int rows = requests * kGroup, full = rows / kUnitRows, rest = rows % kUnitRows;
    const int each = hkv * ((len + kTileKeys - 1) / kTileKeys);
    return make_int2(rest > 0 && rest <= kStreamRows ? each : 0, each * (full + (rest > kStreamRows)));
}

// Blocks of k_own for `pages` list entries beside that prefix work; every warp
// that calls it gets the same answer.
__device__ __forceinline__ int own_blocks(int pages, int2 work, int blocks)
{
    if (work.x + work.y == 0) return blocks;
    if (pages == 0) return 0;
    const float own = kOwnPageTime * static_cast<float>(pages);
    const float pre = kNarrowTime * static_cast<float>(work.x) + kWideTime * static_cast<float>(work.y);
    float best = INFINITY;
    int at = 1;
    // k_prefix keeps at least one team
    for (int x = 1 + (threadIdx.x & 31); x <= blocks - kMaxTeam; x += 32) {
        const float t = fmaxf(kOwnStart + __fdividef(own, static_cast<float>(x)),
                              kPrefixStart + __fdividef(pre, static_cast<float>(blocks - x)));
        if (t < best) {
            best = t;
            at = x;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, best, o);
        const int x = __shfl_xor_sync(0xffffffffu, at, o);
        if (t < best || (t == best && x < at)) {
            best = t;
            at = x;
        }
    }
    return at;
}

// n shares of W list entries; the first W % n have one entry more.  Share w's
// partial of list u lies at slot w + u.
struct OwnSplit {
    int n, q, rem;
    __device__ __forceinline__ OwnSplit(int W, int blocks)
    {
        n = min(blocks * kOwnWarps, (W + kOwnMinPages - 1) / kOwnMinPages);
        q = n > 0 ? W / n : 0;
        rem = n > 0 ? W - q * n : 0;
    }
    __device__ __forceinline__ int lo(int w) const { return w * q + min(w, rem); }
    __device__ __forceinline__ int share_of(int k) const
    {
        const int big = rem * (q + 1);
        return k < big ? k / (q + 1) : rem + (k - big) / q;
    }
};

}  // namespace moira
