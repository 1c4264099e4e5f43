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
// k_prefix leaves it the memory) and as much again a list, and 1.7 us a prefix
// tile of 128 keys, 2.5 us with more than 128 query rows (the slopes of a call's
// time in the prefix's length, 16k to 128k).
// (One after the other against side by side: 32 requests behind 8k 50 and 45 us,
// 256 behind 32k 263 and 230 us, with the kernels of the time, now 41 and 200 us.
// With no time for the lists, 256 requests of one own token behind 64k take
// 364 us instead of 302.)
constexpr float kOwnStart = 14.f, kOwnPageTime = 0.085f, kOwnListTime = 0.085f;
constexpr float kPrefixStart = 19.f, kNarrowTime = 1.7f, kWideTime = 2.5f;

// The prefix work of one group in key tiles, of row tiles with at most and with
// more than 128 rows.
__device__ __forceinline__ int2 prefix_work(int requests, int len, int hkv)
{
    const int rows = requests * kGroup, full = rows / kUnitRows, rest = rows % kUnitRows;
    const int each = hkv * ((len + kTileKeys - 1) / kTileKeys);
    return make_int2(rest > 0 && rest <= kStreamRows ? each : 0, each * (full + (rest > kStreamRows)));
}

// Blocks of k_own for `pages` entries of `lists` lists that have any beside that
// prefix work; every warp that calls it gets the same answer.
__device__ __forceinline__ int own_blocks(int pages, int lists, int2 work, int blocks)
{
    if (work.x + work.y == 0) return blocks;
    if (pages == 0) return 0;
    const float own = kOwnPageTime * static_cast<float>(pages) + kOwnListTime * static_cast<float>(lists);
    const float pre = kNarrowTime * static_cast<float>(work.x) + kWideTime * static_cast<float>(work.y);
    const float tiles = static_cast<float>(work.x + work.y), tile = __fdividef(pre, tiles), all = static_cast<float>(blocks);
    // where kOwnStart + own / x = kPrefixStart + pre / (all - x); lane i looks at
    // the i-th of the 32 counts around it, in whole tiles a block
    constexpr float d = kPrefixStart - kOwnStart;
    const float b = d * all + pre + own;
    const float x0 = __fdividef(2.f * own * all, b + sqrtf(fmaxf(b * b - 4.f * d * own * all, 0.f)));
    const int most = max(blocks - kMaxTeam, 1);                  // k_prefix keeps at least one team
    const int from = min(max(static_cast<int>(x0) - 15, 1), most);
    const int lane = threadIdx.x & 31, x = min(from + lane, most);
    const float t = fmaxf(kOwnStart + __fdividef(own, static_cast<float>(x)),
                          kPrefixStart + tile * ceilf(__fdividef(tiles, static_cast<float>(blocks - x))));
    const uint32_t key = static_cast<uint32_t>(fminf(t * 16.f, 67108863.f)) << 5 | lane;
    return min(from + static_cast<int>(__reduce_min_sync(0xffffffffu, key) & 31u), most);
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
