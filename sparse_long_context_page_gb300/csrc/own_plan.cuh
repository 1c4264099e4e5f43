// How the own lists, laid end to end, are split over the warps of k_own, and
// where k_finish finds a list's partials.
#pragma once

#include "moira_device.cuh"

namespace moira {

constexpr int kOwnMinPages = 2;                     // fewest pages a warp takes (fewer, longer partials to join)

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
