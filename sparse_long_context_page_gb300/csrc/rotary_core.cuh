// Norm and rotation of one head row, shared by the kernels of rotate.cu.
//
// A pair (a, b) of a row at position p turns by the angle p * f, f the pair's
// inverse frequency.  The angle matters modulo a turn alone, and p * f of a far
// token has lost its fraction in 32 bits (p = 200000, f = 1: 2^-7 of a radian
// is one unit in the last place).  So f is kept as a fraction of a turn in
// 64-bit fixed point, u = f / 2 pi * 2^64: the integer product p * u wraps at
// whole turns by itself and its upper half is the angle, exact to 2^-32 of a
// turn for every int32 position.  No fp64, whose rate on this GPU is 1/64 of
// fp32's.
#pragma once

#include "moira_device.cuh"

namespace moira {

constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kMaxAxes = 4;

// The public moira_rotary by value (a kernel parameter).
struct RotaryArgs {
    int pairs;                       // 0: no rotation
    int interleaved;                 // pair i is elements (2i, 2i + 1), else (i, i + pairs)
    float scale;                     // multiplies cosine and sine
    unsigned long long turns[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

// (cos, sin) of position `pos` for a pair that turns `u` a position.
__device__ __forceinline__ float2 turn_of(unsigned long long u, int pos, float scale)
{
    const unsigned long long w = u * static_cast<unsigned long long>(static_cast<long long>(pos));
    const int frac = static_cast<int>(w >> 32);                      // of a turn, [-1/2, 1/2) in units of 2^-32
    float s, c;
    sincospif(static_cast<float>(frac) * 0x1p-31f, &s, &c);
    return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ float2 rotated(float a, float b, float2 cs)
{
    return make_float2(a * cs.x - b * cs.y, b * cs.x + a * cs.y);
}

// 1 / sqrt(mean square + eps) from the row's sum of squares.
__device__ __forceinline__ float norm_factor(float sum_sq, float eps)
{
    return 1.f / sqrtf(sum_sq * (1.f / kHeadDim) + eps);
}

}  // namespace moira
