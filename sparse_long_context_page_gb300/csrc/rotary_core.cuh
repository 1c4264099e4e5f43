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

#include "token_device.cuh"

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

// 1 / sqrt(mean square + eps) from the row's sum of squares.
__device__ __forceinline__ float norm_factor(float sum_sq, float eps)
{
    return rsqrtf(sum_sq * (1.f / kHeadDim) + eps);
}

// The sums of four values over `kLanes` lanes (16 or 32) each, left in every
// lane's f[k] as norm factors: the lanes first share out the values, so that
// four sums take 5 or 6 shuffles and one root, and 4 shuffles back.
template <int kLanes>
__device__ __forceinline__ void norm_factors4(float (&f)[4], float eps)
{
    const int lane = threadIdx.x & 31;
    const bool hi = lane & (kLanes / 2), odd = lane & (kLanes / 4);
    float a = hi ? f[2] : f[0], b = hi ? f[3] : f[1];
    a += __shfl_xor_sync(0xffffffffu, hi ? f[0] : f[2], kLanes / 2);
    b += __shfl_xor_sync(0xffffffffu, hi ? f[1] : f[3], kLanes / 2);
    float s = odd ? b : a;
    s += __shfl_xor_sync(0xffffffffu, odd ? a : b, kLanes / 4);
#pragma unroll
    for (int o = kLanes / 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s = norm_factor(s, eps);
    // value k lies with the lanes whose two upper bits are k
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __shfl_sync(0xffffffffu, s, k * (kLanes / 4), kLanes);
}

// Four neighbouring elements of a row, as two pairs of floats.
struct Run4 {
    uint64_t x[2];
};
__device__ __forceinline__ Run4 unpack4(uint2 v)
{
    return {{pack_b32x2(v.x << 16, v.x & 0xFFFF0000u), pack_b32x2(v.y << 16, v.y & 0xFFFF0000u)}};
}
__device__ __forceinline__ uint2 pack4(const Run4 &r)
{
    return make_uint2(pack_bf16x2(f32x2_lo(r.x[0]), f32x2_hi(r.x[0])), pack_bf16x2(f32x2_lo(r.x[1]), f32x2_hi(r.x[1])));
}
__device__ __forceinline__ Run4 run4(float4 v) { return {{pack_f32x2(v.x, v.y), pack_f32x2(v.z, v.w)}}; }
__device__ __forceinline__ Run4 mul4(const Run4 &a, const Run4 &b)
{
    return {{mul_f32x2(a.x[0], b.x[0]), mul_f32x2(a.x[1], b.x[1])}};
}
__device__ __forceinline__ Run4 fma4(const Run4 &a, const Run4 &b, const Run4 &c)
{
    return {{fma_f32x2(a.x[0], b.x[0], c.x[0]), fma_f32x2(a.x[1], b.x[1], c.x[1])}};
}
__device__ __forceinline__ Run4 scale4(const Run4 &a, float f)
{
    const uint64_t f2 = pack_f32x2(f, f);
    return {{mul_f32x2(a.x[0], f2), mul_f32x2(a.x[1], f2)}};
}
__device__ __forceinline__ Run4 swap4(const Run4 &a)                 // neighbours change places
{
    return {{pack_f32x2(f32x2_hi(a.x[0]), f32x2_lo(a.x[0])), pack_f32x2(f32x2_hi(a.x[1]), f32x2_lo(a.x[1]))}};
}
// The run's pair coefficients where pairs are neighbours: pair p and p + 1 of
// (cos, sin) over the run's four elements, the sines to be multiplied by the
// swapped run.
__device__ __forceinline__ Run4 twice(float2 v) { return {{pack_f32x2(v.x, v.x), pack_f32x2(v.y, v.y)}}; }
__device__ __forceinline__ Run4 twice_signed(float2 v) { return {{pack_f32x2(-v.x, v.x), pack_f32x2(-v.y, v.y)}}; }
__device__ __forceinline__ float sum_sq4(const Run4 &a)
{
    const uint64_t q = fma_f32x2(a.x[0], a.x[0], mul_f32x2(a.x[1], a.x[1]));
    return f32x2_lo(q) + f32x2_hi(q);
}
__device__ __forceinline__ float sum_sq8(const Run4 &a, const Run4 &b)
{
    const uint64_t q = fma_f32x2(a.x[0], a.x[0], fma_f32x2(a.x[1], a.x[1], fma_f32x2(b.x[0], b.x[0], mul_f32x2(b.x[1], b.x[1]))));
    return f32x2_lo(q) + f32x2_hi(q);
}

}  // namespace moira
