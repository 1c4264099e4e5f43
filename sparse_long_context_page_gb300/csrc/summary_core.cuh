// A page's summary from its 16 keys: the exact token-order mean and its three
// formats, shared by the kernels that make or renew summaries (summarize.cu,
// evict.cu).
#pragma once

#include <cuda_bf16.h>

#include "moira_device.cuh"

namespace moira {

// Round a double to the nearest bf16 (ties to even) in one step, by integer
// arithmetic on the binary64 encoding: keep sign, exponent and the top 7
// fraction bits, adding half an ulp minus one plus the kept lsb before
// truncating.  Magnitudes below 2^-126 land on the bf16 subnormal grid
// (multiples of 2^-133), reached by exact scaling and rint().
__device__ __forceinline__ uint32_t f64_to_bf16_rne(double x)
{
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    const uint32_t sign = static_cast<uint32_t>(u >> 48) & 0x8000u;
    const unsigned long long a = u & 0x7FFFFFFFFFFFFFFFull;
    if (a > 0x7FF0000000000000ull) return 0x7FC0u;                  // NaN
    const int biased = static_cast<int>(a >> 52);
    if (biased >= 1023 - 126) {                                       // |x| >= 2^-126
        const unsigned long long r = a + ((1ull << 44) - 1ull) + ((a >> 45) & 1ull);
        const int e_bf = static_cast<int>(r >> 52) - 1023 + 127;
        if (e_bf >= 255) return sign | 0x7F80u;                       // overflow / inf
        return sign | (static_cast<uint32_t>(e_bf) << 7) | static_cast<uint32_t>((r >> 45) & 0x7Full);
    }
    const double grid = rint(fabs(x) * 0x1p133);                      // in [0, 128]
    return sign | static_cast<uint32_t>(grid);
}

// The exact sum, in token order, of one dimension of a page's 16 bf16 keys
// (bit patterns in the low 16 bits of v[t]), when their exponents allow it:
//  * a key is sig * 2^(e - 134) with an integer significand sig < 256 (e = the
//    exponent field, 1 for subnormals).  When the nonzero keys' exponents span
//    at most 40, every partial sum is an integer multiple of 2^(emin - 134)
//    below 2^52 in magnitude, so the sequential fp64 sum is exact and equals
//    the 64-bit integer sum of the significands shifted to the smallest
//    exponent: returns true with that sum in `acc` and emin in `emin`
//    (acc == 0 when every key is +-0 or they cancel: the fp64 sum is +0);
//  * wider spreads, infinities and NaNs return false.
__device__ __forceinline__ bool page_dim_sum_fixed(const uint32_t (&v)[kPageSize], long long &acc, int &emin_out)
{
    int emax = -1, emin = 1 << 30;
    bool special = false;
#pragma unroll
    for (int t = 0; t < kPageSize; ++t) {
        const int e = static_cast<int>((v[t] >> 7) & 0xFFu);
        special |= e == 0xFF;
        if (v[t] & 0x7FFFu) {                           // nonzero
            const int es = e > 0 ? e : 1;
            emax = max(emax, es);
            emin = min(emin, es);
        }
    }
    acc = 0;
    emin_out = 1;
    if (emax < 0) return true;                          // every key is +-0: 0 + ... = +0
    if (special || emax - emin > 40) return false;
#pragma unroll
    for (int t = 0; t < kPageSize; ++t) {
        const int e = static_cast<int>((v[t] >> 7) & 0xFFu);
        const long long sig = static_cast<long long>((v[t] & 0x7Fu) | (e > 0 ? 0x80u : 0u));
        const long long term = sig << max((e > 0 ? e : 1) - emin, 0);     // zeros: sig 0
        acc += (v[t] & 0x8000u) ? -term : term;
    }
    emin_out = emin;
    return true;
}

// The fp64 sum of the same keys in token order, starting from +0.
__device__ __forceinline__ double page_dim_sum_f64(const uint32_t (&v)[kPageSize])
{
    double sum = 0.0;
#pragma unroll
    for (int t = 0; t < kPageSize; ++t) sum += static_cast<double>(__uint_as_float(v[t] << 16));
    return sum;
}

// The fp64 sum of one dimension's 16 keys in token order, bit-exact (the
// integer form where it applies, fp64 adds otherwise).
__device__ __forceinline__ double page_dim_sum(const uint32_t (&v)[kPageSize])
{
    long long acc;
    int emin;
    if (page_dim_sum_fixed(v, acc, emin)) return ldexp(static_cast<double>(acc), emin - 134);
    return page_dim_sum_f64(v);
}

// acc * 2^e2 (|acc| < 2^62, finite and within the bf16 range once rounded)
// rounded to the nearest bf16, ties to even, by integer arithmetic.  The
// result's last place is 2^(e_lead - 7) for a leading bit of weight
// 2^e_lead >= 2^-126, else the subnormal step 2^-133; q, the rounded
// significand on that place, then gives the encoding as
// ((place + 133) << 7) + q for both kinds, a carry to q = 256 included.
__device__ __forceinline__ uint32_t fixed_to_bf16_rne(long long acc, int e2)
{
    if (acc == 0) return 0u;                            // an exact sum of 0 is +0
    const uint32_t sign = acc < 0 ? 0x8000u : 0u;
    const unsigned long long m =
        acc < 0 ? 0ull - static_cast<unsigned long long>(acc) : static_cast<unsigned long long>(acc);
    const int e_lead = 63 - __clzll(static_cast<long long>(m)) + e2;
    const int place = max(e_lead - 7, -133);
    const int sh = place - e2;                          // bits of m below the result's last place
    unsigned long long q;
    if (sh <= 0) {
        q = m << (-sh);
    } else {
        q = m >> sh;
        const unsigned long long rem = m & ((1ull << sh) - 1ull), half = 1ull << (sh - 1);
        q += (rem > half || (rem == half && (q & 1ull))) ? 1ull : 0ull;
    }
    return sign | (static_cast<uint32_t>(place + 133) << 7) + static_cast<uint32_t>(q);
}

// The low-bit record of KV head j from the warp's 128 fp64 means (lane l holds
// dimensions 4l .. 4l+3); the same quantiser as store_lowbit.
template <int kBits>
__device__ void store_lowbit_warp(const double (&mean)[4], uint8_t *rec, int j, int hkv)
{
    constexpr int kCb = lowbit_code_bytes(kBits);
    constexpr double kHalf = static_cast<double>(1 << (kBits - 1));
    const int lane = threadIdx.x & 31;
    bool bad = false;
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bad |= !isfinite(mean[i]);
        a = fmax(a, fabs(mean[i]));
    }
    if (bad) a = 0.0;
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmax(a, __shfl_xor_sync(0xffffffffu, a, o));
    const bool any_bad = __any_sync(0xffffffffu, bad);
    const float step = any_bad ? 0.f : __double2float_rn(a / (kHalf - 0.5));
    int c[4] = {0, 0, 0, 0};
    if (step > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = static_cast<int>(fmin(fmax(floor(mean[i] / static_cast<double>(step)), -kHalf), kHalf - 1.0));
    }
    const int gh = lowbit_group_heads(hkv), jj = j % gh;
    uint8_t *grp = rec + (j / gh) * lowbit_group_bytes(kBits, hkv);
    if constexpr (kBits == 8) {
        *reinterpret_cast<uint32_t *>(grp + jj * kCb + 4 * lane) =
            static_cast<uint32_t>(c[0] & 0xFF) | (static_cast<uint32_t>(c[1] & 0xFF) << 8) |
            (static_cast<uint32_t>(c[2] & 0xFF) << 16) | (static_cast<uint32_t>(c[3] & 0xFF) << 24);
    } else {
        // element i sits in bits 2*(i%4) of byte i/4: the lane's 4 elements are byte `lane`
        grp[jj * kCb + lane] = static_cast<uint8_t>((c[0] + 2) | ((c[1] + 2) << 2) | ((c[2] + 2) << 4) |
                                                    ((c[3] + 2) << 6));
    }
    if (lane == 0) *reinterpret_cast<float *>(grp + gh * kCb + 4 * jj) = step;
    if (jj == 0 && lane < kSummGroup - gh)                  // padding words after the steps
        *reinterpret_cast<uint32_t *>(grp + gh * kCb + 4 * (gh + lane)) = 0u;
}

// The summary of (page p, KV head j) in format kFmt from the warp's keys: lane l
// holds 8 bytes (dimensions 4l .. 4l+3) of each of the page's 16 token rows.
// Every lane of the warp calls it.
template <int kFmt>
__device__ __forceinline__ void store_summary_warp(const uint2 (&row)[kPageSize], uint8_t *summ, int p, int j,
                                                   int hkv)
{
    const int lane = threadIdx.x & 31;
    const size_t blk = static_cast<size_t>(p) * hkv + j;
    if constexpr (kFmt == kSummBf16) {
        // exponent fields of the lane's 4 dimensions (16-bit halves of the two
        // words), smallest and largest over the 16 tokens
        uint32_t mn[2] = {0xFFFFFFFFu, 0xFFFFFFFFu}, mx[2] = {0u, 0u};
#pragma unroll
        for (int t = 0; t < kPageSize; ++t) {
            const uint32_t ex = row[t].x & 0x7F807F80u, ey = row[t].y & 0x7F807F80u;
            mn[0] = __vminu2(mn[0], ex);
            mx[0] = __vmaxu2(mx[0], ex);
            mn[1] = __vminu2(mn[1], ey);
            mx[1] = __vmaxu2(mx[1], ey);
        }
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int sh = 16 * (i & 1);
            const uint32_t lo = (mn[i >> 1] >> sh) & 0xFFFFu, hi = (mx[i >> 1] >> sh) & 0xFFFFu;
            // every key normal (exponent field >= 1, so no zeros either), the
            // largest below 2^124 (16 of them stay below the fp32 limit) and a
            // span of at most 12: every fp32 partial sum is exact
            if (lo >= (1u << 7) && hi <= (250u << 7) && hi - lo <= (12u << 7)) {
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < kPageSize; ++t) {
                    const uint32_t w = i < 2 ? row[t].x : row[t].y;
                    sum += __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
                }
                out[i] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(sum * (1.f / kPageSize))));
            } else {
                uint32_t v[kPageSize];
#pragma unroll
                for (int t = 0; t < kPageSize; ++t) v[t] = ((i < 2 ? row[t].x : row[t].y) >> sh) & 0xFFFFu;
                long long acc;
                int emin;
                out[i] = page_dim_sum_fixed(v, acc, emin)
                             ? fixed_to_bf16_rne(acc, emin - 134 - 4)
                             : f64_to_bf16_rne(page_dim_sum_f64(v) * (1.0 / kPageSize));
            }
        }
        reinterpret_cast<uint2 *>(summ)[blk * (kHeadDim / 4) + lane] =
            make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
    } else {
        double mean[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v[kPageSize];
#pragma unroll
            for (int t = 0; t < kPageSize; ++t) v[t] = ((i < 2 ? row[t].x : row[t].y) >> (16 * (i & 1))) & 0xFFFFu;
            mean[i] = page_dim_sum(v) * (1.0 / kPageSize);
        }
        store_lowbit_warp<summ_bits(kFmt)>(mean, summ + static_cast<size_t>(p) * summ_page_bytes(kFmt, hkv), j,
                                           hkv);
    }
}

}  // namespace moira
