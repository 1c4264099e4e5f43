// Attention of a chunk of tokens over the paged cache.
//
// Request r's new tokens are rows [starts[r], starts[r + 1]); the i-th of n
// sees the first vis = L - n + i + 1 of the request's L cached tokens (causal)
// or all L of them:
//   out_h = sum_{t < vis} e^{s_t} v_t / sum_{t < vis} e^{s_t},  s_t = scale q_h . k_t
// and zero where vis <= 0.
//
// One warp per (row, KV head): lane l holds elements 4l .. 4l + 3 of the
// group's four query rows and of the key and value of one token at a time;
// running maximum and sum in fp32.
#include "moira_device.cuh"
#include "moira_launch.h"

namespace moira {

constexpr int kChunkWarps = 4;

__global__ void __launch_bounds__(kChunkWarps * 32) k_chunk(const ChunkArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kChunkWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (item >= static_cast<long long>(a.tokens) * a.hkv) return;
    const int t = static_cast<int>(item / a.hkv), j = static_cast<int>(item - static_cast<long long>(t) * a.hkv);
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.token_starts + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int from = __ldg(a.token_starts + lo), end = __ldg(a.token_starts + lo + 1);
    if (t < from || t >= end) return;
    int L = __ldg(a.seq_lens + lo);
    if (L < 0 || L > a.max_pages * kPageSize) {
        if (lane == 0) raise_status(a.status, kDevBadLen);
        L = min(max(L, 0), a.max_pages * kPageSize);
    }
    const int vis = a.causal ? L - (end - from) + (t - from) + 1 : L;
    const size_t row = (static_cast<size_t>(t) * a.hkv + j) * kGroup * (kHeadDim / 4) + lane;
    float q[kGroup][4], o[kGroup][4] = {}, m[kGroup], l[kGroup] = {};
#pragma unroll
    for (int h = 0; h < kGroup; ++h) {
        const uint2 v = __ldg(static_cast<const uint2 *>(a.q) + row + h * (kHeadDim / 4));
        q[h][0] = bf16_lo(v.x) * a.scale_log2, q[h][1] = bf16_hi(v.x) * a.scale_log2;
        q[h][2] = bf16_lo(v.y) * a.scale_log2, q[h][3] = bf16_hi(v.y) * a.scale_log2;
        m[h] = -INFINITY;
    }
    for (int s = 0; s < vis; ++s) {
        const int p = __ldg(a.page_table + static_cast<size_t>(lo) * a.max_pages + s / kPageSize);
        if (p < 0 || p >= a.num_pages) {
            if (lane == 0) raise_status(a.status, kDevBadPage);
            s |= kPageSize - 1;
            continue;
        }
        const size_t at = ((static_cast<size_t>(p) * a.hkv + j) * kPageSize + s % kPageSize) * (kHeadDim / 4) + lane;
        const uint2 kv = __ldg(static_cast<const uint2 *>(a.k_pool) + at), vv = __ldg(static_cast<const uint2 *>(a.v_pool) + at);
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
            float d = q[h][0] * bf16_lo(kv.x) + q[h][1] * bf16_hi(kv.x) + q[h][2] * bf16_lo(kv.y) + q[h][3] * bf16_hi(kv.y);
#pragma unroll
            for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            const float mn = fmaxf(m[h], d), f = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn), e = exp2f(d - mn);
            l[h] = l[h] * f + e;
            o[h][0] = o[h][0] * f + e * bf16_lo(vv.x), o[h][1] = o[h][1] * f + e * bf16_hi(vv.x);
            o[h][2] = o[h][2] * f + e * bf16_lo(vv.y), o[h][3] = o[h][3] * f + e * bf16_hi(vv.y);
            m[h] = mn;
        }
    }
#pragma unroll
    for (int h = 0; h < kGroup; ++h) {
        const float f = l[h] == 0.f ? 0.f : 1.f / l[h];
        static_cast<uint2 *>(a.out)[row + h * (kHeadDim / 4)] =
            make_uint2(pack_bf16x2(o[h][0] * f, o[h][1] * f), pack_bf16x2(o[h][2] * f, o[h][3] * f));
    }
}

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t stream)
{
    const long long items = static_cast<long long>(a.tokens) * a.hkv;
    return launch_pdl(k_chunk, dim3(static_cast<unsigned>((items + kChunkWarps - 1) / kChunkWarps)),
                      dim3(kChunkWarps * 32), 0, stream, a);
}

}  // namespace moira
