// Norm and rotation of queries and keys (k_rotate), and the append of rotated
// tokens to a paged cache (k_append_rotated).
//
// A head row x of 128 elements, bf16 in and out, fp32 between, rounded once:
//   y = x / sqrt(mean(x^2) + eps) * w                    (with norm weights w)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)     for its first 2 * pairs elements
// with t the pair's angle at the token's position on the pair's axis
// (rotary_core.cuh).  All heads of a token turn by the same angles, so a block
// takes a few tokens with all their heads and leaves (cos, sin) of every
// (token, pair) in shared memory first.
//
// Tokens are rows of a ragged batch: request r's new tokens are rows
// [starts[r], starts[r + 1]), the last of its seq_lens[r] tokens.  A block of
// k_append_rotated takes the queries of its rows, and the keys and values of
// the pages whose first new token is among them, whole: one warp a (page, KV
// head) holds the page's 16 keys in registers, so the summary of a page that
// fills needs no second pass and no word from another block.
#include "moira_launch.h"
#include "rotary_core.cuh"
#include "summary_core.cuh"

namespace moira {

constexpr int kRotateThreads = 256;
constexpr int kRotateRows = 16;                          // most rows of a block
constexpr int kRotateReach = kRotateRows + kPageSize - 1;    // rows its pages may reach
constexpr int kHeadRun = 4;                              // heads that a half warp takes at a time

struct RotateSmem {
    float2 cs[kRotateReach][kMaxPairs];
    int at[kRotateReach];                                // index of the row's token in its request; -1: no token
    int page[kRotateRows];                               // pages to write: physical id,
    int first[kRotateRows];                              // block's row of its first new token,
    int slot[kRotateRows], count[kRotateRows];           // that token's slot, tokens
    int pages;
};

// (cos, sin) of every (row, pair) of the block's first n rows; at[row] is the
// position where `positions` is null.
__device__ void fill_angles(const RotaryArgs &rot, const int32_t *positions, int tokens, int row0, int n,
                            RotateSmem &sm)
{
    for (int e = threadIdx.x; e < n * rot.pairs; e += kRotateThreads) {
        const int i = e / rot.pairs, p = e - i * rot.pairs;
        const int pos = positions ? __ldg(positions + static_cast<size_t>(rot.axis[p]) * tokens + row0 + i) : sm.at[i];
        sm.cs[i][p] = turn_of(rot.turns[p], pos, rot.scale);
    }
}

// A half warp's rows: lane l holds two runs of four elements that turn with
// each other (a: first elements, b: second) or, behind the rotated part, lie
// side by side.
struct RowRuns {
    int a, b;                                            // first element of each run
    int pair;                                            // pair of element a, -1: not rotated
    bool interleaved;
    __device__ RowRuns(const RotaryArgs &rot, int l)
    {
        interleaved = rot.interleaved != 0;
        const int turned = rot.pairs / 4;                // lanes that hold rotated elements
        if (interleaved) {
            a = 8 * l;
            b = a + 4;
        } else if (l < turned) {
            a = 4 * l;
            b = a + rot.pairs;
        } else {
            a = 2 * rot.pairs + 8 * (l - turned);
            b = a + 4;
        }
        pair = l < turned ? 4 * l : -1;
    }
};

__device__ __forceinline__ void unpack4(uint2 v, float (&f)[4])
{
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
}
__device__ __forceinline__ uint2 pack4(const float (&f)[4])
{
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// kHeadRun heads of one token by a half warp: src and dst are the first head's
// rows, n the heads that exist, most the larger n of the warp's halves.
__device__ __forceinline__ void turn_heads(const uint16_t *src, uint16_t *dst, int n, int most, const RowRuns &r,
                                           const float2 *cs, const float *norm, float eps)
{
    uint2 xa[kHeadRun], xb[kHeadRun];
#pragma unroll
    for (int h = 0; h < kHeadRun; ++h) {
        xa[h] = xb[h] = make_uint2(0u, 0u);
        if (h < n) {
            xa[h] = *reinterpret_cast<const uint2 *>(src + h * kHeadDim + r.a);
            xb[h] = *reinterpret_cast<const uint2 *>(src + h * kHeadDim + r.b);
        }
    }
    float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
    if (norm) {
        wa = __ldg(reinterpret_cast<const float4 *>(norm + r.a));
        wb = __ldg(reinterpret_cast<const float4 *>(norm + r.b));
    }
    float2 t[4];
    if (r.pair >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = cs[r.pair + i];
    }
#pragma unroll
    for (int h = 0; h < kHeadRun; ++h)
        if (h < most) {                                  // uniform over the warp
            float a[4], b[4];
            unpack4(xa[h], a);
            unpack4(xb[h], b);
            if (norm) {
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
#pragma unroll
                for (int o = 8; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                const float f = norm_factor(sq, eps);
                a[0] *= f * wa.x, a[1] *= f * wa.y, a[2] *= f * wa.z, a[3] *= f * wa.w;
                b[0] *= f * wb.x, b[1] *= f * wb.y, b[2] *= f * wb.z, b[3] *= f * wb.w;
            }
            if (r.pair >= 0) {
                if (r.interleaved) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 y = rotated(a[2 * i], a[2 * i + 1], t[i]);
                        const float2 z = rotated(b[2 * i], b[2 * i + 1], t[2 + i]);
                        a[2 * i] = y.x, a[2 * i + 1] = y.y;
                        b[2 * i] = z.x, b[2 * i + 1] = z.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 y = rotated(a[i], b[i], t[i]);
                        a[i] = y.x, b[i] = y.y;
                    }
                }
            }
            if (h < n) {
                *reinterpret_cast<uint2 *>(dst + h * kHeadDim + r.a) = pack4(a);
                *reinterpret_cast<uint2 *>(dst + h * kHeadDim + r.b) = pack4(b);
            }
        }
}

// All heads of the block's rows that hold a token; a warp's two halves take
// different (row, run of heads) items and stay together for the shuffles.
__device__ void turn_rows(const TokenRows &x, int heads, int row0, int rows, const RowRuns &r, const RotateSmem &sm,
                          float eps, int warp, int warps)
{
    const int half = (threadIdx.x >> 4) & 1, runs = (heads + kHeadRun - 1) / kHeadRun, items = rows * runs;
    for (int it = 2 * warp; it < items; it += 2 * warps) {
        const int mine = min(it + half, items - 1), i = mine / runs, h = (mine - i * runs) * kHeadRun;
        // a half without an item of its own repeats the last one, without its heads
        const int n = it + half < items && sm.at[i] >= 0 ? min(kHeadRun, heads - h) : 0;
        const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 16));
        if (most == 0) continue;
        const size_t row = static_cast<size_t>(row0 + i);
        turn_heads(static_cast<const uint16_t *>(x.in) + row * x.stride + h * kHeadDim,
                   static_cast<uint16_t *>(x.out) + (row * heads + h) * kHeadDim, n, most, r, sm.cs[i], x.norm, eps);
    }
}

__global__ void __launch_bounds__(kRotateThreads) k_rotate(const __grid_constant__ RotaryArgs rot, const RotateArgs a)
{
    __shared__ RotateSmem sm;
    const int row0 = blockIdx.x * a.rows, rows = min(a.rows, a.tokens - row0), warp = threadIdx.x >> 5;
    if (threadIdx.x < rows) sm.at[threadIdx.x] = 0;
    pdl_wait();
    pdl_trigger();
    fill_angles(rot, a.positions, a.tokens, row0, rows, sm);
    __syncthreads();
    const RowRuns r(rot, threadIdx.x & 15);
    if (a.q.in) turn_rows(a.q, a.hq, row0, rows, r, sm, a.eps, warp, kRotateThreads / 32);
    if (a.k.in) turn_rows(a.k, a.hkv, row0, rows, r, sm, a.eps, warp, kRotateThreads / 32);
}

// One page's new keys and values of KV head j by a warp: lane l holds elements
// 4l .. 4l + 3 of every row.
template <int kFmt>
__device__ void append_page(const RotaryArgs &rot, const AppendArgs &a, const RotateSmem &sm, int row0, int e, int j)
{
    const int lane = threadIdx.x & 31, slot = sm.slot[e], count = sm.count[e], first = sm.first[e];
    const size_t blk = (static_cast<size_t>(sm.page[e]) * a.hkv + j) * (kPageSize * kHeadDim / 4) + lane;
    uint2 *kp = static_cast<uint2 *>(a.k_pool) + blk, *vp = static_cast<uint2 *>(a.v_pool) + blk;
    const uint16_t *k = static_cast<const uint16_t *>(a.k.in) + static_cast<size_t>(row0 + first) * a.k.stride + j * kHeadDim;
    const uint16_t *v = static_cast<const uint16_t *>(a.v) + static_cast<size_t>(row0 + first) * a.v_stride + j * kHeadDim;
    const bool fills = a.summ && slot + count == kPageSize;
    uint2 row[kPageSize], val[kPageSize];
#pragma unroll
    for (int t = 0; t < kPageSize; ++t) {
        row[t] = make_uint2(0u, 0u);
        const int i = t - slot;
        if (i >= 0 && i < count) {
            row[t] = __ldg(reinterpret_cast<const uint2 *>(k + static_cast<size_t>(i) * a.k.stride) + lane);
            val[t] = __ldg(reinterpret_cast<const uint2 *>(v + static_cast<size_t>(i) * a.v_stride) + lane);
        } else if (fills && i < 0) {
            row[t] = kp[t * (kHeadDim / 4)];
        }
    }
    float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.k.norm) w = __ldg(reinterpret_cast<const float4 *>(a.k.norm) + lane);
    // the pairs of the lane's elements, and the lane that holds their partners
    const bool inter = rot.interleaved != 0, turned = 4 * lane < 2 * rot.pairs, second = 4 * lane >= rot.pairs;
    const int pair = inter ? 2 * lane : 4 * lane - (second ? rot.pairs : 0);
    const int other = turned && !inter ? (second ? lane - rot.pairs / 4 : lane + rot.pairs / 4) : lane;
#pragma unroll
    for (int t = 0; t < kPageSize; ++t) {
        const int i = t - slot;
        if (i < 0 || i >= count) continue;
        float x[4];
        unpack4(row[t], x);
        if (a.k.norm) {
            float sq = fmaf(x[0], x[0], fmaf(x[1], x[1], fmaf(x[2], x[2], x[3] * x[3])));
#pragma unroll
            for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float f = norm_factor(sq, a.eps);
            x[0] *= f * w.x, x[1] *= f * w.y, x[2] *= f * w.z, x[3] *= f * w.w;
        }
        if (rot.pairs) {
            const float2 *cs = sm.cs[first + i];
            if (inter) {
                if (turned) {
                    const float2 y = rotated(x[0], x[1], cs[pair]), z = rotated(x[2], x[3], cs[pair + 1]);
                    x[0] = y.x, x[1] = y.y, x[2] = z.x, x[3] = z.y;
                }
            } else {
                float o[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = __shfl_sync(0xffffffffu, x[c], other);
                if (turned) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 t2 = cs[pair + c];
                        x[c] = second ? x[c] * t2.x + o[c] * t2.y : x[c] * t2.x - o[c] * t2.y;
                    }
                }
            }
        }
        row[t] = pack4(x);
        kp[t * (kHeadDim / 4)] = row[t];
        vp[t * (kHeadDim / 4)] = val[t];
    }
    if (fills) store_summary_warp<kFmt>(row, static_cast<uint8_t *>(a.summ), sm.page[e], j, a.hkv);
}

template <int kFmt>
__global__ void __launch_bounds__(kRotateThreads, 2)
    k_append_rotated(const __grid_constant__ RotaryArgs rot, const AppendArgs a)
{
    extern __shared__ int starts[];                      // [batch + 1]
    __shared__ RotateSmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, row0 = blockIdx.x * a.rows;
    const int reach = min(a.rows + kPageSize - 1, a.tokens - row0), rows = min(a.rows, a.tokens - row0);
    if (tid == 0) sm.pages = 0;
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i <= a.batch; i += kRotateThreads) starts[i] = __ldg(a.token_starts + i);
    __syncthreads();
    if (tid < reach) {
        // the last request that starts at or before the row
        const int t = row0 + tid;
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int from = starts[lo], n = starts[lo + 1] - from, nth = t - from;
        int at = -1;
        if (from >= 0 && nth >= 0 && nth < n && n <= a.tokens) {
            const int L = __ldg(a.seq_lens + lo);
            if (L >= n && L <= a.max_pages * kPageSize) at = L - n + nth;
        }
        sm.at[tid] = at;
        if (tid < rows && at >= 0 && (nth == 0 || at % kPageSize == 0)) {
            const int page = __ldg(a.page_table + static_cast<size_t>(lo) * a.max_pages + at / kPageSize);
            if (page >= 0 && page < a.num_pages) {
                const int e = atomicAdd(&sm.pages, 1);
                sm.page[e] = page;
                sm.first[e] = tid;
                sm.slot[e] = at % kPageSize;
                // the request's rows lie inside [0, tokens)
                sm.count[e] = min(min(kPageSize - at % kPageSize, n - nth), a.tokens - t);
            }
        }
    }
    __syncthreads();
    if (rot.pairs) {
        // rows behind the block's own, as far as its pages reach
        int need = rows;
        for (int e = 0; e < sm.pages; ++e) need = max(need, sm.first[e] + sm.count[e]);
        fill_angles(rot, a.positions, a.tokens, row0, need, sm);
        __syncthreads();
    }
    for (int it = warp; it < sm.pages * a.hkv; it += kRotateThreads / 32)
        append_page<kFmt>(rot, a, sm, row0, it / a.hkv, it & (a.hkv - 1));
    if (a.q.in)
        turn_rows(a.q, a.hkv * kGroup, row0, rows, RowRuns(rot, tid & 15), sm, a.eps, warp, kRotateThreads / 32);
}

namespace {

// Rows of a block: enough blocks for every SM twice while there are tokens.
int rows_per_block(int tokens, int sms)
{
    int rows = 1;
    while (rows < kRotateRows && tokens / (2 * rows) >= 2 * sms) rows *= 2;
    return rows;
}

}  // namespace

cudaError_t launch_rotate(const RotaryArgs &rot, RotateArgs a, int sms, cudaStream_t stream)
{
    a.rows = rows_per_block(a.tokens, sms);
    return launch_pdl(k_rotate, dim3((a.tokens + a.rows - 1) / a.rows), dim3(kRotateThreads), 0, stream, rot, a);
}

cudaError_t launch_append_rotated(const RotaryArgs &rot, AppendArgs a, int fmt, int sms, cudaStream_t stream)
{
    a.rows = rows_per_block(a.tokens, sms);
    const dim3 grid((a.tokens + a.rows - 1) / a.rows);
    const size_t smem = sizeof(int) * (static_cast<size_t>(a.batch) + 1);
    if (fmt == kSummQ8) return launch_pdl(k_append_rotated<kSummQ8>, grid, dim3(kRotateThreads), smem, stream, rot, a);
    if (fmt == kSummQ2) return launch_pdl(k_append_rotated<kSummQ2>, grid, dim3(kRotateThreads), smem, stream, rot, a);
    return launch_pdl(k_append_rotated<kSummBf16>, grid, dim3(kRotateThreads), smem, stream, rot, a);
}

}  // namespace moira
