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
// head), so the summary of a page that fills needs no word from another block.
#include "rotary_core.cuh"
#include "summary_core.cuh"
#include "token_launch.h"

namespace moira {

constexpr int kRotateThreads = 256;
constexpr int kTurnRows = 8;                             // most rows of a block that only turns them
constexpr int kRotateRows = 16;                          // most rows of a block that writes pages
constexpr int kRotateReach = kRotateRows + kPageSize - 1;    // rows its pages may reach
constexpr int kHeadRun = 8;                              // heads that a half warp takes at a time,
constexpr int kAppendRun = 4;                            // in the append, which has fewer registers

struct alignas(16) RotateSmem {                          // the tables are read 16 bytes at a time
    float cos[kRotateReach][kMaxPairs], sin[kRotateReach][kMaxPairs];
    int at[kRotateReach];                                // index of the row's token in its request; -1: no token
    int page[kRotateRows];                               // pages to write: physical id,
    int first[kRotateRows];                              // block's row of its first new token,
    int slot[kRotateRows], count[kRotateRows];           // that token's slot, tokens
    int pages;
};

// Bytes beside it of an append: the starts and lengths of its requests.
constexpr size_t append_smem(int batch) { return sizeof(int) * (2 * static_cast<size_t>(batch) + 1); }
static_assert(sizeof(RotateSmem) + append_smem(kMaxUnits) <= 48 * 1024, "more needs a limit raised at the launch");

// Asks for the rows of `heads` heads of tokens row0 .. row0 + n in L2, ahead of
// what the block has to work out before it can use them.
__device__ __forceinline__ void ask_rows(const void *in, long long stride, int heads, int row0, int n)
{
    const int shift = 32 - __clz(heads);                 // two lines a head
    for (int e = threadIdx.x; e < n << shift; e += kRotateThreads) {
        const int i = e >> shift;
        prefetch_l2(static_cast<const uint8_t *>(in) + (static_cast<size_t>(row0 + i) * stride) * 2 + (e - (i << shift)) * 128);
    }
}

// (cos, sin) of every (row, pair) of the block's first n rows; at[row] is the
// position where `positions` is null.
__device__ void fill_angles(const RotaryArgs &rot, const int32_t *positions, int tokens, int row0, int n,
                            RotateSmem &sm)
{
    if (rot.pairs == 0) return;
    // a row is as many threads wide as it has pairs; four rows a thread, whose positions are under way together
    const int shift = 32 - __clz(rot.pairs - 1), step = kRotateThreads >> shift, p = threadIdx.x & ((1 << shift) - 1);
    if (p >= rot.pairs) return;
    const int32_t *at = positions ? positions + static_cast<size_t>(rot.axis[p]) * tokens + row0 : nullptr;
#pragma unroll 1
    for (int i0 = threadIdx.x >> shift; i0 < n; i0 += 4 * step) {
        int pos[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = min(i0 + k * step, n - 1);
            pos[k] = at ? __ldg(at + i) : sm.at[i];
        }
#pragma unroll 1                                             // one sine and cosine in the code
        for (int i = i0; i < min(n, i0 + 4 * step); i += step) {
            const float2 t = turn_of(rot.turns[p], pos[0], rot.scale);
            sm.cos[i][p] = t.x;
            sm.sin[i][p] = t.y;
            pos[0] = pos[1], pos[1] = pos[2], pos[2] = pos[3];
        }
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

// kRun heads of one token by a half warp: src and dst are the first head's
// rows, n the heads that exist, most the larger n of the warp's halves.  The
// weights are multiplied into the pair's coefficients, once for all heads.
template <int kRun, bool kInter, bool kNorm>
__device__ __forceinline__ void turn_heads(const uint16_t *src, uint16_t *dst, int n, int most, const RowRuns &r,
                                           const float *cos, const float *sin, const float *norm, float eps)
{
    uint2 xa[kRun], xb[kRun];
#pragma unroll
    for (int h = 0; h < kRun; ++h) {
        xa[h] = xb[h] = make_uint2(0u, 0u);
        if (h < n) {
            xa[h] = *reinterpret_cast<const uint2 *>(src + h * kHeadDim + r.a);
            xb[h] = *reinterpret_cast<const uint2 *>(src + h * kHeadDim + r.b);
        }
    }
    Run4 wa = run4(make_float4(1.f, 1.f, 1.f, 1.f)), wb = wa;
    if (kNorm) {
        wa = run4(__ldg(reinterpret_cast<const float4 *>(norm + r.a)));
        wb = run4(__ldg(reinterpret_cast<const float4 *>(norm + r.b)));
    }
    // a' = a ca + (b, or a's neighbours) sa; b' alike
    Run4 ca = wa, cb = wb, sa = wa, sb = wb;
    const bool turned = r.pair >= 0;
    if (turned) {
        const float4 c = *reinterpret_cast<const float4 *>(cos + r.pair), s = *reinterpret_cast<const float4 *>(sin + r.pair);
        if (kInter) {
            ca = mul4(wa, twice(make_float2(c.x, c.y)));
            cb = mul4(wb, twice(make_float2(c.z, c.w)));
            sa = mul4(swap4(wa), twice_signed(make_float2(s.x, s.y)));
            sb = mul4(swap4(wb), twice_signed(make_float2(s.z, s.w)));
        } else {
            const Run4 s4 = run4(s);
            ca = mul4(wa, run4(c));
            cb = mul4(wb, run4(c));
            sa = mul4(scale4(wb, -1.f), s4);
            sb = mul4(wa, s4);
        }
    }
#pragma unroll
    for (int h0 = 0; h0 < kRun; h0 += 4) {
        if (h0 >= most) break;                           // uniform over the warp
        float f[4];
        if (kNorm) {
#pragma unroll
            for (int h = 0; h < 4; ++h) f[h] = sum_sq8(unpack4(xa[h0 + h]), unpack4(xb[h0 + h]));
            norm_factors4<16>(f, eps);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + k;
            Run4 a = unpack4(xa[h]), b = unpack4(xb[h]);
            if (kNorm) {
                a = scale4(a, f[k]);
                b = scale4(b, f[k]);
            }
            Run4 ya, yb;
            if (!turned) {
                ya = mul4(a, ca);
                yb = mul4(b, cb);
            } else if (kInter) {
                ya = fma4(a, ca, mul4(swap4(a), sa));
                yb = fma4(b, cb, mul4(swap4(b), sb));
            } else {
                ya = fma4(a, ca, mul4(b, sa));
                yb = fma4(b, cb, mul4(a, sb));
            }
            if (h < n) {
                *reinterpret_cast<uint2 *>(dst + h * kHeadDim + r.a) = pack4(ya);
                *reinterpret_cast<uint2 *>(dst + h * kHeadDim + r.b) = pack4(yb);
            }
        }
    }
}

// All heads of the block's rows that hold a token; a warp's two halves take
// different (row, run of heads) items and stay together for the shuffles.
template <int kRun, bool kInter, bool kNorm>
__device__ __forceinline__ void turn_rows_as(const TokenRows &x, int heads, int row0, int rows, const RowRuns &r,
                                             const RotateSmem &sm, float eps)
{
    const int half = (threadIdx.x >> 4) & 1, warp = threadIdx.x >> 5;
    const int shift = 31 - __clz(max(heads / kRun, 1)), items = rows << shift;       // the head counts are powers of two
    for (int it = 2 * warp; it < items; it += 2 * (kRotateThreads / 32)) {
        const int mine = min(it + half, items - 1), i = mine >> shift, h = (mine - (i << shift)) * kRun;
        // a half without an item of its own repeats the last one, without its heads
        const int n = it + half < items && sm.at[i] >= 0 ? min(kRun, heads - h) : 0;
        const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 16));
        if (most == 0) continue;
        const size_t row = static_cast<size_t>(row0 + i);
        turn_heads<kRun, kInter, kNorm>(static_cast<const uint16_t *>(x.in) + row * x.stride + h * kHeadDim,
                                  static_cast<uint16_t *>(x.out) + (row * heads + h) * kHeadDim, n, most, r, sm.cos[i],
                                  sm.sin[i], x.norm, eps);
    }
}
template <int kRun>
__device__ __forceinline__ void turn_rows(const TokenRows &x, int heads, int row0, int rows, const RowRuns &r,
                                          const RotateSmem &sm, float eps)
{
    if (r.interleaved) {
        if (x.norm) turn_rows_as<kRun, true, true>(x, heads, row0, rows, r, sm, eps);
        else turn_rows_as<kRun, true, false>(x, heads, row0, rows, r, sm, eps);
    } else {
        if (x.norm) turn_rows_as<kRun, false, true>(x, heads, row0, rows, r, sm, eps);
        else turn_rows_as<kRun, false, false>(x, heads, row0, rows, r, sm, eps);
    }
}

// Bound by memory: the queries and keys of 32k tokens, 32 + 8 heads, norms and three
// axes take 106 us, 6.3 TB/s.
__global__ void __launch_bounds__(kRotateThreads) k_rotate(const __grid_constant__ RotaryArgs rot, const RotateArgs a)
{
    __shared__ RotateSmem sm;
    const int row0 = blockIdx.x * a.rows, rows = min(a.rows, a.tokens - row0);
    if (threadIdx.x < rows) sm.at[threadIdx.x] = 0;
    pdl_wait();
    pdl_trigger();
    if (a.q.in) ask_rows(a.q.in, a.q.stride, a.hq, row0, rows);
    if (a.k.in) ask_rows(a.k.in, a.k.stride, a.hkv, row0, rows);
    fill_angles(rot, a.positions, a.tokens, row0, rows, sm);
    __syncthreads();
    const RowRuns r(rot, threadIdx.x & 15);
    if (a.q.in) turn_rows<kHeadRun>(a.q, a.hq, row0, rows, r, sm, a.eps);
    if (a.k.in) turn_rows<kHeadRun>(a.k, a.hkv, row0, rows, r, sm, a.eps);
}

// One page's new values of KV head j by a warp: lane l holds elements 4l .. 4l + 3
// of every row.
__device__ __forceinline__ void append_values(const AppendArgs &a, const RotateSmem &sm, int row0, int e, int j)
{
    const int lane = threadIdx.x & 31, slot = sm.slot[e], count = sm.count[e];
    uint2 *vp = static_cast<uint2 *>(a.v_pool) + (static_cast<size_t>(sm.page[e]) * a.hkv + j) * (kPageSize * kHeadDim / 4) + lane;
    const uint16_t *v = static_cast<const uint16_t *>(a.v) + static_cast<size_t>(row0 + sm.first[e]) * a.v_stride + j * kHeadDim;
    uint2 row[kPageSize];
#pragma unroll
    for (int i = 0; i < kPageSize; ++i)
        if (i < count) row[i] = __ldg(reinterpret_cast<const uint2 *>(v + static_cast<size_t>(i) * a.v_stride) + lane);
#pragma unroll
    for (int i = 0; i < kPageSize; ++i)
        if (i < count) vp[(slot + i) * (kHeadDim / 4)] = row[i];
}

// Its new keys, normed and rotated, four at a time with the next four under way: a
// rolled loop, since all 16 rows at once are more code than the instruction cache
// holds beside the rest (prompt of 16k tokens 79 us, so 74; its 16 keys then come
// back from L2 for the summary).
template <bool kInter, bool kNorm>
__device__ __forceinline__ void append_keys(const RotaryArgs &rot, const AppendArgs &a, const RotateSmem &sm, int row0, int e,
                                            int j, uint2 *kp)
{
    const int lane = threadIdx.x & 31, slot = sm.slot[e], count = sm.count[e], first = sm.first[e];
    const uint16_t *k = static_cast<const uint16_t *>(a.k.in) + static_cast<size_t>(row0 + first) * a.k.stride + j * kHeadDim + 4 * lane;
    auto load = [&](int i, uint2 (&x)[4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = i + r < count ? __ldg(reinterpret_cast<const uint2 *>(k + static_cast<size_t>(i + r) * a.k.stride)) : make_uint2(0u, 0u);
    };
    uint2 next[4];
    load(0, next);
    // the pairs of the lane's elements, and the lane that holds their partners
    const bool turned = 4 * lane < 2 * rot.pairs, second = 4 * lane >= rot.pairs;
    const int pair = kInter ? 2 * lane : 4 * lane - (second ? rot.pairs : 0);
    const int other = turned && !kInter ? (second ? lane - rot.pairs / 4 : lane + rot.pairs / 4) : lane;
    // weights of the elements and of their partners, the sine's sign with the latter
    Run4 w = run4(make_float4(1.f, 1.f, 1.f, 1.f)), wo = w;
    if (kNorm) {
        w = run4(__ldg(reinterpret_cast<const float4 *>(a.k.norm) + lane));
        wo = kInter ? swap4(w) : run4(__ldg(reinterpret_cast<const float4 *>(a.k.norm) + other));
    }
    if (!kInter && !second) wo = scale4(wo, -1.f);
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += 4) {
        uint2 row[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) row[r] = next[r];
        load(i0 + 4, next);
        float f[4];
        if (kNorm) {
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] = sum_sq4(unpack4(row[r]));
            norm_factors4<32>(f, a.eps);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r;
            if (i >= count) break;                               // uniform over the warp
            Run4 x = unpack4(row[r]), o = x, y;
            if (!kInter) o = unpack4(make_uint2(__shfl_sync(0xffffffffu, row[r].x, other), __shfl_sync(0xffffffffu, row[r].y, other)));
            if (kNorm) {
                x = scale4(x, f[r]);
                o = scale4(o, f[r]);
            }
            if (!turned) {
                y = mul4(x, w);
            } else if (kInter) {
                const float2 c = *reinterpret_cast<const float2 *>(&sm.cos[first + i][pair]);
                const float2 s = *reinterpret_cast<const float2 *>(&sm.sin[first + i][pair]);
                y = fma4(x, mul4(w, twice(c)), mul4(swap4(x), mul4(wo, twice_signed(s))));
            } else {
                const Run4 c = run4(*reinterpret_cast<const float4 *>(&sm.cos[first + i][pair]));
                const Run4 s = run4(*reinterpret_cast<const float4 *>(&sm.sin[first + i][pair]));
                y = fma4(x, mul4(w, c), mul4(o, mul4(wo, s)));
            }
            kp[(slot + i) * (kHeadDim / 4)] = pack4(y);
        }
    }
}

// Bound by memory for long prompts (16k tokens of 32 + 16 heads 74 us, 5.5 TB/s), by
// its blocks' chains of loads for ragged ones (37 requests of up to 1531 tokens 34 us,
// 4 TB/s): starts, page, positions, rows.  Four blocks an SM hide more of them
// than three, although 64 registers spill a little around the summary (36 us).
template <int kFmt>
__global__ void __launch_bounds__(kRotateThreads, 4)
    k_append_rotated(const __grid_constant__ RotaryArgs rot, const AppendArgs a)
{
    extern __shared__ int starts[];                      // [batch + 1], then the lengths
    int *const lens = starts + a.batch + 1;
    __shared__ RotateSmem sm;
    // the first blocks take keys and values, the others queries
    const int page_blocks = (a.tokens + a.rows - 1) / a.rows;
    const bool queries = blockIdx.x >= page_blocks;
    const int tid = threadIdx.x, warp = tid >> 5, most = queries ? a.q_rows : a.rows;
    const int row0 = (queries ? blockIdx.x - page_blocks : blockIdx.x) * most, rows = min(most, a.tokens - row0);
    const int reach = queries ? rows : min(most + kPageSize - 1, a.tokens - row0);
    if (tid == 0) sm.pages = 0;
    pdl_wait();
    pdl_trigger();
    if (queries) {
        ask_rows(a.q.in, a.q.stride, a.hkv * kGroup, row0, rows);
    } else {
        ask_rows(a.k.in, a.k.stride, a.hkv, row0, rows);
        ask_rows(a.v, a.v_stride, a.hkv, row0, rows);
    }
    for (int i = tid; i <= a.batch; i += kRotateThreads) {
        starts[i] = __ldg(a.token_starts + i);
        if (i < a.batch) lens[i] = __ldg(a.seq_lens + i);
    }
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
            const int L = lens[lo];
            if (L >= n && L <= a.max_pages * kPageSize) at = L - n + nth;
        }
        sm.at[tid] = at;
        if (!queries && tid < rows && at >= 0 && (nth == 0 || at % kPageSize == 0)) {
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
    if (!queries) {
        // the values need no angles
        const int shift = 31 - __clz(a.hkv), pages = sm.pages << shift;
        for (int it = warp; it < pages; it += kRotateThreads / 32)
            append_values(a, sm, row0, it >> shift, it & (a.hkv - 1));
    }
    if (rot.pairs) {
        int need = rows;
        if (!queries) {
            // the rows that the pages reach; none where no page begins
            need = 0;
            for (int e = 0; e < sm.pages; ++e) need = max(need, sm.first[e] + sm.count[e]);
        }
        fill_angles(rot, a.positions, a.tokens, row0, need, sm);
        __syncthreads();
    }
    if (queries) {
        turn_rows<kAppendRun>(a.q, a.hkv * kGroup, row0, rows, RowRuns(rot, tid & 15), sm, a.eps);
    } else {
        const int shift = 31 - __clz(a.hkv), pages = sm.pages << shift;
        // by the warps that the values have left free first
        for (int it = (warp + pages) % (kRotateThreads / 32); it < pages; it += kRotateThreads / 32) {
            const int e = it >> shift, j = it & (a.hkv - 1);
            uint2 *kp = static_cast<uint2 *>(a.k_pool) + (static_cast<size_t>(sm.page[e]) * a.hkv + j) * (kPageSize * kHeadDim / 4) + (tid & 31);
            if (rot.interleaved) {
                if (a.k.norm) append_keys<true, true>(rot, a, sm, row0, e, j, kp);
                else append_keys<true, false>(rot, a, sm, row0, e, j, kp);
            } else {
                if (a.k.norm) append_keys<false, true>(rot, a, sm, row0, e, j, kp);
                else append_keys<false, false>(rot, a, sm, row0, e, j, kp);
            }
            if (a.summ && sm.slot[e] + sm.count[e] == kPageSize) {
                // the page is full: its rows, each lane's as it wrote them, come back from L2
                uint2 row[kPageSize];
#pragma unroll
                for (int t = 0; t < kPageSize; ++t) row[t] = kp[t * (kHeadDim / 4)];
                store_summary_warp<kFmt>(row, static_cast<uint8_t *>(a.summ), sm.page[e], j, a.hkv);
            }
        }
    }
}

namespace {

// Rows of a block: enough blocks for every SM twice while there are tokens.
int rows_per_block(int tokens, int most, int sms)
{
    int rows = 1;
    while (rows < most && tokens / (2 * rows) >= 2 * sms) rows *= 2;
    return rows;
}

}  // namespace

cudaError_t launch_rotate(const RotaryArgs &rot, RotateArgs a, int sms, cudaStream_t stream)
{
    a.rows = rows_per_block(a.tokens, kTurnRows, sms);
    return launch_pdl(k_rotate, dim3((a.tokens + a.rows - 1) / a.rows), dim3(kRotateThreads), 0, stream, rot, a);
}

cudaError_t launch_append_rotated(const RotaryArgs &rot, AppendArgs a, int fmt, int sms, cudaStream_t stream)
{
    a.rows = rows_per_block(a.tokens, kRotateRows, sms);
    a.q_rows = rows_per_block(a.tokens, kTurnRows, sms);
    const dim3 grid((a.tokens + a.rows - 1) / a.rows + (a.q.in ? (a.tokens + a.q_rows - 1) / a.q_rows : 0));
    const size_t smem = append_smem(a.batch);
    if (fmt == kSummQ8) return launch_pdl(k_append_rotated<kSummQ8>, grid, dim3(kRotateThreads), smem, stream, rot, a);
    if (fmt == kSummQ2) return launch_pdl(k_append_rotated<kSummQ2>, grid, dim3(kRotateThreads), smem, stream, rot, a);
    return launch_pdl(k_append_rotated<kSummBf16>, grid, dim3(kRotateThreads), smem, stream, rot, a);
}

}  // namespace moira
