// Eviction of cached tokens by accumulated attention weight.
//
// Per (request, KV head) with n > budget tokens, the `budget` tokens that come
// first in the order
//   protected (position < sinks, or among the `recent` newest) before others,
//   then larger weight, NaN last, then lower slot
// stay.  The kept tokens at slots >= budget move into the evicted slots below
// it, the i-th into the i-th (both ascending), so a token that stays below
// the budget is not touched and the moves are disjoint: they run in any order.
// k_evict_plan finds the cut and the pairs, k_evict_move moves keys, values,
// weights and positions and renews the summaries of the pages whose keys
// changed.
#include "moira_launch.h"
#include "summary_core.cuh"

namespace moira {

constexpr int kPlanThreads = 1024;

// A token's place in the order as an unsigned key, larger first.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (isnan(w)) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);                 // -0 counts as 0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);           // ascending with w; +inf is 0xFF800000
}
constexpr uint32_t kKeyProtected = 0xFFFFFFFFu;

// Positions of a unit's tokens.  A slot without one (negative) continues after
// the largest stored position in slot order; `first` is the lowest such slot.
struct Positions {
    int last, first, newest, sinks, recent;
    __device__ __forceinline__ int of(int stored, int t) const { return stored >= 0 ? stored : last + 1 + (t - first); }
    __device__ __forceinline__ bool safe(int pos) const { return pos < sinks || pos > newest - recent; }
};

// Exclusive scan of one int per thread over the block; `total` to everyone.
__device__ __forceinline__ int block_scan(int v, int *s_warp, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s_warp[lane] = y;
    }
    __syncthreads();
    total = s_warp[31];
    const int before = (warp ? s_warp[warp - 1] : 0) + x - v;
    __syncthreads();
    return before;
}

__global__ void __launch_bounds__(kPlanThreads, 1) k_evict_plan(const EvictArgs a)
{
    __shared__ int s_warp[32];
    __shared__ uint32_t s_hist[256];
    __shared__ int s_last, s_first, s_top, s_bad, s_need;
    __shared__ uint32_t s_prefix;
    const int tid = threadIdx.x, u = blockIdx.x, r = u / a.hkv, j = u % a.hkv;
    pdl_wait();
    const int raw = a.seq_lens[r], cap = a.max_pages * kPageSize;
    const int n = min(max(raw, 0), cap), m = min(n, a.budget);
    if (raw != n && tid == 0) raise_status(a.status, kDevBadLen);
    if (n <= m) {
        if (tid == 0) a.counts[u] = make_int2(0, n);
        return;
    }
    if (tid == 0) {
        s_last = -1;
        s_first = 0x7FFFFFFF;
        s_top = -1;
        s_bad = 0;
    }
    __syncthreads();
    const int32_t *table = a.page_table + static_cast<size_t>(r) * a.max_pages;
    for (int p = tid; p * kPageSize < n; p += kPlanThreads) {
        const int pid = table[p];
        if (pid < 0 || pid >= a.num_pages) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {                                                 // the request is left as it is
        if (tid == 0) {
            raise_status(a.status, kDevBadPage);
            a.counts[u] = make_int2(-1, n);
        }
        return;
    }
    auto at = [&](int t) { return (static_cast<size_t>(table[t / kPageSize]) * a.hkv + j) * kPageSize + t % kPageSize; };
    int last = -1, first = 0x7FFFFFFF, top = -1;
    for (int t = tid; t < n; t += kPlanThreads) {
        const int s = a.positions[at(t)];
        if (s >= 0) {
            last = max(last, s);
        } else {
            first = min(first, t);
            top = t;
        }
    }
    atomicMax(&s_last, last);
    atomicMin(&s_first, first);
    atomicMax(&s_top, top);
    __syncthreads();
    Positions ps{s_last, s_first, s_last, a.sinks, a.recent};
    if (s_top >= 0) ps.newest = ps.of(-1, s_top);
    auto key_of = [&](int t) {
        const size_t i = at(t);
        return ps.safe(ps.of(a.positions[i], t)) ? kKeyProtected : weight_key(a.weights[i]);
    };
    // radix descent to the m-th largest key: `need` of the tokens that equal it stay
    uint32_t prefix = 0;
    int need = m;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        for (int t = tid; t < n; t += kPlanThreads) {
            const uint32_t k = key_of(t);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[k >> shift & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, bin = 255;
            while (static_cast<int>(s_hist[bin]) < left) left -= s_hist[bin--];
            s_need = left;
            s_prefix = prefix | static_cast<uint32_t>(bin) << shift;
        }
        __syncthreads();
        need = s_need;
        prefix = s_prefix;
        __syncthreads();
    }
    // pairs in slot order; evicted slots of the cut part are cleared here, the
    // moved ones by k_evict_move once it has read them
    int equal = 0, holes = 0, movers = 0;
    int2 *moves = a.moves + static_cast<size_t>(u) * (a.max_pages * (kPageSize / 2));
    for (int base = 0; base < n; base += kPlanThreads) {
        const int t = base + tid;
        const uint32_t k = t < n ? key_of(t) : 0u;
        const bool eq = t < n && k == prefix;
        int total;
        const int rank = equal + block_scan(eq, s_warp, total);
        equal += total;
        const bool keep = t < n && (k > prefix || (eq && rank < need));
        const bool hole = t < m && !keep, mover = t >= m && keep;
        const int hi = holes + block_scan(hole, s_warp, total);
        holes += total;
        const int mi = movers + block_scan(mover, s_warp, total);
        movers += total;
        if (hole) moves[hi].x = t;
        if (mover) moves[mi].y = t;
        if (t < n) {
            const size_t i = at(t);
            if (keep) {
                const int s = a.positions[i];
                if (s < 0) a.positions[i] = ps.of(s, t);
            } else if (t >= m) {
                a.positions[i] = -1;
                a.weights[i] = 0.f;
            }
        }
    }
    if (tid == 0) a.counts[u] = make_int2(holes, m);
}

// A warp takes the pairs of one destination page: the lanes hold 8 bytes of
// each of its 16 rows.
constexpr int kMoveWarps = 8;

template <int kFmt>
__global__ void __launch_bounds__(kMoveWarps * 32) k_evict_move(const EvictArgs a)
{
    pdl_wait();
    const int u = blockIdx.y, r = u / a.hkv, j = u % a.hkv, lane = threadIdx.x & 31;
    const int2 cnt = a.counts[u];
    if (blockIdx.x == 0 && threadIdx.x == 0 && j == 0) a.new_lens[r] = cnt.y;
    const int32_t *table = a.page_table + static_cast<size_t>(r) * a.max_pages;
    const int2 *moves = a.moves + static_cast<size_t>(u) * (a.max_pages * (kPageSize / 2));
    uint2 *kp = static_cast<uint2 *>(a.k_pool), *vp = static_cast<uint2 *>(a.v_pool);
    for (int i = blockIdx.x * kMoveWarps + (threadIdx.x >> 5); i < cnt.x; i += gridDim.x * kMoveWarps) {
        const int page = moves[i].x / kPageSize;
        if (i > 0 && moves[i - 1].x / kPageSize == page) continue;   // the page's first pair does the page
        const int p = table[page];
        const size_t blk = static_cast<size_t>(p) * a.hkv + j;
        uint2 row[kPageSize];
        // the source of each row: lane t holds row t's
        int src = -1;
        if (lane < kPageSize && i + lane < cnt.x) {
            const int2 mv = moves[i + lane];
            if (mv.x / kPageSize == page) src = mv.y | (mv.x % kPageSize) << 24;
        }
        int from = -1;                                              // lane t: the slot that moves into row t
#pragma unroll
        for (int t = 0; t < kPageSize; ++t) {
            const int s = __shfl_sync(0xffffffffu, src, t);
            if (s >= 0 && (s >> 24) == lane) from = s & 0xFFFFFF;
        }
        if (lane < kPageSize && from >= 0) {
            const size_t si = (static_cast<size_t>(table[from / kPageSize]) * a.hkv + j) * kPageSize + from % kPageSize;
            const size_t di = blk * kPageSize + lane;
            a.weights[di] = a.weights[si];
            a.positions[di] = a.positions[si];
            a.weights[si] = 0.f;
            a.positions[si] = -1;
        }
        const bool renew = a.summ != nullptr && (page + 1) * kPageSize <= cnt.y;
#pragma unroll
        for (int t = 0; t < kPageSize; ++t) {
            const int f = __shfl_sync(0xffffffffu, from, t);
            row[t] = make_uint2(0u, 0u);
            const size_t d = (blk * kPageSize + t) * (kHeadDim / 4) + lane;
            if (f >= 0) {
                const size_t s = ((static_cast<size_t>(table[f / kPageSize]) * a.hkv + j) * kPageSize + f % kPageSize) *
                                     (kHeadDim / 4) + lane;
                row[t] = kp[s];
                kp[d] = row[t];
                vp[d] = vp[s];
            } else if (renew) {
                row[t] = kp[d];
            }
        }
        if (renew) store_summary_warp<kFmt>(row, static_cast<uint8_t *>(a.summ), p, j, a.hkv);
    }
}

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream)
{
    const int units = a.batch * a.hkv;
    k_evict_plan<<<units, kPlanThreads, 0, stream>>>(a);
    const int per = (sms * 8 + units - 1) / units;
    const int most = (a.max_pages * (kPageSize / 2) + kMoveWarps - 1) / kMoveWarps;
    const dim3 grid(per < most ? per : most, units);
    if (a.fmt == kSummQ8)
        k_evict_move<kSummQ8><<<grid, kMoveWarps * 32, 0, stream>>>(a);
    else if (a.fmt == kSummQ2)
        k_evict_move<kSummQ2><<<grid, kMoveWarps * 32, 0, stream>>>(a);
    else
        k_evict_move<kSummBf16><<<grid, kMoveWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace moira
