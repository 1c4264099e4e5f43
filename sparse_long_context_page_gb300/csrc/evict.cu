// Eviction of cached tokens by accumulated attention weight.
//
// Per (request, KV head) with n > budget tokens, the `budget` tokens that come
// first in the order
//   protected (position < sinks, or among the `recent` newest) before others,
//   then larger weight, NaN last, then lower slot
// stay.  The kept tokens at slots >= budget move into the evicted slots below
// it, the i-th into the i-th (both ascending), so a token that stays below
// the budget is not touched and the moves are disjoint: they run in any order.
//
// k_evict_plan finds the cut and the pairs.  A token's place in the order is a
// 32-bit key; the m-th largest is found by a radix descent of 11, 11 and 10
// bits with histograms in shared memory, where the keys stay (every weight and
// position is read once, 8 bytes a token: the kernel's bound for long
// requests, latency for short ones).  Long requests of a small batch are
// split over a thread-block cluster, whose blocks add their histograms and
// scan their counts through distributed shared memory.
// k_evict_move moves keys, values, weights and positions and renews the
// summaries of the pages whose keys changed: bound by the rows' bytes.  Where
// each list has only a few moves, its block of k_evict_plan does them at once.
// Measured: 32 requests of 4112 tokens, 8 heads, cut to 4096: 19 us, latency (in
// two launches 22 us).  Plan and move: two requests of 64k cut to 8192: 24 us
// (eight blocks a list; four take 30 us, two 47 us) and 30 us; 64 of 500 to
// 20,000 cut to 2037: 36 us and 65 us at 4.5 TB/s (in one launch 122 us: its
// warps, short of registers, have half the rows in flight).  Summaries of 8 or 2
// bits cost more to renew: from a cold cache the 32 requests take 27 us with
// bf16 summaries, 50 us with either and 23 us without any, the two prompts 64,
// 113 and 56 us.
#include "moira_launch.h"
#include "summary_core.cuh"

namespace moira {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBins = 2048;                     // of a histogram, in groups of 32
constexpr int kPlanGroups = kPlanBins / 32;
static_assert(kPlanGroups * 8 == kPlanThreads && kPlanGroups % kPlanWarps == 0, "a thread for every (group, block)");
constexpr int kPlanHeld = 4;                        // quads a thread loads together
constexpr int kPlanMaxCluster = 8;                  // the portable size; 8 blocks hold the longest request

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

struct PlanSmem {
    int group[2][kPlanGroups];                      // sums of a histogram's groups, the passes in turn
    int group_all[kPlanGroups], bin_all[32];        // over the cluster: of the groups, of the cut's group's bins
    int2 warp[kPlanWarps];
    int last, first, top, bad;                      // of this block
    int last_all, first_all, top_all, bad_all;      // of the cluster
    int2 total[2];                                  // of this block, in the two scans
    int2 prefix, sum;                               // of the blocks before, of the cluster
    int2 start, mine;                               // the block's pairs in the lists: first, behind the last
};

// ---- the blocks of a cluster (one block: no exchange) --------------------------
__device__ __forceinline__ uint32_t plan_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t plan_blocks()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void plan_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *local, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    return a;
}
__device__ __forceinline__ int remote_int(const int *local, uint32_t rank)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}
// Exclusive scan of a pair of counts per thread over the block; the sums to everyone.
__device__ __forceinline__ int2 block_scan(int2 v, PlanSmem &sm, int2 &sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x.x, o), z = __shfl_up_sync(0xffffffffu, x.y, o);
        if (lane >= o) {
            x.x += y;
            x.y += z;
        }
    }
    __syncthreads();                                             // the last scan's sums are read
    if (lane == 31) sm.warp[warp] = x;
    __syncthreads();
    int2 before = make_int2(x.x - v.x, x.y - v.y);
    sum = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const int2 s = sm.warp[w];
        if (w < warp) {
            before.x += s.x;
            before.y += s.y;
        }
        sum.x += s.x;
        sum.y += s.y;
    }
    return before;
}

// The same over the cluster; `nth`: the kernel's first or second such scan.
__device__ __forceinline__ int2 cluster_scan(int2 v, PlanSmem &sm, uint32_t C, uint32_t rank, int nth, int2 &sum)
{
    int2 mine, before = block_scan(v, sm, mine);
    sum = mine;
    if (C > 1) {
        if (threadIdx.x == 0) sm.total[nth] = mine;
        plan_cluster_sync();
        if (threadIdx.x < 32) {
            int2 t = make_int2(0, 0);
            if (threadIdx.x < C)
                t = make_int2(remote_int(&sm.total[nth].x, threadIdx.x), remote_int(&sm.total[nth].y, threadIdx.x));
            const int ax = __reduce_add_sync(0xffffffffu, t.x), ay = __reduce_add_sync(0xffffffffu, t.y);
            const int px = __reduce_add_sync(0xffffffffu, threadIdx.x < rank ? t.x : 0);
            const int py = __reduce_add_sync(0xffffffffu, threadIdx.x < rank ? t.y : 0);
            if (threadIdx.x == 0) {
                sm.prefix = make_int2(px, py);
                sm.sum = make_int2(ax, ay);
            }
        }
        __syncthreads();
        before.x += sm.prefix.x;
        before.y += sm.prefix.y;
        sum = sm.sum;
    }
    return before;
}

// Shared memory of a block's keys and flags.
__host__ __device__ constexpr size_t plan_keys_bytes(int tokens)
{
    return static_cast<size_t>(tokens) * 4 + static_cast<size_t>(tokens / 4 + 15) / 16 * 16;
}

// ---- the moves ------------------------------------------------------------------
// A warp looks at a window of pairs and does every destination page whose first
// pair lies in it: the lanes hold 8 bytes of each of the page's 16 rows.  A few
// evictions a request lie each in another page: the window shrinks to the pairs
// there are for a warp, so that none does pages in a row while others have none
// (256 lists cut by 48 tokens: 42 us with windows of eight, 34 us so); at most
// eight, about half of a page's pairs.  (Looking the next window up while a
// page's rows load takes 7% longer, rows through a ring of 256-byte bulk copies
// 20%.)
constexpr int kMoveWarps = 8;
constexpr int kMoveBlocks = 2;                      // per SM
constexpr int kMoveWindow = 8;                      // a page's pairs reach at most 15 further

// Warp `warp` of `warps` moves its part of the n pairs of a list cut to m tokens.
// dst_of(i): pair i's destination slot; src_of(i): its source slot, weight and
// position, or the slot alone, which `complete` completes given the token's place
// in the pools.  kBoth: keys and values in flight together, else the values first.
template <int kFmt, bool kBoth, typename Dst, typename Src, typename Complete>
__device__ __forceinline__ void move_pages(const EvictArgs &a, int r, int j, int n, int m, int warp, int warps, Dst dst_of,
                                           Src src_of, Complete complete)
{
    constexpr int kRow = kHeadDim / 4;                            // uint2 of a row
    const int lane = threadIdx.x & 31;
    const int32_t *table = a.page_table + static_cast<size_t>(r) * a.max_pages;
    const uint2 *kp = static_cast<const uint2 *>(a.k_pool) + lane, *vp = static_cast<const uint2 *>(a.v_pool) + lane;
    const int window = min((n + warps - 1) / warps, kMoveWindow);
    for (int base = warp * window; base < n; base += warps * window) {
        // lane i: pair base + i, its destination page and the rows' places
        const int i = base + lane;
        int dst = -1, dpage = -1, prev = -1, dphys = 0, from = 0;
        int4 src = make_int4(0, 0, 0, 0);
        if (lane == 0 && base > 0) prev = dst_of(base - 1) / kPageSize;
        if (lane < window + kPageSize - 1 && i < n) {
            dst = dst_of(i);
            src = src_of(i);
            dpage = dst / kPageSize;
            dphys = __ldg(table + dpage);
            from = (__ldg(table + src.x / kPageSize) * a.hkv + j) * kPageSize + src.x % kPageSize;
            complete(src, from);
        }
        const int left = __shfl_up_sync(0xffffffffu, dpage, 1);
        if (lane > 0) prev = left;
        unsigned todo = __ballot_sync(0xffffffffu, lane < window && dpage >= 0 && dpage != prev);
        while (todo) {
            const int lead = __ffs(todo) - 1;
            todo &= todo - 1;
            const int page = __shfl_sync(0xffffffffu, dpage, lead), p = __shfl_sync(0xffffffffu, dphys, lead);
            const size_t blk = static_cast<size_t>(p) * a.hkv + j;
            const bool renew = a.summ != nullptr && (page + 1) * kPageSize <= m;
            if (dpage == page) {
                a.weights[blk * kPageSize + dst % kPageSize] = __int_as_float(src.y);
                a.positions[blk * kPageSize + dst % kPageSize] = src.z;
            }
            // members are in the order of their rows: row t's is the lead's
            // popc(filled rows below t)-th
            const unsigned filled = __reduce_or_sync(0xffffffffu, dpage == page ? 1u << (dst % kPageSize) : 0u);
            const int row_of = __shfl_sync(0xffffffffu, from, (lead + __popc(filled & ((1u << lane) - 1u))) & 31);
            const int own = static_cast<int>(blk) * kPageSize;
            uint2 *kd = static_cast<uint2 *>(a.k_pool) + blk * kPageSize * kRow + lane;
            uint2 *vd = static_cast<uint2 *>(a.v_pool) + blk * kPageSize * kRow + lane;
            uint2 row[kPageSize], val[kPageSize];
            auto load = [&](int t, bool keys, bool values) {
                const bool fill = filled >> t & 1u;
                const int f = __shfl_sync(0xffffffffu, row_of, t);
                const size_t at = static_cast<size_t>(fill ? f : own + t) * kRow;
                if (keys) row[t] = fill || renew ? kp[at] : make_uint2(0u, 0u);
                if (values) val[t] = fill ? vp[at] : make_uint2(0u, 0u);
            };
            if constexpr (!kBoth) {
#pragma unroll
                for (int t = 0; t < kPageSize; ++t) load(t, false, true);
#pragma unroll
                for (int t = 0; t < kPageSize; ++t)
                    if (filled >> t & 1u) vd[t * kRow] = val[t];
            }
#pragma unroll
            for (int t = 0; t < kPageSize; ++t) load(t, true, kBoth);
#pragma unroll
            for (int t = 0; t < kPageSize; ++t)
                if (filled >> t & 1u) {
                    kd[t * kRow] = row[t];
                    if constexpr (kBoth) vd[t * kRow] = val[t];
                }
            if (renew) store_summary_warp<kFmt>(row, static_cast<uint8_t *>(a.summ), p, j, a.hkv);
        }
    }
}

// kMove: one block a list, which also does its moves (kFmt: the summaries' format).
template <bool kMove, int kFmt>
__global__ void __launch_bounds__(kPlanThreads, 2) k_evict_plan(const EvictArgs a, int tokens)
{
    extern __shared__ uint4 keys4[];                             // [tokens / 4]: positions, then keys
    // a quad's tokens without a position (low four bits) and, later, the kept ones (high)
    uint8_t *flags = reinterpret_cast<uint8_t *>(keys4 + tokens / 4);
    // histograms: of a cluster's block two, which the passes use in turn (other
    // blocks may still read the last one)
    uint32_t *hists = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(keys4) + plan_keys_bytes(tokens));
    __shared__ PlanSmem sm;
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t C = kMove ? 1u : plan_blocks(), rank = kMove ? 0u : plan_rank();
    const int u = blockIdx.x / C, r = u / a.hkv, j = u & (a.hkv - 1);
    pdl_wait();
    pdl_trigger();
    const int raw = a.seq_lens[r], cap = a.max_pages * kPageSize;
    const int n = min(max(raw, 0), cap), m = min(n, a.budget);
    if (raw != n && tid == 0 && rank == 0) raise_status(a.status, kDevBadLen);
    if (n <= m) {                                                // the same for the whole cluster, and for every head
        if (tid == 0 && rank == 0) {
            if constexpr (!kMove) a.counts[u] = make_int2(0, n);
            else if (j == 0) a.new_lens[r] = n;
        }
        return;
    }
    // this block's tokens: whole pages [p0, ..), tokens t0 .. t0 + cnt - 1, in quads of four
    const int pages = (n + kPageSize - 1) / kPageSize, per = (pages + static_cast<int>(C) - 1) / static_cast<int>(C);
    const int p0 = min(static_cast<int>(rank) * per, pages), t0 = p0 * kPageSize;
    const int cnt = max(0, min(n, (p0 + per) * kPageSize) - t0), nq = (cnt + 3) / 4;
    const int32_t *table = a.page_table + static_cast<size_t>(r) * a.max_pages + p0;
    // a quad's first token in the pools, given its page
    auto quad_in = [&](int pid, int q) { return (static_cast<size_t>(pid) * a.hkv + j) * kPageSize + (q & 3) * 4; };
    auto quad_at = [&](int q) { return quad_in(__ldg(table + (q >> 2)), q); };
    if (tid == 0) {
        sm.last = -1;
        sm.first = 0x7FFFFFFF;
        sm.top = -1;
        sm.bad = 0;
    }
    __syncthreads();
    // new_lens may be seq_lens: of a request's blocks the last one here, after all
    // have read the length, writes it (the counter wraps to zero)
    bool writes = kMove && a.hkv == 1;
    if (kMove && a.hkv > 1 && tid == 0) {
        __threadfence();
        writes = atomicInc(&a.arrived[r], a.hkv - 1) == static_cast<uint32_t>(a.hkv - 1);
    }
    auto result = [&](int pairs, int len) {                      // of the list: for k_evict_move, or the new length itself
        if (tid != 0 || rank != 0) return;
        if constexpr (!kMove) a.counts[u] = make_int2(pairs, len);
        else if (writes) a.new_lens[r] = len;
    };

    // ---- positions; the first quads' weights load with them ---------------------
    int last = -1, first = 0x7FFFFFFF, top = -1, bad = 0;
    float4 held[kPlanHeld];
    for (int base = tid; base < nq; base += kPlanHeld * kPlanThreads) {
        int pid[kPlanHeld];
        int4 pos[kPlanHeld];
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            const int q = base + i * kPlanThreads;
            pid[i] = q < nq ? __ldg(table + (q >> 2)) : 0;
            if (pid[i] < 0 || pid[i] >= a.num_pages) {
                bad = 1;
                pid[i] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            const int q = base + i * kPlanThreads;
            if (q < nq) pos[i] = *reinterpret_cast<const int4 *>(a.positions + quad_in(pid[i], q));
            if (q < nq && base == tid) held[i] = *reinterpret_cast<const float4 *>(a.weights + quad_in(pid[i], q));
        }
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i) {
            const int q = base + i * kPlanThreads;
            if (q >= nq) continue;
            const int pv[4] = {pos[i].x, pos[i].y, pos[i].z, pos[i].w};
            uint32_t bits = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * q + e;
                if (t >= cnt) continue;
                if (pv[e] >= 0) {
                    last = max(last, pv[e]);
                } else {
                    first = min(first, t0 + t);
                    top = max(top, t0 + t);
                    bits |= 1u << e;
                }
            }
            keys4[q] = make_uint4(pos[i].x, pos[i].y, pos[i].z, pos[i].w);
            flags[q] = static_cast<uint8_t>(bits);
        }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    first = __reduce_min_sync(0xffffffffu, first);
    top = __reduce_max_sync(0xffffffffu, top);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        atomicMax(&sm.last, last);
        atomicMin(&sm.first, first);
        atomicMax(&sm.top, top);
        if (bad) sm.bad = 1;
    }
    __syncthreads();
    if (C > 1) plan_cluster_sync();
    else __syncthreads();
    if (tid < 32) {
        int l = -1, f = 0x7FFFFFFF, tp = -1, b = 0;
        if (tid < static_cast<int>(C)) {
            l = remote_int(&sm.last, tid);
            f = remote_int(&sm.first, tid);
            tp = remote_int(&sm.top, tid);
            b = remote_int(&sm.bad, tid);
        }
        l = __reduce_max_sync(0xffffffffu, l);
        f = __reduce_min_sync(0xffffffffu, f);
        tp = __reduce_max_sync(0xffffffffu, tp);
        b = __any_sync(0xffffffffu, b);
        if (tid == 0) {
            sm.last_all = l;
            sm.first_all = f;
            sm.top_all = tp;
            sm.bad_all = b;
        }
    }
    __syncthreads();
    if (sm.bad_all) {                                            // the request is left as it is, by every block
        if (C > 1) plan_cluster_sync();                          // none ends while another reads its shared memory
        if (tid == 0 && rank == 0) raise_status(a.status, kDevBadPage);
        result(-1, n);
        return;
    }
    Positions ps{sm.last_all, sm.first_all, sm.last_all, a.sinks, a.recent};
    if (sm.top_all >= 0) ps.newest = ps.of(-1, sm.top_all);

    // ---- keys ---------------------------------------------------------------
    auto make_keys = [&](int q, const float4 &w) {
        const uint4 p = keys4[q];
        const int t = t0 + 4 * q;
        auto key = [&](uint32_t pos, float x, int e) {
            return ps.safe(ps.of(static_cast<int>(pos), t + e)) ? kKeyProtected : weight_key(x);
        };
        keys4[q] = make_uint4(key(p.x, w.x, 0), key(p.y, w.y, 1), key(p.z, w.z, 2), key(p.w, w.w, 3));
    };
    for (int base = tid; base < nq; base += kPlanHeld * kPlanThreads) {
        if (base != tid) {
#pragma unroll
            for (int i = 0; i < kPlanHeld; ++i)
                if (base + i * kPlanThreads < nq)
                    held[i] = *reinterpret_cast<const float4 *>(a.weights + quad_at(base + i * kPlanThreads));
        }
#pragma unroll
        for (int i = 0; i < kPlanHeld; ++i)
            if (base + i * kPlanThreads < nq) make_keys(base + i * kPlanThreads, held[i]);
    }

    // ---- radix descent to the m-th largest key --------------------------------
    uint32_t cut = 0u;
    int need = m;                                                // of the keys that share the cut's prefix
    bool whole = false;                                          // every key that shares it stays
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
        uint32_t *hist = hists + (C > 1 ? (pass & 1) * kPlanBins : 0);
        int *group = sm.group[pass & 1];
        if (C == 1 && pass > 0) __syncthreads();                 // the last pass is read
        reinterpret_cast<uint4 *>(hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        int safe = 0;                                            // protected tokens, one bin of their own in pass 0
        for (int base = 0; base < nq; base += kPlanThreads) {
            const int q = base + tid;
            const uint4 k4 = q < nq ? keys4[q] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t kv[4] = {k4.x, k4.y, k4.z, k4.w};
            uint32_t bin[4];
            bool in[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t k = kv[e];
                in[e] = 4 * q + e < cnt && (pass == 0 || (k >> (above & 31)) == (cut >> (above & 31)));
                if (pass == 0 && in[e] && k == kKeyProtected) {
                    ++safe;
                    in[e] = false;
                }
                bin[e] = (k >> shift) & (pass == 2 ? 1023u : kPlanBins - 1u);
            }
            // weights tie in runs (new tokens have none yet): a quad of one bin adds
            // once, and a warp of one bin once for all
            if (in[0] && in[1] && in[2] && in[3] && bin[0] == bin[1] && bin[0] == bin[2] && bin[0] == bin[3]) {
                const unsigned act = __activemask();
                int same;
                __match_all_sync(act, bin[0], &same);
                if (!same) atomicAdd(&hist[bin[0]], 4u);
                else if (lane == __ffs(act) - 1) atomicAdd(&hist[bin[0]], 4u * __popc(act));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (in[e]) atomicAdd(&hist[bin[e]], 1u);
            }
        }
        if (pass == 0) {
            safe = __reduce_add_sync(0xffffffffu, safe);
            if (lane == 0 && safe) atomicAdd(&hist[kPlanBins - 1], static_cast<uint32_t>(safe));
        }
        __syncthreads();
        // The cut's group of 32 bins, then its bin, from the top; the sums over the
        // cluster's blocks are one value a thread (group or bin tid / 8 of block tid % 8).
#pragma unroll
        for (int i = 0; i < kPlanGroups / kPlanWarps; ++i) {
            const int g = (tid >> 5) * (kPlanGroups / kPlanWarps) + i;
            const int s = static_cast<int>(__reduce_add_sync(0xffffffffu, hist[g * 32 + lane]));
            if (lane == 0) group[g] = s;
        }
        if (C > 1) plan_cluster_sync();
        else __syncthreads();
        auto over_blocks = [&](const int *mine) {
            int v = (tid & 7) < static_cast<int>(C) ? remote_int(mine, tid & 7) : 0;
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            return v + __shfl_xor_sync(0xffffffffu, v, 1);
        };
        const int *groups = group;                               // of one block: where they are
        if (C > 1) {
            const int v = over_blocks(group + (tid >> 3));
            if ((tid & 7) == 0) sm.group_all[tid >> 3] = v;
            __syncthreads();
            groups = sm.group_all;
        }
        // lane i: groups 63 - 2i and 62 - 2i (every warp finds the same)
        const int g0 = groups[kPlanGroups - 1 - 2 * lane], g1 = groups[kPlanGroups - 2 - 2 * lane];
        int upto = g0 + g1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        int at = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;
        int before = __shfl_sync(0xffffffffu, upto - g0 - g1, at);
        const int first_of = __shfl_sync(0xffffffffu, g0, at);
        int cut_group = kPlanGroups - 1 - 2 * at;
        if (before + first_of < need) {
            before += first_of;
            --cut_group;
        }
        need -= before;
        const int *bins = reinterpret_cast<const int *>(hist) + cut_group * 32;
        if (C > 1) {
            if (tid < 256) {
                const int v = over_blocks(bins + (tid >> 3));
                if ((tid & 7) == 0) sm.bin_all[tid >> 3] = v;
            }
            __syncthreads();
            bins = sm.bin_all;
        }
        const int h = bins[31 - lane];
        upto = h;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        at = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;
        need -= __shfl_sync(0xffffffffu, upto - h, at);
        whole = need == __shfl_sync(0xffffffffu, h, at);
        cut |= static_cast<uint32_t>(cut_group * 32 + 31 - at) << shift;
    }

    // ---- pairs in slot order: thread tid takes consecutive quads ---------------
    const int each = (nq + kPlanThreads - 1) / kPlanThreads, q0 = min(nq, tid * each), q1 = min(nq, q0 + each);
    auto key_of = [](const uint4 &k4, int e) { return e == 0 ? k4.x : e == 1 ? k4.y : e == 2 ? k4.z : k4.w; };
    int rank_eq = 0;                                             // equal keys before this thread's tokens
    if (!whole) {
        int eq = 0;
        int2 sum;
        for (int q = q0; q < q1; ++q) {
            const uint4 k4 = keys4[q];
#pragma unroll
            for (int e = 0; e < 4; ++e) eq += 4 * q + e < cnt && key_of(k4, e) == cut;
        }
        rank_eq = cluster_scan(make_int2(eq, 0), sm, C, rank, 0, sum).x;
    }
    // the quad's kept tokens as bits; equals stay in slot order while they are needed
    auto kept = [&](int q, int &eq) {
        const uint4 k4 = keys4[q];
        uint32_t bits = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t k = key_of(k4, e);
            if (4 * q + e >= cnt) continue;
            const bool keep = k > cut || (k == cut && (whole || eq < need)) || (whole && k >= cut);
            eq += k == cut;
            bits |= static_cast<uint32_t>(keep) << e;
        }
        return bits;
    };
    // bits of a quad's tokens below m, and of those that exist
    auto below = [&](int q) {
        const int left = m - (t0 + 4 * q);
        return left >= 4 ? 0xFu : left <= 0 ? 0u : (1u << left) - 1u;
    };
    auto exist = [&](int q) {
        const int left = cnt - 4 * q;
        return left >= 4 ? 0xFu : (1u << left) - 1u;
    };
    int eq = rank_eq, holes = 0, movers = 0;
    for (int q = q0; q < q1; ++q) {
        const uint32_t keep = kept(q, eq), low = below(q), is = exist(q);
        holes += __popc(low & is & ~keep);
        movers += __popc(~low & keep);
        flags[q] |= static_cast<uint8_t>(keep << 4);
    }
    int2 pairs;
    const int2 at_pair = cluster_scan(make_int2(holes, movers), sm, C, rank, 1, pairs);
    // the last look at other blocks: none ends before all have had it
    if (C > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    // the lists in shared memory first (the keys are done with): this block's
    // holes from the front, its movers behind them, so that the stores below are
    // of whole warps
    int *order = reinterpret_cast<int *>(keys4);
    __syncthreads();
    if (tid == 0) sm.start = at_pair;                            // of the block's first pair in the list
    if (tid == kPlanThreads - 1) sm.mine = make_int2(at_pair.x + holes, at_pair.y + movers);
    __syncthreads();
    const int2 start = sm.start;
    const int n_holes = sm.mine.x - start.x, n_movers = sm.mine.y - start.y;
    int hi = at_pair.x - start.x, mi = n_holes + at_pair.y - start.y;
    for (int q = q0; q < q1; ++q) {
        const uint32_t keep = flags[q] >> 4, low = below(q), is = exist(q);
        for (uint32_t b = low & is & ~keep; b; b &= b - 1) order[hi++] = 4 * q + __ffs(b) - 1;
        for (uint32_t b = keep & ~low; b; b &= b - 1) order[mi++] = 4 * q + __ffs(b) - 1;
    }
    __syncthreads();
    if constexpr (kMove) {
        move_pages<kFmt, false>(
            a, r, j, n_holes, m, tid >> 5, kPlanWarps, [&](int i) { return order[i]; },
            [&](int i) { return make_int4(order[n_holes + i], 0, 0, 0); },
            [&](int4 &src, int at) {
                src.y = __float_as_int(a.weights[at]);
                src.z = ps.of(a.positions[at], src.x);
            });
    } else {
        const size_t list = static_cast<size_t>(u) * (a.max_pages * (kPageSize / 2));
        for (int k = tid; k < n_holes; k += kPlanThreads) a.dst[list + start.x + k] = t0 + order[k];
#pragma unroll 4
        for (int k = tid; k < n_movers; k += kPlanThreads) {
            const int t = order[n_holes + k];
            const size_t at = quad_at(t >> 2) + (t & 3);
            a.src[list + start.y + k] =
                make_int4(t0 + t, __float_as_int(a.weights[at]), ps.of(a.positions[at], t0 + t), 0);
        }
    }
    result(pairs.x, m);
    __syncthreads();                                             // the moved tokens are read
    // ---- the slots from m on, and positions of kept tokens that had none -------
#pragma unroll 4
    for (int q = tid; q < nq; q += kPlanThreads) {
        const uint32_t low = below(q), clear = exist(q) & ~low, fill = (flags[q] >> 4) & flags[q] & low;
        if (!(clear | fill)) continue;
        const size_t at = quad_at(q);
        if (clear == 0xFu) {
            *reinterpret_cast<float4 *>(a.weights + at) = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<int4 *>(a.positions + at) = make_int4(-1, -1, -1, -1);
            continue;
        }
        const int t = t0 + 4 * q;
        if (fill == 0xFu) {
            *reinterpret_cast<int4 *>(a.positions + at) =
                make_int4(ps.of(-1, t), ps.of(-1, t + 1), ps.of(-1, t + 2), ps.of(-1, t + 3));
            continue;
        }
        for (uint32_t b = clear; b; b &= b - 1) {
            a.weights[at + __ffs(b) - 1] = 0.f;
            a.positions[at + __ffs(b) - 1] = -1;
        }
        for (uint32_t b = fill; b; b &= b - 1) a.positions[at + __ffs(b) - 1] = ps.of(-1, t + __ffs(b) - 1);
    }
    if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int kFmt>
__global__ void __launch_bounds__(kMoveWarps * 32, kMoveBlocks) k_evict_move(const EvictArgs a)
{
    pdl_wait();
    const int u = blockIdx.y, r = u / a.hkv, j = u & (a.hkv - 1);
    const int2 cnt = a.counts[u];
    if (blockIdx.x == 0 && threadIdx.x == 0 && j == 0) a.new_lens[r] = cnt.y;
    const size_t list = static_cast<size_t>(u) * (a.max_pages * (kPageSize / 2));
    move_pages<kFmt, true>(
        a, r, j, cnt.x, cnt.y, blockIdx.x * kMoveWarps + (threadIdx.x >> 5), gridDim.x * kMoveWarps,
        [&](int i) { return a.dst[list + i]; }, [&](int i) { return a.src[list + i]; }, [](int4 &, int) {});
}

namespace {
std::atomic<int> g_plan_smem_seen[64], g_move_smem_seen[3][64];
constexpr size_t kPairSmem = 110 * 1024;                          // of each of two blocks of a SM

template <int kFmt>
cudaError_t launch_plan_move(const EvictArgs &a, int tokens, size_t smem, cudaStream_t stream)
{
    const cudaError_t e = raise_smem_limit(k_evict_plan<true, kFmt>, smem, g_move_smem_seen[kFmt]);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_evict_plan<true, kFmt>, dim3(a.batch * a.hkv), dim3(kPlanThreads), smem, stream, a, tokens);
}
}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream)
{
    const int units = a.batch * a.hkv;
    // The page table's width stands for the longest request (the lengths are on
    // the device).  Blocks of a (request, head): enough to fill the SMs, but at least one quad
    // a thread, and as many as the longest request needs to keep its keys in
    // shared memory (48k tokens a block).
    const long long longest = static_cast<long long>(a.max_pages) * kPageSize;
    int C = 1;
    while (C < kPlanMaxCluster &&
           (longest > 49152LL * C || (units * C < sms && longest >= 2LL * C * 4 * kPlanThreads)))
        C *= 2;
    const int tokens = (a.max_pages + C - 1) / C * kPageSize;
    const size_t smem = plan_keys_bytes(tokens) + sizeof(uint32_t) * kPlanBins * (C > 1 ? 2 : 1);
    // One launch where a list's block does its few moves as well: no list has more
    // moves than the block has warps, or windows if there are lists for all SMs.
    // (Lists of 4096 + x tokens cut by x, one launch against two: 256 lists 16:
    // 21 / 25 us, 128: 60 / 65 us, 512: 118 / 120 us; 512 lists 128: 109 / 110 us,
    // 512: 217 / 211 us.)
    const long long moves = longest - a.budget < a.budget ? longest - a.budget : a.budget;
    if (C == 1 && smem <= kPairSmem && moves <= (units >= sms ? kPlanWarps * kMoveWindow : kPlanWarps)) {
        if (a.fmt == kSummQ8) return launch_plan_move<kSummQ8>(a, tokens, smem, stream);
        if (a.fmt == kSummQ2) return launch_plan_move<kSummQ2>(a, tokens, smem, stream);
        return launch_plan_move<kSummBf16>(a, tokens, smem, stream);
    }
    cudaError_t e = raise_smem_limit(k_evict_plan<false, 0>, smem, g_plan_smem_seen);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * C);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, k_evict_plan<false, 0>, a, tokens);
    if (e != cudaSuccess) return e;
    const int per = (sms * 2 * kMoveBlocks + units - 1) / units;
    const int most = (a.max_pages * (kPageSize / 2) + kMoveWarps * kMoveWindow - 1) / (kMoveWarps * kMoveWindow);
    const dim3 grid(per < most ? per : most, units);
    const dim3 block(kMoveWarps * 32);
    if (a.fmt == kSummQ8) return launch_pdl(k_evict_move<kSummQ8>, grid, block, 0, stream, a);
    if (a.fmt == kSummQ2) return launch_pdl(k_evict_move<kSummQ2>, grid, block, 0, stream, a);
    return launch_pdl(k_evict_move<kSummBf16>, grid, block, 0, stream, a);
}

}  // namespace moira
