// The device-side plan of the shared-prefix attention: which block computes
// which part of which prefix, from the group starts and prefix lengths alone,
// and where its partials lie (k_prefix in shared.cu, k_finish in finish.cu).
#pragma once

#include "moira_device.cuh"
#include "moira_launch.h"
#include "own_plan.cuh"

namespace moira {

constexpr int kTilePages = kTileKeys / kPageSize;

// The blocks work in teams of R: the members of a team take the same keys at
// the same time for R row tiles, so that a key tile comes from memory once and
// from L2 for the others (256 requests on a 32k prefix, 4 row tiles: without
// teams the keys and values were read 4.3 times from memory).  R is the
// number of row tiles when every group with a prefix has the same, else 1; more
// than kMaxTeam row tiles are done in rounds.  Groups of unequal row tiles so
// read each key tile once a row tile (two groups behind 32k tokens each, 8 heads:
// 128 and 128 requests 176 us, 64 and 192 183 us, 200 and 56 210 us; 100, 100
// and 100 239 us, 20, 70 and 200 276 us).
// The groups' work, laid end to end: group g has hkv * rounds(g) units of
// tiles(g) key tiles each, unit = head * rounds + round.
struct GroupPlan {
    int team;                                       // R
    int woff[kMaxGroups + 1];                       // key tiles before the group
    uint16_t start[kMaxGroups + 1];                 // first request (sanitised: ascending, within the batch)
};
static_assert(kMaxUnits < 65536, "request indices fit 16 bits");

// The plan as block 0 leaves it in the workspace for the merge.
struct PlanRecord {
    int team, blocks;                               // R; blocks of k_prefix that take part
    int start[kMaxGroups + 1], woff[kMaxGroups + 1];
    int uoff[kMaxGroups + 1];                       // units before the group
};
static_assert(sizeof(PlanRecord) <= kPlanBytes, "the workspace's plan record");

__host__ __device__ __forceinline__ int rtiles_of(int requests)
{
    return (requests * kGroup + kUnitRows - 1) / kUnitRows;
}
// The team when the groups that have work have rt_min to rt_max row tiles.
__host__ __device__ __forceinline__ int team_of(int rt_min, int rt_max)
{
    if (rt_min != rt_max) return 1;
    const int rounds = (rt_max + kMaxTeam - 1) / kMaxTeam;
    return rounds == 1 ? rt_max : (rt_max + rounds - 1) / rounds;
}
__host__ __device__ __forceinline__ int rounds_of(int requests, int team)
{
    const int rt = rtiles_of(requests);
    return team == 1 ? rt : rt <= team ? (rt > 0) : (rt + team - 1) / team;
}
__host__ __device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }
// Units of a group, for one head.  A group without a prefix has none: every
// unit takes a team's partial slots, and the team is that of the groups with
// work, so prefix_units_max counts the units of those alone.
__host__ __device__ __forceinline__ int group_units(int requests, int len, int team)
{
    return len > 0 ? rounds_of(requests, team) : 0;
}
__device__ __forceinline__ int prefix_len(const SharedArgs &a, int g)
{
    return min(max(__ldcg(a.prefix_lens + g), 0), a.prefix_pages * kPageSize);
}

// One warp of the block fills the plan; block 0 records it.  `total`: the
// work, for the split of the SMs.
__device__ __forceinline__ void plan_groups(const SharedArgs &a, GroupPlan &p, int2 &total)
{
    const int lane = threadIdx.x & 31;
    const int cap = a.prefix_pages * kPageSize;
    int before = 0;                                 // carried over the chunks of 32 groups
    bool bad = false;
    int rt_min = 0x7FFFFFFF, rt_max = 1;
    int req = 0, len = 0;                           // of the lane's group in the last chunk
#pragma unroll 1
    for (int base = 0; base < a.groups; base += 32) {
        const int g = base + lane;
        const bool in = g < a.groups;
        int raw = 0, next = 0;
        len = 0;
        if (in) {
            raw = __ldcg(a.group_starts + g);
            next = __ldcg(a.group_starts + g + 1);
            len = __ldcg(a.prefix_lens + g);
        }
        bad |= in && (raw < 0 || next < raw || next > a.batch || len < 0 || len > cap);
        // running maxima make the starts ascending whatever was given
        int s = max(min(max(raw, 0), a.batch), before);
        const int e = min(max(next, 0), a.batch);
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s = max(s, y);
        }
        int sn = __shfl_down_sync(0xffffffffu, s, 1);           // the next group's start
        if (g == a.groups - 1 || lane == 31) sn = max(e, s);
        req = in ? max(sn - s, 0) : 0;
        if (req > 0 && len > 0) {
            rt_min = min(rt_min, rtiles_of(req));
            rt_max = max(rt_max, rtiles_of(req));
        }
        if (in) {
            p.start[g] = static_cast<uint16_t>(s);
            if (g == a.groups - 1) p.start[a.groups] = static_cast<uint16_t>(s + req);
        }
        before = __shfl_sync(0xffffffffu, s + req, 31);
    }
    if (bad) raise_status(a.status, kDevBadLen);
    rt_min = __reduce_min_sync(0xffffffffu, rt_min);
    rt_max = __reduce_max_sync(0xffffffffu, rt_max);
    const int team = team_of(rt_min, rt_max);
    PlanRecord *rec = static_cast<PlanRecord *>(a.plan);
    const bool write = blockIdx.x == 0;
    if (lane == 0) {
        p.team = team;
        if (write) rec->team = team;
    }
    __syncwarp();
    int w = 0, u = 0, narrow = 0, wide = 0;
#pragma unroll 1
    for (int base = 0; base < a.groups; base += 32) {
        const int g = base + lane;
        const bool in = g < a.groups;
        if (a.groups > 32) {
            req = in ? p.start[g + 1] - p.start[g] : 0;
            len = in ? __ldcg(a.prefix_lens + g) : 0;
        }
        const int units = in ? a.hkv * group_units(req, len, team) : 0;
        const int work = units * tiles_of(min(max(len, 0), cap));
        if (in) {
            const int2 pw = prefix_work(req, min(max(len, 0), cap), a.hkv);
            narrow += pw.x;
            wide += pw.y;
        }
        int wi = work, ui = units;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int yw = __shfl_up_sync(0xffffffffu, wi, o), yu = __shfl_up_sync(0xffffffffu, ui, o);
            if (lane >= o) {
                wi += yw;
                ui += yu;
            }
        }
        const bool last = g == a.groups - 1;
        if (in) {
            p.woff[g] = w + wi - work;
            if (last) p.woff[a.groups] = w + wi;
            if (write) {
                rec->start[g] = p.start[g];
                rec->woff[g] = w + wi - work;
                rec->uoff[g] = u + ui - units;
                if (last) {
                    rec->start[a.groups] = p.start[a.groups];
                    rec->woff[a.groups] = w + wi;
                }
            }
        }
        w += __shfl_sync(0xffffffffu, wi, 31);
        u += __shfl_sync(0xffffffffu, ui, 31);
    }
    narrow = __reduce_add_sync(0xffffffffu, narrow);
    wide = __reduce_add_sync(0xffffffffu, wide);
    if (lane == 0) total = make_int2(narrow, wide);
}

// Team b's share of W work items on n teams is [b*W/n, (b+1)*W/n).  The
// products stay below 2^32: n is at most the SM count, W at most 9 million
// (32 heads, 128 requests in as many groups, 2048 key tiles each).
__host__ __device__ __forceinline__ int share_lo(int b, int W, int n)
{
    return static_cast<int>(static_cast<uint32_t>(b) * static_cast<uint32_t>(W) / static_cast<uint32_t>(n));
}
// The team whose share holds item k.
__host__ __device__ __forceinline__ int share_of(int k, int W, int n)
{
    return static_cast<int>((static_cast<uint32_t>(k + 1) * static_cast<uint32_t>(n) - 1u) / static_cast<uint32_t>(W));
}

// The partial of team `team`, unit `unit`, member `member`.
__host__ __device__ __forceinline__ size_t partial_slot(int team, int unit, int member, int R)
{
    return (static_cast<size_t>(team) + unit) * R + member;
}

// The tensor cores add into fp32 accumulators by truncation, so a long chain of
// adds drifts towards zero (about 1.7e-8 of the value per 16-key step); after
// this many tiles a stream adds its accumulator to its partial in fp32.  (Never:
// 1.5e-5 off on 128k tokens.  With more than 128 rows, where the softmax warps
// have no time to spare, every 8 tiles: 2.9e-6, every 4 2.1e-6 and 8% longer,
// every tile 1.6e-6 and 55%.  With at most 128 rows they wait for the loads: 8
// requests on 128k, every 8 tiles 2.7e-6 and 108 us, every 2 1.6e-6 and 105 us,
// every tile 1.2e-6 and 105 us, but 32 requests then 152 us, not 125.  A share of
// a few tiles does not stop for it: 32 requests on 8k, 1.7e-6 and 40 us, every 2
// tiles 1.3e-6 and 43 us.)
constexpr int kChainTiles = 8, kChainNarrow = 2;

// A block's part of one unit: key tiles [t0, t1) of group g for the rows
// [row0, row0 + rows) of KV head j (row = request of the group * 4 + head).
struct Segment {
    int g, j, unit, row0, rows, t0, t1;
    // more than 128 rows: each stream has its own rows and takes every tile;
    // else both have the same rows and take alternate tiles
    __host__ __device__ __forceinline__ bool wide() const { return rows > kStreamRows; }
    __host__ __device__ __forceinline__ int tiles(int stream) const { return wide() ? t1 - t0 : (t1 - t0 + 1 - stream) >> 1; }
    // tiles that O adds up in tensor memory (a power of two)
    __host__ __device__ __forceinline__ int chain(int stream) const
    {
        return wide() || tiles(stream) <= kChainTiles ? kChainTiles : kChainNarrow;
    }
};

// Walks the segments of the block's share; every role of the block walks its
// own.  (hkv is a power of two; one round of row tiles is the usual case: a
// segment costs one division.)
struct SegmentWalk {
    const GroupPlan &p;
    int hkv, hshift, member, w, w1, g, u;           // member of the team; u: units before group g
    __host__ __device__ __forceinline__ bool next(Segment &s)
    {
        while (w < w1) {
            int req = p.start[g + 1] - p.start[g];
            while (p.woff[g + 1] <= w) {
                if (p.woff[g + 1] > p.woff[g]) u += rounds_of(req, p.team) << hshift;
                ++g;
                req = p.start[g + 1] - p.start[g];
            }
            const int rounds = rounds_of(req, p.team);
            uint32_t tiles = static_cast<uint32_t>(p.woff[g + 1] - p.woff[g]) >> hshift;
            if (rounds > 1) tiles /= static_cast<uint32_t>(rounds);
            const uint32_t at = static_cast<uint32_t>(w - p.woff[g]), ug = at / tiles;
            const int round = rounds > 1 ? static_cast<int>(ug % static_cast<uint32_t>(rounds)) : 0;
            s.g = g;
            s.t0 = static_cast<int>(at - ug * tiles);
            s.t1 = min(static_cast<int>(tiles), s.t0 + w1 - w);
            s.j = static_cast<int>(rounds > 1 ? ug / static_cast<uint32_t>(rounds) : ug);
            s.unit = u + static_cast<int>(ug);
            s.row0 = (round * p.team + member) * kUnitRows;
            s.rows = min(kUnitRows, req * kGroup - s.row0);
            w += s.t1 - s.t0;
            if (s.rows > 0) return true;            // the last round may have fewer row tiles than the team members
        }
        return false;
    }
};

}  // namespace moira
