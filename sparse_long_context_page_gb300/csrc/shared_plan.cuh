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
// number of row tiles when every group has the same, else 1; more than
// kMaxTeam row tiles are done in rounds.
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

__device__ __forceinline__ int rtiles_of(int requests) { return (requests * kGroup + kUnitRows - 1) / kUnitRows; }
__device__ __forceinline__ int rounds_of(int requests, int team) 
{
    const int rt = rtiles_of(requests);
    return team == 1 ? rt : rt <= team ? (rt > 0) : (rt + team - 1) / team;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }
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
    int team = 1;
    if (rt_min == rt_max) {
        const int rounds = (rt_max + kMaxTeam - 1) / kMaxTeam;
        team = rounds == 1 ? rt_max : (rt_max + rounds - 1) / rounds;
    }
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
        const int units = in ? a.hkv * rounds_of(req, team) : 0;
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
// products stay below 2^32: n is at most the SM count, W at most 8 heads of a
// few hundred row tiles and groups times 2048 key tiles.
__device__ __forceinline__ int share_lo(int b, int W, int n)
{
    return static_cast<int>(static_cast<uint32_t>(b) * static_cast<uint32_t>(W) / static_cast<uint32_t>(n));
}
// The team whose share holds item k.
__device__ __forceinline__ int share_of(int k, int W, int n)
{
    return static_cast<int>((static_cast<uint32_t>(k + 1) * static_cast<uint32_t>(n) - 1u) / static_cast<uint32_t>(W));
}

// The partial of team `team`, unit `unit`, member `member`.
__device__ __forceinline__ size_t partial_slot(int team, int unit, int member, int R)
{
    return (static_cast<size_t>(team) + unit) * R + member;
}

}  // namespace moira
