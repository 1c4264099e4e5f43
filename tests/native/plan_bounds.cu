// The shared-prefix attention's plan on the host: over random group tables
// (empty groups, empty prefixes, every head count) the walk of all blocks takes
// every (row tile, head, key tile) once, and every partial slot it names lies in
// the workspace.  Prints the first violation and ends with status 1.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "shared_plan.cuh"

using namespace moira;

struct Table {
    int hkv, batch, cap;                            // cap: tokens of a prefix table row
    std::vector<int> requests, lens;                // of each group
};

// plan_groups on the host (the table is in order: nothing to mend)
static void plan(const Table &t, GroupPlan &p, std::vector<int> &uoff)
{
    int rt_min = 0x7FFFFFFF, rt_max = 1;
    for (size_t g = 0; g < t.lens.size(); ++g)
        if (t.requests[g] > 0 && t.lens[g] > 0) {
            rt_min = min(rt_min, rtiles_of(t.requests[g]));
            rt_max = max(rt_max, rtiles_of(t.requests[g]));
        }
    p.team = team_of(rt_min, rt_max);
    int at = 0, w = 0, u = 0;
    for (size_t g = 0; g < t.lens.size(); ++g) {
        const int units = t.hkv * group_units(t.requests[g], t.lens[g], p.team);
        p.start[g] = static_cast<uint16_t>(at);
        p.woff[g] = w;
        uoff.push_back(u);
        at += t.requests[g];
        w += units * tiles_of(t.lens[g]);
        u += units;
    }
    p.start[t.lens.size()] = static_cast<uint16_t>(at);
    p.woff[t.lens.size()] = w;
}

static bool check(const Table &t, int sms, int blocks)
{
    static GroupPlan p;
    std::vector<int> uoff;
    plan(t, p, uoff);
    const int groups = static_cast<int>(t.lens.size()), R = p.team, W = p.woff[groups];
    auto bad = [&](const char *what, long long x, long long y) {
        std::printf("%s: %lld, %lld (hkv %d, batch %d, groups %d, team %d, blocks %d)\n", what, x, y, t.hkv, t.batch,
                    groups, R, blocks);
        for (int g = 0; g < groups && g < 20; ++g) std::printf("  %d requests, %d tokens\n", t.requests[g], t.lens[g]);
        return false;
    };
    if (static_cast<uint64_t>(W) * sms >= 1ull << 32) return bad("share products", W, sms);
    const int n = min(blocks / R, W);
    const size_t room = static_cast<size_t>(sms) + prefix_units_max(t.batch, t.hkv, groups);
    std::set<size_t> slots;
    long long done = 0, want = 0;
    for (int g = 0; g < groups; ++g)
        want += static_cast<long long>(t.hkv) * rtiles_of(t.requests[g]) * tiles_of(t.lens[g]);
    for (int block = 0; block < n * R; ++block) {
        const int b = block / R;
        SegmentWalk walk{p, t.hkv, 31 - __builtin_clz(t.hkv), block - b * R, share_lo(b, W, n), share_lo(b + 1, W, n), 0, 0};
        Segment s;
        while (walk.next(s)) {
            if (s.g < 0 || s.g >= groups || s.t0 < 0 || s.t1 > tiles_of(t.lens[s.g]) || s.t0 >= s.t1)
                return bad("segment", s.t0, s.t1);
            if (s.j < 0 || s.j >= t.hkv || s.row0 < 0 || s.row0 + s.rows > t.requests[s.g] * kGroup)
                return bad("rows", s.row0, s.rows);
            done += s.t1 - s.t0;
            const size_t slot = partial_slot(b, s.unit, walk.member, R);
            if (slot >= room) return bad("slot, room", slot, room);
            if (!slots.insert(slot).second) return bad("slot named twice", slot, s.unit);
            // where k_finish looks for it
            const int rounds = rounds_of(t.requests[s.g], R), rt = s.row0 / kUnitRows, round = rt / R;
            const int tiles = (p.woff[s.g + 1] - p.woff[s.g]) / (t.hkv * rounds);
            const int w0 = p.woff[s.g] + (s.j * rounds + round) * tiles;
            if (s.unit != uoff[s.g] + s.j * rounds + round || walk.member != rt - round * R) return bad("unit", s.unit, rt);
            if (b < share_of(w0, W, n) || b > share_of(w0 + tiles - 1, W, n)) return bad("team", b, w0);
        }
    }
    return done == want ? true : bad("tiles taken", done, want);
}

int main(int argc, char **argv)
{
    const int tables = argc > 1 ? std::atoi(argv[1]) : 2000;
    std::mt19937 rng(1);
    auto below = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
    auto spread = [&](int n) { return 1 + below(1 + below(n)); };
    auto run = [&](Table t, int blocks) {
        t.batch = 0;
        for (int r : t.requests) t.batch += r;
        if (t.batch == 0) t.batch = 1;
        return check(t, 152, blocks);
    };
    // empty prefixes before a group of several row tiles
    for (int hkv : {1, 2, 4, 8})
        for (int empty : {1, 3, 10, 255})
            for (int big : {33, 65, 129, 150, 300, 512}) {
                if (hkv * (empty + big) > kMaxUnits) continue;
                Table t{hkv, 0, 0, std::vector<int>(empty, 1), std::vector<int>(empty, 0)};
                t.requests.push_back(big);
                t.lens.push_back(32768);
                if (!run(t, 152)) return 1;
            }
    for (int i = 0; i < tables; ++i) {
        Table t{1 << below(6), 0, 0, {}, {}};
        const int most = kMaxUnits / t.hkv, groups = spread(min(kMaxGroups, most));
        // equal sizes (teams) or any; prefixes empty with any odds; the longest 256k tokens
        const int same = below(3) ? 0 : spread(most / groups), empty = below(4) * 33, longest = 1 << below(19);
        int left = most;
        for (int g = 0; g < groups; ++g) {
            int r = same ? same - below(2) : below(5) ? spread(max(1, 2 * left / (groups - g))) : 0;
            const int len = below(100) < empty ? 0 : spread(longest);
            if (same && len == 0) r = below(min(left, 300) + 1);      // other sizes without a prefix
            r = min(r, left);
            left -= r;
            t.requests.push_back(r);
            t.lens.push_back(len);
        }
        if (!run(t, below(3) ? 152 : kMaxTeam + below(152 - kMaxTeam + 1))) return 1;
    }
    std::printf("ok\n");
    return 0;
}
