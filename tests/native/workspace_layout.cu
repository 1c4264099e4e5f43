// What the kernels keep at zero between calls (counters, barriers, histograms)
// must not be scratch of a call for other sizes on the same workspace.  Compares
// random pairs of layouts; prints the first overlap and ends with status 1.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "moira_device.cuh"

using namespace moira;

struct Range {
    const char *name;
    size_t from, to;
};

int main(int argc, char **argv)
{
    const int pairs = argc > 1 ? std::atoi(argv[1]) : 1000;
    std::mt19937 rng(1);
    auto below = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
    auto spread = [&](int n) { return 1 + below(1 + below(n)); };
    struct Call {
        int hkv, batch, pages, groups;
        bool weights;
        SharedLayout s;
        std::vector<Range> kept, scratch;
    };
    const int sms = 152, blocks = 304;
    auto make = [&]() {
        Call c{1 << below(6), 0, spread(kMaxPagesPerSeq), below(2) * spread(kMaxGroups), below(2) == 0, {}, {}, {}};
        c.batch = spread(below(2) ? kMaxUnits / c.hkv : 8);
        c.s = shared_layout(c.batch, c.hkv * kGroup, c.pages, blocks, c.groups, c.weights, sms);
        const WsLayout &w = c.s.base;
        const int units = c.batch * c.hkv;
        const size_t fu = units < kFusedMaxUnits ? units : kFusedMaxUnits, hq = static_cast<size_t>(c.hkv) * kGroup;
        c.kept = {{"status", w.status, w.status + 256},
                  {"counters", w.counters, w.counters + 4 * static_cast<size_t>(kMaxUnits)},
                  {"group counters", w.gcounters, w.gcounters + 4 * static_cast<size_t>(blocks + units)},
                  {"barriers", w.fbars, w.fbars + 4 * static_cast<size_t>(kBarWords) * (kFusedMaxUnits + 1)},
                  {"histograms", w.fl1, w.fl1 + 4 * static_cast<size_t>(kL1Stride) * fu}};
        c.scratch = {{"weights", w.scores, w.scores + 4 * c.batch * hq * weights_ld(c.pages)},
                     {"chunks", w.chunks, w.chunks + 4 * c.batch * hq * chunks_ld(c.pages)},
                     {"partials", w.partials, w.partials + 4 * static_cast<size_t>(kPartFloats) * (blocks + units)},
                     {"masses", w.fmass, w.fmass + 4 * fu * weights_ld(c.pages)},
                     {"shared", c.s.offsets, c.s.total}};
        return c;
    };
    for (int i = 0; i < pairs; ++i) {
        const Call a = make(), b = make();
        for (const Call *c : {&a, &b})
            for (const Range &x : c->kept)
                if (x.from % 256 != 0 || x.to > c->s.base.total) {
                    std::printf("%s: %zu to %zu of %zu\n", x.name, x.from, x.to, c->s.base.total);
                    return 1;
                }
        for (const Call *p : {&a, &b})
            for (const Call *q : {&a, &b})
                for (const Range &k : p->kept)
                    for (const Range &s : q->scratch)
                        if (k.from < s.to && s.from < k.to) {
                            std::printf("%s of %d requests, %d heads, %d pages (%zu to %zu) under %s of %d, %d, %d (%zu to %zu)\n",
                                        k.name, p->batch, p->hkv, p->pages, k.from, k.to, s.name, q->batch, q->hkv, q->pages,
                                        s.from, s.to);
                            return 1;
                        }
        for (size_t k = 0; k < a.kept.size(); ++k)
            for (size_t l = 0; l < b.kept.size(); ++l)
                if (k != l && a.kept[k].from < b.kept[l].to && b.kept[l].from < a.kept[k].to) {
                    std::printf("%s under %s\n", a.kept[k].name, b.kept[l].name);
                    return 1;
                }
    }
    std::printf("ok\n");
    return 0;
}
