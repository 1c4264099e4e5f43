// The chunk attention's plan on the CPU: for random batches, bad row starts and
// lengths among them, the blocks' shares cover every tile's key tiles once and
// in order, split tiles lie in neighbouring blocks with one partial slot each,
// and the shares differ by little; the workspace's parts lie apart.  Ends with status 1 and a message otherwise.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "chunk_plan.cuh"

using namespace moira;

using I = long long;

int check(int cases)
{
    std::mt19937 rng(1);
    auto below = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
    auto spread = [&](int n) { return below(1 + below(1 + below(n))); };
    for (int c = 0; c < cases; ++c) {
        const int hkv = 1 << below(6), batch = 1 + spread(below(4) ? 40 : kMaxUnits / hkv), grid = below(3) ? 152 : 1 + below(200);
        const int max_pages = 1 + spread(below(4) ? 600 : kMaxPagesPerSeq), most = max_pages * kPageSize;
        const bool causal = below(3) != 0, bad = below(8) == 0;
        std::vector<int32_t> starts{0}, lens;
        for (int r = 0; r < batch; ++r) {
            const int n = below(5) ? spread(below(3) ? 300 : 9000) : 0;
            lens.push_back(below(4) ? std::min(most, n + spread(most)) : spread(most));
            starts.push_back(starts.back() + n);
            if (bad && below(3) == 0) starts.back() = static_cast<int32_t>(rng()) >> below(31), lens.back() = static_cast<int32_t>(rng()) >> below(31);
            if (bad && (starts.back() > 100000 || starts.back() < -100000)) starts.back() %= 100000;
        }
        const int tokens = std::max(1, (bad ? below(20000) : starts.back()) + spread(20));
        I W = 0;
        ChunkSums sums;
        std::vector<I> at;
        std::map<std::tuple<int, int, int>, int> want, done;
        for (int r = 0; r < batch; ++r) {
            const ChunkRequest q = chunk_request(starts.data(), lens.data(), r, tokens, max_pages);
            const ChunkTiles t(q, causal);
            at.push_back(W);
            I sum = 0;
            for (int i = 0; i < t.tiles; ++i) {
                // K from its definition
                const long long last = std::min<long long>(q.n, 64LL * (i + 1));
                long long vis = causal ? static_cast<long long>(q.L) - q.n + last : q.L;
                const int K = static_cast<int>(std::max<long long>(1, (std::max(vis, 0LL) + 127) / 128));
                const ChunkCost cost = chunk_cost(std::min(64, q.n - 64 * i));
                if (t.before(i) != sum || t.keys(i) != K) {
                    std::printf("tile %d of n %d L %d: before %lld not %lld, keys %d not %d\n", i, q.n, q.L, (long long)t.before(i), (long long)sum, t.keys(i), K);
                    return 1;
                }
                sum += cost.start + cost.key * K;
                for (int j = 0; j < hkv; ++j) want[{r, j, i}] = K;
            }
            if (t.total() != sum) return std::printf("total\n"), 1;
            W += sum * hkv;
            sums.add(t, hkv);
        }
        if (W == 0) continue;
        if (sums.units != W) return std::printf("sums\n"), 1;
        const int n = chunk_blocks(sums, grid);
        if (n < 1 || n > grid) return std::printf("blocks\n"), 1;
        const ChunkShare share(W, n);
        auto place = [&](I x) {
            if (x >= W) return ChunkPlace{batch, 0, 0, 0, W};
            int r = static_cast<int>(std::upper_bound(at.begin(), at.end(), x) - at.begin()) - 1;
            return chunk_place(ChunkTiles(chunk_request(starts.data(), lens.data(), r, tokens, max_pages), causal), r, x - at[r], at[r], share.each);
        };
        std::vector<int> used(2 * grid, 0);
        long long worst = 0;
        std::tuple<int, int, int> open{-1, 0, 0};
        int owner = -1, first = -1, last = -1;
        for (int b = 0; b < n; ++b) {
            const ChunkPlace lo = place(share.begin(b)), hi = place(share.begin(b + 1));
            if (lo.at > share.begin(b) || hi.at < lo.at) return std::printf("share of block %d\n", b), 1;
            worst = std::max(worst, hi.at - lo.at - W / n);
            ChunkWalk w{starts.data(), lens.data(), tokens, max_pages, batch, hkv, causal};
            w.begin(lo, hi);
            ChunkSegment s;
            long long cost = 0;
            int parts = 0;
            while (true) {
                const long long tile = w.tile;
                if (!w.next(s)) break;
                chunk_parts(share, static_cast<I>(tile), s.rows, s.keys, b, s.t0, s.t1, s.first, s.last);
                if (s.whole() && (s.first != b || s.last != b)) return std::printf("a whole tile has parts\n"), 1;
                const ChunkRequest q = chunk_request(starts.data(), lens.data(), s.r, tokens, max_pages);
                const std::tuple<int, int, int> key{s.r, s.j, (s.row - q.from) / kChunkTokens};
                cost += (s.t0 == 0 ? chunk_cost(s.rows).start : 0) + chunk_cost(s.rows).key * (s.t1 - s.t0);
                if (s.rows < 1 || s.rows > 64 || s.row < 0 || s.row + s.rows > tokens || s.keys != want[key] || done[key] != s.t0 ||
                    s.t1 <= s.t0 || s.t1 > s.keys || s.most > q.L || s.most < 0 || s.tiles(0) + (s.wide() ? 0 : s.tiles(1)) != s.t1 - s.t0 ||
                    (s.keys - 1) * kTileKeys >= std::max(1, s.most) || s.keys * kTileKeys < s.most)
                    return std::printf("segment of block %d: r %d j %d row %d rows %d keys [%d, %d) of %d\n", b, s.r, s.j, s.row, s.rows, s.t0, s.t1, s.keys), 1;
                done[key] = s.t1;
                if (!s.whole()) {
                    const int slot = chunk_slot(b, s.t0 == 0);
                    if (used[slot]++) return std::printf("slot %d twice\n", slot), 1;
                    ++parts;
                    // the chain that the join follows: owner, then the next blocks without a gap
                    if (s.t0 == 0) open = key, owner = b;
                    else if (open != key || owner != b - 1) return std::printf("chain broken at block %d\n", b), 1;
                    else owner = b;
                    if (s.t0 == 0) {
                        first = b, last = s.last;
                        if (s.first != b || last <= b) return std::printf("block %d begins a tile of blocks %d to %d\n", b, s.first, s.last), 1;
                    } else if (s.first != first || s.last != last || (s.t1 == s.keys) != (b == last)) {
                        return std::printf("block %d: parts of %d to %d, not %d to %d\n", b, s.first, s.last, first, last), 1;
                    }
                }
            }
            if (cost != hi.at - lo.at || parts > 2) return std::printf("block %d: %lld of %lld units, %d parts\n", b, cost, hi.at - lo.at, parts), 1;
        }
        if (want != done) return std::printf("tiles left out\n"), 1;
        if (worst > chunk_cost(64).start + (2 * kMinPart + W / n / 96 * 2 + 2) * chunk_cost(64).key + 1) return std::printf("a share is %lld units too long\n", worst), 1;
    }
    return 0;
}

int main(int argc, char **argv)
{
    const int cases = argc > 1 ? std::atoi(argv[1]) : 1000;
    if (check(cases)) return 1;
    // quotients of large lines
    for (long long W : {1LL, 151LL, 1LL << 31, (1LL << 45) + 12345, (1LL << 62) - 1})
        for (int n : {1, 7, 152, 1000})
            for (int b = 0; b <= n; ++b) {
                const __int128 want = static_cast<__int128>(W) * b / n;
                if (ChunkShare(W, n).begin(b) != static_cast<long long>(want)) return std::printf("share\n"), 1;
            }
    // the attention's workspace: its scratch begins behind what every other call keeps at zero
    for (int units = 1; units <= kMaxUnits; units += 13)
        for (int pages : {1, 100, kMaxPagesPerSeq}) {
            const WsLayout w = ws_layout(units, kGroup, pages, units, 304);
            const ChunkLayout c = chunk_layout(304, 152);
            if (c.records != w.scores || c.counters != w.counters || c.status != w.status || c.counters + 4 * 152 > w.gcounters ||
                c.records % 256 || c.partials % 256 || c.partials < c.records + 16 * 2 * 152 ||
                c.total < c.partials + 4ull * kChunkPart * 2 * 152)
                return std::printf("layout\n"), 1;
        }
    std::printf("ok\n");
    return 0;
}
