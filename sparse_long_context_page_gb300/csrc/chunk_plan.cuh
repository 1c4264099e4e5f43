// The device-side plan of the attention of a chunk of tokens: which block
// computes which part, from the requests' rows and lengths alone (k_chunk and
// k_chunk_join in chunk.cu).
//
// A request's n rows are cut into tiles of kChunkTokens; tile i of a KV head
// needs the first K_i key tiles of kTileKeys tokens (those that one of its rows
// sees, at least one).  All tiles laid end to end in the order (request, head,
// tile) make a line that the blocks share equally.  Its unit is about 900 clocks:
// a tile takes 7 units and 3 for each key tile, or, with half of its rows or less
// (narrow), 4 and 2 (over the blocks of ragged batches a tile took 7300 + 2700 K
// and 4700 + 1800 K clocks, before what it takes beside its key tiles became
// shorter; ragged batch 64.4 us with 8 and 5 units, 62.5 with 7 and 4, 67.1 with 6
// and 4, 63.0 with 9 and 6: one batch, where the cuts fall by chance counts as well).
// A share may begin and end inside a tile, whose keys are then split between
// neighbouring blocks and joined afterwards.
#pragma once

#include "token_device.cuh"

namespace moira {

// Loops that are to stay short code in the kernel.
#ifdef __CUDA_ARCH__
#define MOIRA_ROLLED _Pragma("unroll 1")
#else
#define MOIRA_ROLLED
#endif

constexpr int kMinPart = 2;                         // key tiles that a split leaves on either side
constexpr int kMinShare = 12;                       // least share of a block
struct ChunkCost {
    int start, key;                                 // of a tile, of one of its key tiles
};
// Key tiles that `units` pay for; the key is 3 or 2, each a product in the machine.
__host__ __device__ __forceinline__ int chunk_keys(int units, ChunkCost c)
{
    return c.key == 3 ? static_cast<int>(static_cast<uint32_t>(units) / 3u) : units >> 1;
}
__host__ __device__ __forceinline__ constexpr bool chunk_wide(int rows) { return rows > kChunkTokens / 2; }
__host__ __device__ __forceinline__ constexpr ChunkCost chunk_cost(int rows)
{
    return chunk_wide(rows) ? ChunkCost{7, 3} : ChunkCost{4, 2};
}
static_assert(chunk_cost(kChunkTokens).key == 3 && chunk_cost(1).key == 2, "chunk_keys divides by them");
// Two cuts never fall into the last part of one tile (chunk_min_part).
static_assert(kMinShare - kMinShare / 32 >= kMinPart * chunk_cost(kChunkTokens).key, "a share between two cuts has a part");

struct ChunkRequest {
    int from, n, L;                                 // first row, rows, tokens in the cache
};

// The rows and tokens of request r, clamped to what exists.
__host__ __device__ __forceinline__ ChunkRequest chunk_request(const int32_t *starts, const int32_t *lens, int r,
                                                               int tokens, int max_pages)
{
    ChunkRequest q;
    const int lo = starts[r], hi = starts[r + 1], L = lens[r], most = max_pages * kPageSize;
    q.from = lo < 0 ? 0 : lo > tokens ? tokens : lo;
    const int to = hi > tokens ? tokens : hi;
    q.n = to > q.from ? to - q.from : 0;
    q.L = L < 0 ? 0 : L > most ? most : L;
    return q;
}

// The tiles of one request for one head.  Causal: row x sees L - n + x + 1
// tokens, so K_i = max(1, (a + i) >> 1) with a = floor((L - n + 191) / 64) but for
// the last tile, whose last row sees all L; else K_i is the same for all.
struct ChunkTiles {
    int a;
    int tiles, last, rest;                          // tiles, K and rows of the last one
    bool causal;
    __host__ __device__ __forceinline__ ChunkTiles(const ChunkRequest &q, bool causal_)
        : a((q.L - q.n + 191) >> 6), tiles((q.n - 1 + kChunkTokens) / kChunkTokens),
          last(q.L > 0 ? (q.L + kTileKeys - 1) / kTileKeys : 1), causal(causal_)
    {
        static_assert(kChunkTokens == 64 && kTileKeys == 128, "K_i counts in halves");
        if (q.n == 0) tiles = 0;
        rest = q.n - (tiles - 1) * kChunkTokens;
    }
    __host__ __device__ __forceinline__ int keys(int i) const
    {
        if (!causal || i == tiles - 1) return last;
        const int k = (a + i) >> 1;
        return k > 1 ? k : 1;
    }
    __host__ __device__ __forceinline__ ChunkCost cost(int i) const { return chunk_cost(i == tiles - 1 ? rest : kChunkTokens); }
    // Cost of the tiles before tile i < tiles, all of them wide.
    __host__ __device__ __forceinline__ long long before(int i) const
    {
        constexpr ChunkCost c = chunk_cost(kChunkTokens);
        if (!causal) return static_cast<long long>(i) * (c.start + c.key * last);
        // the first x0 tiles need one key tile, the others (a + x) >> 1
        const int x0 = a >= 2 ? 0 : 2 - a < i ? 2 - a : i;
        return static_cast<long long>(i) * c.start + c.key * (x0 + (x0 < i ? halves(a + i) - halves(a + x0) : 0));
    }
    __host__ __device__ __forceinline__ long long total() const
    {
        if (tiles == 0) return 0;
        const ChunkCost c = cost(tiles - 1);
        return before(tiles - 1) + c.start + c.key * last;
    }

private:
    // sum of j >> 1 over 0 <= j < m
    __host__ __device__ static __forceinline__ long long halves(int m)
    {
        return m > 1 ? static_cast<long long>(static_cast<uint64_t>(m - 1) * static_cast<uint32_t>(m - 1) >> 2) : 0;
    }
};

// A place on the line: key tile k of tile i of head j of request r (k = 0: the
// tile's start), `at` units from the line's start.
struct ChunkPlace {
    int r, j, i, k;
    long long at;
};

// Key tiles that a cut leaves on either side of a tile of K: cuts that would
// split off a small part of a tile, and of a share, move to the tile's ends.
__host__ __device__ __forceinline__ int chunk_min_part(int K, long long share)
{
    const int of_tile = K / 32;
    return kMinPart + (share < 96 * of_tile ? static_cast<int>(static_cast<uint32_t>(share) / 96u) : of_tile);
}

// The place nearest before unit c of request r (c counted from the request's
// own first unit, which lies at `start`) where a share may begin; `share` is the
// shares' length.
__host__ __device__ __forceinline__ ChunkPlace chunk_place(const ChunkTiles &t, int r, long long c, long long start,
                                                           long long share)
{
    const long long head = t.total();
    ChunkPlace p;
    p.r = r;
    p.j = 0;
    p.at = start;
    MOIRA_ROLLED
    for (; c >= head; c -= head) {                  // at most 32 heads
        ++p.j;
        p.at += head;
    }
    int lo = 0, hi = t.tiles;                       // the last tile that starts at or before it
    MOIRA_ROLLED
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.before(mid) <= c) lo = mid;
        else hi = mid;
    }
    const long long first = t.before(lo);
    const int K = t.keys(lo);
    const ChunkCost cost = t.cost(lo);
    const int into = static_cast<int>(c - first) - cost.start;
    p.i = lo;
    const int part = chunk_min_part(K, share);      // a tile of less than two parts is never split
    p.k = into < part * cost.key ? 0 : chunk_keys(into, cost);
    if (p.k > K - part) p.k = K - part;
    if (p.k < part) p.k = 0;
    p.at += first + (p.k ? cost.start + cost.key * p.k : 0);
    return p;
}

constexpr int kL2Tiles = 1500;                      // key tiles, keys and values, that L2 holds (98 MB)

// What the number of blocks goes by, summed over the requests.
struct ChunkSums {
    long long units = 0;                            // the line's length
    int tiles = 0;
    int longest = 0;                                // units of the longest tile
    int cached = 0;                                 // key tiles of all heads; of one request, no more than matter
    __host__ __device__ __forceinline__ void add(const ChunkTiles &t, int hkv)
    {
        if (t.tiles == 0) return;
        units += hkv * t.total();
        tiles += hkv * t.tiles;
        const ChunkCost c = t.cost(t.tiles > 1 ? t.tiles - 2 : 0);      // the last tile may be narrow
        const int most = c.start + c.key * t.last;
        longest = most > longest ? most : longest;
        const int here = hkv * t.last;
        cached += here <= kL2Tiles ? here : kL2Tiles + 1;
    }
};

// Blocks that take part.  With a cache beyond L2, every key tile comes from
// memory once for each tile of q whose block is elsewhere in the keys at the
// time (512 tokens behind 128k: 4.3 of 0.5 GB, all that memory gives).  So where
// the tiles are alike and a number of blocks that gives each the same tiles, or
// the same part of one, takes 4 of 5 of the grid, that number it is: the blocks
// of a head then run through the keys side by side.  With 8 heads on 152 SMs that is
// so for 512, 1024, 2048 and 4096 tokens, and not for most numbers between them or for
// prompts of different lengths, whose shares are equal and lie anywhere in the keys.
__host__ __device__ __forceinline__ int chunk_blocks(const ChunkSums &s, int grid)
{
    const int most = s.units < static_cast<long long>(kMinShare) * grid ? static_cast<int>(s.units) / kMinShare : grid;
    const int n = most < 1 ? 1 : most;
    if (s.cached <= kL2Tiles || s.units < static_cast<long long>(s.tiles) * (s.longest - s.longest / 8)) return n;
    const int rounds = (s.tiles + grid - 1) / grid;
    const int even = s.tiles <= grid ? s.tiles * (grid / s.tiles) : (s.tiles + rounds - 1) / rounds;
    return even <= n && 5 * even >= 4 * n ? even : n;
}
// Where block b's share of W units begins, b W / n; the quotient is taken 16 bits
// at a time (a 64-bit division is a call, which would fix the kernel's registers).
struct ChunkShare {
    long long each;                                 // W / n
    uint32_t rest, n;                               // W % n
    ChunkShare() = default;
    __host__ __device__ __forceinline__ ChunkShare(long long W, int n_) : each(0), rest(0), n(static_cast<uint32_t>(n_))
    {
        MOIRA_ROLLED
        for (int i = 48; i >= 0; i -= 16) {
            const uint32_t cur = rest << 16 | static_cast<uint32_t>(W >> i & 0xFFFF);
            each = each << 16 | cur / n;
            rest = cur % n;
        }
    }
    __host__ __device__ __forceinline__ long long begin(int b) const
    {
        return each * b + static_cast<int>(rest * static_cast<uint32_t>(b) / n);
    }
};

// The blocks that have a part of a tile of `rows` rows which begins at unit `tile`
// and needs `keys` key tiles, of which block b has [t0, t1).
__host__ __device__ __forceinline__ void chunk_parts(const ChunkShare &share, long long tile, int rows, int keys, int b, int t0,
                                                     int t1, int &first, int &last)
{
    const ChunkCost cost = chunk_cost(rows);
    const long long keys_at = tile + cost.start;
    first = last = b;
    if (t0 > 0)                                     // back to the share that begins no later than the tile
        MOIRA_ROLLED while (share.begin(first) - keys_at >= chunk_min_part(keys, share.each) * cost.key) --first;
    if (t1 < keys)                                  // on to the share after which the tile is over
        MOIRA_ROLLED while (share.begin(last + 1) - keys_at < keys * cost.key) ++last;
}

// A part of a tile: key tiles [t0, t1) of `keys`.
struct ChunkSegment {
    int r, j, row, rows;                            // rows of q: first, count (1 .. kChunkTokens)
    int t0, t1, keys;
    int sees;                                       // tokens that the tile's first row sees (may be <= 0)
    int most;                                       // tokens that its last row sees (0 .. L)
    int first, last;                                // blocks that have a part of the tile
    bool causal;
    // More than half a tile: the streams hold different rows and share the
    // keys; else they hold the same rows and take alternate key tiles.
    __host__ __device__ __forceinline__ bool wide() const { return chunk_wide(rows); }
    __host__ __device__ __forceinline__ int tiles(int stream) const
    {
        return wide() ? t1 - t0 : (t1 - t0 + 1 - stream) >> 1;
    }
    __host__ __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == keys; }
    // Key tiles from here on hold tokens that some row does not see.
    __host__ __device__ __forceinline__ int edge() const { return sees > 0 ? sees / kTileKeys : 0; }
};

// The segments of one block's share, in order.
struct ChunkWalk {
    const int32_t *starts, *lens;
    int tokens, max_pages, batch, hkv;
    bool causal;
    ChunkPlace p;
    long long left;
    long long tile;                                 // where the current tile begins
    ChunkRequest q;
    __host__ __device__ __forceinline__ void begin(const ChunkPlace &from, const ChunkPlace &to)
    {
        p = from;
        left = to.at - from.at;
        tile = from.at;
        if (left <= 0) return;
        q = chunk_request(starts, lens, p.r, tokens, max_pages);
        const ChunkCost cost = ChunkTiles(q, causal).cost(p.i);
        if (p.k) tile -= cost.start + cost.key * p.k;
    }
    __host__ __device__ __forceinline__ bool next(ChunkSegment &s)
    {
        if (left <= 0) return false;
        const ChunkTiles t(q, causal);
        const int K = t.keys(p.i);
        const ChunkCost cost = t.cost(p.i);
        const int start = p.k == 0 ? cost.start : 0;
        int take = K - p.k;
        if (left < start + cost.key * take) take = chunk_keys(static_cast<int>(left - start), cost);
        if (left <= start || take <= 0) return false;
        s.r = p.r;
        s.j = p.j;
        s.row = q.from + p.i * kChunkTokens;
        s.rows = q.n - p.i * kChunkTokens < kChunkTokens ? q.n - p.i * kChunkTokens : kChunkTokens;
        s.t0 = p.k;
        s.t1 = p.k + take;
        s.keys = K;
        s.causal = causal;
        s.sees = s.most = q.L;
        if (causal) {
            s.sees = q.L - q.n + p.i * kChunkTokens + 1;
            s.most = s.sees + s.rows - 1 > 0 ? s.sees + s.rows - 1 : 0;
        }
        left -= start + cost.key * take;
        p.k = s.t1;
        if (p.k == K) {
            p.k = 0;
            tile += cost.start + cost.key * K;
            if (++p.i == t.tiles) {
                p.i = 0;
                if (++p.j == hkv) {
                    p.j = 0;
                    if (left > 0)
                        MOIRA_ROLLED
                        do {
                            if (++p.r >= batch) {
                                left = 0;
                                break;
                            }
                            q = chunk_request(starts, lens, p.r, tokens, max_pages);
                        } while (q.n == 0);
                }
            }
        }
        return true;
    }
};

// Where a part of a split tile leaves its partial: the part that begins the
// tile (and does not end it) in its block's second slot, every later part, of
// which a block has one at most, in the first.
__host__ __device__ __forceinline__ int chunk_slot(int block, bool begins) { return 2 * block + (begins ? 1 : 0); }

}  // namespace moira
