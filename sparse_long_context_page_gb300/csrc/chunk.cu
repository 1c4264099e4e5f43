// Attention of a chunk of tokens over the paged cache.
//
// Request r's new tokens are rows [starts[r], starts[r + 1]) of q; the i-th of n
// sees the first vis = L - n + i + 1 of the request's L cached tokens (causal)
// or all L of them:
//   out_h = sum_{t < vis} e^{s_t} v_t / sum_{t < vis} e^{s_t},  s_t = scale q_h . k_t
// and zero where vis <= 0.  The four query heads of a KV head are rows of one
// product: 64 tokens make a tile of 256 query rows, row 4 * token + head.
//
// k_chunk: one block per SM walks its share of all (tile, key tile) pairs
// (chunk_plan.cuh), its warps in four roles around two streams of 128 query
// rows (the 128 lanes of the tensor memory):
//   producer (1 warp)  works out the segments and hands them to the others; TMA
//                      page loads of keys and values into a ring of 32 KB tiles (128 tokens)
//   checker  (1 warp)  TMA loads of the queries; passes the value tiles on, once
//                      what some row does not see holds no value that is not finite
//   issuers  (2 warps) issue the tcgen05 products, one of each stream, in turns
//   softmax  (2 x 4 warps, one thread per row)
// Per key tile and stream
//   S = Q K^T   128 x 128 x 128, Q and K in shared memory (128-byte swizzle, K-major)
//   P = 2^(S - m), bf16, overwrites S in tensor memory
//   O += P V    A = P from tensor memory, B = V from shared memory (MN-major)
// While one stream is in its softmax the tensor cores work for the other.
// The row reference m moves only when a tile's maximum passes it by 2^8, so O
// in tensor memory is rarely rescaled.  Sums are fp32.  P enters its product as one
// bf16, at most 2^-8 of itself away, while the row sums take it unrounded: a second
// term would be a second product, 1024 clocks more a key tile.  Together with the
// output's own rounding, which alone leaves 0.0017 in relative L2, that leaves 0.0019
// to 0.0021.
//
// A token that some row of the tile does not see has P = 0 for that row, but
// 0 times an infinity is not 0.  So the checker zeroes such tokens' values that
// are not finite (no others) and marks the tile, and the softmax warps add them
// to the rows that do see them at the end: only then, so it costs nothing.
//
// The parts of tiles that were split between blocks are joined by their maxima
// and sums: by the last of the tile's blocks to be done with its part, or, where
// there are few tiles and each may have a part of every block, by k_chunk_join.
//
// What bounds it (8 KV heads): over long caches the turns of products and softmax;
// the products of a tile of 64 x 128 tokens take 2048 clocks, the tile 2700, under
// the power limit at 1.4 to 1.9 GHz (8k prompt 404 us, 512 tokens behind 128k 805 us:
// 1.35 PFLOP/s of what the mask leaves).  Few rows behind long caches: memory (5
// tokens of 16 requests behind 4k to 32k 137 us, 6.1 TB/s).  Short requests: what a
// tile costs beside its key tiles, 6000 to 7000 clocks, and a block some 15,000 at its
// ends, much of it instructions: the roles' code is 98 KB (and 8 KB that only tiles
// of more than four parts run), of which every tile runs most once, and more than the
// SM's instruction cache holds (one token on encoder states: 26% of its requests
// missed with 118 KB of code and the next level was busy 60% of the time, 57 us; 19%,
// 54% and 50 us with 98 KB).  So what runs once a tile is kept short, in rolled loops;
// the loops over key tiles are unrolled.
//
// Tried without gain (8k prompt where not said): a softmax without the tile's own
// maximum, checked afterwards, 413 to 441 us; exponentials in a rolled loop or with
// the scores read again, 434 to 450; keys and values by two producers, none; parts
// joined at the block's end, ragged batch 9 us more; the last part joined from
// tensor memory without a trip through L2, ragged batch 1 us, one token on encoder
// states 4 us more (its code); parts published while the block goes on, 2 us more.
#include "chunk_plan.cuh"
#include "token_launch.h"

namespace moira {

namespace {

constexpr int kSlots = 5;                                        // of the ring
constexpr int kTileBytes = kTileKeys * kHeadDim * 2;              // 32 KB
constexpr int kHalfTile = kTileKeys * 128;                       // of the queries: 128 rows x 128 B
// A page of keys or values is one copy of 4 KB that leaves its two groups of 8
// tokens one after the other, each as two halves of 64 elements (8 rows x 128
// B, the swizzle's unit): the groups of all pages then lie kGroupBytes apart.
constexpr int kPageBytes = kPageSize * kHeadDim * 2, kAtomBytes = 1024, kGroupBytes = 2 * kAtomBytes;
constexpr int kTilePages = kTileKeys / kPageSize;
constexpr int kStreamTokens = kChunkTokens / 2;                  // rows of q of one stream
constexpr int kSoftmaxWarps = 4;                                 // of one stream
constexpr int kProducerWarp = 2 * kSoftmaxWarps, kCheckerWarp = kProducerWarp + 1, kIssuerWarp = kProducerWarp + 2;
constexpr int kChunkThreads = (kIssuerWarp + 2) * 32;            // whole warpgroups
// Registers of a thread: 168 at launch, then the softmax warpgroups take what the third leaves.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 96;
static_assert(2 * kSoftmaxWarps * 32 * kSoftmaxRegs + 128 * kOtherRegs <= kChunkThreads * 168, "what the block was launched with");
constexpr int kNoteRing = 16;                                    // tiles whose notes are kept
constexpr int kSegments = 4;                                     // segments handed out and not yet taken by all
constexpr int kReaders = 2 * kSoftmaxWarps + 3;                  // warps that take them
constexpr float kMaxSlack = 8.f;                                 // log2 units a row's maximum may pass its reference by

struct ChunkSmem {
    unsigned long long full[kSlots], empty[kSlots];
    unsigned long long landed[kSlots];                           // a value tile's copies, before the checker passes it on
    unsigned long long q_full[2], q_free[2], s_full[2], o_full[2], half_full, half_free, done;
    unsigned long long p_full[2][2];                             // [stream][half of the keys]
    unsigned long long turn[2];                                  // the stream whose products are issued next
    uint32_t tmem;
    int abort;
    struct {
        long long units;
        int tiles, longest, cached;
    } sums[kChunkThreads / 32];                                  // of the plan's scan, by warps
    ChunkPlace place[2];                                         // the block's share
    ChunkShare share;
    int takes_part;                                              // it has one
    unsigned long long part_done, join_told;
    uint32_t join_here;                                          // this block joins the tile's parts
    unsigned long long seg_full[kSegments], seg_free[kSegments];
    ChunkSegment segment[kSegments];                             // one without rows ends the share
    uint32_t pages[kNoteRing];                                   // a tile's pages that are there, one bit each
    uint32_t spoilt[kNoteRing];                                  // set: the tile held values that are not finite
    float half_m[kStreamRows], half_l[kStreamRows];              // stream 1's, for stream 0 (narrow tiles)
};
constexpr int kChunkSmemBytes = (2 + kSlots) * kTileBytes + static_cast<int>(sizeof(ChunkSmem));
static_assert(kChunkSmemBytes <= 227 * 1024, "one block's shared memory");

// mbar_wait_g as one short piece of code: the roles' code together is larger than the
// SM's instruction cache, and this stands in it often.
__device__ __forceinline__ bool mbar_wait_c(uint32_t bar, uint32_t parity, const WaitGuard &g)
{
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        ".reg .b64 t0, t;\n"
        ".reg .b32 f;\n"
        "mov.b32 %0, 1;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "@p bra DONE;\n"
        "mov.u64 t0, %%globaltimer;\n"
        "AGAIN:\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "@p bra DONE;\n"
        "mov.b32 %0, 0;\n"
        "ld.volatile.shared::cta.b32 f, [%3];\n"
        "setp.ne.b32 p, f, 0;\n"
        "@p bra DONE;\n"
        "mov.b32 %0, 1;\n"
        "mov.u64 t, %%globaltimer;\n"
        "sub.u64 t, t, t0;\n"
        "setp.le.u64 p, t, %5;\n"
        "@p bra AGAIN;\n"
        "mov.b32 f, 1;\n"
        "st.volatile.shared::cta.b32 [%3], f;\n"
        "mov.b32 f, %6;\n"
        "red.or.b32 [%4], f;\n"
        "mov.b32 %0, 0;\n"
        "DONE:\n"
        "}"
        : "=&r"(done)
        : "r"(bar), "r"(parity), "r"(smem_u32(g.flag)), "l"(g.status), "n"(kWaitLimitNs), "n"(kDevTimeout)
        : "memory");
    return done != 0u;
}

// Columns of the tensor memory: S / P of the two streams, then O of the two.
__device__ __forceinline__ uint32_t tmem_s(uint32_t base, int stream) { return base + stream * 128; }
__device__ __forceinline__ uint32_t tmem_o(uint32_t base, int stream) { return base + 256 + stream * 128; }

// Position in the ring: slot and the parity of its current round.
struct Ring {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void advance()
    {
        if (++slot == kSlots) {
            slot = 0;
            round ^= 1u;
        }
    }
};

// The segments as the producer hands them out, one after the other.
struct Segments {
    int slot = 0;
    uint32_t round = 0;
    // False after the last one, or when a wait of the block has run out.
    __device__ __forceinline__ bool next(ChunkSmem &sm, ChunkSegment &s, const WaitGuard &wg)
    {
        if (!mbar_wait_c(smem_u32(&sm.seg_full[slot]), round, wg)) return false;
        s = sm.segment[slot];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.seg_free[slot]));
        advance();
        return s.rows > 0;
    }
    __device__ __forceinline__ void advance()
    {
        if (++slot == kSegments) {
            slot = 0;
            round ^= 1u;
        }
    }
};

// The ring holds a segment's tiles in the order in which the issuers first use
// them: `ahead` key tiles, then values and the next keys in turn.
__device__ __forceinline__ int keys_ahead(const ChunkSegment &s) { return s.wide() ? 1 : 2; }

// ---------------------------------------------------------------- the plan
// Every block finds its own share: each thread sums the costs of a run of
// requests, and the threads whose runs hold the share's two ends place them.
__device__ __forceinline__ void plan_share(const ChunkArgs &a, ChunkSmem &sm)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    const int each = (a.batch + kChunkThreads - 1) / kChunkThreads, r0 = min(tid * each, a.batch), r1 = min(r0 + each, a.batch);
    const int warps = (a.batch + 32 * each - 1) / (32 * each);       // those that have requests
    auto request = [&](int r) { return chunk_request(a.token_starts, a.seq_lens, r, a.tokens, a.max_pages); };
    long long sum = 0, upto = 0;
    if (warp < warps) {
        ChunkSums own;
#pragma unroll 1
        for (int r = r0; r < r1; ++r) {
            const ChunkRequest q = request(r);
            if (q.L != a.seq_lens[r]) raise_status(a.status, kDevBadLen);
            own.add(ChunkTiles(q, a.causal), a.hkv);
        }
        sum = upto = own.units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        own.tiles = __reduce_add_sync(0xffffffffu, own.tiles);
        own.longest = __reduce_max_sync(0xffffffffu, own.longest);
        own.cached = __reduce_add_sync(0xffffffffu, own.cached);
        if (lane == 31) sm.sums[warp] = {upto, own.tiles, own.longest, own.cached};
    }
    // up to 32 requests are one warp's, which the others need not wait for
    if (warps > 1) __syncthreads();
    else if (warp == 0) __syncwarp();
    else return;
    if (warp >= warps) {
        __syncthreads();
        return;
    }
    long long before = upto - sum;
    ChunkSums all;
#pragma unroll 1
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += sm.sums[w].units;
        all.units += sm.sums[w].units;
        all.tiles += sm.sums[w].tiles;
        all.longest = max(all.longest, sm.sums[w].longest);
        all.cached += sm.sums[w].cached;
    }
    const long long W = all.units;
    const int n = W == 0 ? 0 : chunk_blocks(all, gridDim.x);
    const ChunkShare share(W, max(n, 1));
    const long long c0 = share.begin(min(b, n)), c1 = share.begin(min(b + 1, n));
    // the threads whose runs hold the share's two ends find their requests, two lanes place them
    if (sum > 0 && c0 < before + sum && c1 >= before) {
        long long at = before;
#pragma unroll 1
        for (int r = r0; r < r1; ++r) {
            const long long cost = each == 1 ? sum : a.hkv * ChunkTiles(request(r), a.causal).total();
            if (c0 >= at && c0 < at + cost) sm.place[0].r = r, sm.place[0].at = at;
            if (c1 >= at && c1 < at + cost) sm.place[1].r = r, sm.place[1].at = at;
            at += cost;
        }
    }
    if (warps > 1) __syncthreads();
    else __syncwarp();
    if (tid < 2) {
        ChunkPlace &p = sm.place[tid];
        const long long c = tid == 0 ? c0 : c1;
        if (b >= n || c >= W) p = ChunkPlace{a.batch, 0, 0, 0, W};
        else p = chunk_place(ChunkTiles(request(p.r), a.causal), p.r, c - p.at, p.at, share.each);
        if (tid == 0) {
            sm.share.each = share.each, sm.share.rest = share.rest, sm.share.n = share.n;
            sm.takes_part = b < n;
        }
    }
}

// A role returns at the first of its waits that runs out (WaitGuard), and starts
// nothing after it; the copies and products it has started are waited for.

// ---------------------------------------------------------------- producer
struct ProducerState {
    Ring pos;
    uint32_t keys = 0u, keys_round = 0u;                         // bit: the slot's last copies are keys; their phase
    uint32_t values = 0u, values_round = 0u;                     // bit: the slot has had values; the next ones' phase
};

__device__ __forceinline__ void chunk_produce(const ChunkArgs &a, const CUtensorMap *map_k, const CUtensorMap *map_v,
                                              uint8_t *ring, ChunkSmem &sm, ProducerState &p, const WaitGuard &wg)
{
    const int lane = threadIdx.x & 31;
    ChunkWalk walk{a.token_starts, a.seq_lens, a.tokens, a.max_pages, a.batch, a.hkv, a.causal != 0};
    walk.begin(sm.place[0], sm.place[1]);
    Segments out;
    int n_keys = 0;                                              // key tiles so far
    while (true) {
        ChunkSegment s;
        const long long tile = walk.tile;
        if (!walk.next(s)) s.rows = 0;
        else chunk_parts(sm.share, tile, s.rows, s.keys, static_cast<int>(blockIdx.x), s.t0, s.t1, s.first, s.last);
        if (!mbar_wait_c(smem_u32(&sm.seg_free[out.slot]), out.round ^ 1u, wg)) return;
        if (lane == 0) {
            sm.segment[out.slot] = s;
            mbar_arrive(smem_u32(&sm.seg_full[out.slot]));
        }
        out.advance();
        if (s.rows == 0) return;
        const int32_t *table = a.page_table + static_cast<size_t>(s.r) * a.max_pages;
        // this lane's page of a key tile (8 lanes, one copy each); -1: nothing to load
        auto page_of = [&](int t) {
            const int x = t * kTilePages + lane;
            return lane < kTilePages && x >= 0 && x * kPageSize < s.most ? __ldg(table + x) : -1;
        };
        // one tile into the next ring slot
        auto load = [&](int t, int pid, bool keys) {
            const bool ok = pid >= 0 && pid < a.num_pages;
            const int slot = p.pos.slot;
            const uint32_t bar = smem_u32(keys ? &sm.full[slot] : &sm.landed[slot]);
            const unsigned there = __ballot_sync(0xffffffffu, ok);
            if (!mbar_wait_c(smem_u32(&sm.empty[slot]), p.pos.round ^ 1u, wg)) return false;
            if (lane == 0) {
                if (keys) sm.pages[n_keys % kNoteRing] = there;
                if (there) mbar_arrive_expect_tx(bar, __popc(there) * kPageBytes);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (ok)
                tma_load_4d(smem_u32(ring + slot * kTileBytes) + lane * kPageBytes, keys ? map_k : map_v, 0, 0, 0,
                            (pid * a.hkv + s.j) * 2, bar);
            else if (keys && lane < kTilePages && (t * kTilePages + lane) * kPageSize < s.most)
                raise_status(a.status, kDevBadPage);
            __syncwarp();
            const uint32_t bit = 1u << slot;
            if (keys) {
                ++n_keys;
                p.keys |= bit;
                p.keys_round = p.pos.round ? p.keys_round | bit : p.keys_round & ~bit;
            } else {
                p.keys &= ~bit;
                p.values |= bit;
                p.values_round ^= bit;
            }
            p.pos.advance();
            return true;
        };
        const int ahead = keys_ahead(s);
        int id[3];                                               // pages of the tiles t, t + 1 and t + 2
#pragma unroll
        for (int x = 0; x < 3; ++x) id[x] = page_of(s.t0 - ahead + x);
#pragma unroll 1
        for (int t = s.t0 - ahead; t < s.t1; ++t) {
            const int far = page_of(t + 3);
            // the values of tile t, the keys of tile t + ahead
            if (t >= s.t0 && !load(t, id[0], false)) return;
            if (t + ahead < s.t1 && !load(t + ahead, ahead == 1 ? id[1] : id[2], true)) return;
            id[0] = id[1], id[1] = id[2], id[2] = far;
        }
    }
}

// ---------------------------------------------------------------- checker
// Whether a 32-bit word holds a bf16 that is not finite, per half: 0xFFFF.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u); }
// The same in two operations: bit 15 or 31 is set (the others are noise).
__device__ __forceinline__ uint32_t infinite2(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }

struct QueryState {
    uint32_t had = 0u, phase = 0u;                               // bit: the stream has had queries; the last ones' phase
};

__device__ __forceinline__ void chunk_check(const CUtensorMap *map_q, uint8_t *q_smem, uint8_t *ring, ChunkSmem &sm,
                                            QueryState &queries, const WaitGuard &wg)
{
    const int lane = threadIdx.x & 31;
    Ring pos;
    uint32_t landed = 0u;                                        // bit: phase of the slot's next value tile
    int n_tiles = 0;                                             // key tiles of the block before this segment
    Segments in;
    ChunkSegment s;
    while (in.next(sm, s, wg)) {
#pragma unroll 1
        for (int st = 0; st < 2; ++st) {
            if (s.tiles(st) == 0) continue;
            // the products with the last segment's queries are done
            if (queries.had >> st & 1u) {
                if (!mbar_wait_c(smem_u32(&sm.q_free[st]), queries.phase >> st & 1u, wg)) return;
                queries.phase ^= 1u << st;
            }
            queries.had |= 1u << st;
            if (lane == 0) {
                const uint32_t bar = smem_u32(&sm.q_full[st]);
                mbar_arrive_expect_tx(bar, kTileBytes);
                // rows behind the request's (or the tensor's) belong to nobody's output here
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    tma_load_3d(smem_u32(q_smem) + st * kTileBytes + h * kHalfTile, map_q, h * 64, s.j * kGroup,
                                s.row + (s.wide() ? st * kStreamTokens : 0), bar);
            }
            __syncwarp();
        }
        const int ahead = keys_ahead(s);
#pragma unroll 1
        for (int x = 0; x < ahead && s.t0 + x < s.t1; ++x) pos.advance();
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t) {
            if (!mbar_wait_c(smem_u32(&sm.landed[pos.slot]), landed >> pos.slot & 1u, wg)) return;
            landed ^= 1u << pos.slot;
            const int note = (n_tiles + t - s.t0) % kNoteRing;
            const uint32_t there = sm.pages[note];
            bool spoilt = false;
            if (t >= s.edge() || there != 0xFFu) {
                uint8_t *v = ring + pos.slot * kTileBytes;
                // rows of the tile that the product reads (whole pages), and the first that some row of q does not see
                const int first = t * kTileKeys, count = min(max(s.most - first, 1), kTileKeys);
                const int end = (count + kPageSize - 1) / kPageSize * kPageSize;
                const uint32_t needed = (2u << (end / kPageSize - 1)) - 1u;
                const int from = (there & needed) != needed ? 0 : max(s.sees - first, 0);
                // a lane's 16 bytes of rows x, x + 2, ..: two rows are 32 lanes wide
                auto at = [&](int row) {
                    const int c = lane & 15;
                    return reinterpret_cast<uint4 *>(v + (row >> 3) * kGroupBytes + (c >> 3) * kAtomBytes + (row & 7) * 128 +
                                                     (((c & 7) ^ (row & 7)) << 4));
                };
                uint32_t found = 0u;
#pragma unroll 1
                for (int row = (from & ~15) + (lane >> 4); row < end; row += kPageSize) {
                    uint4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = *at(row + 2 * k);
#pragma unroll
                    for (int k = 0; k < 8; ++k) found |= infinite2(x[k].x) | infinite2(x[k].y) | infinite2(x[k].z) | infinite2(x[k].w);
                }
                if (__any_sync(0xffffffffu, (found & 0x80008000u) != 0u) || end > count || (there & needed) != needed) {
#pragma unroll 1
                    for (int row = from + (lane >> 4); row < end; row += 2) {
                        if (first + row >= s.most || !(there >> (row / kPageSize) & 1u)) {
                            *at(row) = make_uint4(0u, 0u, 0u, 0u);       // no row sees it, or its page is not there
                        } else if (first + row >= s.sees) {
                            const uint4 x = *at(row);
                            const uint4 m = make_uint4(not_finite2(x.x), not_finite2(x.y), not_finite2(x.z), not_finite2(x.w));
                            if (m.x | m.y | m.z | m.w) {
                                *at(row) = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
                                spoilt = true;
                            }
                        }
                    }
                }
            }
            spoilt = __any_sync(0xffffffffu, spoilt);
            if (lane == 0) sm.spoilt[note] = spoilt ? 1u : 0u;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.full[pos.slot]));
            pos.advance();
            if (t + ahead < s.t1) pos.advance();
        }
        n_tiles += s.t1 - s.t0;
    }
}

// ---------------------------------------------------------------- issuers
// One stream's products, by a warp of its own.  The tensor cores take products
// from a short queue, so whatever the issuing warp waits for between two groups
// of them (a barrier that is complete costs 100 to 200 clocks) leaves them idle:
// one warp for both streams issued a product every 111 clocks, which take 64.
// So each stream's warp waits for its tiles and for P first, then for its turn,
// and passes the turn on with its products queued.  Left to themselves, without
// turns, the two fall into step, both products first and then both softmaxes
// (8k prompt, before what has come since: one issuer 480 us, two without turns 514).
//   group 0: S of the first tile; group n: O += P V of tile n - 1, S of tile n
// The whole warp walks and waits, so that addresses and loop counts stay in
// uniform registers, which the product instructions read; one lane issues.
__device__ __forceinline__ void chunk_issue(uint32_t q_base, uint32_t ring, ChunkSmem &sm, int st, const WaitGuard &wg)
{
    constexpr uint32_t kIdescS = umma_idesc_bf16(128, kTileKeys, false);
    constexpr uint32_t kIdescO = umma_idesc_bf16(128, kHeadDim, true);
    constexpr uint32_t kTileStep = kTileBytes >> 4;
    const uint32_t tmem = warp_uniform(sm.tmem), tS = tmem_s(tmem, st), tO = tmem_o(tmem, st);
    // descriptors differ in the start address alone, in units of 16 bytes
    const uint32_t q_desc = umma_desc_lo(q_base, 16) + st * kTileStep, k_desc = umma_desc_lo(ring, 16),
                   v_desc = umma_desc_lo(ring, kAtomBytes);
    Ring pos;
    uint32_t q_par = 0u, p_par = 0u, turn_par = 0u;
    auto my_turn = [&]() {
        turn_par ^= 1u;
        return mbar_wait_c(smem_u32(&sm.turn[st]), turn_par ^ 1u, wg);
    };
    auto next_turn = [&]() {
        if (elect_one()) mbar_arrive(smem_u32(&sm.turn[st ^ 1]));
        __syncwarp();
    };
    auto wait_tile = [&](const Ring &r) { return mbar_wait_c(smem_u32(&sm.full[r.slot]), r.round, wg); };
    // an entry of the other stream's: seen, so that no round of the slot is missed, and left
    auto pass = [&](const Ring &r) {
        if (!wait_tile(r)) return false;
        if (elect_one()) mbar_arrive(smem_u32(&sm.empty[r.slot]));
        __syncwarp();
        return true;
    };
    auto take = [&]() {
        const Ring r = pos;
        pos.advance();
        return r;
    };
    // S of a key tile, by one lane; a slot is free when both streams are done with it
    auto qk = [&](const Ring &r, bool last) {
        const uint32_t kt = k_desc + r.slot * kTileStep;
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
            const uint32_t off_q = ((ks >> 2) * kHalfTile + (ks & 3) * 32) >> 4;
            const uint32_t off_k = ((ks >> 2) * kAtomBytes + (ks & 3) * 32) >> 4;
            umma_ss(tS, umma_desc(q_desc + off_q, 1024), umma_desc(kt + off_k, kGroupBytes), kIdescS, ks > 0);
        }
        umma_commit(smem_u32(&sm.s_full[st]));
        umma_commit(smem_u32(&sm.empty[r.slot]));
        if (last) umma_commit(smem_u32(&sm.q_free[st]));
    };
    Segments in;
    ChunkSegment s;
    while (in.next(sm, s, wg)) {
        const int T = warp_uniform(s.t1 - s.t0), t0 = warp_uniform(s.t0), most = warp_uniform(s.most);
        const bool wide = warp_uniform(s.wide());
        const int tiles = wide ? T : (T + 1 - st) >> 1, ahead = wide ? 1 : 2;
        if (tiles > 0) {
            if (!mbar_wait_c(smem_u32(&sm.q_full[st]), q_par, wg)) return;
            q_par ^= 1u;
        }
#pragma unroll 1
        for (int x = 0; x < min(ahead, T); ++x) {
            const Ring r = take();
            if (wide || x == st) {
                if (!wait_tile(r) || !my_turn()) return;
                tcgen05_fence_after();
                if (elect_one()) qk(r, tiles == 1);
                __syncwarp();
                next_turn();
            } else if (!pass(r)) {
                return;
            }
        }
        int n = 0;                                                // tiles of this stream so far
#pragma unroll 1
        for (int i = 0; i < T; ++i) {
            const bool more = i + ahead < T;
            const Ring vr = take();
            if (!wide && (i & 1) != st) {
                if (!pass(vr) || (more && !pass(take()))) return;
                continue;
            }
            Ring kr = vr;
            if (!wait_tile(vr)) return;
            if (more) {
                kr = take();
                if (!wait_tile(kr)) return;
            }
            // pages that some row sees
            const int pages = max(1, min(kTilePages, (most - (t0 + i) * kTileKeys + kPageSize - 1) / kPageSize));
            const uint32_t vt = v_desc + vr.slot * kTileStep;
            auto pv = [&](int ks, bool acc) {
                umma_ts(tO, tS + ks * 8, umma_desc(vt + ks * (kPageBytes >> 4), kGroupBytes), kIdescO, acc);
            };
            if (!mbar_wait_c(smem_u32(&sm.p_full[st][0]), p_par, wg) || !my_turn()) return;
            tcgen05_fence_after();
            if (elect_one()) {
                if (pages >= 4) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) pv(ks, ks > 0 || n > 0);
                } else {
#pragma unroll 1
                    for (int ks = 0; ks < pages; ++ks) pv(ks, ks > 0 || n > 0);
                }
            }
            __syncwarp();
            if (!mbar_wait_c(smem_u32(&sm.p_full[st][1]), p_par, wg)) return;
            tcgen05_fence_after();
            if (elect_one()) {
                if (pages == kTilePages) {
#pragma unroll
                    for (int ks = 4; ks < kTilePages; ++ks) pv(ks, true);
                } else {
#pragma unroll 1
                    for (int ks = 4; ks < pages; ++ks) pv(ks, true);
                }
                if (n + 1 == tiles) umma_commit(smem_u32(&sm.o_full[st]));
                if (more) qk(kr, n + 2 == tiles);
                umma_commit(smem_u32(&sm.empty[vr.slot]));
            }
            __syncwarp();
            next_turn();
            p_par ^= 1u;
            ++n;
        }
        // a narrow segment gives stream 0 up to two groups more: stream 1 passes on as many turns
        if (!wide && st == 1)
#pragma unroll 1
            for (int x = tiles > 0 ? tiles + 1 : 0; x < ((T + 1) >> 1) + 1; ++x) {
                if (!my_turn()) return;
                next_turn();
            }
    }
}

// ---------------------------------------------------------------- softmax
// Which of the 32 keys from `first` on a row counts: those of pages that are
// there (two bits) and below `vis`.
__device__ __forceinline__ uint32_t key_bits(uint32_t pages, int vis, int first)
{
    const uint32_t there = ((pages & 1u) ? 0xFFFFu : 0u) | ((pages & 2u) ? 0xFFFF0000u : 0u);
    const int n = vis - first;
    return there & (n >= 32 ? 0xFFFFFFFFu : n > 0 ? (1u << n) - 1u : 0u);
}

// The values that are not finite of the segment's tokens that some row does not
// see, added to 16 columns of a row that sees them.
__device__ __forceinline__ void add_spoilt(const ChunkArgs &a, const ChunkSegment &s, int vis, int run, float (&o)[16])
{
#pragma unroll 1
    for (int t = max(max(s.sees, 0), s.t0 * kTileKeys); t < min(vis, s.t1 * kTileKeys); ++t) {
        const int pid = __ldg(a.page_table + static_cast<size_t>(s.r) * a.max_pages + t / kPageSize);
        if (pid < 0 || pid >= a.num_pages) continue;
        const uint4 *v = static_cast<const uint4 *>(a.v_pool) +
                         ((static_cast<size_t>(pid) * a.hkv + s.j) * kPageSize + t % kPageSize) * 16 + run * 2;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint4 x = __ldg(v + c);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t m = not_finite2(w[i]);
                if (m & 0xFFFFu) o[8 * c + 2 * i] += bf16_lo(w[i]);
                if (m >> 16) o[8 * c + 2 * i + 1] += bf16_hi(w[i]);
            }
        }
    }
}

// Joins the parts of a split tile, each (m, l, o) of its rows:
//   M = max m,  out = sum 2^(m - M) o / sum 2^(m - M) l
// Part x of the tile belongs to sum x mod kJoinSplit; each sum runs in the order of
// its parts, relative to its own maximum, and the sums are added in theirs.  Here and
// in k_chunk_join alike (a zero's sign is +), so the result depends neither on which
// block joins nor on which of the two does.  Up to kJoinSplit parts are sums of one
// part each, which are one sum in order.
constexpr int kJoinSplit = 4;

// Tiles of more parts, which long requests among many short ones have (80 of one
// token behind 300 and 16 behind 131072, one head: 84 us): as join_parts, one run of
// 16 columns at a time, three parts under way together.
__device__ __forceinline__ void join_many_parts(const ChunkArgs &a, const ChunkSegment &s, int row, int run, int step, bool mine)
{
    auto part = [&](int b) { return a.partials + static_cast<size_t>(chunk_slot(b, b == s.first)) * kChunkPart; };
    float top[kJoinSplit], M = -INFINITY;                        // the sums' maxima
#pragma unroll
    for (int q = 0; q < kJoinSplit; ++q) top[q] = -INFINITY;
#pragma unroll 1
    for (int b = s.first; b <= s.last; b += kJoinSplit)
#pragma unroll
        for (int q = 0; q < kJoinSplit; ++q)
            if (b + q <= s.last) top[q] = fmaxf(top[q], __ldcg(part(b + q) + kChunkRows * kHeadDim + row));
#pragma unroll
    for (int q = 0; q < kJoinSplit; ++q) M = fmaxf(M, top[q]);
#pragma unroll 1
    for (int c = run; c < 8; c += step) {
        float o[16] = {}, l = 0.f;
#pragma unroll 1
        for (int q = 0; q < kJoinSplit; ++q) {
            const float Mq = q == 0 ? top[0] : q == 1 ? top[1] : q == 2 ? top[2] : top[3];
            float oq[16] = {}, lq = 0.f;
#pragma unroll 3
            for (int b = s.first + q; b <= s.last; b += kJoinSplit) {
                const float *p = part(b);
                float4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = __ldcg(reinterpret_cast<const float4 *>(p) + (4 * c + k) * kChunkRows + row);
                const float m = __ldcg(p + kChunkRows * kHeadDim + row), f = m == -INFINITY ? 0.f : exp2f(m - Mq);
                lq = fmaf(f, __ldcg(p + kChunkRows * kHeadDim + kChunkRows + row), lq);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    oq[4 * k] = fmaf(f, x[k].x, oq[4 * k]);
                    oq[4 * k + 1] = fmaf(f, x[k].y, oq[4 * k + 1]);
                    oq[4 * k + 2] = fmaf(f, x[k].z, oq[4 * k + 2]);
                    oq[4 * k + 3] = fmaf(f, x[k].w, oq[4 * k + 3]);
                }
            }
            const float f = Mq == -INFINITY ? 0.f : exp2f(Mq - M);
            l = fmaf(f, lq, l);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(f, oq[k], o[k]);
        }
        const float g = l > 0.f ? 1.f / l : l;                   // NaN stays
        uint4 *out = reinterpret_cast<uint4 *>(a.out) +
                     ((static_cast<size_t>(s.row) + row / kGroup) * a.hkv * kGroup + s.j * kGroup + row % kGroup) * 16 + 2 * c;
        if (mine)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                out[k] = make_uint4(pack_bf16x2(fmaf(o[8 * k], g, 0.f), fmaf(o[8 * k + 1], g, 0.f)),
                                    pack_bf16x2(fmaf(o[8 * k + 2], g, 0.f), fmaf(o[8 * k + 3], g, 0.f)),
                                    pack_bf16x2(fmaf(o[8 * k + 4], g, 0.f), fmaf(o[8 * k + 5], g, 0.f)),
                                    pack_bf16x2(fmaf(o[8 * k + 6], g, 0.f), fmaf(o[8 * k + 7], g, 0.f)));
    }
}

// A warp holds runs of 16 columns of 32 rows, one row a lane, as the parts are laid
// out, two such runs at a time; the tile's rows and columns are shared by 8 warps.
__device__ __forceinline__ void join_parts(const ChunkArgs &a, const ChunkSegment &s)
{
    constexpr int kRuns = 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = s.rows * kGroup, most = rows > 128 ? 8 : rows > 64 ? 4 : rows > 32 ? 2 : 1;      // runs of 32 rows
    const int row = (warp & (most - 1)) * 32 + lane, step = 8 / most;
    if ((row & ~31) >= rows) return;
    if (s.last - s.first >= kJoinSplit) {
        join_many_parts(a, s, row, warp / most, step, row < rows);
        return;
    }
    auto part = [&](int b) { return a.partials + static_cast<size_t>(chunk_slot(b, b == s.first)) * kChunkPart; };
    float M = -INFINITY;
#pragma unroll 2
    for (int b = s.first; b <= s.last; ++b) M = fmaxf(M, __ldcg(part(b) + kChunkRows * kHeadDim + row));
    uint4 *out = reinterpret_cast<uint4 *>(a.out) +
                 ((static_cast<size_t>(s.row) + row / kGroup) * a.hkv * kGroup + s.j * kGroup + row % kGroup) * 16;
#pragma unroll 1
    for (int c0 = warp / most; c0 < 8; c0 += kRuns * step) {
        float o[kRuns][16] = {}, l = 0.f;
#pragma unroll 1
        for (int b = s.first; b <= s.last; ++b) {
            const float *p = part(b);
            float4 x[kRuns][4];
            const float m = __ldcg(p + kChunkRows * kHeadDim + row), lb = __ldcg(p + kChunkRows * kHeadDim + kChunkRows + row);
#pragma unroll
            for (int h = 0; h < kRuns; ++h)
                if (c0 + h * step < 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[h][k] = __ldcg(reinterpret_cast<const float4 *>(p) + (4 * (c0 + h * step) + k) * kChunkRows + row);
            const float f = m == -INFINITY ? 0.f : exp2f(m - M);
            l = fmaf(f, lb, l);
#pragma unroll
            for (int h = 0; h < kRuns; ++h)
                if (c0 + h * step < 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[h][4 * k] = fmaf(f, x[h][k].x, o[h][4 * k]);
                        o[h][4 * k + 1] = fmaf(f, x[h][k].y, o[h][4 * k + 1]);
                        o[h][4 * k + 2] = fmaf(f, x[h][k].z, o[h][4 * k + 2]);
                        o[h][4 * k + 3] = fmaf(f, x[h][k].w, o[h][4 * k + 3]);
                    }
        }
        const float g = l > 0.f ? 1.f / l : l;                   // NaN stays
        if (row < rows)
#pragma unroll
            for (int h = 0; h < kRuns; ++h)
                if (c0 + h * step < 8)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        out[2 * (c0 + h * step) + k] =
                            make_uint4(pack_bf16x2(fmaf(o[h][8 * k], g, 0.f), fmaf(o[h][8 * k + 1], g, 0.f)),
                                       pack_bf16x2(fmaf(o[h][8 * k + 2], g, 0.f), fmaf(o[h][8 * k + 3], g, 0.f)),
                                       pack_bf16x2(fmaf(o[h][8 * k + 4], g, 0.f), fmaf(o[h][8 * k + 5], g, 0.f)),
                                       pack_bf16x2(fmaf(o[h][8 * k + 6], g, 0.f), fmaf(o[h][8 * k + 7], g, 0.f)));
    }
}

// One softmax stream: 4 warps, thread = row = lane of the tensor memory.
__device__ __forceinline__ void chunk_softmax(const ChunkArgs &a, ChunkSmem &sm, int stream, const WaitGuard &wg)
{
    const int row = threadIdx.x & (kStreamRows - 1), lane = threadIdx.x & 31;
    const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
    const uint32_t ts = tmem_s(sm.tmem, stream) + lanes, to = tmem_o(sm.tmem, stream) + lanes;
    const float c = a.scale_log2;
    const uint64_t c2 = pack_f32x2(c, c);
    uint32_t s_par = 0u, o_par = 0u, half_par = 0u, join_par = 0u;
    int n_tiles = 0;                                             // key tiles of the block before this segment
    Segments in;
    ChunkSegment s;
    while (in.next(sm, s, wg)) {
        const int T = s.tiles(stream);
        const bool wide = s.wide();
        const int base_tile = n_tiles;
        n_tiles += s.t1 - s.t0;
        const int token = (wide ? stream * kStreamTokens : 0) + row / kGroup;      // of the tile
        const int vis = s.causal ? s.sees + token : s.sees;
        const bool live = (row & ~31) < (s.rows - (wide ? stream * kStreamTokens : 0)) * kGroup;   // the warp has a row
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < T; ++i) {
            const int nth = wide ? i : 2 * i + stream, t = s.t0 + nth;
            if (!mbar_wait_c(smem_u32(&sm.s_full[stream]), s_par, wg)) return;
            s_par ^= 1u;
            tcgen05_fence_after();
            if (live) {
                // the scores come in two halves; the first one's maximum is taken while the second is on its way
                uint32_t x[4][32];
                float mx[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
                const uint32_t pages = sm.pages[(base_tile + nth) % kNoteRing];
                const bool edge = t >= s.edge() || pages != 0xFFu;
                tmem_ld32(ts, x[0]);
                tmem_ld32(ts + 32, x[1]);
                tmem_wait_ld(x[0]);
                tmem_wait_ld(x[1]);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    if (p == 0) {
                        tmem_ld32(ts + 64, x[2]);
                        tmem_ld32(ts + 96, x[3]);
                    } else {
                        tmem_wait_ld(x[2]);
                        tmem_wait_ld(x[3]);
                    }
                    if (edge) {
#pragma unroll
                        for (int b = 2 * p; b < 2 * p + 2; ++b) {
                            const uint32_t bits = key_bits(pages >> (2 * b), vis, t * kTileKeys + b * 32);
                            if (__any_sync(0xffffffffu, bits != 0xFFFFFFFFu)) {
#pragma unroll
                                for (int k = 0; k < 32; ++k) x[b][k] = (bits >> k & 1u) ? x[b][k] : 0xFF800000u;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        mx[k & 7] = max3(mx[k & 7], __uint_as_float(x[2 * p][k]), __uint_as_float(x[2 * p + 1][k]));
                }
                const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * c;
                // has a row of the warp passed its reference?  Rarely
                const bool move = mt > m + kMaxSlack || (m == -INFINITY && mt > -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    const float mn = move ? mt : m;
                    const float al = m == -INFINITY ? (move ? 0.f : 1.f) : exp2f(m - mn);
                    l *= al;
                    m = mn;
                    if (i > 0) {
                        // the previous product is complete (S of this tile was issued after it)
#pragma unroll 1
                        for (int b = 0; b < 8; ++b) {
                            uint32_t o[16];
                            tmem_ld16(to + b * 16, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                            tmem_st16(to + b * 16, o);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.f : m;
                const uint64_t mu2 = pack_f32x2(-mu, -mu);
                uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t p[8];                           // 16 scores -> 8 registers of P
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint64_t e = fma_f32x2(pack_b32x2(x[b][16 * h + 2 * k], x[b][16 * h + 2 * k + 1]), c2, mu2);
                            const float p0 = ex2_approx(f32x2_lo(e)), p1 = ex2_approx(f32x2_hi(e));
                            ls[k & 1] = add_f32x2(ls[k & 1], pack_f32x2(p0, p1));
                            p[k] = pack_bf16x2(p0, p1);
                        }
                        tmem_st8(ts + b * 16 + 8 * h, p);
                    }
                    if (b == 1) {                                // the first half may go
                        tmem_wait_st();
                        tcgen05_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[stream][0]));
                    }
                }
                const uint64_t lsum = add_f32x2(ls[0], ls[1]);
                l += f32x2_lo(lsum) + f32x2_hi(lsum);
                tmem_wait_st();
            }
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!live) mbar_arrive(smem_u32(&sm.p_full[stream][0]));
                mbar_arrive(smem_u32(&sm.p_full[stream][1]));
            }
        }
        if (T > 0) {
            if (!mbar_wait_c(smem_u32(&sm.o_full[stream]), o_par, wg)) return;
            o_par ^= 1u;
            tcgen05_fence_after();
        }
        // a narrow tile's streams saw different keys: stream 0 takes in what stream 1 has
        float f0 = 1.f, f1 = 0.f;
        const bool two = !wide && s.t1 - s.t0 > 1;
        if (two && stream == 1) {
            sm.half_m[row] = m;
            sm.half_l[row] = l;
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.half_full));
            if (!mbar_wait_c(smem_u32(&sm.half_free), half_par, wg)) return;
            half_par ^= 1u;
            tcgen05_fence_after();
        } else if (two) {
            if (!mbar_wait_c(smem_u32(&sm.half_full), half_par, wg)) return;
            half_par ^= 1u;
            tcgen05_fence_after();
            const float m1 = sm.half_m[row], l1 = sm.half_l[row], mm = fmaxf(m, m1);
            f0 = m == -INFINITY ? 0.f : exp2f(m - mm);
            f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - mm);
            l = l * f0 + l1 * f1;
            m = mm;
        }
        // values that were zeroed on the way (noted before the products that are now complete were issued)
        bool spoilt = false;
#pragma unroll 1
        for (int t = max(s.edge(), s.t0); t < s.t1; ++t) spoilt |= sm.spoilt[(base_tile + t - s.t0) % kNoteRing] != 0u;
        const bool whole = s.whole();
        if (live && (wide || stream == 0)) {
            const bool mine = token < s.rows;
            const float g = whole ? (l > 0.f ? 1.f / l : l) : 1.f;      // NaN stays
            f0 *= g;
            f1 *= g;
            const int slot = chunk_slot(blockIdx.x, s.t0 == 0);
            float *part = a.partials + static_cast<size_t>(slot) * kChunkPart;
            const int part_row = (wide ? stream * kStreamRows : 0) + row;
            uint4 *out = reinterpret_cast<uint4 *>(a.out) +
                         ((static_cast<size_t>(s.row) + token) * a.hkv * kGroup + s.j * kGroup + (row & 2)) * 16 + (row & 1);
            // a short loop: code that runs once a tile comes slowly from the instruction cache
#pragma unroll 1
            for (int b = 0; b < 8; ++b) {
                uint32_t o[16];
                float v[16];
                tmem_ld16(to + b * 16, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]) * f0;
                if (two) {
                    tmem_ld16(to + 128 + b * 16, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = fmaf(__uint_as_float(o[k]), f1, v[k]);
                }
                if (spoilt && mine) add_spoilt(a, s, vis, b, v);
                if (whole) {
                    // two heads of a token trade 16-byte pieces, so that each store writes whole sectors
                    const bool odd = row & 1;
                    uint4 x = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                    uint4 y = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                                         pack_bf16x2(v[14], v[15]));
                    uint4 give = odd ? x : y;
                    give.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
                    give.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
                    give.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
                    give.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
                    if (mine) {
                        out[2 * b] = odd ? give : x;             // of the even head
                        out[2 * b + 16] = odd ? y : give;        // of the odd head
                    }
                } else if (mine) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<float4 *>(part)[(b * 4 + k) * kChunkRows + part_row] =
                            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
            if (!whole && mine) {
                part[kChunkRows * kHeadDim + part_row] = m;
                part[kChunkRows * kHeadDim + kChunkRows + part_row] = l;
            }
            if (!whole && !a.counters && stream == 0 && row == 0) a.records[slot] = make_int4(s.row, s.rows, s.j, s.t1 == s.keys ? 2 : 1);
        }
        tcgen05_fence_before();
        if (two && stream == 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.half_free));
        }
        if (!whole && a.counters) {
            // the softmax warps have written their part: has the tile got all of them?
            __threadfence();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.part_done));
            if (threadIdx.x < 32) {
                if (!mbar_wait_c(smem_u32(&sm.part_done), join_par, wg)) return;
                if (lane == 0) {
                    const uint32_t own = s.t1 - s.t0, before = atomic_add_acq_rel_gpu(a.counters + s.first, own);
                    sm.join_here = before + own == static_cast<uint32_t>(s.keys);
                    if (sm.join_here) a.counters[s.first] = 0u;
                    mbar_arrive(smem_u32(&sm.join_told));
                }
                __syncwarp();
            }
            if (!mbar_wait_c(smem_u32(&sm.join_told), join_par, wg)) return;
            join_par ^= 1u;
            if (sm.join_here) join_parts(a, s);
        }
    }
}

}  // namespace

__global__ void __launch_bounds__(kChunkThreads, 1)
    k_chunk(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
            const __grid_constant__ CUtensorMap map_v, const ChunkArgs a)
{
    extern __shared__ __align__(1024) uint8_t tiles[];           // the swizzled tiles start on 1024-byte boundaries
    ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>(tiles + (2 + kSlots) * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5;
    const WaitGuard wg{&sm.abort, a.status};
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), 2);
            mbar_init(smem_u32(&sm.landed[i]), 1);
        }
#pragma unroll 1
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(smem_u32(&sm.seg_full[i]), 1);
            mbar_init(smem_u32(&sm.seg_free[i]), kReaders);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), 1);
            mbar_init(smem_u32(&sm.q_free[i]), 1);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i][0]), kSoftmaxWarps);
            mbar_init(smem_u32(&sm.p_full[i][1]), kSoftmaxWarps);
            mbar_init(smem_u32(&sm.o_full[i]), 1);
            mbar_init(smem_u32(&sm.turn[i]), 1);
        }
        mbar_init(smem_u32(&sm.half_full), kSoftmaxWarps);
        mbar_init(smem_u32(&sm.half_free), kSoftmaxWarps);
        mbar_init(smem_u32(&sm.part_done), 2 * kSoftmaxWarps);
        mbar_init(smem_u32(&sm.join_told), 1);
        mbar_init(smem_u32(&sm.done), 2);
        mbar_fence_init();
        mbar_arrive(smem_u32(&sm.turn[0]));                      // stream 0 begins
    }
    if (warp == kIssuerWarp) tmem_alloc512(smem_u32(&sm.tmem));
    if (tid == kProducerWarp * 32) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    if (tid == kCheckerWarp * 32) tma_prefetch_desc(&map_q);
    pdl_wait();
    pdl_trigger();
    if (tid == 0) {
        guard_init(wg);
        a.records[chunk_slot(blockIdx.x, false)] = a.records[chunk_slot(blockIdx.x, true)] = make_int4(0, 0, 0, 0);
    }
    plan_share(a, sm);
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (sm.takes_part) {
        uint8_t *ring = tiles + 2 * kTileBytes;
        if (warp < kProducerWarp) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            chunk_softmax(a, sm, warp / kSoftmaxWarps, wg);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
            if (warp == kProducerWarp) {
                ProducerState p;
                chunk_produce(a, &map_k, &map_v, ring, sm, p, wg);
                // after a give-up the copies still in flight land before the block ends
                if ((tid & 31) == 0 && guard_failed(wg)) {
                    const uint64_t deadline = globaltimer() + kDrainLimitNs;
                    for (int i = 0; i < kSlots; ++i) {
                        if (p.keys >> i & 1u) mbar_drain(smem_u32(&sm.full[i]), p.keys_round >> i & 1u, deadline);
                        if (p.values >> i & 1u) mbar_drain(smem_u32(&sm.landed[i]), (p.values_round >> i & 1u) ^ 1u, deadline);
                    }
                }
            } else if (warp == kCheckerWarp) {
                QueryState queries;
                chunk_check(&map_q, tiles, ring, sm, queries, wg);
                if ((tid & 31) == 0 && guard_failed(wg)) {
                    const uint64_t deadline = globaltimer() + kDrainLimitNs;
                    for (int i = 0; i < 2; ++i)
                        if (queries.had >> i & 1u) mbar_drain(smem_u32(&sm.q_full[i]), queries.phase >> i & 1u, deadline);
                }
            } else {
                chunk_issue(smem_u32(tiles), smem_u32(ring), sm, warp - kIssuerWarp, wg);
                // nothing may be in flight when the tensor memory is freed
                if (elect_one()) umma_commit(smem_u32(&sm.done));
                __syncwarp();
                if (!mbar_wait_c(smem_u32(&sm.done), 0u, wg))
                    mbar_drain(smem_u32(&sm.done), 0u, globaltimer() + kDrainLimitNs);
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (warp == kIssuerWarp) tmem_free512(sm.tmem);
}

// ---------------------------------------------------------------- join
// Where there are few tiles a tile may have a part of every block (64 rows behind
// 128k tokens, one head: 152): four warps share the parts of 16 columns of 32
// rows, 16 blocks the tile.  grid (tiles at most, 16); the x-th split tile is
// found in the records that k_chunk left.
constexpr int kMostParts = 8;                       // that the last block joins where tiles are few
constexpr int kJoinWarps = 16, kJoinBlocks = 64 * kJoinSplit / kJoinWarps;

__global__ void __launch_bounds__(kJoinWarps * 32) k_chunk_join(const ChunkArgs a, int blocks)
{
    __shared__ float red[kJoinWarps / kJoinSplit][kJoinSplit][18][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    // the tile's first block, and the one that ends it
    int first = -1, last = -1, nth = blockIdx.x;
    for (int b = 0; b < blocks && first < 0; b += 32) {
        unsigned begins = __ballot_sync(0xffffffffu, b + lane < blocks && __ldcg(a.records + chunk_slot(min(b + lane, blocks - 1), true)).w != 0);
        const int n = __popc(begins);
        if (nth < n) {
            for (; nth > 0; --nth) begins &= begins - 1u;
            first = b + __ffs(begins) - 1;
        } else {
            nth -= n;
        }
    }
    if (first < 0) return;
    const int4 rec = __ldcg(a.records + chunk_slot(first, true));
    for (int b = first + 1; b < blocks && last < 0; b += 32) {
        const unsigned ends = __ballot_sync(0xffffffffu, b + lane < blocks && __ldcg(a.records + chunk_slot(min(b + lane, blocks - 1), false)).w == 2);
        if (ends) last = b + __ffs(ends) - 1;
    }
    if (last < 0) return;
    const int share = warp % kJoinSplit, unit = (blockIdx.y * kJoinWarps + warp) / kJoinSplit;
    const int c = unit >> 3, row = (unit & 7) * 32 + lane;
    // a narrow tile has 128 rows, in the same places
    auto part = [&](int b) { return a.partials + static_cast<size_t>(chunk_slot(b, b == first)) * kChunkPart; };
    float M = -INFINITY, l = 0.f, o[16] = {};
    if ((unit & 7) * 32 < rec.y * kGroup) {
#pragma unroll 4
        for (int b = first + share; b <= last; b += kJoinSplit) M = fmaxf(M, __ldcg(part(b) + kChunkRows * kHeadDim + row));
#pragma unroll 4
        for (int b = first + share; b <= last; b += kJoinSplit) {
            const float *p = part(b);
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __ldcg(reinterpret_cast<const float4 *>(p) + (4 * c + k) * kChunkRows + row);
            const float m = __ldcg(p + kChunkRows * kHeadDim + row), f = m == -INFINITY ? 0.f : exp2f(m - M);
            l = fmaf(f, __ldcg(p + kChunkRows * kHeadDim + kChunkRows + row), l);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[4 * k] = fmaf(f, x[k].x, o[4 * k]);
                o[4 * k + 1] = fmaf(f, x[k].y, o[4 * k + 1]);
                o[4 * k + 2] = fmaf(f, x[k].z, o[4 * k + 2]);
                o[4 * k + 3] = fmaf(f, x[k].w, o[4 * k + 3]);
            }
        }
    }
    float(&mine)[18][32] = red[warp / kJoinSplit][share];
    mine[16][lane] = M;
    mine[17][lane] = l;
#pragma unroll
    for (int k = 0; k < 16; ++k) mine[k][lane] = o[k];
    __syncthreads();
    if (share != 0 || row >= rec.y * kGroup) return;
    const float own = M;
    for (int q = 1; q < kJoinSplit; ++q) M = fmaxf(M, red[warp / kJoinSplit][q][16][lane]);
    float f = own == -INFINITY ? 0.f : exp2f(own - M);
    l *= f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= f;
    for (int q = 1; q < kJoinSplit; ++q) {
        const float(&x)[18][32] = red[warp / kJoinSplit][q];
        f = x[16][lane] == -INFINITY ? 0.f : exp2f(x[16][lane] - M);
        l = fmaf(f, x[17][lane], l);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = fmaf(f, x[k][lane], o[k]);
    }
    const float g = l > 0.f ? 1.f / l : l;
    uint4 *out = reinterpret_cast<uint4 *>(a.out) +
                 ((static_cast<size_t>(rec.x) + row / kGroup) * a.hkv * kGroup + rec.z * kGroup + row % kGroup) * 16 + 2 * c;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        out[k] = make_uint4(pack_bf16x2(fmaf(o[8 * k], g, 0.f), fmaf(o[8 * k + 1], g, 0.f)),
                            pack_bf16x2(fmaf(o[8 * k + 2], g, 0.f), fmaf(o[8 * k + 3], g, 0.f)),
                            pack_bf16x2(fmaf(o[8 * k + 4], g, 0.f), fmaf(o[8 * k + 5], g, 0.f)),
                            pack_bf16x2(fmaf(o[8 * k + 6], g, 0.f), fmaf(o[8 * k + 7], g, 0.f)));
}

namespace {
std::atomic<int> g_chunk_smem_seen[64];
}

cudaError_t launch_chunk(const CUtensorMap &map_q, const CUtensorMap &map_k, const CUtensorMap &map_v, ChunkArgs a, int blocks,
                         cudaStream_t stream)
{
    cudaError_t e = raise_smem_limit(k_chunk, kChunkSmemBytes, g_chunk_smem_seen);
    if (e != cudaSuccess) return e;
    // By what the host knows, the sizes and not the lengths: tiles there may be, and
    // parts of one.  With a tile for every other block it has two or three parts on
    // average (a long request among many short ones has more), and a table of less than
    // 232 pages has no more than a few.  Behind a wider table a call of few tiles pays
    // the second launch whatever its lengths: 7 tokens behind 519 15.2 us, 12.1 with
    // their own 33 pages (both in a captured graph).
    const long long tiles = a.hkv * (static_cast<long long>(a.tokens) / kChunkTokens + a.batch);
    constexpr ChunkCost c = chunk_cost(kChunkTokens);
    const int parts = 1 + (c.start + c.key * (a.max_pages * kPageSize / kTileKeys + 1)) / kMinShare;
    const bool few = 2 * tiles < blocks && parts > kMostParts;
    if (few) a.counters = nullptr;
    e = launch_pdl(k_chunk, dim3(blocks), dim3(kChunkThreads), kChunkSmemBytes, stream, map_q, map_k, map_v, a);
    if (e != cudaSuccess || !few) return e;
    return launch_pdl(k_chunk_join, dim3(static_cast<unsigned>(tiles), kJoinBlocks), dim3(kJoinWarps * 32), 0, stream, a, blocks);
}

}  // namespace moira
