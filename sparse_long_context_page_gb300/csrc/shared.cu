// Attention of a batch whose requests share a long prefix, and the
// accumulation of attention weights over each request's own tokens.
//
// Every group of consecutive requests [start_g, start_{g+1}) shares the first
// len_g tokens of one page list.  For a query row (request r, head h) the
// softmax runs over the prefix and the request's own tokens together; both
// parts are computed apart and joined by their log-sum-exp:
//   own:    k_attend over the request's lists (attend.cu, recording variant)
//   prefix: k_prefix, all query rows of a (group, KV head) against each key
//           tile, so the prefix is read once for the group and not once per
//           request; the keys are split over the grid and every split leaves
//           a partial (max, sum, unnormalised output)
//   joint:  k_shared_merge joins a row's prefix partials and its own part
// The weights of the own tokens need the joint log-sum-exp, so they are added
// last (k_weights) from the logits that the own part left in the workspace.
#include "moira_device.cuh"
#include "moira_launch.h"

namespace moira {

constexpr int kTileKeys = 128;                      // keys of one prefix work item
constexpr int kTilePages = kTileKeys / kPageSize;

// The groups' work, laid end to end: group g has hkv * rtiles(g) units of
// tiles(g) key tiles each, unit = head * rtiles + row tile.
struct GroupPlan {
    int woff[kMaxGroups + 1];                       // key tiles before the group
    uint16_t start[kMaxGroups + 1];                 // first request (sanitised: ascending, within the batch)
};
static_assert(kMaxUnits < 65536, "request indices fit 16 bits");

__device__ __forceinline__ int rtiles_of(int requests) { return (requests * kGroup + kUnitRows - 1) / kUnitRows; }
__device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }
__device__ __forceinline__ int prefix_len(const PrefixArgs &a, int g)
{
    return min(max(a.prefix_lens[g], 0), a.prefix_pages * kPageSize);
}

// One warp of the block fills the plan.
__device__ __forceinline__ void plan_groups(const PrefixArgs &a, GroupPlan &p)
{
    const int lane = threadIdx.x & 31;
    int before = 0, w = 0;                          // carried over the chunks of 32 groups
    bool bad = false;
    for (int base = 0; base < a.groups; base += 32) {
        const int g = base + lane;
        const bool in = g < a.groups;
        int raw = 0, next = 0, len = 0;
        if (in) {
            raw = a.group_starts[g];
            next = a.group_starts[g + 1];
            len = a.prefix_lens[g];
        }
        const int cap = a.prefix_pages * kPageSize;
        bad |= in && (raw < 0 || next < raw || next > a.batch || len < 0 || len > cap);
        len = min(max(len, 0), cap);
        // running maxima make the starts ascending whatever was given
        int s = max(min(max(raw, 0), a.batch), before);
        const int e = min(max(next, 0), a.batch);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s = max(s, y);
        }
        int sn = __shfl_down_sync(0xffffffffu, s, 1);           // the next group's start
        if (g == a.groups - 1 || lane == 31) sn = max(e, s);
        const int req = in ? max(sn - s, 0) : 0;
        const int work = a.hkv * rtiles_of(req) * tiles_of(len);
        int wi = work;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o) wi += y;
        }
        if (in) {
            p.start[g] = static_cast<uint16_t>(s);
            p.woff[g] = w + wi - work;
            if (g == a.groups - 1) {
                p.start[a.groups] = static_cast<uint16_t>(s + req);
                p.woff[a.groups] = w + wi;
            }
        }
        before = __shfl_sync(0xffffffffu, s + req, 31);
        w += __shfl_sync(0xffffffffu, wi, 31);
    }
    if (bad) raise_status(a.status, kDevBadLen);
}

// Block b's share of W work items on n blocks is [b*W/n, (b+1)*W/n).
__device__ __forceinline__ int share_lo(int b, int W, int n) { return static_cast<int>(static_cast<long long>(b) * W / n); }
// The block whose share holds item k.
__device__ __forceinline__ int share_of(int k, int W, int n)
{
    return static_cast<int>(((static_cast<long long>(k) + 1) * n - 1) / W);
}

// A block's part of one unit: key tiles [t0, t1) of group g for the rows
// [row0, row0 + rows) of KV head j (row = request of the group * 4 + head).
struct Segment {
    int g, j, unit, row0, rows, t0, t1;
    // more than 128 rows: each stream has its own rows and takes every tile;
    // else both have the same rows and take alternate tiles
    __device__ __forceinline__ bool wide() const { return rows > kStreamRows; }
    __device__ __forceinline__ int tiles(int stream) const { return wide() ? t1 - t0 : (t1 - t0 + 1 - stream) >> 1; }
};

// Walks the segments of the block's share; every role of the block walks its own.
struct SegmentWalk {
    const GroupPlan &p;
    int hkv, w, w1, g, u;                           // u: units before group g
    __device__ __forceinline__ bool next(Segment &s)
    {
        if (w >= w1) return false;
        int req = p.start[g + 1] - p.start[g];
        while (p.woff[g + 1] <= w) {
            u += hkv * rtiles_of(req);
            ++g;
            req = p.start[g + 1] - p.start[g];
        }
        const int rt = rtiles_of(req);
        const int tiles = (p.woff[g + 1] - p.woff[g]) / (hkv * rt);
        const int ug = (w - p.woff[g]) / tiles;
        s.g = g;
        s.t0 = w - p.woff[g] - ug * tiles;
        s.t1 = min(tiles, s.t0 + w1 - w);
        s.j = ug / rt;
        s.unit = u + ug;
        s.row0 = (ug % rt) * kUnitRows;
        s.rows = min(kUnitRows, req * kGroup - s.row0);
        w += s.t1 - s.t0;
        return true;
    }
};

// ---------------------------------------------------------------- prefix attention
// k_prefix: one block per SM, its warps in four roles around two streams of
// 128 query rows (the 128 lanes of the tensor memory):
//   producer  (1 warp)  TMA page loads into a ring of 32 KB tiles (keys or values of 128 tokens)
//   issuer    (1 warp)  one thread issues the tcgen05 products
//   softmax   (2 x 4 warps, one thread per row) S -> P in tensor memory
// Per key tile and stream
//   S = Q K^T   128 x 128 x 128, Q and K in shared memory (128-byte swizzle, K-major)
//   P           2^(S - m), bf16 and bf16 residual, overwrites S in tensor memory
//               (32 columns of scores become 16 of each)
//   O += P V    A = P from tensor memory, B = V from shared memory (MN-major), both halves of P
// While one stream is in its softmax the tensor cores work for the other.
// With more than 128 rows the streams hold different rows and share each K/V
// tile; else they hold the same rows and take alternate tiles.
// The row reference m moves only when a tile's maximum passes it by 2^8
// (P then stays below 2^8 and nothing is lost in its significand), so O in
// tensor memory is rarely rescaled.
constexpr int kRingSlots = 5;
constexpr int kTileBytes = kTileKeys * kHeadDim * 2;              // 32 KB
constexpr int kHalfTile = kTileKeys * 128;                       // 128 rows x 128 B
constexpr int kPrefixThreads = 320;
constexpr int kProducerWarp = 8, kIssuerWarp = 9;
constexpr int kMaskRing = 16;                                    // tiles whose key masks are kept
constexpr float kMaxSlack = 8.f;                                 // log2 units a row's maximum may pass its reference by
// The tensor cores add into fp32 accumulators by truncation, so a long chain of
// adds drifts towards zero (about 1.7e-8 of the value per 16-key step); after
// this many tiles a stream adds its accumulator to its partial in fp32.
constexpr int kChainTiles = 8;

struct PrefixSmem {
    unsigned long long full[kRingSlots], empty[kRingSlots];
    unsigned long long q_full[2], s_full[2], p_full[2], o_full[2], done;
    uint32_t tmem;
    int abort;
    uint4 mask[kMaskRing];                                       // keys of a tile that count
    GroupPlan plan;
};
constexpr int kPrefixSmemBytes = 1024 + (2 + kRingSlots) * kTileBytes + static_cast<int>(sizeof(PrefixSmem));
static_assert(kPrefixSmemBytes <= 227 * 1024, "one block's shared memory");

// Columns of the tensor memory: S / P of the two streams, then O of the two.
__device__ __forceinline__ uint32_t tmem_s(uint32_t base, int stream) { return base + stream * 128; }
__device__ __forceinline__ uint32_t tmem_o(uint32_t base, int stream) { return base + 256 + stream * 128; }

// Position in a ring of kRingSlots: slot and the parity of its current round.
struct RingPos {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void advance()
    {
        if (++slot == kRingSlots) {
            slot = 0;
            round ^= 1u;
        }
    }
};

__device__ void prefix_produce(const PrefixArgs &a, const CUtensorMap *mk, const CUtensorMap *mv, uint8_t *ring,
                               PrefixSmem &sm, SegmentWalk walk, const WaitGuard &wg)
{
    const int lane = threadIdx.x & 31, page = lane & 7, half = (lane >> 3) & 1;
    RingPos pos;
    int n_tiles = 0;                                             // K tiles so far
    Segment s;
    while (walk.next(s)) {
        const int len = prefix_len(a, s.g);
        const int32_t *table = a.prefix_table + static_cast<size_t>(s.g) * a.prefix_pages;
        // one tile's keys or values into the next ring slot; lane (half, page) copies one box
        auto load = [&](int tile, bool keys) {
            const int p = tile * kTilePages + page, tok = len - p * kPageSize;     // tokens from this page on
            const int pid = tok > 0 ? table[p] : -1;
            const bool ok = tok > 0 && pid >= 0 && pid < a.num_pages;
            mbar_wait_g(smem_u32(&sm.empty[pos.slot]), pos.round ^ 1u, wg);
            uint8_t *dst = ring + pos.slot * kTileBytes;
            const uint32_t full = smem_u32(&sm.full[pos.slot]);
            // values of tokens that do not count must be finite (their P is 0): a
            // partly filled page is copied by hand, a missing one is zeroed
            const bool whole = ok && (keys || tok >= kPageSize);
            if (keys) {
                if (tok > 0 && !ok && lane < 8) raise_status(a.status, kDevBadPage);
                uint32_t bits = ok ? (tok >= kPageSize ? 0xFFFFu : (1u << tok) - 1u) : 0u;
                bits |= __shfl_down_sync(0xffffffffu, bits, 1) << 16;
                if (lane < 8 && (lane & 1) == 0)
                    reinterpret_cast<uint32_t *>(&sm.mask[n_tiles % kMaskRing])[lane >> 1] = bits;
            } else {
                unsigned by_hand = __ballot_sync(0xffffffffu, lane < 8 && !whole);
                while (by_hand) {
                    const int pg = __ffs(by_hand) - 1;
                    by_hand &= by_hand - 1;
                    const int id = __shfl_sync(0xffffffffu, ok ? pid : -1, pg);
                    const int cnt = __shfl_sync(0xffffffffu, tok, pg);
                    for (int e = lane; e < kPageSize * 16; e += 32) {
                        const int t = e >> 4, c = e & 15, row = pg * kPageSize + t;
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (id >= 0 && t < cnt)
                            x = reinterpret_cast<const uint4 *>(a.v_pool)[((static_cast<size_t>(id) * a.hkv + s.j) *
                                                                              kPageSize + t) * 16 + c];
                        *reinterpret_cast<uint4 *>(dst + (c >> 3) * kHalfTile + row * 128 +
                                                   (((c & 7) ^ (row & 7)) << 4)) = x;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            const unsigned copies = __ballot_sync(0xffffffffu, lane < 16 && whole);
            if (lane == 0) {
                if (copies) mbar_arrive_expect_tx(full, __popc(copies) * kHalfBytes);
                else mbar_arrive(full);
            }
            __syncwarp();
            if (lane < 16 && whole)
                tma_load_2d(smem_u32(dst) + half * kHalfTile + page * kHalfBytes, keys ? mk : mv, half * 64,
                            (pid * a.hkv + s.j) * kPageSize, full);
            __syncwarp();
            if (keys) ++n_tiles;
            pos.advance();
        };
        // the order in which the issuer first uses the tiles
        const int ahead = s.wide() ? 1 : 2;
        for (int t = s.t0; t < min(s.t1, s.t0 + ahead); ++t) load(t, true);
        for (int t = s.t0; t < s.t1; ++t) {
            load(t, false);
            if (t + ahead < s.t1) load(t + ahead, true);
        }
    }
    // after a give-up, let the copies still in flight land before the block ends
    if (lane == 0 && guard_failed(wg)) {
        const uint64_t deadline = globaltimer() + kDrainLimitNs;
        for (int i = 0; i < kRingSlots; ++i) {
            // the slot's last round, if it had one
            const bool wrapped = i < pos.slot;
            mbar_drain(smem_u32(&sm.full[i]), wrapped ? pos.round : pos.round ^ 1u, deadline);
        }
    }
}

// The issuing thread: S and O products of both streams in the ring's order.
__device__ void prefix_issue(uint32_t q_base, uint32_t ring, PrefixSmem &sm, SegmentWalk walk, const WaitGuard &wg)
{
    constexpr uint32_t kIdescS = umma_idesc_bf16(128, kTileKeys, false);
    constexpr uint32_t kIdescO = umma_idesc_bf16(128, kHeadDim, true);
    const uint32_t tmem = sm.tmem;
    RingPos pos;
    uint32_t q_par = 0u, p_par = 0u;                              // bit s: stream s
    Segment s;
    auto bump = [](uint32_t &par, int st) { par ^= 1u << st; };
    while (walk.next(s)) {
        const int T = s.t1 - s.t0;
        const bool wide = s.wide();
        for (int st = 0; st < 2; ++st)
            if (s.tiles(st) > 0) {
                mbar_wait_g(smem_u32(&sm.q_full[st]), (q_par >> st) & 1u, wg);
                bump(q_par, st);
            }
        tcgen05_fence_after();
        auto qk = [&](int st, uint32_t kt) {
#pragma unroll
            for (int ks = 0; ks < kHeadDim / 16; ++ks) {
                const uint32_t off = (ks >> 2) * kHalfTile + (ks & 3) * 32;
                umma_ss(tmem_s(tmem, st), umma_desc(q_base + st * kTileBytes + off, 16, 1024),
                        umma_desc(kt + off, 16, 1024), kIdescS, ks > 0);
            }
            umma_commit(smem_u32(&sm.s_full[st]));
        };
        auto pv = [&](int st, uint32_t vt, int nth) {
            mbar_wait_g(smem_u32(&sm.p_full[st]), (p_par >> st) & 1u, wg);
            bump(p_par, st);
            tcgen05_fence_after();
            bool acc = nth % kChainTiles != 0;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < kTileKeys / 16; ++ks) {
                    umma_ts(tmem_o(tmem, st), tmem_s(tmem, st) + (ks >> 1) * 32 + part * 16 + (ks & 1) * 8,
                            umma_desc(vt + ks * 2048, kHalfTile, 1024), kIdescO, acc);
                    acc = true;
                }
            if (nth + 1 == s.tiles(st)) umma_commit(smem_u32(&sm.o_full[st]));
        };
        auto wait_tile = [&](const RingPos &r) {
            mbar_wait_g(smem_u32(&sm.full[r.slot]), r.round, wg);
            tcgen05_fence_after();
            return ring + r.slot * kTileBytes;
        };
        if (wide) {
            uint32_t kt = wait_tile(pos);
            qk(0, kt);
            qk(1, kt);
            umma_commit(smem_u32(&sm.empty[pos.slot]));
            pos.advance();
            for (int i = 0; i < T; ++i) {
                const RingPos vp = pos;
                RingPos kp = pos;
                kp.advance();
                const uint32_t vt = wait_tile(vp);
                pv(0, vt, i);
                if (i + 1 < T) {
                    kt = wait_tile(kp);
                    qk(0, kt);
                }
                pv(1, vt, i);
                umma_commit(smem_u32(&sm.empty[vp.slot]));
                pos.advance();
                if (i + 1 < T) {
                    qk(1, kt);
                    umma_commit(smem_u32(&sm.empty[kp.slot]));
                    pos.advance();
                }
            }
        } else {
            for (int i = 0; i < min(T, 2); ++i) {
                qk(i, wait_tile(pos));
                umma_commit(smem_u32(&sm.empty[pos.slot]));
                pos.advance();
            }
            for (int i = 0; i < T; ++i) {
                const uint32_t vt = wait_tile(pos);
                pv(i & 1, vt, i >> 1);
                umma_commit(smem_u32(&sm.empty[pos.slot]));
                pos.advance();
                if (i + 2 < T) {
                    qk(i & 1, wait_tile(pos));
                    umma_commit(smem_u32(&sm.empty[pos.slot]));
                    pos.advance();
                }
            }
        }
    }
    umma_commit(smem_u32(&sm.done));
}

// One softmax stream: 4 warps, thread = row.
__device__ void prefix_softmax(const PrefixArgs &a, uint8_t *q_smem, PrefixSmem &sm, SegmentWalk walk, int stream,
                               const WaitGuard &wg)
{
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
    const uint32_t ts = tmem_s(sm.tmem, stream) + lanes, to = tmem_o(sm.tmem, stream) + lanes;
    const float c = a.scale_log2;
    uint32_t s_par = 0u, o_par = 0u;
    int n_tiles = 0;                                             // K tiles of the block before this segment
    Segment s;
    while (walk.next(s)) {
        const int T = s.tiles(stream);
        const bool wide = s.wide();
        const int base_tile = n_tiles;
        n_tiles += s.t1 - s.t0;
        if (T == 0) continue;
        const int first = s.row0 + (wide ? stream * kStreamRows : 0);
        const int rows = min(kStreamRows, s.rows - (wide ? stream * kStreamRows : 0));
        // the stream's query rows (the last segment's products are complete: o_full)
        const uint16_t *q = static_cast<const uint16_t *>(a.q) +
                            (static_cast<size_t>(walk.p.start[s.g]) * a.hq + s.j * kGroup) * kHeadDim;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int e = row + i * kStreamRows, r = e >> 4, ch = e & 15, rr = first + r;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows)
                x = *reinterpret_cast<const uint4 *>(q + (static_cast<size_t>(rr / kGroup) * a.hq + rr % kGroup) *
                                                             kHeadDim + ch * 8);
            *reinterpret_cast<uint4 *>(q_smem + (ch >> 3) * kHalfTile + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(smem_u32(&sm.q_full[stream]));

        float *part = a.partials + (static_cast<size_t>(blockIdx.x + s.unit) * 2 + stream) * kPrefixPart;
        const bool live = (row & ~31) < rows;                    // this warp has a row that counts
        float m = -INFINITY, l = 0.f, m_part = -INFINITY;
        // adds O to the partial in global memory (the first time: writes it)
        auto flush = [&](bool fresh) {
            const float f = m_part == -INFINITY ? 0.f : exp2f(m_part - m);
            float4 *pp = reinterpret_cast<float4 *>(part) + row;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t o[32];
                tmem_ld32(to + b * 32, o);
                float4 old[8];
                if (!fresh && row < rows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) old[i] = pp[(b * 8 + i) * kStreamRows];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                tmem_wait_ld(o);
                if (row < rows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        pp[(b * 8 + i) * kStreamRows] =
                            make_float4(fmaf(old[i].x, f, __uint_as_float(o[4 * i])),
                                        fmaf(old[i].y, f, __uint_as_float(o[4 * i + 1])),
                                        fmaf(old[i].z, f, __uint_as_float(o[4 * i + 2])),
                                        fmaf(old[i].w, f, __uint_as_float(o[4 * i + 3])));
                }
            }
            m_part = m;
        };
        for (int i = 0; i < T; ++i) {
            const bool chain_start = i % kChainTiles == 0;
            mbar_wait_g(smem_u32(&sm.s_full[stream]), s_par, wg);
            s_par ^= 1u;
            tcgen05_fence_after();
            if (live) {
                if (chain_start && i > 0) flush(i == kChainTiles);
                const uint4 mask = sm.mask[(base_tile + (wide ? i : 2 * i + stream)) % kMaskRing];
                const bool part_tile = (mask.x & mask.y & mask.z & mask.w) != 0xFFFFFFFFu;
                // the row's scores are read twice, 32 columns at a time: for the
                // maximum, then for P (held at once they would not fit the registers)
                auto scores = [&](int b, uint32_t (&x)[32]) {
                    if (part_tile) {
                        const uint32_t mw = b == 0 ? mask.x : b == 1 ? mask.y : b == 2 ? mask.z : mask.w;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(mw >> k & 1u)) x[k] = 0xFF800000u;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int b = 0; b < 4; b += 2) {
                    uint32_t x[32], y[32];
                    tmem_ld32(ts + b * 32, x);
                    tmem_ld32(ts + b * 32 + 32, y);
                    tmem_wait_ld(x);
                    tmem_wait_ld(y);
                    scores(b, x);
                    scores(b + 1, y);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        mx[k & 3] = fmaxf(mx[k & 3], fmaxf(__uint_as_float(x[k]), __uint_as_float(y[k])));
                }
                const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool move = mt > m + kMaxSlack || (m == -INFINITY && mt > -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    const float mn = move ? mt : m;
                    const float al = m == -INFINITY ? (move ? 0.f : 1.f) : exp2f(m - mn);
                    l *= al;
                    m = mn;
                    if (!chain_start) {
                        // the previous product is complete (S of this tile was issued after it)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            uint32_t o[32];
                            tmem_ld32(to + b * 32, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                            tmem_st32(to + b * 32, o);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.f : m;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t x[32], hi[16], lo[16];
                    tmem_ld32(ts + b * 32, x);
                    tmem_wait_ld(x);
                    scores(b, x);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float p0 = ex2_approx(fmaf(__uint_as_float(x[2 * k]), c, -mu));
                        const float p1 = ex2_approx(fmaf(__uint_as_float(x[2 * k + 1]), c, -mu));
                        l0 += p0;
                        l1 += p1;
                        hi[k] = pack_bf16x2(p0, p1);
                        lo[k] = pack_bf16x2(p0 - bf16_lo(hi[k]), p1 - bf16_hi(hi[k]));
                    }
                    tmem_st16(ts + b * 32, hi);
                    tmem_st16(ts + b * 32 + 16, lo);
                }
                l += l0 + l1;
                tmem_wait_st();
            }
            tcgen05_fence_before();
            mbar_arrive(smem_u32(&sm.p_full[stream]));
        }
        mbar_wait_g(smem_u32(&sm.o_full[stream]), o_par, wg);
        o_par ^= 1u;
        tcgen05_fence_after();
        if (live) {
            flush(T <= kChainTiles);
            if (row < rows) {
                part[kStreamRows * kHeadDim + row] = m;
                part[kStreamRows * kHeadDim + kStreamRows + row] = l;
            }
        }
        tcgen05_fence_before();
    }
}

__global__ void __launch_bounds__(kPrefixThreads, 1)
    k_prefix(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
             const PrefixArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    PrefixSmem &sm = *reinterpret_cast<PrefixSmem *>(tiles + (2 + kRingSlots) * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5;
    const WaitGuard wg{&sm.abort, a.status};
    if (tid == 0) {
        for (int i = 0; i < kRingSlots; ++i) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), kStreamRows);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i]), kStreamRows);
            mbar_init(smem_u32(&sm.o_full[i]), 1);
        }
        mbar_init(smem_u32(&sm.done), 1);
        mbar_fence_init();
        guard_init(wg);
    }
    if (warp == kIssuerWarp) tmem_alloc512(smem_u32(&sm.tmem));
    if (warp == kProducerWarp) {
        if ((tid & 31) == 0) {
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
        }
    }
    pdl_wait();
    if (warp == kProducerWarp) plan_groups(a, sm.plan);
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();

    const int W = sm.plan.woff[a.groups], n = min(static_cast<int>(gridDim.x), W), b = blockIdx.x;
    if (b < n) {
        SegmentWalk walk{sm.plan, a.hkv, share_lo(b, W, n), share_lo(b + 1, W, n), 0, 0};
        uint8_t *ring = tiles + 2 * kTileBytes;
        if (warp == kProducerWarp) {
            prefix_produce(a, &tmap_k, &tmap_v, ring, sm, walk, wg);
        } else if (warp == kIssuerWarp) {
            if ((tid & 31) == 0) {
                prefix_issue(smem_u32(tiles), smem_u32(ring), sm, walk, wg);
                // nothing may be in flight when the tensor memory is freed
                if (!mbar_try_wait(smem_u32(&sm.done), 0u))
                    mbar_drain(smem_u32(&sm.done), 0u, globaltimer() + kDrainLimitNs);
            }
            __syncwarp();
        } else {
            prefix_softmax(a, tiles + (warp >> 2) * kTileBytes, sm, walk, warp >> 2, wg);
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (warp == kIssuerWarp) tmem_free512(sm.tmem);
}

int prefix_blocks(int sms) { return sms; }

namespace {
std::atomic<int> g_prefix_smem_seen[64];
}

cudaError_t launch_prefix(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const PrefixArgs &a,
                          cudaStream_t stream)
{
    const cudaError_t e = raise_smem_limit(k_prefix, kPrefixSmemBytes, g_prefix_smem_seen);
    if (e != cudaSuccess) return e;
    k_prefix<<<a.blocks, kPrefixThreads, kPrefixSmemBytes, stream>>>(tmap_k, tmap_v, a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- joint softmax
// One block per (request, KV head): thread (head, 4 dims).
__global__ void __launch_bounds__(128) k_shared_merge(const PrefixArgs a)
{
    __shared__ GroupPlan p;
    pdl_wait();
    if (threadIdx.x < 32) plan_groups(a, p);
    __syncthreads();
    const int r = blockIdx.x / a.hkv, j = blockIdx.x % a.hkv;
    int g = 0, u = 0;                                            // u: units before group g
    while (g < a.groups && r >= p.start[g + 1]) {
        u += a.hkv * rtiles_of(p.start[g + 1] - p.start[g]);
        ++g;
    }
    if (g < a.groups && r < p.start[g]) return;                  // a request before the first group
    if (g == a.groups || p.woff[g + 1] == p.woff[g]) return;     // no prefix: the own part is the result
    const int W = p.woff[a.groups], n = min(a.blocks, W);
    const int h = threadIdx.x >> 5, d4 = threadIdx.x & 31;
    const int req = p.start[g + 1] - p.start[g], rt = rtiles_of(req);
    const int tiles = (p.woff[g + 1] - p.woff[g]) / (a.hkv * rt);
    const int row = (r - p.start[g]) * kGroup + h;
    const int ug = j * rt + row / kUnitRows, in = row % kUnitRows;
    const int w0 = p.woff[g] + ug * tiles;
    const int b0 = share_of(w0, W, n), b1 = share_of(w0 + tiles - 1, W, n);
    const float *part = a.partials + static_cast<size_t>(u + ug) * 2 * kPrefixPart;
    // a unit of more than 128 rows: the row's own stream; else both streams
    // (the second has none where the block took a single tile)
    const int rows = min(kUnitRows, req * kGroup - row / kUnitRows * kUnitRows);
    const bool wide = rows > kStreamRows;
    const int rr = in % kStreamRows, st0 = wide ? in / kStreamRows : 0;
    const size_t at = static_cast<size_t>(r) * a.hq + j * kGroup + h;
    float4 *outp = reinterpret_cast<float4 *>(a.out + at * kHeadDim) + d4;
    float m = a.lse[at], l = m == -INFINITY ? 0.f : 1.f;         // the own part: normalised, weight 2^lse
    float4 o = *outp;
    __syncwarp();
    for (int b = b0; b <= b1; ++b) {
        const int mine = min(share_lo(b + 1, W, n), w0 + tiles) - max(share_lo(b, W, n), w0);
        const int st1 = wide || mine < 2 ? st0 : 1;
        for (int st = st0; st <= st1; ++st) {
            const float *pp = part + (static_cast<size_t>(b) * 2 + st) * kPrefixPart;
            const float pm = pp[kStreamRows * kHeadDim + rr], pl = pp[kStreamRows * kHeadDim + kStreamRows + rr];
            const float4 po = *reinterpret_cast<const float4 *>(pp + (d4 * kStreamRows + rr) * 4);
            const float mn = fmaxf(m, pm), mu = mn == -INFINITY ? 0.f : mn;
            const float e0 = exp2f(m - mu), e1 = exp2f(pm - mu);
            o.x = o.x * e0 + po.x * e1;
            o.y = o.y * e0 + po.y * e1;
            o.z = o.z * e0 + po.z * e1;
            o.w = o.w * e0 + po.w * e1;
            l = l * e0 + pl * e1;
            m = mn;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *outp = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (d4 == 0) a.lse[at] = m == -INFINITY ? m : m + log2f(l);
}

cudaError_t launch_shared_merge(const PrefixArgs &a, cudaStream_t stream)
{
    k_shared_merge<<<a.batch * a.hkv, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- attention weights
// Adds every listed token's attention weight, summed over the group's heads,
// to weights[page][head][slot].  One thread per (list entry, 4 tokens); the
// adds are reductions at L2, so a page listed by several requests collects
// all their weights (in no fixed order), and a page listed once gets exactly
// one add per token.
__global__ void __launch_bounds__(256) k_weights(const float *__restrict__ logits, const float *__restrict__ lse,
                                                 const int32_t *__restrict__ lists,
                                                 const int32_t *__restrict__ lengths,
                                                 const int32_t *__restrict__ seq_lens, int hkv, int max_pages,
                                                 long long num_pages, float *weights)
{
    pdl_wait();
    const int u = blockIdx.y, r = u / hkv, j = u % hkv;
    const int len = min(max(lengths[u], 0), max_pages);
    int L = seq_lens[r];
    L = min(max(L, 0), max_pages * kPageSize);
    const int tail = L % kPageSize;
    float z[kGroup];
#pragma unroll
    for (int h = 0; h < kGroup; ++h) z[h] = lse[static_cast<size_t>(r) * hkv * kGroup + j * kGroup + h];
    for (int e = blockIdx.x * blockDim.x + threadIdx.x; e < len * 4; e += gridDim.x * blockDim.x) {
        const int i = e >> 2, t0 = (e & 3) * 4;
        const int pid = lists[static_cast<size_t>(u) * max_pages + i];
        if (pid < 0 || pid >= num_pages) continue;               // the attention skipped it and flagged it
        const float4 *lg = reinterpret_cast<const float4 *>(logits + (static_cast<size_t>(u) * max_pages + i) * kLogitPage + t0);
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
            const float4 s = lg[h * 4];
            w[0] += exp2f(s.x - z[h]);
            w[1] += exp2f(s.y - z[h]);
            w[2] += exp2f(s.z - z[h]);
            w[3] += exp2f(s.w - z[h]);
        }
        const int ntok = i == len - 1 && tail ? tail : kPageSize;
        float *dst = weights + (static_cast<size_t>(pid) * hkv + j) * kPageSize + t0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (t0 + x < ntok) atomicAdd(dst + x, w[x]);
    }
}

cudaError_t launch_weights(const float *logits, const float *lse, const int32_t *lists, const int32_t *lengths,
                           const int32_t *seq_lens, int batch, int hkv, int max_pages, long long num_pages,
                           float *weights, cudaStream_t stream)
{
    const int bx = (max_pages * 4 + 255) / 256;
    k_weights<<<dim3(bx, batch * hkv), 256, 0, stream>>>(logits, lse, lists, lengths, seq_lens, hkv, max_pages,
                                                          num_pages, weights);
    return cudaGetLastError();
}

}  // namespace moira
