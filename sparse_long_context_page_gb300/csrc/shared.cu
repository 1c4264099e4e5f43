// Attention over the prefixes that groups of requests share, the middle part
// of the shared-prefix attention.
//
// Every group of consecutive requests [start_g, start_{g+1}) shares the first
// len_g tokens of one page list.  For a query row (request r, head h) the
// softmax runs over the prefix and the request's own tokens together; both
// parts are computed apart and joined by their log-sum-exp:
//   own:    k_own, over the request's lists (own.cu)
//   prefix: k_prefix, all query rows of a (group, KV head) against each key
//           tile, so the prefix is read once for the group and not once per
//           request; the keys are split over the grid and every split leaves
//           a partial (max, sum, unnormalised output)
//   joint:  k_finish (finish.cu)
#include "own_plan.cuh"
#include "shared_plan.cuh"

namespace moira {

// ---------------------------------------------------------------- prefix attention
// k_prefix: one block per SM, its warps in four roles around two streams of
// 128 query rows (the 128 lanes of the tensor memory):
//   producers (2 warps) TMA page loads into a ring of 32 KB tiles (128 tokens): one loads the keys', one the values'
//   issuer    (1 warp)  issues the tcgen05 products
//   softmax   (2 x 8 warps, two threads per row, 64 of the tile's 128 scores each) S -> P in tensor memory
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
// What bounds it: up to 128 rows the prefix's bytes (8 requests on 128k tokens,
// 8 heads, 537 MB: 94 us, 5.7 TB/s, of which 6 us pass before the first tile is
// there).  Above, the turn of a stream through its products and its softmax
// (256 requests on 32k: 173 us beside the own lists, on 124 of the SMs, where
// the products alone, P's residual among them, would take 107 us).  Half of P's
// products less would save 9%, its stores to tensor memory 7%: no one part
// bounds it.  Tried without gain: two S buffers of 64 keys a stream with the
// softmax in turns or a softmax warpgroup for each (-0.5%, +15%), the products
// of P in two steps (-1%), 104 registers for the softmax warps (+1%).
// Rounding: S and O are fp32 sums of the tensor cores, P enters with 16 bits;
// outputs are 1e-6 to 3e-6 off (relative L2), by P's 16 bits and the drift of
// a chain (kChainTiles) in about equal parts.  A third term of P would need 128 more columns of
// tensor memory than there are.
constexpr int kRingSlots = 5;
constexpr int kTileBytes = kTileKeys * kHeadDim * 2;              // 32 KB
constexpr int kHalfTile = kTileKeys * 128;                       // 128 rows x 128 B
constexpr int kSoftmaxWarps = 8;                                 // of one stream
constexpr int kKeyWarp = 2 * kSoftmaxWarps, kValueWarp = kKeyWarp + 1, kIssuerWarp = kKeyWarp + 2;
constexpr int kPrefixThreads = (kIssuerWarp + 1) * 32;
constexpr int kMaskRing = 16;                                    // tiles whose key masks are kept
constexpr float kMaxSlack = 8.f;                                 // log2 units a row's maximum may pass its reference by
constexpr float kPartSlack = 60.f;                               // the same for a partial's, whose sums stay far below 2^127
struct PrefixSmem {
    unsigned long long full[kRingSlots], empty[kRingSlots];
    unsigned long long q_full[2], s_full[2], p_full[2], o_full[2], done;
    uint32_t tmem;
    int abort;
    int own_pages, own_lists;                                    // list entries, lists that have any, and the
    int2 work;                                                   // prefix work, for the split of the SMs
    float row_max[2][kStreamRows];                               // exchange between a row's two threads, per stream
    uint4 mask[kMaskRing];                                       // keys of a tile that count
    GroupPlan plan;
};
constexpr int kPrefixSmemBytes = (2 + kRingSlots) * kTileBytes + static_cast<int>(sizeof(PrefixSmem));
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

// The producer of the keys' or the values' tiles; both walk the whole ring.
template <bool keys>
__device__ void prefix_produce(const SharedArgs &a, const CUtensorMap *map, uint8_t *ring, PrefixSmem &sm,
                               SegmentWalk walk, const WaitGuard &wg)
{
    const int lane = threadIdx.x & 31, page = lane & 7, half = (lane >> 3) & 1;
    RingPos pos;
    int n_tiles = 0;                                             // K tiles so far
    Segment s;
    while (walk.next(s)) {
        const int len = prefix_len(a, s.g);
        const int32_t *table = a.prefix_table + static_cast<size_t>(s.g) * a.prefix_pages;
        // one tile's keys or values into the next ring slot; lane (half, page) copies one box
        auto load = [&](int tile, bool its_keys) {
            if (its_keys != keys) {
                pos.advance();
                return;
            }
            const int p = tile * kTilePages + page, tok = len - p * kPageSize;     // tokens from this page on
            const int pid = tok > 0 ? __ldcg(table + p) : -1;
            const bool ok = tok > 0 && pid >= 0 && pid < a.num_pages;
            mbar_wait_g(smem_u32(&sm.empty[pos.slot]), pos.round ^ 1u, wg);
            uint8_t *dst = ring + pos.slot * kTileBytes;
            const uint32_t full = smem_u32(&sm.full[pos.slot]);
            // values of tokens that do not count must be finite (their P is 0): a
            // partly filled page is copied by hand, a missing one is zeroed
            const bool whole = ok && (keys || tok >= kPageSize);
            if constexpr (keys) {
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
                            x = __ldcg(reinterpret_cast<const uint4 *>(a.v_pool) +
                                       ((static_cast<size_t>(id) * a.hkv + s.j) * kPageSize + t) * 16 + c);
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
                tma_load_2d(smem_u32(dst) + half * kHalfTile + page * kHalfBytes, map, half * 64,
                            (pid * a.hkv + s.j) * kPageSize, full);
            __syncwarp();
            if constexpr (keys) ++n_tiles;
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
        for (int i = 0; i < kRingSlots; ++i)                     // every slot's last round, if it had one
            mbar_drain(smem_u32(&sm.full[i]), i < pos.slot ? pos.round : pos.round ^ 1u, deadline);
    }
}

// The issuing warp: S and O products of both streams in the ring's order.  The
// whole warp walks and waits, so that addresses and loop counts stay in uniform
// registers, which the product instructions read; one lane issues.
__device__ void prefix_issue(uint32_t q_base, uint32_t ring, PrefixSmem &sm, SegmentWalk walk, const WaitGuard &wg)
{
    constexpr uint32_t kIdescS = umma_idesc_bf16(128, kTileKeys, false);
    constexpr uint32_t kIdescO = umma_idesc_bf16(128, kHeadDim, true);
    const uint32_t tmem = warp_uniform(sm.tmem);
    // descriptors differ in the start address alone, in units of 16 bytes
    const uint32_t q_desc = umma_desc_lo(q_base, 16), k_desc = umma_desc_lo(ring, 16), v_desc = umma_desc_lo(ring, kHalfTile);
    constexpr uint32_t kTileStep = kTileBytes >> 4;
    RingPos pos;
    uint32_t q_par = 0u, p_par = 0u;                              // bit s: stream s
    Segment s;
    while (walk.next(s)) {
        const int T = warp_uniform(s.t1 - s.t0);
        const bool wide = warp_uniform(s.wide());
        for (int st = 0; st < 2; ++st)
            if (s.tiles(st) > 0) {
                mbar_wait_g(smem_u32(&sm.q_full[st]), (q_par >> st) & 1u, wg);
                q_par ^= 1u << st;
            }
        tcgen05_fence_after();
        auto qk = [&](int st, uint32_t kt) {
            if (elect_one()) {
                const uint32_t qd = q_desc + st * kTileStep, d = tmem_s(tmem, st);
#pragma unroll
                for (int ks = 0; ks < kHeadDim / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalfTile + (ks & 3) * 32) >> 4;
                    umma_ss(d, umma_desc(qd + off, 1024), umma_desc(kt + off, 1024), kIdescS, ks > 0);
                }
                umma_commit(smem_u32(&sm.s_full[st]));
            }
            __syncwarp();
        };
        auto pv = [&](int st, uint32_t vt, int nth) {
            mbar_wait_g(smem_u32(&sm.p_full[st]), (p_par >> st) & 1u, wg);
            p_par ^= 1u << st;
            tcgen05_fence_after();
            const bool acc = (nth & (s.chain(st) - 1)) != 0;
            const bool last = nth + 1 == s.tiles(st);
            if (elect_one()) {
                const uint32_t d = tmem_o(tmem, st), p = tmem_s(tmem, st);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < kTileKeys / 16; ++ks)
                        umma_ts(d, p + (ks >> 1) * 32 + part * 16 + (ks & 1) * 8, umma_desc(vt + ks * (2048 >> 4), 1024),
                                kIdescO, part || ks ? true : acc);
                if (last) umma_commit(smem_u32(&sm.o_full[st]));
            }
            __syncwarp();
        };
        // the low words of the descriptors of a ring slot, once its tile is there
        auto wait_tile = [&](const RingPos &r, uint32_t base) {
            mbar_wait_g(smem_u32(&sm.full[r.slot]), r.round, wg);
            tcgen05_fence_after();
            return base + r.slot * kTileStep;
        };
        auto release = [&]() {                                   // the ring's oldest tile, once its products are done
            if (elect_one()) umma_commit(smem_u32(&sm.empty[pos.slot]));
            __syncwarp();
            pos.advance();
        };
        if (wide) {
            uint32_t kt = wait_tile(pos, k_desc);
            qk(0, kt);
            qk(1, kt);
            release();
            for (int i = 0; i < T; ++i) {
                RingPos kp = pos;
                kp.advance();
                const uint32_t vt = wait_tile(pos, v_desc);
                const bool more = i + 1 < T;
                pv(0, vt, i);
                if (more) {
                    kt = wait_tile(kp, k_desc);
                    qk(0, kt);
                }
                pv(1, vt, i);
                release();
                if (more) {
                    qk(1, kt);
                    release();
                }
            }
        } else {
            for (int i = 0; i < min(T, 2); ++i) {
                qk(i, wait_tile(pos, k_desc));
                release();
            }
            for (int i = 0; i < T; ++i) {
                pv(i & 1, wait_tile(pos, v_desc), i >> 1);
                release();
                if (i + 2 < T) {
                    qk(i & 1, wait_tile(pos, k_desc));
                    release();
                }
            }
        }
    }
    if (elect_one()) umma_commit(smem_u32(&sm.done));
    __syncwarp();
}

// The two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int bar) { asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory"); }
__device__ __forceinline__ bool bar_any(int bar, bool v)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(bar), "r"(v ? 1u : 0u)
                 : "memory");
    return any != 0;
}

// One softmax stream: 8 warps; warp w and w + 4 share 32 rows (the lanes of the
// tensor memory that they reach), thread = (row, half of the columns).
__device__ void prefix_softmax(const SharedArgs &a, uint8_t *q_smem, PrefixSmem &sm, SegmentWalk walk, int stream,
                               const WaitGuard &wg)
{
    const int tid = threadIdx.x & (kSoftmaxWarps * 32 - 1), row = tid & 127, lane = tid & 31, half = tid >> 7;
    const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
    const uint32_t ts = tmem_s(sm.tmem, stream) + lanes + half * 64, to = tmem_o(sm.tmem, stream) + lanes + half * 64;
    const int pair_bar = 1 + stream * 4 + (row >> 5);            // named barrier of the two warps of these rows
    const float c = a.scale_log2;
    uint32_t s_par = 0u, o_par = 0u;
    int n_tiles = 0;                                             // K tiles of the block before this segment
    Segment s;
    while (walk.next(s)) {
        const int T = s.tiles(stream), chain = s.chain(stream);
        const bool wide = s.wide();
        const int base_tile = n_tiles;
        n_tiles += s.t1 - s.t0;
        if (T == 0) continue;
        const int first = s.row0 + (wide ? stream * kStreamRows : 0);
        const int rows = min(kStreamRows, s.rows - (wide ? stream * kStreamRows : 0));
        // the stream's query rows (the last segment's products are complete: o_full)
        const uint16_t *q = static_cast<const uint16_t *>(a.q) +
                            (static_cast<size_t>(walk.p.start[s.g]) * a.hq + s.j * kGroup) * kHeadDim;
        {
            constexpr int kLoads = kStreamRows * 16 / (kSoftmaxWarps * 32);
            uint4 x[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int e = tid + i * kSoftmaxWarps * 32, r = e >> 4, ch = e & 15, rr = first + r;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows)
                    x[i] = __ldcg(reinterpret_cast<const uint4 *>(
                        q + (static_cast<size_t>(rr / kGroup) * a.hq + rr % kGroup) * kHeadDim + ch * 8));
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int e = tid + i * kSoftmaxWarps * 32, r = e >> 4, ch = e & 15;
                *reinterpret_cast<uint4 *>(q_smem + (ch >> 3) * kHalfTile + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x[i];
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[stream]));

        const int R = walk.p.team;
        float *part = a.prefix + (partial_slot(blockIdx.x / R, s.unit, walk.member, R) * 2 + stream) * kPrefixPart;
        float4 *part_o = reinterpret_cast<float4 *>(part) + half * 16 * kStreamRows + row;
        const bool live = (row & ~31) < rows;                    // this warp has a row that counts
        float m = -INFINITY, l = 0.f, m_part = -INFINITY;
        bool fresh = true;                                       // nothing of this segment in the partial yet
        // adds O (this thread's 64 columns) to the partial in global memory, whose
        // reference stays at m_part: the first time it writes it, later the adds
        // are reductions at L2 that nothing waits for.  Only a reference that has
        // moved on by 2^kPartSlack rescales what is there.
        auto flush = [&](bool first) {
            if (first) m_part = m;
            const bool rebase = !first && m - m_part > kPartSlack;
            const float f = rebase ? exp2f(m_part - m) : 1.f;
            if (rebase) m_part = m;
            const float g = m_part == -INFINITY ? 1.f : exp2f(m - m_part);
            const bool slow = __any_sync(0xffffffffu, rebase);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t o[32];
                tmem_ld32(to + b * 32, o);
                tmem_wait_ld(o);
                if (row < rows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4 *pp = part_o + (b * 8 + i) * kStreamRows;
                        float4 v = make_float4(__uint_as_float(o[4 * i]) * g, __uint_as_float(o[4 * i + 1]) * g,
                                               __uint_as_float(o[4 * i + 2]) * g, __uint_as_float(o[4 * i + 3]) * g);
                        if (first) {
                            *pp = v;
                        } else if (slow) {
                            const float4 old = __ldcg(pp);
                            *pp = make_float4(fmaf(old.x, f, v.x), fmaf(old.y, f, v.y), fmaf(old.z, f, v.z),
                                              fmaf(old.w, f, v.w));
                        } else {
                            red_add_f32x4(pp, v);
                        }
                    }
                }
            }
        };
        for (int i = 0; i < T; ++i) {
            const bool chain_start = (i & (chain - 1)) == 0;
            mbar_wait_g(smem_u32(&sm.s_full[stream]), s_par, wg);
            s_par ^= 1u;
            tcgen05_fence_after();
            if (live) {
                if (chain_start && i > 0) {
                    flush(fresh);
                    fresh = false;
                }
                const uint2 mask = reinterpret_cast<const uint2 *>(
                    &sm.mask[(base_tile + (wide ? i : 2 * i + stream)) % kMaskRing])[half];
                // keys that do not count, in a prefix's last tile and in missing pages
                // alone: their scores are overwritten first, out of the others' way
                if ((mask.x & mask.y) != 0xFFFFFFFFu) {
#pragma unroll 1
                    for (int b = 0; b < 8; ++b) {
                        uint32_t v[8];
                        tmem_ld8(ts + b * 8, v);
                        tmem_wait_ld(v);
                        const uint32_t bits = (b < 4 ? mask.x : mask.y) >> (b & 3) * 8;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (!(bits >> k & 1u)) v[k] = 0xFF800000u;
                        tmem_st8(ts + b * 8, v);
                    }
                    tmem_wait_st();
                }
                // the thread's 64 scores, 32 at a time; the second half is read again
                // for P (held at once with what else lives here they would spill)
                uint32_t x[32], y[32];
                tmem_ld32(ts, x);
                tmem_ld32(ts + 32, y);
                tmem_wait_ld(x);
                tmem_wait_ld(y);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; k += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = max3(mx[e], __uint_as_float(x[k + e]), __uint_as_float(y[k + e]));
                float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                // has a row of the pair's 32 passed its reference?  Rarely: then the
                // halves exchange their maxima and move the reference together
                mt *= c;
                const bool pass = mt > m + kMaxSlack || (m == -INFINITY && mt > -INFINITY);
                if (bar_any(pair_bar, pass)) {
                    if (half) sm.row_max[stream][row] = mt;
                    pair_sync(pair_bar);
                    if (!half) sm.row_max[stream][row] = mt = fmaxf(mt, sm.row_max[stream][row]);
                    pair_sync(pair_bar);
                    if (half) mt = sm.row_max[stream][row];
                    const bool move = mt > m + kMaxSlack || (m == -INFINITY && mt > -INFINITY);
                    const float mn = move ? mt : m;
                    const float al = m == -INFINITY ? (move ? 0.f : 1.f) : exp2f(m - mn);
                    l *= al;
                    m = mn;
                    if (!chain_start) {
                        // the previous product is complete (S of this tile was issued after it)
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            uint32_t o[8];
                            tmem_ld8(to + b * 8, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                            tmem_st8(to + b * 8, o);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.f : m;
                const uint64_t c2 = pack_f32x2(c, c), mu2 = pack_f32x2(-mu, -mu), minus1 = pack_f32x2(-1.f, -1.f);
                uint64_t ls[2] = {0ull, 0ull};
                // 16 scores -> 8 registers of P and 8 of its residual
                auto emit = [&](const uint32_t (&v)[32], int h, uint32_t to_p) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t e = fma_f32x2(pack_b32x2(v[16 * h + 2 * k], v[16 * h + 2 * k + 1]), c2, mu2);
                        const float p0 = ex2_approx(f32x2_lo(e)), p1 = ex2_approx(f32x2_hi(e));
                        const uint64_t p = pack_f32x2(p0, p1);
                        ls[k & 1] = add_f32x2(ls[k & 1], p);
                        hi[k] = pack_bf16x2(p0, p1);
                        const uint64_t r = fma_f32x2(pack_f32x2(bf16_lo(hi[k]), bf16_hi(hi[k])), minus1, p);
                        lo[k] = pack_bf16x2(f32x2_lo(r), f32x2_hi(r));
                    }
                    tmem_st8(to_p + 8 * h, hi);
                    tmem_st8(to_p + 16 + 8 * h, lo);
                };
                emit(x, 0, ts);
                tmem_ld32(ts + 32, y);
                emit(x, 1, ts);
                tmem_wait_ld(y);
                emit(y, 0, ts + 32);
                emit(y, 1, ts + 32);
                const uint64_t lsum = add_f32x2(ls[0], ls[1]);
                l += f32x2_lo(lsum) + f32x2_hi(lsum);
                tmem_wait_st();
            }
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[stream]));
        }
        mbar_wait_g(smem_u32(&sm.o_full[stream]), o_par, wg);
        o_par ^= 1u;
        tcgen05_fence_after();
        if (live) {
            flush(fresh);
            // the row's two sums
            if (half) sm.row_max[stream][row] = l;
            pair_sync(pair_bar);
            if (!half && row < rows) {
                part[kStreamRows * kHeadDim + row] = m_part;
                part[kStreamRows * kHeadDim + kStreamRows + row] =
                    (l + sm.row_max[stream][row]) * (m_part == -INFINITY ? 1.f : exp2f(m - m_part));
            }
            pair_sync(pair_bar);
        }
        tcgen05_fence_before();
    }
}

__global__ void __launch_bounds__(kPrefixThreads, 1)
    k_prefix(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
             const SharedArgs a)
{
    extern __shared__ __align__(1024) uint8_t tiles[];           // the swizzled tiles start on 1024-byte boundaries
    PrefixSmem &sm = *reinterpret_cast<PrefixSmem *>(tiles + (2 + kRingSlots) * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5;
    const WaitGuard wg{&sm.abort, a.status};
    if (tid == 0) {
        for (int i = 0; i < kRingSlots; ++i) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), kSoftmaxWarps);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i]), kSoftmaxWarps);
            mbar_init(smem_u32(&sm.o_full[i]), 1);
        }
        mbar_init(smem_u32(&sm.done), 1);
        mbar_fence_init();
        guard_init(wg);
        sm.own_pages = sm.own_lists = 0;
    }
    if (warp == kIssuerWarp) tmem_alloc512(smem_u32(&sm.tmem));
    if (tid == kKeyWarp * 32) tma_prefetch_desc(&tmap_k);
    if (tid == kValueWarp * 32) tma_prefetch_desc(&tmap_v);
    // No wait for k_own here: the two share nothing but the merge, and k_own lets
    // this kernel start only after its own wait, when the results of earlier
    // kernels are in memory (they are read past L1).
    pdl_trigger();
    // the softmax warps count the list entries, the key warp plans
    int pages = 0, some = 0;
    if (warp < kKeyWarp)
        for (int u = tid; u < a.units; u += kKeyWarp * 32) {
            const int len = min(max(__ldcg(a.lengths + u), 0), a.max_pages);
            pages += len;
            some += len > 0;
        }
    if (warp == kKeyWarp) plan_groups(a, sm.plan, sm.work);
    tcgen05_fence_before();
    __syncthreads();
    if (warp < kKeyWarp) {
        pages = __reduce_add_sync(0xffffffffu, pages);
        some = __reduce_add_sync(0xffffffffu, some);
        if ((tid & 31) == 0 && some) {
            atomicAdd(&sm.own_pages, pages);
            atomicAdd(&sm.own_lists, some);
        }
    }
    __syncthreads();
    tcgen05_fence_after();

    const int blocks = gridDim.x - (sm.plan.woff[a.groups] > 0 ? own_blocks(sm.own_pages, sm.own_lists, sm.work, gridDim.x) : 0);
    if (blockIdx.x == 0 && tid == 0) static_cast<PlanRecord *>(a.plan)->blocks = blocks;
    const int R = sm.plan.team, W = sm.plan.woff[a.groups];
    const int n = min((R == 1 ? blocks : static_cast<int>(static_cast<uint32_t>(blocks) / static_cast<uint32_t>(R))), W);
    const int b = R == 1 ? blockIdx.x : static_cast<uint32_t>(blockIdx.x) / static_cast<uint32_t>(R);
    if (b < n) {
        const SegmentWalk walk{sm.plan, a.hkv, 31 - __clz(a.hkv), static_cast<int>(blockIdx.x) - b * R, share_lo(b, W, n),
                               share_lo(b + 1, W, n), 0, 0};
        uint8_t *ring = tiles + 2 * kTileBytes;
        if (warp == kKeyWarp) {
            prefix_produce<true>(a, &tmap_k, ring, sm, walk, wg);
        } else if (warp == kValueWarp) {
            prefix_produce<false>(a, &tmap_v, ring, sm, walk, wg);
        } else if (warp == kIssuerWarp) {
            prefix_issue(smem_u32(tiles), smem_u32(ring), sm, walk, wg);
            // nothing may be in flight when the tensor memory is freed
            if (!mbar_try_wait(smem_u32(&sm.done), 0u))
                mbar_drain(smem_u32(&sm.done), 0u, globaltimer() + kDrainLimitNs);
        } else {
            prefix_softmax(a, tiles + warp / kSoftmaxWarps * kTileBytes, sm, walk, warp / kSoftmaxWarps, wg);
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (warp == kIssuerWarp) tmem_free512(sm.tmem);
    pdl_wait();                                                  // k_finish, which waits for this kernel, reads k_own's partials too
}

namespace {
std::atomic<int> g_prefix_smem_seen[64];
}

cudaError_t launch_prefix(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const SharedArgs &a,
                          cudaStream_t stream)
{
    const cudaError_t e = raise_smem_limit(k_prefix, kPrefixSmemBytes, g_prefix_smem_seen);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_prefix, dim3(a.blocks), dim3(kPrefixThreads), kPrefixSmemBytes, stream, tmap_k, tmap_v, a);
}

}  // namespace moira
