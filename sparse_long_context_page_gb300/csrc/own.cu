// Attention over each request's own page lists as partials, the first part of
// the shared-prefix and the weight-accumulating attention.
//
// The lists, laid end to end, are split evenly over all warps of the grid, and
// a warp works alone: it streams its pages through its own ring of TMA loads,
// keeps the running maximum, sum and output of the list it is in, and leaves a
// partial per (warp, list) in the workspace.  There is no barrier and no
// arrival between warps after the plan, so many short lists cost no more than
// few long ones (256 requests of 128 to 1024 tokens, 8 heads, 450 MB: k_attend,
// whose blocks combine five warps at every list's end, takes 146 us).  What
// joins the partials is k_finish, which joins the prefix's too.  (The same 450 MB
// take 71 us here on all SMs; one request of 128k tokens, 546 MB with the
// logits, 89 us, 6.1 TB/s.)  Twelve warps of two slots each: 192 KB in flight a
// SM; eight of three slots take 2% longer.
//
// Per page (16 tokens) and the group's 4 heads
//   S^T[h][t] = q_h . k_t : mma.m16n8k16, A = q (rows 0-3 and 4-7 both hold the
//                           4 heads), B = K^T via ldmatrix
//   O^T[d][h] += V^T P^T  : A = V^T via ldmatrix.trans, B columns 0-3 bf16(P),
//                           columns 4-7 its bf16 residual; a second product
//                           adds what these leave (P keeps 24 bits)
// in fp32, log2 domain.  The tensor cores add by truncation, so a page's product
// starts from zero and joins O by an fp32 multiply-add (3e-7 to 6e-7 off in
// relative L2; with two terms of P and O as the accumulator 1e-6, for 0.7% less
// time).  mma.sync and not tcgen05: 4 rows against 16 keys leave
// the tensor cores 97% idle in any shape, and the pages' bytes are the bound.
// With weights the scaled logits go to the workspace too (256 B beside the 8 KB
// that a page's keys and values take), since the weights need the joint sum.
#include "moira_device.cuh"
#include "moira_launch.h"
#include "own_plan.cuh"

namespace moira {

constexpr int kOwnSlots = 2;                        // pages of one warp in flight or in use
constexpr int kOwnPage = 2 * kPageSize * kHeadDim * 2;          // K and V of one (page, head)

struct OwnSmem {
    unsigned long long full[kOwnWarps][kOwnSlots];
    int tokens[kOwnWarps][kOwnSlots];               // of the slot's page; 0: skipped
    int wsum[kOwnWarps];
    int lists;                                      // that have pages
    int2 work;                                      // of the prefixes
    int abort;
};

__host__ __device__ constexpr size_t own_smem_bytes(int units)
{
    return static_cast<size_t>(kOwnWarps) * kOwnSlots * kOwnPage + sizeof(OwnSmem) + sizeof(int) * (units + 1);
}

__global__ void __launch_bounds__(kOwnWarps * 32, 1)
    k_own(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const SharedArgs a)
{
    extern __shared__ __align__(1024) uint8_t stage[];           // the swizzled boxes start on 1024-byte boundaries
    OwnSmem &sm = *reinterpret_cast<OwnSmem *>(stage + kOwnWarps * kOwnSlots * kOwnPage);
    int *s_off = reinterpret_cast<int *>(&sm + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.units;
    const WaitGuard wg{&sm.abort, a.status};
    if (tid < kOwnWarps * kOwnSlots) mbar_init(smem_u32(&sm.full[0][0] + tid), 1);
    if (tid == 0) {
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        guard_init(wg);
        sm.work = make_int2(0, 0);
        sm.lists = 0;
    }
    mbar_fence_init();
    pdl_wait();
    if (tid == 0) __threadfence();
    pdl_trigger();                                               // from here on earlier kernels' results are in memory

    // ---- plan: exclusive scan of the list lengths --------------------------
    {
        constexpr int kHeld = 8;                                 // lengths a thread keeps in registers
        const int per = (units + kOwnWarps * 32 - 1) / (kOwnWarps * 32);
        const int ub = min(units, tid * per), ue = min(units, ub + per);
        bool bad = false;
        auto length_of = [&](int u) {
            const int len = a.lengths[u];
            bad |= len < 0 || len > a.max_pages;
            return min(max(len, 0), a.max_pages);
        };
        // a thread's group, for the prefixes' work (k_prefix checks and mends the groups)
        static_assert(kMaxGroups <= kOwnWarps * 32, "a thread for every group");
        int gs = 0, ge = 0, glen = 0;
        if (tid < a.groups) {
            gs = min(max(a.group_starts[tid], 0), a.batch);
            ge = min(max(a.group_starts[tid + 1], gs), a.batch);
            glen = min(max(a.prefix_lens[tid], 0), a.prefix_pages * kPageSize);
        }
        int held[kHeld], mine = 0, some = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            held[i] = ub + i < ue ? length_of(ub + i) : 0;
            mine += held[i];
            some += held[i] > 0;
        }
        for (int u = ub + kHeld; u < ue; ++u) {
            const int len = length_of(u);
            mine += len;
            some += len > 0;
        }
        const int2 work = prefix_work(ge - gs, glen, a.hkv);
        if (bad) raise_status(a.status, kDevBadLen);
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sm.wsum[warp] = x;
        __syncthreads();
        if (work.x) atomicAdd(&sm.work.x, work.x);
        if (work.y) atomicAdd(&sm.work.y, work.y);
        some = __reduce_add_sync(0xffffffffu, some);
        if (lane == 0 && some) atomicAdd(&sm.lists, some);
        int run = x - mine;
        for (int w = 0; w < warp; ++w) run += sm.wsum[w];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (ub + i < ue) s_off[ub + i] = run;
            run += held[i];
        }
        for (int u = ub + kHeld; u < ue; ++u) {
            s_off[u] = run;
            run += length_of(u);
        }
        if (tid == kOwnWarps * 32 - 1) s_off[units] = run;
    }
    __syncthreads();
    const int blocks = own_blocks(s_off[units], sm.lists, sm.work, gridDim.x);
    if (blockIdx.x == 0) {
        for (int u = tid; u <= units; u += kOwnWarps * 32) a.offsets[u] = s_off[u];
        if (tid == 0) a.offsets[units + 1] = blocks;
    }
    if (static_cast<int>(blockIdx.x) >= blocks) return;

    const OwnSplit split(s_off[units], blocks);
    // neighbouring shares lie on different SMs
    const int gw = warp * blocks + blockIdx.x;
    if (gw >= split.n) return;
    const int k0 = split.lo(gw), k1 = split.lo(gw + 1);

    // ---- the warp's entries: lane i holds entry base + i of a batch of 32 ---
    auto list_of = [&](int k) {                                  // largest u with s_off[u] <= k
        int lo = 0, hi = units;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_off[mid] <= k) lo = mid; else hi = mid;
        }
        return lo;
    };
    int cu = 0, cn = 0, cp = 0, nu = 0, nn = 0, np = 0;          // list, valid tokens, page: this and the next batch
    auto look = [&](int k, int &u, int &ntok, int &pid) {
        u = ntok = pid = 0;
        if (k >= k1) return;
        u = list_of(k);
        const int i = k - s_off[u], len = s_off[u + 1] - s_off[u];
        pid = a.lists[static_cast<size_t>(u) * a.max_pages + i];
        const int L = min(max(a.seq_lens[u / a.hkv], 0), a.max_pages * kPageSize), tail = L % kPageSize;
        ntok = i == len - 1 && tail ? tail : kPageSize;
    };
    const uint64_t pol = l2_evict_first();
    uint8_t *ring = stage + warp * kOwnSlots * kOwnPage;
    int issued = 0, islot = 0;                                   // entries issued, the next one's slot
    look(k0 + lane, nu, nn, np);
    auto issue = [&]() {
        if (k0 + issued >= k1) return;
        const int at = issued & 31;
        if (at == 0) {
            cu = nu;
            cn = nn;
            cp = np;
            if (cn > 0 && (cp < 0 || cp >= a.num_pages)) {
                cn = 0;
                raise_status(a.status, kDevBadPage);
            }
            look(k0 + issued + 32 + lane, nu, nn, np);
        }
        const int u = __shfl_sync(0xffffffffu, cu, at), n = __shfl_sync(0xffffffffu, cn, at);
        const int pid = __shfl_sync(0xffffffffu, cp, at);
        if (lane == 0) {
            const uint32_t full = smem_u32(&sm.full[warp][islot]);
            sm.tokens[warp][islot] = n;
            if (n > 0) {
                const uint32_t dst = smem_u32(ring + islot * kOwnPage);
                const int row = (pid * a.hkv + (u & (a.hkv - 1))) * kPageSize;
                mbar_arrive_expect_tx(full, kOwnPage);
                tma_load_2d_hint(dst, &tmap_k, 0, row, full, pol);
                tma_load_2d_hint(dst + kHalfBytes, &tmap_k, 64, row, full, pol);
                tma_load_2d_hint(dst + 2 * kHalfBytes, &tmap_v, 0, row, full, pol);
                tma_load_2d_hint(dst + 3 * kHalfBytes, &tmap_v, 64, row, full, pol);
            } else {
                mbar_arrive(full);
            }
        }
        __syncwarp();
        ++issued;
        if (++islot == kOwnSlots) islot = 0;
    };
#pragma unroll
    for (int i = 0; i < kOwnSlots; ++i) issue();

    const int hq_row = (lane >> 2) & 3, tq = 2 * (lane & 3);      // this lane's row and columns of S^T
    const int hn0 = tq & 3;                                      // its first column of O^T
    const bool lo_lane = lane >= 16;                             // holds the residual columns of P
    const float c = a.scale_log2;
    auto load_q = [&](int u, uint32_t (&f)[8][2]) {
        const uint16_t *row = static_cast<const uint16_t *>(a.q) +
                              (static_cast<size_t>(u) * kGroup + hq_row) * kHeadDim + tq;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            f[ks][0] = __ldg(reinterpret_cast<const uint32_t *>(row + ks * 16));
            f[ks][1] = __ldg(reinterpret_cast<const uint32_t *>(row + ks * 16 + 8));
        }
    };
    int u = list_of(k0), slot = 0;
    uint32_t phase = 0u, aq[8][2];
    load_q(u, aq);
    for (int k = k0; k < k1;) {
        const int end = min(k1, s_off[u + 1]);
        int un = u;                                              // the next list; its queries load meanwhile
        uint32_t aqn[8][2];
        if (end < k1) {
            ++un;
            while (s_off[un + 1] == s_off[un]) ++un;
            load_q(un, aqn);
        }
        float m_run = -INFINITY, l_run = 0.f;
        float D[8][4];
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) D[mt][0] = D[mt][1] = D[mt][2] = D[mt][3] = 0.f;
        for (; k < end; ++k) {
            mbar_wait_g(smem_u32(&sm.full[warp][slot]), phase, wg);
            const int ntok = sm.tokens[warp][slot];
            if (ntok > 0) {
                const uint32_t kb = smem_u32(ring + slot * kOwnPage), vb = kb + 2 * kHalfBytes;
                float acc[4][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
                {
                    const int t = (lane & 7) + ((lane >> 4) << 3), sw = t & 7;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const int ch = 2 * ks + ((lane >> 3) & 1);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(kb + (ch >> 3) * kHalfBytes + t * 128 + (((ch & 7) ^ sw) << 4), b0, b1, b2, b3);
                        const int par = (ks & 1) * 2;
                        mma_bf16_16816(acc[par], aq[ks][0], 0u, aq[ks][1], 0u, b0, b1);
                        mma_bf16_16816(acc[par + 1], aq[ks][0], 0u, aq[ks][1], 0u, b2, b3);
                    }
                }
                float s[4] = {(acc[0][0] + acc[2][0]) * c, (acc[0][1] + acc[2][1]) * c,
                              (acc[1][0] + acc[3][0]) * c, (acc[1][1] + acc[3][1]) * c};
                uint32_t msk01 = 0xFFFFFFFFu, msk23 = 0xFFFFFFFFu;
                if (ntok < kPageSize) {
                    // tokens behind the last: no weight, and values (garbage, maybe NaN) as zeros
                    if (tq >= ntok) s[0] = -INFINITY;
                    if (tq + 1 >= ntok) s[1] = -INFINITY;
                    if (tq + 8 >= ntok) s[2] = -INFINITY;
                    if (tq + 9 >= ntok) s[3] = -INFINITY;
                    msk01 = (tq < ntok ? 0x0000FFFFu : 0u) | (tq + 1 < ntok ? 0xFFFF0000u : 0u);
                    msk23 = (tq + 8 < ntok ? 0x0000FFFFu : 0u) | (tq + 9 < ntok ? 0xFFFF0000u : 0u);
                }
                if (a.logits) {
                    // lanes 0-15 store tokens tq, tq+1 of their head, lanes 16-31
                    // (copies of the same heads) tokens tq+8, tq+9: 256 B in one go
                    float *lg = a.logits + (static_cast<size_t>(u) * a.max_pages + (k - s_off[u])) * kLogitPage +
                                hq_row * kPageSize + tq + (lo_lane ? 8 : 0);
                    *reinterpret_cast<float2 *>(lg) = lo_lane ? make_float2(s[2], s[3]) : make_float2(s[0], s[1]);
                }
                float pm = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
                pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 1));
                pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 2));
                const float m_new = fmaxf(m_run, pm), m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = ex2_approx(m_run - m_use);
                float p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) p[x] = ex2_approx(s[x] - m_use);
                l_run = l_run * alpha + (p[0] + p[1]) + (p[2] + p[3]);
                m_run = m_new;
                const uint32_t h01 = pack_bf16x2(p[0], p[1]), h23 = pack_bf16x2(p[2], p[3]);
                const float e0 = p[0] - bf16_lo(h01), e1 = p[1] - bf16_hi(h01);
                const float e2 = p[2] - bf16_lo(h23), e3 = p[3] - bf16_hi(h23);
                const uint32_t r01 = pack_bf16x2(e0, e1), r23 = pack_bf16x2(e2, e3);
                const uint32_t bp0 = lo_lane ? r01 : h01, bp1 = lo_lane ? r23 : h23;
                // what the first two leave
                const uint32_t t01 = lo_lane ? 0u : pack_bf16x2(e0 - bf16_lo(r01), e1 - bf16_hi(r01));
                const uint32_t t23 = lo_lane ? 0u : pack_bf16x2(e2 - bf16_lo(r23), e3 - bf16_hi(r23));
                const float al0 = __shfl_sync(0xffffffffu, alpha, 4 * hn0);
                const float al1 = __shfl_sync(0xffffffffu, alpha, 4 * (hn0 + 1));
                {
                    const int mi = lane >> 3, t = (lane & 7) + ((mi >> 1) << 3), sw = t & 7;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        const int ch = 2 * mt + (mi & 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4_trans(vb + (ch >> 3) * kHalfBytes + t * 128 + (((ch & 7) ^ sw) << 4), a0, a1, a2, a3);
                        float w[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_bf16_16816(w, a0 & msk01, a1 & msk01, a2 & msk23, a3 & msk23, t01, t23);
                        mma_bf16_16816(w, a0 & msk01, a1 & msk01, a2 & msk23, a3 & msk23, bp0, bp1);
                        D[mt][0] = fmaf(D[mt][0], al0, w[0]);
                        D[mt][1] = fmaf(D[mt][1], al1, w[1]);
                        D[mt][2] = fmaf(D[mt][2], al0, w[2]);
                        D[mt][3] = fmaf(D[mt][3], al1, w[3]);
                    }
                }
            }
            __syncwarp();                                        // the slot is read: refill it
            issue();
            if (++slot == kOwnSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        // the list's (or the share's) end: the warp's partial m[4], l[4], o[4][d]
        float *part = a.own + static_cast<size_t>(gw + u) * kPartFloats;
        float lsum = l_run + __shfl_xor_sync(0xffffffffu, l_run, 1);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
        if (lane < 16 && (lane & 3) == 0) {
            part[lane >> 2] = m_run;
            part[kGroup + (lane >> 2)] = lsum;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float v = D[mt][x] + __shfl_xor_sync(0xffffffffu, D[mt][x], 2);
                if ((lane & 3) < 2)
                    part[2 * kGroup + (tq + (x & 1)) * kHeadDim + 16 * mt + (lane >> 2) + (x >= 2 ? 8 : 0)] = v;
            }
        if (end < k1) {
            u = un;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                aq[ks][0] = aqn[ks][0];
                aq[ks][1] = aqn[ks][1];
            }
        }
    }
    // after a give-up, let the copies still in flight land before the block ends
    if (lane == 0 && guard_failed(wg)) {
        const uint64_t deadline = globaltimer() + kDrainLimitNs;
        const int n = k1 - k0;
        for (int s = 0; s < kOwnSlots && s < n; ++s) {
            const int last = n - 1 - (n - 1 - s) % kOwnSlots;    // the last entry on slot s
            mbar_drain(smem_u32(&sm.full[warp][s]), static_cast<uint32_t>(last / kOwnSlots) & 1u, deadline);
        }
    }
}

namespace {
std::atomic<int> g_own_smem_seen[64];
}

cudaError_t launch_own(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const SharedArgs &a, cudaStream_t stream)
{
    const size_t smem = own_smem_bytes(a.units);
    const cudaError_t e = raise_smem_limit(k_own, smem, g_own_smem_seen);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_own, dim3(a.blocks), dim3(kOwnWarps * 32), smem, stream, tmap_k, tmap_v, a);
}

}  // namespace moira
