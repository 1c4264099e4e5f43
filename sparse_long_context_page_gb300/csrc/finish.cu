// The last part of the shared-prefix and the weight-accumulating attention:
// joins a (request, KV head)'s partials over its own list (k_own) and over its
// group's prefix (k_prefix) into the output, and adds the own tokens'
// attention weights.
//
// With partials (m_k, l_k, o_k) of the row, M = max m_k:
//   out = sum_k 2^(m_k - M) o_k / Z,  Z = sum_k 2^(m_k - M) l_k
//   weight of token t = sum over the 4 heads of 2^(s_t - M) / Z
// grid (x, list): every block of a list first forms M and Z from the partials'
// maxima and sums (a few KB), then block x takes its slice of the output's
// dimensions (the first few blocks) and of the list's pages.  Bound by latency
// (about 8 us from the last partial to the last weight, 12 us for 2048 lists;
// its loads are batched so that every step is one trip to L2); the weights read
// 256 B and add 64 B a page.
#include "own_plan.cuh"
#include "shared_plan.cuh"

namespace moira {

constexpr int kFinishThreads = 256;
constexpr int kFinishBatch = 256;                   // partials joined at a time
constexpr uint32_t kNoPartial = 0xFFFFFFFFu;
constexpr int kFinishOut = 16;                      // most blocks of a list that share its output (8 dims each)

struct FinishSmem {
    float e[kFinishBatch][kGroup];                  // a partial's weight
    uint32_t at[kFinishBatch];                      // its address: (own slot << 1) or (prefix half unit << 1 | 1)
    float red[kFinishThreads / 32][kGroup];
    float4 sum[kFinishThreads];
    int g, start, req, woff, wnext, uoff;
};

// More blocks a SM without weights, which keep logits in registers.
template <bool kWeights>
__global__ void __launch_bounds__(kFinishThreads, kWeights ? 2 : 4) k_finish(const SharedArgs a)
{
    __shared__ FinishSmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.y, r = u / a.hkv, j = u & (a.hkv - 1);
    const int outs = min(1 << (31 - __clz(gridDim.x)), kFinishOut);      // a power of two
    if (tid == 0) sm.g = -1;
    pdl_wait();
    // ---- where the partials lie ----------------------------------------------
    const int o0 = a.offsets[u], o1 = a.offsets[u + 1], entries = o1 - o0;
    const OwnSplit split(a.offsets[a.units], a.offsets[a.units + 1]);
    const PlanRecord &plan = *static_cast<const PlanRecord *>(a.plan);
    int R = 1, W = 0, blocks = 0;
    if (a.groups > 0) {
        R = plan.team;
        blocks = plan.blocks;
        W = plan.woff[a.groups];
        __syncthreads();
        for (int g = tid; g < a.groups; g += kFinishThreads) {
            const int s = plan.start[g], sn = plan.start[g + 1], w = plan.woff[g], wn = plan.woff[g + 1];
            if (s <= r && r < sn && w < wn) {
                sm.g = g;
                sm.start = s;
                sm.req = sn - s;
                sm.woff = w;
                sm.wnext = wn;
                sm.uoff = plan.uoff[g];
            }
        }
        __syncthreads();
    }
    int n_own = 0, w_first = 0;
    if (entries > 0) {
        w_first = split.share_of(o0);
        n_own = split.share_of(o1 - 1) - w_first + 1;
    }
    int n_pre = 0, b0 = 0, w0 = 0, tiles = 0, unit = 0, member = 0, n_team = 1, in = 0;
    bool wide = false;
    if (a.groups > 0 && sm.g >= 0) {
        const int rounds = rounds_of(sm.req, R);
        tiles = (sm.wnext - sm.woff) / (a.hkv * rounds);
        const int row0 = (r - sm.start) * kGroup, rt = row0 / kUnitRows, round = rt / R;
        in = row0 % kUnitRows;
        member = rt - round * R;
        unit = sm.uoff + j * rounds + round;
        n_team = min(blocks / R, W);
        w0 = sm.woff + (j * rounds + round) * tiles;
        b0 = share_of(w0, W, n_team);
        // a unit of more than 128 rows: the row's own stream; else both streams
        wide = min(kUnitRows, sm.req * kGroup - rt * kUnitRows) > kStreamRows;
        n_pre = (share_of(w0 + tiles - 1, W, n_team) - b0 + 1) * (wide ? 1 : 2);
    }
    const int count = n_own + n_pre;

    // the first entry's logits load while the partials are joined
    const int32_t *list = a.lists + static_cast<size_t>(u) * a.max_pages;
    const float4 *lg = reinterpret_cast<const float4 *>(a.logits + static_cast<size_t>(u) * a.max_pages * kLogitPage);
    const int e_step = gridDim.x * kFinishThreads;
    int e = blockIdx.x * kFinishThreads + tid, pid = -1;
    float4 s4[kGroup];
    auto fetch = [&]() {
        if (e >= entries * 4) return;
        pid = __ldg(list + (e >> 2));
#pragma unroll
        for (int h = 0; h < kGroup; ++h)
            s4[h] = __ldcs(lg + static_cast<size_t>(e >> 2) * (kLogitPage / 4) + h * 4 + (e & 3));
    };
    if constexpr (kWeights) fetch();

    // ---- joint maximum and sum, and this block's slice of the output ---------
    // output thread: (partial slice, 4 dims and head) with the heads in
    // neighbouring lanes; `outs` blocks take 128 / outs dims each
    const bool has_out = static_cast<int>(blockIdx.x) < outs;
    const int cols = kHeadDim / outs / 4 * kGroup;               // threads of one partial slice: 128 to 8
    const int hh = tid & 3, d4 = static_cast<int>(blockIdx.x) * (kHeadDim / outs / 4) + (tid % cols) / kGroup;
    const int slice = tid / cols, slices = kFinishThreads / cols;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, Z = 0.f;                                // of head hh
    for (int k0 = 0; k0 < count; k0 += kFinishBatch) {
        const int cnt = min(kFinishBatch, count - k0);
        if (k0 > 0) __syncthreads();
        // thread (partial, head): its maximum and sum; a thread's loads are all
        // in flight together
        constexpr int kEach = kFinishBatch * kGroup / kFinishThreads;
        float mx = -INFINITY, mv[kEach], lv[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = (tid >> 2) + i * (kFinishThreads / kGroup), kk = k0 + k;
            uint32_t at = kNoPartial;
            const float *pp = nullptr;
            int l_off = kGroup;
            if (k < cnt) {
                if (kk < n_own) {
                    const uint32_t s = static_cast<uint32_t>(w_first + kk + u);
                    pp = a.own + static_cast<size_t>(s) * kPartFloats + hh;
                    at = s << 1;
                } else {
                    const int x = kk - n_own, b = b0 + (wide ? x : x >> 1), st = wide ? in / kStreamRows : x & 1;
                    // the second stream has nothing where the team took a single tile
                    if (wide || st == 0 ||
                        min(share_lo(b + 1, W, n_team), w0 + tiles) - max(share_lo(b, W, n_team), w0) >= 2) {
                        const uint32_t s = static_cast<uint32_t>(partial_slot(b, unit, member, R) * 2 + st);
                        pp = a.prefix + static_cast<size_t>(s) * kPrefixPart + kStreamRows * kHeadDim +
                             in % kStreamRows + hh;
                        l_off = kStreamRows;
                        at = s << 1 | 1u;
                    }
                }
                if (hh == 0) sm.at[k] = at;
            }
            mv[i] = pp ? __ldcg(pp) : -INFINITY;
            lv[i] = pp ? __ldcg(pp + l_off) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) mx = fmaxf(mx, mv[i]);
        // over the threads of this head: lanes 4 apart, then the warps
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        if (lane < kGroup) sm.red[warp][lane] = mx;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kFinishThreads / 32; ++w) mx = fmaxf(mx, sm.red[w][hh]);
        const float mn = fmaxf(M, mx), mu = mn == -INFINITY ? 0.f : mn, e0 = exp2f(M - mu);
        M = mn;
        Z *= e0;
        o.x *= e0;
        o.y *= e0;
        o.z *= e0;
        o.w *= e0;
        float ls = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = (tid >> 2) + i * (kFinishThreads / kGroup);
            if (k >= cnt) continue;
            const float e = exp2f(mv[i] - mu);
            sm.e[k][hh] = e;
            ls += e * lv[i];
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
        __syncthreads();                                         // red is read, e is written
        if (lane < kGroup) sm.red[warp][lane] = ls;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kFinishThreads / 32; ++w) Z += sm.red[w][hh];
        if (has_out) {
            constexpr int kInFlight = kWeights ? 8 : 4;
            for (int k = slice; k < cnt; k += slices * kInFlight) {
                float4 v[kInFlight];
#pragma unroll
                for (int i = 0; i < kInFlight; ++i) {
                    const int kk = k + i * slices;
                    const uint32_t at = kk < cnt ? sm.at[kk] : kNoPartial;
                    const float *pp = (at & 1u) ? a.prefix + static_cast<size_t>(at >> 1) * kPrefixPart +
                                                      (d4 * kStreamRows + in % kStreamRows + hh) * 4
                                                : a.own + static_cast<size_t>(at >> 1) * kPartFloats + 2 * kGroup +
                                                      hh * kHeadDim + d4 * 4;
                    v[i] = at != kNoPartial ? __ldcg(reinterpret_cast<const float4 *>(pp))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < kInFlight; ++i) {
                    const int kk = k + i * slices;
                    const float e = kk < cnt ? sm.e[kk][hh] : 0.f;
                    o.x = fmaf(e, v[i].x, o.x);
                    o.y = fmaf(e, v[i].y, o.y);
                    o.z = fmaf(e, v[i].z, o.z);
                    o.w = fmaf(e, v[i].w, o.w);
                }
            }
        }
    }
    if (has_out) {
        sm.sum[tid] = o;
        __syncthreads();
        if (slice == 0) {
            for (int s = 1; s < slices; ++s) {
                const float4 v = sm.sum[s * cols + tid];
                o.x += v.x;
                o.y += v.y;
                o.z += v.z;
                o.w += v.w;
            }
            const float inv = Z == 0.f ? 0.f : 1.f / Z;
            reinterpret_cast<float4 *>(a.out + (static_cast<size_t>(u) * kGroup + hh) * kHeadDim)[d4] =
                make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
    }

    // ---- weights: thread (list entry, 4 tokens) -------------------------------
    // The adds are reductions at L2: a page listed by several requests collects
    // all their weights (in no fixed order), a page listed once gets exactly one
    // add per token.
    if (!kWeights || entries == 0) return;
    float z[kGroup];                                             // log2 of every head's sum
    {
        const float mine = M == -INFINITY ? M : M + log2f(Z);
#pragma unroll
        for (int h = 0; h < kGroup; ++h) z[h] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + h);
    }
    const int L = min(max(a.seq_lens[r], 0), a.max_pages * kPageSize), tail = L % kPageSize;
    for (; e < entries * 4; e += e_step, fetch()) {
        const int i = e >> 2, q = e & 3;
        if (pid < 0 || pid >= a.num_pages) continue;             // k_own skipped it and flagged it
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
            w.x += ex2_approx(s4[h].x - z[h]);
            w.y += ex2_approx(s4[h].y - z[h]);
            w.z += ex2_approx(s4[h].z - z[h]);
            w.w += ex2_approx(s4[h].w - z[h]);
        }
        float *dst = a.weights + (static_cast<size_t>(pid) * a.hkv + j) * kPageSize + q * 4;
        const int ntok = i == entries - 1 && tail ? tail - q * 4 : 4;
        if (ntok >= 4) {
            red_add_f32x4(reinterpret_cast<float4 *>(dst), w);
        } else {                                                 // slots behind the last token stay as they are
            if (ntok > 0) atomicAdd(dst, w.x);
            if (ntok > 1) atomicAdd(dst + 1, w.y);
            if (ntok > 2) atomicAdd(dst + 2, w.z);
        }
    }
}

cudaError_t launch_finish(const SharedArgs &a, cudaStream_t stream)
{
    // Blocks of a list: about two a SM over all lists, so that a list's output
    // (few lists have many partials each) is spread over up to kFinishOut of
    // them; more only where its weights have pages for them (64 a block and pass).
    const int fill = (a.blocks * 2 + a.units - 1) / a.units;
    int x = fill < kFinishOut ? fill : kFinishOut;
    if (a.weights) {
        const int pages = (a.max_pages * 4 + kFinishThreads - 1) / kFinishThreads;
        const int want = fill < pages ? fill : pages;
        if (want > x) x = want;
    }
    if (a.weights) return launch_pdl(k_finish<true>, dim3(x, a.units), dim3(kFinishThreads), 0, stream, a);
    return launch_pdl(k_finish<false>, dim3(x, a.units), dim3(kFinishThreads), 0, stream, a);
}

}  // namespace moira
