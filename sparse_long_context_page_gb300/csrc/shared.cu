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

constexpr int kTileKeys = 64;                       // keys of one prefix work item

// The groups' work, laid end to end: group g has hkv * rtiles(g) units of
// tiles(g) key tiles each, unit = head * rtiles + row tile.
struct GroupPlan {
    int start[kMaxGroups + 1];                      // first request (sanitised: ascending, within the batch)
    int len[kMaxGroups];                            // prefix tokens
    int woff[kMaxGroups + 1];                       // key tiles before the group
    int uoff[kMaxGroups + 1];                       // units before the group
};

__device__ __forceinline__ int rtiles_of(int requests) { return (requests * kGroup + kUnitRows - 1) / kUnitRows; }
__device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }

// Every warp of the block may call it with its own plan; one warp fills it.
__device__ __forceinline__ void plan_groups(const PrefixArgs &a, GroupPlan &p)
{
    const int lane = threadIdx.x & 31;
    int before = 0, w = 0, u = 0;                   // carried over the chunks of 32 groups
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
        int s = max(min(max(raw, 0), a.batch), before), e = min(max(next, 0), a.batch);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s = max(s, y);
        }
        int sn = __shfl_down_sync(0xffffffffu, s, 1);           // the next group's start
        if (g == a.groups - 1 || lane == 31) sn = max(e, s);
        const int req = in ? max(sn - s, 0) : 0;
        const int units = a.hkv * rtiles_of(req), work = units * tiles_of(len);
        int wi = work, ui = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yw = __shfl_up_sync(0xffffffffu, wi, o), yu = __shfl_up_sync(0xffffffffu, ui, o);
            if (lane >= o) {
                wi += yw;
                ui += yu;
            }
        }
        if (in) {
            p.start[g] = s;
            p.start[g + 1] = s + req;
            p.len[g] = len;
            p.woff[g] = w + wi - work;
            p.uoff[g] = u + ui - units;
            if (g == a.groups - 1) {
                p.woff[a.groups] = w + wi;
                p.uoff[a.groups] = u + ui;
            }
        }
        before = __shfl_sync(0xffffffffu, s + req, 31);
        w += __shfl_sync(0xffffffffu, wi, 31);
        u += __shfl_sync(0xffffffffu, ui, 31);
        __syncwarp();
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

// ---------------------------------------------------------------- prefix attention
constexpr int kPrefixWarps = 16;

struct PrefixSmem {
    uint4 k[kTileKeys * 16];                        // [key][16 chunks of 8 dims], chunk ^ (key & 7)
    uint4 v[kTileKeys * 16];
    GroupPlan plan;
    unsigned long long valid;                       // keys of the tile that count
};

__global__ void __launch_bounds__(kPrefixWarps * 32, 1) k_prefix(const PrefixArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    PrefixSmem &sm = *reinterpret_cast<PrefixSmem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    if (warp == 0) plan_groups(a, sm.plan);
    __syncthreads();
    const GroupPlan &p = sm.plan;
    const int W = p.woff[a.groups], n = min(static_cast<int>(gridDim.x), W), b = blockIdx.x;
    if (b >= n) return;
    int w = share_lo(b, W, n);
    const int w1 = share_lo(b + 1, W, n);
    int g = 0;
    while (w < w1) {
        while (p.woff[g + 1] <= w) ++g;
        const int req = p.start[g + 1] - p.start[g], rt = rtiles_of(req), tiles = tiles_of(p.len[g]);
        const int ug = (w - p.woff[g]) / tiles, t0 = (w - p.woff[g]) % tiles;
        const int t1 = min(tiles, t0 + w1 - w);
        const int j = ug / rt, row0 = (ug % rt) * kUnitRows, rows = min(kUnitRows, req * kGroup - row0);
        float *part = a.partials + static_cast<size_t>(b + p.uoff[g] + ug) * 2 * kPrefixPart;
        const bool mine = warp * 16 < rows;
        // this lane's two rows of the warp's 16, clamped to the last valid row
        const int ra = warp * 16 + (lane >> 2), rb = ra + 8;
        uint32_t aq[8][4];
        if (mine) {
            auto qrow = [&](int r) {
                r = min(r, rows - 1) + row0;
                return static_cast<const uint16_t *>(a.q) +
                       (static_cast<size_t>(p.start[g] + r / kGroup) * a.hq + j * kGroup + r % kGroup) * kHeadDim +
                       2 * (lane & 3);
            };
            const uint16_t *qa = qrow(ra), *qb = qrow(rb);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                aq[ks][0] = *reinterpret_cast<const uint32_t *>(qa + ks * 16);
                aq[ks][1] = *reinterpret_cast<const uint32_t *>(qb + ks * 16);
                aq[ks][2] = *reinterpret_cast<const uint32_t *>(qa + ks * 16 + 8);
                aq[ks][3] = *reinterpret_cast<const uint32_t *>(qb + ks * 16 + 8);
            }
        }
        float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
        for (int t = t0; t < t1; ++t) {
            __syncthreads();                                     // the previous tile is consumed
            if (tid == 0) sm.valid = 0ull;
            __syncthreads();
            for (int e = tid; e < kTileKeys * 16; e += kPrefixWarps * 32) {
                const int key = e >> 4, ch = e & 15, tok = t * kTileKeys + key;
                const int pid = tok < p.len[g] ? a.prefix_table[static_cast<size_t>(g) * a.prefix_pages + tok / kPageSize]
                                               : 0;
                const bool ok = tok < p.len[g] && pid >= 0 && pid < a.num_pages;
                if (tok < p.len[g] && !ok && ch == 0) raise_status(a.status, kDevBadPage);
                uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
                if (ok) {
                    const size_t off = ((static_cast<size_t>(pid) * a.hkv + j) * kPageSize + tok % kPageSize) * 16 + ch;
                    kv = reinterpret_cast<const uint4 *>(a.k_pool)[off];
                    vv = reinterpret_cast<const uint4 *>(a.v_pool)[off];
                    if (ch == 0) atomicOr(&sm.valid, 1ull << key);
                }
                sm.k[key * 16 + (ch ^ (key & 7))] = kv;
                sm.v[key * 16 + (ch ^ (key & 7))] = vv;
            }
            __syncthreads();
            if (!mine) continue;
            const unsigned long long valid = sm.valid;
            float s[8][4];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                const int key = nt * 8 + (lane & 7);
#pragma unroll
                for (int ks = 0; ks < 8; ks += 2) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(smem_u32(&sm.k[key * 16 + ((2 * ks + (lane >> 3)) ^ (key & 7))]), b0, b1, b2, b3);
                    mma_bf16_16816(s[nt], aq[ks][0], aq[ks][1], aq[ks][2], aq[ks][3], b0, b1);
                    mma_bf16_16816(s[nt], aq[ks + 1][0], aq[ks + 1][1], aq[ks + 1][2], aq[ks + 1][3], b2, b3);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int kk = nt * 8 + 2 * (lane & 3) + (x & 1);
                    s[nt][x] = (valid >> kk & 1ull) ? s[nt][x] * a.scale_log2 : -INFINITY;
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = m[r];
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mu = mx == -INFINITY ? 0.f : mx, al = exp2f(m[r] - mu);
                m[r] = mx;
                l[r] *= al;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    o[x][2 * r] *= al;
                    o[x][2 * r + 1] *= al;
                }
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                    s[nt][2 * r] = exp2f(s[nt][2 * r] - mu);
                    s[nt][2 * r + 1] = exp2f(s[nt][2 * r + 1] - mu);
                    l[r] += s[nt][2 * r] + s[nt][2 * r + 1];
                }
            }
            // P enters as bf16 and its bf16 residual (16 significant bits)
#pragma unroll
            for (int kc = 0; kc < 4; ++kc) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p0 = s[2 * kc + (x >> 1)][2 * (x & 1)], p1 = s[2 * kc + (x >> 1)][2 * (x & 1) + 1];
                    const uint32_t h0 = f32_to_bf16_rne(p0), h1 = f32_to_bf16_rne(p1);
                    hi[x] = h0 | (h1 << 16);
                    lo[x] = f32_to_bf16_rne(p0 - __uint_as_float(h0 << 16)) |
                            (f32_to_bf16_rne(p1 - __uint_as_float(h1 << 16)) << 16);
                }
#pragma unroll
                for (int dt = 0; dt < 16; dt += 2) {
                    const int key = kc * 16 + (lane & 15), ch = dt + (lane >> 4);
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_trans(smem_u32(&sm.v[key * 16 + (ch ^ (key & 7))]), b0, b1, b2, b3);
                    mma_bf16_16816(o[dt], hi[0], hi[1], hi[2], hi[3], b0, b1);
                    mma_bf16_16816(o[dt], lo[0], lo[1], lo[2], lo[3], b0, b1);
                    mma_bf16_16816(o[dt + 1], hi[0], hi[1], hi[2], hi[3], b2, b3);
                    mma_bf16_16816(o[dt + 1], lo[0], lo[1], lo[2], lo[3], b2, b3);
                }
            }
        }
        if (mine) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                const int row = r ? rb : ra;
                if (row >= rows) continue;
                float *pp = part + (row / kStreamRows) * kPrefixPart;
                const int rr = row % kStreamRows;
#pragma unroll
                for (int dt = 0; dt < 16; ++dt) {
                    const int d = dt * 8 + 2 * (lane & 3);
                    *reinterpret_cast<float2 *>(pp + ((d >> 2) * kStreamRows + rr) * 4 + (d & 3)) =
                        make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
                }
                if ((lane & 3) == 0) {
                    pp[kStreamRows * kHeadDim + rr] = m[r];
                    pp[kStreamRows * kHeadDim + kStreamRows + rr] = l[r];
                }
            }
        }
        w += t1 - t0;
    }
}

int prefix_blocks(int sms) { return sms; }

cudaError_t launch_prefix(const PrefixArgs &a, cudaStream_t stream)
{
    static std::atomic<int> seen[64];
    const size_t smem = sizeof(PrefixSmem) + 128;
    const cudaError_t e = raise_smem_limit(k_prefix, smem, seen);
    if (e != cudaSuccess) return e;
    k_prefix<<<a.blocks, kPrefixWarps * 32, smem, stream>>>(a);
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
    int g = 0;
    while (g < a.groups && !(p.start[g] <= r && r < p.start[g + 1])) ++g;
    if (g == a.groups || p.len[g] == 0) return;                  // no prefix: the own part is the result
    const int W = p.woff[a.groups], n = min(a.blocks, W);
    const int h = threadIdx.x >> 5, d4 = threadIdx.x & 31;
    const int req = p.start[g + 1] - p.start[g], rt = rtiles_of(req), tiles = tiles_of(p.len[g]);
    const int row = (r - p.start[g]) * kGroup + h;
    const int ug = j * rt + row / kUnitRows, in = row % kUnitRows;
    const int w0 = p.woff[g] + ug * tiles;
    const int b0 = share_of(w0, W, n), b1 = share_of(w0 + tiles - 1, W, n);
    const float *part = a.partials + static_cast<size_t>(p.uoff[g] + ug) * 2 * kPrefixPart +
                        (in / kStreamRows) * kPrefixPart;
    const int rr = in % kStreamRows;
    const size_t at = static_cast<size_t>(r) * a.hq + j * kGroup + h;
    float4 *outp = reinterpret_cast<float4 *>(a.out + at * kHeadDim) + d4;
    float m = a.lse[at], l = m == -INFINITY ? 0.f : 1.f;         // the own part: normalised, weight 2^lse
    float4 o = *outp;
    __syncwarp();
    for (int b = b0; b <= b1; ++b) {
        const float *pp = part + static_cast<size_t>(b) * 2 * kPrefixPart;
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
