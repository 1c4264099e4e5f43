// C ABI of the operators that fill the cache and attend to it with many tokens
// a request: norm and rotation, the append of rotated tokens, the attention of
// a chunk.  Host-side argument checks, workspace carving and kernel launches;
// nothing here allocates, synchronises or reads device memory.
#include <cmath>
#include <cstring>

#include "../../include/moira.h"
#include "checks.h"
#include "rotary_core.cuh"
#include "token_device.cuh"
#include "token_launch.h"

using namespace moira;

namespace {

static_assert(MOIRA_MAX_PAIRS == kMaxPairs && MOIRA_MAX_AXES == kMaxAxes, "public limits match the kernels'");

// The kernels' copy of a rotary; false where a field is out of range.
bool rotary_args(RotaryArgs &r, const moira_rotary *rotary)
{
    std::memset(&r, 0, sizeof r);
    r.scale = 1.f;
    if (!rotary) return true;
    if (rotary->pairs < 0 || rotary->pairs > kMaxPairs || rotary->pairs % 4 != 0) return false;
    if (rotary->axes < 1 || rotary->axes > kMaxAxes || !std::isfinite(rotary->scale)) return false;
    for (int i = 0; i < rotary->pairs; ++i)
        if (rotary->axis[i] >= rotary->axes) return false;
    r.pairs = rotary->pairs;
    r.interleaved = rotary->interleaved != 0;
    r.scale = rotary->scale;
    std::memcpy(r.turns, rotary->turns, sizeof r.turns);
    std::memcpy(r.axis, rotary->axis, sizeof r.axis);
    return true;
}

// Token rows of `heads` heads: 16-byte aligned, rows that do not overlap.
bool rows_ok(const void *p, int64_t stride, int heads)
{
    return p && aligned16(p) && stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * kHeadDim;
}

// Whether dense rows `out` of `tokens` tokens hold no byte of as many rows `in`,
// `stride` elements apart.  Blocks write their rows of one while others still
// read theirs of the other.
bool rows_apart(const void *in, int64_t stride, int in_heads, const void *out, int out_heads, int32_t tokens)
{
    const int64_t row = 2 * static_cast<int64_t>(in_heads) * kHeadDim, len = 2 * static_cast<int64_t>(out_heads) * kHeadDim * tokens;
    const int64_t from = static_cast<int64_t>(reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(in));
    const int64_t i = from < row ? 0 : (from - row) / (2 * stride) + 1;      // the first row of `in` that ends behind out's begin
    return i >= tokens || 2 * stride * i >= from + len;
}

// The same rows, or none of their memory.
bool same_or_apart(const void *in, int64_t stride, const void *out, int heads, int32_t tokens)
{
    if (in == out) return stride == static_cast<int64_t>(heads) * kHeadDim || tokens == 1;
    return rows_apart(in, stride, heads, out, heads, tokens);
}

bool eps_ok(float eps) { return std::isfinite(eps) && eps >= 0.f; }

moira_status status_of(cudaError_t e) { return e == cudaSuccess ? MOIRA_OK : MOIRA_ECUDA; }

}  // namespace

extern "C" {

moira_status moira_make_rotary(moira_rotary *rotary, const double *inv_freq, const int32_t *axis, int32_t pairs,
                               int32_t axes, int32_t interleaved, float scale)
{
    if (!rotary || !inv_freq || pairs <= 0 || pairs > kMaxPairs || pairs % 4 != 0) return MOIRA_EINVAL;
    if (axes < 1 || axes > kMaxAxes || !std::isfinite(scale)) return MOIRA_EINVAL;
    for (int i = 0; i < pairs; ++i)
        if (!(std::fabs(inv_freq[i]) <= 0x1p20) || (axis && (axis[i] < 0 || axis[i] >= axes))) return MOIRA_EINVAL;
    std::memset(rotary, 0, sizeof *rotary);
    rotary->pairs = pairs;
    rotary->axes = axes;
    rotary->interleaved = interleaved != 0;
    rotary->scale = scale;
    // 1 / 2 pi in two doubles: the product keeps 2^-64 of a turn
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    for (int i = 0; i < pairs; ++i) {
        const double f = std::fabs(inv_freq[i]);
        const double hi = f * kHi, lo = std::fma(f, kHi, -hi) + f * kLo;
        const double part = std::ldexp(hi - std::floor(hi), 64);     // exact, [0, 2^64)
        const uint64_t u = static_cast<uint64_t>(part) + static_cast<uint64_t>(std::llrint(std::ldexp(lo, 64)));
        rotary->turns[i] = inv_freq[i] < 0.0 ? 0u - u : u;
        rotary->axis[i] = static_cast<uint8_t>(axis ? axis[i] : 0);
    }
    return MOIRA_OK;
}

moira_status moira_rotate_qk(const moira_shape *shape, const moira_rotary *rotary, const void *q, int64_t q_stride,
                             const void *k, int64_t k_stride, const float *q_norm, const float *k_norm, float eps,
                             const int32_t *positions, int32_t tokens, void *q_out, void *k_out,
                             moira_stream_t stream)
{
    moira_status st = check_shape(shape);
    if (st != MOIRA_OK) return st;
    RotaryArgs rot;
    if (!rotary_args(rot, rotary) || !eps_ok(eps) || tokens < 0) return MOIRA_EINVAL;
    if (tokens == 0) return MOIRA_OK;
    if ((!q && !k) || (rot.pairs && !positions)) return MOIRA_EINVAL;
    if (q && (!rows_ok(q, q_stride, shape->num_q_heads) || !q_out || !aligned16(q_out))) return MOIRA_EINVAL;
    if (k && (!rows_ok(k, k_stride, shape->num_kv_heads) || !k_out || !aligned16(k_out))) return MOIRA_EINVAL;
    if (q && !same_or_apart(q, q_stride, q_out, shape->num_q_heads, tokens)) return MOIRA_EINVAL;
    if (k && !same_or_apart(k, k_stride, k_out, shape->num_kv_heads, tokens)) return MOIRA_EINVAL;
    if (q && k) {
        const int hq = shape->num_q_heads, hkv = shape->num_kv_heads;
        if (!rows_apart(k, k_stride, hkv, q_out, hq, tokens) || !rows_apart(q, q_stride, hq, k_out, hkv, tokens) ||
            !rows_apart(q_out, static_cast<int64_t>(hq) * kHeadDim, hq, k_out, hkv, tokens))
            return MOIRA_EINVAL;
    }
    if (!aligned16(q_norm) || !aligned16(k_norm)) return MOIRA_EINVAL;
    RotateArgs a = {};
    a.q = {q, q_out, q_norm, q_stride};
    a.k = {k, k_out, k_norm, k_stride};
    a.positions = positions;
    a.eps = eps;
    a.tokens = tokens;
    a.hq = shape->num_q_heads;
    a.hkv = shape->num_kv_heads;
    const int sms = current_sm_count();
    if (sms <= 0) return MOIRA_ECUDA;
    return status_of(launch_rotate(rot, a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moira_status moira_append_rotated(const moira_shape *shape, int32_t format, const moira_rotary *rotary, const void *q,
                                  int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                  const float *q_norm, const float *k_norm, float eps, const int32_t *positions,
                                  const int32_t *token_starts, int32_t tokens, void *k_pool, void *v_pool, void *summ,
                                  const int32_t *page_table, const int32_t *seq_lens, int32_t batch,
                                  int32_t max_pages, void *q_out, moira_stream_t stream)
{
    moira_status st = check_shape(shape);
    if (st != MOIRA_OK) return st;
    if ((st = check_batch(shape, batch, max_pages)) != MOIRA_OK) return st;
    RotaryArgs rot;
    if (!valid_format(format) || !rotary_args(rot, rotary) || !eps_ok(eps) || tokens < 0) return MOIRA_EINVAL;
    if (tokens == 0) return MOIRA_OK;
    if (!token_starts || !k_pool || !v_pool || !page_table || !seq_lens) return MOIRA_EINVAL;
    if (!rows_ok(k, k_stride, shape->num_kv_heads) || !rows_ok(v, v_stride, shape->num_kv_heads)) return MOIRA_EINVAL;
    if (q && (!rows_ok(q, q_stride, shape->num_q_heads) || !q_out || !aligned16(q_out))) return MOIRA_EINVAL;
    if (q && (!same_or_apart(q, q_stride, q_out, shape->num_q_heads, tokens) ||
              !rows_apart(k, k_stride, shape->num_kv_heads, q_out, shape->num_q_heads, tokens) ||
              !rows_apart(v, v_stride, shape->num_kv_heads, q_out, shape->num_q_heads, tokens)))
        return MOIRA_EINVAL;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(summ) || !aligned16(q_norm) || !aligned16(k_norm))
        return MOIRA_EINVAL;
    AppendArgs a = {};
    a.q = {q, q_out, q_norm, q_stride};
    a.k = {k, nullptr, k_norm, k_stride};
    a.v = v;
    a.v_stride = v_stride;
    a.positions = positions;
    a.token_starts = token_starts;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.summ = summ;
    a.eps = eps;
    a.tokens = tokens;
    a.batch = batch;
    a.hkv = shape->num_kv_heads;
    a.max_pages = max_pages;
    a.num_pages = shape->num_phys_pages;
    const int sms = current_sm_count();
    if (sms <= 0) return MOIRA_ECUDA;
    return status_of(launch_append_rotated(rot, a, format, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moira_chunk_workspace_bytes(const moira_shape *shape, int32_t batch, int32_t max_pages, int32_t tokens)
{
    if (check_shape(shape) != MOIRA_OK || check_batch(shape, batch, max_pages) != MOIRA_OK || tokens <= 0) return 0;
    const int sms = current_sm_count();
    return sms <= 0 ? 0 : chunk_layout(attend_blocks(), sms).total;
}

moira_status moira_attend_chunk(const moira_shape *shape, const void *q, const void *k_pool, const void *v_pool,
                                const int32_t *page_table, const int32_t *seq_lens, const int32_t *token_starts,
                                int32_t batch, int32_t max_pages, int32_t tokens, int32_t causal, float sm_scale,
                                void *out, void *workspace, size_t ws_bytes, moira_stream_t stream)
{
    moira_status st = check_shape(shape);
    if (st != MOIRA_OK) return st;
    if ((st = check_batch(shape, batch, max_pages)) != MOIRA_OK) return st;
    if (!finite_pos(sm_scale) || tokens < 0) return MOIRA_EINVAL;
    if (tokens == 0) return MOIRA_OK;
    if (!q || !k_pool || !v_pool || !page_table || !seq_lens || !token_starts || !out) return MOIRA_EINVAL;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return MOIRA_EINVAL;
    if (q == out || !same_or_apart(q, static_cast<int64_t>(shape->num_q_heads) * kHeadDim, out, shape->num_q_heads, tokens)) return MOIRA_EINVAL;
    const int sms = current_sm_count();
    const ChunkLayout L = chunk_layout(attend_blocks(), sms);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < L.total) return MOIRA_EWORKSPACE;
    if (sms <= 0 || sms > kMaxUnits) return MOIRA_ECUDA;         // a counter a block
    uint8_t *w = static_cast<uint8_t *>(workspace);
    CUtensorMap mq, mk, mv;
    if (!make_query_map(&mq, q, tokens, kChunkTokens / 2, shape) || !make_page_map(&mk, k_pool, shape) ||
        !make_page_map(&mv, v_pool, shape))
        return MOIRA_ECUDA;
    ChunkArgs a = {};
    a.v_pool = v_pool;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.token_starts = token_starts;
    a.out = out;
    a.records = reinterpret_cast<int4 *>(w + L.records);
    a.partials = reinterpret_cast<float *>(w + L.partials);
    a.counters = reinterpret_cast<uint32_t *>(w + L.counters);
    a.status = reinterpret_cast<uint32_t *>(w + L.status);
    a.batch = batch;
    a.tokens = tokens;
    a.hkv = shape->num_kv_heads;
    a.max_pages = max_pages;
    a.causal = causal != 0;
    a.num_pages = shape->num_phys_pages;
    a.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
    return status_of(launch_chunk(mq, mk, mv, a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
