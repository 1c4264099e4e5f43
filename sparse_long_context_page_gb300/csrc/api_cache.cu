// C ABI of the cache operators: attention of requests that share a prefix,
// attention that accumulates the cached tokens' weights, and eviction by them.
// Host-side argument checks, workspace carving and kernel launches; nothing
// here allocates, synchronises or reads device memory.
#include "../../include/moira.h"
#include "checks.h"
#include "moira_device.cuh"
#include "moira_launch.h"

using namespace moira;

namespace {

moira_status check_groups(int32_t groups, int32_t prefix_pages)
{
    if (groups < 0) return MOIRA_EINVAL;
    if (groups > kMaxGroups) return MOIRA_EUNSUPPORTED;
    if (groups == 0) return MOIRA_OK;
    if (prefix_pages <= 0) return MOIRA_EINVAL;
    return prefix_pages > kMaxPagesPerSeq ? MOIRA_EUNSUPPORTED : MOIRA_OK;
}

SharedLayout shared_layout_for(const moira_shape *s, int32_t batch, int32_t max_pages, int32_t groups, bool weights)
{
    return shared_layout(batch, s->num_q_heads, max_pages, attend_blocks(), groups, weights, current_sm_count());
}

bool ws_ok(const void *ws, size_t bytes, size_t need)
{
    return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && bytes >= need;
}

float log2_scale(float sm_scale) { return static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634); }

moira_status attend_shared_impl(const moira_shape *shape, const void *q, const void *k_pool, const void *v_pool,
                                const int32_t *prefix_table, const int32_t *prefix_lens,
                                const int32_t *group_starts, int32_t groups, int32_t prefix_pages,
                                const int32_t *lists, const int32_t *lengths, const int32_t *seq_lens,
                                int32_t batch, int32_t max_pages, float sm_scale, float *weights, float *out,
                                void *workspace, size_t ws_bytes, cudaStream_t stream)
{
    moira_status st = check_shape(shape);
    if (st != MOIRA_OK) return st;
    if ((st = check_batch(shape, batch, max_pages)) != MOIRA_OK) return st;
    if ((st = check_groups(groups, prefix_pages)) != MOIRA_OK) return st;
    if (!finite_pos(sm_scale)) return MOIRA_EINVAL;
    if (!q || !k_pool || !v_pool || !lists || !lengths || !seq_lens || !out) return MOIRA_EINVAL;
    if (groups > 0 && (!prefix_table || !prefix_lens || !group_starts)) return MOIRA_EINVAL;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned16(weights))
        return MOIRA_EINVAL;
    const SharedLayout L = shared_layout_for(shape, batch, max_pages, groups, weights != nullptr);
    if (!ws_ok(workspace, ws_bytes, L.total)) return MOIRA_EWORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    CUtensorMap mk, mv;
    if (!make_pool_map(&mk, k_pool, shape) || !make_pool_map(&mv, v_pool, shape)) return MOIRA_ECUDA;
    SharedArgs a = {};
    a.q = q;
    a.v_pool = v_pool;
    a.prefix_table = prefix_table;
    a.prefix_lens = prefix_lens;
    a.group_starts = group_starts;
    a.lists = lists;
    a.lengths = lengths;
    a.seq_lens = seq_lens;
    a.offsets = reinterpret_cast<int32_t *>(w + L.offsets);
    a.own = reinterpret_cast<float *>(w + L.own);
    a.logits = weights ? reinterpret_cast<float *>(w + L.logits) : nullptr;
    a.plan = w + L.plan;
    a.prefix = reinterpret_cast<float *>(w + L.prefix);
    a.weights = weights;
    a.out = out;
    a.status = reinterpret_cast<uint32_t *>(w + L.base.status);
    a.groups = groups;
    a.prefix_pages = prefix_pages;
    a.batch = batch;
    a.hq = shape->num_q_heads;
    a.hkv = shape->num_kv_heads;
    a.units = batch * shape->num_kv_heads;
    a.max_pages = max_pages;
    a.blocks = current_sm_count();
    a.num_pages = shape->num_phys_pages;
    a.scale_log2 = log2_scale(sm_scale);
    if (launch_own(mk, mv, a, stream) != cudaSuccess) return MOIRA_ECUDA;
    if (groups > 0 && launch_prefix(mk, mv, a, stream) != cudaSuccess) return MOIRA_ECUDA;
    return launch_finish(a, stream) == cudaSuccess ? MOIRA_OK : MOIRA_ECUDA;
}

}  // namespace

extern "C" {

size_t moira_shared_workspace_bytes(const moira_shape *shape, int32_t batch, int32_t max_pages, int32_t groups,
                                    int32_t with_weights)
{
    if (check_shape(shape) != MOIRA_OK || check_batch(shape, batch, max_pages) != MOIRA_OK) return 0;
    if (check_groups(groups, 1) != MOIRA_OK || attend_blocks() <= 0) return 0;
    return shared_layout_for(shape, batch, max_pages, groups, with_weights != 0).total;
}

moira_status moira_attend_shared(const moira_shape *shape, const void *q, const void *k_pool, const void *v_pool,
                                 const int32_t *prefix_table, const int32_t *prefix_lens,
                                 const int32_t *group_starts, int32_t groups, int32_t prefix_pages,
                                 const int32_t *lists, const int32_t *lengths, const int32_t *seq_lens,
                                 int32_t batch, int32_t max_pages, float sm_scale, float *weights, float *out,
                                 void *workspace, size_t ws_bytes, moira_stream_t stream)
{
    return attend_shared_impl(shape, q, k_pool, v_pool, prefix_table, prefix_lens, group_starts, groups, prefix_pages,
                              lists, lengths, seq_lens, batch, max_pages, sm_scale, weights, out, workspace, ws_bytes,
                              reinterpret_cast<cudaStream_t>(stream));
}

moira_status moira_attend_weights(const moira_shape *shape, const void *q, const void *k_pool, const void *v_pool,
                                  const int32_t *lists, const int32_t *lengths, const int32_t *seq_lens,
                                  int32_t batch, int32_t max_pages, float sm_scale, float *weights, float *out,
                                  void *workspace, size_t ws_bytes, moira_stream_t stream)
{
    if (!weights) return MOIRA_EINVAL;
    return attend_shared_impl(shape, q, k_pool, v_pool, nullptr, nullptr, nullptr, 0, 0, lists, lengths, seq_lens,
                              batch, max_pages, sm_scale, weights, out, workspace, ws_bytes,
                              reinterpret_cast<cudaStream_t>(stream));
}

size_t moira_evict_workspace_bytes(const moira_shape *shape, int32_t batch, int32_t max_pages)
{
    if (check_shape(shape) != MOIRA_OK || check_batch(shape, batch, max_pages) != MOIRA_OK) return 0;
    return evict_layout(batch * shape->num_kv_heads, max_pages).total;
}

moira_status moira_evict(const moira_shape *shape, int32_t format, void *k_pool, void *v_pool, void *summ,
                         float *weights, int32_t *positions, const int32_t *page_table, const int32_t *seq_lens,
                         int32_t batch, int32_t max_pages, int32_t budget, int32_t sinks, int32_t recent,
                         int32_t *new_lens, void *workspace, size_t ws_bytes, moira_stream_t stream)
{
    moira_status st = check_shape(shape);
    if (st != MOIRA_OK) return st;
    if ((st = check_batch(shape, batch, max_pages)) != MOIRA_OK) return st;
    if (!valid_format(format)) return MOIRA_EINVAL;
    if (budget <= 0 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks) return MOIRA_EINVAL;
    if (!k_pool || !v_pool || !weights || !positions || !page_table || !seq_lens || !new_lens) return MOIRA_EINVAL;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(summ) || !aligned16(weights) || !aligned16(positions))
        return MOIRA_EINVAL;
    const EvictLayout L = evict_layout(batch * shape->num_kv_heads, max_pages);
    if (!ws_ok(workspace, ws_bytes, L.total)) return MOIRA_EWORKSPACE;
    const int sms = current_sm_count();
    if (sms <= 0) return MOIRA_ECUDA;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    EvictArgs a;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.summ = summ;
    a.weights = weights;
    a.positions = positions;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.arrived = reinterpret_cast<uint32_t *>(w + L.arrived);
    a.counts = reinterpret_cast<int2 *>(w + L.counts);
    a.dst = reinterpret_cast<int32_t *>(w + L.dst);
    a.src = reinterpret_cast<int4 *>(w + L.src);
    a.status = reinterpret_cast<uint32_t *>(w + L.status);
    a.fmt = format;
    a.batch = batch;
    a.hkv = shape->num_kv_heads;
    a.max_pages = max_pages;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.num_pages = shape->num_phys_pages;
    return launch_evict(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOIRA_OK : MOIRA_ECUDA;
}

}  // extern "C"
