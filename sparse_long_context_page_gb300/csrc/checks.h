// Host-side argument checks and launch plumbing shared by the C ABI's entry
// points (api.cu, api_cache.cu and noalloc.cu), so that every entry point
// rejects the same bad arguments the same way.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "../../include/moira.h"

namespace moira {

// Shape, batch and max_pages: MOIRA_EINVAL for nonsense, MOIRA_EUNSUPPORTED
// for sizes the kernels are not built for.
moira_status check_shape(const moira_shape *s);
moira_status check_batch(const moira_shape *s, int32_t batch, int32_t max_pages);

// Everything moira_select_ex checks except the workspace: the shape and
// batch as above, the summary format, the rule and its parameter, a finite
// positive sm_scale, non-null buffers, and q and the summaries on 16-byte
// boundaries.
moira_status check_select_args(const moira_shape *shape, int32_t fmt, const void *q, const void *summ,
                               const int32_t *page_table, const int32_t *seq_lens, int32_t batch,
                               int32_t max_pages, int32_t rule, float param, float sm_scale,
                               const int32_t *lists, const int32_t *lengths);

bool finite_pos(float x);
bool valid_format(int32_t fmt);
bool aligned16(const void *p);

int current_sm_count();                  // of the current device; 0 if it cannot be read
int attend_blocks();                     // the attention grid on the current device
// One layer's pool as the TMA tensor map that the attention kernels load from.
bool make_pool_map(CUtensorMap *map, const void *pool, const moira_shape *s);

}  // namespace moira
