// Arguments and launches of the token operators' kernels (rotate.cu, chunk.cu).
#pragma once

#include "moira_launch.h"

namespace moira {

// Norm and rotation of queries and keys, and the append of rotated tokens
// (rotate.cu).  `in` is bf16 [tokens][heads][d], a token's rows `stride`
// elements after the last one's; `out` is dense.
struct TokenRows {
    const void *in;                  // or null
    void *out;
    const float *norm;               // fp32 [d], or null
    long long stride;
};
struct RotateArgs {
    TokenRows q, k;
    const int32_t *positions;        // [axes][tokens]
    float eps;
    int tokens, hq, hkv;
    int rows;                        // of a block, set by the launch
};
struct AppendArgs {
    TokenRows q, k;                  // k.out is unused
    const void *v;
    long long v_stride;
    const int32_t *positions;        // [axes][tokens], or null: the token's index in its request
    const int32_t *token_starts;     // [batch + 1]
    const int32_t *page_table;
    const int32_t *seq_lens;
    void *k_pool;
    void *v_pool;
    void *summ;                      // or null
    float eps;
    int tokens, batch, hkv, max_pages;
    int rows, q_rows;                // of a block that writes pages and of one of queries, set by the launch
    long long num_pages;
};
struct RotaryArgs;
cudaError_t launch_rotate(const RotaryArgs &rot, RotateArgs args, int sms, cudaStream_t stream);
cudaError_t launch_append_rotated(const RotaryArgs &rot, AppendArgs args, int fmt, int sms, cudaStream_t stream);

// Attention of a chunk of tokens over the paged cache (chunk.cu).
struct ChunkArgs {
    const void *v_pool;
    const int32_t *page_table;       // [batch][max_pages]
    const int32_t *seq_lens;         // [batch]
    const int32_t *token_starts;     // [batch + 1]
    void *out;                       // bf16 [tokens][Hq][d]
    int4 *records;                   // [2 * blocks] split tiles: first row, rows, head, 0 none / 1 goes on / 2 ends
    float *partials;                 // [2 * blocks][kChunkPart]
    uint32_t *counters;              // [blocks] key tiles done of the split tile that a block begins, zero between calls
    uint32_t *status;
    int batch, tokens, hkv, max_pages, causal;
    long long num_pages;
    float scale_log2;
};
cudaError_t launch_chunk(const CUtensorMap &tmap_q, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                         ChunkArgs args, int blocks, cudaStream_t stream);

}  // namespace moira
