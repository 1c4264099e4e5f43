// What the token operators (rotate.cu, chunk.cu) need of the device beside
// moira_device.cuh: the workspace of the attention of a chunk, copies of 3-D and
// 4-D tensors, pieces of 16 columns of the tensor memory.
#pragma once

#include "moira_device.cuh"

namespace moira {

// ---- workspace of the attention of a chunk of tokens -----------------------------
// What starts at zero as in ws_layout (the status word and the counters are
// used), then, where ws_layout's scratch begins,
// records                     : int4 [2 * blocks]               split tiles, see chunk.cu
// partials                    : fp32 [2 * blocks][kChunkPart]
constexpr int kChunkTokens = 64;                    // rows of q of one tile: 256 query rows of a KV head
constexpr int kChunkRows = kChunkTokens * kGroup;
// one partial: o [d / 4][row] float4, then m [row], l [row]
constexpr int kChunkPart = kChunkRows * kHeadDim + 2 * kChunkRows;

struct ChunkLayout {
    size_t status, counters, records, partials, total;
};

__host__ __device__ inline ChunkLayout chunk_layout(int attend_blocks, int blocks)
{
    ChunkLayout c;
    const WsLayout base = ws_layout(1, kGroup, 1, 1, attend_blocks);
    c.status = base.status;
    c.counters = base.counters;
    size_t o = base.scores;
    c.records = o;  o = align_up(o + sizeof(int4) * 2 * (size_t)blocks, 256);
    c.partials = o; o = align_up(o + sizeof(float) * kChunkPart * 2 * (size_t)blocks, 256);
    c.total = o;
    return c;
}

// ---- instructions ----------------------------------------------------------------
// tma_load_2d of a 3-D tensor.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// The same of a 4-D tensor.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Ask for the line that holds `p` in L2.
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 16 columns of the tensor memory, a lane a row.
#define MOIRA_X16(c, r) c((r)[0]), c((r)[1]), c((r)[2]), c((r)[3]), c((r)[4]), c((r)[5]), c((r)[6]), c((r)[7]), c((r)[8]), \
                        c((r)[9]), c((r)[10]), c((r)[11]), c((r)[12]), c((r)[13]), c((r)[14]), c((r)[15])
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : MOIRA_X16("=r", r)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::MOIRA_X16("r", r), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : MOIRA_X16("+r", r)::"memory");
}
#undef MOIRA_X16

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace moira
