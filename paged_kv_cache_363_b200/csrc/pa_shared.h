// Launch interface of pa_decode_shared (pa_shared.cu).
#pragma once

#include "pa_group.cuh"
#include "pa_internal.h"

namespace pa {

struct SharedArgs {
    GroupArgs g;               // the shared tokens' kernel and the merge
    DecodeArgs d;              // the own tokens' kernel; plan_list has uint4 entries
    const int32_t* group_rows;
    const int32_t* group_start;
    const int32_t* shared_lens;
    void* row_info;            // [S] 16 bytes: what the plan says about a row
    int* listed;               // [S] times a row is listed (this and the next three: batches over 1024 rows)
    int* ctx;                  // [S] context length
    int* lead_blocks;          // [S] shared blocks of a row
    int* lead_states;          // [S] partial states of its shared tokens
    int* group_ok;             // [groups]
    int num_groups;
    int num_group_rows;
    int max_shared_len;
    int max_chunks;
    int wait_first;            // the finish has to wait for the plan itself before it begins
};

// Own tokens that the finish reads itself: up to eight steps of its four warps.  Longer rows are
// split into partitions that several CTAs share.
constexpr int kDirectTokens = 512;

// Own tokens per partition at least: 512, doubled until a row has at most 16 partitions (a
// partial state per partition is kept for every row) or a partition is as long as it may be.
inline int shared_partition(int64_t max_context)
{
    int p = 512;
    while (p < kMaxPartitionTokens && (max_context + p - 1) / p > 16) p *= 2;
    return p;
}

// Rows of a tile: 64 where the groups have that many rows or fewer on average (half the shared
// memory for Q, and more of it for K and V), else 128.
inline int shared_tile_rows(int64_t groups, int64_t rows, int group)
{
    return rows * group <= 64 * groups ? 64 : 128;
}

struct SharedWorkspace {
    GroupWorkspace g;
    size_t entries, plan, list, row_info, listed, ctx, lead_blocks, lead_states, group_ok, acc, ml, total;
    int chunks, parts;
};

inline SharedWorkspace shared_workspace(size_t S, size_t Hq, int Hkv, int D, int max_context, int max_shared,
                                        size_t groups, size_t rows)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    SharedWorkspace w{};
    const int G = (int)(Hq / (size_t)Hkv);
    const int P = shared_partition(max_context);
    w.chunks = group_max_chunks(max_shared, (int64_t)rows, G, Hkv);
    w.parts = max_context > 0 ? (max_context + P - 1) / P : 1;
    w.entries = max_shared > 0 && rows > 0 ? (groups + rows / (size_t)(shared_tile_rows((int64_t)groups, (int64_t)rows, G) / G)) * (size_t)w.chunks : 0;
    w.g = group_workspace(0, w.entries, 0);
    w.plan = w.g.end;
    w.list = w.plan + 256;
    w.row_info = up(w.list + 16 * S * (size_t)w.parts);
    w.listed = up(w.row_info + 16 * S);
    w.ctx = up(w.listed + 4 * S);
    w.lead_blocks = up(w.ctx + 4 * S);
    w.lead_states = up(w.lead_blocks + 4 * S);
    w.group_ok = up(w.lead_states + 4 * S);
    w.acc = up(w.group_ok + 4 * groups);
    const size_t states = S * Hq * (size_t)(w.chunks + w.parts);
    w.ml = up(w.acc + states * (size_t)D * 4);
    w.total = up(w.ml + states * 8);
    return w;
}

cudaError_t launch_shared(const SharedArgs& a, int head_dim, int block_size, int group, cudaStream_t stream);

}  // namespace pa
