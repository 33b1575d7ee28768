// Launch interface of pa_decode_shared (pa_shared.cu).
#pragma once

#include <algorithm>

#include "pa_group.cuh"
#include "pa_internal.h"

namespace pa {

// Own tokens of one query row: all of them, or one of several parts.
struct OwnItem {
    int row;
    int tok0, ntok;
    int lead;         // partial states of the row's shared tokens
    int part, parts;
    int table_row;    // row of block_tables
    int pad;
};

struct SharedArgs {
    GroupArgs g;               // the shared tokens' kernel; counts: [0] its entries, [2] those of the own tokens
    const int32_t* context_lens;
    const int32_t* group_rows;
    const int32_t* group_start;
    const int32_t* shared_lens;
    OwnItem* own;              // [S * max_parts] rows' own tokens, in parts
    unsigned* arrived;         // [S * Hkv] parts of a row and kv head that are done
    int* listed;               // [S] times a row is listed (this and the next three: batches over 1024 rows)
    int* ctx;                  // [S] context length
    int* lead_blocks;          // [S] shared blocks of a row
    int* lead_states;          // [S] partial states of its shared tokens
    int* group_ok;             // [groups]
    int num_seqs;
    int num_groups;
    int num_group_rows;
    int max_context_len;
    int max_shared_len;
    int max_chunks;            // of the shared tokens
    int max_parts;             // of a row's own tokens
    int wait_first;            // the own tokens' kernel follows the plan itself
};

// Most parts of a row's own tokens (the workspace has a partial state per part of every row): as many as
// make four units per warp of the device (about 4,800), and where contexts are long, up to 32 of 1024
// tokens or more; none below 256 tokens.
inline int shared_max_parts(int64_t seqs, int64_t num_kv_heads, int64_t max_context)
{
    const int64_t want = (4800 + seqs * num_kv_heads - 1) / (seqs * num_kv_heads);
    const int64_t lengthy = std::min<int64_t>(32, (max_context + 1023) / 1024);
    return (int)std::max<int64_t>(1, std::min<int64_t>((max_context + 255) / 256, std::max(std::min<int64_t>(want, 32), lengthy)));
}

// Rows of a tile: 64 where the groups have that many rows or fewer on average (half the shared
// memory for Q, and more of it for K and V), else 128.
inline int shared_tile_rows(int64_t groups, int64_t rows, int group)
{
    return rows * group <= 64 * groups ? 64 : 128;
}

struct SharedWorkspace {
    GroupWorkspace g;
    size_t entries, own, arrived, listed, ctx, lead_blocks, lead_states, group_ok, acc, ml, total;
    int chunks, parts;
};

inline SharedWorkspace shared_workspace(size_t S, size_t Hq, int Hkv, int D, int max_context, int max_shared,
                                        size_t groups, size_t rows)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    SharedWorkspace w{};
    const int G = (int)(Hq / (size_t)Hkv);
    w.chunks = group_max_chunks(max_shared, (int64_t)rows, G, Hkv);
    w.parts = shared_max_parts((int64_t)S, Hkv, max_context);
    w.entries = max_shared > 0 && rows > 0 && groups > 0
                    ? (groups + rows / (size_t)(shared_tile_rows((int64_t)groups, (int64_t)rows, G) / G)) * (size_t)w.chunks
                    : 0;
    w.g = group_workspace(0, w.entries, 0);
    w.own = w.g.end;
    w.arrived = up(w.own + sizeof(OwnItem) * S * (size_t)w.parts);
    w.listed = up(w.arrived + 4 * S * (size_t)Hkv);
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

cudaError_t launch_shared(const SharedArgs& a, int head_dim, int group, cudaStream_t stream);

// pa_cross_attention with at most one query row per sequence: the own tokens' kernel alone.  Of `a`: g (lse
// too), context_lens, own, arrived, num_seqs, max_context_len, max_parts.
cudaError_t launch_cross_single(const SharedArgs& a, const int32_t* q_start, int num_query_tokens, int head_dim, int group,
                                cudaStream_t stream);

}  // namespace pa
