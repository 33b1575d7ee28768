// Attention of packed query rows to one block table each, without a mask: the tensor-core
// kernel that pa_cross_attention and the shared tokens of pa_decode_shared run on, its work
// entries, and the merge of a row's partial states.
#pragma once

#include <cstdint>

#include "pa_internal.h"

namespace pa {

// One entry: the members (query tokens) that share a 128-row tile, and the tokens they attend to.
struct GroupItem {
    int table_row;   // row of block_tables
    int row0;        // first member: an index into rows[] (or the query row itself when rows is null)
    int members;     // at most the launch's rows of a tile (64 or 128) / G
    int chunk;       // partial state this entry writes, or -1: it writes the output
    int kv0, kvlen;  // tokens [kv0, kv0 + kvlen); kv0 a multiple of 64
    int pad[2];
};

struct GroupArgs {
    void* out;                    // [rows][num_heads][D] bf16
    float* lse;                   // [rows][num_heads] or null
    const void* q;                // [rows][num_heads][D] bf16
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* rows;          // query row of each member, or null
    const GroupItem* items;
    const unsigned* counts;       // [0] entries, [1] rows to merge
    const uint2* merge_list;      // (row, its partial states)
    float* ws_acc;                // [rows][num_heads][num_partitions][D]
    float* ws_ml;                 // [rows][num_heads][num_partitions][2]
    unsigned int* status;
    int num_heads;
    int num_kv_heads;
    int max_blocks_per_seq;
    int num_blocks;
    int block_size;
    int num_partitions;           // partial states kept per (row, head)
    int lead_partitions;          // pa_decode_shared: of them, those of the shared tokens (the others follow)
    int max_entries;              // host bounds: entries, and rows to merge
    int max_merges;
    float scale_log2;
};

// Bytes of the entries, the merge list and the header, from a 256-byte aligned base.
struct GroupWorkspace {
    size_t header, items, merges, end;
};

inline GroupWorkspace group_workspace(size_t base, size_t max_entries, size_t max_merges)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    GroupWorkspace w{};
    w.header = base;
    w.items = base + 256;
    w.merges = up(w.items + max_entries * sizeof(GroupItem));
    w.end = up(w.merges + max_merges * sizeof(uint2));
    return w;
}

// Most chunks a table's tokens are split into: enough that about 1200 units exist (four per
// resident CTA) whatever the batch, chunks of 256 tokens or more, at most 32.
inline int group_max_chunks(int64_t max_len, int64_t rows, int group, int num_kv_heads)
{
    const int64_t by_len = (max_len + 255) / 256;
    const int64_t tiles = rows * group / 128 > 1 ? rows * group / 128 : 1;
    const int64_t want = (1200 + num_kv_heads * tiles - 1) / (num_kv_heads * tiles);
    int64_t n = by_len < want ? by_len : want;
    n = n < 1 ? 1 : n;
    return (int)(n < 32 ? n : 32);
}

#ifdef __CUDACC__
// The chunk length of a plan.  Split or not, from a few sums: `tiles` (tiles of rows x kv heads), `steps` (those
// x tiles of 64 tokens), the longest table, and the (row, head) pairs.  Unsplit, the time is the longest table's or the mean
// load's, at about 1 us a step; split into the mean load of a CTA (256 tokens at least), that load's and the
// partial states' (written and read at 5 TB/s), and 4 us where a split brings a merge with it.
// A chunk is long enough for the units to fit one round of the CTAs, where the tiles are few enough to tell (each ends
// in a part of a chunk, taken as 3/4); or, where the states are joined anyway, two rounds, if those are the shorter at
// three steps of overhead a unit.  155 rows on three documents of 23,000 to 32,000 tokens, 32 query heads on 8, the
// whole call: 202 us with half the mean load (608 units for 296 CTAs), 197 fitted to two rounds, 183 to one; 12 rows on
// each of 24 of 3,000: 85 fitted to two, 91 to one.
// (Splitting every batch into two units per CTA cost 16 sequences x 64 rows x 1500 tokens 90 us, 60 unsplit.)
__device__ __forceinline__ int plan_chunk(float steps, float tiles, int ctas, int longest, float pairs, int max_chunks, int D, bool merge_anyway)
{
    const float load = steps / (float)ctas;
    const int least = (longest + max_chunks - 1) / max_chunks;
    float fit = 64.f * load, best = 3e38f;
    for (int rounds = 1; rounds <= (merge_anyway ? 2 : 1); ++rounds) {
        const float units = (float)(rounds * ctas) - 0.75f * tiles;
        if (units < 0.5f * (float)(rounds * ctas)) continue;
        const float c = fmaxf(fmaxf(64.f * steps / units, (float)least), 256.f);
        const float cost = (float)rounds * ((float)longest / ceilf((float)longest / c) * (1.f / 64.f) + 3.f);
        if (cost < best) {
            best = cost;
            fit = c;
        }
    }
    const int c = (max(max((int)fminf(fit, 1e9f), least), 256) + 63) / 64 * 64;
    if (c >= longest) return max(longest, 1);
    const float whole = fmaxf((float)longest * (1.f / 64.f), load);
    const float states = pairs * ceilf((float)longest / (float)c);
    const float parts = fmaxf((float)c * (1.f / 64.f), load) + states * (float)D * (8.f / 5e6f) + (merge_anyway ? 0.f : 4.f);
    return whole <= parts ? longest : c;
}

// Weight of a partial state (m, l, O) in a join whose largest maximum is M.  NaN logits are no maximum, they show in
// the sum alone: a state without a maximum weighs nothing, unless its sum is NaN.
__device__ __forceinline__ float state_weight(float m, float l, float M)
{
    return m != -INFINITY ? exp2f(m - M) : (l == l ? 0.f : l);
}
// The natural log-sum-exp of a row: -inf without a sum, NaN where that is NaN.
__device__ __forceinline__ float row_lse(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Entries go longest first, by sixteenths of the chunk: a CTA's units then are one of every length.
constexpr int kLenClasses = 16;
__device__ __forceinline__ int len_class(int kvlen, int chunk)
{
    return kLenClasses - 1 - min(kLenClasses - 1, (int)((float)kvlen / (float)chunk * kLenClasses));
}
#endif

// CTAs of the kernel resident on the device at once.
int group_resident_ctas(int sms);

// The kernel over the entries a plan kernel (just launched on the stream) wrote, tiles of
// tile_rows rows, on at most `ctas` CTAs; and the merge of the rows the plan listed.
cudaError_t launch_group(const GroupArgs& a, int head_dim, int group, int tile_rows, int ctas, cudaStream_t stream);
cudaError_t launch_group_merge(const GroupArgs& a, int head_dim, cudaStream_t stream);

// pa_cross_attention: plan, kernel, merge.
struct CrossArgs {
    GroupArgs g;
    const int32_t* context_lens;
    const int32_t* q_start;
    int num_seqs;
    int num_query_tokens;
    int max_query_len;
    int max_context_len;
    int max_chunks;
};

cudaError_t launch_cross(const CrossArgs& a, int head_dim, int group, cudaStream_t stream);

}  // namespace pa
