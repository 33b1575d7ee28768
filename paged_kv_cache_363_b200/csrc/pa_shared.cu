// Decode attention of a batch in groups whose sequences share leading blocks, for sm_100a.
//
// What it computes: pa_decode's output.  Row s of group g attends to the group's n_g shared
// tokens and to its own tokens n_g .. L_s - 1; the softmax over both is joined from the two
// partial states (m, l, O) = (maximum, sum of 2^(x - m), weighted V):
//   out = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p,  M = max m_p.
// The shared tokens of a kv head are one dense product of all the group's rows x G query
// heads with the same K and V: the tensor-core kernel of pa_group.cu reads each shared byte
// once per tile of rows, where pa_decode reads it once per sequence (from L2 when it is lucky).
//
// Three kernels: a plan, the shared tokens, and the own tokens with the join.  The last needs
// the plan alone to begin, so the shared tokens' kernel lets it start once it has itself seen
// the plan finish, and its CTAs fill the places that the other's leave.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pa_decode_mma.cuh"
#include "pa_group.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"
#include "pa_shared.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;

// Entry i, or one without tokens past the end.
__device__ __forceinline__ OwnItem load_own(const OwnItem* items, unsigned i, unsigned n)
{
    if (i >= n) return OwnItem{0, 0, 0, 0, 0, 1, 0, 0};
    const int4 x = __ldcg(reinterpret_cast<const int4*>(items + i)), y = __ldcg(reinterpret_cast<const int4*>(items + i) + 1);
    return OwnItem{x.x, x.y, x.z, x.w, y.x, y.y, y.z, 0};
}

// Half a warp's share of `tokens` own tokens, and the tokens of a row's parts (all the same but the last):
// at least that share and 256 (joining costs some 4 us: with 128, 16 rows on each of eight groups took 54 us for 46;
// with 512, 24 rows of 33 to 1500 tokens x 16 heads 30 for 26), and no more parts than the row has
// partial states for.
__device__ __forceinline__ int own_share(unsigned tokens, int rows, int num_kv_heads, int own_warps)
{
    const float units = (float)rows * (float)num_kv_heads, warps = (float)own_warps;
    return (int)fminf((float)tokens * (float)num_kv_heads / (3.f * units <= warps ? warps - 0.75f * units : 2.f * warps), 1e9f);
}
__device__ __forceinline__ int own_part(int own, int share, int max_parts)
{
    const int p0 = max(share, 256);
    if (own <= p0) return max(own, 1);
    const int p = (max(p0, (own + max_parts - 1) / max_parts) + 15) / 16 * 16;
    const int n = (own + p - 1) / p;
    return n <= 1 ? own : ((own + n - 1) / n + 15) / 16 * 16;
}

// The plan, in one CTA.
//  1. Groups are checked (starts in order, rows in range and listed once, whole blocks, no more
//     tokens than any member's context).  A bad one raises PA_DEV_BAD_CONTEXT and is not
//     shared: its rows attend to all their tokens on their own, which is the same result.
//  2. Entries of the shared tokens: (tile of rows, chunk), a chunk's tiles next to each other.
//  3. Entries of the own tokens: a row, or one of its parts, the longer half of the entries
//     first.
// A batch of up to 1024 rows keeps its per-row values in shared memory: the plan is on the
// critical path, and most of it was trips to L2.
__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_kernel(const SharedArgs a, int T, int D, int group_ctas, int own_warps)
{
    __shared__ int s_listed[kPlanThreads], s_ctx[kPlanThreads], s_lead[kPlanThreads], s_states[kPlanThreads];
    __shared__ int s_rows[kPlanThreads], s_start[kPlanThreads + 1], s_len[kPlanThreads], s_ok[kPlanThreads];
    __shared__ unsigned s_steps, s_tiles, s_members, s_own, s_class[kLenClasses];
    __shared__ unsigned s_items, s_big, s_front, s_back;
    __shared__ int s_bad, s_longest;
    pdl_launch_dependents();
    const int B = a.g.block_size, S = a.num_seqs, NG = a.num_groups, R = a.num_group_rows;
    const int bshift = B == 16 ? 4 : 5;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool small = S <= kPlanThreads && NG <= kPlanThreads;  // (R <= S)
    volatile int* listed = small ? s_listed : a.listed;
    volatile int* ctx = small ? s_ctx : a.ctx;
    volatile int* lead_blocks = small ? s_lead : a.lead_blocks;
    volatile int* lead_states = small ? s_states : a.lead_states;
    volatile int* group_ok = small ? s_ok : a.group_ok;
    const int* rows = small ? s_rows : a.group_rows;
    const int* start = small ? s_start : a.group_start;
    const int* lens = small ? s_len : a.shared_lens;
    if (tid == 0) {
        s_steps = s_tiles = s_members = s_own = 0;
        s_items = s_big = s_front = s_back = 0;
        s_bad = s_longest = 0;
    }
    if (tid < kLenClasses) s_class[tid] = 0;
    if (small) {
        // everything the plan reads, in one trip
        const int r = tid < R ? __ldg(a.group_rows + tid) : 0;
        const int n = tid < NG ? __ldg(a.shared_lens + tid) : 0;
        const int g0 = NG > 0 && tid <= NG ? __ldg(a.group_start + tid) : 0;
        if (tid < R) s_rows[tid] = r;
        if (tid < NG) s_len[tid] = n;
        if (tid <= NG) s_start[tid] = g0;
        if (tid == 0 && NG == kPlanThreads) s_start[NG] = __ldg(a.group_start + NG);
    }
    const int cap = min(a.max_context_len, table_tokens(a.g.max_blocks_per_seq, B));
    for (int s = tid; s < S; s += kPlanThreads) {
        int L = __ldg(a.context_lens + s);
        if (L < 0 || L > cap) {
            atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
            L = L < 0 ? 0 : cap;
        }
        listed[s] = 0;
        lead_blocks[s] = 0;
        lead_states[s] = 0;
        ctx[s] = L;
    }
    __syncthreads();
    for (int g = tid; g < NG; g += kPlanThreads) {
        const int r0 = start[g], r1 = start[g + 1];
        if (r0 < 0 || r1 < r0 || r1 > R) s_bad = 1;
    }
    for (int i = tid; i < R; i += kPlanThreads) {
        const int s = rows[i];
        if ((unsigned)s < (unsigned)S) atomicAdd(const_cast<int*>(listed) + s, 1);
    }
    __syncthreads();
    if (tid == 0 && s_bad) atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
    const int ngroups = s_bad ? 0 : NG;
    for (int g = warp; g < ngroups; g += kPlanThreads / 32) {
        const int r0 = start[g], r1 = start[g + 1], n = lens[g];
        bool ok = n >= 0 && n <= a.max_shared_len && (n & (B - 1)) == 0;
        for (int i = r0 + lane; i < r1; i += 32) {
            const int s = rows[i];
            ok = ok && (unsigned)s < (unsigned)S;
            ok = ok && listed[s] == 1 && n <= ctx[s];
        }
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (lane == 0) {
            group_ok[g] = ok && n > 0 && r1 > r0;
            if (!ok) atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
            else if (n > 0) {
                const unsigned tiles = (unsigned)((r1 - r0 + T - 1) / T);
                atomicAdd(&s_tiles, tiles);
                atomicAdd(&s_steps, tiles * (unsigned)((n + 63) / 64));
                atomicAdd(&s_members, (unsigned)(r1 - r0));
                atomicMax(&s_longest, n);
            }
        }
    }
    __syncthreads();
    if (s_steps > 0 && !a.wait_first) {
        const int chunk = plan_chunk((float)s_steps * (float)a.g.num_kv_heads, (float)s_tiles * (float)a.g.num_kv_heads,
                                     group_ctas, s_longest, (float)s_members * (float)a.g.num_heads, a.max_chunks, D, true);
        auto chunks_of = [&](int n, int& per) {
            const int want = (n + chunk - 1) / chunk;
            per = ((n + want - 1) / want + 63) / 64 * 64;
            return (n + per - 1) / per;
        };
        for (int g = tid; g < ngroups; g += kPlanThreads)
            if (group_ok[g]) {
                int per;
                const int nch = chunks_of(lens[g], per);
                atomicAdd(&s_class[len_class(per, chunk)], (unsigned)(nch * ((start[g + 1] - start[g] + T - 1) / T)));
            }
        __syncthreads();
        if (warp == 0) {
            const unsigned c = lane < kLenClasses ? s_class[lane] : 0u;
            unsigned x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane < kLenClasses) s_class[lane] = x - c;
            if (lane == 31) s_items = x;
        }
        __syncthreads();
        GroupItem* items = const_cast<GroupItem*>(a.g.items);
        for (int g = warp; g < ngroups; g += kPlanThreads / 32) {
            if (!group_ok[g]) continue;
            const int r0 = start[g], r1 = start[g + 1], n = lens[g];
            const int tiles = (r1 - r0 + T - 1) / T;
            int per;
            const int nch = chunks_of(n, per);
            unsigned i0 = 0;
            if (lane == 0) i0 = atomicAdd(&s_class[len_class(per, chunk)], (unsigned)(tiles * nch));
            i0 = __shfl_sync(0xffffffffu, i0, 0);
            const int first = rows[r0];
            for (int i = lane; i < tiles * nch; i += 32) {
                const int ch = i / tiles, tile = i % tiles;
                GroupItem it{};
                it.table_row = first;
                it.row0 = r0 + tile * T;
                it.members = min(T, r1 - r0 - tile * T);
                it.chunk = ch;
                it.kv0 = ch * per;
                it.kvlen = min(per, n - ch * per);
                items[i0 + i] = it;
            }
            for (int i = r0 + lane; i < r1; i += 32) {
                const int s = rows[i];
                lead_blocks[s] = n >> bshift;
                lead_states[s] = nch;
            }
        }
        __syncthreads();
    }
    unsigned tok = 0;
    for (int s = tid; s < S; s += kPlanThreads) tok += (unsigned)(ctx[s] - lead_blocks[s] * B);
    tok = __reduce_add_sync(0xffffffffu, tok);
    if (lane == 0 && tok) atomicAdd(&s_own, tok);
    __syncthreads();
    const int share = own_share(s_own, S, a.g.num_kv_heads, own_warps);
    auto part_of = [&](int own) { return own_part(own, share, a.max_parts); };
    const int big = max(32, share / 2);  // an entry of the first half
    unsigned nbig = 0;
    for (int s = tid; s < S; s += kPlanThreads) {
        const int own = ctx[s] - lead_blocks[s] * B, per = part_of(own);
        nbig += per > big ? (own <= per ? 1u : (unsigned)((own + per - 1) / per)) : 0u;
    }
    if (nbig) atomicAdd(&s_big, nbig);
    __syncthreads();
    for (int s = tid; s < S; s += kPlanThreads) {
        const int tok0 = lead_blocks[s] * B, own = ctx[s] - tok0, lead = lead_states[s];
        const int per = part_of(own), parts = own <= per ? 1 : (own + per - 1) / per;
        const unsigned i0 = per > big ? atomicAdd(&s_front, (unsigned)parts) : s_big + atomicAdd(&s_back, (unsigned)parts);
        for (int p = 0; p < parts; ++p)
            a.own[i0 + p] = OwnItem{s, tok0 + p * per, min(per, own - p * per), lead, p, parts, s, 0};
        if (parts > 1)
            for (int h = 0; h < a.g.num_kv_heads; ++h) a.arrived[(size_t)s * a.g.num_kv_heads + h] = 0u;
    }
    __syncthreads();
    if (tid == 0) {
        unsigned* counts = const_cast<unsigned*>(a.g.counts);
        counts[0] = s_items;
        counts[2] = s_big + s_back;
    }
}

// The plan of single query rows (pa_cross_attention): an entry per sequence with a row, or per part of it.
__global__ void __launch_bounds__(kPlanThreads, 1)
    single_plan_kernel(const SharedArgs a, const int32_t* q_start, int num_query_tokens, int own_warps)
{
    __shared__ unsigned s_own, s_big, s_front, s_back;
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, S = a.num_seqs;
    const int cap = min(a.max_context_len, table_tokens(a.g.max_blocks_per_seq, a.g.block_size));
    if (tid == 0) s_own = s_big = s_front = s_back = 0;
    // row and tokens of sequence s; no row where its data is bad
    auto load = [&](int s, int& row, int& L, bool flag) {
        const int q0 = __ldg(q_start + s), q1 = __ldg(q_start + s + 1);
        L = __ldg(a.context_lens + s);
        const bool bad = q0 < 0 || q1 > num_query_tokens || q1 < q0 || q1 - q0 > 1 || L < 0 || L > cap;
        if (bad && flag) atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
        row = bad || q1 == q0 ? -1 : q0;
    };
    int row0 = -1, L0 = 0;  // this thread's first sequence, loaded once
    unsigned tok = 0;
    for (int s = tid; s < S; s += kPlanThreads) {
        int row, L;
        load(s, row, L, true);
        if (s == tid) {
            row0 = row;
            L0 = L;
        }
        if (row >= 0) tok += (unsigned)L;
    }
    tok = __reduce_add_sync(0xffffffffu, tok);
    __syncthreads();
    if (lane == 0 && tok) atomicAdd(&s_own, tok);
    __syncthreads();
    const int share = own_share(s_own, S, a.g.num_kv_heads, own_warps), big = max(32, share / 2);
    unsigned nbig = 0;
    for (int s = tid; s < S; s += kPlanThreads) {
        int row = row0, L = L0;
        if (s != tid) load(s, row, L, false);
        const int per = own_part(L, share, a.max_parts);
        if (row >= 0 && per > big) nbig += L <= per ? 1u : (unsigned)((L + per - 1) / per);
    }
    if (nbig) atomicAdd(&s_big, nbig);
    __syncthreads();
    for (int s = tid; s < S; s += kPlanThreads) {
        int row = row0, L = L0;
        if (s != tid) load(s, row, L, false);
        if (row < 0) continue;
        const int per = own_part(L, share, a.max_parts), parts = L <= per ? 1 : (L + per - 1) / per;
        const unsigned i0 = per > big ? atomicAdd(&s_front, (unsigned)parts) : s_big + atomicAdd(&s_back, (unsigned)parts);
        for (int p = 0; p < parts; ++p) a.own[i0 + p] = OwnItem{row, p * per, min(per, L - p * per), 0, p, parts, s, 0};
        if (parts > 1)
            for (int h = 0; h < a.g.num_kv_heads; ++h) a.arrived[(size_t)row * a.g.num_kv_heads + h] = 0u;
    }
    __syncthreads();
    if (tid == 0) const_cast<unsigned*>(a.g.counts)[2] = s_big + s_back;
}

// The own tokens and the join.
//
// A unit is one kv head of a row, or of a part of it, and one warp's.  Thousands of them are
// short (a sampled stream's own tokens are 1 to 40), so what counts is that no unit waits for
// another and that the next one's bytes are under way while one ends: every warp streams its
// units' K and V, 16 tokens a step, through a ring of its own (cp.async, swizzled as TMA's 128
// bytes would be), and a unit's q comes with its first step.  The copies run ahead by the ring's
// stages, across units; the units' entries and blocks are fetched ahead of that.  (With TMA boxes
// of a block's 16 tokens the step was as long again: a thread takes 200 to 250 cycles to issue
// one, 1,100 a step, where the step's arithmetic takes 1,000 to 1,200 and these copies 200.)
//
// A step's products are m16n8k16 MMAs (fp32 accumulation).  An MMA's order of k is free as long
// as both operands agree, and so is the order of output rows, so every lane reads 16 contiguous
// bytes at a time and nothing is transposed:
//   S^T[heads][tokens] = q K^T: lane (g, t) holds dims 8t .. 8t+7 of each 32 for head g (A) and
//     for tokens g and g + 8 (B);
//   O^T[dims][heads] += V^T P: lane (g, t) holds dims 8g .. 8g+7 of each 64 for tokens 2t, 2t+1,
//     2t+8, 2t+9; pairs of tokens are packed per dim (A), and P comes out of S^T's accumulators
//     in B's layout as it is.  P is split into a bf16 head and remainder, as in pa_decode.
// Lane (g, t) ends with dims 8g .. 8g+7 of each 64 of heads 2t and 2t + 1, and reads the other
// states of the row the same way, 32 contiguous bytes each.
constexpr int kOwnThreads = 128, kOwnWarps = 4, kStep = 16;
constexpr int own_ctas(int head_dim) { return head_dim == 64 ? 4 : 2; }  // per SM

template <int D, int G>
struct OwnCfg {
    static constexpr int NH = D / 64;
    static constexpr int HALF = kStep * 128;               // 64 columns of a step's K or V
    static constexpr int CTAS = own_ctas(D);
    static constexpr int STAGE = 2 * NH * HALF + (G * D * 2 + 127) / 128 * 128;
    static constexpr int NST = (227 * 1024 / CTAS - 1024) / (kOwnWarps * STAGE);
    static constexpr int SMEM = kOwnWarps * NST * STAGE;
    static_assert(NST >= 2 && CTAS * (SMEM + 1024) <= 227 * 1024, "two stages a warp");
};

__device__ __forceinline__ uint32_t lo_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// A warp's softmax state of one kv head.
template <int D>
struct OwnState {
    static constexpr int NV = D / 64;
    float m, l;          // head g: running maximum, and this lane's share of the sum (all of it after finish)
    float o[NV * 4][4];  // dims 64c + 8g + j, heads 2t and 2t + 1; then dims + 4

    __device__ __forceinline__ void clear()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    // the output columns by a factor per head g
    __device__ __forceinline__ void scale(float f, int t)
    {
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) {
            o[i][0] *= f0;
            o[i][1] *= f1;
            o[i][2] *= f0;
            o[i][3] *= f1;
        }
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// q of a unit from shared memory ([G][D]) into the A operand's registers.
template <int D, int G>
__device__ __forceinline__ void load_q(uint32_t qs, uint4 (&q)[D / 32])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) q[c] = g < G ? lds16(qs + g * D * 2 + c * 64 + t * 16) : make_uint4(0, 0, 0, 0);
}

// One step: 16 tokens of K at ks and of V at vs (halves of 64 columns, 128-byte swizzle), `left` of them valid.
template <int D, int G>
__device__ __forceinline__ void own_step(uint32_t ks, uint32_t vs, int left, float sl, const uint4 (&q)[D / 32], OwnState<D>& st)
{
    constexpr int NC = D / 32, NV = D / 64, HALF = kStep * 128;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // (two chains of MMAs for each half of the tokens: the step is bound by its latency)
    float x[2][4], x2[2][4];
    uint4 k[2][NC];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
        x2[n][0] = x2[n][1] = x2[n][2] = x2[n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ch = c * 4 + t;  // 16-byte chunk of the row: its half, and its place there
            k[n][c] = lds16(ks + (ch >> 3) * HALF + (n * 8 + g) * 128 + (((ch & 7) ^ g) << 4));
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const uint32_t a0[4] = {q[c].x, 0u, q[c].y, 0u}, a1[4] = {q[c].z, 0u, q[c].w, 0u};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma_bf16(x[n], a0, k[n][c].x, k[n][c].y);
            mma_bf16(x2[n], a1, k[n][c].z, k[n][c].w);
        }
    }
    uint32_t w[NV][4][4];
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int vt = 2 * t + (i & 1) + (i >> 1) * 8;
            // (tokens past the context: their weight is 0, and 0 must not meet a NaN left in the pool)
            const uint4 v = vt < left ? lds16(vs + c * HALF + vt * 128 + ((g ^ (vt & 7)) << 4)) : make_uint4(0, 0, 0, 0);
            w[c][i][0] = v.x;
            w[c][i][1] = v.y;
            w[c][i][2] = v.z;
            w[c][i][3] = v.w;
        }
    // logits of head g for tokens 2t, 2t+1, 2t+8, 2t+9
    float y[4];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int vt = 2 * t + (i & 1) + (i >> 1) * 8;
        y[i] = vt < left ? (x[i >> 1][i & 1] + x2[i >> 1][i & 1]) * sl : -INFINITY;
        mx = fmaxf(mx, y[i]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(st.m, mx);
    if (__any_sync(0xffffffffu, mn > st.m)) {
        const float al = st.m == -INFINITY ? 0.f : ex2(st.m - mn);
        st.m = mn;
        st.l *= al;
        st.scale(al, t);
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = y[i] == -INFINITY ? 0.f : ex2(y[i] - st.m);
        st.l += p[i];
    }
    const uint32_t h0 = pack_bf16(p[0], p[1]), h1 = pack_bf16(p[2], p[3]);
    const uint32_t r0 = pack_bf16(p[0] - __uint_as_float(h0 << 16), p[1] - __uint_as_float(h0 & 0xffff0000u));
    const uint32_t r1 = pack_bf16(p[2] - __uint_as_float(h1 << 16), p[3] - __uint_as_float(h1 & 0xffff0000u));
#pragma unroll
    for (int c = 0; c < NV; ++c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // output rows g: dim 8g + j, rows g + 8: dim 8g + j + 4 (of 64)
            const int e = j >> 1;
            uint32_t af[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x0 = w[c][(i >> 1) * 2][e + (i & 1) * 2], x1 = w[c][(i >> 1) * 2 + 1][e + (i & 1) * 2];
                af[i] = (j & 1) ? hi_pair(x0, x1) : lo_pair(x0, x1);
            }
            mma_bf16(st.o[c * 4 + j], af, h0, h1);
            mma_bf16(st.o[c * 4 + j], af, r0, r1);
        }
    }
}

// Adds the states slot(first), slot(first + step), ... (below n) of the row and kv head to the warp's.  The
// output columns of heads G and up are nobody's, so their lanes take states of their own: 4 / HP at a time.
template <int D, int G, class Slot>
__device__ __forceinline__ void absorb_states(const SharedArgs& a, size_t row0, OwnState<D>& st, int n, int first, int step,
                                              Slot slot)
{
    constexpr int NV = D / 64, HP = G >= 2 ? G / 2 : 1, SPL = 4 / HP;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int hp = t % HP, sub = t / HP;
    const int np = a.g.num_partitions;
    const int cnt = (n - first + step - 1) / step;
    if (cnt <= 0) return;
    const float2* ml = reinterpret_cast<const float2*>(a.g.ws_ml) + row0 * np;
    float M = st.m;
    for (int i = t; i < cnt; i += 4) M = fmaxf(M, __ldcg(ml + (size_t)(g < G ? g : 0) * np + slot(first + i * step)).x);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
    const float f = st.m == -INFINITY ? 0.f : exp2f(st.m - M);
    st.m = M;
    st.l *= f;
    st.scale(f, t);
    if (t >= HP) {
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
    }
    const float M0 = __shfl_sync(0xffffffffu, M, 8 * hp), M1 = __shfl_sync(0xffffffffu, M, 8 * hp + 4);
    float l0 = 0.f, l1 = 0.f;
    for (int i = 0; i < cnt; i += SPL) {
        const bool valid = i + sub < cnt;
        const int p = slot(first + min(i + sub, cnt - 1) * step);
        const float4* acc = reinterpret_cast<const float4*>(a.g.ws_acc + ((row0 + 2 * hp) * np + p) * D + 8 * g);
        float4 x[G >= 2 ? 2 : 1][NV][2];
        float2 v[2];
#pragma unroll
        for (int h = 0; h < (G >= 2 ? 2 : 1); ++h) {
            v[h] = __ldcg(ml + (size_t)(2 * hp + h) * np + p);
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                x[h][c][0] = __ldcg(acc + (size_t)h * np * (D / 4) + c * 16);
                x[h][c][1] = __ldcg(acc + (size_t)h * np * (D / 4) + c * 16 + 1);
            }
        }
#pragma unroll
        for (int h = 0; h < (G >= 2 ? 2 : 1); ++h) {
            const float w = valid ? state_weight(v[h].x, v[h].y, h ? M1 : M0) : 0.f;
            if (h) l1 = fmaf(w, v[h].y, l1);
            else l0 = fmaf(w, v[h].y, l0);
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                const float4 lo = x[h][c][0], hi = x[h][c][1];
                st.o[c * 4 + 0][h] = fmaf(w, lo.x, st.o[c * 4 + 0][h]);
                st.o[c * 4 + 1][h] = fmaf(w, lo.y, st.o[c * 4 + 1][h]);
                st.o[c * 4 + 2][h] = fmaf(w, lo.z, st.o[c * 4 + 2][h]);
                st.o[c * 4 + 3][h] = fmaf(w, lo.w, st.o[c * 4 + 3][h]);
                st.o[c * 4 + 0][h + 2] = fmaf(w, hi.x, st.o[c * 4 + 0][h + 2]);
                st.o[c * 4 + 1][h + 2] = fmaf(w, hi.y, st.o[c * 4 + 1][h + 2]);
                st.o[c * 4 + 2][h + 2] = fmaf(w, hi.z, st.o[c * 4 + 2][h + 2]);
                st.o[c * 4 + 3][h + 2] = fmaf(w, hi.w, st.o[c * 4 + 3][h + 2]);
            }
        }
    }
#pragma unroll
    for (int x = HP; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
#pragma unroll
        for (int i = 0; i < NV * 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[i][e] += __shfl_xor_sync(0xffffffffu, st.o[i][e], x);
    }
    // the sums belong with head g: lane t = (g / 2) has them for heads 2t and 2t + 1
    const float s0 = __shfl_sync(0xffffffffu, l0, (g >> 1) % HP), s1 = __shfl_sync(0xffffffffu, l1, (g >> 1) % HP);
    st.l += (g & 1) ? s1 : s0;
}

// A warp's state of a unit to and from its partial state `slot`.
template <int D, int G>
__device__ __forceinline__ void store_state(const SharedArgs& a, size_t row0, int slot, const OwnState<D>& st)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, np = a.g.num_partitions;
    if (t == 0 && g < G) *reinterpret_cast<float2*>(a.g.ws_ml + ((row0 + g) * np + slot) * 2) = make_float2(st.m, st.l);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (2 * t + h < G) {
            float4* acc = reinterpret_cast<float4*>(a.g.ws_acc + ((row0 + 2 * t + h) * np + slot) * D + 8 * g);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                acc[c * 16] = make_float4(st.o[c * 4][h], st.o[c * 4 + 1][h], st.o[c * 4 + 2][h], st.o[c * 4 + 3][h]);
                acc[c * 16 + 1] =
                    make_float4(st.o[c * 4][h + 2], st.o[c * 4 + 1][h + 2], st.o[c * 4 + 2][h + 2], st.o[c * 4 + 3][h + 2]);
            }
        }
}

template <int D, int G>
__device__ __forceinline__ void load_state(const SharedArgs& a, size_t row0, int slot, OwnState<D>& st)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, np = a.g.num_partitions;
    st.clear();
    if (g < G) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(a.g.ws_ml) + (row0 + g) * np + slot);
        st.m = v.x;
        st.l = v.y;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (2 * t + h < G) {
            const float4* acc = reinterpret_cast<const float4*>(a.g.ws_acc + ((row0 + 2 * t + h) * np + slot) * D + 8 * g);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 lo = __ldcg(acc + c * 16), hi = __ldcg(acc + c * 16 + 1);
                st.o[c * 4][h] = lo.x;
                st.o[c * 4 + 1][h] = lo.y;
                st.o[c * 4 + 2][h] = lo.z;
                st.o[c * 4 + 3][h] = lo.w;
                st.o[c * 4][h + 2] = hi.x;
                st.o[c * 4 + 1][h + 2] = hi.y;
                st.o[c * 4 + 2][h + 2] = hi.z;
                st.o[c * 4 + 3][h + 2] = hi.w;
            }
        }
}

template <int D, int G>
__device__ __forceinline__ void write_row(const SharedArgs& a, size_t row0, OwnState<D>& st)
{
    constexpr int NV = D / 64;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (a.g.lse && t == 0 && g < G)
        a.g.lse[row0 + g] = row_lse(st.m, st.l);
    st.scale(st.l > 0.f ? 1.f / st.l : 0.f, t);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (2 * t + h < G) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.g.out) + (row0 + 2 * t + h) * D + 8 * g);
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                uint4 pk;
                pk.x = pack_bf16(st.o[c * 4 + 0][h], st.o[c * 4 + 1][h]);
                pk.y = pack_bf16(st.o[c * 4 + 2][h], st.o[c * 4 + 3][h]);
                pk.z = pack_bf16(st.o[c * 4 + 0][h + 2], st.o[c * 4 + 1][h + 2]);
                pk.w = pack_bf16(st.o[c * 4 + 2][h + 2], st.o[c * 4 + 3][h + 2]);
                out[c * 8] = pk;
            }
        }
}

template <int D, int G>
__global__ void __launch_bounds__(kOwnThreads, own_ctas(D)) shared_own_kernel(const __grid_constant__ SharedArgs a)
{
    using C = OwnCfg<D, G>;
    constexpr int NST = C::NST, CPR = D / 8;  // 16-byte chunks of a row
    extern __shared__ __align__(1024) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned Hkv = (unsigned)a.g.num_kv_heads;
    const uint32_t ring = smem_u32(smem) + warp * NST * C::STAGE;
    if (a.wait_first) pdl_wait_primary();
    const unsigned entries = __ldcg(a.g.counts + 2), total = entries * Hkv;
    const unsigned first = blockIdx.x * kOwnWarps + warp, hop = gridDim.x * kOwnWarps;

    const int bshift = a.g.block_size == 16 ? 4 : 5;
    // The copying cursor: unit iu (kv head ikvh) at token itk, the block of that step, and the entry of the unit after.
    auto table_at = [&](const OwnItem& it, int tk) {
        return it.ntok > 0 ? __ldg(a.g.block_tables + (size_t)it.table_row * a.g.max_blocks_per_seq + (tk >> bshift)) : 0;
    };
    unsigned iu = first;
    OwnItem icur = load_own(a.own, iu / Hkv, iu < total ? entries : 0u);
    OwnItem inext = load_own(a.own, (iu + hop) / Hkv, iu + hop < total ? entries : 0u);
    int itk = icur.tok0, iphys = table_at(icur, itk), ikvh = (int)(iu % Hkv), ist = 0;
    // lane's chunk of rows lane / CPR, + 32 / CPR, ...: the swizzle repeats every 8 rows
    constexpr int RPI = 32 / CPR;
    const int crow = lane / CPR, cch = lane % CPR;
    auto issue = [&]() {
        if (iu < total) {
            const uint32_t dst = ring + ist * C::STAGE;
            if (icur.ntok > 0) {
                int phys = iphys;
                if ((unsigned)phys >= (unsigned)a.g.num_blocks) {
                    if (lane == 0) atomicOr(a.g.status, PA_DEV_BAD_BLOCK);
                    phys = 0;
                }
                const unsigned row = ((unsigned)phys * Hkv + ikvh) * (1u << bshift) + (itk & ((1 << bshift) - 1));  // < 2^31
                const size_t off = (size_t)row * (D * 2) + lane * 16;
                const char* kp = static_cast<const char*>(a.g.k_cache) + off;
                const char* vp = static_cast<const char*>(a.g.v_cache) + off;
#pragma unroll
                for (int i = 0; i < kStep / RPI; ++i) {
                    const int r = crow + i * RPI;
                    const uint32_t d = dst + (cch >> 3) * C::HALF + r * 128 + (((cch & 7) ^ (r & 7)) << 4);
                    cp_async16(d, kp + i * 512);
                    cp_async16(d + C::NH * C::HALF, vp + i * 512);
                }
                if (itk == icur.tok0) {
                    const char* qp = static_cast<const char*>(a.g.q) +
                                     ((size_t)icur.row * a.g.num_heads + (size_t)ikvh * G) * (D * 2);
#pragma unroll
                    for (int i = 0; i < (G * CPR + 31) / 32; ++i)
                        if (i * 32 + lane < G * CPR)
                            cp_async16(dst + 2 * C::NH * C::HALF + (i * 32 + lane) * 16, qp + (i * 32 + lane) * 16);
                }
            }
            // on to the next step (a unit without tokens takes one, without bytes): its block is asked for now
            if (itk + kStep < icur.tok0 + icur.ntok) {
                itk += kStep;
            } else {
                iu += hop;
                ikvh = (int)(iu % Hkv);
                icur = inext;
                inext = load_own(a.own, (iu + hop) / Hkv, iu + hop < total ? entries : 0u);
                itk = icur.tok0;
            }
            iphys = table_at(icur, itk);
        }
        ist = ist + 1 == NST ? 0 : ist + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < NST; ++i) issue();

    bool waited = a.wait_first != 0;
    // A unit whose row has shared tokens is joined with their states, which come late: the join is put off until this
    // warp has nothing else to do (its last unit's state stays in registers), and `back` is the trip over those.
    bool put_off = false, back = false;
    int sg = 0;  // stage of the next step
    OwnState<D> st;
    OwnItem it = load_own(a.own, first / Hkv, first < total ? entries : 0u);
    for (unsigned u = first; u < total;) {
        const bool final = u + hop >= total;
        const unsigned un = final ? first : u + hop;
        const OwnItem next = load_own(a.own, un / Hkv, entries);
        const unsigned kvh = u % Hkv;
        const size_t row0 = (size_t)it.row * a.g.num_heads + (size_t)kvh * G;
        bool later;
        if (!back) {
            st.clear();
            uint4 q[D / 32];
            const int n = max(1, (it.ntok + kStep - 1) / kStep);
            for (int j = 0; j < n; ++j) {
                asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
                __syncwarp();
                const uint32_t base = ring + sg * C::STAGE;
                if (it.ntok > 0) {
                    if (j == 0) load_q<D, G>(base + 2 * C::NH * C::HALF, q);
                    own_step<D, G>(base, base + C::NH * C::HALF, it.ntok - j * kStep, a.g.scale_log2, q, st);
                }
                __syncwarp();  // every lane has read the stage
                sg = sg + 1 == NST ? 0 : sg + 1;
                issue();
            }
            st.l += __shfl_xor_sync(0xffffffffu, st.l, 1);
            st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
            later = it.lead > 0 && !waited && !final;
            put_off |= later;
            if (it.parts > 1 || later) store_state<D, G>(a, row0, a.g.lead_partitions + it.part, st);
        } else {
            later = it.lead == 0 || final;  // (joined already)
            if (!later && it.parts == 1) load_state<D, G>(a, row0, a.g.lead_partitions, st);
        }
        if (!later) {
            if (it.lead > 0 && !waited) {
                pdl_wait_primary();
                waited = true;
            }
            // of several parts the last one here joins them all, in order
            bool last = true;
            if (it.parts > 1) {
                __threadfence();
                __syncwarp();
                unsigned before = 0;
                if (lane == 0) before = atomicAdd(a.arrived + (size_t)it.row * Hkv + kvh, 1u);
                before = __shfl_sync(0xffffffffu, before, 0);
                __threadfence();
                last = before == (unsigned)it.parts - 1;
                if (last) st.clear();
            }
            if (last) {
                const int lead = it.lead, skip = a.g.lead_partitions - lead;
                absorb_states<D, G>(a, row0, st, lead + (it.parts > 1 ? it.parts : 0), 0, 1,
                                    [lead, skip](int p) { return p < lead ? p : p + skip; });
                write_row<D, G>(a, row0, st);
            }
        }
        if (final) {
            if (back || !put_off) break;
            back = true;
            __syncwarp();  // the states of this warp, read by other lanes than wrote them
        }
        u = un;
        it = next;
    }
    // whatever waits for this grid may count on the shared tokens' kernel having finished too
    if (!waited) pdl_wait_primary();
}

template <int D, int G>
cudaError_t launch_shared_dg(const SharedArgs& a, cudaStream_t stream)
{
    using C = OwnCfg<D, G>;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaFuncSetAttribute(shared_own_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int tile_rows = shared_tile_rows(a.num_groups, a.num_group_rows, G);
    const int gctas = group_resident_ctas(sms);
    const int64_t units = (int64_t)a.num_seqs * a.max_parts * a.g.num_kv_heads;
    // Rows so short that their warps read them in twelve steps, and few enough for a warp per row and kv head: the
    // shared tokens' kernel would take longer than reading them once per row.  Shared / not, graph replay, us: 4 rows x 8
    // heads of 116 tokens 14.9 / 11.5 (head_dim 64), 16.4 / 13.4 (128), 212 tokens 15.3 / 14.6 and 16.8 / 17.4; 128 rows x
    // 8 heads x 4 of 116 tokens 18.1 / 13.5 and 21.8 / 16.2, 212 tokens 18.7 / 17.4 and 22.0 / 21.8, 308 20.2 / 22.8 and 24.9 / 35.6.
    const bool brief = a.max_context_len <= 192 && (int64_t)a.num_seqs * a.g.num_kv_heads <= (int64_t)C::CTAS * sms * kOwnWarps;
    const bool shares = a.g.max_entries > 0 && !brief;
    SharedArgs args = a;
    args.wait_first = shares ? 0 : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((units + kOwnWarps - 1) / kOwnWarps, (int64_t)C::CTAS * sms);
    shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(args, tile_rows / G, D, gctas, C::CTAS * sms * kOwnWarps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (shares && (e = launch_group(args.g, D, G, tile_rows, gctas, stream)) != cudaSuccess) return e;
    return launch_pdl(shared_own_kernel<D, G>, dim3(grid), dim3(kOwnThreads), (size_t)C::SMEM, stream, args);
}

template <int D>
cudaError_t launch_shared_d(const SharedArgs& a, int group, cudaStream_t stream)
{
    switch (group) {
        case 1: return launch_shared_dg<D, 1>(a, stream);
        case 2: return launch_shared_dg<D, 2>(a, stream);
        case 4: return launch_shared_dg<D, 4>(a, stream);
        case 8: return launch_shared_dg<D, 8>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

namespace {

template <int D, int G>
cudaError_t launch_single_dg(const SharedArgs& a, const int32_t* q_start, int num_query_tokens, cudaStream_t stream)
{
    using C = OwnCfg<D, G>;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaFuncSetAttribute(shared_own_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    SharedArgs args = a;
    args.wait_first = 1;
    const int64_t units = (int64_t)a.num_seqs * a.max_parts * a.g.num_kv_heads;
    const unsigned grid = (unsigned)std::min<int64_t>((units + kOwnWarps - 1) / kOwnWarps, (int64_t)C::CTAS * sms);
    single_plan_kernel<<<1, kPlanThreads, 0, stream>>>(args, q_start, num_query_tokens, C::CTAS * sms * kOwnWarps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_pdl(shared_own_kernel<D, G>, dim3(grid), dim3(kOwnThreads), (size_t)C::SMEM, stream, args);
}

template <int D>
cudaError_t launch_single_d(const SharedArgs& a, const int32_t* q_start, int num_query_tokens, int group, cudaStream_t stream)
{
    switch (group) {
        case 1: return launch_single_dg<D, 1>(a, q_start, num_query_tokens, stream);
        case 2: return launch_single_dg<D, 2>(a, q_start, num_query_tokens, stream);
        case 4: return launch_single_dg<D, 4>(a, q_start, num_query_tokens, stream);
        case 8: return launch_single_dg<D, 8>(a, q_start, num_query_tokens, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_cross_single(const SharedArgs& a, const int32_t* q_start, int num_query_tokens, int head_dim, int group,
                                cudaStream_t stream)
{
    return head_dim == 64 ? launch_single_d<64>(a, q_start, num_query_tokens, group, stream)
                          : launch_single_d<128>(a, q_start, num_query_tokens, group, stream);
}

cudaError_t launch_shared(const SharedArgs& a, int head_dim, int group, cudaStream_t stream)
{
    return head_dim == 64 ? launch_shared_d<64>(a, group, stream) : launch_shared_d<128>(a, group, stream);
}

}  // namespace pa
