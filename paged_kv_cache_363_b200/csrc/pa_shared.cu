// Decode attention of a batch in groups whose sequences share leading blocks, for sm_100a.
//
// What it computes: pa_decode's output.  Row s of group g attends to the group's n_g shared
// tokens and to its own tokens n_g .. L_s - 1; the softmax over both is joined from the two
// partial states (m, l, O) = (maximum, sum of 2^(x - m), weighted V):
//   out = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p,  M = max m_p.
// The shared tokens of a kv head are one dense product of all the group's rows x G query
// heads with the same K and V: the tensor-core kernel of pa_group.cu reads each shared byte
// once per 128 rows, where pa_decode reads it once per sequence (from L2 when it is lucky).
// A row's own tokens are read by the kernel that also joins the states, unless they are many;
// those go through pa_decode's persistent kernel, from the block behind the shared ones.
//
// Four kernels: a plan, the shared tokens, the long rows' own tokens, the finish.  The last two
// need the plan alone to begin, so the shared tokens' kernel lets them start once it has itself
// seen the plan finish, and the CTAs of all share the device until the work is gone.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_persist.cuh"
#include "pa_group.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_shared.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;

// 16 bytes of the K/V stream, read once
__device__ __forceinline__ uint4 ldg_stream(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// What the plan says about a row.
struct RowInfo {
    int lead_blocks;   // shared blocks before its own tokens
    int lead_states;   // partial states of its shared tokens
    int own_parts;     // partial states of its own tokens (kDirect: none, the finish attends to them itself)
    int L;             // context length (clamped)
};
constexpr int kDirect = -1;

// The plan, in one CTA.
//  1. Groups are checked (starts in order, rows in range and listed once, whole blocks, no more
//     tokens than any member's context).  A bad one raises PA_DEV_BAD_CONTEXT and is not
//     shared: its rows attend to all their tokens on their own, which is the same result.
//  2. Entries of the shared tokens: (tile of rows, chunk), a chunk's tiles next to each other.
//     The chunk length is the work over twice the resident CTAs, at least 256 tokens.
//  3. The long rows' own tokens as units for the decode kernel, longest first, as pa_decode's
//     plan lists them, each entry with the blocks before it and the number of shared states
//     (which makes it write its own state).
// A batch of up to 1024 rows keeps its per-row values in shared memory: the plan is on the
// critical path, and most of it was trips to L2.
__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_kernel(const SharedArgs a, int T, int group_ctas)
{
    __shared__ int bucket[kMaxPartitionTokens / 16 + 1];
    __shared__ int s_listed[kPlanThreads], s_ctx[kPlanThreads], s_lead[kPlanThreads], s_states[kPlanThreads];
    __shared__ unsigned long long s_work, s_tok;
    __shared__ unsigned s_items;
    __shared__ int s_bad, s_max, s_pb;
    pdl_launch_dependents();
    const DecodeArgs& d = a.d;
    const int B = a.g.block_size;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool small = d.num_seqs <= kPlanThreads;
    volatile int* listed = small ? s_listed : a.listed;
    volatile int* ctx = small ? s_ctx : a.ctx;
    volatile int* lead_blocks = small ? s_lead : a.lead_blocks;
    volatile int* lead_states = small ? s_states : a.lead_states;
    if (tid == 0) {
        s_work = s_tok = 0;
        s_items = 0;
        s_bad = s_max = 0;
    }
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        listed[s] = 0;
        lead_blocks[s] = 0;
        lead_states[s] = 0;
        ctx[s] = clamped_context(d, s, B, true);
    }
    __syncthreads();
    for (int g = tid; g < a.num_groups; g += kPlanThreads) {
        const int r0 = __ldg(a.group_start + g), r1 = __ldg(a.group_start + g + 1);
        if (r0 < 0 || r1 < r0 || r1 > a.num_group_rows) s_bad = 1;
    }
    for (int i = tid; i < a.num_group_rows; i += kPlanThreads) {
        const int s = __ldg(a.group_rows + i);
        if ((unsigned)s < (unsigned)d.num_seqs) atomicAdd(const_cast<int*>(listed) + s, 1);
    }
    __syncthreads();
    if (tid == 0 && s_bad) atomicOr(d.status, PA_DEV_BAD_CONTEXT);
    const int ngroups = s_bad ? 0 : a.num_groups;
    for (int g = warp; g < ngroups; g += kPlanThreads / 32) {
        const int r0 = __ldg(a.group_start + g), r1 = __ldg(a.group_start + g + 1), n = __ldg(a.shared_lens + g);
        bool ok = n >= 0 && n <= a.max_shared_len && n % B == 0;
        for (int i = r0 + lane; i < r1; i += 32) {
            const int s = __ldg(a.group_rows + i);
            ok = ok && (unsigned)s < (unsigned)d.num_seqs;
            ok = ok && listed[s] == 1 && n <= ctx[s];
        }
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (lane == 0) {
            a.group_ok[g] = ok && n > 0 && r1 > r0;
            if (!ok) atomicOr(d.status, PA_DEV_BAD_CONTEXT);
            else if (n > 0) atomicAdd(&s_work, (unsigned long long)((r1 - r0 + T - 1) / T) * n);
        }
    }
    __syncthreads();
    if (s_work > 0) {
        const unsigned long long share = s_work * d.num_kv_heads / (2ull * group_ctas);
        const int least = (a.max_shared_len + a.max_chunks - 1) / a.max_chunks;
        const int chunk = (max(max((int)min(share, 1ull << 30), least), 256) + 63) / 64 * 64;
        GroupItem* items = const_cast<GroupItem*>(a.g.items);
        for (int g = warp; g < ngroups; g += kPlanThreads / 32) {
            if (!*(volatile int*)(a.group_ok + g)) continue;
            const int r0 = __ldg(a.group_start + g), r1 = __ldg(a.group_start + g + 1), n = __ldg(a.shared_lens + g);
            const int tiles = (r1 - r0 + T - 1) / T;
            const int want = (n + chunk - 1) / chunk;
            const int per = ((n + want - 1) / want + 63) / 64 * 64;
            const int nch = (n + per - 1) / per;
            unsigned i0 = 0;
            if (lane == 0) i0 = atomicAdd(&s_items, (unsigned)(tiles * nch));
            i0 = __shfl_sync(0xffffffffu, i0, 0);
            const int first = __ldg(a.group_rows + r0);
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
                const int s = __ldg(a.group_rows + i);
                lead_blocks[s] = n / B;
                lead_states[s] = nch;
            }
        }
        __syncthreads();
    }
    // ---- the own tokens of long rows
    auto long_len = [&](int s) {
        const int own = ctx[s] - lead_blocks[s] * B;
        return own > kDirectTokens ? own : 0;
    };
    unsigned long long tok = 0;
    int lmax = 0;
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        const int L = long_len(s);
        tok += (unsigned long long)L;
        lmax = max(lmax, L);
    }
    if (tok > 0) {
        atomicAdd(&s_tok, tok);
        atomicMax(&s_max, lmax);
    }
    __syncthreads();
    const bool any = s_max > 0;
    int pb = d.partition_blocks;
    if (any) {
        if (tid == 0) {
            const int max_pb = kMaxPartitionTokens / B;
            const double share = (double)s_tok / (double)(d.num_ctas > 0 ? d.num_ctas : 1);
            while (2 * pb <= max_pb && pb * B < s_max && (double)min(2 * pb * B, s_max) * 4.0 <= share) pb *= 2;
            s_pb = pb;
        }
        for (int i = tid; i < kMaxPartitionTokens / 16 + 1; i += kPlanThreads) bucket[i] = 0;
        __syncthreads();
        pb = s_pb;
    }
    const int P = pb * B;
    RowInfo* info = reinterpret_cast<RowInfo*>(a.row_info);
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        const int L = long_len(s), np = (L + P - 1) / P;
        if (np > 0) {
            const int last = (L - (np - 1) * P + B - 1) / B;
            if (np > 1) atomicAdd(&bucket[pb], np - 1);
            atomicAdd(&bucket[last], 1);
        }
        const RowInfo r{lead_blocks[s], lead_states[s], np > 0 ? np : kDirect, ctx[s]};
        *reinterpret_cast<int4*>(info + s) = make_int4(r.lead_blocks, r.lead_states, r.own_parts, r.L);
    }
    if (any) {
        __syncthreads();
        if (warp == 0) {
            int running = 0;  // start of each size, largest first
            for (int base = pb; base >= 0; base -= 32) {
                const int sz = base - lane;
                const int c = sz >= 0 ? bucket[sz] : 0;
                int x = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (sz >= 0) bucket[sz] = running + x - c;
                running += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) d.plan[1] = (unsigned)running;
        }
        __syncthreads();
        uint4* list = reinterpret_cast<uint4*>(d.plan_list);
        for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
            const int L = long_len(s), np = (L + P - 1) / P;
            const int last = (L - (np - 1) * P + B - 1) / B;
            for (int p = 0; p < np; ++p) {
                const int pos = atomicAdd(&bucket[p < np - 1 ? pb : last], 1);
                list[pos] = make_uint4(((unsigned)s << 11) | (unsigned)p, (unsigned)ctx[s], (unsigned)lead_blocks[s],
                                       (unsigned)lead_states[s]);
            }
        }
    } else if (tid == 0) {
        d.plan[1] = 0u;
    }
    if (tid == 0) {
        d.plan[0] = 0u;
        d.plan[2] = (unsigned)pb;
        d.plan[4] = 0u;
        const_cast<unsigned*>(a.g.counts)[0] = s_items;
    }
}

// The finish, a CTA per (row, kv head): the row's own tokens (up to kDirectTokens of them),
// and the join with the partial states of its shared tokens (or of its own ones, when they were
// long).  The own tokens are read while the shared tokens' kernel still runs; only the join
// waits for it.
//
// The own tokens, 16 at a time per warp, straight from global memory into the operands of
// m16n8k16 MMAs (fp32 accumulation).  An MMA's order of k is free as long as both operands
// agree, and so is the order of output rows, so every lane loads 16 contiguous bytes:
//   S^T[heads][tokens] = q K^T: lane (g, t) holds dims 8t .. 8t+7 of each 32 for head g (A) and
//     for tokens g and g + 8 (B);
//   O^T[dims][heads] += V^T P: lane (g, t) holds dims 8g .. 8g+7 of each 64 for tokens 2t, 2t+1,
//     2t+8, 2t+9; pairs of tokens are packed per dim (A), and P comes out of S^T's accumulators
//     in B's layout as it is.  P is split into a bf16 head and remainder, as in pa_decode.
// Small units bound this part (a sampled stream's own tokens are 1 to 40): a unit of the
// persistent kernel costs some 3 us however small, a CTA here has all its loads in flight at once.
constexpr int kFinThreads = 128, kFinWarps = 4;

__device__ __forceinline__ uint32_t lo_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

template <int D, int G>
__global__ void __launch_bounds__(kFinThreads, 3) shared_finish_kernel(const SharedArgs a)
{
    constexpr int NC = D / 32;                         // 16-byte chunks of a K row per lane
    constexpr int NV = D / 64;                         // and of a V row
    __shared__ float s_o[kFinWarps][G][D];
    __shared__ float s_inv[G];
    extern __shared__ float s_ml[];                    // [G][states] maxima (then weights), [G][states] sums
    const DecodeArgs& d = a.d;
    const int max_states = kFinWarps + d.num_partitions;
    float* s_m = s_ml;
    float* s_l = s_ml + G * max_states;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (a.wait_first) pdl_wait_primary();
    const int s = blockIdx.x / d.num_kv_heads, kvh = blockIdx.x % d.num_kv_heads;
    const int4 ri = __ldcg(reinterpret_cast<const int4*>(a.row_info) + s);
    const int B = a.g.block_size, lead = ri.y, parts = ri.z == kDirect ? 0 : ri.z, L = ri.w;
    if (lead == 0 && parts == 1) return;  // one partition and nothing shared: the decode kernel wrote the row
    const int tok0 = ri.x * B;
    float m = -INFINITY, l = 0.f;         // head g, this lane's tokens' sum
    float o[NV * 4][4];
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    if (ri.z == kDirect && tok0 + warp * 16 < L) {
        const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(d.k_cache);
        const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(d.v_cache);
        const int32_t* table = d.block_tables + (size_t)s * d.max_blocks_per_seq;
        const float sl = d.scale_log2;
        uint4 q[NC];
        const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(d.q) +
                                                         ((size_t)s * d.num_heads + (size_t)kvh * G + (g < G ? g : 0)) * D);
#pragma unroll
        for (int c = 0; c < NC; ++c) q[c] = g < G ? __ldg(qp + c * 4 + t) : make_uint4(0, 0, 0, 0);
        int phys = __ldg(table + (tok0 + warp * 16) / B);
        for (int tk = tok0 + warp * 16; tk < L; tk += kFinWarps * 16) {
            if ((unsigned)phys >= (unsigned)d.num_blocks) {
                if (lane == 0) atomicOr(d.status, PA_DEV_BAD_BLOCK);
                phys = 0;
            }
            const size_t base = (((size_t)phys * d.num_kv_heads + kvh) * B + tk % B) * D;
            const int left = L - tk;  // tokens of this step
            uint4 k[2][NC], v[4][NV];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    k[n][c] = ldg_stream(reinterpret_cast<const uint4*>(kc + base + (size_t)(n * 8 + g) * D) + c * 4 + t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int vt = 2 * t + (i & 1) + (i >> 1) * 8;
#pragma unroll
                for (int c = 0; c < NV; ++c)
                    // (tokens past the context: their weight is 0, and 0 must not meet a NaN left in the pool)
                    v[i][c] = vt < left ? ldg_stream(reinterpret_cast<const uint4*>(vc + base + (size_t)vt * D) + c * 8 + g)
                                        : make_uint4(0, 0, 0, 0);
            }
            if (tk + kFinWarps * 16 < L) phys = __ldg(table + (tk + kFinWarps * 16) / B);
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint32_t a0[4] = {q[c].x, 0u, q[c].y, 0u}, a1[4] = {q[c].z, 0u, q[c].w, 0u};
                    mma_bf16(x[n], a0, k[n][c].x, k[n][c].y);
                    mma_bf16(x[n], a1, k[n][c].z, k[n][c].w);
                }
            }
            // logits of head g for tokens 2t, 2t+1, 2t+8, 2t+9
            float y[4];
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int vt = 2 * t + (i & 1) + (i >> 1) * 8;
                y[i] = vt < left ? x[i >> 1][i & 1] * sl : -INFINITY;
                mx = fmaxf(mx, y[i]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m, mx);
            if (__any_sync(0xffffffffu, mn > m)) {
                const float al = m == -INFINITY ? 0.f : exp2f(m - mn);
                m = mn;
                l *= al;
                // heads 2t and 2t + 1 of the output columns
                const float al0 = __shfl_sync(0xffffffffu, al, 8 * t), al1 = __shfl_sync(0xffffffffu, al, 8 * t + 4);
#pragma unroll
                for (int i = 0; i < NV * 4; ++i) {
                    o[i][0] *= al0;
                    o[i][1] *= al1;
                    o[i][2] *= al0;
                    o[i][3] *= al1;
                }
            }
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = y[i] == -INFINITY ? 0.f : exp2f(y[i] - m);
                l += p[i];
            }
            const uint32_t h0 = pack_bf16(p[0], p[1]), h1 = pack_bf16(p[2], p[3]);
            const uint32_t r0 = pack_bf16(p[0] - __uint_as_float(h0 << 16), p[1] - __uint_as_float(h0 & 0xffff0000u));
            const uint32_t r1 = pack_bf16(p[2] - __uint_as_float(h1 << 16), p[3] - __uint_as_float(h1 & 0xffff0000u));
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                const uint32_t* w[4] = {&v[0][c].x, &v[1][c].x, &v[2][c].x, &v[3][c].x};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // output rows g: dim 8g + j, rows g + 8: dim 8g + j + 4 (of 64)
                    const int e = j >> 1;
                    uint32_t af[4];
                    if (j & 1) {
                        af[0] = hi_pair(w[0][e], w[1][e]);
                        af[1] = hi_pair(w[0][e + 2], w[1][e + 2]);
                        af[2] = hi_pair(w[2][e], w[3][e]);
                        af[3] = hi_pair(w[2][e + 2], w[3][e + 2]);
                    } else {
                        af[0] = lo_pair(w[0][e], w[1][e]);
                        af[1] = lo_pair(w[0][e + 2], w[1][e + 2]);
                        af[2] = lo_pair(w[2][e], w[3][e]);
                        af[3] = lo_pair(w[2][e + 2], w[3][e + 2]);
                    }
                    mma_bf16(o[c * 4 + j], af, h0, h1);
                    mma_bf16(o[c * 4 + j], af, r0, r1);
                }
            }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
    }
    // the warps' states to shared memory
    if (t == 0 && g < G) {
        s_m[g * max_states + warp] = m;
        s_l[g * max_states + warp] = l;
    }
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) {
        const int dim = (i >> 2) * 64 + 8 * g + (i & 3);
        if (2 * t < G) {
            s_o[warp][2 * t][dim] = o[i][0];
            s_o[warp][2 * t][dim + 4] = o[i][2];
        }
        if (2 * t + 1 < G) {
            s_o[warp][2 * t + 1][dim] = o[i][1];
            s_o[warp][2 * t + 1][dim + 4] = o[i][3];
        }
    }
    // everything else the row's states need is written from here on
    if (!a.wait_first) pdl_wait_primary();
    const int nst = kFinWarps + lead + parts;
    const size_t row0 = (size_t)s * d.num_heads + (size_t)kvh * G;
    auto slot = [&](int p) { return p < lead ? p : d.lead_partitions + p - lead; };
    for (int i = threadIdx.x; i < G * (lead + parts); i += kFinThreads) {
        const int h = i / (lead + parts), p = i % (lead + parts);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(d.ws_ml) + (row0 + h) * d.num_partitions + slot(p));
        s_m[h * max_states + kFinWarps + p] = ml.x;
        s_l[h * max_states + kFinWarps + p] = ml.y;
    }
    __syncthreads();
    for (int h = warp; h < G; h += kFinWarps) {
        float M = -INFINITY, den = 0.f;
        for (int i = lane; i < nst; i += 32) M = fmaxf(M, s_m[h * max_states + i]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        for (int i = lane; i < nst; i += 32) {
            const float mi = s_m[h * max_states + i], w = mi == -INFINITY ? 0.f : exp2f(mi - M);
            s_m[h * max_states + i] = w;
            den = fmaf(w, s_l[h * max_states + i], den);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(0xffffffffu, den, x);
        if (lane == 0) s_inv[h] = den > 0.f ? 1.f / den : 0.f;
    }
    __syncthreads();
    // two columns a thread
    constexpr int TPH = D / 2;
    for (int h = threadIdx.x / TPH; h < G; h += kFinThreads / TPH) {
        const int col = (threadIdx.x % TPH) * 2;
        float n0 = 0.f, n1 = 0.f;
#pragma unroll
        for (int w = 0; w < kFinWarps; ++w) {
            const float wt = s_m[h * max_states + w];
            if (wt != 0.f) {
                n0 = fmaf(wt, s_o[w][h][col], n0);
                n1 = fmaf(wt, s_o[w][h][col + 1], n1);
            }
        }
        const float* acc = d.ws_acc + (row0 + h) * d.num_partitions * D + col;
        for (int p0 = 0; p0 < lead + parts; p0 += 8) {
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __ldcg(reinterpret_cast<const float2*>(acc + (size_t)slot(min(p0 + i, lead + parts - 1)) * D));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wt = p0 + i < lead + parts ? s_m[h * max_states + kFinWarps + p0 + i] : 0.f;
                if (wt != 0.f) {
                    n0 = fmaf(wt, x[i].x, n0);
                    n1 = fmaf(wt, x[i].y, n1);
                }
            }
        }
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(d.out) + (row0 + h) * D + col) =
            pack_bf16(n0 * s_inv[h], n1 * s_inv[h]);
    }
}

template <class Cons, int BS>
cudaError_t launch_shared_c(const SharedArgs& a, int group, cudaStream_t stream)
{
    using P = Persist<Cons, BS>;
    CUtensorMap tk, tv;
    std::memset(&tk, 0, sizeof(tk));
    std::memset(&tv, 0, sizeof(tv));
    cudaError_t e;
    if constexpr (Cons::kTensorLoads) {
        const uint64_t rows = (uint64_t)a.d.num_blocks * a.d.num_kv_heads * BS;
        if ((e = encode_pool_map(&tk, a.d.k_cache, rows, P::D, P::TR)) != cudaSuccess) return e;
        if ((e = encode_pool_map(&tv, a.d.v_cache, rows, P::D, P::TR)) != cudaSuccess) return e;
    }
    int ctas = 0;
    if ((e = resident_ctas<Cons, BS, kModeOwn>(&ctas)) != cudaSuccess) return e;
    const int64_t units = (int64_t)a.d.num_kv_heads * a.d.num_seqs * (a.d.num_partitions - a.d.lead_partitions);
    const unsigned grid = (unsigned)(units < ctas ? units : ctas);
    SharedArgs args = a;
    args.d.num_ctas = (int)grid;
    const bool shares = a.g.max_entries > 0;
    args.d.wait_first = shares ? 0 : 1;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int tile_rows = shared_tile_rows(a.num_groups, a.num_group_rows, group);
    const int gctas = group_resident_ctas(sms);
    shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(args, tile_rows / group, gctas);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (shares && (e = launch_group(args.g, P::D, group, tile_rows, gctas, stream)) != cudaSuccess) return e;
    // without a context longer than kDirectTokens the finish has every own token
    const bool longs = a.d.max_context_len > kDirectTokens;
    if (longs) {
        e = launch_pdl(decode_persistent_kernel<Cons, BS, kModeOwn>, dim3(grid), dim3(P::THREADS), (size_t)P::SMEM,
                       stream, args.d, tk, tv);
        if (e != cudaSuccess) return e;
    }
    args.wait_first = shares ? 0 : 1;
    const size_t smem = 2 * sizeof(float) * P::G * (size_t)(kFinWarps + a.d.num_partitions);
    e = cudaFuncSetAttribute(shared_finish_kernel<P::D, P::G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(shared_finish_kernel<P::D, P::G>, dim3((unsigned)(a.d.num_seqs * a.d.num_kv_heads)),
                      dim3(kFinThreads), smem, stream, args);
}

template <int D, int BS>
cudaError_t launch_shared_db(const SharedArgs& a, int group, cudaStream_t stream)
{
    switch (group) {
        case 1: return launch_shared_c<FmaConsumer<__nv_bfloat16, D, 16, 1>, BS>(a, group, stream);
        case 2: return launch_shared_c<MmaConsumer<D, 16, 2>, BS>(a, group, stream);
        case 4: return launch_shared_c<MmaConsumer<D, 16, 4>, BS>(a, group, stream);
        case 8: return launch_shared_c<MmaConsumer<D, 16, 8>, BS>(a, group, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_shared(const SharedArgs& a, int head_dim, int block_size, int group, cudaStream_t stream)
{
    if (head_dim == 64)
        return block_size == 16 ? launch_shared_db<64, 16>(a, group, stream) : launch_shared_db<64, 32>(a, group, stream);
    return block_size == 16 ? launch_shared_db<128, 16>(a, group, stream) : launch_shared_db<128, 32>(a, group, stream);
}

}  // namespace pa
