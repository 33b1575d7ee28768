// Decode attention of a batch in groups whose sequences share leading blocks, for sm_100a.
//
// What it computes: pa_decode's output.  Row s of group g attends to the group's n_g shared
// tokens and to its own tokens n_g .. L_s - 1; the softmax over both is joined from the two
// partial states (m, l, O) = (maximum, sum of 2^(x - m), weighted V):
//   out = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p,  M = max m_p.
// The shared tokens of a kv head are one dense product of all the group's rows x G query
// heads with the same K and V: the tensor-core kernel of pa_group.cu reads each shared byte
// once per 128 rows, where pa_decode reads it once per sequence (from L2 when it is lucky).
// The own tokens go through pa_decode's persistent kernel, from the block behind the shared
// ones.  The two write partial states side by side and a merge joins them.
//
// Four kernels: a plan (below), the shared tokens, the own tokens, the merge.  The own tokens'
// kernel needs the plan alone, so the shared tokens' kernel lets it start once it has itself
// seen the plan finish, and the CTAs of both share the device until the work is gone.
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

// The plan, in one CTA.
//  1. Groups are checked (starts in order, rows in range and listed once, whole blocks, no more
//     tokens than any member's context).  A bad one raises PA_DEV_BAD_CONTEXT and is not
//     shared: its rows attend to all their tokens on their own, which is the same result.
//  2. Entries of the shared tokens: (tile of 128 / G rows, chunk), a chunk's tiles next to each
//     other.  The chunk length is the work over twice the resident CTAs, at least 256 tokens.
//  3. The own tokens' list, longest first, as pa_decode's plan makes it, each entry with the
//     blocks before it and the number of shared states (which makes it write its own state).
//  4. The rows to merge.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs a, int group, int group_ctas)
{
    __shared__ int bucket[kMaxPartitionTokens / 16 + 1];
    __shared__ unsigned long long s_work, s_tok;
    __shared__ unsigned s_items, s_merges;
    __shared__ int s_bad, s_max, s_pb;
    pdl_launch_dependents();
    const DecodeArgs& d = a.d;
    const int B = a.g.block_size, T = 128 / group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        s_work = s_tok = 0;
        s_items = s_merges = 0;
        s_bad = s_max = 0;
    }
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        a.listed[s] = 0;
        a.lead_blocks[s] = 0;
        a.lead_states[s] = 0;
    }
    __syncthreads();
    for (int g = tid; g < a.num_groups; g += kPlanThreads) {
        const int r0 = __ldg(a.group_start + g), r1 = __ldg(a.group_start + g + 1);
        if (r0 < 0 || r1 < r0 || r1 > a.num_group_rows) s_bad = 1;
    }
    for (int i = tid; i < a.num_group_rows; i += kPlanThreads) {
        const int s = __ldg(a.group_rows + i);
        if ((unsigned)s < (unsigned)d.num_seqs) atomicAdd(a.listed + s, 1);
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
            ok = ok && __ldcg(a.listed + s) == 1 && n <= clamped_context(d, s, B, false);
        }
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (lane == 0) {
            a.group_ok[g] = ok && n > 0 && r1 > r0;
            if (!ok) atomicOr(d.status, PA_DEV_BAD_CONTEXT);
            else if (n > 0) atomicAdd(&s_work, (unsigned long long)((r1 - r0 + T - 1) / T) * n);
        }
    }
    __syncthreads();
    {
        const unsigned long long share = s_work * d.num_kv_heads / (2ull * group_ctas);
        const int least = (a.max_shared_len + a.max_chunks - 1) / a.max_chunks;
        const int chunk = (max(max((int)min(share, 1ull << 30), least), 256) + 63) / 64 * 64;
        GroupItem* items = const_cast<GroupItem*>(a.g.items);
        for (int g = warp; g < ngroups; g += kPlanThreads / 32) {
            if (!a.group_ok[g]) continue;
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
                a.lead_blocks[s] = n / B;
                a.lead_states[s] = nch;
            }
        }
    }
    // ---- the own tokens
    __syncthreads();
    auto own_len = [&](int s, bool flag) {
        return max(0, clamped_context(d, s, B, flag) - __ldcg(a.lead_blocks + s) * B);
    };
    unsigned long long tok = 0;
    int lmax = 0;
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        const int L = own_len(s, true);
        tok += (unsigned long long)L;
        lmax = max(lmax, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        tok += __shfl_xor_sync(0xffffffffu, tok, o);
        lmax = max(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    }
    if (lane == 0) {
        atomicAdd(&s_tok, tok);
        atomicMax(&s_max, lmax);
    }
    __syncthreads();
    if (tid == 0) {
        int pb = d.partition_blocks;
        const int max_pb = kMaxPartitionTokens / B;
        const double share = (double)s_tok / (double)(d.num_ctas > 0 ? d.num_ctas : 1);
        while (2 * pb <= max_pb && pb * B < s_max && (double)min(2 * pb * B, s_max) * 4.0 <= share) pb *= 2;
        s_pb = pb;
        d.plan[2] = (unsigned)pb;
    }
    __syncthreads();
    const int pb = s_pb, P = pb * B;
    for (int i = tid; i <= pb; i += kPlanThreads) bucket[i] = 0;
    __syncthreads();
    // partitions of a sequence: none when the shared tokens are all it has, one when it has no token
    auto parts = [&](int s, int L) { return L > 0 ? (L + P - 1) / P : (__ldcg(a.lead_states + s) > 0 ? 0 : 1); };
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        const int L = own_len(s, false), np = parts(s, L), lead = __ldcg(a.lead_states + s);
        if (np > 0) {
            const int last = L > 0 ? (L - (np - 1) * P + B - 1) / B : 0;
            if (np > 1) atomicAdd(&bucket[pb], np - 1);
            atomicAdd(&bucket[last], 1);
        }
        if (lead > 0 || np > 1)
            const_cast<uint2*>(a.g.merge_list)[atomicAdd(&s_merges, 1u)] =
                make_uint2((unsigned)s, (unsigned)lead | (unsigned)np << 16);
    }
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
        if (lane == 0) {
            d.plan[0] = 0u;
            d.plan[4] = 0u;
            d.plan[1] = (unsigned)running;
            unsigned* counts = const_cast<unsigned*>(a.g.counts);
            counts[0] = s_items;
            counts[1] = s_merges;
        }
    }
    __syncthreads();
    uint4* list = reinterpret_cast<uint4*>(d.plan_list);
    for (int s = tid; s < d.num_seqs; s += kPlanThreads) {
        const int L = own_len(s, false), np = parts(s, L);
        const int last = L > 0 ? (L - (np - 1) * P + B - 1) / B : 0;
        const unsigned lead = (unsigned)__ldcg(a.lead_states + s), blocks = (unsigned)__ldcg(a.lead_blocks + s);
        for (int p = 0; p < np; ++p) {
            const int pos = atomicAdd(&bucket[p < np - 1 ? pb : last], 1);
            list[pos] = make_uint4(((unsigned)s << 11) | (unsigned)p, (unsigned)(blocks * B + L), blocks, lead);
        }
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
    shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(args, group, group_resident_ctas(sms));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (shares && (e = launch_group(args.g, P::D, group, stream)) != cudaSuccess) return e;
    e = launch_pdl(decode_persistent_kernel<Cons, BS, kModeOwn>, dim3(grid), dim3(P::THREADS), (size_t)P::SMEM, stream,
                   args.d, tk, tv);
    if (e != cudaSuccess) return e;
    return launch_group_merge(args.g, P::D, stream);
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
