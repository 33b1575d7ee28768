// Eviction from the paged cache by accumulated attention weight, for sm_100a.
//
// What it computes, for every (sequence, kv head): of L cached tokens the n that stay are
// the recent ones (position within num_recent of the largest) and then those of the largest
// score, ties to the lowest slot.  The n first slots then hold them: a kept token before
// slot n stays where it is, and the kept tokens behind it move, in order, into the gaps the
// dropped ones leave.  Attention does not depend on the order of cached tokens (a key row
// carries its own position), so nothing else has to move: sum_s (gaps) rows are read and
// written instead of the whole kept context.  Sources (slots >= n) and destinations (slots
// < n) are disjoint, so the moves run in any order.
//
// Two kernels.  evict_select (one CTA per (sequence, kv head)) finds the n-th largest key by
// radix selection, 8 bits a pass, marks the kept tokens in a bit mask in shared memory, ranks
// gaps and movers by prefix sums over the mask's words, and writes the move list and the new
// scores and positions.  evict_move copies the K and V rows of the list.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

// Scores in an unsigned order: larger is better, -0 and +0 alike, NaN above +inf, and every
// recent token above all of them.
__device__ __forceinline__ uint32_t rank_key(float score, int pos, int first_recent)
{
    if (pos >= first_recent) return 0xffffffffu;
    if (score != score) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(score + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix sum of one value per thread over the CTA; *total receives the sum.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp,
                                                         unsigned long long* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        unsigned long long w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[kSelThreads / 32 - 1];
    const unsigned long long base = warp ? s_warp[warp - 1] : 0ull;
    __syncthreads();
    return base + x - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a)
{
    extern __shared__ uint32_t s_mask[];  // kept tokens, then (second half) the ties: one bit each
    __shared__ unsigned s_hist[256];
    __shared__ unsigned long long s_warp[kSelThreads / 32];
    __shared__ unsigned s_prefix, s_need;
    __shared__ int s_max[kSelThreads / 32];
    const int sh = blockIdx.x;
    const int s = sh / a.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L = __ldg(a.context_lens + s), n = __ldg(a.keep_lens + s);
    pdl_launch_dependents();
    if (L < 0 || n < 0 || L > a.max_context_len || L > a.max_blocks_per_seq * a.block_size) {
        if (tid == 0) {
            a.counts[sh] = 0;
            if (sh % a.num_kv_heads == 0) atomicOr(a.status, PA_DEV_BAD_CONTEXT);
        }
        return;
    }
    n = min(n, L);
    const size_t row = (size_t)sh * a.score_stride;
    const float* sc = a.scores + row;
    const int* pos = a.positions + row;
    float* nsc = a.new_scores + row;
    int* npos = a.new_positions + row;
    if (n == L || n == 0) {
        for (int i = tid; i < n; i += kSelThreads) {
            nsc[i] = sc[i];
            npos[i] = pos[i];
        }
        if (tid == 0) a.counts[sh] = 0;
        return;
    }
    // the recent tokens: positions within num_recent of the largest
    int mx = INT32_MIN;
    for (int i = tid; i < L; i += kSelThreads) mx = max(mx, pos[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
    mx = s_max[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const long long fr = (long long)mx - min(a.num_recent, n) + 1;
    const int first_recent = fr < (long long)INT32_MIN ? INT32_MIN : (int)fr;  // mx + 1 (none recent) needs fr > mx
    const bool none_recent = min(a.num_recent, n) == 0;
    auto key = [&](int i) {
        return none_recent ? rank_key(sc[i], -1, 0) : rank_key(sc[i], pos[i], first_recent);
    };
    // radix selection of the n-th largest key
    unsigned prefix = 0, need = (unsigned)n;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        const unsigned hi_mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i = tid; i < L; i += kSelThreads) {
            const uint32_t k = key(i);
            if ((k & hi_mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds bins 255 - 8l .. 248 - 8l, from the top
            unsigned c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[j] = s_hist[255 - 8 * lane - j];
            unsigned x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            unsigned above = x - sum;
            if (above < need && need <= x) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (above < need && need <= above + c[j]) {
                        s_prefix = prefix | ((unsigned)(255 - 8 * lane - j) << shift);
                        s_need = need - above;
                    }
                    above += c[j];
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        __syncthreads();
    }
    // masks of the keys above the threshold, and of those equal to it
    const int words = (L + 31) / 32;
    uint32_t* s_tie = s_mask + words;
    for (int w = warp; w < words; w += kSelThreads / 32) {
        const int i = w * 32 + lane;
        const uint32_t k = i < L ? key(i) : 0u;
        const uint32_t gt = __ballot_sync(0xffffffffu, i < L && k > prefix);
        const uint32_t eq = __ballot_sync(0xffffffffu, i < L && k == prefix);
        if (lane == 0) {
            s_mask[w] = gt;
            s_tie[w] = eq;
        }
    }
    __syncthreads();
    // the first `need` ties stay: every thread ranks a run of words
    const int per = (words + kSelThreads - 1) / kSelThreads;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    unsigned long long cnt = 0, total;
    for (int w = w0; w < w1; ++w) cnt += __popc(s_tie[w]);
    unsigned long long rank = block_scan(cnt, s_warp, &total);
    cnt = 0;
    for (int w = w0; w < w1; ++w) {
        uint32_t t = s_tie[w], take = 0;
        while (t && rank < need) {
            take |= t & (0u - t);
            t &= t - 1;
            ++rank;
        }
        const uint32_t kept = s_mask[w] | take;
        s_mask[w] = kept;
        const int below = n - w * 32;  // tokens of this word before slot n
        const uint32_t front = below >= 32 ? 0xffffffffu : (below <= 0 ? 0u : (1u << below) - 1u);
        cnt += (unsigned long long)__popc(~kept & front) | (unsigned long long)__popc(kept & ~front) << 32;
    }
    // gaps before slot n (low half) and kept tokens behind it (high half): as many of each
    rank = block_scan(cnt, s_warp, &total);
    uint2* moves = a.moves + (size_t)sh * a.move_stride;
    unsigned gap = (unsigned)rank, mover = (unsigned)(rank >> 32);
    for (int w = w0; w < w1; ++w) {
        const uint32_t kept = s_mask[w];
        const int below = n - w * 32;
        const uint32_t front = below >= 32 ? 0xffffffffu : (below <= 0 ? 0u : (1u << below) - 1u);
        for (uint32_t b = ~kept & front; b; b &= b - 1) moves[gap++].x = (unsigned)(w * 32 + __ffs(b) - 1);
        for (uint32_t b = kept & ~front; b; b &= b - 1) moves[mover++].y = (unsigned)(w * 32 + __ffs(b) - 1);
    }
    if (tid == 0) a.counts[sh] = (unsigned)total;
    __syncthreads();
    // the scores and positions of the slots before n (these arrays may be the old ones: a slot
    // before n is only ever written with its own value or one from behind n)
    for (int i = tid; i < n; i += kSelThreads)
        if (s_mask[i / 32] >> (i % 32) & 1u) {
            nsc[i] = sc[i];
            npos[i] = pos[i];
        }
    for (unsigned r = tid; r < (unsigned)total; r += kSelThreads) {
        const uint2 m = moves[r];
        nsc[m.x] = sc[m.y];
        npos[m.x] = pos[m.y];
    }
}

// CPR threads per row (16 bytes each), the K and the V row of a move together.
template <int CPR>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int splits)
{
    pdl_wait_primary();
    constexpr int RPI = kMoveThreads / CPR;  // moves per step of the CTA
    const int sh = blockIdx.x / splits, part = blockIdx.x % splits;
    const int s = sh / a.num_kv_heads, kvh = sh % a.num_kv_heads;
    const unsigned count = __ldg(a.counts + sh);
    const uint2* moves = a.moves + (size_t)sh * a.move_stride;
    const int32_t* table = a.block_tables + (size_t)s * a.max_blocks_per_seq;
    const int c = threadIdx.x % CPR;
    uint4* kc = static_cast<uint4*>(a.k_cache);
    uint4* vc = static_cast<uint4*>(a.v_cache);
    auto row_of = [&](unsigned tok, bool& ok) -> size_t {
        const int b = __ldg(table + tok / (unsigned)a.block_size);
        if ((unsigned)b >= (unsigned)a.num_blocks) {
            if (c == 0) atomicOr(a.status, PA_DEV_BAD_BLOCK);
            ok = false;
            return 0;
        }
        return (((size_t)b * a.num_kv_heads + kvh) * a.block_size + tok % (unsigned)a.block_size) * CPR + c;
    };
    for (unsigned r = part * RPI + threadIdx.x / CPR; r < count; r += splits * RPI) {
        const uint2 m = __ldg(moves + r);
        bool ok = true;
        const size_t dst = row_of(m.x, ok), src = row_of(m.y, ok);
        if (ok) {
            const uint4 kv = kc[src], vv = vc[src];
            kc[dst] = kv;
            vc[dst] = vv;
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int head_dim, int elt_bytes, cudaStream_t stream)
{
    const int rows = a.num_seqs * a.num_kv_heads;
    const size_t smem = (size_t)((a.max_context_len + 31) / 32) * 8;
    cudaError_t e;
    if (smem > 40 * 1024) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    evict_select_kernel<<<rows, kSelThreads, smem, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // enough CTAs to fill the device, but none with less than one step of the longest list
    const int cpr = head_dim * elt_bytes / 16;
    const int steps = (a.move_stride + kMoveThreads / cpr - 1) / (kMoveThreads / cpr);
    int splits = (148 * 16 + rows - 1) / rows;
    splits = splits < steps ? splits : steps;
    splits = splits < 1 ? 1 : splits;
    const dim3 grid((unsigned)rows * (unsigned)splits);
    switch (cpr) {
        case 8: return launch_pdl(evict_move_kernel<8>, grid, dim3(kMoveThreads), 0, stream, a, splits);
        case 16: return launch_pdl(evict_move_kernel<16>, grid, dim3(kMoveThreads), 0, stream, a, splits);
        case 32: return launch_pdl(evict_move_kernel<32>, grid, dim3(kMoveThreads), 0, stream, a, splits);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
