// Paged decode attention that also adds every token's attention weight to a running score
// per (sequence, kv head, token), the statistic pa_evict ranks tokens by.
//
// What it computes: with x = scale * q_h . K_i in base-2 units, M_h the row's maximum and
// l_h = sum_i 2^(x_i - M_h), the output is pa_decode's and the weight of token i is
//   w_i = sum over the kv head's query heads of 2^(x_i - M_h) / l_h .
// A weight needs the whole row's maximum and sum, which one pass over the keys has only at
// its end.  Reading K again for it would cost half of the K/V traffic once more.  Instead
// the decode kernel writes each logit it has in registers (4 bytes per query head and token
// beside the 2 * D * elt bytes of K and V it has just read: 3 % for bf16 with D = 128 and a
// group of 4), and a second kernel, below, turns logits into weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_persist.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kScoreThreads = 256;

// One (sequence, partition) of the plan and one kv head at a time: the row statistics of
// the group's heads from the partitions' (max, sum) pairs, a warp per head, then a token
// per thread.  The heads are added in order, so a score's bits do not depend on the grid.
template <int G>
__global__ void __launch_bounds__(kScoreThreads) decode_scores_kernel(const DecodeArgs a, int block_size)
{
    __shared__ float s_m[G], s_inv[G];
    pdl_wait_primary();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int P = (int)__ldg(a.plan + 2) * block_size;
    const unsigned units = __ldg(a.plan + 1) * (unsigned)a.num_kv_heads;
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
        const uint2 e = __ldg(a.plan_list + u / (unsigned)a.num_kv_heads);
        const int kvh = (int)(u % (unsigned)a.num_kv_heads);
        const int s = (int)(e.x >> 11), L = (int)e.y;
        const int lo = (int)(e.x & 2047u) * P, hi = min(L, lo + P);
        if (warp < G) {
            const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) +
                               ((size_t)s * a.num_heads + (size_t)kvh * G + warp) * a.num_partitions;
            const int np = (L + P - 1) / P;
            float M = -INFINITY, l = 0.f;
            for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldg(&ml[p].x));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            for (int p = lane; p < np; p += 32) {
                const float2 v = __ldg(ml + p);
                if (v.x != -INFINITY) l = fmaf(exp2f(v.x - M), v.y, l);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) {
                s_m[warp] = M;
                s_inv[warp] = l > 0.f ? 1.f / l : 0.f;
            }
        }
        __syncthreads();
        const float* lg = a.logits + ((size_t)s * a.num_kv_heads + kvh) * a.max_context_len * G;
        float* sc = a.scores + ((size_t)s * a.num_kv_heads + kvh) * a.score_stride;
        for (int i = lo + (int)threadIdx.x; i < hi; i += kScoreThreads) {
            const float* x = lg + (size_t)i * G;
            float w = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) w = fmaf(exp2f(__ldg(x + g) - s_m[g]), s_inv[g], w);
            sc[i] = i == L - 1 ? w : sc[i] + w;  // the step's own token has no history
        }
        __syncthreads();
    }
}

template <int G>
cudaError_t launch_scores(const DecodeArgs& a, int block_size, cudaStream_t stream)
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t units = (int64_t)a.num_seqs * a.num_partitions * a.num_kv_heads;
    const unsigned grid = (unsigned)(units < 8LL * sms ? units : 8LL * sms);
    return launch_pdl(decode_scores_kernel<G>, dim3(grid), dim3(kScoreThreads), 0, stream, a, block_size);
}

}  // namespace

cudaError_t launch_decode_scores(const DecodeArgs& a, pa_dtype dtype, int head_dim, int block_size, int group,
                                 cudaStream_t stream)
{
    const cudaError_t e = dtype == PA_DTYPE_F32
                              ? dispatch_dim<float, kModeScores>(a, head_dim, block_size, group, stream)
                              : dispatch_dim<__nv_bfloat16, kModeScores>(a, head_dim, block_size, group, stream);
    if (e != cudaSuccess) return e;
    switch (group) {
        case 1: return launch_scores<1>(a, block_size, stream);
        case 2: return launch_scores<2>(a, block_size, stream);
        case 4: return launch_scores<4>(a, block_size, stream);
        case 8: return launch_scores<8>(a, block_size, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
