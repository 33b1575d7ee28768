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
// group of 4), and a second kernel, below, turns logits into weights and joins split
// sequences' partial outputs at the same time.  A small batch, whose every unit is a whole
// sequence and has a CTA, needs neither that kernel nor a plan: one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_persist.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kScoreThreads = 256;

// The first `mblocks` blocks join the split sequences' partial outputs, nwr warps per (sequence, query head), as
// decode_merge_kernel does: the same chunks of 8 partitions to the same sums, added in the same order, so the
// same bits.  The others take one partition and kv head of a sequence at a time: a warp per head takes the
// row statistics from the partitions' (max, sum) pairs, then a token per thread.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreThreads, 6) decode_scores_kernel(const DecodeArgs a, int block_size, int nwr, int mblocks)
{
    constexpr int EPL = D / 32, CH = 8, NW = kScoreThreads / 32;
    __shared__ float s_m[G], s_inv[G];
    __shared__ float s_num[NW][D], s_den[NW];
    pdl_wait_primary();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int P = (int)__ldg(a.plan + 2) * block_size;
    if ((int)blockIdx.x < mblocks) {
        const int H = a.num_heads, rows = (int)__ldg(a.plan + 3) * H;
        const int rpc = NW / nwr, sub = warp % nwr;
        for (int r0 = blockIdx.x * rpc; r0 < rows; r0 += mblocks * rpc) {
            const int r = r0 + warp / nwr;
            float num[EPL], den = 0.f;
#pragma unroll
            for (int k = 0; k < EPL; ++k) num[k] = 0.f;
            size_t row = 0;
            if (r < rows) {
                const uint2 e = __ldg(a.split_list + r / H);
                const int np = ((int)e.y + P - 1) / P;
                row = (size_t)e.x * H + r % H;
                const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * a.num_partitions;
                const float* acc = a.ws_acc + row * a.num_partitions * D + lane * EPL;
                float M = -INFINITY;
                for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldg(&ml[p].x));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                for (int c = sub; c * CH < np; c += nwr) {
                    float x[CH][EPL];
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const float* src = acc + (size_t)min(c * CH + i, np - 1) * D;
                        if constexpr (EPL == 4)
                            *reinterpret_cast<float4*>(x[i]) = __ldg(reinterpret_cast<const float4*>(src));
                        else
                            *reinterpret_cast<float2*>(x[i]) = __ldg(reinterpret_cast<const float2*>(src));
                    }
                    const int pw = c * CH + (lane & (CH - 1));
                    float wt = 0.f;
                    if (lane < CH && pw < np) {
                        const float2 v = __ldg(ml + pw);
                        wt = v.x == -INFINITY ? 0.f : exp2f(v.x - M);
                        den = fmaf(wt, v.y, den);
                    }
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const float wi = __shfl_sync(0xffffffffu, wt, i);
#pragma unroll
                        for (int k = 0; k < EPL; ++k) num[k] = fmaf(wi, x[i][k], num[k]);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
            }
#pragma unroll
            for (int k = 0; k < EPL; ++k) s_num[warp][lane * EPL + k] = num[k];
            if (lane == 0) s_den[warp] = den;
            __syncthreads();
            if (r < rows && sub == 0) {
                for (int j = 1; j < nwr; ++j) {
#pragma unroll
                    for (int k = 0; k < EPL; ++k) num[k] += s_num[warp + j][lane * EPL + k];
                    den += s_den[warp + j];
                }
                const float inv = den > 0.f ? 1.f / den : 0.f;
                T* o = static_cast<T*>(a.out) + row * D + lane * EPL;
#pragma unroll
                for (int k = 0; k < EPL; ++k) o[k] = from_f32<T>(num[k] * inv);
            }
            __syncthreads();
        }
        return;
    }
    const unsigned units = __ldg(a.plan + 1) * (unsigned)a.num_kv_heads;
    for (unsigned u = blockIdx.x - mblocks; u < units; u += gridDim.x - mblocks) {
        const uint2 e = __ldg(a.plan_list + u / (unsigned)a.num_kv_heads);
        const int kvh = (int)(u % (unsigned)a.num_kv_heads);
        const int s = (int)(e.x >> 11), L = (int)e.y;
        const int lo = (int)(e.x & 2047u) * P, hi = min(L, lo + P);
        const size_t srow = (size_t)s * a.num_kv_heads + kvh;
        const float* lg = a.logits + srow * a.max_context_len * G;
        float* sc = a.scores + srow * a.score_stride;
        WeightTokens<G, kScoreThreads, 2> w;  // on their way while the statistics are taken
        w.load(lg, sc, lo, hi, threadIdx.x);
        if (warp < G) {
            const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) +
                               ((size_t)s * a.num_heads + (size_t)kvh * G + warp) * a.num_partitions;
            const int np = (L + P - 1) / P;
            float2 v = make_float2(-INFINITY, 0.f);  // the lane's partitions, joined
            for (int p = lane; p < np; p += 32) {
                const float2 x = __ldg(ml + p);
                const float M = fmaxf(v.x, x.x);
                if (M != -INFINITY) v = make_float2(M, v.y * exp2f(v.x - M) + x.y * exp2f(x.x - M));
            }
            float M = v.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            float l = v.x == -INFINITY ? 0.f : v.y * exp2f(v.x - M);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) {
                s_m[warp] = M;
                s_inv[warp] = l > 0.f ? 1.f / l : 0.f;
            }
        }
        __syncthreads();
        w.add(sc, lo, hi, L, threadIdx.x, s_m, s_inv);
        for (int i = lo + 2 * kScoreThreads; i < hi; i += 2 * kScoreThreads) {
            w.load(lg, sc, i, hi, threadIdx.x);
            w.add(sc, i, hi, L, threadIdx.x, s_m, s_inv);
        }
        __syncthreads();
    }
}

template <typename T, int D, int G>
cudaError_t launch_scores(const DecodeArgs& a, int block_size, cudaStream_t stream)
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t units = (int64_t)a.num_seqs * a.num_partitions * a.num_kv_heads;
    const unsigned grid = (unsigned)(units < 8LL * sms ? units : 8LL * sms);
    const int nwr = a.num_partitions <= 8 ? 1 : (a.num_partitions <= 16 ? 2 : 4);  // as launch_merge
    const int64_t rows = a.num_partitions > 1 ? ((int64_t)a.num_seqs * a.num_heads * nwr + 7) / 8 : 0;
    const int mblocks = (int)(rows < 4LL * sms ? rows : 4LL * sms);
    return launch_pdl(decode_scores_kernel<T, D, G>, dim3(grid + mblocks), dim3(kScoreThreads), 0, stream, a, block_size, nwr,
                      mblocks);
}

template <typename T, int D>
cudaError_t launch_scores_td(const DecodeArgs& a, int block_size, int group, cudaStream_t stream)
{
    switch (group) {
        case 1: return launch_scores<T, D, 1>(a, block_size, stream);
        case 2: return launch_scores<T, D, 2>(a, block_size, stream);
        case 4: return launch_scores<T, D, 4>(a, block_size, stream);
        case 8: return launch_scores<T, D, 8>(a, block_size, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t launch_scores_t(const DecodeArgs& a, int head_dim, int block_size, int group, cudaStream_t stream)
{
    return head_dim == 64 ? launch_scores_td<T, 64>(a, block_size, group, stream)
                          : launch_scores_td<T, 128>(a, block_size, group, stream);
}

}  // namespace

cudaError_t launch_decode_scores(const DecodeArgs& a, pa_dtype dtype, int head_dim, int block_size, int group,
                                 cudaStream_t stream)
{
    const bool f32 = dtype == PA_DTYPE_F32;
    int planless = 0;
    DecodeArgs d = a;
    d.was_planless = &planless;
    const cudaError_t e = f32 ? dispatch_dim<float, kModeScores>(d, head_dim, block_size, group, stream)
                              : dispatch_dim<__nv_bfloat16, kModeScores>(d, head_dim, block_size, group, stream);
    if (e != cudaSuccess || planless) return e;
    return f32 ? launch_scores_t<float>(a, head_dim, block_size, group, stream)
               : launch_scores_t<__nv_bfloat16>(a, head_dim, block_size, group, stream);
}

}  // namespace pa
