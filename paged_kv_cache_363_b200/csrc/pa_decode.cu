// Paged decode attention for sm_100a.
//
// What it computes ("PagedAttention and vLLM Architecture", section 2, "PagedAttention
// Attention CUDA Kernel Mechanics"): for each sequence's single new query, walk the
// physical blocks named by the block table in logical order, dot q with every key of
// each gathered block, keep an online softmax (running max and sum) across blocks and
// fold the weighted V rows of the same blocks into the output in the same pass.
// Token i of a sequence lives in physical block T[i / B] at offset i % B
// ("PagedAttention Paper Breakdown", section 2, Address Translation Formula).
//
// B200 design:
//  * Work units are (sequence, context partition, kv head).  All query heads of the
//    kv head's group are packed into one unit, so each K/V byte leaves HBM once.
//  * A plan kernel lists the (sequence, partition) pairs longest first; a persistent
//    kernel (a few CTAs per SM) takes units from that list with an atomic counter, so
//    the grid holds no empty CTAs and the short units are the ones left at the end.
//  * In each CTA one warp fetches units ahead of use (block-table slice and q into a
//    small shared ring), one thread streams the units' K/V tiles into a ring of
//    shared-memory stages with the TMA engine (1-D bulk copies of whole tiles, or 2-D
//    tensor boxes with the 128-byte swizzle for the tensor-core consumer; each CTA
//    loads its own tiles) and four consumer warps take alternate blocks.  The stream of tiles
//    runs across unit boundaries, so the pipeline does not drain between units.
//  * Consumers: CUDA cores (fp32; bf16 with one query head per kv head) or tensor
//    cores (bf16 with 2, 4 or 8 query heads per kv head); see the two policy headers.
//  * At the end of a unit each warp leaves its softmax state in shared memory and goes
//    on with the next unit; the warp that consumed the unit's last tile merges the four
//    states.  A sequence longer than one partition leaves (max, sum, unnormalised
//    output) per partition in the workspace and a log-sum-exp merge kernel combines
//    them.  Plan, persistent and merge kernels are chained with programmatic dependent
//    launch.
//  * The first wave of CTAs does not wait for the plan: when the partition length is
//    fixed, CTA b starts on partition 0 of sequence b / Hkv (kv head b % Hkv), which
//    the plan lists at position b / Hkv, while the plan kernel still runs.
//  * Logits are kept in base-2 units (q pre-scaled by scale*log2 e) and exponentials
//    use exp2f, the reformulation of online softmax by Milakov & Gimelshein (2018).
//  * Every wait is bounded: a wait that runs out raises PA_DEV_WAIT_TIMEOUT and the
//    CTA winds down instead of hanging.  Bad block indices or context lengths raise a
//    status bit and are clamped instead of being dereferenced.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "pa_decode_persist.cuh"
#include "pa_internal.h"

namespace pa {

// ---------------------------------------------------------------- tensor maps

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

unsigned long long current_context_id()
{
    using GetCurrent = CUresult (*)(CUcontext*);
    using GetId = CUresult (*)(CUcontext, unsigned long long*);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<GetCurrent>(p);
        p = nullptr;
        if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<GetId>(p);
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// The pool [num_blocks][kv_heads][B][D] as a 2-D bf16 tensor of rows of D elements;
// boxes of 64 columns x `B` rows (one stage tile), 128-byte swizzle.
cudaError_t encode_pool_map(CUtensorMap* out, const void* pool, uint64_t rows, int D, int B)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    std::memset(out, 0, sizeof(*out));
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)B};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_pool_atoms(CUtensorMap* out, const void* pool, uint64_t rows, int D, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    std::memset(out, 0, sizeof(*out));
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)D / 64, (cuuint64_t)rows / 8};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)box_rows / 8};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// encode_pool_map's maps from a small cache, which avoids re-encoding the maps of the same pools on every call.
cudaError_t tensor_map(CUtensorMap* out, const void* pool, uint64_t rows, int D, int B)
{
    struct Entry {
        const void* ptr;
        uint64_t rows;
        int d, b, dev;
        CUtensorMap map;
    };
    static std::mutex mu;
    static Entry cache[16] = {};
    static int next = 0;
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess) return ce;
    {
        std::lock_guard<std::mutex> lk(mu);
        for (auto& en : cache)
            if (en.ptr == pool && en.rows == rows && en.d == D && en.b == B && en.dev == dev) {
                *out = en.map;
                return cudaSuccess;
            }
    }
    CUtensorMap m;
    ce = encode_pool_map(&m, pool, rows, D, B);
    if (ce != cudaSuccess) return ce;
    std::lock_guard<std::mutex> lk(mu);
    Entry& en = cache[next];
    next = (next + 1) % 16;
    en.ptr = pool;
    en.rows = rows;
    en.d = D;
    en.b = B;
    en.dev = dev;
    en.map = m;
    *out = m;
    return cudaSuccess;
}

bool decode_uses_tensor_cores(pa_dtype dtype, int head_dim, int group)
{
    return dtype == PA_DTYPE_BF16 && (head_dim == 64 || head_dim == 128) && (group == 2 || group == 4 || group == 8);
}

cudaError_t launch_decode(const DecodeArgs& a, pa_dtype dtype, int head_dim, int block_size, int group,
                          cudaStream_t stream)
{
    if (dtype == PA_DTYPE_F32) return dispatch_dim<float, kModePlain>(a, head_dim, block_size, group, stream);
    return dispatch_dim<__nv_bfloat16, kModePlain>(a, head_dim, block_size, group, stream);
}

}  // namespace pa
