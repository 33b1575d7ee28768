// C ABI of libpa.so (declared in include/pa.h): argument validation, dispatch to
// the kernels, the device status word, and the per-thread error message.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "pa.h"
#include "pa_group.cuh"
#include "pa_internal.h"
#include "pa_shared.h"

namespace pa {

static thread_local std::string g_err;

void set_error(const std::string& msg) { g_err = msg; }

namespace {

// Device status word: kernels OR PA_DEV_* bits into it.  Host code reaches it
// through its per-device address (the symbol itself is only a host-side handle).
__device__ unsigned int g_status_word;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned int* g_status_ptr[kMaxDevices] = {};
unsigned long long g_status_ctx[kMaxDevices] = {};  // context id each cached address belongs to

pa_status cuda_fail(const char* what, cudaError_t e)
{
    set_error(std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
    return PA_ERR_CUDA;
}

// Address of the status word on the current device: resolved once per device and
// context, and again after a device reset has re-created the context.
pa_status status_ptr(unsigned int** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) {
        set_error("device index out of range");
        return PA_ERR_INVALID;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    const unsigned long long ctx = current_context_id();
    if (!g_status_ptr[dev] || ctx == 0 || g_status_ctx[dev] != ctx) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_status_word);
        if (e != cudaSuccess) return cuda_fail("cudaGetSymbolAddress(status word)", e);
        g_status_ptr[dev] = static_cast<unsigned int*>(p);
        g_status_ctx[dev] = current_context_id();  // current now, if it was not before the lookup
    }
    *out = g_status_ptr[dev];
    return PA_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elt_bytes(pa_dtype dt) { return dt == PA_DTYPE_F32 ? 4 : 2; }

pa_status check_common(const char* fn, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                       pa_dtype dtype)
{
    if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) {
        set_error(std::string(fn) + ": dtype must be PA_DTYPE_F32 or PA_DTYPE_BF16");
        return PA_ERR_UNSUPPORTED;
    }
    if (head_dim != 64 && head_dim != 128) {
        set_error(std::string(fn) + ": head_dim must be 64 or 128");
        return PA_ERR_UNSUPPORTED;
    }
    if (block_size != 16 && block_size != 32) {
        set_error(std::string(fn) + ": block_size must be 16 or 32");
        return PA_ERR_UNSUPPORTED;
    }
    if (num_kv_heads <= 0 || num_kv_heads > 65535 || num_blocks <= 0) {
        set_error(std::string(fn) + ": num_kv_heads and num_blocks must be > 0 (num_kv_heads <= 65535)");
        return PA_ERR_INVALID;
    }
    return PA_OK;
}

constexpr int kAutoPartitionTokens = 512;

// Partition tokens for the arguments, or a negative pa_status.
int resolve_partition(int block_size, int max_context_len, int partition_size)
{
    int p = partition_size > 0 ? partition_size : kAutoPartitionTokens;
    if (p % block_size != 0 || p > kMaxPartitionTokens) {
        set_error("partition_size must be a multiple of block_size and at most " +
                  std::to_string(kMaxPartitionTokens));
        return PA_ERR_INVALID;
    }
    const long np = ((long)max_context_len + p - 1) / p;
    if (np > kMaxPartitions) {
        set_error("max_context_len / partition_size exceeds " + std::to_string(kMaxPartitions) +
                  " partitions; use a larger partition_size");
        return PA_ERR_UNSUPPORTED;
    }
    return p;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

const char* pa_last_error_string(void) { return g_err.c_str(); }

int pa_decode_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int max_context_len, int partition_size)
{
    (void)num_seqs;
    (void)num_heads;
    (void)num_kv_heads;
    (void)head_dim;
    if (block_size != 16 && block_size != 32) {
        set_error("pa_decode_partition_size: block_size must be 16 or 32");
        return PA_ERR_UNSUPPORTED;
    }
    if (max_context_len < 0 || partition_size < 0) {
        set_error("pa_decode_partition_size: negative size");
        return PA_ERR_INVALID;
    }
    return resolve_partition(block_size, max_context_len, partition_size);
}

size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                int max_context_len, int partition_size)
{
    const int p = pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                           max_context_len, partition_size);
    if (p <= 0 || num_seqs <= 0 || num_heads <= 0 || head_dim <= 0) return 0;
    const size_t np = max_context_len > 0 ? ((size_t)max_context_len + p - 1) / p : 1;
    return decode_workspace((size_t)num_seqs, (size_t)num_heads, (size_t)head_dim, np).total;
}

}  // extern "C"

namespace pa {
namespace {

// pa_decode, pa_decode_plan and pa_decode_run: the same checks and arguments, then the
// plan kernel, the persistent kernel and merge, or both.  The plan phase does not
// touch out, q or the caches (they may be null).
pa_status decode_call(const char* fn, int phases, void* out, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                      int num_blocks, int max_context_len, float scale, int partition_size, void* workspace,
                      size_t workspace_bytes, pa_dtype dtype, void* stream, bool with_scores = false,
                      float* scores = nullptr, int score_stride = 0)
{
    const char* const name = fn;
    auto set_error = [name](const std::string& msg) { pa::set_error(std::string(name) + msg); };
    pa_status st = check_common(fn, num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || num_seqs > 65535 || num_heads <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
        partition_size < 0 || !std::isfinite(scale)) {
        set_error(": bad size or scale");
        return PA_ERR_INVALID;
    }
    if (num_heads % num_kv_heads != 0) {
        set_error(": num_heads must be a multiple of num_kv_heads");
        return PA_ERR_INVALID;
    }
    const int group = num_heads / num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) {
        set_error(": num_heads / num_kv_heads must be 1, 2, 4 or 8");
        return PA_ERR_UNSUPPORTED;
    }
    if (with_scores && score_stride < max_context_len) {
        set_error(": score_stride must be at least max_context_len");
        return PA_ERR_INVALID;
    }
    if (num_seqs == 0) return PA_OK;
    const bool run = (phases & kDecodeRun) != 0;
    if ((run && (!out || !q || !k_cache || !v_cache)) || (with_scores && !scores && max_context_len > 0) || !block_tables || !context_lens) {
        set_error(": null pointer");
        return PA_ERR_INVALID;
    }
    if ((run && (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(scores, 4)) {
        set_error(": misaligned pointer (q, out, caches need 16 bytes)");
        return PA_ERR_INVALID;
    }
    if (decode_uses_tensor_cores(dtype, head_dim, group) &&
        (int64_t)num_blocks * num_kv_heads * block_size > (int64_t)INT32_MAX) {
        set_error(": num_blocks * num_kv_heads * block_size must stay below 2^31 (tensor-copy row index)");
        return PA_ERR_UNSUPPORTED;
    }
    const int p = resolve_partition(block_size, max_context_len, partition_size);
    if (p < 0) return (pa_status)p;
    const int np = max_context_len > 0 ? (max_context_len + p - 1) / p : 1;
    const ScoresWorkspace sl =
        scores_workspace((size_t)num_seqs, (size_t)num_heads, (size_t)head_dim, (size_t)np, (size_t)max_context_len);
    const DecodeWorkspace& wl = sl.d;
    const size_t need = with_scores ? sl.total : wl.total;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) {
        set_error(": workspace missing, too small (need " + std::to_string(need) +
                  " bytes) or not 16-byte aligned");
        return PA_ERR_INVALID;
    }
    DecodeArgs a{};
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.plan = reinterpret_cast<unsigned int*>(ws + wl.plan);
    a.plan_list = reinterpret_cast<uint2*>(ws + wl.list);
    a.split_list = reinterpret_cast<uint2*>(ws + wl.splits);
    if (np > 1) {
        a.ws_acc = reinterpret_cast<float*>(ws + wl.acc);
        a.ws_ml = reinterpret_cast<float*>(ws + wl.ml);
    }
    if (with_scores) {
        a.ws_ml = reinterpret_cast<float*>(ws + sl.ml);
        a.logits = reinterpret_cast<float*>(ws + sl.logits);
        a.scores = scores;
        a.score_stride = score_stride;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = status;
    a.num_seqs = num_seqs;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.max_context_len = max_context_len;
    a.partition_blocks = p / block_size;
    a.adaptive = partition_size == 0 ? 1 : 0;
    a.num_partitions = np;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.phases = phases;
    const cudaError_t e = (with_scores ? launch_decode_scores : launch_decode)(a, dtype, head_dim, block_size,
                                                                               group, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail((std::string(name) + " launch").c_str(), e);
    return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_heads,
                    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                    int max_context_len, float scale, int partition_size, void* workspace,
                    size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_decode");
    return decode_call("pa_decode", kDecodePlan | kDecodeRun, out, q, k_cache, v_cache, block_tables, context_lens,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                       max_context_len, scale, partition_size, workspace, workspace_bytes, dtype, stream);
}

pa_status pa_decode_plan(const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_heads,
                         int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                         int max_context_len, int partition_size, void* workspace, size_t workspace_bytes,
                         pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_decode_plan");
    return decode_call("pa_decode_plan", kDecodePlan, nullptr, nullptr, nullptr, nullptr, block_tables, context_lens,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                       max_context_len, 1.0f, partition_size, workspace, workspace_bytes, dtype, stream);
}

pa_status pa_decode_run(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_heads,
                        int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                        int max_context_len, float scale, int partition_size, void* workspace,
                        size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_decode_run");
    return decode_call("pa_decode_run", kDecodeRun, out, q, k_cache, v_cache, block_tables, context_lens, num_seqs,
                       num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                       max_context_len, scale, partition_size, workspace, workspace_bytes, dtype, stream);
}

size_t pa_decode_scores_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                       int max_context_len, int partition_size)
{
    const int p = pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                                           partition_size);
    if (p <= 0 || num_seqs <= 0 || num_heads <= 0 || head_dim <= 0) return 0;
    const size_t np = max_context_len > 0 ? ((size_t)max_context_len + p - 1) / p : 1;
    return scores_workspace((size_t)num_seqs, (size_t)num_heads, (size_t)head_dim, np, (size_t)max_context_len).total;
}

pa_status pa_decode_scores(void* out, float* scores, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                           int max_context_len, int score_stride, float scale, int partition_size, void* workspace,
                           size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_decode_scores");
    return decode_call("pa_decode_scores", kDecodePlan | kDecodeRun, out, q, k_cache, v_cache, block_tables,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                       num_blocks, max_context_len, scale, partition_size, workspace, workspace_bytes, dtype, stream,
                       true, scores, score_stride);
}

static size_t evict_counts_bytes(size_t rows) { return (rows * sizeof(unsigned) + 255) / 256 * 256; }
static size_t evict_list_bytes(size_t rows, int max_context_len)
{
    return rows * sizeof(unsigned) * (size_t)std::max(1, max_context_len / 2);
}

size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_context_len)
{
    if (num_seqs <= 0 || num_kv_heads <= 0 || max_context_len < 0 || max_context_len > kMaxEvictContext) return 0;
    const size_t rows = (size_t)num_seqs * num_kv_heads;
    return evict_counts_bytes(rows) + 2 * evict_list_bytes(rows, max_context_len) +
           rows * sizeof(uint32_t) * (size_t)((max_context_len + 31) / 32);
}

pa_status pa_evict(void* k_cache, void* v_cache, float* new_scores, int32_t* new_positions, const float* scores,
                   const int32_t* positions, const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* keep_lens, int num_recent, int num_seqs, int num_kv_heads, int head_dim,
                   int block_size, int max_blocks_per_seq, int num_blocks, int max_context_len, int score_stride,
                   void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_evict");
    pa_status st = check_common("pa_evict", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_recent < 0 || num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
        score_stride < max_context_len) {
        set_error("pa_evict: bad size (score_stride must be at least max_context_len)");
        return PA_ERR_INVALID;
    }
    if (max_context_len > kMaxEvictContext || (int64_t)num_seqs * num_kv_heads > (1 << 20)) {
        set_error("pa_evict: max_context_len at most " + std::to_string(kMaxEvictContext) +
                  ", num_seqs * num_kv_heads at most 1048576");
        return PA_ERR_UNSUPPORTED;
    }
    if (num_seqs == 0 || max_context_len == 0) return PA_OK;
    if (!k_cache || !v_cache || !new_scores || !new_positions || !scores || !positions || !block_tables ||
        !context_lens || !keep_lens) {
        set_error("pa_evict: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(new_scores, 4) || !aligned(new_positions, 4) ||
        !aligned(scores, 4) || !aligned(positions, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(keep_lens, 4)) {
        set_error("pa_evict: misaligned pointer (caches need 16 bytes)");
        return PA_ERR_INVALID;
    }
    const size_t need = pa_evict_workspace_size(num_seqs, num_kv_heads, max_context_len);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) {
        set_error("pa_evict: workspace missing, too small (need " + std::to_string(need) +
                  " bytes) or not 16-byte aligned");
        return PA_ERR_INVALID;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    EvictArgs a{};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.new_scores = new_scores;
    a.new_positions = new_positions;
    a.scores = scores;
    a.positions = positions;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.keep_lens = keep_lens;
    a.counts = static_cast<unsigned*>(workspace);
    unsigned char* lists = static_cast<unsigned char*>(workspace) + evict_counts_bytes((size_t)num_seqs * num_kv_heads);
    const size_t list = evict_list_bytes((size_t)num_seqs * num_kv_heads, max_context_len);
    a.dst = reinterpret_cast<unsigned*>(lists);
    a.src = reinterpret_cast<unsigned*>(lists + list);
    a.masks = reinterpret_cast<uint32_t*>(lists + 2 * list);
    a.status = status;
    a.num_recent = num_recent;
    a.num_seqs = num_seqs;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.max_context_len = max_context_len;
    a.score_stride = score_stride;
    a.move_stride = std::max(1, max_context_len / 2);
    const cudaError_t e = launch_evict(a, head_dim, elt_bytes(dtype), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_evict launch", e);
    return PA_OK;
}

pa_status pa_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_reshape_and_cache");
    pa_status st = check_common("pa_reshape_and_cache", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_tokens < 0) {
        set_error("pa_reshape_and_cache: num_tokens < 0");
        return PA_ERR_INVALID;
    }
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) {
        set_error("pa_reshape_and_cache: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slot_mapping, 8)) {
        set_error("pa_reshape_and_cache: misaligned pointer");
        return PA_ERR_INVALID;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    ReshapeArgs a{key, value, k_cache, v_cache, slot_mapping, status, num_tokens, num_kv_heads, num_blocks};
    const cudaError_t e =
        launch_reshape_and_cache(a, elt_bytes(dtype), head_dim, block_size, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_reshape_and_cache launch", e);
    return PA_OK;
}

pa_status pa_check_block_mapping(const int64_t* block_mapping, int num_pairs, int num_blocks)
{
    if (num_pairs < 0 || num_blocks <= 0 || (num_pairs > 0 && !block_mapping)) {
        set_error("pa_check_block_mapping: bad count or null array");
        return PA_ERR_INVALID;
    }
    // (block, pair index) of every destination, then of every source, sorted by block
    std::vector<std::pair<int64_t, int>> dst, src;
    dst.reserve(num_pairs);
    src.reserve(num_pairs);
    for (int i = 0; i < num_pairs; ++i) {
        const int64_t s = block_mapping[2 * i], d = block_mapping[2 * i + 1];
        if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
            set_error("pa_check_block_mapping: pair " + std::to_string(i) + " names a block outside [0, num_blocks)");
            return PA_ERR_INVALID;
        }
        dst.emplace_back(d, i);
        src.emplace_back(s, i);
    }
    std::sort(dst.begin(), dst.end());
    std::sort(src.begin(), src.end());
    for (size_t k = 1; k < dst.size(); ++k)
        if (dst[k].first == dst[k - 1].first) {
            set_error("pa_check_block_mapping: pairs " + std::to_string(dst[k - 1].second) + " and " +
                      std::to_string(dst[k].second) + " write the same block " + std::to_string(dst[k].first));
            return PA_ERR_INVALID;
        }
    for (size_t k = 0, m = 0; k < dst.size(); ++k) {
        while (m < src.size() && src[m].first < dst[k].first) ++m;
        if (m < src.size() && src[m].first == dst[k].first) {
            set_error("pa_check_block_mapping: block " + std::to_string(dst[k].first) + " is written by pair " +
                      std::to_string(dst[k].second) + " and read by pair " + std::to_string(src[m].second));
            return PA_ERR_INVALID;
        }
    }
    return PA_OK;
}

pa_status pa_check_slot_mapping(const int64_t* slot_mapping, int num_tokens, int num_blocks, int block_size)
{
    if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || (num_tokens > 0 && !slot_mapping)) {
        set_error("pa_check_slot_mapping: bad count or size, or null array");
        return PA_ERR_INVALID;
    }
    const int64_t nslots = (int64_t)num_blocks * block_size;
    std::vector<std::pair<int64_t, int>> slots;
    slots.reserve(num_tokens);
    for (int t = 0; t < num_tokens; ++t) {
        const int64_t s = slot_mapping[t];
        if (s < 0) continue;  // padding
        if (s >= nslots) {
            set_error("pa_check_slot_mapping: token " + std::to_string(t) + " has slot " + std::to_string(s) +
                      ", past the pool's " + std::to_string(nslots) + " slots");
            return PA_ERR_INVALID;
        }
        slots.emplace_back(s, t);
    }
    std::sort(slots.begin(), slots.end());
    for (size_t k = 1; k < slots.size(); ++k)
        if (slots[k].first == slots[k - 1].first) {
            set_error("pa_check_slot_mapping: tokens " + std::to_string(slots[k - 1].second) + " and " +
                      std::to_string(slots[k].second) + " share slot " + std::to_string(slots[k].first));
            return PA_ERR_INVALID;
        }
    return PA_OK;
}

pa_status pa_copy_blocks(void* k_cache, void* v_cache, const int64_t* block_mapping, int num_pairs,
                         int num_kv_heads, int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                         void* stream)
{
    pa::CallRange range("pa_copy_blocks");
    pa_status st = check_common("pa_copy_blocks", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_pairs < 0 || num_pairs > 65535) {
        set_error("pa_copy_blocks: num_pairs must be in [0, 65535]");
        return PA_ERR_INVALID;
    }
    if (num_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !block_mapping) {
        set_error("pa_copy_blocks: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_mapping, 8)) {
        set_error("pa_copy_blocks: misaligned pointer");
        return PA_ERR_INVALID;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    CopyArgs a{};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_mapping = block_mapping;
    a.status = status;
    a.num_pairs = num_pairs;
    a.num_blocks = num_blocks;
    a.block_bytes = (size_t)num_kv_heads * block_size * head_dim * elt_bytes(dtype);
    const cudaError_t e = launch_copy_blocks(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_copy_blocks launch", e);
    return PA_OK;
}

static pa_status prefill_impl(const char* name, void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables,
                     const int32_t* context_lens, const int32_t* q_start, int num_seqs, int num_heads,
                     int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                     int num_query_tokens, int max_query_len, float scale, pa_dtype dtype, void* stream,
                              void* workspace, size_t workspace_bytes)
{
    pa::CallRange range(name);
    pa_status st = check_common("pa_prefill", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (dtype != PA_DTYPE_BF16 || head_dim != 128) {
        set_error("pa_prefill: bf16 with head_dim 128 only (the tensor-core tile)");
        return PA_ERR_UNSUPPORTED;
    }
    if (num_seqs < 0 || num_seqs > 65535 || num_heads <= 0 || num_heads % num_kv_heads != 0 ||
        num_query_tokens < 0 || max_query_len < 0 || max_blocks_per_seq < 0 || !(scale == scale) ||
        scale == INFINITY || scale == -INFINITY) {
        set_error("pa_prefill: bad sizes or scale");
        return PA_ERR_INVALID;
    }
    const int group = num_heads / num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) {
        set_error("pa_prefill: num_heads / num_kv_heads must be 1, 2, 4 or 8");
        return PA_ERR_UNSUPPORTED;
    }
    if (workspace && (workspace_bytes < pa_prefill_workspace_size() || !aligned(workspace, 16))) {
        set_error("pa_prefill_ws: workspace smaller than pa_prefill_workspace_size() or not 16-byte aligned");
        return PA_ERR_INVALID;
    }
    if (num_seqs == 0 || num_query_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !q_start) {
        set_error("pa_prefill: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) {
        set_error("pa_prefill: misaligned pointer (q, out, caches need 16 bytes)");
        return PA_ERR_INVALID;
    }
    if ((int64_t)num_blocks * num_kv_heads * block_size > (int64_t)INT32_MAX) {
        set_error("pa_prefill: num_blocks * num_kv_heads * block_size must stay below 2^31 (tensor-copy row index)");
        return PA_ERR_UNSUPPORTED;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    PrefillArgs a{};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.q_start = q_start;
    a.status = status;
    a.sched = static_cast<unsigned int*>(workspace);
    a.num_seqs = num_seqs;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.num_query_tokens = num_query_tokens;
    a.max_query_len = max_query_len;
    a.scale_log2 = scale * 1.4426950408889634f;
    if (workspace) {
        // the item counter starts at zero on every call, in stream order
        const cudaError_t z = cudaMemsetAsync(workspace, 0, sizeof(unsigned int), static_cast<cudaStream_t>(stream));
        if (z != cudaSuccess) return cuda_fail("pa_prefill_ws counter reset", z);
    }
    const cudaError_t e =
        launch_prefill(a, group, num_query_tokens, max_query_len, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_prefill launch", e);
    return PA_OK;
}

namespace {

// Layout of pa_cross_attention's workspace: entries and merge list (or, with at most one query row per
// sequence, the own tokens' entries and counters), then the partial states.
struct CrossWorkspace {
    GroupWorkspace g;
    size_t entries, merges, own, arrived, acc, ml, total;
    int chunks;
    bool single;
};

CrossWorkspace cross_workspace(size_t S, size_t Hq, int Hkv, int D, size_t Nq, int max_query_len, int max_context_len)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    CrossWorkspace w{};
    const int G = (int)(Hq / (size_t)Hkv);
    w.single = max_query_len <= 1;
    if (w.single) {
        w.chunks = shared_max_parts((int64_t)S, Hkv, max_context_len);
        w.g = group_workspace(0, 0, 0);
        w.own = w.g.end;
        w.arrived = up(w.own + sizeof(OwnItem) * S * (size_t)w.chunks);
        w.acc = up(w.arrived + 4 * Nq * (size_t)Hkv);
        const size_t states = w.chunks > 1 ? Nq * Hq * (size_t)w.chunks : 0;
        w.ml = up(w.acc + states * (size_t)D * 4);
        w.total = up(w.ml + states * 8);
        w.entries = S * (size_t)w.chunks;
        return w;
    }
    const size_t T = ((int64_t)max_query_len * G <= 64 ? 64 : 128) / (size_t)G;
    w.chunks = group_max_chunks(max_context_len, (int64_t)Nq, G, Hkv);
    w.entries = (S + Nq / T) * (size_t)w.chunks;
    w.merges = w.chunks > 1 ? Nq : 0;
    w.g = group_workspace(0, w.entries, w.merges);
    const size_t states = w.chunks > 1 ? Nq * Hq * (size_t)w.chunks : 0;
    w.acc = w.g.end;
    w.ml = up(w.acc + states * (size_t)D * 4);
    w.total = up(w.ml + states * 8);
    return w;
}

// The checks that the two tensor-core calls over packed rows share.
pa_status check_group(const char* fn, int num_heads, int num_kv_heads, int num_blocks, int block_size, pa_dtype dtype)
{
    if (dtype != PA_DTYPE_BF16) {
        set_error(std::string(fn) + ": bf16 only (the tensor-core tile)");
        return PA_ERR_UNSUPPORTED;
    }
    if (num_heads <= 0 || num_heads % num_kv_heads != 0) {
        set_error(std::string(fn) + ": num_heads must be a multiple of num_kv_heads");
        return PA_ERR_INVALID;
    }
    const int group = num_heads / num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) {
        set_error(std::string(fn) + ": num_heads / num_kv_heads must be 1, 2, 4 or 8");
        return PA_ERR_UNSUPPORTED;
    }
    if ((int64_t)num_blocks * num_kv_heads * block_size > (int64_t)INT32_MAX) {
        set_error(std::string(fn) +
                  ": num_blocks * num_kv_heads * block_size must stay below 2^31 (tensor-copy row index)");
        return PA_ERR_UNSUPPORTED;
    }
    return PA_OK;
}

}  // namespace

size_t pa_cross_attention_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                         int num_query_tokens, int max_query_len, int max_context_len)
{
    if (num_seqs <= 0 || num_query_tokens <= 0 || max_query_len < 0 || max_context_len < 0 ||
        check_common("pa_cross_attention_workspace_size", num_kv_heads, head_dim, block_size, 1, PA_DTYPE_BF16) != PA_OK ||
        check_group("pa_cross_attention_workspace_size", num_heads, num_kv_heads, 1, block_size, PA_DTYPE_BF16) != PA_OK)
        return 0;
    return cross_workspace((size_t)num_seqs, (size_t)num_heads, num_kv_heads, head_dim, (size_t)num_query_tokens,
                           std::min(max_query_len, num_query_tokens), max_context_len)
        .total;
}

pa_status pa_cross_attention(void* out, float* lse, const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_start,
                             int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int max_blocks_per_seq, int num_blocks, int num_query_tokens, int max_query_len,
                             int max_context_len, float scale, void* workspace, size_t workspace_bytes, pa_dtype dtype,
                             void* stream)
{
    pa::CallRange range("pa_cross_attention");
    pa_status st = check_common("pa_cross_attention", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    st = check_group("pa_cross_attention", num_heads, num_kv_heads, num_blocks, block_size, dtype);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || num_seqs > 65535 || num_query_tokens < 0 || max_query_len < 0 || max_context_len < 0 ||
        max_blocks_per_seq < 0 || !std::isfinite(scale)) {
        set_error("pa_cross_attention: bad size or scale");
        return PA_ERR_INVALID;
    }
    if (num_seqs == 0 || num_query_tokens == 0 || max_query_len == 0) return PA_OK;
    // no sequence has more rows than there are; the bound chooses the kernel and counts its work items
    max_query_len = std::min(max_query_len, num_query_tokens);
    if (!out || !q || !k_cache || !v_cache || (!block_tables && max_blocks_per_seq > 0) || !context_lens || !q_start) {
        set_error("pa_cross_attention: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lse, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(q_start, 4)) {
        set_error("pa_cross_attention: misaligned pointer (q, out, caches need 16 bytes)");
        return PA_ERR_INVALID;
    }
    const CrossWorkspace w = cross_workspace((size_t)num_seqs, (size_t)num_heads, num_kv_heads, head_dim,
                                             (size_t)num_query_tokens, max_query_len, max_context_len);
    if (w.entries * (size_t)num_kv_heads > (size_t)INT32_MAX || w.merges * (size_t)num_heads > (size_t)INT32_MAX) {
        set_error("pa_cross_attention: too many query rows");
        return PA_ERR_UNSUPPORTED;
    }
    if (!workspace || workspace_bytes < w.total || !aligned(workspace, 16)) {
        set_error("pa_cross_attention: workspace missing, too small (need " + std::to_string(w.total) +
                  " bytes) or not 16-byte aligned");
        return PA_ERR_INVALID;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    CrossArgs a{};
    a.g.out = out;
    a.g.lse = lse;
    a.g.q = q;
    a.g.k_cache = k_cache;
    a.g.v_cache = v_cache;
    a.g.block_tables = block_tables;
    a.g.items = reinterpret_cast<const GroupItem*>(ws + w.g.items);
    a.g.counts = reinterpret_cast<const unsigned*>(ws + w.g.header);
    a.g.merge_list = reinterpret_cast<const uint2*>(ws + w.g.merges);
    a.g.ws_acc = reinterpret_cast<float*>(ws + w.acc);
    a.g.ws_ml = reinterpret_cast<float*>(ws + w.ml);
    a.g.status = status;
    a.g.num_heads = num_heads;
    a.g.num_kv_heads = num_kv_heads;
    a.g.max_blocks_per_seq = max_blocks_per_seq;
    a.g.num_blocks = num_blocks;
    a.g.block_size = block_size;
    a.g.num_partitions = w.chunks;
    a.g.max_entries = (int)w.entries;
    a.g.max_merges = (int)w.merges;
    a.g.scale_log2 = scale * 1.4426950408889634f;
    a.context_lens = context_lens;
    a.q_start = q_start;
    a.num_seqs = num_seqs;
    a.num_query_tokens = num_query_tokens;
    a.max_query_len = max_query_len;
    a.max_context_len = max_context_len;
    a.max_chunks = w.chunks;
    cudaError_t e;
    if (w.single) {
        SharedArgs o{};
        o.g = a.g;
        o.context_lens = context_lens;
        o.own = reinterpret_cast<OwnItem*>(ws + w.own);
        o.arrived = reinterpret_cast<unsigned*>(ws + w.arrived);
        o.num_seqs = num_seqs;
        o.max_context_len = max_context_len;
        o.max_parts = w.chunks;
        e = launch_cross_single(o, q_start, num_query_tokens, head_dim, num_heads / num_kv_heads,
                                static_cast<cudaStream_t>(stream));
    } else {
        e = launch_cross(a, head_dim, num_heads / num_kv_heads, static_cast<cudaStream_t>(stream));
    }
    if (e != cudaSuccess) return cuda_fail("pa_cross_attention launch", e);
    return PA_OK;
}

size_t pa_decode_shared_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                       int max_context_len, int max_shared_len, int num_groups, int num_group_rows)
{
    if (num_seqs <= 0 || max_context_len < 0 || max_shared_len < 0 || num_groups < 0 || num_group_rows < 0 ||
        check_common("pa_decode_shared_workspace_size", num_kv_heads, head_dim, block_size, 1, PA_DTYPE_BF16) != PA_OK ||
        check_group("pa_decode_shared_workspace_size", num_heads, num_kv_heads, 1, block_size, PA_DTYPE_BF16) != PA_OK)
        return 0;
    return shared_workspace((size_t)num_seqs, (size_t)num_heads, num_kv_heads, head_dim, max_context_len, max_shared_len,
                            (size_t)num_groups, (size_t)num_group_rows)
        .total;
}

pa_status pa_decode_shared(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, const int32_t* group_rows,
                           const int32_t* group_start, const int32_t* shared_lens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                           int num_groups, int num_group_rows, int max_context_len, int max_shared_len, float scale,
                           void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_decode_shared");
    pa_status st = check_common("pa_decode_shared", num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    st = check_group("pa_decode_shared", num_heads, num_kv_heads, num_blocks, block_size, dtype);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || max_context_len < 0 || max_shared_len < 0 ||
        num_groups < 0 || num_groups > 65535 || num_group_rows < 0 || num_group_rows > num_seqs ||
        !std::isfinite(scale)) {
        set_error("pa_decode_shared: bad size or scale (a row is in one group at most)");
        return PA_ERR_INVALID;
    }
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens ||
        (num_groups > 0 && (!group_start || !shared_lens)) || (num_group_rows > 0 && !group_rows)) {
        set_error("pa_decode_shared: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(group_rows, 4) || !aligned(group_start, 4) ||
        !aligned(shared_lens, 4)) {
        set_error("pa_decode_shared: misaligned pointer (q, out, caches need 16 bytes)");
        return PA_ERR_INVALID;
    }
    const SharedWorkspace w =
        shared_workspace((size_t)num_seqs, (size_t)num_heads, num_kv_heads, head_dim, max_context_len, max_shared_len,
                         (size_t)num_groups, (size_t)num_group_rows);
    if (std::max(w.entries, (size_t)num_seqs * (size_t)w.parts) * (size_t)num_kv_heads > (size_t)INT32_MAX ||
        (size_t)num_seqs * (size_t)num_heads > (size_t)INT32_MAX) {
        set_error("pa_decode_shared: too many rows");
        return PA_ERR_UNSUPPORTED;
    }
    if (!workspace || workspace_bytes < w.total || !aligned(workspace, 16)) {
        set_error("pa_decode_shared: workspace missing, too small (need " + std::to_string(w.total) +
                  " bytes) or not 16-byte aligned");
        return PA_ERR_INVALID;
    }
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    SharedArgs a{};
    a.g.out = out;
    a.g.q = q;
    a.g.k_cache = k_cache;
    a.g.v_cache = v_cache;
    a.g.block_tables = block_tables;
    a.g.rows = group_rows;
    a.g.items = reinterpret_cast<const GroupItem*>(ws + w.g.items);
    a.g.counts = reinterpret_cast<const unsigned*>(ws + w.g.header);
    a.g.ws_acc = reinterpret_cast<float*>(ws + w.acc);
    a.g.ws_ml = reinterpret_cast<float*>(ws + w.ml);
    a.g.status = status;
    a.g.num_heads = num_heads;
    a.g.num_kv_heads = num_kv_heads;
    a.g.max_blocks_per_seq = max_blocks_per_seq;
    a.g.num_blocks = num_blocks;
    a.g.block_size = block_size;
    a.g.num_partitions = w.chunks + w.parts;
    a.g.lead_partitions = w.chunks;
    a.g.max_entries = (int)w.entries;
    a.g.scale_log2 = scale * 1.4426950408889634f;
    a.context_lens = context_lens;
    a.group_rows = group_rows;
    a.group_start = group_start;
    a.shared_lens = shared_lens;
    a.own = reinterpret_cast<OwnItem*>(ws + w.own);
    a.arrived = reinterpret_cast<unsigned*>(ws + w.arrived);
    a.listed = reinterpret_cast<int*>(ws + w.listed);
    a.ctx = reinterpret_cast<int*>(ws + w.ctx);
    a.lead_blocks = reinterpret_cast<int*>(ws + w.lead_blocks);
    a.lead_states = reinterpret_cast<int*>(ws + w.lead_states);
    a.group_ok = reinterpret_cast<int*>(ws + w.group_ok);
    a.num_seqs = num_seqs;
    a.num_groups = num_groups;
    a.num_group_rows = num_group_rows;
    a.max_context_len = max_context_len;
    a.max_shared_len = max_shared_len;
    a.max_chunks = w.chunks;
    a.max_parts = w.parts;
    const cudaError_t e = launch_shared(a, head_dim, num_heads / num_kv_heads, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_decode_shared launch", e);
    return PA_OK;
}

size_t pa_prefill_workspace_size(void) { return 256; }

pa_status pa_prefill(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     const int32_t* context_lens, const int32_t* q_start, int num_seqs, int num_heads,
                     int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                     int num_query_tokens, int max_query_len, float scale, pa_dtype dtype, void* stream)
{
    return prefill_impl("pa_prefill", out, q, k_cache, v_cache, block_tables, context_lens, q_start, num_seqs,
                        num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                        num_query_tokens, max_query_len, scale, dtype, stream, nullptr, 0);
}

pa_status pa_prefill_ws(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_start,
                        int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                        int max_blocks_per_seq, int num_blocks, int num_query_tokens, int max_query_len, float scale,
                        void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream)
{
    if (!workspace) {
        set_error("pa_prefill_ws: null workspace");
        return PA_ERR_INVALID;
    }
    return prefill_impl("pa_prefill_ws", out, q, k_cache, v_cache, block_tables, context_lens, q_start, num_seqs,
                        num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                        num_query_tokens, max_query_len, scale, dtype, stream, workspace, workspace_bytes);
}

// Address a kernel can use for p: device memory as is, pinned (page-locked) host
// memory through its device mapping; anything else is refused.
static pa_status kernel_address(const char* who, const char* what, const void* p, const void** out)
{
    cudaPointerAttributes at{};
    const cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_error(std::string(who) + ": cannot query " + what + ": " + cudaGetErrorString(e));
        return PA_ERR_INVALID;
    }
    if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) {
        *out = p;
        return PA_OK;
    }
    if (at.type == cudaMemoryTypeHost && at.devicePointer) {
        *out = at.devicePointer;
        return PA_OK;
    }
    set_error(std::string(who) + ": " + what + " must be device memory or pinned host memory");
    return PA_ERR_INVALID;
}

pa_status pa_swap_blocks(void* dst_k_cache, void* dst_v_cache, const void* src_k_cache, const void* src_v_cache,
                         const int64_t* block_mapping, int num_pairs, int num_kv_heads, int head_dim, int block_size,
                         int num_src_blocks, int num_dst_blocks, pa_dtype dtype, void* stream)
{
    pa::CallRange range("pa_swap_blocks");
    pa_status st = check_common("pa_swap_blocks", num_kv_heads, head_dim, block_size, num_src_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_dst_blocks <= 0) {
        set_error("pa_swap_blocks: num_dst_blocks must be > 0");
        return PA_ERR_INVALID;
    }
    if (num_pairs < 0 || num_pairs > 65535) {
        set_error("pa_swap_blocks: num_pairs must be in [0, 65535]");
        return PA_ERR_INVALID;
    }
    if (num_pairs == 0) return PA_OK;
    if (!dst_k_cache || !dst_v_cache || !src_k_cache || !src_v_cache || !block_mapping) {
        set_error("pa_swap_blocks: null pointer");
        return PA_ERR_INVALID;
    }
    if (!aligned(dst_k_cache, 16) || !aligned(dst_v_cache, 16) || !aligned(src_k_cache, 16) ||
        !aligned(src_v_cache, 16) || !aligned(block_mapping, 8)) {
        set_error("pa_swap_blocks: misaligned pointer");
        return PA_ERR_INVALID;
    }
    SwapArgs a{};
    const void* p = nullptr;
    if ((st = kernel_address("pa_swap_blocks", "dst_k_cache", dst_k_cache, &p)) != PA_OK) return st;
    a.dst_k = const_cast<void*>(p);
    if ((st = kernel_address("pa_swap_blocks", "dst_v_cache", dst_v_cache, &p)) != PA_OK) return st;
    a.dst_v = const_cast<void*>(p);
    if ((st = kernel_address("pa_swap_blocks", "src_k_cache", src_k_cache, &a.src_k)) != PA_OK) return st;
    if ((st = kernel_address("pa_swap_blocks", "src_v_cache", src_v_cache, &a.src_v)) != PA_OK) return st;
    if ((st = kernel_address("pa_swap_blocks", "block_mapping", block_mapping, &p)) != PA_OK) return st;
    a.block_mapping = static_cast<const int64_t*>(p);
    unsigned int* status = nullptr;
    st = status_ptr(&status);
    if (st != PA_OK) return st;
    a.status = status;
    a.num_pairs = num_pairs;
    a.num_src_blocks = num_src_blocks;
    a.num_dst_blocks = num_dst_blocks;
    a.block_bytes = (size_t)num_kv_heads * block_size * head_dim * elt_bytes(dtype);
    const cudaError_t e = launch_swap_blocks(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_swap_blocks launch", e);
    return PA_OK;
}

pa_status pa_selftest_bounded_wait(uint64_t* waited_ns, void* stream)
{
    unsigned int* status = nullptr;
    pa_status st = status_ptr(&status);
    if (st != PA_OK) return st;
    unsigned long long ns = 0;
    const cudaError_t e = launch_wait_selftest(status, &ns, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("pa_selftest_bounded_wait", e);
    if (waited_ns) *waited_ns = (uint64_t)ns;
    return PA_OK;
}

pa_status pa_device_status(uint32_t* flags, void* stream)
{
    if (!flags) return PA_ERR_INVALID;
    unsigned int* status = nullptr;
    pa_status st = status_ptr(&status);
    if (st != PA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, status, sizeof(v), cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return cuda_fail("pa_device_status read", e);
    e = cudaMemsetAsync(status, 0, sizeof(unsigned int), s);
    if (e != cudaSuccess) return cuda_fail("pa_device_status clear", e);
    e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail("pa_device_status sync", e);
    *flags = v;
    return PA_OK;
}

}  // extern "C"
