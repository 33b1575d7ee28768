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
// Two kernels.  evict_select (one CTA per (sequence, kv head)) finds the n-th largest key,
// marks the kept tokens in a bit mask in shared memory, ranks gaps and movers by prefix sums
// over the mask's words, and writes the mask and the list of moves.  evict_move copies the K
// and V rows of the list, and brings scores and positions along.
//
// The selection counts the keys in 2048 equal bins between the smallest and the largest (a
// fixed split by leading bits would put most scores into a few bins, whose counters then take
// them one by one), goes on in the bin of the n-th, and compares its last 256 or fewer keys
// with one another: one or two passes, where fixed digits of 11 bits take three.
// The selection is a chain of passes over the head's tokens, each a trip to memory long, and
// there may be fewer heads than SMs: scores and positions are read once, eight loads in flight
// per thread, and the keys stay in shared memory (contexts up to kCachedContext; longer ones
// read them again in every pass).
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_evict_select.h"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kBins = kEvictBins;
constexpr int kCachedContext = 49152;  // keys (4 bytes) and two masks of a context in shared memory
constexpr unsigned kFew = 256;         // keys of one bin that are compared with one another
constexpr int kSmallContext = 4096;    // scores, positions, blocks and the move list as well

// Where the head's tokens are kept while they are selected.
constexpr int kFromGlobal = 0;  // nowhere: read again in every pass
constexpr int kKeysCached = 1;  // their keys in shared memory
constexpr int kAllCached = 2;   // scores, positions and the move list too; the CTA may move the rows itself

// Exclusive prefix sum of one value per thread over the CTA; *total receives the sum.
template <int THREADS>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp,
                                                         unsigned long long* total)
{
    constexpr int NW = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    unsigned long long w = lane < NW ? s_warp[lane] : 0ull;  // every warp adds up the warps' sums itself
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, NW - 1);
    const unsigned long long base = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return (warp > 0 ? base : 0ull) + x - v;
}

// CPR: with kAllCached, 16-byte chunks of a K or V row when this kernel moves the rows too, else 0.
template <int THREADS, int WHERE, int CPR>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const EvictArgs a)
{
    constexpr bool CACHED = WHERE != kFromGlobal, ALL = WHERE == kAllCached, MOVE = CPR > 0;
    constexpr int UN = THREADS == 1024 ? 16 : 8;  // loads in flight per thread
    constexpr int UW = 4;                         // words of a warp at a time
    constexpr int BPT = kBins / THREADS;          // bins per thread
    extern __shared__ uint32_t s_mask[];          // kept tokens, then the ties: one bit each; then what is cached
    __shared__ unsigned s_hist[kBins];
    __shared__ unsigned long long s_warp[THREADS / 32];
    __shared__ unsigned s_prefix, s_need, s_count, s_recent, s_few;
    __shared__ int s_max[THREADS / 32];
    __shared__ unsigned s_lo[THREADS / 32], s_hi[THREADS / 32];
    const int sh = blockIdx.x;
    const int s = sh / a.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L = __ldg(a.context_lens + s), n = __ldg(a.keep_lens + s);
    if constexpr (!MOVE) pdl_launch_dependents();
    if (L < 0 || n < 0 || L > a.max_context_len || L > table_tokens(a.max_blocks_per_seq, a.block_size)) {
        if (tid == 0) {
            if constexpr (!MOVE) a.counts[sh] = ~0u;
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
        for (int i = tid; i < n; i += THREADS) {
            nsc[i] = sc[i];
            npos[i] = pos[i];
        }
        if constexpr (!MOVE)
            if (tid == 0) a.counts[sh] = ~0u;
        return;
    }
    const int words = (L + 31) / 32;
    uint32_t* s_tie = s_mask + words;
    uint32_t* s_key = s_tie + words;
    float* s_sc = reinterpret_cast<float*>(s_key + L);
    int* s_pos = reinterpret_cast<int*>(s_sc + L);
    int* s_blk = s_pos + L;                                       // the table's row, where rows are moved here
    const int nblk = MOVE ? (L + a.block_size - 1) / a.block_size : 0;
    uint16_t* s_gap = reinterpret_cast<uint16_t*>(s_blk + nblk);  // [L / 2]
    uint16_t* s_mover = s_gap + L / 2;                            // [L / 2]
    if constexpr (MOVE)
        for (int i = tid; i < nblk; i += THREADS) s_blk[i] = __ldg(a.block_tables + (size_t)s * a.max_blocks_per_seq + i);
    // keys and their range, and the largest position
    int mx = INT32_MIN;
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int i0 = tid; i0 < L; i0 += THREADS * UN) {
        float x[UN];
        int p[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int i = i0 + k * THREADS;
            p[k] = i < L ? pos[i] : INT32_MIN;
            x[k] = i < L ? sc[i] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            mx = max(mx, p[k]);
            const int i = i0 + k * THREADS;
            if (i < L) {
                const uint32_t y = score_key(x[k]);
                lo = min(lo, y);
                hi = max(hi, y);
                if constexpr (CACHED) s_key[i] = y;
                if constexpr (ALL) {
                    s_sc[i] = x[k];
                    s_pos[i] = p[k];
                }
            }
        }
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        s_max[warp] = mx;
        s_lo[warp] = lo;
        s_hi[warp] = hi;
    }
    if (tid == 0) s_recent = s_few = 0;
    for (int i = tid; i < kBins; i += THREADS) s_hist[i] = 0;
    __syncthreads();
    mx = __reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? s_max[lane] : INT32_MIN);
    lo = __reduce_min_sync(0xffffffffu, lane < THREADS / 32 ? s_lo[lane] : 0xffffffffu);
    hi = __reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? s_hi[lane] : 0u);
    // the recent tokens: positions within num_recent of the largest
    const int recent = min(a.num_recent, n);
    const long long fr = (long long)mx - recent + 1;
    const int first_recent = fr < (long long)INT32_MIN ? INT32_MIN : (int)min(fr, (long long)INT32_MAX);
    if constexpr (CACHED) {
        if (recent > 0) {
            for (int i0 = tid; i0 < L; i0 += THREADS * UN) {
                int p[UN];
#pragma unroll
                for (int k = 0; k < UN; ++k)
                    p[k] = i0 + k * THREADS < L ? (ALL ? s_pos[i0 + k * THREADS] : pos[i0 + k * THREADS]) : INT32_MIN;
#pragma unroll
                for (int k = 0; k < UN; ++k)
                    if (i0 + k * THREADS < L && p[k] >= first_recent) s_key[i0 + k * THREADS] = kRecentKey;
            }
        }
        // (a thread reads back the keys it wrote itself until the masks below)
    }
    auto key = [&](int i) -> uint32_t {
        if constexpr (CACHED) return s_key[i];
        return recent > 0 && pos[i] >= first_recent ? kRecentKey : score_key(sc[i]);
    };
    // the n-th largest key, `prefix`, and how many of its equals are among the n; the recent tokens lie above [lo, hi]
    unsigned prefix = kRecentKey, need = (unsigned)n;
    KeyRange range{lo, hi};
    for (int pass = 0; pass < kEvictPasses; ++pass) {
        const bool first = pass == 0;
        const int shift = range.shift();
        unsigned seen = 0;  // recent tokens
        for (int i0 = tid; i0 < L; i0 += THREADS * 8) {
            uint32_t k[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = i0 + j * THREADS < L ? key(i0 + j * THREADS) : 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (i0 + j * THREADS < L && range.has(k[j])) atomicAdd(&s_hist[range.bin(k[j], shift)], 1u);
                seen += k[j] == kRecentKey ? 1u : 0u;
            }
        }
        if (first) {
            seen = __reduce_add_sync(0xffffffffu, seen);
            if (lane == 0 && seen) atomicAdd(&s_recent, seen);
        }
        __syncthreads();
        if (first) {
            if (s_recent >= need) break;
            need -= s_recent;
        }
        // thread t holds bins kBins - 1 - BPT * t and down
        unsigned c[BPT], sum = 0;
#pragma unroll
        for (int j = 0; j < BPT; ++j) {
            const int bin = kBins - 1 - BPT * tid - j;
            sum += c[j] = s_hist[bin];
            s_hist[bin] = 0;  // for the next pass
        }
        unsigned long long total;
        unsigned above = (unsigned)block_scan<THREADS>(sum, s_warp, &total);
        if (above < need && need <= above + sum) {
            bool found = false;
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
                if (!found && need <= above + c[j]) {
                    found = true;
                    s_prefix = range.first((unsigned)(kBins - 1 - BPT * tid - j), shift);
                    s_need = need - above;
                    s_count = c[j];
                }
                above += c[j];
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        const unsigned count = s_count;
        if (shift == 0) break;
        range = range.narrow(prefix, shift);
        if (count > kFew) continue;
        // few left: each is compared with all
        for (int i0 = tid; i0 < L; i0 += THREADS * 8) {
            uint32_t k[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = i0 + j * THREADS < L ? key(i0 + j * THREADS) : kRecentKey;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (range.has(k[j])) {
                    const unsigned at = atomicAdd(&s_few, 1u);
                    if (at < kFew) s_hist[at] = k[j];
                }
        }
        __syncthreads();
        if (tid < count) {
            const uint32_t mine = s_hist[tid];
            unsigned more = 0, same = 0;
            for (unsigned j = 0; j < count; ++j) {
                const uint32_t k = s_hist[j];
                more += k > mine ? 1u : 0u;
                same += k == mine ? 1u : 0u;
            }
            if (more < need && need <= more + same) {  // (the same from every equal)
                s_prefix = mine;
                s_need = need - more;
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        break;
    }
    // masks of the keys above the threshold, and of those equal to it
    for (int wb = warp; wb < words; wb += THREADS / 32 * UW) {
        uint32_t k[UW];
#pragma unroll
        for (int j = 0; j < UW; ++j) {
            const int i = (wb + j * (THREADS / 32)) * 32 + lane;
            k[j] = i < L ? key(i) : 0u;
        }
#pragma unroll
        for (int j = 0; j < UW; ++j) {
            const int w = wb + j * (THREADS / 32), i = w * 32 + lane;
            const uint32_t gt = __ballot_sync(0xffffffffu, i < L && k[j] > prefix);
            const uint32_t eq = __ballot_sync(0xffffffffu, i < L && k[j] == prefix);
            if (lane == 0 && w < words) {
                s_mask[w] = gt;
                s_tie[w] = eq;
            }
        }
    }
    __syncthreads();
    // the first `need` ties stay: every thread ranks a run of words
    const int per = (words + THREADS - 1) / THREADS;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    unsigned long long cnt = 0, total;
    for (int w = w0; w < w1; ++w) cnt += __popc(s_tie[w]);
    unsigned long long rank = block_scan<THREADS>(cnt, s_warp, &total);
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
    // gaps before slot n (low half) and kept tokens behind it (high half): as many of each.  A word has one kind or
    // the other, but for the one that slot n is in, whose kept tokens are the first to move.
    rank = block_scan<THREADS>(cnt, s_warp, &total);
    if ((unsigned)total != (unsigned)(total >> 32)) {
        // not n tokens: scores or positions changed between the passes.  The lists below have room for as many gaps
        // as movers alone.
        if (tid == 0) {
            if constexpr (!MOVE) a.counts[sh] = ~0u;
            atomicOr(a.status, PA_DEV_BAD_CONTEXT);
        }
        return;
    }
    for (int w = w0; w < w1; ++w) {
        const uint32_t kept = s_mask[w];
        const int below = n - w * 32;
        const uint32_t front = below >= 32 ? 0xffffffffu : (below <= 0 ? 0u : (1u << below) - 1u);
        s_tie[w] = below > 0 ? (unsigned)rank : (unsigned)(rank >> 32);
        rank += (unsigned long long)__popc(~kept & front) | (unsigned long long)__popc(kept & ~front) << 32;
    }
    __syncthreads();
    const size_t list = (size_t)sh * a.move_stride;
    for (int wb = warp; wb < words; wb += THREADS / 32 * UW) {
        uint32_t kepts[UW], base[UW];
#pragma unroll
        for (int j = 0; j < UW; ++j) {
            const int w = wb + j * (THREADS / 32);
            kepts[j] = w < words ? s_mask[w] : 0u;
            base[j] = w < words ? s_tie[w] : 0u;
        }
#pragma unroll
        for (int j = 0; j < UW; ++j) {
            const int w = wb + j * (THREADS / 32), i = w * 32 + lane;
            if (w >= words) break;
            const uint32_t kept = kepts[j], lt = (1u << lane) - 1u;
            const bool in = kept >> lane & 1u;
            const int below = n - w * 32;
            const uint32_t front = below >= 32 ? 0xffffffffu : (below <= 0 ? 0u : (1u << below) - 1u);
            if (i < n) {
                const unsigned r = base[j] + __popc(~kept & lt);
                if (!in) {
                    if constexpr (ALL) s_gap[r] = (uint16_t)i;
                    if constexpr (!MOVE) a.dst[list + r] = (unsigned)i;
                }
            } else if (in) {
                const unsigned r = (below > 0 ? 0u : base[j]) + __popc(kept & ~front & lt);
                if constexpr (ALL) s_mover[r] = (uint16_t)i;
                if constexpr (!MOVE) a.src[list + r] = (unsigned)i;
            }
        }
    }
    if constexpr (!ALL)
        for (int w = tid; w < words; w += THREADS) a.masks[(size_t)sh * ((a.max_context_len + 31) / 32) + w] = s_mask[w];
    const unsigned count = (unsigned)total;
    if constexpr (!MOVE)
        if (tid == 0) a.counts[sh] = count;
    if constexpr (!ALL) return;  // the moving kernel brings the scores and positions along
    __syncthreads();
    if constexpr (MOVE) {
        // the rows first: they are what takes the time
        constexpr int RPI = THREADS / CPR, MU = 4;  // rows of a step, steps in flight
        const int kvh = sh % a.num_kv_heads, c = tid % CPR;
        uint4* kc = static_cast<uint4*>(a.k_cache);
        uint4* vc = static_cast<uint4*>(a.v_cache);
        const int bshift = a.block_size == 16 ? 4 : 5;
        for (unsigned r0 = tid / CPR; r0 < count; r0 += RPI * MU) {
            uint4 kv[MU], vv[MU];
            size_t dst[MU];
            bool ok[MU];
#pragma unroll
            for (int k = 0; k < MU; ++k) {
                const unsigned r = r0 + k * RPI;
                ok[k] = r < count;
                if (!ok[k]) continue;
                const int f = s_mover[r], d = s_gap[r];
                const int fb = s_blk[f >> bshift], db = s_blk[d >> bshift];
                if ((unsigned)fb >= (unsigned)a.num_blocks || (unsigned)db >= (unsigned)a.num_blocks) {
                    if (c == 0) atomicOr(a.status, PA_DEV_BAD_BLOCK);
                    ok[k] = false;
                    continue;
                }
                const size_t src = ((((size_t)fb * a.num_kv_heads + kvh) << bshift) + (f & (a.block_size - 1))) * CPR + c;
                dst[k] = ((((size_t)db * a.num_kv_heads + kvh) << bshift) + (d & (a.block_size - 1))) * CPR + c;
                kv[k] = kc[src];
                vv[k] = vc[src];
            }
#pragma unroll
            for (int k = 0; k < MU; ++k)
                if (ok[k]) {
                    kc[dst[k]] = kv[k];
                    vc[dst[k]] = vv[k];
                }
        }
    }
    // the scores and positions of the slots before n (these arrays may be the old ones: a slot
    // before n is only ever written with its own value or one from behind n)
    if constexpr (ALL) {
        for (int i = tid; i < n; i += THREADS)
            if (s_mask[i / 32] >> (i % 32) & 1u) {
                nsc[i] = s_sc[i];
                npos[i] = s_pos[i];
            }
        for (unsigned r = tid; r < count; r += THREADS) {
            const int f = s_mover[r], d = s_gap[r];
            nsc[d] = s_sc[f];
            npos[d] = s_pos[f];
        }
    }
}

// `splits` CTAs move each head's rows, CPR threads per row (16 bytes each), the K and the V row of a move together.
// `carry` more CTAs before them (0: none) bring its scores and positions along, those of the slots before n, as above.
template <int CPR>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int carry, int splits)
{
    pdl_wait_primary();
    constexpr int RPI = kMoveThreads / CPR;  // moves per step of the CTA
    const int sh = blockIdx.x / (carry + splits), part = (int)(blockIdx.x % (carry + splits)) - carry;
    const int s = sh / a.num_kv_heads, kvh = sh % a.num_kv_heads;
    const unsigned count = __ldcg(a.counts + sh);
    if (count == ~0u) return;
    const size_t list = (size_t)sh * a.move_stride;
    if (part < 0) {
        const size_t row = (size_t)sh * a.score_stride;
        const uint32_t* mask = a.masks + (size_t)sh * ((a.max_context_len + 31) / 32);
        const int n = min(__ldg(a.keep_lens + s), __ldg(a.context_lens + s)), hop = carry * kMoveThreads;
        const int first = (part + carry) * kMoveThreads + threadIdx.x;
        constexpr int UN = 4;
        for (int r0 = first; r0 < (int)count; r0 += hop * UN) {
            unsigned d[UN], f[UN];
            float x[UN];
            int p[UN];
#pragma unroll
            for (int k = 0; k < UN; ++k)
                if (r0 + k * hop < (int)count) {
                    d[k] = __ldcg(a.dst + list + r0 + k * hop);
                    f[k] = __ldcg(a.src + list + r0 + k * hop);
                }
#pragma unroll
            for (int k = 0; k < UN; ++k)
                if (r0 + k * hop < (int)count) {
                    x[k] = a.scores[row + f[k]];
                    p[k] = a.positions[row + f[k]];
                }
#pragma unroll
            for (int k = 0; k < UN; ++k)
                if (r0 + k * hop < (int)count) {
                    a.new_scores[row + d[k]] = x[k];
                    a.new_positions[row + d[k]] = p[k];
                }
        }
        for (int i0 = first; i0 < n; i0 += hop * UN) {
            uint32_t m[UN];
            float x[UN];
            int p[UN];
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const int i = i0 + k * hop;
                m[k] = i < n ? __ldcg(mask + i / 32) : 0u;
                x[k] = i < n ? a.scores[row + i] : 0.f;
                p[k] = i < n ? a.positions[row + i] : 0;
            }
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const int i = i0 + k * hop;
                if (i < n && (m[k] >> (i % 32) & 1u)) {
                    a.new_scores[row + i] = x[k];
                    a.new_positions[row + i] = p[k];
                }
            }
        }
        return;
    }
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
        const unsigned d = __ldcg(a.dst + list + r), f = __ldcg(a.src + list + r);
        bool ok = true;
        const size_t dst = row_of(d, ok), src = row_of(f, ok);
        if (ok) {
            const uint4 kv = kc[src], vv = vc[src];
            kc[dst] = kv;
            vc[dst] = vv;
        }
    }
}

}  // namespace

// Dynamic shared memory of the selection for contexts of up to max_context tokens.
static size_t evict_smem(int max_context)
{
    const size_t n = (size_t)max_context;
    size_t bytes = (n + 31) / 32 * 8 + (max_context <= kCachedContext ? n * 4 : 0);
    if (max_context <= kSmallContext) bytes += n * 8 + n / 2 * 4 + (n / 16 + 1) * 4;
    return bytes;
}

cudaError_t launch_evict(const EvictArgs& a, int head_dim, int elt_bytes, cudaStream_t stream)
{
    const int rows = a.num_seqs * a.num_kv_heads;
    const int cpr = head_dim * elt_bytes / 16;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // Contexts of up to 4096 tokens take 256 threads (cheaper barriers) and keep all they need in shared
    // memory.  With a CTA per SM or more they also move their rows, which saves the second kernel's
    // launch and the list's way through memory; fewer CTAs would leave the moving to too few SMs.
    const bool small = a.max_context_len <= kSmallContext, fused = small && rows >= sms;
    const bool cached = a.max_context_len <= kCachedContext;
    auto kernel = cached ? evict_select_kernel<1024, kKeysCached, 0> : evict_select_kernel<1024, kFromGlobal, 0>;
    if (small) kernel = evict_select_kernel<256, kAllCached, 0>;
    if (fused) {
        switch (cpr) {
            case 8: kernel = evict_select_kernel<256, kAllCached, 8>; break;
            case 16: kernel = evict_select_kernel<256, kAllCached, 16>; break;
            case 32: kernel = evict_select_kernel<256, kAllCached, 32>; break;
            default: return cudaErrorInvalidValue;
        }
    }
    // the most that any call of this kernel needs, not this call's need: another thread's call may come between here
    // and the launch
    const size_t most = evict_smem(small ? kSmallContext : (cached ? kCachedContext : kMaxEvictContext));
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) != cudaSuccess) return e;
    kernel<<<rows, small ? 256 : 1024, evict_smem(a.max_context_len), stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || fused) return e;
    // enough CTAs to fill the device, but none with less than one step of the longest list
    const int steps = (a.move_stride + kMoveThreads / cpr - 1) / (kMoveThreads / cpr);
    int splits = (sms * 16 + rows - 1) / rows;
    splits = splits < steps ? splits : steps;
    splits = splits < 1 ? 1 : splits;
    const int carry = small ? 0 : (a.max_context_len + 8191) / 8192;
    const dim3 grid((unsigned)rows * (unsigned)(carry + splits));
    switch (cpr) {
        case 8: return launch_pdl(evict_move_kernel<8>, grid, dim3(kMoveThreads), 0, stream, a, carry, splits);
        case 16: return launch_pdl(evict_move_kernel<16>, grid, dim3(kMoveThreads), 0, stream, a, carry, splits);
        case 32: return launch_pdl(evict_move_kernel<32>, grid, dim3(kMoveThreads), 0, stream, a, carry, splits);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
