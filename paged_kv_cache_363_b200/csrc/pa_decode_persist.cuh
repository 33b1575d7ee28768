// The persistent decode kernel and its launch, shared by pa_decode (pa_decode.cu) and
// pa_decode_scores (pa_decode_scores.cu).  MODE picks what a unit does beside its attention;
// the plain form's code has nothing of the other's (it is resolved at compile time).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pa_decode_common.cuh"
#include "pa_decode_fma.cuh"
#include "pa_decode_mma.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kModePlain = 0;   // pa_decode
constexpr int kModeScores = 1;  // also writes every token's logits and every partition's (max, sum)

constexpr int kEndUnit = 1;    // no more work for this CTA
constexpr int kSplitUnit = 2;  // the sequence spans several partitions

struct UnitInfo {
    int s, kvh, part, nb, b0, first, L, flags, np, pad[3];
};

// Shared-memory budget of one CTA: two CTAs per SM, each with about 96 KB of K/V
// stages in flight, keep enough bytes moving to cover the HBM latency under load.
constexpr int kCtaSmemBudget = 110 * 1024;

// Cons: the consumer policy (tiles of Cons::B = 16 tokens); BS: the physical block
// size.  A stage holds one 16-token tile of K and of V; a block of BS tokens is
// BS / 16 consecutive tiles.
template <class Cons, int BS>
struct Persist {
    using T = typename Cons::T;
    static constexpr int D = Cons::D, G = Cons::G;
    static constexpr int TR = Cons::B;                  // tokens per stage
    static constexpr int SPB = BS / TR;                 // stages per physical block
    static constexpr int TILE_BYTES = TR * D * (int)sizeof(T);
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K tile, then V tile
    static constexpr int NCW = 4;                       // consumer warps
    static constexpr int UR = 2;                        // units held: the current one and the next
    static constexpr int MAX_PBLK = kMaxPartitionTokens / 16;
    static constexpr int QBYTES = G * D * (int)sizeof(T);
    static constexpr int SLOT_BYTES = (QBYTES + MAX_PBLK * 4 + (int)sizeof(UnitInfo) + 127) / 128 * 128;
    static constexpr int THREADS = (NCW + 2) * 32;      // consumers, tile producer, unit producer
    static constexpr int MERGE_FLOATS = NCW * G * (D + 2);
    static constexpr int NBAR_FIXED = 3 * UR + 2;
    static constexpr int FIXED_BYTES = UR * SLOT_BYTES + MERGE_FLOATS * 4 + NCW * Cons::SCRATCH_FLOATS * 4 +
                                       NBAR_FIXED * 8 + 16 + 1024;
    // Stage i of the CTA's stream is consumed by warp i % NCW.  With NSTAGES a multiple
    // of NCW the warp that waits for a stage's n-th fill also consumed its (n-1)-th, so
    // a one-bit phase parity is never stale.
    static constexpr int NSTAGES =
        cmax(NCW, cmin(24, ((kCtaSmemBudget - FIXED_BYTES - 16 * 24) / STAGE_BYTES) / NCW * NCW));
    static constexpr int OFF_SLOT = NSTAGES * STAGE_BYTES;
    static constexpr int OFF_MERGE = OFF_SLOT + UR * SLOT_BYTES;
    static constexpr int OFF_SCRATCH = OFF_MERGE + MERGE_FLOATS * 4;
    static constexpr int OFF_BAR = (OFF_SCRATCH + NCW * Cons::SCRATCH_FLOATS * 4 + 7) / 8 * 8;
    static constexpr int NBAR = 2 * NSTAGES + NBAR_FIXED;
    static constexpr int OFF_ABORT = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_ABORT + 16 + 1024;  // + slack to align the base to 1024 bytes

    static_assert(BS % TR == 0, "block size must be a multiple of the stage tile");
    static_assert(NSTAGES % NCW == 0, "stage ring must be a multiple of the consumer warps");
    static_assert(TILE_BYTES % 1024 == 0, "tiles keep the 1024-byte alignment of the swizzle atoms");
    static_assert(QBYTES % 16 == 0, "q rows are bulk-copied");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// Moves 16-token tile h of one physical block's K and V into a stage; completion is
// counted on bar.
template <class Cons, int BS>
__device__ __forceinline__ void issue_tile(unsigned char* stage, const DecodeArgs& a, const CUtensorMap* tk,
                                           const CUtensorMap* tv, int phys, int kvh, int h, uint64_t* bar,
                                           uint64_t policy)
{
    using P = Persist<Cons, BS>;
    mbar_arrive_expect_tx(bar, 2 * P::TILE_BYTES);
    if constexpr (Cons::kTensorLoads) {
        const int row = (phys * a.num_kv_heads + kvh) * BS + h * P::TR;
        const uint32_t dk = smem_u32(stage);
#pragma unroll
        for (int hh = 0; hh < Cons::NHALF; ++hh) {
            tma_load_2d(dk + hh * Cons::HALF_BYTES, tk, hh * 64, row, bar, policy);
            tma_load_2d(dk + P::TILE_BYTES + hh * Cons::HALF_BYTES, tv, hh * 64, row, bar, policy);
        }
    } else {
        const size_t off = (((size_t)phys * a.num_kv_heads + kvh) * BS + (size_t)h * P::TR) * P::D * sizeof(typename P::T);
        bulk_g2s_hint(stage, static_cast<const unsigned char*>(a.k_cache) + off, P::TILE_BYTES, bar, policy);
        bulk_g2s_hint(stage + P::TILE_BYTES, static_cast<const unsigned char*>(a.v_cache) + off, P::TILE_BYTES,
                      bar, policy);
    }
}

template <class Cons, int BS, int MODE>
__global__ void __launch_bounds__(Persist<Cons, BS>::THREADS, 2)
    decode_persistent_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v)
{
    using P = Persist<Cons, BS>;
    using T = typename Cons::T;
    constexpr int D = P::D, B = BS, G = P::G, NCW = P::NCW, NS = P::NSTAGES, UR = P::UR, TR = P::TR,
                  SPB = P::SPB;

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::OFF_BAR);
    uint64_t* full = bars;            // stage filled (tx bytes)
    uint64_t* empty = bars + NS;      // stage consumed
    uint64_t* ufull = bars + 2 * NS;  // unit slot filled (q bytes)
    uint64_t* uempty = ufull + UR;    // unit slot released (consumers and tile producer)
    uint64_t* utab = uempty + UR;     // unit slot's block-table slice written (tile producer)
    uint64_t* mg_full = utab + UR;    // every consumer warp's state of the unit is in the merge buffer
    uint64_t* mg_free = mg_full + 1;  // the unit's finish has read the merge buffer
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::OFF_ABORT);
    float* mg_m = reinterpret_cast<float*>(smem + P::OFF_MERGE);
    float* mg_l = mg_m + NCW * G;
    float* mg_acc = mg_l + NCW * G;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int st = 0; st < NS; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], 1);
        }
        for (int u = 0; u < UR; ++u) {
            mbar_init(&ufull[u], 1);
            mbar_init(&uempty[u], 2);
            mbar_init(&utab[u], 1);
        }
        mbar_init(mg_full, NCW);
        mbar_init(mg_free, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // A CTA of the first wave starts on its own unit while the plan kernel still runs:
    // only its unit producer waits for the plan, before its second unit.  Every other
    // CTA waits here; the plan kernel's list and counters are visible after the wait.
    const bool early = (int)blockIdx.x < a.first_wave;
    const bool planless = MODE == kModeScores && a.planless != 0;  // every unit is in the first wave: no plan was made
    if (!early) pdl_wait_primary();

    auto slot = [&](int k) { return smem + P::OFF_SLOT + (k % UR) * P::SLOT_BYTES; };
    auto slot_table = [&](int k) { return reinterpret_cast<int*>(slot(k) + P::QBYTES); };
    auto slot_info = [&](int k) { return reinterpret_cast<UnitInfo*>(slot(k) + P::QBYTES + P::MAX_PBLK * 4); };

    if (warp == NCW + 1) {
        // ---------------- unit producer: takes units from the plan, fills the unit ring
        // The first unit's list entry is requested together with the pair count, not
        // after it: its index is inside the list whatever the count (the grid has at
        // most one CTA per unit the list can hold).  A first-wave CTA knows its first
        // unit without the list: partition 0 of sequence b / Hkv (the plan puts that
        // pair at list position b / Hkv).
        unsigned nunits = 0;
        uint2 e_first;
        auto plan_ready = [&]() { nunits = __ldcg(a.plan + 1) * (unsigned)a.num_kv_heads; };
        if (early) {
            const int s0 = (int)(blockIdx.x / (unsigned)a.num_kv_heads);
            e_first = make_uint2((unsigned)s0 << 11, (unsigned)clamped_context(a, s0, B, planless));
        } else {
            e_first = __ldcg(a.plan_list + blockIdx.x / (unsigned)a.num_kv_heads);
            plan_ready();
        }
        // This CTA takes no more units.  The last CTA to stop (at the end marker or on
        // a wait that gave up) resets the work counter, so the plan in the workspace
        // serves the next run as it is (one plan per decode step, one run per layer);
        // it happens while the CTAs still finish their last units, off the kernel's
        // critical path.  Lane 0 only.
        auto leave = [&]() {
            if (planless) return;
            if (atomicAdd(a.plan + 4, 1u) == gridDim.x - 1) {
                a.plan[0] = 0u;
                a.plan[4] = 0u;
            }
        };
        int first = 0;
        int k = 0;
        bool ended = false;
        for (;; ++k) {
            if (k >= UR && !mbar_wait_warp(&uempty[k % UR], ((k / UR) & 1) ^ 1, abort_flag)) {
                if (lane == 0) {
                    atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
                    leave();
                }
                *abort_flag = 1;
                break;
            }
            UnitInfo* info = slot_info(k);
            // the first unit of CTA b is unit b; later ones come from the counter
            unsigned u = blockIdx.x;
            if (planless && k > 0) {
                u = 0u;  // (nunits is 0: the end)
            } else if (k > 0) {
                if (k == 1 && early) {
                    pdl_wait_primary();
                    plan_ready();
                }
                if (lane == 0) u = gridDim.x + atomicAdd(a.plan, 1u);
                u = __shfl_sync(0xffffffffu, u, 0);
            }
            if (u >= nunits && !(k == 0 && early)) {
                if (lane == 0) {
                    info->flags = kEndUnit;
                    mbar_arrive(&utab[k % UR]);
                    mbar_arrive(&ufull[k % UR]);
                    leave();
                }
                ended = true;
                break;
            }
            const uint2 e = k == 0 ? e_first : a.plan_list[u / (unsigned)a.num_kv_heads];
            const int kvh = (int)(u % (unsigned)a.num_kv_heads);
            const int s = (int)(e.x >> 11);
            const int part = (int)(e.x & 2047u);
            const int L = (int)e.y;
            const int nblk_seq = (L + B - 1) / B;
            const int pb = (k == 0 && early) ? a.partition_blocks : (int)a.plan[2];  // equal when early
            const int b0 = part * pb;
            const int nb = max(0, min(pb, nblk_seq - b0));
            int* tab = slot_table(k);
            // A first-wave unit reads its table slice (partition 0: the row's first pb
            // entries, all inside the row) in the same trip to memory as its context
            // length, not after it; entries past the context are loaded but never used.
            const int nload = (k == 0 && early) ? min(pb, a.max_blocks_per_seq) : nb;
            for (int i = lane; i < nload; i += 32)
                tab[i] = __ldg(a.block_tables + (size_t)s * a.max_blocks_per_seq + b0 + i);
            if (lane == 0) {
                info->s = s;
                info->kvh = kvh;
                info->part = part;
                info->nb = nb;
                info->b0 = b0;
                info->first = first;
                info->L = L;
                info->flags = nblk_seq > pb ? kSplitUnit : 0;
                info->np = (nblk_seq + pb - 1) / pb;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&utab[k % UR]);  // the tile producer may start on this unit
                mbar_arrive_expect_tx(&ufull[k % UR], P::QBYTES);
                bulk_g2s(slot(k), static_cast<const T*>(a.q) + ((size_t)s * a.num_heads + (size_t)kvh * G) * D,
                         P::QBYTES, &ufull[k % UR]);
            }
            first += nb * SPB;
        }
        // No q copy may still be landing in shared memory at exit: wait for the fills of
        // the last units.  After an end marker, slot k % UR has moved on past unit k - UR
        // (a parity wait on that older phase would alias), so only units k-UR+1 .. k-1.
        if (lane == 0) {
            volatile int never = 0;
            const int j0 = k - UR + (ended ? 1 : 0);
            for (int j = j0 < 0 ? 0 : j0; j < k; ++j)
                if (!mbar_wait_bounded(&ufull[j % UR], (j / UR) & 1, &never)) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
        }
    } else if (warp == NCW) {
        // ---------------- tile producer: one thread streams K/V tiles into the stages
        if (lane == 0) {
            const uint64_t policy = policy_evict_first();
            int i = 0;  // blocks issued so far (the CTA's stream index)
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (!mbar_wait_bounded(&utab[k % UR], (k / UR) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const UnitInfo* info = slot_info(k);
                if (info->flags & kEndUnit) break;
                const int nt = info->nb * SPB;
                const int kvh = info->kvh;
                const int* tab = slot_table(k);
                int phys = 0;
                for (int j = 0; j < nt; ++j, ++i) {
                    const int st = i % NS;
                    if (i >= NS && !mbar_wait_bounded(&empty[st], ((i / NS) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (j % SPB == 0) {
                        phys = tab[j / SPB];
                        if ((unsigned)phys >= (unsigned)a.num_blocks) {
                            atomicOr(a.status, PA_DEV_BAD_BLOCK);
                            phys = 0;
                        }
                    }
                    issue_tile<Cons, BS>(smem + st * P::STAGE_BYTES, a, &tmap_k, &tmap_v, phys, kvh, j % SPB,
                                         &full[st], policy);
                }
                // done with this unit's table: the slot may be refilled once the consumers are done too
                if (ok) mbar_arrive(&uempty[k % UR]);
            }
            if (!ok) {
                atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            // no tile copy may still be landing in shared memory at exit
            volatile int never = 0;
            for (int j = i - NS < 0 ? 0 : i - NS; j < i; ++j)
                if (!mbar_wait_bounded(&full[j % NS], (j / NS) & 1, &never)) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
        }
    } else {
        // ---------------- consumers
        // At a unit's end each warp puts its state in the merge buffer and moves on to
        // the next unit without waiting.  The warp that consumed the unit's last tile
        // (usually the last to get there) waits for the other states, merges them and
        // writes the result, then frees the buffer and the unit slot.  A warp may write
        // its state for unit k only after the finish of unit k-1 has freed the buffer,
        // so arrivals on mg_full for unit k all belong to phase k, and one-bit parities
        // on both barriers are never stale.
        Cons cons;
        cons.init(reinterpret_cast<float*>(smem + P::OFF_SCRATCH) + warp * Cons::SCRATCH_FLOATS, lane);
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!mbar_wait_bounded(&ufull[k % UR], (k / UR) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const UnitInfo* info = slot_info(k);
            if (info->flags & kEndUnit) break;
            const int first = info->first, nt = info->nb * SPB, L = info->L;
            const int tok0 = info->b0 * B;  // first token of the unit
            cons.begin_unit(reinterpret_cast<const T*>(slot(k)), a.scale_log2);
            for (int i = first + ((warp - first % NCW) + NCW) % NCW; i < first + nt; i += NCW) {
                const int st = i % NS;
                if (!mbar_wait_bounded(&full[st], (i / NS) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                unsigned char* stage = smem + st * P::STAGE_BYTES;
                float* lg = nullptr;
                if constexpr (MODE == kModeScores)
                    lg = a.logits + (((size_t)info->s * a.num_kv_heads + info->kvh) * a.max_context_len + tok0 +
                                     (i - first) * TR) * G;
                cons.template block<MODE == kModeScores>(stage, stage + P::TILE_BYTES,
                                                         min(TR, L - tok0 - (i - first) * TR), lg);
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            if (!ok) break;
            if (k > 0 && !mbar_wait_bounded(mg_free, (k - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            cons.end_unit(mg_m, mg_l, mg_acc, warp);
            __syncwarp();
            if (lane == 0) mbar_arrive(mg_full);
            const int finisher = ((first + nt - 1) % NCW + NCW) % NCW;
            if (warp == finisher) {
                if (!mbar_wait_bounded(mg_full, k & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const bool split = (info->flags & kSplitUnit) != 0;
                finish_unit_warp<T, D, G, NCW, MODE == kModeScores>(a, mg_m, mg_l, mg_acc, info->s, info->kvh,
                                                                    info->part, split, first % NCW, lane);
                // Without a plan this is the CTA's only unit, and the whole sequence's: the weights follow here.
                // (With one, a second kernel adds them: a warp that left the stream for the 3 us that takes held
                // the ring up, 69 -> 81 us on 128 sequences of 16 to 4096 tokens.)
                const bool score = planless && L > 0;
                float hm[G], hinv[G];
                const float* lg = nullptr;
                float* sc = nullptr;
                if (score) {
                    unit_stats<G, NCW>(mg_m, mg_l, first % NCW, hm, hinv);
                    const size_t row = (size_t)info->s * a.num_kv_heads + info->kvh;
                    lg = a.logits + row * a.max_context_len * G;
                    sc = a.scores + row * a.score_stride;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(mg_free);
                    mbar_arrive(&uempty[k % UR]);
                }
                if (score) {
                    WeightTokens<G, 32, 2> w;
                    for (int i = 0; i < L; i += 64) {
                        w.load(lg, sc, i, L, lane);
                        w.add(sc, i, L, L, lane, hm, hinv);
                    }
                }
            }
        }
        if (!ok) {
            if (lane == 0) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
            *abort_flag = 1;
        }
    }
}

// CTAs of the persistent kernel resident on the current device at once (cached per device).
template <class Cons, int BS, int MODE>
cudaError_t resident_ctas(int* out)
{
    using P = Persist<Cons, BS>;
    static std::atomic<int> cached[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int d = dev & 63;
    int v = cached[d].load();
    if (v == 0) {
        e = cudaFuncSetAttribute(decode_persistent_kernel<Cons, BS, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 P::SMEM);
        if (e != cudaSuccess) return e;
        int occ = 0, sms = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, decode_persistent_kernel<Cons, BS, MODE>, P::THREADS,
                                                          P::SMEM);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        v = (occ < 1 ? 1 : occ) * sms;
        cached[d].store(v);
    }
    *out = v;
    return cudaSuccess;
}

// Plan, persistent kernel and merge of one call (kModePlain, kModeScores).
template <class Cons, int BS, int MODE>
cudaError_t launch_persistent(const DecodeArgs& a, cudaStream_t stream)
{
    using P = Persist<Cons, BS>;
    CUtensorMap tk, tv;
    std::memset(&tk, 0, sizeof(tk));
    std::memset(&tv, 0, sizeof(tv));
    if constexpr (Cons::kTensorLoads) {
        if (a.phases & kDecodeRun) {
            const uint64_t rows = (uint64_t)a.num_blocks * a.num_kv_heads * BS;
            auto map = MODE == kModePlain ? tensor_map : encode_pool_map;
            cudaError_t e = map(&tk, a.k_cache, rows, P::D, P::TR);
            if (e != cudaSuccess) return e;
            e = map(&tv, a.v_cache, rows, P::D, P::TR);
            if (e != cudaSuccess) return e;
        }
    }
    int ctas = 0;
    cudaError_t e = resident_ctas<Cons, BS, MODE>(&ctas);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.num_kv_heads * a.num_seqs * a.num_partitions;
    const unsigned grid = (unsigned)(units < ctas ? units : ctas);
    DecodeArgs args = a;
    args.num_ctas = (int)grid;
    // An automatic partition starts at 1024 tokens instead of 512 when units twice as long still balance and
    // halving the partitions saves merge work: at least three (sequence, kv head) pairs per CTA with a context
    // bound of 3072 tokens or more (long sequences split into half as many partitions), or at least ten pairs
    // per CTA (many sequences just over one partition).  Plan and run calls take the same arguments, so they
    // make the same choice.
    const int64_t pairs_all = (int64_t)a.num_seqs * a.num_kv_heads;
    if (a.adaptive && a.partition_blocks * BS == 512 &&
        ((pairs_all >= 3LL * grid && a.max_context_len >= 3072) || pairs_all >= 10LL * grid))
        args.partition_blocks = 1024 / BS;
    // The first wave: with the partition fixed, CTA b < first_wave starts on kv head
    // b % Hkv of partition 0 of sequence b / Hkv without waiting for the plan.  The plan
    // grows an automatic partition only when the tokens of all sequences exceed
    // 4 x partition x CTAs, which the bound num_seqs x max_context_len rules out here.
    // Only behind the call's own plan kernel, which itself starts when everything before it has finished: a run on an
    // earlier plan may follow a kernel that lets its dependents start (another run, an unsplit pa_cross_attention, a
    // pa_decode_scores in one launch) and whose output may be this run's q.
    args.planless = MODE == kModeScores && a.num_partitions == 1 && units <= ctas ? 1 : 0;
    const bool fixed_partition =
        !a.adaptive || (int64_t)a.num_seqs * a.max_context_len <= 4LL * args.partition_blocks * BS * (int64_t)grid;
    const int64_t pairs0 = (int64_t)a.num_seqs * a.num_kv_heads;
    const bool behind_plan = (a.phases & kDecodePlan) != 0;
    args.first_wave = (fixed_partition && behind_plan) || args.planless ? (int)(pairs0 < (int64_t)grid ? pairs0 : (int64_t)grid) : 0;

    if (a.was_planless) *a.was_planless = args.planless;
    if (args.planless) {
        // no kernel of this call comes before it, so it may not overlap the one that does
        decode_persistent_kernel<Cons, BS, MODE><<<grid, P::THREADS, (size_t)P::SMEM, stream>>>(args, tk, tv);
        return cudaGetLastError();
    }
    if (a.phases & kDecodePlan) {
        // one CTA; fewer threads for small batches keep its barriers short
        const int plan_threads = a.num_seqs <= 256 ? 256 : (a.num_seqs <= 512 ? 512 : 1024);
        decode_plan_kernel<<<1, plan_threads, 0, stream>>>(args, BS);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!(a.phases & kDecodeRun)) return cudaSuccess;
    e = launch_pdl(decode_persistent_kernel<Cons, BS, MODE>, dim3(grid), dim3(P::THREADS), (size_t)P::SMEM, stream,
                   args, tk, tv);
    if (e != cudaSuccess || a.num_partitions <= 1 || MODE == kModeScores) return e;
    return launch_merge<typename Cons::T, P::D>(args, BS, stream);
}

template <typename T, int MODE, int D, int B>
cudaError_t dispatch_group(const DecodeArgs& a, int group, cudaStream_t stream)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        switch (group) {
            case 1: return launch_persistent<FmaConsumer<T, D, 16, 1>, B, MODE>(a, stream);
            case 2: return launch_persistent<MmaConsumer<D, 16, 2>, B, MODE>(a, stream);
            case 4: return launch_persistent<MmaConsumer<D, 16, 4>, B, MODE>(a, stream);
            case 8: return launch_persistent<MmaConsumer<D, 16, 8>, B, MODE>(a, stream);
            default: return cudaErrorInvalidValue;
        }
    } else {
        switch (group) {
            case 1: return launch_persistent<FmaConsumer<T, D, 16, 1>, B, MODE>(a, stream);
            case 2: return launch_persistent<FmaConsumer<T, D, 16, 2>, B, MODE>(a, stream);
            case 4: return launch_persistent<FmaConsumer<T, D, 16, 4>, B, MODE>(a, stream);
            case 8: return launch_persistent<FmaConsumer<T, D, 16, 8>, B, MODE>(a, stream);
            default: return cudaErrorInvalidValue;
        }
    }
}

template <typename T, int MODE, int D>
cudaError_t dispatch_block(const DecodeArgs& a, int block_size, int group, cudaStream_t stream)
{
    switch (block_size) {
        case 16: return dispatch_group<T, MODE, D, 16>(a, group, stream);
        case 32: return dispatch_group<T, MODE, D, 32>(a, group, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <typename T, int MODE>
cudaError_t dispatch_dim(const DecodeArgs& a, int head_dim, int block_size, int group, cudaStream_t stream)
{
    switch (head_dim) {
        case 64: return dispatch_block<T, MODE, 64>(a, block_size, group, stream);
        case 128: return dispatch_block<T, MODE, 128>(a, block_size, group, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace pa
