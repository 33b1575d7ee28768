// Attention of packed query rows to one block table each, without a mask, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory), for sm_100a.
//
// What it computes: an entry's rows are its members (query tokens) x the G query heads of
// one kv head, at most 128; all of them attend to the same tokens [kv0, kv0 + kvlen) of one
// block table.  With x = scale * q . K in base-2 units the rows keep a running maximum m, the
// sum l of 2^(x - m) and the weighted sum of V rows, and end in out = O / l (and
// lse = ln 2 * (m + log2 l)), or, when a table's tokens are split into chunks, in the state
// (m, l, O) that the merge kernel below joins.
//
// Few rows share a table (a decode step's requests, one or a few target tokens), so the K/V
// bytes bound it: every K/V byte is loaded once for all rows of the tile.  A 128-row tile is
// padded by whatever the group lacks, which costs nothing: a 64-token tile of K and V (32 KB
// at D = 128) takes 0.74 us at a 148th of the measured copy rate, its two products 0.27 us.
//
// A CTA runs every grid-th unit (entry, kv head), there and back; two CTAs per SM, each with
//   - warps 4 and 5: K and V by TMA, a block and kv head per box (a box per half of the
//     columns took 1 to 2 us more of 70 to 97), 128-byte swizzle, rings of ST stages that run
//     on across units;
//   - warp 6 (one thread): S = Q K^T (M = 128, N = 64) into one of two tensor-memory buffers
//     and O += P V (A = P from tensor memory, V MN-major); S of the next tile is issued before
//     P V of this one, so the tensor core works while the softmax does;
//   - warps 0-3: the softmax, a thread per row, which also fetch the rows of Q (cp.async,
//     swizzled by hand: members may be any rows) while the unit before ends.  Warps without a
//     valid row only keep the barriers going.
// P goes as bf16 over its S: one rounding of at most 2^-8 of each weight, which the sum l
// does not see; it averages out over a row's tokens to the size of the output's own rounding.
// O is rescaled only when the maximum grows by more than 8 (a weight is then at most 2^8).
// Every wait is bounded; on expiry the CTA raises PA_DEV_WAIT_TIMEOUT, drains its own copies
// and MMAs, frees its tensor memory and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "pa_group.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;      // rows of an MMA tile
constexpr int kTok = 64;        // tokens per K/V tile
constexpr int kNBox = kTok / 16;  // blocks per K/V tile, at most (a TMA box is a block's rows)
constexpr int kThreads = 224;   // 4 softmax warps, producers of K and of V, MMA issuer
constexpr int kKWarp = 4, kVWarp = 5, kMmaWarp = 6;
constexpr uint32_t kTmemCols = 256;  // S 0..63 and 64..127 (P over their first 32), O 128..
constexpr float kLazy = 8.f;    // base-2 units

// QR: the rows of Q kept in shared memory (a unit's most).  The MMA always takes 128 rows: those past QR
// are whatever lies behind Q (the K stages), give rows of S and O that nobody reads, and leave 16 KB more
// for K and V where few rows share them.
template <int D, int QR>
struct Cfg {
    static constexpr int NH = D / 64;             // 64-column halves
    static constexpr int QHALF = QR * 128;        // bytes of a half of Q
    static constexpr int ATOM = 8 * 128;          // 8 rows of a half of K or V (the halves of 8 rows lie together)
    static constexpr int TILE = NH * kTok * 128;
    static constexpr int ST = (D == 128 ? 1 : 2) * (QR == 64 ? 3 : 2);  // stages of K and of V
    static constexpr int OFF_K = NH * QHALF;
    static constexpr int OFF_V = OFF_K + ST * TILE;
    static constexpr int OFF_BAR = OFF_V + ST * TILE;
    static constexpr int NBAR = 4 * ST + 8;       // k_full, k_empty, v_full, v_empty [ST], q_full, s_full[2], p_full[2],
                                                  // o_done, o_free, drain
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
};
static_assert(2 * (Cfg<128, 64>::SMEM + 1024) <= 227 * 1024 && 2 * (Cfg<128, 128>::SMEM + 1024) <= 227 * 1024 &&
                  2 * (Cfg<64, 64>::SMEM + 1024) <= 227 * 1024 && 2 * (Cfg<64, 128>::SMEM + 1024) <= 227 * 1024,
              "two CTAs per SM");
static_assert(Cfg<64, 64>::OFF_K + Cfg<64, 64>::ST * Cfg<64, 64>::TILE >= 128 * 128 &&
                  Cfg<128, 64>::OFF_K + Cfg<128, 64>::ST * Cfg<128, 64>::TILE >= Cfg<128, 64>::QHALF + 128 * 128,
              "128 rows from either half of Q lie inside the tiles");

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pack2f(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

// (x0, x1) = (s0, s1) * b + c, elementwise over the pairs b and c
__device__ __forceinline__ void ffma2(float& x0, float& x1, uint32_t s0, uint32_t s1, uint64_t b, uint64_t c)
{
    asm("{\n\t.reg .b64 ra, rd;\n\tmov.b64 ra, {%2, %3};\n\t"
        "fma.rn.f32x2 rd, ra, %4, %5;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(x0), "=f"(x1)
        : "r"(s0), "r"(s1), "l"(b), "l"(c));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The entry of a unit, or an empty one past the end.  Every role asks for a unit's entry a whole unit before
// it needs it, so that no trip to memory stands between two units.
__device__ __forceinline__ GroupItem load_item(const GroupArgs& a, unsigned unit, unsigned nunits)
{
    if (unit >= nunits) return GroupItem{0, 0, 0, 0, 0, 0, {0, 0}};
    const int4* p = reinterpret_cast<const int4*>(a.items + unit / (unsigned)a.num_kv_heads);
    const int4 x = __ldcg(p), y = __ldcg(p + 1);
    GroupItem it;
    it.table_row = x.x;
    it.row0 = x.y;
    it.members = x.z;
    it.chunk = x.w;
    it.kv0 = y.x;
    it.kvlen = y.y;
    return it;
}

template <int D, int G, int QR>
__global__ void __launch_bounds__(kThreads, 2)
    group_attention_kernel(const __grid_constant__ GroupArgs a, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v)
{
    using C = Cfg<D, QR>;
    constexpr int ST = C::ST, NH = C::NH;
    // dynamic shared memory starts on a 1024-byte boundary here (no static part; there is no room for a slack)
    extern __shared__ __align__(1024) unsigned char smem[];
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
        return;
    }
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + ST;
    uint64_t* v_full = k_empty + ST;
    uint64_t* v_empty = v_full + ST;
    uint64_t* q_full = v_empty + ST;   // a unit's Q written (4 warps)
    uint64_t* s_full = q_full + 1;     // [2] S = Q K^T in tensor memory
    uint64_t* p_full = s_full + 2;     // [2] P written (4 warps)
    uint64_t* o_done = p_full + 2;     // P V finished
    uint64_t* o_free = o_done + 1;     // a unit's O read out (4 warps)
    uint64_t* drain = o_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(drain + 1) + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(q_full, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(o_done, 1);
        mbar_init(o_free, 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_primary();       // the plan's entries are visible from here on
    pdl_launch_dependents();  // after it: a kernel that only needs the plan may start now
    const unsigned nunits = __ldcg(a.counts) * (unsigned)a.num_kv_heads;
    // This CTA's k-th unit, there and back: entries come longest first, so each pair of rounds is the same for all.
    auto unit_at = [&](unsigned k) {
        return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    };

    if (warp == kKWarp || warp == kVWarp) {
        const bool is_k = warp == kKWarp;
        uint64_t* full = is_k ? k_full : v_full;
        uint64_t* empty = is_k ? k_empty : v_empty;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        const uint32_t ring = smem_u32(smem) + (is_k ? C::OFF_K : C::OFF_V);
        const uint64_t pol = policy_evict_normal();
        const int B = a.block_size;
        bool ok = true;
        int t = 0;  // tiles issued
        // physical block of box `lane` of tile j of a unit
        auto lookup = [&](const GroupItem& it, int j) -> int {
            const int tok = j * kTok + lane * B;
            return lane < kTok / B && tok < it.kvlen
                       ? __ldg(a.block_tables + (size_t)it.table_row * a.max_blocks_per_seq + (it.kv0 + tok) / B)
                       : 0;
        };
        GroupItem it = load_item(a, unit_at(0), nunits), nit = load_item(a, unit_at(1), nunits);
        int next = lookup(it, 0);
        unsigned u;
        for (unsigned k = 0; (u = unit_at(k)) < nunits && ok; ++k) {
            const GroupItem after = load_item(a, unit_at(k + 2), nunits);
            const int kvh = (int)(u % (unsigned)a.num_kv_heads);
            const int n = (it.kvlen + kTok - 1) / kTok;
            if (n == 0) next = lookup(nit, 0);
            for (int j = 0; j < n; ++j, ++t) {
                int phys = next;
                next = j + 1 < n ? lookup(it, j + 1) : lookup(nit, 0);
                const int nbox = min(kTok, it.kvlen - j * kTok + B - 1) / B;
                if ((unsigned)phys >= (unsigned)a.num_blocks) {
                    atomicOr(a.status, PA_DEV_BAD_BLOCK);
                    phys = 0;
                }
                const int grp = (phys * a.num_kv_heads + kvh) * (B / 8);
                int groups[kNBox];
#pragma unroll
                for (int b = 0; b < kNBox; ++b) groups[b] = __shfl_sync(0xffffffffu, grp, b);
                const int st = t % ST;
                // one thread issues the boxes (lanes of a warp that each issue one take turns, and take longer)
                if (lane == 0) {
                    if (t >= ST && !mbar_wait_bounded(&empty[st], ((t / ST) & 1) ^ 1, abort_flag)) ok = false;
                    if (ok) {
                        mbar_arrive_expect_tx(&full[st], (uint32_t)(nbox * B * 128 * NH));
#pragma unroll
                        for (int b = 0; b < kNBox; ++b)
                            if (b < nbox)
                                tma_load_4d(ring + st * C::TILE + b * B * 128 * NH, map, 0, 0, 0, groups[b], &full[st], pol);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
            }
            it = nit;
            nit = after;
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            // nothing may still be landing in shared memory when the CTA exits
            volatile int never = 0;
            for (int i = max(0, t - ST); i < t; ++i)
                if (!mbar_wait_bounded(&full[i % ST], (i / ST) & 1, &never)) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t idesc_qk = umma_idesc_bf16(kRows, kTok, false);
            constexpr uint32_t idesc_pv = umma_idesc_bf16(kRows, D, true);
            const uint32_t sq = smem_u32(smem), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
            // S of tile t (the K stages' position), `first`: its unit's Q has to be waited for
            int units = 0;  // units whose first S was issued
            auto issue_qk = [&](int t, bool first) -> bool {
                // The buffer held P of tile t - 2: after its P V has finished.  Inside a unit that is
                // the last one issued; at a unit's start P V of tile t - 1 is issued too, and a one-bit
                // parity is only good for the last one, so that one is waited for.
                const int last = first ? t - 1 : t - 2;
                if (last >= 0 && !mbar_wait_bounded(o_done, last & 1, abort_flag)) return false;
                if (first && !mbar_wait_bounded(q_full, units++ & 1, abort_flag)) return false;
                if (!mbar_wait_bounded(&k_full[t % ST], (t / ST) & 1, abort_flag)) return false;
                tc_fence_after_sync();
                const uint32_t kb = sk + (t % ST) * C::TILE;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t kk = (k & 3) * 32;
                    umma_bf16_ss(tmem + (t & 1) * kTok, umma_desc_sw128(sq + (k >> 2) * C::QHALF + kk, 16, 1024),
                                 umma_desc_sw128(kb + (k >> 2) * C::ATOM + kk, 16, NH * C::ATOM), idesc_qk, k > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[t & 1]);
                umma_commit(&k_empty[t % ST]);
                return true;
            };
            bool ok = true;
            int t = 0;       // tiles whose P V was issued
            int done = 0;    // units with tokens finished
            auto tiles_of = [&](unsigned unit) {
                return unit < nunits ? (__ldcg(&a.items[unit / (unsigned)a.num_kv_heads].kvlen) + kTok - 1) / kTok : 0;
            };
            int n = tiles_of(unit_at(0)), nn = tiles_of(unit_at(1));
            if (n > 0) ok = issue_qk(0, true);
            for (unsigned k = 0; ok && unit_at(k) < nunits; ++k) {
                const int after = tiles_of(unit_at(k + 2));
                for (int j = 0; j < n && ok; ++j, ++t) {
                    if (j + 1 < n && !(ok = issue_qk(t + 1, false))) break;
                    if (!mbar_wait_bounded(&p_full[t & 1], (t >> 1) & 1, abort_flag) ||
                        (j == 0 && done > 0 && !mbar_wait_bounded(o_free, (done - 1) & 1, abort_flag)) ||
                        !mbar_wait_bounded(&v_full[t % ST], (t / ST) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t vb = sv + (t % ST) * C::TILE, p = tmem + (t & 1) * kTok;
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        umma_bf16_ts(tmem + 128, p + k * 8, umma_desc_sw128(vb + k * 2 * NH * C::ATOM, C::ATOM, NH * C::ATOM), idesc_pv,
                                     (j > 0 || k > 0) ? 1u : 0u);
                    umma_commit(o_done);
                    umma_commit(&v_empty[t % ST]);
                }
                done += n > 0 ? 1 : 0;
                n = nn;
                nn = after;
                if (ok && n > 0) ok = issue_qk(t, true);
            }
            if (!ok) {
                atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            umma_commit(drain);
            volatile int never = 0;
            if (!mbar_wait_bounded(drain, 0, &never)) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
        }
    } else {
        const int r = threadIdx.x;  // row of the tile
        const int member = r / G, head = r % G;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const bool neg = a.scale_log2 < 0.f;
        const float sl = neg ? -a.scale_log2 : a.scale_log2;
        const uint64_t slp = pack2f(sl, sl);
        bool ok = true;
        int t = 0;
        auto query_row = [&](const GroupItem& it) {
            const int i = it.row0 + max(0, min(member, it.members - 1));
            return a.rows && it.members > 0 ? __ldg(a.rows + i) : i;
        };
        // this row of the unit's Q into shared memory, 16 bytes at a time
        auto fetch_q = [&](const GroupItem& it, int row, int kvh) {
            if (member >= it.members) return;
            const char* src = static_cast<const char*>(a.q) +
                              (((size_t)row * a.num_heads) + (size_t)kvh * G + head) * (D * 2);
            const uint32_t dst = smem_u32(smem) + r * 128;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                cp_async16(dst + (c >> 3) * C::QHALF + (((c & 7) ^ (r & 7)) << 4), src + c * 16);
        };
        auto q_ready = [&]() {
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        };
        GroupItem it = load_item(a, unit_at(0), nunits), nit = load_item(a, unit_at(1), nunits);
        int row = query_row(it);
        if (it.kvlen > 0) {
            fetch_q(it, row, (int)(unit_at(0) % (unsigned)a.num_kv_heads));
            q_ready();
        }
        unsigned u;
        for (unsigned k = 0; (u = unit_at(k)) < nunits; ++k) {
            const GroupItem after = load_item(a, unit_at(k + 2), nunits);
            const int nrow = query_row(nit);
            const int kvh = (int)(u % (unsigned)a.num_kv_heads);
            const int nkvh = (int)(unit_at(k + 1) % (unsigned)a.num_kv_heads);
            const int n = (it.kvlen + kTok - 1) / kTok;
            const bool valid = member < it.members;
            const bool active = (warp * 32) / G < it.members;  // the warp has a valid row
            const size_t o_row = (size_t)row * a.num_heads + (size_t)kvh * G + head;
            if (n == 0) {
                // no tokens: the rows are zero
                if (valid) {
                    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o_row * D);
                    for (int c = 0; c < D / 8; ++c) out[c] = make_uint4(0, 0, 0, 0);
                    if (a.lse) a.lse[o_row] = -INFINITY;
                }
                if (nit.kvlen > 0) {
                    fetch_q(nit, nrow, nkvh);
                    q_ready();
                }
                it = nit;
                nit = after;
                row = nrow;
                continue;
            }
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j, ++t) {
                if (!mbar_wait_warp(&s_full[t & 1], (t >> 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                // every Q K^T of the unit has finished: the next unit's Q may take its place
                if (j == n - 1 && nit.kvlen > 0) fetch_q(nit, nrow, nkvh);
                const int left = it.kvlen - j * kTok;  // tokens from this tile on
                if (active) {
                    uint32_t sr[2][32];
                    tmem_ld32(tmem + (t & 1) * kTok + lane_base, sr[0]);
                    tmem_ld32(tmem + (t & 1) * kTok + 32 + lane_base, sr[1]);
                    tmem_wait_ld();
                    if (neg) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) sr[c][e] ^= 0x80000000u;
                    }
                    if (left < kTok) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c * 32 + e >= left) sr[c][e] = __float_as_uint(-INFINITY);
                    }
                    float mx[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(sr[c][e]));
                    const float mraw = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                             fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                    const float m_new = fmaxf(m_used, mraw == -INFINITY ? -INFINITY : mraw * sl);
                    // (rows that are not valid hold whatever was in shared memory: they may not cause the others work)
                    const bool rescale = valid && m_used != -INFINITY && m_new > m_used + kLazy;
                    const float alpha = rescale ? ex2(m_used - m_new) : 1.f;
                    if (rescale || m_used == -INFINITY) m_used = m_new;
                    const float mref = m_used == -INFINITY ? 0.f : m_used;
                    const uint64_t mrp = pack2f(-mref, -mref);
                    float rs[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            ffma2(x0, x1, sr[c][2 * e], sr[c][2 * e + 1], slp, mrp);
                            float p0 = ex2(x0), p1 = ex2(x1);
                            if (left < kTok) {  // (-inf * 0 is no -inf: a scale of zero)
                                p0 = c * 32 + 2 * e < left ? p0 : 0.f;
                                p1 = c * 32 + 2 * e + 1 < left ? p1 : 0.f;
                            }
                            rs[(e & 1) * 2] += p0;
                            rs[(e & 1) * 2 + 1] += p1;
                            p[c * 16 + e] = pack_bf16(p0, p1);
                        }
                    tmem_st32(tmem + (t & 1) * kTok + lane_base, p);
                    l = l * alpha + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
                    if (__any_sync(0xffffffffu, rescale)) {
                        // O may be changed once the last P V has finished
                        if (!mbar_wait_warp(o_done, (t - 1) & 1, abort_flag)) ok = false;
                        tc_fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tmem + 128 + lane_base + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tmem + 128 + lane_base + c * 32, o);
                        }
                    }
                    tmem_wait_st();
                }
                if (!ok) break;
                if (left < kTok) {
                    // rows past the tokens: their weight is 0, and 0 must not meet a NaN left in the pool
                    if (!mbar_wait_warp(&v_full[t % ST], (t / ST) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    for (int i = r; i < (kTok - left) * NH * 8; i += 128) {
                        const int vr = left + i / (NH * 8), h = (i >> 3) % NH;
                        *reinterpret_cast<uint4*>(smem + C::OFF_V + (t % ST) * C::TILE + ((vr >> 3) * NH + h) * C::ATOM +
                                                  (vr & 7) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                // S of this tile was issued before P V of the tile before it, which may still be waiting for a
                // slower warp.  The wait for this tile's P V below is on a one-bit parity, so P V of the tile
                // before has to be known finished first, and while this tile's cannot be.
                if (j > 0 && j == n - 1 && !mbar_wait_warp(o_done, (t - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t & 1]);
            }
            if (!ok) break;
            if (nit.kvlen > 0) q_ready();
            if (!mbar_wait_warp(o_done, (t - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            if (active) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tmem + 128 + lane_base + c * 32, o);
                    tmem_wait_ld();
                    if (valid && it.chunk < 0) {
                        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o_row * D + c * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint4 pk;
                            pk.x = pack_bf16(__uint_as_float(o[e * 8 + 0]) * inv, __uint_as_float(o[e * 8 + 1]) * inv);
                            pk.y = pack_bf16(__uint_as_float(o[e * 8 + 2]) * inv, __uint_as_float(o[e * 8 + 3]) * inv);
                            pk.z = pack_bf16(__uint_as_float(o[e * 8 + 4]) * inv, __uint_as_float(o[e * 8 + 5]) * inv);
                            pk.w = pack_bf16(__uint_as_float(o[e * 8 + 6]) * inv, __uint_as_float(o[e * 8 + 7]) * inv);
                            out[e] = pk;
                        }
                    } else if (valid) {
                        uint4* acc = reinterpret_cast<uint4*>(
                            a.ws_acc + (o_row * a.num_partitions + it.chunk) * D + c * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = make_uint4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
                    }
                }
                if (valid) {
                    if (it.chunk >= 0) {
                        *reinterpret_cast<float2*>(a.ws_ml + (o_row * a.num_partitions + it.chunk) * 2) =
                            make_float2(m_used, l);
                    } else if (a.lse) {
                        a.lse[o_row] = row_lse(m_used, l);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            it = nit;
            nit = after;
            row = nrow;
        }
        if (!ok) {
            cp_async_wait_all();
            if (lane == 0) atomicOr(a.status, PA_DEV_WAIT_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial states of the listed rows, a warp per (row, query head): M = max m_p,
// out = sum 2^(m_p - M) acc_p / sum 2^(m_p - M) l_p, in list order of the states.  Eight
// states are in flight at a time; a lane owns D / 32 columns.
template <int D>
__global__ void __launch_bounds__(128) group_merge_kernel(const GroupArgs a)
{
    constexpr int EPL = D / 32, CH = 8;
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const unsigned total = __ldcg(a.counts + 1) * (unsigned)a.num_heads;
    for (unsigned w = blockIdx.x * 4 + (threadIdx.x >> 5); w < total; w += gridDim.x * 4) {
        const uint2 e = __ldcg(a.merge_list + w / (unsigned)a.num_heads);
        const int h = (int)(w % (unsigned)a.num_heads);
        const int np = (int)e.y;
        const size_t row = (size_t)e.x * a.num_heads + h;
        const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * a.num_partitions;
        const float* acc = a.ws_acc + row * a.num_partitions * D + lane * EPL;
        float M = -INFINITY;
        for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldcg(ml + p).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float num[EPL], den = 0.f;
#pragma unroll
        for (int k = 0; k < EPL; ++k) num[k] = 0.f;
        for (int c = 0; c < np; c += CH) {
            float x[CH][EPL];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const float* src = acc + (size_t)min(c + i, np - 1) * D;
                if constexpr (EPL == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                    x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                    x[i][0] = v.x; x[i][1] = v.y;
                }
            }
            float wt = 0.f;  // lane i < 8: the weight of state c + i
            if (lane < CH && c + lane < np) {
                const float2 v = __ldcg(ml + c + lane);
                wt = state_weight(v.x, v.y, M);
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
        const float inv = den > 0.f ? 1.f / den : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D + lane * EPL;
        if constexpr (EPL == 4) {
            uint2 pk;
            pk.x = pack_bf16(num[0] * inv, num[1] * inv);
            pk.y = pack_bf16(num[2] * inv, num[3] * inv);
            *reinterpret_cast<uint2*>(out) = pk;
        } else {
            *reinterpret_cast<uint32_t*>(out) = pack_bf16(num[0] * inv, num[1] * inv);
        }
        if (a.lse && lane == 0) a.lse[row] = row_lse(M, den);
    }
}

// pa_cross_attention's plan: one entry per (sequence, tile of query tokens, chunk of its tokens), the tiles
// of a chunk next to each other (they read the same K/V), and the query rows of sequences with several
// chunks for the merge.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads, 1) cross_plan_kernel(const CrossArgs a, int T, int D, int ctas)
{
    __shared__ unsigned s_steps, s_tiles, s_rows, s_class[kLenClasses], s_merges, s_over;
    __shared__ int s_longest;
    __shared__ int s_q0[kPlanThreads], s_n[kPlanThreads], s_len[kPlanThreads];
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, S = a.num_seqs;
    const int cap = min(a.max_context_len, table_tokens(a.g.max_blocks_per_seq, a.g.block_size));
    const bool split = a.max_chunks > 1;
    if (tid < kLenClasses) s_class[tid] = 0;
    if (tid == 0) {
        s_steps = s_tiles = s_rows = 0;
        s_merges = s_over = 0;
        s_longest = 0;
    }
    // rows and tokens of sequence s; no rows where its data is bad
    auto load = [&](int s, bool flag) {
        const int q0 = __ldg(a.q_start + s), q1 = __ldg(a.q_start + s + 1), L = __ldg(a.context_lens + s);
        const bool bad = q0 < 0 || q1 > a.num_query_tokens || q1 < q0 || q1 - q0 > a.max_query_len || L < 0 || L > cap;
        if (bad && flag) atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
        s_q0[tid] = q0;
        s_n[tid] = bad ? 0 : q1 - q0;
        s_len[tid] = L;
    };
    const bool one = S <= kPlanThreads;  // a batch this small is loaded once
    // f(rows, tokens) for this thread's sequences
    auto each = [&](bool first, auto f) {
        for (int s = tid; s < S; s += kPlanThreads) {
            if (first || !one) load(s, first);
            if (s_n[tid] > 0) f(s_n[tid], s_len[tid]);
        }
    };
    // (sums may wrap for absurd batches: the chunk length is then a poor one, and no more)
    unsigned steps = 0, tiles = 0, nrows = 0;
    int longest = 0;
    each(true, [&](int rows, int L) {
        steps += (unsigned)((rows + T - 1) / T) * (unsigned)((L + kTok - 1) / kTok);
        tiles += (unsigned)((rows + T - 1) / T);
        nrows += (unsigned)rows;
        longest = max(longest, L);
    });
    __syncthreads();
    int chunk = 0;
    if (split) {
        longest = __reduce_max_sync(0xffffffffu, longest);
        steps = __reduce_add_sync(0xffffffffu, steps);
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        nrows = __reduce_add_sync(0xffffffffu, nrows);
        if (lane == 0 && nrows) {
            atomicAdd(&s_steps, steps);
            atomicAdd(&s_tiles, tiles);
            atomicAdd(&s_rows, nrows);
            atomicMax(&s_longest, longest);
        }
        __syncthreads();
        chunk = plan_chunk((float)s_steps * (float)a.g.num_kv_heads, (float)s_tiles * (float)a.g.num_kv_heads, ctas, s_longest,
                           (float)s_rows * (float)a.g.num_heads, a.max_chunks, D, false);
    }
    // tokens of a sequence's chunks, all the same but the last, and their number
    auto chunks_of = [&](int L, int& per) {
        if (!split || L <= chunk) {
            per = max(L, 1);
            return 1;
        }
        const int want = (L + chunk - 1) / chunk;
        per = ((L + want - 1) / want + kTok - 1) / kTok * kTok;
        return (L + per - 1) / per;
    };
    const int top = split ? max(chunk, 1) : max(a.max_context_len, 1);
    each(false, [&](int rows, int L) {
        int per;
        const int n = chunks_of(L, per);
        atomicAdd(&s_class[len_class(per, top)], (unsigned)(n * ((rows + T - 1) / T)));
    });
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
        if (lane == 31) s_over = x;  // all entries
    }
    __syncthreads();
    const unsigned entries = s_over;
    GroupItem* items = const_cast<GroupItem*>(a.g.items);
    uint2* merges = const_cast<uint2*>(a.g.merge_list);
    const unsigned room = (unsigned)a.g.max_entries, mroom = (unsigned)a.g.max_merges;
    for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
        if (!one) {
            __syncthreads();
            if (s0 + tid < S) load(s0 + tid, false);
            __syncthreads();
        }
        for (int i = warp; i < min(kPlanThreads, S - s0); i += kPlanThreads / 32) {
            const int q0 = s_q0[i], rows = s_n[i], L = s_len[i];
            if (rows == 0) continue;
            const int tiles = (rows + T - 1) / T;
            int per;
            const int nch = chunks_of(L, per);
            unsigned i0 = 0, m0 = 0;
            if (lane == 0) {
                i0 = atomicAdd(&s_class[len_class(per, top)], (unsigned)(tiles * nch));
                m0 = nch > 1 ? atomicAdd(&s_merges, (unsigned)rows) : 0u;
            }
            i0 = __shfl_sync(0xffffffffu, i0, 0);
            m0 = __shfl_sync(0xffffffffu, m0, 0);
            // rows listed twice (q_start running backwards elsewhere) can ask for more than there is room for
            const bool fits = i0 + tiles * nch <= room && (nch == 1 || m0 + rows <= mroom);
            if (!fits && lane == 0) atomicOr(a.g.status, PA_DEV_BAD_CONTEXT);
            for (int k = lane; k < tiles * nch; k += 32) {
                if (i0 + k >= room) break;
                const int ch = nch > 1 ? k / tiles : 0, tile = k - ch * tiles;
                GroupItem it{};
                if (fits) {
                    it.table_row = s0 + i;
                    it.row0 = q0 + tile * T;
                    it.members = min(T, rows - tile * T);
                    it.chunk = nch > 1 ? ch : -1;
                    it.kv0 = ch * per;
                    it.kvlen = min(per, L - ch * per);
                }
                items[i0 + k] = it;
            }
            if (nch > 1)
                for (int k = lane; k < rows; k += 32)
                    if (m0 + k < mroom) merges[m0 + k] = make_uint2((unsigned)(q0 + k), fits ? (unsigned)nch : 0u);
        }
    }
    __syncthreads();
    if (tid == 0) {
        unsigned* counts = const_cast<unsigned*>(a.g.counts);
        counts[0] = min(entries, room);
        counts[1] = min(s_merges, mroom);
    }
}

int sm_count()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int D, int G, int QR>
cudaError_t launch_group_dgq(const GroupArgs& a, int ctas, cudaStream_t stream)
{
    using C = Cfg<D, QR>;
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    cudaError_t e = encode_pool_atoms(&tk, a.k_cache, rows, D, a.block_size);
    if (e != cudaSuccess) return e;
    if ((e = encode_pool_atoms(&tv, a.v_cache, rows, D, a.block_size)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(group_attention_kernel<D, G, QR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  C::SMEM)) != cudaSuccess)
        return e;
    const int64_t units = (int64_t)a.max_entries * a.num_kv_heads;
    const unsigned grid = (unsigned)std::min<int64_t>(units, ctas);
    return launch_pdl(group_attention_kernel<D, G, QR>, dim3(grid), dim3(kThreads), (size_t)C::SMEM, stream, a, tk, tv);
}

template <int D, int G>
cudaError_t launch_group_dg(const GroupArgs& a, int tile_rows, int ctas, cudaStream_t stream)
{
    return tile_rows == 64 ? launch_group_dgq<D, G, 64>(a, ctas, stream) : launch_group_dgq<D, G, 128>(a, ctas, stream);
}

template <int D>
cudaError_t launch_group_d(const GroupArgs& a, int group, int tile_rows, int ctas, cudaStream_t stream)
{
    switch (group) {
        case 1: return launch_group_dg<D, 1>(a, tile_rows, ctas, stream);
        case 2: return launch_group_dg<D, 2>(a, tile_rows, ctas, stream);
        case 4: return launch_group_dg<D, 4>(a, tile_rows, ctas, stream);
        case 8: return launch_group_dg<D, 8>(a, tile_rows, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int group_resident_ctas(int sms) { return 2 * sms; }

// Many query rows: two query tiles of 128 rows per CTA share every K/V tile (pa_prefill.cu), where a sequence
// fills them on average and there are enough of them to keep a third of the SMs busy.  Measured at head_dim
// 128, tiles shared / this file's kernel, us:
//   16 sequences of 1500 tokens, 32 query heads on 8: 64 rows 45.9 / 51, 128 rows 77.6 / 90
//   4 sequences of 2000 tokens, 32 on 8: 64 rows (32 pairs of tiles) 50 / 43.8, 128 rows (64) 51.5 / 56.5
//   64 sequences of 1500 tokens, 32 on 8: 32 rows (128 of a pair's 256) 115 / 95, 64 rows 141 / 146
//   16 sequences of 1500 tokens, 16 on 16: 64 rows 66 / 49.7, 256 rows 79 / 91.5; 64 of 100 rows 203 / 160
static bool cross_many_rows(int64_t rows, int64_t max_rows, int seqs, int group, int num_kv_heads, int sms)
{
    return max_rows * group >= 256 && rows * group >= 192LL * seqs && rows * group / 256 * num_kv_heads >= sms / 3;
}

cudaError_t launch_group(const GroupArgs& a, int head_dim, int group, int tile_rows, int ctas, cudaStream_t stream)
{
    return head_dim == 64 ? launch_group_d<64>(a, group, tile_rows, ctas, stream)
                          : launch_group_d<128>(a, group, tile_rows, ctas, stream);
}

cudaError_t launch_group_merge(const GroupArgs& a, int head_dim, cudaStream_t stream)
{
    const int64_t ctas = ((int64_t)a.max_merges * a.num_heads + 3) / 4;
    const unsigned grid = (unsigned)std::min<int64_t>(ctas, 16LL * sm_count());
    return head_dim == 64 ? launch_pdl(group_merge_kernel<64>, dim3(grid), dim3(128), 0, stream, a)
                          : launch_pdl(group_merge_kernel<128>, dim3(grid), dim3(128), 0, stream, a);
}

cudaError_t launch_cross(const CrossArgs& a, int head_dim, int group, cudaStream_t stream)
{
    const int sms = sm_count(), ctas = group_resident_ctas(sms);
    if (head_dim == 128 &&
        cross_many_rows(a.num_query_tokens, a.max_query_len, a.num_seqs, group, a.g.num_kv_heads, sms)) {
        PrefillArgs p{};
        p.out = a.g.out;
        p.q = a.g.q;
        p.k_cache = a.g.k_cache;
        p.v_cache = a.g.v_cache;
        p.block_tables = a.g.block_tables;
        p.context_lens = a.context_lens;
        p.q_start = a.q_start;
        p.status = a.g.status;
        p.sched = const_cast<unsigned*>(a.g.counts);
        p.num_seqs = a.num_seqs;
        p.num_heads = a.g.num_heads;
        p.num_kv_heads = a.g.num_kv_heads;
        p.max_blocks_per_seq = a.g.max_blocks_per_seq;
        p.num_blocks = a.g.num_blocks;
        p.block_size = a.g.block_size;
        p.num_query_tokens = a.num_query_tokens;
        p.max_query_len = a.max_query_len;
        p.scale_log2 = a.g.scale_log2;
        p.lse = a.g.lse;
        p.max_context_len = a.max_context_len;
        p.order = reinterpret_cast<int*>(const_cast<GroupItem*>(a.g.items));  // (as many entries as sequences at least)
        return launch_cross_rows(p, group, a.num_query_tokens, a.max_query_len, stream);
    }
    const int tile_rows = (int64_t)a.max_query_len * group <= 64 ? 64 : 128;
    cross_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, tile_rows / group, head_dim, ctas);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((e = launch_group(a.g, head_dim, group, tile_rows, ctas, stream)) != cudaSuccess) return e;
    return a.max_chunks > 1 ? launch_group_merge(a.g, head_dim, stream) : cudaSuccess;
}

}  // namespace pa
