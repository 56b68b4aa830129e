// Attention of the newest tokens of ragged sequences over a paged cache of keys
// and values, bf16, on the tensor cores.
//
// out_i = sum_j w_ij v_j / sum_j w_ij, w_ij = 2^(c q_i.k_j - m_i), c = scale
// log2(e), in one pass over the keys with the running maximum m_i and sum.
//
// A tile is 128 rows = (token, head of the group) pairs that share one key head:
// tpt = floor(128 / group) tokens.  An item is two tiles of one sequence and key
// head; its keys come in chunks of 128, loaded by TMA page by page into K and V
// rings.  The kernel runs the chunks as attn3_kernel does (ac_attn3.cu holds the
// ordering argument): TMEM holds S_0 | S_1 | O_0 | O_1, softmax warpgroup t
// turns S_t(j) into P_t(j) in place, the MMA warp issues O_t += P_t(j) V_j and
// S_t(j+1) = Q_t K_{j+1}^T, so that the tensor core works on one tile while the
// softmax works on the other.  An item of one tile (a few new tokens) takes the
// even chunks on tile 0 and the odd ones on tile 1 and merges the two.
//
// What differs from attn3_kernel:
//  - keys lie in pages: a lane per page reads the block table one chunk ahead
//    and issues that page's copies; pages past the sequence's end, and pages wholly
//    before the unit's lowest visible key, are not read;
//  - a chunk that runs past the sequence's end, or begins before that key, holds
//    foreign rows (whatever the cache or the stage has there, NaN too): their scores
//    are replaced by -inf, and the MMA warp (past the end) or the V producer (before that
//    key) overwrites their V rows with zeros before P.V reads them;
//  - each row has its own range of keys [lo, hi) (causal blocks, window); a warp
//    masks only chunks that cross its rows' bounds, and stores zeros for chunks
//    none of its rows sees;
//  - units: the items of the last, partial wave over the SMs are split into
//    `nsplit` runs of chunks, so that few items fill the GPU too; their sums go
//    to the workspace unnormalised, and merge_kernel joins them.
//
// Bound by each tile's chain softmax -> P.V -> next S (tensor pipe 63% active at
// d = 128, 36% at d = 64): of some 2,900 cycles a chunk takes at d = 64, a softmax
// warp works 2,000, beside the other tile's warp for half of them, and waits 850 for
// its next S; at d = 128 3,150, 1,800 and 1,300, at the 1.4 GHz that the power limit
// leaves.  One frame of 3,600 tokens over 75,600 keys, 40 heads, d = 128: 4.97 to 5.24 ms
// on several B200s, 1.12 to 1.06 PFLOP/s; two ragged sequences of up to 2,700 tokens
// over 17,550 keys, 30 heads, d = 64: 774 to 826 us, 0.71 to 0.66.
// Every mbarrier wait is bounded; on expiry the CTA records ST_TIMEOUT, drains
// its copies and MMAs, frees TMEM and returns.
#include <algorithm>

#include "ac_cache.cuh"
#include "ac_softmax.cuh"

namespace ac {
namespace {

constexpr int CHUNK = 128;

template <int D> struct CCfg {
    static constexpr int DB = D / 64;
    static constexpr int Q_BYTES = 128 * D * 2;     // one query tile
    static constexpr int KV_BYTES = CHUNK * D * 2;  // one stage of K (or of V)
    static constexpr int KST = D == 128 ? 3 : 4, VST = D == 128 ? 2 : 4;
    static constexpr int OFF_Q = 0;                 // tile 1 at + Q_BYTES
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + VST * KV_BYTES;
    static constexpr int OFF_X = OFF_BAR + 448;     // (max, sum) of tile 1 per row, when tiles share rows
    static constexpr int OFF_SCHED = OFF_X + 128 * 8;  // ring of scheduled units
    static constexpr int SCHED = 4;                 // its depth
    static constexpr int SMEM_RAW = OFF_SCHED + 4 * SCHED + 1024;
    // threads that read each ring entry: V producer warp, MMA warp, both softmax warpgroups
    static constexpr int SCHED_READERS = 32 + 32 + 256;
    // at least 116 KB so that two CTAs never share an SM (each takes all of TMEM)
    static constexpr int SMEM = SMEM_RAW > 116 * 1024 ? SMEM_RAW : 116 * 1024;
    // warps 0-3 softmax tile 0, 4-7 softmax tile 1, 8 TMA (Q, K), 9 MMA, 10 TMA (V), 11 idle
    static constexpr int NTHREADS = 384;
    static constexpr int REGS_LAUNCH = 168, REGS_LOW = 136, REGS_HIGH = 184;
    static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= NTHREADS * REGS_LAUNCH, "register split");
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr int TM_S = 0, TM_O = 256;      // + 128 t, + D t
    static_assert(TM_O + 2 * D <= (int)TMEM_COLS, "TMEM budget");
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr int EMU_PER8 = 2;              // exponentials per 8 key pairs on the FMA pipe
};

// How the call's work is cut (host side).
struct Plan {
    int tpt;       // tokens per tile
    int blocks;    // items per sequence and key head
    int whole;     // items taken whole: units 0 .. whole - 1
    int nsplit;    // pieces of each later item
    int units;
    int *next;           // units handed out beyond the CTAs' first ones (0 between calls)
    unsigned *done;      // CTAs that are through (0 between calls)
    float *part_o;   // [units - whole, 256, D]
    float2 *part_ml; // [units - whole, 256]
};

// One unit of work, decoded alike by every role.
struct Unit {
    int s, kvh;
    int row0, nq;    // first row of the stacked tensors, tokens (<= 2 tpt; 0: nothing to do)
    int p0;          // position of the first token
    int len;         // the sequence's keys
    int c0, nch;     // chunks of this unit
    int lo;          // lowest key that any of its tokens sees
    int slot;        // partial slot, or -1: whole
    int nt;          // tiles at work
    bool two;        // two tiles of rows (else both tiles share one)
    int nc0, nc1;    // chunks of tile 0 / tile 1
};

__device__ __forceinline__ Unit decode(const CacheAttnArgs &a, const Plan &pl, int u, bool report) {
    Unit w;
    int item = u, piece = 0;
    w.slot = -1;
    if (u >= pl.whole) {
        w.slot = u - pl.whole;
        item = pl.whole + w.slot / pl.nsplit;
        piece = w.slot % pl.nsplit;
        if (pl.nsplit == 1) w.slot = -1;
    }
    const int b = item % pl.blocks, sh = item / pl.blocks;
    w.s = sh / a.kv_heads;
    w.kvh = sh - w.s * a.kv_heads;
    sequence(a, w.s, w.row0, w.nq, w.p0, w.len, report);
    const int t0 = b * 2 * pl.tpt;
    w.row0 += t0;
    w.p0 += t0;
    w.nq = max(0, min(2 * pl.tpt, w.nq - t0));
    w.c0 = w.nch = w.lo = 0;
    if (w.nq) {
        int hi, x;
        key_range(a, w.p0, w.len, w.lo, x);
        key_range(a, w.p0 + w.nq - 1, w.len, x, hi);
        if (hi > w.lo) {
            const int first = w.lo / CHUNK, all = (hi + CHUNK - 1) / CHUNK - first;
            const int np = w.slot < 0 ? 1 : pl.nsplit, per = (all + np - 1) / np;
            w.c0 = first + piece * per;
            w.nch = max(0, min(per, all - piece * per));
        }
    }
    w.two = w.nq > pl.tpt;
    const bool share = !w.two && w.nch >= 2;
    w.nt = w.two || share ? 2 : 1;
    w.nc0 = share ? (w.nch + 1) / 2 : w.nch;
    w.nc1 = share ? w.nch / 2 : (w.two ? w.nch : 0);
    return w;
}

template <int D>
__device__ __forceinline__ void issue_s(uint32_t ld, uint32_t d, uint64_t qdesc, uint64_t kdesc) {
    using C = CCfg<D>;
    constexpr uint32_t idesc = idesc_make(128, CHUNK, 1, false);
#pragma unroll
    for (int kb = 0; kb < C::DB; kb++) {
#pragma unroll
        for (int k4 = 0; k4 < 4; k4++) umma_f16_p(ld, d, qdesc + 2 * k4, kdesc + 2 * k4, idesc, (kb | k4) ? 1u : 0u);
        qdesc += (128 * 128) >> 4;
        kdesc += (CHUNK * 128) >> 4;
    }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t ld, uint32_t d, uint32_t p, uint64_t vdesc, bool first) {
    constexpr uint32_t idesc = idesc_make(128, D, 1, true);
#pragma unroll
    for (int ks = 0; ks < CHUNK / 16; ks++)
        umma_ts_f16_p(ld, d, p + ks * 8, vdesc + (uint64_t)((ks * 16 * 128) >> 4), idesc, (!first || ks > 0) ? 1u : 0u);
}

__device__ __forceinline__ void tma_load_3d_hint_p(uint32_t leader, void *dst, const CUtensorMap *map, uint64_t *bar,
                                                   int x, int y, int z, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy), "r"(leader)
        : "memory");
}

// Rows [from, to) of a V stage become zeros, for the MMAs issued after a barrier
// that the calling warp arrives on next.
template <int D> __device__ __forceinline__ void zero_rows(unsigned char *st, int from, int to, int lane) {
    for (int i = from * 8 + lane; i < to * 8; i += 32)
#pragma unroll
        for (int kb = 0; kb < CCfg<D>::DB; kb++)
            *reinterpret_cast<uint4 *>(st + kb * (CHUNK * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CacheAttnArgs a,
                      const __grid_constant__ Plan pl) {
    using C = CCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                          ~(uintptr_t)1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint64_t *q_full = bars + 0, *q_empty = bars + 1;
    uint64_t *k_full = bars + 2, *k_empty = k_full + C::KST;          // [KST]
    uint64_t *v_full = k_empty + C::KST, *v_empty = v_full + C::VST;  // [VST]
    uint64_t *s_full = v_empty + C::VST;  // [tile]: one phase per chunk
    uint64_t *p_full = s_full + 2;        // [tile]: one phase per chunk, 128 arrivals
    uint64_t *o_free = p_full + 2;        // [tile], 128 arrivals
    uint64_t *o_done = o_free + 2;        // [tile]: one phase per unit, after its last P.V
    uint64_t *xchg = o_done + 2;          // shared rows: tile 1's (max, sum) written; 128 arrivals
    uint64_t *comb_done = xchg + 1;       // shared rows: tile 0 has read O_1; 128 arrivals
    uint64_t *sched_full = comb_done + 1;           // [SCHED], 1 arrival
    uint64_t *sched_empty = sched_full + C::SCHED;  // [SCHED], SCHED_READERS arrivals
    uint64_t *drain_bar = sched_empty + C::SCHED;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(drain_bar + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < C::KST; i++) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < C::VST; i++) {
            mbar_init(v_full + i, 1);
            mbar_init(v_empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 128);
            mbar_init(o_free + i, 128);
            mbar_init(o_done + i, 1);
        }
        mbar_init(xchg, 128);
        mbar_init(comb_done, 128);
        for (int i = 0; i < C::SCHED; i++) {
            mbar_init(sched_full + i, 1);
            mbar_init(sched_empty + i, C::SCHED_READERS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // CTA i begins with unit i.  The others are handed out as CTAs get free: the
    // TMA warp draws the next one from a counter and publishes it in a shared
    // ring, which every other role reads in the same order (-1 ends it).
    const bool dealt = pl.units > (int)gridDim.x;
    volatile int *sched_ring = reinterpret_cast<volatile int *>(sm + C::OFF_SCHED);
    uint32_t sched_pos = 0;
    // the next unit for a reading role (whole warp or warpgroup); -2 on abort
    auto unit_after = [&]() -> int {
        if (!dealt) return -1;
        const int qs = (int)(sched_pos % C::SCHED);
        if (!mbar_wait_warp(sched_full + qs, (sched_pos / C::SCHED) & 1, abort_flag, a.status)) return -2;
        const int unit = sched_ring[qs];
        mbar_arrive(sched_empty + qs);
        sched_pos++;
        return unit;
    };
    // ... and for the TMA warp
    auto unit_drawn = [&]() -> int {
        if (!dealt) return -1;
        int unit = 0;
        if (lane == 0) unit = atomicAdd(pl.next, 1) + (int)gridDim.x;
        unit = __shfl_sync(0xffffffffu, unit, 0);
        if (unit >= pl.units) unit = -1;
        const int qs = (int)(sched_pos % C::SCHED);
        if (sched_pos >= (uint32_t)C::SCHED &&
            !mbar_wait_warp(sched_empty + qs, ((sched_pos / C::SCHED) - 1) & 1, abort_flag, a.status))
            return -2;
        if (lane == 0) {
            sched_ring[qs] = unit;
            mbar_arrive(sched_full + qs);
        }
        __syncwarp();
        sched_pos++;
        return unit;
    };

    if (warp >= 8) {
    regs_dec3<C::REGS_LOW>();
    if (warp == 8 || warp == 10) {
        // ------------------------------------------------------ TMA producers
        // Warp 8 loads Q and K, warp 10 loads V, converged; lane i < pages of a
        // chunk issues the copies of page i.
        const bool kq = warp == 8;
        const uint32_t leader = elect_leader();
        // K/V rows are re-read by the head's other items: keep them in L2
        const uint64_t pol_keep = l2_policy_evict_last(), pol_stream = l2_policy_evict_first();
        uint64_t *full = kq ? k_full : v_full, *empty = kq ? k_empty : v_empty;
        const int nst = kq ? C::KST : C::VST;
        unsigned char *ring = sm + (kq ? C::OFF_K : C::OFF_V);
        const CUtensorMap *map = kq ? &tmK : &tmV;
        const int page = 1 << a.page_log2, box = min(page, CHUNK);
        uint32_t qi = 0, nloads = 0;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = blockIdx.x, next_u; u >= 0 && ok; u = next_u) {
            // drawn ahead of the unit's loads: the other roles need not wait for it
            next_u = kq ? unit_drawn() : unit_after();
            if (next_u == -2) { ok = false; break; }
            const Unit w = decode(a, pl, u, kq && lane == 0);
            if (!w.nq || !w.nch) continue;
            if (kq) {
                if (qi >= 1 && !mbar_wait_warp(q_empty, (qi - 1) & 1, abort_flag, a.status)) { ok = false; break; }
                const int nqt = w.two ? 2 : 1;
                mbar_arrive_expect_tx_p(leader, q_full, nqt * C::DB * pl.tpt * a.group * 128);
                for (int t = 0; t < nqt; t++)
                    for (int kb = 0; kb < C::DB; kb++)
                        tma_load_3d_hint_p(leader, sm + C::OFF_Q + t * C::Q_BYTES + kb * (128 * 128), &tmQ, q_full,
                                           kb * 64, w.kvh * a.group, w.row0 + t * pl.tpt, pol_stream);
                qi++;
            }
            const int32_t *table = a.block_table + (long long)w.s * a.max_pages;
            // rows of the pool where chunk c's page `lane` begins; -1: none (past the
            // end, or before every window: such a page may have been given back)
            auto page_row = [&](int c) -> int {
                const int j = c * CHUNK + lane * box;
                if (lane * box >= CHUNK || j >= w.len || j + box <= w.lo) return -1;
                int id = __ldg(table + (j >> a.page_log2));
                if (id < 0 || id >= a.num_pages) {
                    set_status(a.status, ST_INVALID);
                    id = id < 0 ? 0 : a.num_pages - 1;
                }
                return ((id * a.kv_heads + w.kvh) << a.page_log2) + (j & (page - 1));
            };
            int next = page_row(w.c0);
            for (int c = 0; c < w.nch; c++) {
                const int row = next;
                if (c + 1 < w.nch) next = page_row(w.c0 + c + 1);
                // the slot's previous chunk (one pass ago) must be consumed
                if (nloads >= (uint32_t)nst && !mbar_wait_warp(empty + slot, phase ^ 1u, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                const int pages = __popc(__ballot_sync(0xffffffffu, row >= 0));
                // pages before every window, at the front of the unit's first chunk: P is
                // 0 there and V must be too (off the MMA warp's chain: 5.22 against 5.31 ms)
                const int front = kq ? 0 : (w.lo & ~(box - 1)) - (w.c0 + c) * CHUNK;
                if (front > 0) zero_rows<D>(ring + slot * C::KV_BYTES, 0, front, lane);
                mbar_arrive_expect_tx_p(leader, full + slot, (uint32_t)(pages * box * 128 * C::DB));
                __syncwarp();
#pragma unroll
                for (int kb = 0; kb < C::DB; kb++)
                    tma_load_2d_hint_p(row >= 0, ring + slot * C::KV_BYTES + kb * (CHUNK * 128) + lane * box * 128, map,
                                       full + slot, kb * 64, row, pol_keep);
                nloads++;
                if (++slot == nst) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok) {
            // wait (bounded) for every copy in flight before the CTA exits
            if (kq && qi >= 1) drain3(q_full, (qi - 1) & 1);
            for (uint32_t i = 0; i < (uint32_t)nst && i < nloads; i++)
                drain3(full + i, ((nloads - 1 - i) / (uint32_t)nst) & 1);
        }
    } else if (warp == 9) {
        // --------------------------------------------------------- MMA issuer
        const uint32_t leader = elect_leader();
        uint32_t qi = 0;
        int kslot = 0, vslot = 0;
        uint32_t kph = 0, vph = 0;
        uint32_t cnt[2] = {0, 0};  // chunks each tile has been through
        uint32_t act[2] = {0, 0};  // units each tile was active in
        bool ok = true;
        const uint64_t qdesc = sdesc_sw128(smem_u32(sm + C::OFF_Q), 16, 1024);
        const uint64_t kdesc0 = sdesc_sw128(smem_u32(sm + C::OFF_K), 16, 1024);
        const uint64_t vdesc0 = sdesc_make(smem_u32(sm + C::OFF_V), CHUNK * 128, 1024, 2u);
        auto k_next = [&]() {
            if (++kslot == C::KST) {
                kslot = 0;
                kph ^= 1u;
            }
        };
        // rows past the sequence's end become zeros (P is 0 there)
        auto zero_tail = [&](unsigned char *st, int valid) { zero_rows<D>(st, valid, CHUNK, lane); };
        // O_t += P_t V once softmax t has written its P of phase c
        auto pv_of = [&](int t, uint32_t c, uint64_t vdesc, bool first) -> bool {
            ok = mbar_wait_warp(p_full + t, c & 1, abort_flag, a.status) &&
                 (!first || act[t] == 0 || mbar_wait_warp(o_free + t, (act[t] - 1) & 1, abort_flag, a.status));
            if (!ok) return false;
            tc_fence_after();
            issue_pv<D>(leader, tmem + C::TM_O + t * D, tmem + C::TM_S + t * 128, vdesc, first);
            return true;
        };
        auto v_next = [&]() {
            if (++vslot == C::VST) {
                vslot = 0;
                vph ^= 1u;
            }
        };
        for (int u = blockIdx.x, next_u; u >= 0; u = next_u) {
            next_u = unit_after();
            if (next_u == -2) { ok = false; break; }
            const Unit w = decode(a, pl, u, false);
            if (!w.nq || !w.nch) continue;
            const int nt = w.nt;
            const bool share = !w.two && nt == 2;
            if (!mbar_wait_warp(q_full, qi & 1, abort_flag, a.status)) { ok = false; break; }
            qi++;
            // Stages in stream order.  Two tiles of rows: stage j serves chunk j
            // of both.  Shared rows: stage 2j + t serves chunk j of tile t.  A
            // stage is waited for by its first user and released after its last.
            const int nc[2] = {w.nc0, w.nc1};
            const uint64_t qd[2] = {qdesc, qdesc + (uint64_t)((w.two ? C::Q_BYTES : 0) >> 4)};
            int k_used = 0;  // K stages released in this unit
#pragma unroll
            for (int t = 0; t < 2; t++) {
                if (t >= nt) break;
                if (share || t == 0) {
                    if (!mbar_wait_warp(k_full + kslot, kph, abort_flag, a.status)) { ok = false; break; }
                    tc_fence_after();
                }
                issue_s<D>(leader, tmem + C::TM_S + t * 128, qd[t], kdesc0 + (uint64_t)((kslot * C::KV_BYTES) >> 4));
                umma_commit_p(leader, s_full + t);
                if (share || t == nt - 1) {
                    umma_commit_p(leader, k_empty + kslot);
                    k_next();
                    if (++k_used == w.nch) umma_commit_p(leader, q_empty);
                }
            }
            if (!share) {
                // both tiles' products of a chunk share its K and V stages; what they
                // need besides P is waited for first and the stages are released last, off
                // the chain P -> P.V -> S (the two ragged sequences 857 -> 775 us)
                for (int j = 0; j < w.nch; j++) {
                    const bool more = j + 1 < w.nch;
                    if (!mbar_wait_warp(v_full + vslot, vph, abort_flag, a.status)) { ok = false; break; }
                    const int valid = w.len - (w.c0 + j) * CHUNK;
                    if (valid < CHUNK) zero_tail(sm + C::OFF_V + vslot * C::KV_BYTES, valid);
                    if (more && !mbar_wait_warp(k_full + kslot, kph, abort_flag, a.status)) { ok = false; break; }
                    const uint64_t vd = vdesc0 + (uint64_t)((vslot * C::KV_BYTES) >> 4);
                    const uint64_t kd = kdesc0 + (uint64_t)((kslot * C::KV_BYTES) >> 4);
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        if (t >= nt) break;
                        if (!pv_of(t, cnt[t] + j, vd, j == 0)) break;
                        if (more) {
                            issue_s<D>(leader, tmem + C::TM_S + t * 128, qd[t], kd);
                            umma_commit_p(leader, s_full + t);
                        } else {
                            umma_commit_p(leader, o_done + t);
                        }
                    }
                    if (!ok) break;
                    umma_commit_p(leader, v_empty + vslot);
                    v_next();
                    if (more) {
                        umma_commit_p(leader, k_empty + kslot);
                        k_next();
                        if (j + 2 == w.nch) umma_commit_p(leader, q_empty);
                    }
                }
            } else {
                // tile t has stages of its own: 2j + t
                int v_used = 0;
                for (int j = 0; j < w.nc0 && ok; j++) {
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        if (j >= nc[t]) break;
                        const bool more = j + 1 < nc[t];
                        if (!mbar_wait_warp(v_full + vslot, vph, abort_flag, a.status)) { ok = false; break; }
                        const int valid = w.len - (w.c0 + v_used++) * CHUNK;
                        if (valid < CHUNK) zero_tail(sm + C::OFF_V + vslot * C::KV_BYTES, valid);
                        if (more && !mbar_wait_warp(k_full + kslot, kph, abort_flag, a.status)) { ok = false; break; }
                        if (!pv_of(t, cnt[t] + j, vdesc0 + (uint64_t)((vslot * C::KV_BYTES) >> 4), j == 0)) break;
                        umma_commit_p(leader, v_empty + vslot);
                        v_next();
                        if (!more) {
                            umma_commit_p(leader, o_done + t);
                            continue;
                        }
                        issue_s<D>(leader, tmem + C::TM_S + t * 128, qd[t], kdesc0 + (uint64_t)((kslot * C::KV_BYTES) >> 4));
                        umma_commit_p(leader, s_full + t);
                        umma_commit_p(leader, k_empty + kslot);
                        k_next();
                        if (++k_used == w.nch) umma_commit_p(leader, q_empty);
                    }
                }
            }
            if (!ok) break;
            cnt[0] += w.nc0;
            act[0]++;
            if (nt > 1) {
                cnt[1] += w.nc1;
                act[1]++;
            }
        }
        if (!ok) {
            umma_commit_p(leader, drain_bar);
            drain3(drain_bar, 0);
        }
    }
    // no code after the role split is shared by warps of different register
    // budgets: all 384 threads meet at barrier 1, then TMEM is freed
    tc_fence_before();
    named_bar_sync(1, C::NTHREADS);
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
        // the last CTA of the call puts the counters back to 0 (atomicInc wraps)
        if (dealt && lane == 0 && atomicInc(pl.done, gridDim.x - 1) == gridDim.x - 1) atomicExch(pl.next, 0);
    }
    } else {
        regs_inc3<C::REGS_HIGH>();
        // ------------------------------------------------ softmax + epilogue
        // Warpgroup t = tile t; one thread per row (= TMEM lane).
        const int t = warp >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + C::TM_S + t * 128;
        const uint32_t o_addr = tmem + lane_addr + C::TM_O + t * D;
        const int rtok = row / a.group, rhead = row - rtok * a.group;
        const float sc = a.scale_log2;
        uint32_t cnt = 0;         // chunks (= s_full / p_full phases) this tile has been through
        uint32_t units_done = 0;  // units (= o_done phases) this tile has finished
        uint32_t shares = 0;      // units with shared rows (= xchg / comb_done phases) so far
        float2 *xs = reinterpret_cast<float2 *>(sm + C::OFF_X);
        bool ok = true;
        for (int u = blockIdx.x, next_u; u >= 0; u = next_u) {
            next_u = unit_after();
            if (next_u == -2) { ok = false; break; }
            const Unit w = decode(a, pl, u, false);
            if (!w.nq) continue;
            const bool share = !w.two && w.nt == 2;
            const int tok = (w.two && t == 1 ? pl.tpt : 0) + rtok;
            const bool valid = rtok < pl.tpt && tok < w.nq;
            if (w.nch == 0) {
                // no key at all (of this piece): zeros, written by tile 0's threads
                // for the rows of both tiles
                for (int k = 0; t == 0 && k < (w.two ? 2 : 1); k++) {
                    const int i = k * pl.tpt + rtok;
                    if (rtok >= pl.tpt || i >= w.nq) continue;
                    const int head = w.kvh * a.group + rhead;
                    if (w.slot >= 0) {
                        pl.part_ml[(size_t)w.slot * 256 + k * 128 + row] = make_float2(-INFINITY, 0.f);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out.p +
                                                               (long long)(w.row0 + i) * a.out.sn +
                                                               (long long)head * a.out.sh);
                        for (int x = 0; x < D / 8; x++) dst[x] = make_uint4(0u, 0u, 0u, 0u);
                        if (a.lse) a.lse[(long long)(w.row0 + i) * a.heads + head] = -INFINITY;
                    }
                }
                continue;
            }
            if (t >= w.nt) continue;
            const int nch = t == 0 ? w.nc0 : w.nc1;
            const int cbase = w.c0 + (share ? t : 0), cstep = share ? 2 : 1;
            // this row's keys, and the warp's: chunks within [wlo, whi) need no
            // mask, chunks outside [alo, ahi) hold no key of any of its rows
            int lo = 0, hi = 0;
            if (valid) key_range(a, w.p0 + tok, w.len, lo, hi);
            const int wlo = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
            const int whi = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
            const int alo = __reduce_min_sync(0xffffffffu, valid ? lo : 0x7fffffff);
            const int ahi = __reduce_max_sync(0xffffffffu, valid ? hi : 0);
            const bool idle = !__any_sync(0xffffffffu, valid);
            float m_ref = -INFINITY, l0 = 0.f, l1 = 0.f;
            for (int j = 0; j < nch; j++) {
                const int cb = (cbase + cstep * j) * CHUNK;
                const uint32_t c = cnt + j;
                if (!mbar_wait_warp(s_full + t, c & 1, abort_flag, a.status)) { ok = false; break; }
                tc_fence_after();
                if (idle) {
                    // no row of this warp is written: its P may stay what S left
                } else if (cb >= ahi || cb + CHUNK <= alo) {
                    tmem_st32_zero(s_addr);
                    tmem_st32_zero(s_addr + 32);
                } else {
                    uint32_t s[128];
                    tmem_ld128(s_addr, s);
                    if (cb < wlo || cb + CHUNK > whi) {
                        const int from = lo - cb;
                        const uint32_t span = hi > lo ? (uint32_t)(hi - lo) : 0u;
#pragma unroll
                        for (int i = 0; i < CHUNK; i++)
                            if ((uint32_t)(i - from) >= span) s[i] = __float_as_uint(-INFINITY);
                    }
                    // row max: four independent chains of 3-input max
                    float mq[4];
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        float m = fmaxf(__uint_as_float(s[32 * q]), __uint_as_float(s[32 * q + 1]));
#pragma unroll
                        for (int i = 2; i < 32; i += 2)
                            m = fmax3(m, __uint_as_float(s[32 * q + i]), __uint_as_float(s[32 * q + i + 1]));
                        mq[q] = m;
                    }
                    const float mx = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]);
                    const float m_new = mx * sc;
                    if (j == 0) m_ref = m_new;
                    // Move the reference max (and rescale O_t and l by f) only when it
                    // grew by more than 2^8; warp-uniform because TMEM access is
                    // collective.  PV_t(j-1) is complete: S_t(j) was issued after it.
                    // Rows in use alone have a say: the others hold the next sequence's
                    // queries, or what an earlier unit left, and would decide how these round.
                    const bool rescale = j > 0 && __any_sync(0xffffffffu, valid && m_new > m_ref + 8.f);
                    float f = 1.f;
                    if (rescale) {
                        const float m_to = fmaxf(m_ref, m_new);
                        // a row with no key yet keeps f = 1 (its O and l are 0)
                        f = m_to == -INFINITY ? 1.f : ex2_approx(m_ref - m_to);
                        m_ref = m_to;
                    }
                    // a row with no key yet: all its scores are -inf and give P = 0
                    const float negm = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t scale2 = pack2(sc, sc), neg2 = pack2(negm, negm);
                    uint64_t la[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
                    uint32_t pk[32];
                    exp_pairs<C::EMU_PER8, 0, 32>(s, pk, scale2, neg2, la);
                    tmem_st32(s_addr, pk);
                    exp_pairs<C::EMU_PER8, 32, 32>(s, pk, scale2, neg2, la);
                    tmem_st32(s_addr + 32, pk);
                    if (rescale) {
#pragma unroll
                        for (int pc = 0; pc < D / 32; pc++) {
                            uint32_t o[32];
                            tmem_ld32(o_addr + pc * 32, o);
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(o_addr + pc * 32, o);
                        }
                    }
                    float a0, a1, b0, b1;
                    unpack2(la[0], a0, a1);
                    unpack2(la[1], b0, b1);
                    l0 = fmaf(l0, f, a0 + b0);
                    l1 = fmaf(l1, f, a1 + b1);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_full + t);
            }
            if (!ok) break;
            if (!mbar_wait_warp(o_done + t, units_done & 1, abort_flag, a.status)) { ok = false; break; }
            tc_fence_after();
            cnt += nch;
            units_done++;
            // m, l and the weights of O_0 and O_1 in this row's result
            float m = m_ref, l = l0 + l1, w0 = 1.f, w1 = 0.f;
            if (share) {
                // Tile 1 hands its max and sum to tile 0, which merges O_0 and O_1
                // (same TMEM lanes) with weights 2^(m_t - m); tile 1 releases O_1
                // once tile 0 has read it.
                const uint32_t ph = shares++ & 1;
                if (t == 1) {
                    xs[row] = make_float2(m, l);
                    tc_fence_before();  // O_1 is final (o_done); tile 0 reads it after xchg
                    mbar_arrive(xchg);
                    if (!mbar_wait_warp(comb_done, ph, abort_flag, a.status)) { ok = false; break; }
                    tc_fence_after();
                    tc_fence_before();
                    mbar_arrive(o_free + 1);
                    continue;
                }
                if (!mbar_wait_warp(xchg, ph, abort_flag, a.status)) { ok = false; break; }
                tc_fence_after();
                const float2 x = xs[row];
                m = fmaxf(m_ref, x.x);
                w0 = weight(m_ref, m);
                w1 = weight(x.x, m);
                l = l * w0 + x.y * w1;
            }
            const int head = w.kvh * a.group + rhead;
            __nv_bfloat16 *orow = (__nv_bfloat16 *)a.out.p + (long long)(w.row0 + tok) * a.out.sn +
                                  (long long)head * a.out.sh;
            const size_t prow = (size_t)w.slot * 256 + (w.two && t == 1 ? 128 : 0) + row;
            // a row without keys has l = 0 and O = 0
            const float inv = w.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            w0 *= inv;
            w1 *= inv;
            if (!idle) {
#pragma unroll
                for (int pc = 0; pc < D / 32; pc++) {
                    uint32_t o[32], o1[32];
                    tmem_ld32(o_addr + pc * 32, o);
                    if (share) {
                        tmem_ld32(o_addr + D + pc * 32, o1);
#pragma unroll
                        for (int i = 0; i < 32; i++)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * w0 + __uint_as_float(o1[i]) * w1);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * w0);
                    }
                    if (!valid) continue;
                    if (w.slot >= 0) {
                        uint4 *dst = reinterpret_cast<uint4 *>(pl.part_o + prow * D + pc * 32);
#pragma unroll
                        for (int i = 0; i < 8; i++) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    } else {
                        uint32_t b[16];
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            __nv_bfloat162 b2 =
                                __floats2bfloat162_rn(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                            b[i] = *reinterpret_cast<uint32_t *>(&b2);
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + pc * 32);
#pragma unroll
                        for (int i = 0; i < 4; i++) dst[i] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
                    }
                }
            }
            tc_fence_before();
            if (share) mbar_arrive(comb_done);
            mbar_arrive(o_free + t);
            if (valid) {
                if (w.slot >= 0)
                    pl.part_ml[prow] = make_float2(m, l);
                else if (a.lse)
                    a.lse[(long long)(w.row0 + tok) * a.heads + head] =
                        l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
            }
        }
        tc_fence_before();
        named_bar_sync(1, C::NTHREADS);
    }
}

// Rows of the split items: sum of the pieces' O with weights 2^(m_i - m), over
// the sum of their l.  One warp per row; bound by the pieces' bytes.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ Plan pl,
                                                    int items, int rows) {
    constexpr int E = D / 32;
    after_previous();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int it = (int)(w / rows), r = (int)(w - (long long)it * rows);
    if (it >= items) return;
    const int tok = r / a.group, head = r - tok * a.group;
    const int item = pl.whole + it, b = item % pl.blocks, sh = item / pl.blocks;
    const int s = sh / a.kv_heads, kvh = sh - s * a.kv_heads;
    int row0, nq, p0, len;
    sequence(a, s, row0, nq, p0, len, false);
    const int t = b * 2 * pl.tpt + tok;
    if (t >= nq) return;
    const size_t at = (size_t)it * pl.nsplit * 256 + (tok >= pl.tpt ? 128 + (tok - pl.tpt) * a.group : tok * a.group) + head;
    float m = -INFINITY;
    for (int i = lane; i < pl.nsplit; i += 32) m = fmaxf(m, pl.part_ml[at + (size_t)i * 256].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float l = 0.f, acc[E];
#pragma unroll
    for (int k = 0; k < E; k++) acc[k] = 0.f;
    for (int i = 0; i < pl.nsplit; i++) {
        const float2 ml = pl.part_ml[at + (size_t)i * 256];
        if (ml.y == 0.f) continue;  // no key in this piece: its O was not written
        const float f = weight(ml.x, m);
        l += f * ml.y;
        const float *o = pl.part_o + (at + (size_t)i * 256) * D + lane * E;
#pragma unroll
        for (int k = 0; k < E; k++) acc[k] += f * o[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int h = kvh * a.group + head;
    __nv_bfloat16 *o = (__nv_bfloat16 *)a.out.p + (long long)(row0 + t) * a.out.sn + (long long)h * a.out.sh + lane * E;
#pragma unroll
    for (int k = 0; k < E; k++) o[k] = __float2bfloat16(acc[k] * inv);
    if (a.lse && lane == 0)
        a.lse[(long long)(row0 + t) * a.heads + h] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(void *fn, CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const cuuint32_t ones[3] = {1, 1, 1};
    return ((EncodeFn)fn)(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int FILL = 2;
int max_slots(int num_sms) { return 2 * FILL * num_sms; }

template <int D> int launch(const CacheAttnArgs &a, const Plan &pl, int num_sms, void *encode_fn, cudaStream_t st) {
    using C = CCfg<D>;
    CUtensorMap mq, mk, mv;
    {
        // strides of a dimension of one element are never used: give them a legal value
        const cuuint64_t sh = a.heads > 1 ? (cuuint64_t)a.q.sh * 2 : (cuuint64_t)D * 2;
        const cuuint64_t sn = a.tokens > 1 ? (cuuint64_t)a.q.sn * 2 : (cuuint64_t)D * 2 * a.heads;
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.heads, (cuuint64_t)a.tokens}, strides[2] = {sh, sn};
        const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)pl.tpt};
        if (!encode(encode_fn, &mq, a.q.p, 3, dims, strides, box)) return -1;
    }
    const int page = 1 << a.page_log2;
    // a cache without pages has no keys: the maps are never used
    const void *kp = a.num_pages ? a.kp : a.q.p, *vp = a.num_pages ? a.vp : a.q.p;
    const cuuint64_t dims[2] = {(cuuint64_t)D, a.num_pages ? (cuuint64_t)a.num_pages * a.kv_heads * page : 1};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)std::min(page, CHUNK)};
    if (!encode(encode_fn, &mk, kp, 2, dims, strides, box) || !encode(encode_fn, &mv, vp, 2, dims, strides, box)) return -1;
    cache_attn_kernel<D><<<std::min(pl.units, num_sms), C::NTHREADS, C::SMEM, st>>>(mq, mk, mv, a, pl);
    note_launch();
    if (pl.nsplit > 1) {
        const int items = (pl.units - pl.whole) / pl.nsplit;
        const int rows = std::min(2 * pl.tpt, a.max_q) * a.group;
        launch_after(merge_kernel<D>, (unsigned)(((long long)items * rows + 7) / 8), 256, st, a, pl, items, rows);
    }
    return 0;
}

// The register split assumes the launch budget ptxas gave the kernel; a larger
// split would make setmaxnreg.inc wait forever, so refuse.
template <int D> int setup() {
    using C = CCfg<D>;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, cache_attn_kernel<D>) != cudaSuccess || fa.numRegs != C::REGS_LAUNCH) return -1;
    return cudaFuncSetAttribute(cache_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) ==
                   cudaSuccess
               ? 0
               : -1;
}

}  // namespace

int cache_attn_setup(int D) {
    if (cache_decode_setup(D)) return -1;
    return D == 64 ? setup<64>() : setup<128>();
}

size_t cache_attn_ws(int num_sms, int D) {
    return (size_t)max_slots(num_sms) * 256 * (D * sizeof(float) + sizeof(float2));
}

int k_cache_attn(const CacheAttnArgs &a, int num_sms, void *encode_fn, cudaStream_t st) {
    if (a.group > 128) return -1;
    const int cs = decode_cluster(a, num_sms);
    if (cs) return k_cache_decode(a, cs, st);
    Plan pl;
    pl.tpt = 128 / a.group;
    pl.blocks = (a.max_q + 2 * pl.tpt - 1) / (2 * pl.tpt);
    const long long items = (long long)a.seqs * a.kv_heads * pl.blocks;
    if (items > 0x3fffffffLL) return -1;
    // Whole items for the full waves over the SMs; the items left over are cut
    // into the number of pieces whose waves take least: a wave of pieces costs
    // their chunks plus about 3 chunks' time to start and to write out.  With
    // several sequences the items differ in length and CTAs get free at different
    // times: then the last num_sms items or more are cut in FILL pieces too, small
    // enough to fill the gaps (the two ragged sequences above 780 us without, 767 with
    // 2 pieces, 752 with 3, 750 with 4, 777 with 8; 2 keep the workspace at 79 MB).
    long long keys = a.max_kv;
    if (a.window) keys = std::min<long long>(keys, (long long)a.window + 2 * pl.tpt + a.causal_block);
    const int chunks = (int)((keys + CHUNK - 1) / CHUNK);
    int left = (int)(items % num_sms);
    pl.nsplit = 1;
    if (a.seqs > 1 && items >= num_sms && chunks >= 4 * FILL) {
        left = std::min((int)items, left + num_sms);
        pl.nsplit = FILL;
    } else if (left) {
        double best = 1e30;
        for (int n = 1; n <= std::max(1, chunks) && left * n <= max_slots(num_sms); n++) {
            const double cost = (double)((left * n + num_sms - 1) / num_sms) * ((chunks + n - 1) / n + (n > 1 ? 3 : 0));
            if (cost < best) {
                best = cost;
                pl.nsplit = n;
            }
        }
    }
    pl.whole = (int)(items - left);
    pl.units = pl.whole + left * pl.nsplit;
    pl.next = a.counters;
    pl.done = (unsigned *)(a.counters + 1);
    pl.part_o = (float *)a.ws;
    pl.part_ml = (float2 *)((char *)a.ws + (size_t)max_slots(num_sms) * 256 * a.D * sizeof(float));
    return a.D == 64 ? launch<64>(a, pl, num_sms, encode_fn, st) : launch<128>(a, pl, num_sms, encode_fn, st);
}

}  // namespace ac
