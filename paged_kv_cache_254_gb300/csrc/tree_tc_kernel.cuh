// Tree attention for launches of 17 to 128 query rows per (sequence, KV head) pair,
// on the 5th-generation tensor core: pa_multi_tc_kernel's tile, stages, roles, lazy
// rescaling and hand-offs, with ancestor masks in place of the causal limit.
//
// A row's visible keys of a 64-key stage are a 64-bit set: ones below the tree, the
// node's mask from there on.  A row of no node looks at every key, so that it never
// takes its warp off the unmasked path; its results go nowhere.  Nodes whose V is not
// finite leave the product, and the rows that see them become NaN.  The CTA finds its
// own place in the work list (tree_start), so there is no pre-pass.
//
// A kernel of its own, not a variant of pa_multi_tc_kernel: sharing the source moved
// that one's code about and cost it 3 to 4 % (8-token chunks 0.863 -> 0.902 ms).
//
// Measured: 256 sequences of 1024-8192 tokens, 8 nodes, 64 / 8 heads, d 128, bf16:
// 0.86 to 0.89 ms, 5.6 TB/s, 0.82 of the copy bandwidth; 4 of 24576-32768, 24 nodes,
// 64 / 64 heads: 0.62 to 0.65 ms, 0.87.  Bound by the softmax warps' instructions next to HBM: in
// scalar fp32 as for chunks it took 1.00 ms with the masks' code added, and stacking
// the hi and lo weights of 64 rows in one product's 128 rows (two thirds of the MMAs)
// 0.87.
//
// The tensor core cuts its fp32 sums where it could round them: 2 steps per 16 keys
// draw the outputs towards zero by 2e-9 of their size per key that one CTA sums up
// (6.5e-5 at 33,000 keys, 2.6e-4 at 131,000; half a step of bf16 is 2e-3 to 4e-3).
#pragma once

#include "multi_tc_kernel.cuh"

namespace pa {

template <int D_, int BS_, bool BF16_>
struct TreeTcTraits : TcTraits<D_, BS_, BF16_> {
    using Tc = TcTraits<D_, BS_, BF16_>;
    // the chunk kernel's barriers and scanned[2]; then its regions, and a TreeStart with a word per warp
    static constexpr int REC_OFF = (Tc::BAR_OFF + 8 * (2 * Tc::R_CAP + Tc::NBAR_FIXED + 2) + 15) / 16 * 16;
    static constexpr int XCH_OFF = REC_OFF + Tc::R_CAP * Tc::REC_BYTES;
    static constexpr int MISC_OFF = XCH_OFF + Tc::XCH_BYTES;  // TMEM base, abort flag, stage count
    static constexpr int START_OFF = MISC_OFF + 16;
    static constexpr int Q_OFF = (START_OFF + 32 + 8 * 12 + 1023) / 1024 * 1024;
    __host__ __device__ static constexpr int ring_stages(int qrows) {
        return (Tc::SMEM_CAP - 1024 - Q_OFF - Tc::HALVES * qrows * 128) / Tc::STAGE_BYTES > Tc::R_CAP
                   ? Tc::R_CAP
                   : (Tc::SMEM_CAP - 1024 - Q_OFF - Tc::HALVES * qrows * 128) / Tc::STAGE_BYTES;
    }
    // a twelfth, idle warp completes the third warpgroup, whose registers the softmax
    // warps take over (masks need more than the even share)
    static constexpr int THREADS = 32 * (Tc::SOFT_WARPS + 4);
    static_assert(ring_stages(Tc::ROWS) >= 3, "three ring stages at least (the MMA issue order relies on it)");
};

// One ring stage as the copy warp describes it to the consumers.
struct alignas(16) TreeTcStage {
    int base, kvh, t0, nkeys;    // first position of the tree, KV head, first key, keys copied (blocks x B)
    int n, ctx, q0, flags;       // nodes, context, first query row of the sequence
    int poison, seg;             // bad block id seen; segment number within the CTA
    uint32_t spoilt[2];          // stage keys (bits) whose V is not finite
};
static_assert(sizeof(TreeTcStage) == 48, "stage record");

template <class Tr>
__global__ void __launch_bounds__(Tr::THREADS, 1)
pa_tree_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const MultiParams mp) {
    constexpr int D = Tr::D, BS = Tr::BS, SB = Tr::SB, HALVES = Tr::HALVES, KEYS = Tr::KEYS;
    constexpr int SW = Tr::SOFT_WARPS;
    constexpr uint32_t IDESC_S = idesc_f16<Tr::BF16>(128, KEYS, false, false);
    constexpr uint32_t IDESC_O = idesc_f16<Tr::BF16>(128, D, false, true);
    const DecodeParams& p = mp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hkv;
    const uint32_t sbase = smem_u32(smem);
    const int qrows = Tr::q_rows(mp.q_box, G);
    const uint32_t q_half = (uint32_t)qrows * 128;            // between the Q tile's column halves
    const int R = Tr::ring_stages(qrows);                     // ring stages
    const uint32_t q_tile = sbase + Tr::Q_OFF;
    const uint32_t ring_off = Tr::Q_OFF + HALVES * q_half;
    const uint32_t ring = sbase + ring_off;
    const uint32_t bars = sbase + Tr::BAR_OFF;
    auto full = [&](int st) -> uint32_t { return bars + 8 * st; };
    auto empty = [&](int st) -> uint32_t { return bars + 8 * (R + st); };
    const uint32_t s_full = bars + 16 * R, s_free = s_full + 16, p_full = s_free + 16, pv_done = p_full + 16;
    const uint32_t q_full = pv_done + 16, q_empty = q_full + 8, fin = q_empty + 8, o_free = fin + 8;
    const uint32_t scanned = o_free + 8;                     // a stream's four warps have looked at the tree's V
    TreeTcStage* recs = reinterpret_cast<TreeTcStage*>(smem + Tr::REC_OFF);
    volatile unsigned long long* xch = reinterpret_cast<volatile unsigned long long*>(smem + Tr::XCH_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Tr::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Tr::MISC_OFF + 4);
    volatile int* n_stages = reinterpret_cast<volatile int*>(smem + Tr::MISC_OFF + 8);   // set at the end record

    if (threadIdx.x == 0) {
        for (int st = 0; st < R; ++st) {
            mbar_init(full(st), 1);
            mbar_init(empty(st), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full + 8 * b, 1);
            mbar_init(s_free + 8 * b, SW / 2);      // the four warps of the stage's stream
            mbar_init(p_full + 8 * b, SW / 2);
            mbar_init(pv_done + 8 * b, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(fin, 2);                      // the score thread and the PV thread
        mbar_init(o_free, SW / 2);              // a segment's output read: the four warps of its last stage
        mbar_init(scanned, SW / 2);
        mbar_init(scanned + 8, SW / 2);
        *abort_flag = 0;
        *n_stages = 0x7fffffff;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < Tr::XCH_BYTES / 8; i += Tr::THREADS) xch[i] = 0ull;   // tag 0: nothing yet
    if (warp == Tr::MMA_WARP) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), Tr::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == Tr::COPY_WARP && lane == 0) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // launched with programmatic stream serialization after the pre-pass:
    // the set-up above overlaps it; nothing the stream wrote is read before
    // it completes.  The merge post-pass may then be placed as CTAs retire.
    griddep_wait();
    griddep_launch_dependents();

    const int32_t* qst = mp.q_start;
    TreeTab tab;
    tab.ctx = p.context_lens;
    tab.qst = qst;
    tab.N = p.N;
    tab.groups = 1;
    tab.group_nodes = mp.group_nodes;
    tab.max_nodes = mp.max_q;
    tab.total_q = mp.total_q;
    tab.MB = p.MB;
    tab.BS = BS;
    // a sequence's tree size, or -1 when it is malformed
    auto chunk_len = [&](int s) -> int {
        const int a = __ldg(qst + s), b = __ldg(qst + s + 1), ctx = __ldg(p.context_lens + s);
        const long long n = (long long)b - a;
        const bool ok = a >= 0 && b <= mp.total_q && n >= 0 && n <= mp.max_q && n <= (ctx > 0 ? ctx : 0);
        return ok ? (int)n : -1;
    };

    // ---- malformed trees and bad context lengths: error bit, NaN rows ----
    for (int s = blockIdx.x; s < p.N; s += gridDim.x) {
        const int n = chunk_len(s);
        const int ctx = __ldg(p.context_lens + s);
        const bool bad_ctx = ctx < 0 || ctx > p.MB * BS;
        if (n >= 0 && !bad_ctx) continue;
        if (threadIdx.x == 0) set_err(p.err, PA_DEVERR_CONTEXT);
        const int a = max(0, __ldg(qst + s));
        const int b = min(mp.total_q, __ldg(qst + s + 1));
        for (long long i = (long long)a * p.Hq * D + threadIdx.x; i < (long long)b * p.Hq * D; i += Tr::THREADS)
            p.out[i] = qnan16<Tr::BF16>();
    }

    Sched sc;
    const TreeStart& at = *reinterpret_cast<TreeStart*>(smem + Tr::START_OFF);
    tree_start<Tr::THREADS>(tab, p.Hkv, SB, reinterpret_cast<long long*>(smem + Tr::START_OFF + 32),
                            reinterpret_cast<TreeStart*>(smem + Tr::START_OFF));
    sc = tree_sched(at.W, gridDim.x, SB);
    const bool has_work = (int)blockIdx.x < sc.NS;
    const long long lo = has_work ? sc.lo(blockIdx.x) : 0, hi = has_work ? sc.lo(blockIdx.x + 1) : 0;

    // 256 x 200 + 128 x 104 registers, the 384 x 168 of the launch
    if (warp >= SW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == Tr::COPY_WARP) {
            const uint64_t kv_pol = l2_evict_first();
            // ================================================================ copies
            int j = 0, st = 0, nseg = 0;            // stage, its ring slot and phase
            uint32_t ph = 0;
            bool ok = true;
            if (lane == 0) mp.starts[blockIdx.x] = at;
            auto claim = [&]() -> bool {            // lane 0: slot st free for stage j (its last use done)
                return j < R || mbar_wait_bounded(empty(st), ph ^ 1u, p.timeout_ns);
            };
            if (has_work) {
                SegIter it;
                it.gi = lo;
                it.s = at.s;
                it.kvh = at.kvh;
                it.b0 = at.b0;
                it.nb = at.nb;
                it.first = 0;
                while (ok && it.gi < hi) {
                    const int len = seg_len(it, hi);
                    const int n = chunk_len(it.s);
                    if (n > 0) {
                        const int ctx = __ldg(p.context_lens + it.s);
                        const int q0 = __ldg(qst + it.s);
                        const long long P0 = it.gi - it.b0;
                        const bool complete = sc.of(P0) == sc.of(P0 + it.nb - 1);
                        const int seg_flags = (complete ? TC_COMPLETE : 0) | (it.gi == lo ? 0 : TC_SLOT1);
                        if (lane == 0) {
                            if (nseg > 0 && !mbar_wait_bounded(q_empty, (uint32_t)((nseg - 1) & 1), p.timeout_ns)) {
                                ok = false;
                            } else {
                                mbar_arrive_expect_tx(q_full, (uint32_t)(HALVES * 128 * G * mp.q_box));
    #pragma unroll
                                for (int h = 0; h < HALVES; ++h)
                                    tma_load_3d(q_tile + h * q_half, &tmap_q, h * 64, it.kvh * G, q0, q_full);
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        ++nseg;
                        const int32_t* trow = p.block_tables + (size_t)it.s * p.MB + it.b0;
                        auto batch = [&](int from) -> int { return lane < len - from ? __ldg(trow + from + lane) : 0; };
                        int ids = batch(0), ids_next = batch(32);
                        const int nst = (len + SB - 1) / SB;
                        for (int k = 0; ok && k < nst; ++k) {
                            const int bb = k * SB;
                            if (bb > 0 && (bb & 31) == 0) {
                                ids = ids_next;
                                ids_next = batch(bb + 32);
                            }
                            const int nbs = min(SB, len - bb);
                            int idv[SB];
    #pragma unroll
                            for (int i = 0; i < SB; ++i) idv[i] = __shfl_sync(0xffffffffu, ids, (bb + i) & 31);
                            if (lane == 0) {
                                if (!claim()) {
                                    ok = false;
                                } else {
                                    int poison = 0;
    #pragma unroll
                                    for (int i = 0; i < SB; ++i)
                                        if (i < nbs && (unsigned)idv[i] >= (unsigned)p.NB) {
                                            poison = 1;
                                            idv[i] = 0;
                                        }
                                    if (poison) set_err(p.err, PA_DEVERR_BLOCK_ID);
                                    TreeTcStage& rc = recs[st];
                                    rc.base = ctx - n;
                                    rc.kvh = it.kvh;
                                    rc.spoilt[0] = rc.spoilt[1] = 0u;
                                    rc.t0 = (it.b0 + bb) * BS;
                                    rc.nkeys = nbs * BS;
                                    rc.n = n;
                                    rc.ctx = ctx;
                                    rc.q0 = q0;
                                    rc.flags = seg_flags | (k == 0 ? TC_FIRST : 0) | (k == nst - 1 ? TC_LAST : 0) |
                                               (k == nst - 2 ? TC_PENULT : 0);
                                    rc.poison = poison;
                                    rc.seg = nseg;
                                    mbar_arrive_expect_tx(full(st), (uint32_t)(nbs * BS * 128 * HALVES * 2));
                                }
                            }
                            ok = __shfl_sync(0xffffffffu, ok, 0);
                            __syncwarp();   // lane 0's claim of the slot orders the other lanes' copies
                            // the stage's copies, one box per lane (the TMA unit takes boxes
                            // one at a time, so each block's K and V go as one box each):
                            // lanes 0 .. SB - 1 the K boxes, the next SB lanes the V boxes
                            {
                                const bool kl = lane < SB;
                                const int ci = kl ? lane : lane - SB;
                                int cid = __shfl_sync(0xffffffffu, ids, (bb + (ci & (SB - 1))) & 31);
                                if ((unsigned)cid >= (unsigned)p.NB) cid = 0;   // flagged and poisoned above
                                const int y = (cid * p.Hkv + it.kvh) * BS;
                                const uint32_t dst = ring + st * Tr::STAGE_BYTES + (kl ? 0 : Tr::KV_BYTES) + ci * Tr::BLK_BYTES;
                                if (ok && lane < 2 * SB && ci < nbs) {
                                    // each block is read once: L2 evict-first
                                    if (kl)
                                        tma_load_4d_hint(dst, &tmap_k, 0, 0, 0, y / 8, full(st), kv_pol);
                                    else
                                        tma_load_3d_hint(dst, &tmap_v, 0, y, 0, full(st), kv_pol);
                                }
                            }
                            ++j;
                            if (++st == R) {
                                st = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                    seg_advance(it, len, p, tab);
                }
            }
            if (lane == 0) {
                // the end record, twice: each softmax stream takes every other stage
                for (int e = 0; e < 2 && ok; ++e) {
                    if (claim()) {
                        recs[st].flags = TC_END;
                        mbar_arrive(full(st));
                        ++j;
                        if (++st == R) {
                            st = 0;
                            ph ^= 1u;
                        }
                    } else {
                        ok = false;
                    }
                }
                if (!ok) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    // copies still in flight land before the CTA's shared memory is released
                    for (int k = j - R > 0 ? j - R : 0; k < j; ++k)
                        mbar_wait_bounded(full(k % R), (uint32_t)((k / R) & 1), p.timeout_ns);
                    if (nseg > 0) mbar_wait_bounded(q_full, (uint32_t)((nseg - 1) & 1), p.timeout_ns);
                }
            }
            __syncwarp();
        } else if (warp == Tr::MMA_WARP) {
            // ================================================================ scores
            // One thread issues S_j as soon as its inputs are ready: the copy of
            // stage j, the scores of stage j - 2 read out of its TMEM buffer
            // (s_free) and, at a segment start, the Q tile.  The PV products are
            // issued by another thread (PV_WARP), so neither kind of MMA waits
            // behind the other's inputs.  At the end record it publishes the
            // number of stages.  No progress for the wait limit: abort.
            if (lane == 0) {
                int js = 0, nseg = 0;                        // next S, Q tiles consumed
                int s_st = 0;                                // ring slot and phase of stage js
                uint32_t s_ph = 0;
                bool ok = true;
                uint64_t t_last = global_timer_ns();
                for (uint32_t spin = 0;; ++spin) {
                    if (mbar_test_wait(full(s_st), s_ph)) {
                        const int flags = recs[s_st].flags;
                        if (flags & TC_END) {
                            *n_stages = js;
                            break;
                        }
                        if ((!(flags & TC_FIRST) || mbar_test_wait(q_full, (uint32_t)(nseg & 1))) &&
                            (js < 2 || mbar_test_wait(s_free + 8 * (js & 1), (uint32_t)(((js - 2) >> 1) & 1)))) {
                            const int b = js & 1;
                            if (flags & TC_FIRST) ++nseg;
                            tc_fence_after();
                            const uint64_t qd = sdesc_sw128(q_tile, 16, 1024);
                            const uint64_t kd = sdesc_sw128(ring + s_st * Tr::STAGE_BYTES, 16, Tr::GROUP_STRIDE);
    #pragma unroll
                            for (int k = 0; k < D / 16; ++k) {      // +32 bytes per K step; per 4: Q's next half tile,
                                                                    // K's next 1024-byte atom (address >> 4)
                                mma_f16(tmem + 64 * b, qd + (uint64_t)((k / 4) * (q_half >> 4) + (k % 4) * 2),
                                        kd + (uint64_t)((k / 4) * (1024 >> 4) + (k % 4) * 2), IDESC_S,
                                        k > 0 ? 1u : 0u);
                            }
                            mma_commit(s_full + 8 * b);
                            if (flags & TC_LAST) mma_commit(q_empty);
                            ++js;
                            if (++s_st == R) {
                                s_st = 0;
                                s_ph ^= 1u;
                            }
                            t_last = global_timer_ns();
                            continue;
                        }
                    }
                    if ((spin & 63u) == 0 && (*abort_flag || global_timer_ns() - t_last > p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                }
                if (!ok) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                }
                // every MMA issued (by both threads) completes before tensor memory is released
                mma_commit(fin);
                mbar_wait_bounded(fin, 0, p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == Tr::PV_WARP) {
            // ================================================================ PV
            // One thread issues PV_j in stage order once P_j is written and, at a
            // segment start, the previous segment's output has been read; the
            // commit frees the stage's ring slot.  It stops at the number of
            // stages the score thread publishes.
            if (lane == 0) {
                int jp = 0, pv_seg = 0;
                bool ok = true;
                while (true) {
                    const int b = jp & 1;
                    bool ready = false;
                    const uint64_t t0 = global_timer_ns();
                    for (uint32_t spin = 0;; ++spin) {
                        if (jp >= *n_stages) break;
                        if (mbar_test_wait(p_full + 8 * b, (uint32_t)((jp >> 1) & 1))) {
                            ready = true;
                            break;
                        }
                        if ((spin & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                    }
                    if (!ready) break;
                    const int st = jp % R;
                    const bool first = (recs[st].flags & TC_FIRST) != 0;
                    // a segment's first PV overwrites O: the previous segment's output must have been read
                    if (first && pv_seg > 0 && !mbar_wait_bounded(o_free, (uint32_t)((pv_seg - 1) & 1), p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (first) ++pv_seg;
                    tc_fence_after();
                    const uint32_t pt = tmem + Tr::P_COL + 64 * b;
                    const uint32_t vbase = ring + st * Tr::STAGE_BYTES + Tr::KV_BYTES;
    #pragma unroll
                    for (int k = 0; k < KEYS / 16; ++k) {
                        // keys 16 k .. 16 k + 15: rows (16 k) % BS .. of block tile (16 k) / BS
                        const uint64_t bv = sdesc_sw128(vbase + ((16 * k) / BS) * Tr::BLK_BYTES + ((16 * k) % BS) * 128,
                                                        Tr::HALF_STRIDE, 1024);
                        mma_f16_ts(tmem + Tr::O_COL, pt + 8 * k, bv, IDESC_O, (first && k == 0) ? 0u : 1u);
                        mma_f16_ts(tmem + Tr::O_COL, pt + 32 + 8 * k, bv, IDESC_O, 1u);
                    }
                    mma_commit(pv_done + 8 * b);
                    mma_commit(empty(st));
                    ++jp;
                }
                if (!ok) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                }
                mma_commit(fin);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ================================================================ softmax
        // Warp w takes rows 32 (w % 4) .. + 31 (its TMEM lane quarter; thread =
        // query row) of every other stage: stream w / 4 takes the stages of its
        // parity, so the two warps of a lane quarter work on consecutive stages
        // at once.  Per row, the softmax reference is handed along a segment's
        // stages (a tagged cell, written once the stage's maximum is known); each
        // stream keeps its own partial row sum, and the segment's last stage adds
        // the other stream's.  O is one accumulator: a stage that moves the
        // reference rescales it after the previous stage's PV has completed.
        const int quarter = warp & 3, stream = warp >> 2;
        const int r = quarter * 32 + lane;                      // query row = TMEM lane
        const int stid = quarter * 32 + lane;                   // thread index within the stream
        // bounded wait whose outcome is the same on every lane of the warp
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.timeout_ns));
        };
        auto get_all = [&](const volatile unsigned long long* cell, uint32_t tag, float& v) -> bool {
            return __all_sync(0xffffffffu, xch_get(cell, tag, p.timeout_ns, v));
        };
        volatile unsigned long long* ref_cell = xch;                      // [4][ROWS] by tag % 4
        volatile unsigned long long* sum_cell = xch + 4 * Tr::ROWS;       // [4][ROWS] partial sums by segment % 4
        volatile unsigned long long* sref_cell = xch + 8 * Tr::ROWS;      // [4][ROWS] their references
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t o_addr = lane_addr + Tr::O_COL;
        const float qnan = __int_as_float(0x7fc00000);
        int j = stream, st = stream;                            // this stream's stage, its ring slot and phase
        uint32_t ph = 0;
        float m_mine = -INFINITY, l = 0.f;                      // reference of this stream's sum, the sum
        int pois = 0, cur_seg = -1, seg_kvh = 0, seg_q0 = 0;
        bool wact = false, ok = true;
        // trees: the nodes this row sees (a row of no node looks at every key, so that
        // it never takes its warp off the unmasked path; its results go nowhere)
        uint64_t sees = 0;
        bool alive = false;
        uint32_t scan_ph = 0;
        const bool flip = !(p.scale_log2 > 0.f);
        const float scale = flip ? 1.f : p.scale_log2;
        while (true) {
            if (*abort_flag) break;
            if (!wait_all(full(st), ph)) {
                ok = false;
                break;
            }
            const int flags = recs[st].flags;
            if (flags & TC_END) break;
            const int t0 = recs[st].t0, nkeys = recs[st].nkeys, ctx = recs[st].ctx, seg = recs[st].seg;
            if (seg != cur_seg) {
                const int n = recs[st].n;
                cur_seg = seg;
                seg_kvh = recs[st].kvh;
                seg_q0 = recs[st].q0;
                m_mine = -INFINITY;
                l = 0.f;
                pois = 0;
                alive = r < n * G;
                sees = alive ? node_bits(__ldg(mp.tree_masks + seg_q0 + r / G), ctx - recs[st].base) : 0;
                wact = __any_sync(0xffffffffu, alive);
            }
            pois |= recs[st].poison;
            const int b = j & 1;
            // P buffer b is free once this stream's previous PV is done.  Every warp
            // of the stream waits for it before arriving for this stage, active or
            // not: a warp that skipped ahead could otherwise count toward the
            // previous stage's P-ready phase before that stage's P was written.
            bool p_free = j < 2;
            auto p_buffer_free = [&]() -> bool {
                if (!p_free) p_free = wait_all(pv_done + 8 * b, (uint32_t)(((j - 2) >> 1) & 1));
                return p_free;
            };
            uint64_t spoilt = 0;
            // Nodes whose V holds an infinity or NaN: a weight of 0 would still spoil
            // the rows that do not see them, so their V leaves the product, and the
            // rows that do see them become NaN.  The stream's warps share the look
            // (while the scores are computed) and meet at a barrier before acting.
            const int from = max(0, recs[st].base - t0), held = min(nkeys, ctx - t0);
            if (from < held) {
                uint8_t* vt = smem + ring_off + st * Tr::STAGE_BYTES + Tr::KV_BYTES;
                auto part_of = [&](int i) -> uint4* {
                    const int key = i / (HALVES * 8), part = i % (HALVES * 8);
                    return reinterpret_cast<uint4*>(vt + (key / BS) * Tr::BLK_BYTES + (part / 8) * Tr::HALF_STRIDE +
                                                    (key % BS) * 128 + (part % 8) * 16);
                };
                uint64_t mine = 0;
                for (int i = from * HALVES * 8 + stid; i < held * HALVES * 8; i += 128)
                    if (vec_not_finite<Tr::BF16>(*part_of(i))) mine |= 1ull << (i / (HALVES * 8));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t bits = __reduce_or_sync(0xffffffffu, (uint32_t)(mine >> (32 * h)));
                    if (lane == 0 && bits) atomicOr(&recs[st].spoilt[h], bits);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(scanned + 8 * stream);
                if (!wait_all(scanned + 8 * stream, scan_ph)) {
                    ok = false;
                    break;
                }
                scan_ph ^= 1u;
                const volatile uint32_t* words = recs[st].spoilt;
                spoilt = (uint64_t)words[0] | ((uint64_t)words[1] << 32);
                if (spoilt) {                            // uniform over the stream
                    for (int i = from * HALVES * 8 + stid; i < held * HALVES * 8; i += 128)
                        if ((spoilt >> (i / (HALVES * 8))) & 1) *part_of(i) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
            }
            if (!wait_all(s_full + 8 * b, (uint32_t)((j >> 1) & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
            float x[KEYS];
            if (wact) {
                uint32_t u0[32], u1[32];
                tmem_ld32(lane_addr + 64 * b, u0);
                tmem_ld32(lane_addr + 64 * b + 32, u1);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    x[k] = __uint_as_float(u0[k]);
                    x[32 + k] = __uint_as_float(u1[k]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free + 8 * b);
            if (wact) {
                uint64_t set = ~0ull;                              // trees: the keys that this row sees here
                float mx;
                // the scores stay as they are (the scale joins the exponent's FMA), unless a
                // scale turns their order
                if (flip)
#pragma unroll
                    for (int k = 0; k < KEYS; ++k) x[k] *= p.scale_log2;
                if (alive)   // t0 < ctx <= base + 64, so the offset is in range
                    set = tree_visible(sees, recs[st].base - t0) & (nkeys < KEYS ? (1ull << nkeys) - 1 : ~0ull);
                if (!__all_sync(0xffffffffu, set == ~0ull)) {
#pragma unroll
                    for (int k = 0; k < KEYS; ++k)
                        if (!(((k < 32 ? (uint32_t)set : (uint32_t)(set >> 32)) >> (k & 31)) & 1u)) x[k] = -INFINITY;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < KEYS; k += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmaxf(m4[i], x[k + i]), x[k + 4 + i]);
                mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
                // the reference after the previous stage of the segment (other stream)
                float m_prev = -INFINITY;
                if (!(flags & TC_FIRST) && !get_all(ref_cell + (j & 3) * Tr::ROWS + r, (uint32_t)j, m_prev)) {
                    ok = false;
                    break;
                }
                if (m_prev != m_mine) {                      // references only grow along a segment
                    l *= m_mine == -INFINITY ? 0.f : ex2(m_mine - m_prev);
                    m_mine = m_prev;
                }
                const float m_new = fmaxf(m_prev, mx);
                const bool need = m_new > m_prev + Tr::TAU && alive;
                if (need) m_mine = m_new;
                if (!(flags & TC_LAST)) xch_put(ref_cell + ((j + 1) & 3) * Tr::ROWS + r, m_mine, (uint32_t)(j + 1));
                const float alpha = need ? ex2(m_prev - m_new) : 1.f;      // m_prev = -inf: 0
                if (need) l *= alpha;
                if (!(flags & TC_FIRST) && __any_sync(0xffffffffu, need)) {
                    // O holds the earlier stages once the previous stage's PV is done
                    if (!wait_all(pv_done + 8 * (b ^ 1), (uint32_t)(((j - 1) >> 1) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t u[32];
                        tmem_ld32(o_addr + 32 * c, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * alpha);
                        tmem_st32(o_addr + 32 * c, u);
                    }
                    tmem_st_wait();
                }
                const float mref = m_mine == -INFINITY ? 0.f : m_mine;      // no visible key yet: weights 0
                if (!p_buffer_free()) {
                    ok = false;
                    break;
                }
                f32x2 sum2[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 2; ++c) {            // 32 keys at a time: hi, lo columns 16 c ..
                    uint32_t hw[16], lw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        // packed: this code has to fit the instruction cache
                        split2(fma2(pair2(x[32 * c + 2 * e], x[32 * c + 2 * e + 1]), pair2(scale, scale),
                                    pair2(-mref, -mref)), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum2[e & 1] = add2(sum2[e & 1], pair2(p0, p1));
                        if constexpr (Tr::BF16) {
                            // hi: the weights cut to bf16 (their top 16 bits); lo: the exact
                            // remainders, rounded to nearest (2^-16 of a weight in all, to either
                            // side; cut as well, all outputs were drawn 2^-17 towards zero)
                            const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                            hw[e] = __byte_perm(u0, u1, 0x7632);
                            float r0, r1;
                            split2(add2(pair2(p0, p1), pair2(-__uint_as_float(u0 & 0xffff0000u),
                                                             -__uint_as_float(u1 & 0xffff0000u))), r0, r1);
                            lw[e] = pack2<true>(r0, r1);
                        } else {
                            const uint32_t hv = pack2<false>(p0, p1);
                            hw[e] = hv;
                            lw[e] = pack2<false>(p0 - lo_of<false>(hv), p1 - hi_of<false>(hv));
                        }
                    }
                    tmem_st16(lane_addr + Tr::P_COL + 64 * b + 16 * c, hw);
                    tmem_st16(lane_addr + Tr::P_COL + 64 * b + 32 + 16 * c, lw);
                }
                float sa, sb;
                split2(add2(sum2[0], sum2[1]), sa, sb);
                l += sa + sb;
                if (spoilt & set) l = qnan;
            }
            // V rows past the context or past the blocks copied are zero for the PV product
            const int vvalid = max(0, min(nkeys, ctx - t0));
            if (vvalid < KEYS) {
                uint8_t* vt = smem + ring_off + st * Tr::STAGE_BYTES + Tr::KV_BYTES;
                const int nz = (KEYS - vvalid) * HALVES * 8;
                for (int i = stid; i < nz; i += 128) {
                    const int key = vvalid + i / (HALVES * 8), part = i % (HALVES * 8);
                    *reinterpret_cast<uint4*>(vt + (key / BS) * Tr::BLK_BYTES + (part / 8) * Tr::HALF_STRIDE +
                                              (key % BS) * 128 + (part % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            if (!p_buffer_free()) {
                ok = false;
                break;
            }
            if (wact) tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * b);
            if ((flags & TC_PENULT) && wact) {
                // this stream's share of the row sums, for the segment's last stage
                xch_put(sum_cell + (seg & 3) * Tr::ROWS + r, l, (uint32_t)(seg + 1));
                xch_put(sref_cell + (seg & 3) * Tr::ROWS + r, m_mine, (uint32_t)(seg + 1));
            }
            if (flags & TC_LAST) {
                if (!wait_all(pv_done + 8 * b, (uint32_t)((j >> 1) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (wact) {
                    float L = l;
                    if (!(flags & TC_FIRST)) {
                        float l2 = 0.f, m2 = -INFINITY;
                        if (!get_all(sum_cell + (seg & 3) * Tr::ROWS + r, (uint32_t)(seg + 1), l2) ||
                            !get_all(sref_cell + (seg & 3) * Tr::ROWS + r, (uint32_t)(seg + 1), m2)) {
                            ok = false;
                            break;
                        }
                        if (m2 != -INFINITY) L += l2 * ex2(m2 - m_mine);
                    }
                    if (flags & TC_COMPLETE) {
                        uint16_t* orow = p.out + ((size_t)(seg_q0 + r / G) * p.Hq + (size_t)seg_kvh * G + r % G) * D;
                        const float inv = L == 0.f ? 0.f : 1.f / L;   // a node that sees no key: zero
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t u[32];
                            tmem_ld32(o_addr + 32 * c, u);
                            tmem_ld_wait();
                            uint32_t w[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float o0 = pois ? qnan : __uint_as_float(u[2 * k]) * inv;
                                const float o1 = pois ? qnan : __uint_as_float(u[2 * k + 1]) * inv;
                                w[k] = pack2<Tr::BF16>(o0, o1);
                            }
                            if (alive) {
                                uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                            }
                        }
                    } else {
                        float* prow = p.partials +
                                      (((size_t)blockIdx.x * 2 + ((flags & TC_SLOT1) ? 1 : 0)) * Tr::ROWS + r) *
                                          Tr::PSTRIDE;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t u[32];
                            tmem_ld32(o_addr + 32 * c, u);
                            tmem_ld_wait();
                            if (alive) {
                                float4* dst = reinterpret_cast<float4*>(prow + 32 * c);
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    float4 v;
                                    v.x = pois ? qnan : __uint_as_float(u[4 * k]);
                                    v.y = pois ? qnan : __uint_as_float(u[4 * k + 1]);
                                    v.z = pois ? qnan : __uint_as_float(u[4 * k + 2]);
                                    v.w = pois ? qnan : __uint_as_float(u[4 * k + 3]);
                                    dst[k] = v;
                                }
                            }
                        }
                        if (alive) {
                            prow[D] = m_mine;
                            prow[D + 1] = L;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
            }
            j += 2;
            st += 2;
            if (st >= R) {
                st -= R;
                ph ^= 1u;
            }
        }
        if (!ok) {
            if (lane == 0) set_err(p.err, PA_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == Tr::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, Tr::TMEM_COLS);
    }
}

template <class Tr>
cudaError_t tree_tc_launch(const MultiLaunch& L) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(L.grid, Tr::THREADS, Tr::SMEM_BYTES, L.stream, attr);
    return cudaLaunchKernelEx(&cfg, pa_tree_tc_kernel<Tr>, *L.tmap_q, *L.tmap_k, *L.tmap_v, L.p);
}

template <class Tr>
MultiKernelInfo tree_tc_info() {
    return MultiKernelInfo{&tree_tc_launch<Tr>,
                           &persistent_ctas<pa_tree_tc_kernel<Tr>, Tr::THREADS, Tr::SMEM_BYTES>, Tr::ROWS};
}

// [d == 128][bs == 32], defined in tree_tc_*.cu.
void tree_tc_table_bf16(MultiKernelInfo (&t)[2][2]);
void tree_tc_table_fp16(MultiKernelInfo (&t)[2][2]);

}  // namespace pa
