// Tree attention for launches of more than 128 query rows per (sequence, KV
// head) pair, on the 5th-generation tensor core: two 128-row tiles per CTA over
// one stream of keys.
//
// Mathematics: as pa_multi_tc_kernel with ancestor masks (online softmax in base
// 2 with a lazily moved reference; weights as a hi + lo pair of 16-bit values, so
// the products keep ~16 bits of each weight).  Rows r = i * g + hh of node i and
// head hh; a group of up to 256 rows (256 / g nodes) is one pass over the pair's
// keys, tile t its rows 128 t .. 128 t + 127.  Keys come in stages of 128:
//
//   S_t  = Q_t K^T   M 128, N 128, K = head_dim   (Q, K: K-major swizzled tiles)
//   O_t += P_t V     M 128, N = head_dim, K 128   (P from tensor memory, V MN-major)
//
// What bounds it: each tile's chain of scores, softmax and products, and the tensor
// core.  A stage costs 2 * (1 + 2) * 512 cycles of MMA at head_dim 128 (the PV
// product runs twice, hi and lo) for 64 KB of keys and values, which HBM delivers in
// about 2800; it takes about 5000.  Two tiles share each copied stage, so the keys
// are read once per 256 rows, and tile 1 follows tile 0 by its score product, so that
// one tile's softmax runs beside the other's products.  N = 128 because an MMA of
// N = 64 takes as long.
//
// Measured: 64 sequences of 1024-8192 tokens, 64 nodes, 64 / 8 heads, d 128, bf16:
// 0.76 to 0.79 ms, 0.79 PFLOP/s with each product counted once (0.40 of cuBLAS).  The
// softmax is short of instructions, not of units: with its loops over the 128 scores
// unrolled, the masks among them and both tiles in step it took 0.92 ms (on a box where it
// takes 0.765 now); 0.90 with
// the weights handed over by the quarter and the wait for the next keys before the
// one for the products, 0.86 with rolled loops, 0.82 with the tiles apart, 0.77 with
// masks and signs out of the loops.  16 softmax warps, two to a row, took 0.89 ms
// (unrolled 1.11).  The products' issue stays unrolled: rolled, an MMA takes 130 cycles to
// issue instead of 64.
//
// Tensor memory (512 columns): S_0, S_1 at 0 and 128, O_0, O_1 at 256 and 384.  P_t
// overwrites S_t, 32 keys at a time (16 columns of hi, 16 of lo, in the 32 columns
// that held their scores), each thread its own row after it has read the row's
// scores.  The next S_t is issued once PV_t has completed, so a tile's chain is
// S, softmax, PV, and its rows' state never leaves their threads.
//
// Roles (384 threads, one CTA per SM):
//   warps 0-3, 4-7   softmax of tile 0, 1: thread = row = TMEM lane
//   warp 8           copies: Q tiles per segment, K and V per stage, one TMA box
//                    per block and operand, a ring of 128-key slots (K and V
//                    alternate)
//   warp 9, 10       MMAs of tile 0, 1 (one thread each)
//   warp 11          looks at each V slot before the products may use it: zeroes
//                    the rows past the context, and takes out nodes whose V is not
//                    finite (their rows would spoil rows that do not see them)
//
// A tile without rows in a segment takes part in every hand-off and skips the
// work.  Every wait is bounded (PA_DEVERR_TIMEOUT).
#pragma once

#include "multi_tc_kernel.cuh"

namespace pa {

template <int D_, int BS_, bool BF16_>
struct WideTraits {
    static constexpr int D = D_;
    static constexpr int BS = BS_;
    static constexpr bool BF16 = BF16_;
    static constexpr int TILE = 128;                         // rows of a tile (M)
    static constexpr int ROWS = 2 * TILE;
    static constexpr int KEYS = 128;                         // keys per stage
    static constexpr int SB = KEYS / BS;                     // blocks per stage
    static constexpr int HALVES = D / 64;
    static constexpr int SLOT_BYTES = KEYS * D * 2;          // a stage's K, or its V
    static constexpr int GROUP_STRIDE = HALVES * 1024;       // between 8-key groups of K
    static constexpr int HALF_STRIDE = BS * 128;             // between the column halves of a V block tile
    static constexpr int BLK_BYTES = HALVES * HALF_STRIDE;
    static constexpr int SMEM_BYTES = 227 * 1024;
    static constexpr int Q_HALF = TILE * 128;                // one column half of a Q tile
    static constexpr int Q_BYTES = 2 * HALVES * Q_HALF;
    static constexpr int NREC = 8;                           // stage records in use at most: slots / 2 + 2
    static constexpr int R_CAP = 8;
    // full, empty, ready; s_full, p_part[4], pv_done; q_full, q_empty; fin; described; lead, follow
    static constexpr int NBAR = 3 * R_CAP + 2 * 6 + 2 + 2 + NREC + 2;
    static constexpr int REC_OFF = (8 * NBAR + 15) / 16 * 16;
    static constexpr int MISC_OFF = REC_OFF + NREC * 48;
    static constexpr int START_OFF = MISC_OFF + 16;          // a TreeStart, a word per warp
    static constexpr int Q_OFF = (START_OFF + 32 + 8 * 12 + 1023) / 1024 * 1024;
    static constexpr int OUT_OFF = Q_OFF + Q_BYTES;          // per softmax warp: 32 rows of 128 bytes on their way out
    static constexpr int OUT_BYTES = 32 * 128;
    static constexpr int RING_OFF = OUT_OFF + 8 * OUT_BYTES;
    static constexpr int R_FIT = (SMEM_BYTES - 1024 - RING_OFF) / SLOT_BYTES;
    static constexpr int R = R_FIT > R_CAP ? R_CAP : R_FIT;  // ring slots
    static constexpr int THREADS = 384;
    static constexpr int COPY_WARP = 8, MMA_WARP = 9, LOOK_WARP = 11;
    static constexpr int TMEM_COLS = 512;
    static constexpr int O_COL = 256;
    static constexpr int PSTRIDE = D + 4;
    static constexpr float TAU = 8.f;                        // lazy-rescale threshold (log2 units)
    static_assert(R >= 4 && R / 2 + 2 <= NREC, "ring");
};

// Keep uses of loaded tensor memory behind the wait that precedes this.
__device__ __forceinline__ void after_wait(uint32_t (&u)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(u[k]));
}

// One stage as the copy warp describes it to the others.
struct alignas(16) WideStage {
    int base, kvh, t0, nkeys;     // first position of the tree, KV head, first key, keys copied
    int n, ctx, q0, flags;        // nodes of the group, context, the group's first query row
    int poison, seg;
    uint32_t spoilt[2];           // nodes (bits) whose V is not finite, as far as this stage holds them
};
static_assert(sizeof(WideStage) == 48, "stage record");

template <class Tr>
__global__ void __launch_bounds__(Tr::THREADS, 1)
pa_tree_wide_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const MultiParams mp) {
    constexpr int D = Tr::D, BS = Tr::BS, SB = Tr::SB, HALVES = Tr::HALVES, KEYS = Tr::KEYS, R = Tr::R;
    constexpr uint32_t IDESC_S = idesc_f16<Tr::BF16>(128, KEYS, false, false);
    constexpr uint32_t IDESC_O = idesc_f16<Tr::BF16>(128, D, false, true);
    const DecodeParams& p = mp.d;
    const int seqs = p.N;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hkv, gs = 31 - __clz(G);           // a power of two
    const uint32_t sbase = smem_u32(smem);
    const uint32_t q_base = sbase + Tr::Q_OFF, ring = sbase + Tr::RING_OFF;
    auto full = [&](int st) -> uint32_t { return sbase + 8 * st; };
    auto empty = [&](int st) -> uint32_t { return sbase + 8 * (Tr::R_CAP + st); };
    auto ready = [&](int st) -> uint32_t { return sbase + 8 * (2 * Tr::R_CAP + st); };
    const uint32_t tile_bars = sbase + 8 * 3 * Tr::R_CAP;
    auto s_full = [&](int t) -> uint32_t { return tile_bars + 48 * t; };
    auto p_part = [&](int t, int c) -> uint32_t { return tile_bars + 48 * t + 8 + 8 * c; };
    auto pv_done = [&](int t) -> uint32_t { return tile_bars + 48 * t + 40; };
    const uint32_t q_full = tile_bars + 96, q_empty = q_full + 8, fin = q_empty + 8;   // fin[2]
    const uint32_t described = fin + 16;                      // [NREC] the stage's record is written
    // tile 1's scores of a stage come after tile 0's, tile 0's next ones after those have been issued
    const uint32_t lead = described + 8 * Tr::NREC, follow = lead + 8;
    WideStage* recs = reinterpret_cast<WideStage*>(smem + Tr::REC_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Tr::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Tr::MISC_OFF + 4);

    if (threadIdx.x == 0) {
        for (int st = 0; st < R; ++st) {
            mbar_init(full(st), 1);
            mbar_init(empty(st), 2);                // both tiles' products are done with it
            mbar_init(ready(st), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            for (int c = 0; c < 4; ++c) mbar_init(p_part(t, c), 4);   // the tile's four warps
            mbar_init(pv_done(t), 1);
            mbar_init(fin + 8 * t, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        for (int i = 0; i < Tr::NREC; ++i) mbar_init(described + 8 * i, 1);
        mbar_init(lead, 1);
        mbar_init(follow, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
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
    griddep_wait();                 // the launch before is complete
    griddep_launch_dependents();

    const int32_t* qst = mp.q_start;
    // a sequence's tree size, or -1 when it is malformed
    auto tree_size = [&](int s) -> int {
        const int a = __ldg(qst + s), b = __ldg(qst + s + 1), ctx = __ldg(p.context_lens + s);
        const long long n = (long long)b - a;
        const bool ok = a >= 0 && b <= mp.total_q && n >= 0 && n <= mp.max_q && n <= (ctx > 0 ? ctx : 0) &&
                        ctx <= p.MB * BS;
        return ok ? (int)n : -1;
    };

    // ---- malformed trees and bad context lengths: error bit, NaN rows ----
    for (int s = blockIdx.x; s < seqs; s += gridDim.x) {
        const int ctx = __ldg(p.context_lens + s);
        if (tree_size(s) >= 0 && ctx >= 0) continue;
        if (threadIdx.x == 0) set_err(p.err, PA_DEVERR_CONTEXT);
        const int a = max(0, __ldg(qst + s));
        const int b = min(mp.total_q, __ldg(qst + s + 1));
        for (long long i = (long long)a * p.Hq * D + threadIdx.x; i < (long long)b * p.Hq * D; i += Tr::THREADS)
            p.out[i] = qnan16<Tr::BF16>();
    }

    TreeTab tab;
    tab.ctx = p.context_lens;
    tab.qst = qst;
    tab.N = seqs;
    tab.groups = mp.groups;
    tab.group_nodes = mp.group_nodes;
    tab.max_nodes = mp.max_q;
    tab.total_q = mp.total_q;
    tab.MB = p.MB;
    tab.BS = BS;
    const TreeStart& at = *reinterpret_cast<TreeStart*>(smem + Tr::START_OFF);
    tree_start<Tr::THREADS>(tab, p.Hkv, SB, reinterpret_cast<long long*>(smem + Tr::START_OFF + 32),
                            reinterpret_cast<TreeStart*>(smem + Tr::START_OFF));
    const Sched sc = tree_sched(at.W, gridDim.x, SB);
    const bool has_work = (int)blockIdx.x < sc.NS;
    const long long lo = has_work ? sc.lo(blockIdx.x) : 0, hi = has_work ? sc.lo(blockIdx.x + 1) : 0;

    if (warp >= Tr::COPY_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == Tr::COPY_WARP) {
            // ============================================================ copies
            // with one group the keys are read once per call; with more, another CTA
            // reads the same keys for the next group at about this time
            const uint64_t kv_pol = mp.groups == 1 ? l2_evict_first() : l2_evict_normal();
            if (lane == 0) mp.starts[blockIdx.x] = at;
            int item = 0, st = 0, j = 0, nseg = 0;   // ring item (two a stage), its slot and phase; stage
            uint32_t ph = 0;
            bool ok = true;
            auto claim = [&]() -> bool {             // lane 0: the slot's last use is over
                return item < R || mbar_wait_bounded(empty(st), ph ^ 1u, p.timeout_ns);
            };
            auto next_slot = [&]() {
                ++item;
                if (++st == R) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            if (has_work) {
                SegIter it{lo, at.s, at.kvh, at.b0, at.nb, 0};
                while (ok && it.gi < hi) {
                    const int len = seg_len(it, hi);
                    const int s = it.s % seqs, skip = it.s / seqs * mp.group_nodes;
                    const int size = tree_size(s), n = min(mp.group_nodes, size - skip);   // > 0: it has blocks
                    const int ctx = __ldg(p.context_lens + s), q0 = __ldg(qst + s) + skip;
                    const long long P0 = it.gi - it.b0;
                    const bool complete = sc.of(P0) == sc.of(P0 + it.nb - 1);
                    const int seg_flags = (complete ? TC_COMPLETE : 0) | (it.gi == lo ? 0 : TC_SLOT1);
                    const int tile_nodes = Tr::TILE >> gs;
                    if (lane == 0) {
                        if (nseg > 0 && !mbar_wait_bounded(q_empty, (uint32_t)((nseg - 1) & 1), p.timeout_ns)) {
                            ok = false;
                        } else {
                            const int tiles = n > tile_nodes ? 2 : 1;
                            mbar_arrive_expect_tx(q_full, (uint32_t)(tiles * HALVES * 128 * G * mp.q_box));
                            for (int t = 0; t < tiles; ++t)
#pragma unroll
                                for (int h = 0; h < HALVES; ++h)
                                    tma_load_3d(q_base + (t * HALVES + h) * Tr::Q_HALF, &tmap_q, h * 64, it.kvh * G,
                                                q0 + t * tile_nodes, q_full);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    ++nseg;
                    const int32_t* trow = p.block_tables + (size_t)s * p.MB + it.b0;
                    auto batch = [&](int from) -> int { return lane < len - from ? __ldg(trow + from + lane) : 0; };
                    int ids = batch(0), ids_next = batch(32);
                    const int nst = (len + SB - 1) / SB;
                    for (int k = 0; ok && k < nst; ++k, ++j) {
                        const int bb = k * SB;
                        if (bb > 0 && (bb & 31) == 0) {
                            ids = ids_next;
                            ids_next = batch(bb + 32);
                        }
                        const int nbs = min(SB, len - bb);
                        int cid = __shfl_sync(0xffffffffu, ids, (bb + lane) & 31);
                        const bool copies = lane < nbs;
                        const bool bad = copies && (unsigned)cid >= (unsigned)p.NB;
                        if (bad) cid = 0;
                        const bool poison = __any_sync(0xffffffffu, bad);
                        const int y = (cid * p.Hkv + it.kvh) * BS;
                        const uint32_t bytes = (uint32_t)(nbs * Tr::BLK_BYTES);
                        for (int op = 0; op < 2; ++op) {          // K, then V
                            if (lane == 0) {
                                if (!claim()) {
                                    ok = false;
                                } else {
                                    if (op == 0) {
                                        if (poison) set_err(p.err, PA_DEVERR_BLOCK_ID);
                                        WideStage& rc = recs[j % Tr::NREC];
                                        rc.base = ctx - size;
                                        rc.kvh = it.kvh;
                                        rc.t0 = (it.b0 + bb) * BS;
                                        rc.nkeys = nbs * BS;
                                        rc.n = n;
                                        rc.ctx = ctx;
                                        rc.q0 = q0;
                                        rc.flags = seg_flags | (k == 0 ? TC_FIRST : 0) | (k == nst - 1 ? TC_LAST : 0);
                                        rc.poison = poison;
                                        rc.seg = nseg;
                                        rc.spoilt[0] = rc.spoilt[1] = 0u;
                                        mbar_arrive(described + 8 * (j % Tr::NREC));
                                    }
                                    mbar_arrive_expect_tx(full(st), bytes);
                                }
                            }
                            ok = __shfl_sync(0xffffffffu, ok, 0);
                            __syncwarp();
                            if (!ok) break;
                            const uint32_t dst = ring + st * Tr::SLOT_BYTES + lane * Tr::BLK_BYTES;
                            if (copies) {
                                if (op == 0)
                                    tma_load_4d_hint(dst, &tmap_k, 0, 0, 0, y / 8, full(st), kv_pol);
                                else
                                    tma_load_3d_hint(dst, &tmap_v, 0, y, 0, full(st), kv_pol);
                            }
                            next_slot();
                        }
                    }
                    seg_advance(it, len, p, tab);
                }
            }
            if (lane == 0) {
                if (ok && claim()) {
                    recs[j % Tr::NREC].flags = TC_END;
                    mbar_arrive(described + 8 * (j % Tr::NREC));
                    mbar_arrive(full(st));
                    next_slot();
                } else {
                    ok = false;
                }
                if (!ok) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    // copies still in flight land before the CTA's shared memory is released
                    for (int k = item - R > 0 ? item - R : 0; k < item; ++k)
                        mbar_wait_bounded(full(k % R), (uint32_t)((k / R) & 1), p.timeout_ns);
                    if (nseg > 0) mbar_wait_bounded(q_full, (uint32_t)((nseg - 1) & 1), p.timeout_ns);
                }
            }
        } else if (warp == Tr::LOOK_WARP) {
            // ============================================================ V rows
            int st = 0, j = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto next_slot = [&]() {
                if (++st == R) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            auto wait_full = [&]() -> bool {
                const bool stop = *abort_flag != 0 || !mbar_wait_bounded(full(st), ph, p.timeout_ns);
                return !__any_sync(0xffffffffu, stop);
            };
            for (;; ++j) {
                if (!wait_full()) {
                    ok = false;
                    break;
                }
                const WideStage& rc = recs[j % Tr::NREC];
                const bool end = rc.flags & TC_END;
                const int t0 = rc.t0, held = min(rc.nkeys, rc.ctx - t0), from = max(0, rc.base - t0);
                __syncwarp();
                if (lane == 0) mbar_arrive(ready(st));            // K, or the end, needs no look
                if (end) break;
                next_slot();
                if (!wait_full()) {
                    ok = false;
                    break;
                }
                if (from < held || held < KEYS) {
                    uint8_t* vt = smem + Tr::RING_OFF + st * Tr::SLOT_BYTES;
                    auto part_of = [&](int i) -> uint4* {
                        const int key = i / (HALVES * 8), part = i % (HALVES * 8);
                        return reinterpret_cast<uint4*>(vt + (key / BS) * Tr::BLK_BYTES + (part / 8) * Tr::HALF_STRIDE +
                                                        (key % BS) * 128 + (part % 8) * 16);
                    };
                    uint64_t spoilt = 0;                          // by node
                    for (int i = from * HALVES * 8 + lane; i < held * HALVES * 8; i += 32)
                        if (vec_not_finite<Tr::BF16>(*part_of(i)))
                            spoilt |= 1ull << (t0 + i / (HALVES * 8) - rc.base);
                    const uint32_t s0 = __reduce_or_sync(0xffffffffu, (uint32_t)spoilt);
                    const uint32_t s1 = __reduce_or_sync(0xffffffffu, (uint32_t)(spoilt >> 32));
                    spoilt = (uint64_t)s0 | ((uint64_t)s1 << 32);
                    if (spoilt) {
                        for (int i = from * HALVES * 8 + lane; i < held * HALVES * 8; i += 32)
                            if ((spoilt >> (t0 + i / (HALVES * 8) - rc.base)) & 1) *part_of(i) = make_uint4(0u, 0u, 0u, 0u);
                        if (lane == 0) {
                            recs[j % Tr::NREC].spoilt[0] = s0;
                            recs[j % Tr::NREC].spoilt[1] = s1;
                        }
                    }
                    for (int i = held * HALVES * 8 + lane; i < KEYS * HALVES * 8; i += 32) *part_of(i) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(ready(st));
                next_slot();
            }
            if (!ok && lane == 0) {
                set_err(p.err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
        } else if (lane == 0) {
            // ============================================================ MMAs of one tile
            const int t = warp - Tr::MMA_WARP;
            const uint32_t s_col = tmem + 128 * t, o_col = tmem + Tr::O_COL + 128 * t;
            const int tile_rows0 = t * (Tr::TILE >> gs);          // first node of the tile
            int st = 0, nseg = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                if (mbar_try_wait(bar, parity)) return true;
                if (*abort_flag || !mbar_wait_bounded(bar, parity, p.timeout_ns)) ok = false;
                return ok;
            };
            auto next_slot = [&]() {
                if (++st == R) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            int flags = 0;
            bool active = false;
            auto keys = [&](int j) -> bool {                      // stage j's keys, and its segment's Q, are there
                if (!wait(ready(st), ph)) return false;           // (the look warp never falls a slot's use behind)
                const WideStage& rc = recs[j % Tr::NREC];
                flags = rc.flags;
                if (flags & TC_END) return false;
                active = rc.n > tile_rows0;
                if (flags & TC_FIRST) {
                    if (!wait(q_full, (uint32_t)(nseg & 1))) return false;
                    ++nseg;
                }
                return true;
            };
            for (int j = 0, more = keys(0); more; ++j) {
                const uint32_t par = (uint32_t)(j & 1);
                // Not with the other tile: its scores, then this tile's, so that one tile's softmax runs
                // beside the other's products (together, each waited for the other: 814 against 770 us).
                if (t == 1 ? !wait(lead, par) : j > 0 && !wait(follow, par ^ 1u)) break;
                if (active) {
                    tc_fence_after();
                    const uint64_t qd = sdesc_sw128(q_base + t * HALVES * Tr::Q_HALF, 16, 1024);
                    const uint64_t kd = sdesc_sw128(ring + st * Tr::SLOT_BYTES, 16, Tr::GROUP_STRIDE);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_f16(s_col, qd + (uint64_t)((k / 4) * (Tr::Q_HALF >> 4) + (k % 4) * 2),
                                kd + (uint64_t)((k / 4) * (1024 >> 4) + (k % 4) * 2), IDESC_S, k > 0 ? 1u : 0u);
                    mma_commit(s_full(t));
                    if (t == 0) mma_commit(lead);
                    mma_commit(empty(st));
                    if (flags & TC_LAST) mma_commit(q_empty);
                } else {
                    mbar_arrive(s_full(t));
                    if (t == 0) mbar_arrive(lead);
                    mbar_arrive(empty(st));
                    if (flags & TC_LAST) mbar_arrive(q_empty);
                }
                if (t == 1) mbar_arrive(follow);
                next_slot();
                if (!wait(ready(st), ph)) break;
                const uint32_t vbase = ring + st * Tr::SLOT_BYTES;
                bool stop = false;
#pragma unroll
                for (int h = 0; h < 4; ++h) {                     // as each quarter of the weights is there
                    if (!wait(p_part(t, h), par)) {
                        stop = true;
                        break;
                    }
                    if (active) {
                        tc_fence_after();
#pragma unroll
                        for (int k = 2 * h; k < 2 * h + 2; ++k) {
                            const uint64_t bv = sdesc_sw128(vbase + ((16 * k) / BS) * Tr::BLK_BYTES + ((16 * k) % BS) * 128,
                                                            Tr::HALF_STRIDE, 1024);
                            const uint32_t pt = s_col + 32 * (k / 2) + 8 * (k % 2);
                            mma_f16_ts(o_col, pt, bv, IDESC_O, (flags & TC_FIRST) && k == 0 ? 0u : 1u);
                            mma_f16_ts(o_col, pt + 16, bv, IDESC_O, 1u);
                        }
                    }
                }
                if (stop) break;
                const bool issued = active;
                if (active) {
                    mma_commit(pv_done(t));
                    mma_commit(empty(st));
                } else {
                    mbar_arrive(pv_done(t));
                    mbar_arrive(empty(st));
                }
                next_slot();
                more = keys(j + 1);
                // the next scores overwrite the weights
                if (issued && more && !wait(pv_done(t), par)) break;
            }
            if (!ok) {
                set_err(p.err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            // every MMA of this thread completes before tensor memory is released
            mma_commit(fin + 8 * t);
            mbar_wait_bounded(fin + 8 * t, 0, p.timeout_ns);
        }
        __syncwarp();
    } else {
        // ================================================================ softmax
        // 256 x 200 + 128 x 104 registers: the 384 x 168 of the launch
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;                        // row of the tile = TMEM lane
        const int node = (t * Tr::TILE + r) >> gs;                // node of the group
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.timeout_ns));
        };
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lane_addr + 128 * t, o_addr = lane_addr + Tr::O_COL + 128 * t;
        const float qnan = __int_as_float(0x7fc00000);
        // scores keep their order under a positive scale; another sign goes into the scores first
        const bool flip = !(p.scale_log2 > 0.f);
        const float scale = flip ? 1.f : p.scale_log2;
        int st = 0, cur_seg = -1, pois = 0, seg_kvh = 0, seg_q0 = 0;
        uint32_t ph = 0;
        float m = -INFINITY, l = 0.f;                             // reference (scaled, log2 units) and sum
        uint64_t sees = 0;
        bool alive = false, active = false, ok = true;
        for (int j = 0;; ++j) {
            const uint32_t par = (uint32_t)(j & 1);
            if (*abort_flag) break;
            if (!wait_all(described + 8 * (j % Tr::NREC), (uint32_t)((j / Tr::NREC) & 1))) {
                ok = false;
                break;
            }
            const WideStage& rc = recs[j % Tr::NREC];
            const int flags = rc.flags;
            if (flags & TC_END) break;
            const int t0 = rc.t0, nkeys = rc.nkeys, base = rc.base, seg = rc.seg;
            if (seg != cur_seg) {
                cur_seg = seg;
                seg_kvh = rc.kvh;
                seg_q0 = rc.q0;
                m = -INFINITY;
                l = 0.f;
                pois = 0;
                alive = node < rc.n;
                active = rc.n > t * (Tr::TILE >> gs);
                sees = alive ? node_bits(__ldg(mp.tree_masks + seg_q0 + node), rc.ctx - base) : 0;
            }
            pois |= rc.poison;
            if (!wait_all(s_full(t), par)) {
                ok = false;
                break;
            }
            // a quarter without rows has nothing to weigh; the tile's other rows go on
            const bool busy = active && __any_sync(0xffffffffu, alive);
            if (busy) {
                tc_fence_after();
                uint32_t u[32];
                // Scores that some row may not see, or whose order a scale turns, are rewritten first,
                // so that the loops below, which every stage runs, stay short: they are bound by
                // instruction fetches.
                if (flip || t0 + KEYS > base || nkeys < KEYS) {
                    auto held = [&](int n) -> uint64_t { return n >= 64 ? ~0ull : n > 0 ? (1ull << n) - 1 : 0ull; };
                    uint64_t s0 = 0, s1 = 0;                      // the keys that the row sees
                    if (alive) {
                        s0 = tree_visible(sees, base - t0) & held(nkeys);
                        s1 = tree_visible(sees, base - t0 - 64) & held(nkeys - 64);
                    }
                    if (base < t0 + nkeys) {                      // the stage holds nodes: their V has been looked at
                        int vs = st + 1;
                        uint32_t vph = ph;
                        if (vs == R) {
                            vs = 0;
                            vph ^= 1u;
                        }
                        if (!wait_all(ready(vs), vph)) {
                            ok = false;
                            break;
                        }
                        const volatile uint32_t* words = rc.spoilt;
                        if (((uint64_t)words[0] | ((uint64_t)words[1] << 32)) & sees) l = qnan;
                    }
#pragma unroll 1
                    for (int c = 0; c < KEYS / 32; ++c) {
                        tmem_ld32(s_addr + 32 * c, u);
                        tmem_ld_wait();
                        after_wait(u);
                        const uint32_t w = (uint32_t)((c < 2 ? s0 : s1) >> (32 * (c & 1)));
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float x = __uint_as_float(u[k]);
                            u[k] = (w >> k) & 1u ? __float_as_uint(flip ? x * p.scale_log2 : x) : 0xff800000u;
                        }
                        tmem_st32(s_addr + 32 * c, u);
                    }
                    tmem_st_wait();
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int c = 0; c < KEYS / 32; c += 2) {
                    uint32_t v[32];
                    tmem_ld32(s_addr + 32 * c, u);
                    tmem_ld32(s_addr + 32 * c + 32, v);
                    tmem_ld_wait();
                    after_wait(u);
                    after_wait(v);
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            m4[i] = fmaxf(fmaxf(m4[i], __uint_as_float(u[k + i])), __uint_as_float(v[k + i]));
                }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
                const bool need = mx > m + Tr::TAU && alive;
                const float alpha = need ? ex2(m - mx) : 1.f;     // m = -inf: 0
                if (need) {
                    m = mx;
                    l *= alpha;
                }
                if (!(flags & TC_FIRST) && __any_sync(0xffffffffu, need)) {
                    // O holds the earlier stages: their products are done (the scores were issued after them)
                    if (!wait_all(pv_done(t), par ^ 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        tmem_ld32(o_addr + 32 * c, u);
                        tmem_ld_wait();
                        after_wait(u);
#pragma unroll
                        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * alpha);
                        tmem_st32(o_addr + 32 * c, u);
                    }
                    tmem_st_wait();
                }
                tmem_ld32(s_addr, u);
                const float mref = m == -INFINITY ? 0.f : m;      // no visible key yet: weights 0
                const f32x2 scale2 = pair2(scale, scale), mref2 = pair2(-mref, -mref);
                f32x2 sum2[2] = {0ull, 0ull};
                tmem_ld_wait();
                after_wait(u);
#pragma unroll 1
                for (int c = 0; c < KEYS / 32; ++c) {
                    uint32_t w[32];                               // 16 columns of hi, 16 of lo
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        split2(fma2(pair2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), scale2, mref2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum2[e & 1] = add2(sum2[e & 1], pair2(p0, p1));
                        if constexpr (Tr::BF16) {
                            // hi: the weights cut to bf16; lo: the exact remainders, rounded to nearest
                            // (2^-16 of a weight in all, to either side)
                            const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                            w[e] = __byte_perm(u0, u1, 0x7632);
                            float r0, r1;
                            split2(add2(pair2(p0, p1), pair2(-__uint_as_float(u0 & 0xffff0000u),
                                                             -__uint_as_float(u1 & 0xffff0000u))), r0, r1);
                            w[16 + e] = pack2<true>(r0, r1);
                        } else {
                            const uint32_t hv = pack2<false>(p0, p1);
                            w[e] = hv;
                            w[16 + e] = pack2<false>(p0 - lo_of<false>(hv), p1 - hi_of<false>(hv));
                        }
                    }
                    if (c + 1 < KEYS / 32) tmem_ld32(s_addr + 32 * c + 32, u);
                    tmem_st32(s_addr + 32 * c, w);
                    tmem_st_wait();                               // a quarter of the weights is there
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_part(t, c));
                    tmem_ld_wait();
                    after_wait(u);
                }
                float sa, sb;
                split2(add2(sum2[0], sum2[1]), sa, sb);
                l += sa + sb;
            } else {
                __syncwarp();
                if (lane == 0)
                    for (int c = 0; c < 4; ++c) mbar_arrive(p_part(t, c));
            }
            if (flags & TC_LAST) {
                if (!wait_all(pv_done(t), par)) {
                    ok = false;
                    break;
                }
                if (busy) {
                    tc_fence_after();
                    // 128 bytes of each row at a time (64 finished values, or 32 of a partial
                    // state) go through shared memory, so that 8 lanes write a row's piece
                    uint8_t* out = smem + Tr::OUT_OFF + warp * Tr::OUT_BYTES;
                    const bool complete = flags & TC_COMPLETE;
                    const float inv = pois ? qnan : complete ? (l == 0.f ? 0.f : 1.f / l) : 1.f;   // a node that sees no key: zero
                    constexpr int PIECES = D / 32;
                    const unsigned rows = __ballot_sync(0xffffffffu, alive);
                    const int row0 = t * Tr::TILE + quarter * 32;                 // the warp's first row of the group
#pragma unroll 1
                    for (int c = 0; c < PIECES; ++c) {
                        uint32_t u[32];
                        tmem_ld32(o_addr + 32 * c, u);
                        tmem_ld_wait();
                        after_wait(u);
                        const int half = complete ? c & 1 : 0;                    // which half of the 128 bytes
#pragma unroll
                        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * inv);
                        if (complete) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                auto two = [&](int i) -> uint32_t {
                                    return pack2<Tr::BF16>(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
                                };
                                *reinterpret_cast<uint4*>(out + lane * 128 + (((4 * half + k) ^ (lane & 7)) << 4)) =
                                    make_uint4(two(8 * k), two(8 * k + 2), two(8 * k + 4), two(8 * k + 6));
                            }
                            if (half == 0) continue;
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                *reinterpret_cast<uint4*>(out + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                    make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                        }
                        __syncwarp();
#pragma unroll 2
                        for (int i = 0; i < 8; ++i) {
                            const int rr = 4 * i + lane / 8, part = lane & 7;
                            const uint4 v = *reinterpret_cast<const uint4*>(out + rr * 128 + ((part ^ (rr & 7)) << 4));
                            if (!((rows >> rr) & 1)) continue;
                            const int row = row0 + rr;
                            if (complete) {
                                uint16_t* orow = p.out + ((size_t)(seg_q0 + (row >> gs)) * p.Hq + (size_t)seg_kvh * G + (row & (G - 1))) * D;
                                *reinterpret_cast<uint4*>(orow + 64 * (c / 2) + 8 * part) = v;
                            } else {
                                float* prow = p.partials + (((size_t)blockIdx.x * 2 + ((flags & TC_SLOT1) ? 1 : 0)) * Tr::ROWS +
                                                            row) * Tr::PSTRIDE;
                                *reinterpret_cast<uint4*>(prow + 32 * c + 4 * part) = v;
                            }
                        }
                        __syncwarp();
                    }
                    if (alive && !complete) {
                        float* prow = p.partials + (((size_t)blockIdx.x * 2 + ((flags & TC_SLOT1) ? 1 : 0)) * Tr::ROWS + row0 +
                                                    lane) * Tr::PSTRIDE;
                        prow[D] = m;
                        prow[D + 1] = l;
                    }
                    tc_fence_before();
                }
            }
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
cudaError_t tree_wide_launch(const MultiLaunch& L) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(L.grid, Tr::THREADS, Tr::SMEM_BYTES, L.stream, attr);
    return cudaLaunchKernelEx(&cfg, pa_tree_wide_kernel<Tr>, *L.tmap_q, *L.tmap_k, *L.tmap_v, L.p);
}

template <class Tr>
MultiKernelInfo tree_wide_info() {
    return MultiKernelInfo{&tree_wide_launch<Tr>,
                           &persistent_ctas<pa_tree_wide_kernel<Tr>, Tr::THREADS, Tr::SMEM_BYTES>, Tr::ROWS};
}

// [d == 128][bs == 32], defined in tree_wide_*.cu.
void tree_wide_table_bf16(MultiKernelInfo (&t)[2][2]);
void tree_wide_table_fp16(MultiKernelInfo (&t)[2][2]);

}  // namespace pa
