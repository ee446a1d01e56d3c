// Attention of chunks of new tokens over the 8-bit cache with a scale for each block and
// KV head, on the 5th-generation tensor core.
//
// Mathematics: decode_bs8.cuh (a value scale in the exponent, weights in proportion to
// their share of the output), causal within the chunk.  Rows r = i * g + hh of token i and
// query head hh; keys in stages of 128:
//
//   S = Q K^T   M 128, N 128, K = head_dim    (fp16; K converted from its codes)
//   O += P V    M 128, N = head_dim, K 128    (P fp16 from tensor memory)
//
// Codes become fp16 in shared memory (exactly) because the products want 11 bits of the
// queries and weights, and the tensor core takes 8-bit operands on both sides or none.
// N = 128 because a product of N = 64 takes as long.
//
// Two arrangements of a CTA's two 128-row tiles:
//  * more than 128 rows per (sequence, KV head): the tiles are 256 rows, both read each
//    converted stage (a stage costs 2 * 2 * 512 cycles of products at head_dim 128);
//  * SPLIT, up to 128 rows: both tiles are the same rows and take every other stage, so that
//    one's softmax runs beside the other's products; their states are joined at a
//    segment's end, where the threads of tile 0 read both outputs from tensor memory.
//
// Tensor memory (512 columns): S_0, S_1 at 0 and 128, O_0, O_1 at 256 and 384; P_t overwrites
// S_t, 16 columns at the start of each 32 that held its scores.  A row's reference moves
// only when its maximum rises by more than 8 (O is rescaled then), so weights are at most
// 2^8.
//
// Roles (512 threads, one CTA per SM):
//   warps 0-3, 4-7   softmax of tile 0, 1: thread = row = TMEM lane
//   warps 8-11       per segment the queries, as fp16 under the swizzle that the products
//                    read; per stage the block scales, the keys, then the values: codes
//                    from shared memory, fp16 back.  Value rows past the context become
//                    zeros, and so do rows of the chunk that hold NaN or infinities
//                    (rows that see them become NaN at the softmax)
//   warps 12, 13     products of tile 0, 1 (one thread each)
//   warp 14          copies: a bulk copy per block for scales and keys, one for values
//
// The work list and the partial states of split rows are those of the tree kernels: each CTA
// takes an equal run of (row group, KV head, block) units; a group's keys end at its
// last token's.  Every wait is bounded (PA_DEVERR_TIMEOUT).
#pragma once

#include <climits>

#include "bs8.cuh"
#include "decode_bs8.cuh"
#include "packed.cuh"
#include "tree_wide_kernel.cuh"

namespace pa {

// The work list: sequence i % N in group i / N, whose tokens see keys up to its last
// token's.  A malformed sequence is nowhere.
struct ChunkTab {
    const int* ctx;
    const int* qst;
    int N, groups, group_nodes, max_nodes, total_q, MB, BS;
    __device__ __forceinline__ int nb(int i) const {
        const int g = groups == 1 ? 0 : i / N, s = i - g * N;
        const int a = qst[s], b = qst[s + 1], c = ctx[s];
        const long long n = (long long)b - a;
        const bool ok = a >= 0 && b <= total_q && n <= max_nodes && n <= c && c > 0 && c <= MB * BS;
        const long long skip = (long long)g * group_nodes;
        if (!ok || n <= skip) return 0;
        const long long last = c - n + min(n, skip + group_nodes);   // keys the group sees
        return (int)((last + BS - 1) / BS);
    }
};

__device__ __forceinline__ void seg_advance(SegIter& it, int len, const DecodeParams& p, const ChunkTab& tab) {
    it.gi += len;
    it.b0 += len;
    if (it.b0 < it.nb) return;
    it.b0 = 0;
    if (++it.kvh < p.Hkv) return;
    it.kvh = 0;
    it.nb = 0;
    for (const int n = tab.N * tab.groups; ++it.s < n;)
        if ((it.nb = tab.nb(it.s)) > 0) break;
}

template <int D_, int BS_, bool BF16_, bool E5M2_, bool SPLIT_>
struct ChunkTraits {
    static constexpr int D = D_;
    static constexpr int BS = BS_;
    static constexpr bool BF16 = BF16_;
    static constexpr bool E5M2 = E5M2_;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int TILE = 128;
    static constexpr int ROWS = SPLIT ? TILE : 2 * TILE;
    static constexpr int KEYS = 128;                         // keys per stage
    static constexpr int SB = KEYS / BS;                     // blocks per stage
    static constexpr int HALVES = D / 64;
    static constexpr int SLOT_BYTES = KEYS * D * 2;          // a stage's keys, or its values, in fp16
    static constexpr int HALF_STRIDE = KEYS * 128;           // between the column halves of a slot
    static constexpr int R = 3;                              // such slots; K and V alternate
    static constexpr int K8_BYTES = BS8_HEAD + BS * D;       // a block's scales and key codes
    static constexpr int V8_BYTES = BS * D;
    static constexpr int SLOT8_BYTES = (SB * K8_BYTES + 127) / 128 * 128;
    static constexpr int SMEM_BYTES = 227 * 1024;
    static constexpr int Q_HALF = TILE * 128;
    static constexpr int Q_BYTES = (SPLIT ? 1 : 2) * HALVES * Q_HALF;
    static constexpr int NREC = 8;
    static constexpr int N8_CAP = 8;
    // full8, empty8; empty, ready; s_full, p_part[4], pv_done per tile; q_full, q_empty; fin;
    // described; lead, follow; joined, o1_free
    static constexpr int NBAR = 2 * N8_CAP + 2 * R + 2 * 6 + 2 + 2 + NREC + 2 + 2;
    static constexpr int REC_OFF = (8 * NBAR + 15) / 16 * 16;
    static constexpr int REC_BYTES = 48 + 4 * SB * 4;
    static constexpr int ROWF_OFF = REC_OFF + NREC * REC_BYTES;   // score factors of the rows, two segments
    static constexpr int XCH_OFF = ROWF_OFF + 2 * 2 * TILE * 4;   // SPLIT: tile 1's (m, l) of a row
    static constexpr int MISC_OFF = XCH_OFF + (SPLIT ? TILE * 8 : 0);   // TMEM base, abort flag
    static constexpr int SPOILT_OFF = MISC_OFF + 16;         // per segment: first position of a value that is not finite
    static constexpr int START_OFF = SPOILT_OFF + NREC * 4;  // a TreeStart, a word per warp
    static constexpr int THREADS = 512;
    static constexpr int Q_OFF = (START_OFF + 32 + 8 * THREADS / 32 + 1023) / 1024 * 1024;
    static constexpr int OUT_OFF = Q_OFF + Q_BYTES;          // per softmax warp: 32 rows of 64 bytes on their way out
    static constexpr int OUT_BYTES = 32 * 64;
    static constexpr int RING_OFF = OUT_OFF + 8 * OUT_BYTES;
    static constexpr int RING8_OFF = RING_OFF + R * SLOT_BYTES;
    static constexpr int N8_FIT = (SMEM_BYTES - 1024 - RING8_OFF) / SLOT8_BYTES / 2 * 2;
    static constexpr int N8 = N8_FIT > N8_CAP ? N8_CAP : N8_FIT;   // slots of codes; keys in the even ones
    static constexpr int CONVERT_WARP = 8, MMA_WARP = 12, COPY_WARP = 14;
    static constexpr int TMEM_COLS = 512;
    static constexpr int O_COL = 256;
    static constexpr int PSTRIDE = D + 4;
    static constexpr float TAU = 8.f;                        // lazy-rescale threshold (log2 units)
    static_assert(N8 >= 2, "shared memory");
};

// One stage: what the copy warp says of it (first the 48 bytes), and its blocks' scales.
template <int SB>
struct alignas(16) ChunkStage {
    int base, kvh, t0, nkeys;     // position of the group's first token, KV head, first key, keys copied
    int n, ctx, q0, flags;        // tokens of the group, context, the group's first query row
    int poison, seg, chunk, pad;  // bad block id or scale; segment number; the chunk's first position
    float ks[SB], lb[SB], back[SB], cut[SB];   // key scale, lb, 2^-lb, f of decode_bs8.cuh
};

// 32 consecutive columns' worth of scores' maximum, 16 columns at a time.
__device__ __forceinline__ float max16(const uint32_t* u) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = fmaxf(fmaxf(__uint_as_float(u[i]), __uint_as_float(u[i + 4])),
                     fmaxf(__uint_as_float(u[i + 8]), __uint_as_float(u[i + 12])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <class Tr>
__global__ void __launch_bounds__(Tr::THREADS, 1)
pa_chunk_bs8_kernel(const MultiParams mp) {
    constexpr int D = Tr::D, BS = Tr::BS, SB = Tr::SB, HALVES = Tr::HALVES, KEYS = Tr::KEYS, R = Tr::R, N8 = Tr::N8;
    constexpr bool SPLIT = Tr::SPLIT;
    constexpr uint32_t IDESC_S = idesc_f16<false>(128, KEYS, false, false);
    constexpr uint32_t IDESC_O = idesc_f16<false>(128, D, false, true);
    using Stage = ChunkStage<SB>;
    static_assert(sizeof(Stage) == Tr::REC_BYTES, "stage record");
    const DecodeParams& p = mp.d;
    const int seqs = p.N;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hkv, gs = 31 - __clz(G);           // a power of two
    const uint32_t sbase = smem_u32(smem);
    const uint32_t q_base = sbase + Tr::Q_OFF, ring = sbase + Tr::RING_OFF, ring8 = sbase + Tr::RING8_OFF;
    auto full8 = [&](int st) -> uint32_t { return sbase + 8 * st; };
    auto empty8 = [&](int st) -> uint32_t { return sbase + 8 * (Tr::N8_CAP + st); };
    const uint32_t slot_bars = sbase + 8 * 2 * Tr::N8_CAP;
    auto empty = [&](int st) -> uint32_t { return slot_bars + 8 * st; };
    auto ready = [&](int st) -> uint32_t { return slot_bars + 8 * (R + st); };
    const uint32_t tile_bars = slot_bars + 8 * 2 * R;
    auto s_full = [&](int t) -> uint32_t { return tile_bars + 48 * t; };
    auto p_part = [&](int t, int c) -> uint32_t { return tile_bars + 48 * t + 8 + 8 * c; };
    auto pv_done = [&](int t) -> uint32_t { return tile_bars + 48 * t + 40; };
    const uint32_t q_full = tile_bars + 96, q_empty = q_full + 8, fin = q_empty + 8;   // fin[2]
    auto described = [&](int j) -> uint32_t { return fin + 16 + 8 * (j % Tr::NREC); };
    // tile 1's scores of a stage come after tile 0's, tile 0's next ones after those have been issued
    const uint32_t lead = fin + 16 + 8 * Tr::NREC, follow = lead + 8;
    // SPLIT: tile 1's state of a segment is there; tile 0 has read it
    const uint32_t joined = follow + 8, o1_free = joined + 8;
    Stage* recs = reinterpret_cast<Stage*>(smem + Tr::REC_OFF);
    float* rowf = reinterpret_cast<float*>(smem + Tr::ROWF_OFF);
    float2* xch = reinterpret_cast<float2*>(smem + Tr::XCH_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Tr::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Tr::MISC_OFF + 4);
    // (of segment s at s % NREC: no role is that many stages ahead of another)
    int* spoilt = reinterpret_cast<int*>(smem + Tr::SPOILT_OFF);

    if (threadIdx.x == 0) {
        for (int i = 0; i < N8; ++i) {
            mbar_init(full8(i), 1);
            mbar_init(empty8(i), 4);                // the converting warps are done with it
        }
        for (int i = 0; i < R; ++i) {
            mbar_init(empty(i), SPLIT ? 1 : 2);     // the products of its tile, or of both
            mbar_init(ready(i), 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            for (int c = 0; c < 4; ++c) mbar_init(p_part(t, c), 4);
            mbar_init(pv_done(t), 1);
            mbar_init(fin + 8 * t, 1);
        }
        mbar_init(q_full, 4);
        mbar_init(q_empty, 2);
        for (int i = 0; i < Tr::NREC; ++i) mbar_init(described(i), 1);
        mbar_init(lead, 1);
        mbar_init(follow, 1);
        mbar_init(joined, 4);
        mbar_init(o1_free, 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == Tr::MMA_WARP) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), Tr::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();                 // the launch before is complete
    griddep_launch_dependents();

    const int32_t* qst = mp.q_start;
    // a sequence's chunk, or -1 when it is malformed
    auto chunk_size = [&](int s) -> int {
        const int a = __ldg(qst + s), b = __ldg(qst + s + 1), ctx = __ldg(p.context_lens + s);
        const long long n = (long long)b - a;
        const bool ok = a >= 0 && b <= mp.total_q && n >= 0 && n <= mp.max_q && n <= (ctx > 0 ? ctx : 0) &&
                        ctx <= p.MB * BS;
        return ok ? (int)n : -1;
    };
    // ---- malformed chunks and bad context lengths: error bit, NaN rows ----
    for (int s = blockIdx.x; s < seqs; s += gridDim.x) {
        if (chunk_size(s) >= 0 && __ldg(p.context_lens + s) >= 0) continue;
        if (threadIdx.x == 0) set_err(p.err, PA_DEVERR_CONTEXT);
        const int a = max(0, __ldg(qst + s));
        const int b = min(mp.total_q, __ldg(qst + s + 1));
        for (long long i = (long long)a * p.Hq * D + threadIdx.x; i < (long long)b * p.Hq * D; i += Tr::THREADS)
            p.out[i] = qnan16<Tr::BF16>();
    }

    ChunkTab tab;
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
    const int tile_nodes = Tr::TILE >> gs;                    // tokens of a tile
    // scores keep their order under a scale that is not negative; a sign goes into the queries
    const float scale_abs = fabsf(p.scale_log2);

    // 256 x 168 + 128 x 104 + 128 x 64 registers: no more than the 512 x 128 of the launch
    if (warp >= Tr::MMA_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == Tr::COPY_WARP) {
            // ============================================================ copies
            // with one group the codes are read once per call; with more, other CTAs read them too
            const uint64_t kv_pol = mp.groups == 1 ? l2_evict_first() : l2_evict_normal();
            if (lane == 0) mp.starts[blockIdx.x] = at;
            int item = 0, st = 0, j = 0, nseg = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto claim = [&]() -> bool {             // lane 0: the slot's last use is over
                return item < N8 || mbar_wait_bounded(empty8(st), ph ^ 1u, p.timeout_ns);
            };
            auto next_slot = [&]() {
                ++item;
                if (++st == N8) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            if (has_work) {
                SegIter it{lo, at.s, at.kvh, at.b0, at.nb, 0};
                while (ok && it.gi < hi) {
                    const int len = seg_len(it, hi);
                    const int s = it.s % seqs, skip = it.s / seqs * mp.group_nodes;
                    const int size = chunk_size(s), n = min(mp.group_nodes, size - skip);   // > 0: it has blocks
                    const int ctx = __ldg(p.context_lens + s), q0 = __ldg(qst + s) + skip;
                    const long long P0 = it.gi - it.b0;
                    const bool complete = sc.of(P0) == sc.of(P0 + it.nb - 1);
                    const int seg_flags = (complete ? TC_COMPLETE : 0) | (it.gi == lo ? 0 : TC_SLOT1);
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
                        const uint8_t* piece = p.kv8 + ((size_t)cid * p.Hkv + it.kvh) * bs8_piece_bytes(BS, D);
                        for (int op = 0; op < 2; ++op) {          // scales and keys, then values
                            if (lane == 0) {
                                if (!claim()) {
                                    ok = false;
                                } else {
                                    if (op == 0) {
                                        if (poison) set_err(p.err, PA_DEVERR_BLOCK_ID);
                                        Stage& rc = recs[j % Tr::NREC];
                                        rc.base = ctx - size + skip;
                                        rc.kvh = it.kvh;
                                        rc.t0 = (it.b0 + bb) * BS;
                                        rc.nkeys = nbs * BS;
                                        rc.n = n;
                                        rc.ctx = ctx;
                                        rc.q0 = q0;
                                        rc.flags = seg_flags | (k == 0 ? TC_FIRST : 0) | (k == nst - 1 ? TC_LAST : 0);
                                        rc.poison = poison;
                                        rc.seg = nseg;
                                        rc.chunk = ctx - size;
                                    }
                                    mbar_arrive_expect_tx(full8(st), (uint32_t)(nbs * (op ? Tr::V8_BYTES : Tr::K8_BYTES)));
                                }
                            }
                            ok = __shfl_sync(0xffffffffu, ok, 0);
                            __syncwarp();
                            if (!ok) break;
                            if (copies) {
                                const uint32_t dst = ring8 + st * Tr::SLOT8_BYTES;
                                if (op == 0)
                                    bulk_load_hint(dst + lane * Tr::K8_BYTES, piece, Tr::K8_BYTES, full8(st), kv_pol);
                                else
                                    bulk_load_hint(dst + lane * Tr::V8_BYTES, piece + Tr::K8_BYTES, Tr::V8_BYTES, full8(st),
                                                   kv_pol);
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
                    mbar_arrive(full8(st));
                    next_slot();
                } else {
                    ok = false;
                }
                if (!ok) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    // copies still in flight land before the CTA's shared memory is released
                    for (int k = item - N8 > 0 ? item - N8 : 0; k < item; ++k)
                        mbar_wait_bounded(full8(k % N8), (uint32_t)((k / N8) & 1), p.timeout_ns);
                }
            }
        } else if (warp < Tr::COPY_WARP && lane == 0) {
            // ============================================================ products of one tile
            const int t = warp - Tr::MMA_WARP;
            const uint32_t s_col = tmem + 128 * t, o_col = tmem + Tr::O_COL + 128 * t;
            const uint32_t q_tile = q_base + (SPLIT ? 0 : t * HALVES * Tr::Q_HALF);
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                if (mbar_try_wait(bar, parity)) return true;
                if (*abort_flag || !mbar_wait_bounded(bar, parity, p.timeout_ns)) ok = false;
                return ok;
            };
            int own = 0, nseg = 0;                                // stages of this tile, segments begun
            bool fresh = true;                                    // O holds nothing of the segment
            bool issued = false;                                  // a PV product of stage own - 1
            for (int j = 0;; ++j) {
                if (!wait(described(j), (uint32_t)((j / Tr::NREC) & 1))) break;
                const Stage& rc = recs[j % Tr::NREC];
                const int flags = rc.flags;
                if (flags & TC_END) break;
                const bool active = SPLIT || rc.n > t * tile_nodes;
                if (flags & TC_FIRST) {
                    if (!wait(q_full, (uint32_t)(nseg & 1))) break;
                    ++nseg;
                    fresh = true;
                }
                if (SPLIT && (j & 1) != t) {                      // the other tile's stage
                    if (flags & TC_LAST) mma_commit(q_empty);
                    continue;
                }
                const int ik = 2 * j, iv = 2 * j + 1;
                const int ks = ik % R, vs = iv % R;
                const uint32_t par = (uint32_t)(own & 1);
                if (!wait(ready(ks), (uint32_t)((ik / R) & 1))) break;
                // the scores overwrite the weights of the stage before
                if (issued && !wait(pv_done(t), par ^ 1u)) break;
                if (!SPLIT && (t == 1 ? !wait(lead, par) : j > 0 && !wait(follow, par ^ 1u))) break;
                if (active) {
                    tc_fence_after();
                    const uint64_t qd = sdesc_sw128(q_tile, 16, 1024);
                    const uint64_t kd = sdesc_sw128(ring + ks * Tr::SLOT_BYTES, 16, 1024);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_f16(s_col, qd + (uint64_t)((k / 4) * (Tr::Q_HALF >> 4) + (k % 4) * 2),
                                kd + (uint64_t)((k / 4) * (Tr::HALF_STRIDE >> 4) + (k % 4) * 2), IDESC_S, k > 0 ? 1u : 0u);
                    mma_commit(s_full(t));
                    if (!SPLIT && t == 0) mma_commit(lead);
                    mma_commit(empty(ks));
                    if (flags & TC_LAST) mma_commit(q_empty);
                } else {
                    mbar_arrive(s_full(t));
                    if (!SPLIT && t == 0) mbar_arrive(lead);
                    mbar_arrive(empty(ks));
                    if (flags & TC_LAST) mbar_arrive(q_empty);
                }
                if (!SPLIT && t == 1) mbar_arrive(follow);
                if (!wait(ready(vs), (uint32_t)((iv / R) & 1))) break;
                const uint64_t vd = sdesc_sw128(ring + vs * Tr::SLOT_BYTES, Tr::HALF_STRIDE, 1024);
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
                        for (int k = 2 * h; k < 2 * h + 2; ++k)
                            mma_f16_ts(o_col, s_col + 32 * (k / 2) + 8 * (k % 2), vd + (uint64_t)(k * (2048 >> 4)), IDESC_O,
                                       fresh && k == 0 ? 0u : 1u);
                    }
                }
                if (stop) break;
                fresh = false;
                issued = active;
                if (active) {
                    mma_commit(pv_done(t));
                    mma_commit(empty(vs));
                } else {
                    mbar_arrive(pv_done(t));
                    mbar_arrive(empty(vs));
                }
                ++own;
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
    } else if (warp >= Tr::CONVERT_WARP) {
        // ================================================================ queries, keys and values to fp16
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const int cw = warp - Tr::CONVERT_WARP;
        // A lane's share of a row: one 16-byte part of codes.  Eight neighbouring lanes hold
        // four parts each of two neighbouring rows (D 128: of different halves), which are read
        // from eight different 16-byte bank groups and, as fp16, written to eight.
        constexpr int RPW = D == 128 ? 4 : 8;                     // rows a warp takes at once
        constexpr int NI = KEYS / (4 * RPW);                      // such rounds in a slot
        const int part = D == 128 ? (lane & 3) | (((lane >> 2) ^ (lane >> 3)) & 1) << 2 : lane & 3;
        const int row0 = cw * RPW + (D == 128 ? ((lane >> 2) & 1) | (lane >> 4) << 1 : lane >> 2);
        int j = 0, st8 = 0, st = 0, nseg = 0;
        uint32_t ph8 = 0, ph = 0;
        bool ok = true;
        float top_lb = -INFINITY;
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait_bounded(bar, parity, p.timeout_ns));
        };
        // codes -> fp16 at (row, part) of the slot
        auto put = [&](uint32_t slot, int row, const uint4& c, uint32_t by, bool scaled) {
            uint32_t h[8];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[2 * i] = fp8x2_to_f16x2<Tr::E5M2>((uint16_t)(w[i] & 0xffffu));
                h[2 * i + 1] = fp8x2_to_f16x2<Tr::E5M2>((uint16_t)(w[i] >> 16));
            }
            if (scaled) {
#pragma unroll
                for (int i = 0; i < 8; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(by));
            }
            const uint32_t a = slot + (part >> 2) * Tr::HALF_STRIDE + row * 128;
            const int c0 = 2 * (part & 3), x = row & 7;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + ((c0 ^ x) << 4)), "r"(h[0]), "r"(h[1]),
                         "r"(h[2]), "r"(h[3]) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + (((c0 + 1) ^ x) << 4)), "r"(h[4]), "r"(h[5]),
                         "r"(h[6]), "r"(h[7]) : "memory");
        };
        auto next = [&](int& s, uint32_t& parity, int n) {
            if (++s == n) {
                s = 0;
                parity ^= 1u;
            }
        };
        for (;; ++j) {
            if (!wait_all(full8(st8), ph8)) {
                ok = false;
                break;
            }
            Stage& rc = recs[j % Tr::NREC];
            const int flags = rc.flags;
            if (flags & TC_END) {
                __syncwarp();
                if (cw == 0 && lane == 0) mbar_arrive(described(j));
                break;
            }
            const int nkeys = rc.nkeys, nbs = nkeys / BS;
            uint8_t* k8 = smem + Tr::RING8_OFF + st8 * Tr::SLOT8_BYTES;
            if (cw == 0) {                                        // the blocks' scales
                if (flags & TC_FIRST) {
                    top_lb = -INFINITY;
                    if (lane == 0) spoilt[rc.seg % Tr::NREC] = INT_MAX;
                }
                float ks = 0.f, lb = -INFINITY;
                bool bad = false;
                if (lane < nbs) {
                    const float2 sc2 = *reinterpret_cast<const float2*>(k8 + lane * Tr::K8_BYTES);
                    bad = !bs8_is_scale(sc2.x) || !bs8_is_scale(sc2.y);
                    ks = sc2.x;
                    lb = fmaxf(__log2f(sc2.y), -126.f);
                }
                float top = lb;
#pragma unroll
                for (int o = 1; o < SB; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top_lb = fmaxf(top_lb, __shfl_sync(0xffffffffu, top, 0));
                if (lane < SB) {
                    const float held = fmaxf(lb, fmaxf(top_lb - BS8_LB_RANGE, BS8_LB_FLOOR));
                    rc.ks[lane] = ks;
                    rc.lb[lane] = held;
                    rc.back[lane] = ex2(-held);
                    rc.cut[lane] = lane < nbs ? ex2(lb - held) : 0.f;
                }
                if (__any_sync(0xffffffffu, bad) && lane == 0) {
                    set_err(p.err, PA_DEVERR_SCALE);
                    rc.poison = 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(described(j));
            }
            if (flags & TC_FIRST) {                               // the segment's queries
                if (nseg > 0 && !wait_all(q_empty, (uint32_t)((nseg - 1) & 1))) {
                    ok = false;
                    break;
                }
                const int rows = min(rc.n << gs, Tr::ROWS), r = 32 * cw + lane;
                for (int t = 0; t < (SPLIT ? 1 : 2); ++t) {
                    const int row = t * Tr::TILE + r;
                    if (!__any_sync(0xffffffffu, row < rows)) {   // nothing but rows that no one reads
                        if (t * Tr::TILE >= rows) break;
                        // (a partly filled tile: they have to be finite)
                    }
                    uint4 x[D / 8];
                    uint32_t top = 0;
                    const uint16_t* src = p.q + ((size_t)(rc.q0 + (row >> gs)) * p.Hq + (size_t)rc.kvh * G + (row & (G - 1))) * D;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        x[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (row < rows) x[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
                    }
                    float2 f = make_float2(1.f, 1.f);
                    if constexpr (Tr::BF16) {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
                            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
                        top = max(top & 0xffffu, top >> 16);
                        f = row_factor((int)(top >> 7));
                    }
                    if (p.scale_log2 < 0.f) f.x = -f.x;
                    rowf[(nseg & 1) * 2 * Tr::TILE + row] = f.y * scale_abs;
                    const uint32_t a = q_base + t * HALVES * Tr::Q_HALF + r * 128;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack2<false>(lo_of<Tr::BF16>(w[e]) * f.x, hi_of<Tr::BF16>(w[e]) * f.x);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + (i / 8) * Tr::Q_HALF + (((i & 7) ^ (r & 7)) << 4)),
                                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                    }
                }
                ++nseg;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            // keys
            const int item = 2 * j;
            if (item >= R && !wait_all(empty(st), ph ^ 1u)) {
                ok = false;
                break;
            }
            {
                const uint32_t slot = ring + st * Tr::SLOT_BYTES;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int row = row0 + i * 4 * RPW, b = row / BS;
                    const uint4 c = *reinterpret_cast<const uint4*>(k8 + b * Tr::K8_BYTES + bs8_key<D>(row % BS, part));
                    put(slot, row, c, 0u, false);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ready(st));
                mbar_arrive(empty8(st8));
            }
            next(st, ph, R);
            next(st8, ph8, N8);
            // values (the scales are in the record: this warp's wait makes warp 8's stores visible)
            if (!wait_all(described(j), (uint32_t)((j / Tr::NREC) & 1)) || !wait_all(full8(st8), ph8) ||
                (item + 1 >= R && !wait_all(empty(st), ph ^ 1u))) {
                ok = false;
                break;
            }
            {
                const uint32_t slot = ring + st * Tr::SLOT_BYTES;
                const uint8_t* v8 = smem + Tr::RING8_OFF + st8 * Tr::SLOT8_BYTES - Tr::K8_BYTES;   // where the pieces' keys would be
                const int t0 = rc.t0, held = min(nkeys, rc.ctx - t0), from = rc.chunk - t0;   // rows with values; of the chunk
                const bool plain = held == KEYS && from >= KEYS;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int row = row0 + i * 4 * RPW, b = row / BS;
                    uint4 c = *reinterpret_cast<const uint4*>(v8 + b * Tr::V8_BYTES + bs8_value<BS, D>(row % BS, part));
                    const float cut = rc.cut[b];
                    if (!plain) {
                        if (row >= held) {
                            c = make_uint4(0u, 0u, 0u, 0u);
                        } else if (row >= from) {
                            // NaN and infinite codes: all but the sign set (E4M3), the exponent all ones (E5M2)
                            auto odd = [](uint32_t w) -> uint32_t {
                                return Tr::E5M2 ? ((w & 0x7f7f7f7fu) + 0x04040404u) & 0x80808080u
                                                : ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            };
                            if (odd(c.x) | odd(c.y) | odd(c.z) | odd(c.w)) {
                                atomicMin(&spoilt[rc.seg % Tr::NREC], t0 + row);
                                c.x &= ~(odd(c.x) / 128 * 255);
                                c.y &= ~(odd(c.y) / 128 * 255);
                                c.z &= ~(odd(c.z) / 128 * 255);
                                c.w &= ~(odd(c.w) / 128 * 255);
                            }
                        }
                    }
                    put(slot, row, c, pack2<false>(cut, cut), cut != 1.f);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ready(st));
                mbar_arrive(empty8(st8));
            }
            next(st, ph, R);
            next(st8, ph8, N8);
        }
        if (!ok && lane == 0) {
            set_err(p.err, PA_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ================================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int t = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;                        // row of the tile = TMEM lane
        const int row_of_group = SPLIT ? r : t * Tr::TILE + r;
        const int token = row_of_group >> gs;                     // of the group
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.timeout_ns));
        };
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lane_addr + 128 * t, o_addr = lane_addr + Tr::O_COL + 128 * t;
        const float qnan = __int_as_float(0x7fc00000);
        int own = 0, cur_seg = 0, pois = 0;
        float m = -INFINITY, l = 0.f, rf = 0.f;                   // reference (log2 units), sum, the row's score factor
        bool alive = false, active = false, fresh = true, ok = true;
        for (int j = 0;; ++j) {
            if (*abort_flag) break;
            if (!wait_all(described(j), (uint32_t)((j / Tr::NREC) & 1))) {
                ok = false;
                break;
            }
            const Stage& rc = recs[j % Tr::NREC];
            const int flags = rc.flags;
            if (flags & TC_END) break;
            if (flags & TC_FIRST) {
                cur_seg = rc.seg;
                m = -INFINITY;
                l = 0.f;
                pois = 0;
                fresh = true;
                alive = token < rc.n;
                active = SPLIT || rc.n > t * tile_nodes;
            }
            pois |= rc.poison;
            const bool mine = !SPLIT || (j & 1) == t;
            const bool busy = active && __any_sync(0xffffffffu, alive);
            if (mine) {
                const uint32_t par = (uint32_t)(own & 1);
                const int seen = rc.base + token - rc.t0 + 1;     // keys of the stage that the row sees
                if (!wait_all(s_full(t), par)) {
                    ok = false;
                    break;
                }
                if (busy) {
                    tc_fence_after();
                    if (fresh) rf = rowf[((cur_seg - 1) & 1) * 2 * Tr::TILE + row_of_group];
                    uint32_t u[32];
                    const int vis = alive ? min(seen, rc.nkeys) : KEYS;
                    const bool masked = __any_sync(0xffffffffu, vis < KEYS);
                    if (masked) {
                        // the last stages of a row: scores become final here, -inf where the row does not
                        // see the key, and the loops below, which every stage runs, stay short
#pragma unroll 1
                        for (int c = 0; c < KEYS / 32; ++c) {
                            tmem_ld32(s_addr + 32 * c, u);
                            tmem_ld_wait();
                            after_wait(u);
                            const float by0 = rc.ks[32 * c / BS] * rf, by1 = rc.ks[(32 * c + 16) / BS] * rf;
                            const float lb0 = rc.lb[32 * c / BS], lb1 = rc.lb[(32 * c + 16) / BS];
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const float x = fmaf(__uint_as_float(u[k]), k < 16 ? by0 : by1, k < 16 ? lb0 : lb1);
                                u[k] = 32 * c + k < vis ? __float_as_uint(x) : 0xff800000u;
                            }
                            tmem_st32(s_addr + 32 * c, u);
                        }
                        tmem_st_wait();
                    }
                    auto factor = [&](int key) -> float { return masked ? 1.f : rc.ks[key / BS] * rf; };
                    auto offset = [&](int key) -> float { return masked ? 0.f : rc.lb[key / BS]; };
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < KEYS / 32; ++c) {
                        tmem_ld32(s_addr + 32 * c, u);
                        tmem_ld_wait();
                        after_wait(u);
                        if constexpr (BS == 16) {
                            mx = fmaxf(mx, fmaxf(fmaf(max16(u), factor(32 * c), offset(32 * c)),
                                                 fmaf(max16(u + 16), factor(32 * c + 16), offset(32 * c + 16))));
                        } else {
                            mx = fmaxf(mx, fmaf(fmaxf(max16(u), max16(u + 16)), factor(32 * c), offset(32 * c)));
                        }
                    }
                    const bool need = mx > m + Tr::TAU && alive;
                    const float alpha = need ? ex2(m - mx) : 1.f;     // m = -inf: 0
                    if (need) {
                        m = mx;
                        l *= alpha;
                    }
                    if (!fresh && __any_sync(0xffffffffu, need)) {
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
                    if (SPLIT && t == 1 && fresh && cur_seg > 1) {    // tile 0 has read the last segment's O
                        if (!wait_all(o1_free, (uint32_t)((cur_seg - 2) & 1))) {
                            ok = false;
                            break;
                        }
                    }
                    tmem_ld32(s_addr, u);
                    const float mref = m == -INFINITY ? 0.f : m;      // no visible key yet: weights 0
                    tmem_ld_wait();
                    after_wait(u);
#pragma unroll 1
                    for (int c = 0; c < KEYS / 32; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float by = factor(32 * c + 16 * b), add = offset(32 * c + 16 * b) - mref;
                            const f32x2 by2 = pair2(by, by), add2x = pair2(add, add);
                            f32x2 sum[2] = {0ull, 0ull};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int i = 16 * b + 2 * e;
                                float p0, p1;
                                split2(fma2(pair2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), by2, add2x), p0, p1);
                                p0 = ex2(p0);
                                p1 = ex2(p1);
                                sum[e & 1] = add2(sum[e & 1], pair2(p0, p1));
                                w[8 * b + e] = pack2<false>(p0, p1);
                            }
                            float sa, sb;
                            split2(add2(sum[0], sum[1]), sa, sb);
                            l = fmaf(sa + sb, rc.back[(32 * c + 16 * b) / BS], l);
                        }
                        if (c + 1 < KEYS / 32) tmem_ld32(s_addr + 32 * c + 32, u);
                        tmem_st16(s_addr + 32 * c, w);
                        tmem_st_wait();                               // a quarter of the weights is there
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_part(t, c));
                        tmem_ld_wait();
                        after_wait(u);
                    }
                } else {
                    __syncwarp();
                    if (lane == 0)
                        for (int c = 0; c < 4; ++c) mbar_arrive(p_part(t, c));
                }
                fresh = false;
                ++own;
            }
            if (flags & TC_LAST) {
                // the tile's last product of the segment, if it had a stage in it
                if (!fresh && !wait_all(pv_done(t), (uint32_t)((own - 1) & 1))) {
                    ok = false;
                    break;
                }
                float f0 = 1.f, f1 = 0.f;                             // SPLIT: the factors of both tiles' states
                bool other = false;
                if constexpr (SPLIT) {
                    if (t == 1) {
                        // (tile 0 has read the last segment's state)
                        if (cur_seg > 1 && !wait_all(o1_free, (uint32_t)((cur_seg - 2) & 1))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();                             // O_1 is complete
                        tc_fence_before();
                        xch[r] = make_float2(fresh ? -INFINITY : m, fresh ? 0.f : l);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(joined);
                        continue;
                    }
                    if (!wait_all(joined, (uint32_t)((cur_seg - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    const float2 x = xch[r];
                    const float top = fmaxf(m, x.x), ref = top == -INFINITY ? 0.f : top;
                    // a tile without a stage left nothing in tensor memory: its output is not read
                    other = __any_sync(0xffffffffu, x.x != -INFINITY || x.y != 0.f);
                    f0 = ex2(m - ref);
                    f1 = ex2(x.x - ref);
                    l = l * f0 + x.y * f1;
                    m = top;
                }
                // the segment's values have all been converted; a row that sees one that is not finite is NaN
                if (*const_cast<const volatile int*>(&spoilt[cur_seg % Tr::NREC]) <= rc.base + token) l = qnan;
                if (busy) {
                    tc_fence_after();
                    // 64 bytes of each row at a time (32 finished values, or 16 of a partial state) go
                    // through shared memory, so that 4 lanes write a row's piece
                    uint8_t* out = smem + Tr::OUT_OFF + warp * Tr::OUT_BYTES;
                    const bool complete = flags & TC_COMPLETE;
                    const float inv = pois ? qnan : complete ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                    f0 *= inv;
                    f1 *= inv;
                    const unsigned rows = __ballot_sync(0xffffffffu, alive);
                    const int row0 = (SPLIT ? 0 : t * Tr::TILE) + quarter * 32;   // the warp's first row of the group
                    float* part0 = p.partials + ((size_t)blockIdx.x * 2 + ((flags & TC_SLOT1) ? 1 : 0)) * Tr::ROWS * Tr::PSTRIDE;
                    const int q0 = rc.q0, kvh = rc.kvh;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t u[32];
                        if (!SPLIT || !fresh) {
                            tmem_ld32(o_addr + 32 * c, u);
                            tmem_ld_wait();
                            after_wait(u);
#pragma unroll
                            for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * f0);
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(pois ? qnan : 0.f);
                        }
                        if (SPLIT && other) {
                            uint32_t v[32];
                            tmem_ld32(o_addr + 128 + 32 * c, v);
                            tmem_ld_wait();
                            after_wait(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                u[k] = __float_as_uint(fmaf(__uint_as_float(v[k]), f1, __uint_as_float(u[k])));
                        }
                        const int pieces = complete ? 1 : 2;
                        for (int hf = 0; hf < pieces; ++hf) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint4 v;
                                if (complete) {
                                    auto two = [&](int i) -> uint32_t {
                                        return pack2<Tr::BF16>(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
                                    };
                                    v = make_uint4(two(8 * k), two(8 * k + 2), two(8 * k + 4), two(8 * k + 6));
                                } else {
                                    v = hf ? make_uint4(u[16 + 4 * k], u[17 + 4 * k], u[18 + 4 * k], u[19 + 4 * k])
                                           : make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                                }
                                *reinterpret_cast<uint4*>(out + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = v;
                            }
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int rr = 8 * i + lane / 4, part = lane & 3;
                                const uint4 v = *reinterpret_cast<const uint4*>(out + rr * 64 + ((part ^ ((rr >> 1) & 3)) << 4));
                                if (!((rows >> rr) & 1)) continue;
                                const int row = row0 + rr;
                                if (complete) {
                                    uint16_t* orow = p.out + ((size_t)(q0 + (row >> gs)) * p.Hq + (size_t)kvh * G + (row & (G - 1))) * D;
                                    *reinterpret_cast<uint4*>(orow + 32 * c + 8 * part) = v;
                                } else {
                                    *reinterpret_cast<uint4*>(part0 + (size_t)row * Tr::PSTRIDE + 32 * c + 16 * hf + 4 * part) = v;
                                }
                            }
                            __syncwarp();
                        }
                    }
                    if (alive && !complete) {
                        float* prow = part0 + (size_t)(row0 + lane) * Tr::PSTRIDE;
                        prow[D] = m;
                        prow[D + 1] = l;
                    }
                    tc_fence_before();
                }
                if (SPLIT) {                                          // (tile 0: tile 1's state has been read)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o1_free);
                }
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
cudaError_t chunk_bs8_launch(const MultiLaunch& L) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(L.grid, Tr::THREADS, Tr::SMEM_BYTES, L.stream, attr);
    return cudaLaunchKernelEx(&cfg, pa_chunk_bs8_kernel<Tr>, L.p);
}

template <class Tr>
MultiKernelInfo chunk_bs8_info() {
    return MultiKernelInfo{&chunk_bs8_launch<Tr>,
                           &persistent_ctas<pa_chunk_bs8_kernel<Tr>, Tr::THREADS, Tr::SMEM_BYTES>, Tr::ROWS};
}

// [e5m2][bs == 32][more than 128 rows], one table per (dtype, head_dim), defined in chunk_bs8_*.cu.
void chunk_bs8_table_bf16_d128(MultiKernelInfo (&t)[2][2][2]);
void chunk_bs8_table_bf16_d64(MultiKernelInfo (&t)[2][2][2]);
void chunk_bs8_table_fp16_d128(MultiKernelInfo (&t)[2][2][2]);
void chunk_bs8_table_fp16_d64(MultiKernelInfo (&t)[2][2][2]);

}  // namespace pa
