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
// S_t, 32 columns at the start of each 64 that held its scores.  Weights are
// 2^(x - m) for a reference m that moves (to the maximum, with O rescaled) only when half a stage's
// add up to more than 2^12: fp16 holds any of them, its relative precision is the same at every
// size, and no stage has to know its maximum before its weights.  l adds up the weights with the 11 bits that
// the products read (not with their fp16 underflow: a block of next to nothing counts in l), so that a weight's
// rounding moves a row only by the distance of its value from the row's output, and not at all where one
// key has the row.  Of outputs in fp16, relative to their size (2.07e-4 of it their own rounding):
//                                drafts, 128 sequences     prompt of 4096 tokens
//   l of weights of 24 bits      2.48e-4,  564 us          2.75e-4,  918 us
//   l of weights of 11 bits      2.26e-4,  604 us          2.38e-4,  972 us    (this kernel)
//   ... border 2^9               2.21e-4,  622 us          2.34e-4,  990 us
//   ... border 2^6               2.13e-4,  667 us          2.26e-4, 1031 us
//
// Roles (one CTA per SM; 640 threads for SPLIT, else 512):
//   warps 0-3, 4-7   softmax of tile 0, 1: thread = row = TMEM lane, half of a stage at a time, so that the
//                    products of the first half run beside the softmax of the second
//   8 or 4 warps     per segment the queries, as fp16 under the swizzle that the products read; per
//                    stage the keys, then the values: codes from shared memory, fp16 back.
//                    Value rows past the context become zeros, and so do rows of the chunk that hold
//                    NaN or infinities (rows that see them become NaN at the softmax)
//   2 warps          products of tile 0, 1
//   1 warp           the plan: each stage's place, blocks and scales, as a record for the others
//   1 warp           copies: a bulk copy per block for its keys, one for its values
//
// Bound by the chain of a stage within a tile, not by a unit: at 256 rows and head_dim 128 a stage
// takes 5,800 cycles (5,400 before l added up rounded weights, when this was stamped), of which 2,700 are products of both tiles and 1,100 exponentials; a tile's
// scores (700), their way to the softmax (200), two halves (1,000 to 1,800 each, the loads
// 300 of it), the last products and their way back (700) follow one another, and the tiles'
// warps share issue slots with the conversion (530 of 2,600 instructions of a stage).
// Measured on GB300: 981 to 987 us for 4096 new tokens of one sequence at context 8192, 64 query and 8 KV heads of
// 128 (840 TFLOP/s of 1,905); 576 to 591 us for 128 sequences of 1 to 16 new tokens at contexts of 1024
// to 8192 (2.2 TB/s).  Also measured, against 1,060 us and 636: 64-key products ahead of the
// softmax (1,470 us for the long prompt), scores of one stage in one piece (1,175), two softmax
// warps to a row (1,250), codes loaded into registers from L2 (1,160), the conversion unrolled over
// both kinds (1,190: the roles' loops then fall out of the SM's instruction cache), polling loops
// in place of held waits (no difference), waits that end when another role gives up (640 us against 589: code
// around every wait; without it the CTA is gone within the limit of one wait, not at once).
//
// The work list and the partial states of split rows are those of the tree kernels: each CTA
// takes an equal run of (row group, KV head, block) units; a group's keys end at its
// last token's.  Every wait is bounded (PA_DEVERR_TIMEOUT); a CTA that gives up gives NaN for all that it
// was to write, so that the merge finds nothing of an earlier call.
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
    // SPLIT is the arrangement that HBM feeds: twice the converting warps
    static constexpr int CONVERT_WARPS = SPLIT ? 8 : 4;
    static constexpr int THREADS = 32 * (8 + CONVERT_WARPS + 4);
    // registers after the roles part, in all no more than the launch's: 640 x 96 or 512 x 128
    static constexpr int SOFT_REGS = SPLIT ? 144 : 168, CONVERT_REGS = SPLIT ? 64 : 104, OTHER_REGS = 64;
    static_assert(256 * SOFT_REGS + 32 * CONVERT_WARPS * CONVERT_REGS + 128 * OTHER_REGS <= THREADS * (SPLIT ? 96 : 128), "registers");
    static constexpr int SLOT_BYTES = KEYS * D * 2;          // a stage's keys, or its values, in fp16
    static constexpr int HALF_STRIDE = KEYS * 128;           // between the column halves of a slot
    static constexpr int SMEM_BYTES = 227 * 1024;
    static constexpr int Q_HALF = TILE * 128;
    static constexpr int Q_BYTES = (SPLIT ? 1 : 2) * HALVES * Q_HALF;
    static constexpr int NREC = 8;
    static constexpr int R_CAP = 6;
    static constexpr int N8_CAP = 8;
    // empty, ready; empty8, full8; s_full, p_half[2], pv_half[2] per tile; q_full, q_empty; fin; described, forgotten;
    // listed; joined, o1_free; stall
    static constexpr int NBAR = 2 * R_CAP + 2 * N8_CAP + 2 * 6 + 2 + 2 + 3 * NREC + 3;
    static constexpr int REC_OFF = (8 * NBAR + 15) / 16 * 16;
    static constexpr int REC_BYTES = 48 + 5 * SB * 4;
    static constexpr int SLOT8_BYTES = KEYS * D;             // a stage's key or value codes
    static constexpr int ROWF_OFF = REC_OFF + NREC * REC_BYTES;   // score factors of the rows, two segments
    static constexpr int XCH_OFF = ROWF_OFF + 2 * 2 * TILE * 4;   // SPLIT: tile 1's (m, l) of a row
    static constexpr int MISC_OFF = XCH_OFF + (SPLIT ? TILE * 8 : 0);   // TMEM base, abort flag
    static constexpr int SPOILT_OFF = MISC_OFF + 16;         // per segment: first position of a bad block or a value that is not finite
    static constexpr int NSEG = 2 * NREC;
    static constexpr int START_OFF = SPOILT_OFF + NSEG * 4;  // a TreeStart, a word per warp
    static constexpr int Q_OFF = (START_OFF + 32 + 8 * THREADS / 32 + 1023) / 1024 * 1024;
    static constexpr int RING_OFF = Q_OFF + Q_BYTES;
    // fp16 slots; K and V alternate.  (SPLIT: with three, a tile's next keys wait for its values' slot, 586 us to 567.)
    static constexpr int R = SPLIT ? 4 : 3;
    // slots of codes on their way, a ring for keys and one for values
    static constexpr int RING8_OFF = RING_OFF + R * SLOT_BYTES;
    static constexpr int N8_FIT = (SMEM_BYTES - 1024 - RING8_OFF) / SLOT8_BYTES;
    static constexpr int N8 = N8_FIT > N8_CAP ? N8_CAP : N8_FIT;
    static constexpr int NK8 = (N8 + 1) / 2, NV8 = N8 / 2;
    static constexpr int CONVERT_WARP = 8, MMA_WARP = CONVERT_WARP + CONVERT_WARPS, PLAN_WARP = MMA_WARP + 2, COPY_WARP = MMA_WARP + 3;
    static constexpr int TMEM_COLS = 512;
    static constexpr int O_COL = 256;
    static constexpr int PSTRIDE = D + 4;
    static constexpr float MOST = 4096.f;                 // that the weights of half a stage may add up to
    static_assert(N8 >= 2 && RING_OFF % 1024 == 0, "shared memory");
};

// One stage as the planning warp describes it, and its blocks.
template <int SB>
struct alignas(16) ChunkStage {
    int base, kvh, t0, nkeys;     // position of the group's first token, KV head, first key, keys copied
    int n, ctx, q0, flags;        // tokens of the group, context, the group's first query row
    int seg, chunk, cuts, spare;  // segment number; the chunk's first position; any cut != 1
    int ids[SB];
    float ks[SB], lb[SB], back[SB], cut[SB];   // key scale, lb, 2^-lb, f of decode_bs8.cuh
};

// Waits with a hint of how long the hardware may hold the warp before the test answers (20 us): a warp that
// polls takes issue slots from the others.  In few instructions, because the roles' loops together
// have to fit the instruction cache.
__device__ __forceinline__ bool try_wait_held(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 20000;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
#pragma unroll 1
    while (!try_wait_held(bar, parity)) {
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) return false;
    }
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The maximum of 16 scores.
__device__ __forceinline__ float max16(const uint32_t* u) {
    auto f = [&](int i) -> float { return __uint_as_float(u[i]); };
    const float a = max3(max3(f(0), f(1), f(2)), f(3), f(4)), b = max3(max3(f(5), f(6), f(7)), f(8), f(9));
    const float c = max3(max3(f(10), f(11), f(12)), f(13), f(14));
    return fmaxf(max3(a, b, c), f(15));
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <class Tr>
__global__ void __launch_bounds__(Tr::THREADS, 1)
pa_chunk_bs8_kernel(const MultiParams mp) {
    constexpr int D = Tr::D, BS = Tr::BS, SB = Tr::SB, HALVES = Tr::HALVES, KEYS = Tr::KEYS, R = Tr::R;
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
    const uint32_t q_base = sbase + Tr::Q_OFF, ring = sbase + Tr::RING_OFF;
    auto empty = [&](int st) -> uint32_t { return sbase + 8 * st; };
    auto ready = [&](int st) -> uint32_t { return sbase + 8 * (Tr::R_CAP + st); };
    auto empty8 = [&](int st) -> uint32_t { return sbase + 8 * (2 * Tr::R_CAP + st); };
    auto full8 = [&](int st) -> uint32_t { return sbase + 8 * (2 * Tr::R_CAP + Tr::N8_CAP + st); };
    // the slot of stage j's key codes (op 0) or value codes (1), and how often it has been used before
    auto slot8 = [&](int op, int j) -> int { return op ? Tr::NK8 + j % Tr::NV8 : j % Tr::NK8; };
    auto uses8 = [&](int op, int j) -> int { return op ? j / Tr::NV8 : j / Tr::NK8; };
    const uint32_t ring8 = sbase + Tr::RING8_OFF;
    const uint32_t tile_bars = sbase + 8 * (2 * Tr::R_CAP + 2 * Tr::N8_CAP);
    auto s_full = [&](int t) -> uint32_t { return tile_bars + 48 * t; };                        // a stage's scores,
    auto p_half = [&](int t, int h) -> uint32_t { return tile_bars + 48 * t + 16 + 8 * h; };    // half of its weights
    auto pv_half = [&](int t, int h) -> uint32_t { return tile_bars + 48 * t + 32 + 8 * h; };   // and its products
    const uint32_t q_full = tile_bars + 96, q_empty = q_full + 8, fin = q_empty + 8;   // fin[2]
    auto described = [&](int j) -> uint32_t { return fin + 16 + 8 * (j % Tr::NREC); };                // stage j's record stands
    auto forgotten = [&](int j) -> uint32_t { return fin + 16 + 8 * (Tr::NREC + j % Tr::NREC); };      // no one reads it any more
    auto listed = [&](int j) -> uint32_t { return fin + 16 + 8 * (2 * Tr::NREC + j % Tr::NREC); };     // its blocks do, without their scales
    // SPLIT: tile 1's state of a segment is there; tile 0 has read it
    const uint32_t joined = fin + 16 + 8 * 3 * Tr::NREC, o1_free = joined + 8;
    const uint32_t stall_bar = o1_free + 8;                    // nothing completes it (pa_set_decode_stall_ns)
    Stage* recs = reinterpret_cast<Stage*>(smem + Tr::REC_OFF);
    float* rowf = reinterpret_cast<float*>(smem + Tr::ROWF_OFF);
    float2* xch = reinterpret_cast<float2*>(smem + Tr::XCH_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Tr::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Tr::MISC_OFF + 4);
    // (of segment s at s % NSEG: no role is that many stages ahead of another)
    int* spoilt = reinterpret_cast<int*>(smem + Tr::SPOILT_OFF);

    if (threadIdx.x == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(empty(i), SPLIT ? 1 : 2);     // its tile is done with it, or both are
            mbar_init(ready(i), Tr::CONVERT_WARPS);
        }
        for (int i = 0; i < Tr::N8; ++i) {
            mbar_init(empty8(i), Tr::CONVERT_WARPS);
            mbar_init(full8(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(p_half(t, h), 4);
                mbar_init(pv_half(t, h), 1);
            }
            mbar_init(fin + 8 * t, 1);
        }
        mbar_init(q_full, Tr::CONVERT_WARPS);
        mbar_init(q_empty, 2);
        for (int i = 0; i < Tr::NREC; ++i) {
            mbar_init(described(i), 1);
            mbar_init(listed(i), 1);
            // converting warps, products, softmax warps, copies
            mbar_init(forgotten(i), Tr::CONVERT_WARPS + 2 + 8 + 1);
        }
        mbar_init(joined, 4);
        mbar_init(o1_free, 4);
        mbar_init(stall_bar, 1);
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

    if (warp >= Tr::MMA_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Tr::OTHER_REGS));
        if (warp == Tr::PLAN_WARP) {
            // ============================================================ the stages, and their blocks' scales
            if (lane == 0) mp.starts[blockIdx.x] = at;
            struct Next {                            // a stage whose blocks' scales are on their way
                int base, kvh, t0, nbs, n, ctx, q0, flags, seg, chunk, id;
                bool bad;
                float2 scales;
            };
            SegIter it{lo, at.s, at.kvh, at.b0, at.nb, 0};
            const int32_t* trow = nullptr;
            int len = 0, k = 0, nseg = 0, ids = 0, ids_next = 0, n = 0, ctx = 0, q0 = 0, size = 0, skip = 0, seg_flags = 0;
            auto batch = [&](int from) -> int { return lane < len - from ? __ldg(trow + from + lane) : 0; };
            auto advance = [&](Next& x) -> bool {
                if (len > 0 && k * SB >= len) {      // the segment is done
                    seg_advance(it, len, p, tab);
                    len = 0;
                }
                if (len == 0) {
                    if (!has_work || it.gi >= hi) return false;
                    len = seg_len(it, hi);
                    k = 0;
                    const int s = it.s % seqs;
                    skip = it.s / seqs * mp.group_nodes;
                    size = chunk_size(s);
                    n = min(mp.group_nodes, size - skip);                      // > 0: it has blocks
                    ctx = __ldg(p.context_lens + s);
                    q0 = __ldg(qst + s) + skip;
                    const long long P0 = it.gi - it.b0;
                    seg_flags = (sc.of(P0) == sc.of(P0 + it.nb - 1) ? TC_COMPLETE : 0) | (it.gi == lo ? 0 : TC_SLOT1);
                    ++nseg;
                    trow = p.block_tables + (size_t)s * p.MB + it.b0;
                    ids = batch(0);
                    ids_next = batch(32);
                }
                const int bb = k * SB;
                if (bb > 0 && (bb & 31) == 0) {
                    ids = ids_next;
                    ids_next = batch(bb + 32);
                }
                x.nbs = min(SB, len - bb);
                x.id = __shfl_sync(0xffffffffu, ids, (bb + lane) & 31);
                const bool held = lane < x.nbs;
                x.bad = held && (unsigned)x.id >= (unsigned)p.NB;
                if (!held || x.bad) x.id = 0;
                x.scales = make_float2(0.f, 0.f);
                if (held && !x.bad) x.scales = __ldg(reinterpret_cast<const float2*>(p.kv8 + ((size_t)x.id * p.Hkv + it.kvh) * bs8_piece_bytes(BS, D)));
                x.base = ctx - size + skip;
                x.kvh = it.kvh;
                x.t0 = (it.b0 + bb) * BS;
                x.n = n;
                x.ctx = ctx;
                x.q0 = q0;
                x.flags = seg_flags | (k == 0 ? TC_FIRST : 0) | (bb + SB >= len ? TC_LAST : 0);
                x.seg = nseg;
                x.chunk = ctx - size;
                ++k;
                return true;
            };
            float top_lb = -INFINITY;                             // R of decode_bs8.cuh
            bool ok = true;
            Next x, y;
            bool more = false;
            for (int j = -1;; ++j) {
                const bool then = (more || j < 0) && advance(y);
                if (j < 0) {
                    x = y;
                    more = then;
                    continue;
                }
                const bool stop = j >= Tr::NREC && (*abort_flag != 0 || !wait_bounded(forgotten(j), (uint32_t)((j / Tr::NREC - 1) & 1), p.timeout_ns));
                if (__any_sync(0xffffffffu, stop)) {
                    ok = false;
                    break;
                }
                Stage& rc = recs[j % Tr::NREC];
                if (!more) {
                    if (lane == 0) {
                        rc.flags = TC_END;
                        mbar_arrive(listed(j));
                        mbar_arrive(described(j));
                    }
                    break;
                }
                if (x.flags & TC_FIRST) {
                    top_lb = -INFINITY;
                    if (lane == 0) spoilt[x.seg % Tr::NSEG] = INT_MAX;
                }
                // what the copies need goes ahead of what waits for the scales
                if (lane < SB) rc.ids[lane] = x.id;
                if (lane == 0) {
                    rc.base = x.base;
                    rc.kvh = x.kvh;
                    rc.t0 = x.t0;
                    rc.nkeys = x.nbs * BS;
                    rc.n = x.n;
                    rc.ctx = x.ctx;
                    rc.q0 = x.q0;
                    rc.flags = x.flags;
                    rc.seg = x.seg;
                    rc.chunk = x.chunk;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(listed(j));
                const bool held_here = lane < x.nbs;
                const bool bad_scale = held_here && (!bs8_is_scale(x.scales.x) || !bs8_is_scale(x.scales.y));
                if (bad_scale) x.scales = make_float2(0.f, 0.f);   // (rows that do not see the block keep their sums)
                const float lb = held_here ? fmaxf(__log2f(x.scales.y), -126.f) : -INFINITY;
                float top = lb;
#pragma unroll
                for (int o = 1; o < SB; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top_lb = fmaxf(top_lb, __shfl_sync(0xffffffffu, top, 0));
                const float held = fmaxf(lb, fmaxf(top_lb - BS8_LB_RANGE, BS8_LB_FLOOR));
                const float cut = held_here ? ex2(lb - held) : 1.f;
                if (lane < SB) {
                    rc.ks[lane] = x.scales.x;
                    rc.lb[lane] = held;
                    rc.back[lane] = ex2(-held);
                    rc.cut[lane] = cut;
                }
                const bool any_id = __any_sync(0xffffffffu, x.bad), any_scale = __any_sync(0xffffffffu, bad_scale);
                const uint32_t bad = __ballot_sync(0xffffffffu, x.bad || bad_scale);
                const bool any_cut = __any_sync(0xffffffffu, cut != 1.f);
                if (lane == 0) {
                    if (any_id) set_err(p.err, PA_DEVERR_BLOCK_ID);
                    if (any_scale) set_err(p.err, PA_DEVERR_SCALE);
                    if (bad) atomicMin(&spoilt[x.seg % Tr::NSEG], x.t0 + (__ffs((int)bad) - 1) * BS);
                    rc.cuts = any_cut;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(described(j));
                x = y;
                more = then;
            }
            if (!ok && lane == 0) {
                set_err(p.err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
        } else if (warp == Tr::COPY_WARP) {
            // ============================================================ copies of the codes
            {
                // with one group the codes are read once per call; with more, other CTAs read them too
                const uint64_t kv_pol = mp.groups == 1 ? l2_evict_first() : l2_evict_normal();
                int copied[2] = {0, 0};
                bool ok = true;
                for (int j = 0; ok; ++j) {
                    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                        const bool good = *abort_flag == 0 && wait_bounded(bar, parity, p.timeout_ns);
                        return __all_sync(0xffffffffu, good);
                    };
                    if (!wait(listed(j), (uint32_t)((j / Tr::NREC) & 1))) {
                        ok = false;
                        break;
                    }
                    const Stage& rc = recs[j % Tr::NREC];
                    if (rc.flags & TC_END) break;
                    const int nbs = rc.nkeys / BS;
                    const uint8_t* codes = p.kv8 + ((size_t)rc.ids[lane < nbs ? lane : 0] * p.Hkv + rc.kvh) * bs8_piece_bytes(BS, D) + BS8_HEAD;
                    for (int op = 0; op < 2; ++op) {              // keys, values
                        const int st = slot8(op, j), n = uses8(op, j);
                        if (n > 0 && !wait(empty8(st), (uint32_t)((n - 1) & 1))) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(full8(st), (uint32_t)(nbs * BS * D));
                        __syncwarp();
                        if (lane < nbs)
                            bulk_load_hint(ring8 + st * Tr::SLOT8_BYTES + lane * BS * D, codes + op * BS * D, BS * D, full8(st), kv_pol);
                        ++copied[op];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(forgotten(j));
                }
                if (!ok && lane == 0) {
                    set_err(p.err, PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                }
                // Copies still in flight land before the CTA's shared memory is released, whoever gave up (the converting
                // warps may have left stages that were copied long before).
                if (lane == 0) {
                    for (int op = 0; op < 2; ++op)
                        for (int k = max(0, copied[op] - (op ? Tr::NV8 : Tr::NK8)); k < copied[op]; ++k)
                            wait_bounded(full8(slot8(op, k)), (uint32_t)(uses8(op, k) & 1), p.timeout_ns);
                }
            }
        } else {
            // ============================================================ products of one tile
            // The whole warp runs the loop and one lane of it issues, so that descriptors and addresses are
            // uniform to the compiler: a loop of one thread issued a product in 150 cycles, not 64 (636 to 596
            // us and 1,061 to 996).  Commits give the slots back, and the next stage's record and keys are
            // waited for before the last products are through (to 585 and 972).
            const int t = __shfl_sync(0xffffffffu, warp, 0) - Tr::MMA_WARP;
            const uint32_t s_col = tmem + 128 * t, o_col = tmem + Tr::O_COL + 128 * t;
            const uint32_t q_tile = q_base + (SPLIT ? 0 : t * HALVES * Tr::Q_HALF);
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                if (__builtin_expect(__all_sync(0xffffffffu, try_wait_held(bar, parity)), 1)) return true;
                if (!__all_sync(0xffffffffu, *abort_flag == 0 && wait_bounded(bar, parity, p.timeout_ns))) ok = false;
                return ok;
            };
            auto arrive = [&](uint32_t bar) {                     // for what all lanes have done
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            int own = 0, nseg = 0;                 // stages of this tile; segments begun
            bool fresh = true;                     // O holds nothing of the segment
            bool active = true;
            for (int j = 0;; ++j) {
                if (!wait(described(j), (uint32_t)((j / Tr::NREC) & 1))) break;
                const Stage& rc = recs[j % Tr::NREC];
                const int flags = rc.flags;
                if (flags & TC_END) break;
                if (flags & TC_FIRST) {
                    if (!wait(q_full, (uint32_t)(nseg & 1))) break;
                    ++nseg;
                    fresh = true;
                    active = SPLIT || rc.n > t * tile_nodes;
                }
                arrive(forgotten(j));
                if (SPLIT && (j & 1) != t) {                      // the other tile's stage
                    if ((flags & TC_LAST) && elect_one()) mma_commit(q_empty);
                    continue;
                }
                const int ks = 2 * j % R, vs = (2 * j + 1) % R;
                const uint32_t par = (uint32_t)(own & 1);
                if (!wait(ready(ks), (uint32_t)((2 * j / R) & 1))) break;
                // the scores overwrite the last stage's weights
                if (own > 0 && !wait(pv_half(t, 1), par ^ 1u)) break;
                if (active) {
                    tc_fence_after();
                    const uint64_t qd = sdesc_sw128(q_tile, 16, 1024), kd = sdesc_sw128(ring + ks * Tr::SLOT_BYTES, 16, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_f16(s_col, qd + (uint64_t)((k / 4) * (Tr::Q_HALF >> 4) + (k % 4) * 2),
                                    kd + (uint64_t)((k / 4) * (Tr::HALF_STRIDE >> 4) + (k % 4) * 2), IDESC_S, k > 0 ? 1u : 0u);
                        mma_commit(s_full(t));
                        mma_commit(empty(ks));
                        if (flags & TC_LAST) mma_commit(q_empty);
                    }
                    __syncwarp();
                } else {
                    arrive(s_full(t));
                    arrive(empty(ks));
                    if (flags & TC_LAST) arrive(q_empty);
                }
                if (!wait(ready(vs), (uint32_t)(((2 * j + 1) / R) & 1))) break;
                bool stop = false;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {                     // as each half of the weights is there
                    if (!wait(p_half(t, h), par)) {
                        stop = true;
                        break;
                    }
                    if (active) {
                        tc_fence_after();
                        const uint64_t vd = sdesc_sw128(ring + vs * Tr::SLOT_BYTES + h * 8192, Tr::HALF_STRIDE, 1024);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f16_ts(o_col, s_col + 64 * h + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), IDESC_O,
                                           fresh && h + k == 0 ? 0u : 1u);
                            mma_commit(pv_half(t, h));
                            if (h == 1) mma_commit(empty(vs));
                        }
                        __syncwarp();
                    } else {
                        arrive(pv_half(t, h));
                        if (h == 1) arrive(empty(vs));
                    }
                }
                if (stop) break;
                fresh = false;
                ++own;
            }
            if (!ok && lane == 0) {
                set_err(p.err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            // every MMA of this thread completes before tensor memory is released
            if (elect_one()) mma_commit(fin + 8 * t);
            __syncwarp();
            wait_bounded(fin + 8 * t, 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp >= Tr::CONVERT_WARP) {
        // ================================================================ queries, keys and values to fp16
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Tr::CONVERT_REGS));
        const int cw = warp - Tr::CONVERT_WARP;
        // A lane's share of a row: one 16-byte part of codes.  Eight neighbouring lanes hold four
        // parts each of two neighbouring rows, a warp 512 consecutive bytes of a piece; as fp16 the eight
        // lanes' parts fall into eight different 16-byte bank groups.
        constexpr int RPW = D == 128 ? 4 : 8;                     // rows a warp takes at once
        constexpr int STEP = Tr::CONVERT_WARPS * RPW;             // rows of a round
        constexpr int NI = KEYS / STEP;                           // rounds of a slot
        const int part = D == 128 ? (lane & 3) | (((lane >> 2) ^ (lane >> 3)) & 1) << 2 : lane & 3;
        const int row0 = cw * RPW + (D == 128 ? ((lane >> 2) & 1) | (lane >> 4) << 1 : lane >> 2);
        const float qnan = __int_as_float(0x7fc00000);
        int nseg = 0;
        bool ok = true;
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            if (__builtin_expect(__all_sync(0xffffffffu, try_wait_held(bar, parity)), 1)) return true;
            return __all_sync(0xffffffffu, *abort_flag == 0 && wait_bounded(bar, parity, p.timeout_ns));
        };
        // sixteen codes -> sixteen values
        auto widen = [&](const uint32_t (&c)[4], uint32_t (&h)[8]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fp8x4_to_f16x4<Tr::E5M2>(c[i], h[2 * i], h[2 * i + 1]);
            }
        };
        // the lane's place in a slot: its two 16-byte parts of row row0; round i is i * STEP rows on
        const uint32_t put0 = (part >> 2) * Tr::HALF_STRIDE + row0 * 128;
        const uint32_t put_a = put0 + (((2 * (part & 3)) ^ (row0 & 7)) << 4), put_b = put0 + (((2 * (part & 3) + 1) ^ (row0 & 7)) << 4);
        auto put = [&](uint32_t slot, int i, const uint32_t (&h)[8]) {
            const uint32_t a = slot + i * (STEP * 128);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + put_a), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + put_b), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                         : "memory");
        };
        auto place = [&](int op, int row) -> uint32_t {           // of the lane's part in a slot of codes
            return (row / BS) * BS * D +
                   (op ? bs8_value<BS, D>(row % BS, part) - BS * D - BS8_HEAD : bs8_key<D>(row % BS, part) - BS8_HEAD);
        };
        // item 2 j (+ 1): keys (values) of stage j, into slot item % R once its last use is over
        auto claim = [&](int item) -> bool { return item < R || wait_all(empty(item % R), (uint32_t)((item / R - 1) & 1)); };
        auto done = [&](int item) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready(item % R));
        };
        ok = wait_all(described(0), 0);
        if (ok && p.stall_ns != 0 && !(recs[0].flags & TC_END))
            ok = __all_sync(0xffffffffu, wait_bounded(stall_bar, 0, p.stall_ns));
        for (int j = 0; ok; ++j) {
            Stage& rc = recs[j % Tr::NREC];
            const int flags = rc.flags;
            if (flags & TC_END) break;
            if (flags & TC_FIRST) {                               // the segment's queries
                if (nseg > 0 && !wait_all(q_empty, (uint32_t)((nseg - 1) & 1))) {
                    ok = false;
                    break;
                }
                // four lanes hold a row; rows past the last one in a tile have to be finite: zeros
                constexpr int NQ = D / 32;                        // 16-byte parts of a lane
                const int rows = min(rc.n << gs, Tr::ROWS), end = (rows + Tr::TILE - 1) / Tr::TILE * Tr::TILE;
#pragma unroll 1
                for (int row = 8 * cw + lane / 4; row < end; row += 8 * Tr::CONVERT_WARPS) {
                    const uint4* src = reinterpret_cast<const uint4*>(
                        p.q + ((size_t)(rc.q0 + (row >> gs)) * p.Hq + (size_t)rc.kvh * G + (row & (G - 1))) * D);
                    uint4 x[NQ];
#pragma unroll
                    for (int i = 0; i < NQ; ++i) x[i] = row < rows ? __ldg(src + (lane & 3) + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < NQ; ++i)
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
                    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = max(top & 0xffffu, top >> 16);
                    float2 f = make_float2(1.f, 1.f);
                    if constexpr (Tr::BF16) f = row_factor((int)(top >> 7));
                    if (p.scale_log2 < 0.f) f.x = -f.x;
                    // an infinite query has infinite scores or NaN: no weights (all at -inf would look like a row that
                    // sees nothing)
                    const bool finite = top < (Tr::BF16 ? 0x7f80u : 0x7c00u);
                    if ((lane & 3) == 0) rowf[(nseg & 1) * 2 * Tr::TILE + row] = finite ? f.y * scale_abs : qnan;
                    const int r = row % Tr::TILE;
                    const uint32_t a = q_base + row / Tr::TILE * (HALVES * Tr::Q_HALF) + r * 128;
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const int c = (lane & 3) + 4 * i;
                        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack2<false>(lo_of<Tr::BF16>(w[e]) * f.x, hi_of<Tr::BF16>(w[e]) * f.x);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + (c / 8) * Tr::Q_HALF + (((c & 7) ^ (r & 7)) << 4)),
                                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                    }
                }
                ++nseg;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const int t0 = rc.t0, held = min(rc.nkeys, rc.ctx - t0), from = rc.chunk - t0;   // rows with values; of the chunk
            const bool cuts = rc.cuts;
#pragma unroll 1
            for (int op = 0; op < 2 && ok; ++op) {                // keys, values
                const int st = slot8(op, j), item = 2 * j + op;
                if (!wait_all(full8(st), (uint32_t)(uses8(op, j) & 1)) || !claim(item)) {
                    ok = false;
                    break;
                }
                const uint32_t src = ring8 + st * Tr::SLOT8_BYTES, slot = ring + (item % R) * Tr::SLOT_BYTES;
                const uint32_t in0 = place(op, row0), in1 = place(op, row0 + STEP);
                const bool care = op && (held < KEYS || from < KEYS || cuts);
#pragma unroll (SPLIT ? 1 : 2)                            // (SPLIT: by two 611 us, by four 677, by one 567)
                for (int i = 0; i < NI; ++i) {
                    uint32_t c[4], h[8];
                    const int row = row0 + i * STEP;
                    lds128(src + (i / 2) * (2 * STEP * D) + (i & 1 ? in1 : in0), c);
                    if (care) {
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t odd = ((c[e] & 0x7f7f7f7fu) + (Tr::E5M2 ? 0x04040404u : 0x01010101u)) & 0x80808080u;
                            if (row >= from) {
                                any |= odd;
                                c[e] &= ~(odd / 128 * 255);
                            }
                            if (row >= held) c[e] = 0u;
                        }
                        if (any && row < held) atomicMin(&spoilt[rc.seg % Tr::NSEG], t0 + row);
                    }
                    widen(c, h);
                    if (care && cuts) {                           // blocks of next to nothing
                        const float cut = rc.cut[row / BS];
                        const uint32_t by = pack2<false>(cut, cut);
#pragma unroll
                        for (int e = 0; e < 8; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(by));
                    }
                    put(slot, i, h);
                }
                done(item);
                if (lane == 0) mbar_arrive(empty8(st));
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(forgotten(j));
            if (!wait_all(described(j + 1), (uint32_t)(((j + 1) / Tr::NREC) & 1))) {
                ok = false;
                break;
            }
        }
        if (!ok && lane == 0) {
            set_err(p.err, PA_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ================================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Tr::SOFT_REGS));
        const int t = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;                        // row of the tile = TMEM lane
        const int row_of_group = SPLIT ? r : t * Tr::TILE + r;
        const int token = row_of_group >> gs;                     // of the group
        auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
            if (__builtin_expect(__all_sync(0xffffffffu, try_wait_held(bar, parity)), 1)) return true;
            return __all_sync(0xffffffffu, wait_bounded(bar, parity, p.timeout_ns));
        };
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lane_addr + 128 * t, o_addr = lane_addr + Tr::O_COL + 128 * t;
        const float qnan = __int_as_float(0x7fc00000);
        int own = 0, cur_seg = 0, seg_q0 = 0, seg_kvh = 0, last_seen = 0;
        float m = -INFINITY, l = 0.f, rf = 0.f;                   // reference (log2 units), sum, the row's score factor
        bool alive = false, active = false, fresh = true, ok = true;
        for (int j = 0;; ++j) {
            if (!wait_all(described(j), (uint32_t)((j / Tr::NREC) & 1))) {
                ok = false;
                break;
            }
            const Stage& rc = recs[j % Tr::NREC];
            const int flags = rc.flags;
            if (flags & TC_END) break;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) {
                ok = false;
                break;
            }
            if (flags & TC_FIRST) {
                cur_seg = rc.seg;
                seg_q0 = rc.q0;                                   // (a record may be written again before a segment's end is over)
                seg_kvh = rc.kvh;
                last_seen = rc.base + token;
                m = -INFINITY;
                l = 0.f;
                fresh = true;
                alive = token < rc.n;
                active = SPLIT || rc.n > t * tile_nodes;
            }
            const bool mine = !SPLIT || (j & 1) == t;
            const bool busy = active && __any_sync(0xffffffffu, alive);
            if (mine) {
                const uint32_t par = (uint32_t)(own & 1);
                const int seen = last_seen - rc.t0 + 1;     // keys of the stage that the row sees
                if (busy) {
                    if (!wait_all(s_full(t), par)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (fresh) rf = rowf[((cur_seg - 1) & 1) * 2 * Tr::TILE + row_of_group];
                    if (SPLIT && t == 1 && fresh && cur_seg > 1) {    // tile 0 has read the last segment's O
                        if (!wait_all(o1_free, (uint32_t)((cur_seg - 2) & 1))) {
                            ok = false;
                            break;
                        }
                    }
                    const int vis = alive ? min(seen, rc.nkeys) : KEYS;
                    const bool masked = __any_sync(0xffffffffu, vis < KEYS);
                    if (masked) {
                        // The last stages of a row: scores become final here, -inf where the row does not see the
                        // key, in tensor memory, so that the loop below, which every stage runs, has one form.
#pragma unroll 1
                        for (int c = 0; c < KEYS / 16; ++c) {
                            uint32_t x[16];
                            tmem_ld16(s_addr + 16 * c, x);
                            const float by = rc.ks[16 * c / BS] * rf, add = rc.lb[16 * c / BS];
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                asm volatile("" : "+r"(x[k]));
                                x[k] = 16 * c + k < vis ? __float_as_uint(fmaf(__uint_as_float(x[k]), by, add)) : 0xff800000u;
                            }
                            tmem_st16(s_addr + 16 * c, x);
                        }
                        tmem_st_wait();
                    }
                    // Half of the scores at a time becomes weights in the first 32 of the 64 columns that held
                    // them, by the row's reference as it stands; only where there is none yet, or the weights
                    // add up to more than fp16 holds with room to spare, are the scores' maxima looked for and
                    // the half done again (the scores are still there).  O is rescaled behind the products of the
                    // half before.
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        bool redo = __any_sync(0xffffffffu, alive && m == -INFINITY);
                        float by[4], add[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            by[b] = masked ? 1.f : rc.ks[(64 * h + 16 * b) / BS] * rf;
                            add[b] = masked ? 0.f : rc.lb[(64 * h + 16 * b) / BS];
                        }
                        uint32_t w[32];
                        float sum, plain;
#pragma unroll 1
                        for (;;) {
                            uint32_t u[64];
                            tmem_ld64_wait(s_addr + 64 * h, u);
                            if (redo) {
                                const float mx = fmaxf(fmaxf(fmaf(max16(u), by[0], add[0]), fmaf(max16(u + 16), by[1], add[1])),
                                                       fmaxf(fmaf(max16(u + 32), by[2], add[2]), fmaf(max16(u + 48), by[3], add[3])));
                                const bool need = mx > m && alive;
                                const float alpha = need ? ex2(m - mx) : 1.f;     // m = -inf: 0
                                if (need) {
                                    m = mx;
                                    l *= alpha;
                                }
                                if ((!fresh || h > 0) && __any_sync(0xffffffffu, need)) {
                                    if (!wait_all(pv_half(t, h ^ 1), h == 0 ? par ^ 1u : par)) {
                                        ok = false;
                                        break;
                                    }
                                    tc_fence_after();
#pragma unroll 1
                                    for (int i = 0; i < D / 16; ++i) {
                                        uint32_t x[16];
                                        tmem_ld16(o_addr + 16 * i, x);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int k = 0; k < 16; ++k) {
                                            asm volatile("" : "+r"(x[k]));
                                            x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
                                        }
                                        tmem_st16(o_addr + 16 * i, x);
                                    }
                                    tmem_st_wait();
                                }
                            }
                            const float mref = m == -INFINITY ? 0.f : m;          // no visible key yet: weights 0
                            sum = plain = 0.f;
                            auto weigh = [&](const uint32_t* x, int b) {          // 16 scores -> 8 columns of weights
                                const f32x2 by2 = pair2(by[b], by[b]), add2x = pair2(add[b] - mref, add[b] - mref);
                                f32x2 s2[2] = {0ull, 0ull};
                                // The weight with fp16's 11 bits: p - 2^13 p rounded to 24 bits, plus 2^13 p, which
                                // stands on the places that were left.  (2^13 p + p - 2^13 p would round weights next below
                                // a power of two to 10 bits, and a row's largest is often the one next below 1.)
                                const f32x2 up2 = pair2(8192.f, 8192.f), down2 = pair2(-8192.f, -8192.f);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    float p0, p1;
                                    split2(fma2(pair2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), by2, add2x), p0, p1);
                                    p0 = ex2(p0);
                                    p1 = ex2(p1);
                                    const f32x2 p2 = pair2(p0, p1);
                                    s2[e & 1] = add2(s2[e & 1], fma2(p2, up2, fma2(p2, down2, p2)));
                                    w[8 * b + e] = pack2<false>(p0, p1);
                                }
                                float sa, sb;
                                split2(add2(s2[0], s2[1]), sa, sb);
                                plain += sa + sb;
                                sum = fmaf(sa + sb, rc.back[(64 * h + 16 * b) / BS], sum);
                            };
                            weigh(u, 0);
                            weigh(u + 16, 1);
                            weigh(u + 32, 2);
                            weigh(u + 48, 3);
                            if (redo) break;
                            // (a weight above 2^114 is -inf or NaN with 11 bits)
                            redo = __any_sync(0xffffffffu, alive && !(fabsf(plain) <= Tr::MOST));
                            if (!redo) break;
                        }
                        if (!ok) break;
                        tmem_st32(s_addr + 64 * h, w);
                        l += sum;
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_half(t, h));
                    }
                    if (!ok) break;
                } else {
                    if (!wait_all(s_full(t), par)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        for (int h = 0; h < 2; ++h) mbar_arrive(p_half(t, h));
                    }
                }
                fresh = false;
                ++own;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(forgotten(j));
            if (flags & TC_LAST) {
                // the tile's last product of the segment, if it had a stage in it
                if (!fresh && !wait_all(pv_half(t, 1), (uint32_t)((own - 1) & 1))) {
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
                // the segment's values have all been converted; a row that sees one that is not finite, or a block with a bad
                // id or scale, is NaN
                if (*const_cast<const volatile int*>(&spoilt[cur_seg % Tr::NSEG]) <= last_seen) l = qnan;
                if (busy) {
                    tc_fence_after();
                    const bool complete = flags & TC_COMPLETE;
                    const float inv = l != l ? qnan : complete ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                    f0 *= inv;
                    f1 *= inv;
                    // Each lane writes its row, 32 columns at a time (rows of one token stand side by side in the output, so
                    // the sectors fill up in L2; exchanging them through shared memory first took 3 us longer
                    // for a short chunk, cold code included, and nothing less for long ones).
                    const int row = (SPLIT ? 0 : t * Tr::TILE) + r;
                    float* prow = p.partials + (((size_t)blockIdx.x * 2 + ((flags & TC_SLOT1) ? 1 : 0)) * Tr::ROWS + row) * Tr::PSTRIDE;
                    uint16_t* orow = p.out + ((size_t)(seg_q0 + (row >> gs)) * p.Hq + (size_t)seg_kvh * G + (row & (G - 1))) * D;
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
                            for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(l != l ? qnan : 0.f);
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
                        if (alive && complete) {
                            auto two = [&](int i) -> uint32_t {
                                return pack2<Tr::BF16>(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
                            };
#pragma unroll
                            for (int k = 0; k < 32; k += 8)
                                *reinterpret_cast<uint4*>(orow + 32 * c + k) = make_uint4(two(k), two(k + 2), two(k + 4), two(k + 6));
                        } else if (alive) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<uint4*>(prow + 32 * c + k) = make_uint4(u[k], u[k + 1], u[k + 2], u[k + 3]);
                        }
                        __syncwarp();
                    }
                    if (alive && !complete) {
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
            // The rows and partial states of the CTA's whole run become NaN, each by the thread that it is written by (an
            // l of NaN is NaN after the merge, whatever stands beside it).  Rows written before are among them.
            // (the run is found again from shared memory: what is kept for it costs the loop registers)
            const volatile TreeStart& from = *reinterpret_cast<TreeStart*>(smem + Tr::START_OFF);
            const Sched sc = tree_sched(from.W, gridDim.x, SB);
            const bool has_rows = (int)blockIdx.x < sc.NS && !(SPLIT && t == 1);
            const long long lo = has_rows ? sc.lo(blockIdx.x) : 0, hi = has_rows ? sc.lo(blockIdx.x + 1) : 0;
            SegIter it{lo, from.s, from.kvh, from.b0, from.nb, 0};
            while (it.gi < hi) {
                const int len = seg_len(it, hi), s = it.s % seqs, skip = it.s / seqs * mp.group_nodes;
                if (token < min(mp.group_nodes, chunk_size(s) - skip)) {
                    const long long P0 = it.gi - it.b0;
                    if (sc.of(P0) == sc.of(P0 + it.nb - 1)) {
                        uint4* orow = reinterpret_cast<uint4*>(
                            p.out + ((size_t)(__ldg(qst + s) + skip + token) * p.Hq + (size_t)it.kvh * G + (row_of_group & (G - 1))) * D);
                        const uint32_t two = qnan16<Tr::BF16>() * 0x10001u;
#pragma unroll 1
                        for (int i = 0; i < D / 8; ++i) orow[i] = make_uint4(two, two, two, two);
                    } else {
                        float* prow = p.partials + (((size_t)blockIdx.x * 2 + (it.gi == lo ? 0 : 1)) * Tr::ROWS + row_of_group) * Tr::PSTRIDE;
                        prow[D] = 0.f;
                        prow[D + 1] = qnan;
                    }
                }
                seg_advance(it, len, p, tab);
            }
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
