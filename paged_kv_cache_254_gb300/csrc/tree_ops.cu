// Bookkeeping of a tree of drafted tokens around the attention call: which
// path of each tree the target model agrees with, and moving that path's keys
// and values to consecutive positions of the cache.
#include "tree_ops.cuh"

#include "launch.cuh"
#include "../../include/pa.h"

namespace pa {

// One warp per sequence; lane l holds nodes l and l + 32 of its tree.
//
//   parent(i)   = highest node below i on i's way (bits of masks[i])
//   match(i)    = draft[i] == target[parent(i)]
//   ok(i)       = i is 0, or match(i) and no lower node with i's parent matches
//   accepted(i) = ok(i) and every node below i on i's way is ok
//
// "Lowest matching child" needs the nodes that share a parent: lanes with equal
// parents find one another with match_any, and the upper 32 nodes ask a bit set
// of the parents that the lower 32 already matched.  With the ok nodes as a
// 64-bit set, accepted(i) is one AND and the path comes out of a population
// count, so the depth of the tree costs nothing.  Bound by the latency of three
// dependent loads (chunk start; mask and tokens; the parent's target).
__global__ void __launch_bounds__(128)
pa_tree_verify_kernel(const VerifyArgs a) {
    const int lane = threadIdx.x & 31;
    const long long b = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (b >= a.N) return;
    const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1), ctx = __ldg(a.context_lens + b);
    const long long len = (long long)q1 - q0;
    const bool bad = q0 < 0 || q1 > a.total_q || len < 0 || len > a.P || ctx < 0 || len > ctx;
    if (bad && lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_CONTEXT);
    const int n = bad ? 0 : (int)len;
    uint64_t below[2];
    int parent[2];
    bool match[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        below[h] = 0;
        parent[h] = -1;
        match[h] = false;
        if (i < n) {
            below[h] = __ldg(a.masks + q0 + i) & ((1ull << i) - 1);
            parent[h] = 63 - __clzll((long long)below[h]);      // -1: no bit
            if (parent[h] >= 0) match[h] = __ldg(a.draft + q0 + i) == __ldg(a.target + q0 + parent[h]);
        }
    }
    const uint32_t all = 0xffffffffu;
    auto lowest = [&](bool m, int p) -> bool {                  // lowest lane with this parent among the matched
        const unsigned peers = __match_any_sync(all, m ? p : -1 - lane);
        return m && lane == __ffs((int)peers) - 1;
    };
    auto spread = [&](bool x, int p, int half) -> unsigned {    // bits 32 half .. of the set of p
        return __reduce_or_sync(all, x && (p >> 5) == half ? 1u << (p & 31) : 0u);
    };
    const bool first_lo = lowest(match[0], parent[0]);
    const uint64_t taken = (uint64_t)spread(match[0], parent[0], 0);    // parents of nodes < 32 are < 32
    const bool first_hi = lowest(match[1] && !((taken >> (parent[1] & 63)) & 1), parent[1]);
    const bool ok0 = (lane == 0 && n > 0) || first_lo;
    const uint64_t ok = (uint64_t)__ballot_sync(all, ok0) | ((uint64_t)__ballot_sync(all, first_hi) << 32);
    const uint64_t acc = (uint64_t)__ballot_sync(all, ok0 && (below[0] & ~ok) == 0) |
                         ((uint64_t)__ballot_sync(all, first_hi && (below[1] & ~ok) == 0) << 32);
    const int count = __popcll((long long)acc);
    int32_t* path = a.path + b * a.P;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        if ((acc >> i) & 1) path[__popcll((long long)(acc & ((1ull << i) - 1)))] = i;
        if (i >= count && i < a.P) path[i] = -1;
    }
    if (lane == 0) {
        a.accepted[b] = count;
        a.next[b] = count > 0 ? __ldg(a.target + q0 + 63 - __clzll((long long)acc)) : -1;
        a.new_lens[b] = ctx - n + count;
    }
}

// Keeps the path's rows: position base + path[d] moves to base + d.  Paths
// ascend strictly, so path[d] >= d: a thread that owns one 16-byte column of
// every row and walks d upwards never reads a row it has written, and needs no
// exchange with any other thread.  KEEP_AHEAD rows are loaded before the first
// of them is stored.  A CTA serves one sequence; its first warp checks the path
// and turns it into row offsets.  Bound by the latency of table, row and store
// for small batches, by HBM traffic (each kept row read and written) for large.
constexpr int KEEP_AHEAD = 8;

__global__ void __launch_bounds__(256)
pa_keep_kernel(const KeepArgs a, int ctas_per_seq) {
    __shared__ long long src[64], dst[64];          // row offsets (16-byte vectors) at KV head 0
    __shared__ int moves;
    const long long b = blockIdx.x / ctas_per_seq;
    const int part = (int)(blockIdx.x % ctas_per_seq);
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const uint32_t all = 0xffffffffu;
        const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1), ctx = __ldg(a.context_lens + b);
        const long long len = (long long)q1 - q0;
        const bool bad_seq = len < 0 || len > a.P || ctx < 0 || ctx > (long long)a.MB * a.BS || len > ctx;
        const int n = bad_seq ? 0 : (int)len, base = ctx - n;
        int p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) p[h] = lane + 32 * h < a.P ? __ldg(a.path + b * a.P + lane + 32 * h) : -1;
        const uint64_t ends = (uint64_t)__ballot_sync(all, p[0] == -1) | ((uint64_t)__ballot_sync(all, p[1] == -1) << 32);
        const int count = ends ? __ffsll((long long)ends) - 1 : 64;
        const int last_lo = __shfl_sync(all, p[0], 31);
        int prev[2] = {__shfl_up_sync(all, p[0], 1), __shfl_up_sync(all, p[1], 1)};
        if (lane == 0) {
            prev[0] = -1;
            prev[1] = last_lo;
        }
        bool bad_path = false, bad_block = false;
        bool moved[2];
        long long so[2], to[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d = lane + 32 * h;
            moved[h] = false;
            if (d >= count) continue;
            if (p[h] <= prev[h] || p[h] >= n) {
                bad_path = true;
                continue;
            }
            if (p[h] == d) continue;                // already in place
            moved[h] = true;
            const int s = base + p[h], t = base + d;
            const int sb = __ldg(a.block_tables + b * a.MB + s / a.BS), tb = __ldg(a.block_tables + b * a.MB + t / a.BS);
            if ((unsigned)sb >= (unsigned)a.NB || (unsigned)tb >= (unsigned)a.NB) bad_block = true;
            so[h] = ((long long)sb * a.Hkv * a.BS + s % a.BS) * a.vec_per_row;
            to[h] = ((long long)tb * a.Hkv * a.BS + t % a.BS) * a.vec_per_row;
        }
        bad_path = __any_sync(all, bad_path);
        bad_block = __any_sync(all, bad_block);
        if (part == 0 && lane == 0 && a.err) {
            const uint32_t e = (bad_seq ? PA_DEVERR_CONTEXT : 0u) | (bad_path && !bad_seq ? PA_DEVERR_PATH : 0u) |
                               (bad_block && !bad_path && !bad_seq ? PA_DEVERR_BLOCK_ID : 0u);
            if (e) atomicOr(a.err, e);
        }
        const bool go = !bad_seq && !bad_path && !bad_block;
        const uint64_t set = (uint64_t)__ballot_sync(all, go && moved[0]) | ((uint64_t)__ballot_sync(all, go && moved[1]) << 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d = lane + 32 * h;
            if (go && moved[h]) {
                const int at = __popcll((long long)(set & ((1ull << d) - 1)));
                src[at] = so[h];
                dst[at] = to[h];
            }
        }
        if (lane == 0) moves = __popcll((long long)set);
    }
    __syncthreads();
    const int m = moves;
    const int cols = a.Hkv * a.vec_per_row;
    const int item = part * 256 + (int)threadIdx.x;
    if (m == 0 || item >= 2 * cols) return;
    const int col = item < cols ? item : item - cols;
    uint4* pool = (item < cols ? a.k_pool : a.v_pool) +
                  (long long)(col / a.vec_per_row) * a.BS * a.vec_per_row + col % a.vec_per_row;
    for (int d = 0; d < m; d += KEEP_AHEAD) {
        uint4 x[KEEP_AHEAD];
#pragma unroll
        for (int i = 0; i < KEEP_AHEAD; ++i)
            if (d + i < m) x[i] = pool[src[d + i]];
#pragma unroll
        for (int i = 0; i < KEEP_AHEAD; ++i)
            if (d + i < m) pool[dst[d + i]] = x[i];
    }
}

cudaError_t tree_verify_launch(const VerifyArgs& a, cudaStream_t stream) {
    return launch(pa_tree_verify_kernel, (unsigned)(((long long)a.N + 3) / 4), 128, 0, stream, a);
}

cudaError_t keep_launch(const KeepArgs& a, cudaStream_t stream) {
    const int per_seq = (2 * a.Hkv * a.vec_per_row + 255) / 256;
    const long long blocks = (long long)a.N * per_seq;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch(pa_keep_kernel, (unsigned)blocks, 256, 0, stream, a, per_seq);
}

}  // namespace pa
