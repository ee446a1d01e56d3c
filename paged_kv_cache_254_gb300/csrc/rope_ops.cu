// Per-head RMS norm, rotary positions and the append of new tokens to the
// paged cache, in one pass over the projection's output.
//
// Mathematics, per token t at position p and per head row x of D values:
//   norm (optional)   y = x / sqrt(mean(x^2) + eps) * w
//   rotation          (a, b) -> (a c - b s, b c + a s) for each pair j < rot / 2,
//                     c = scale cos(p f_j), s = scale sin(p f_j);
//                     pairs (j, j + rot / 2), or (2j, 2j + 1) when interleaved;
//                     values from rot on pass through
// for queries (to q_out) and keys (to the pool); values go to the pool as they
// are.  Everything is fp32 and rounded once, to the 16-bit type.
//
// Angles.  p f_j reaches 10^6 radians and more, where an fp32 product keeps no
// digit of the turn.  Here the frequency is held as turns per position in
// 64-bit fixed point, u_j = frac(f_j / 2 pi) * 2^64: p * u_j modulo 2^64 is the
// fraction of a turn (whole turns fall off the top; a negative p works alike) with
// an error below p * 2^-64 turns.  Its top 32 bits, as one fp32 number of half turns
// (rounded by up to 2^-25), go to sincospif.  u_j comes from the fp32 frequency's mantissa times 1 / 2 pi in
// integer arithmetic: no fp64 (2 operations per clock and SM here).  An infinite or
// NaN frequency has no such number: its pairs' cosines and sines are NaN.
//
// What bounds it: HBM at first (every value is read once and written once), then
// the instructions around it.  A row of D values is held by D / 16 lanes, 16
// values each in two 16-byte vectors that hold both halves of the lane's eight
// pairs, so the rotation needs no shuffle.  A warp computes its token's angles
// once, one per lane, and walks the token's rows (queries, keys, values end to
// end) in groups of 2 * 32 / LPR, all branch-free inside so that the two rows a
// lane works on hide one another's latencies, in packed fp32 pairs; the next
// group's loads, the next token's too, are under way meanwhile.  Few tokens are
// split over several warps each.
//
// Measured: 8192 tokens of 64 / 8 heads, d 128, norm and rotation: 62 us, 0.80 of
// the copy bandwidth on 336 MB (first version, angles per lane and loads per
// step: 95 us; angles shared and loads ahead: 64 us).  Asynchronous copies to
// shared memory instead of the registers ahead, 4 to 10 steps deep, were no
// faster (63 us): bytes in flight are not the limit.  One row a lane on three
// CTAs: 73 us; three rows: registers spill.
#include "rope_ops.cuh"

#include <cuda_fp16.h>

#include "decode_common.cuh"
#include "launch.cuh"
#include "packed.cuh"
#include "ptx.cuh"
#include "../../include/pa.h"

namespace pa {

// frac(f / 2 pi) * 2^64.  1 / 2 pi = C * 2^-66; f = m * 2^e with a 24-bit
// integer m, so the fraction is m * C * 2^(e - 2) modulo 2^64.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    constexpr uint64_t C = 0xA2F9836E4E441529ull;   // floor(2^66 / 2 pi)
    const uint32_t bits = __float_as_uint(f);
    const int ex = (int)((bits >> 23) & 0xffu);
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int shift = 152 - (ex ? ex : 1);          // 2 - e
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    uint64_t u;
    if (shift <= 0) {
        u = shift > -64 ? lo << -shift : 0;         // f >= 2^25: whole turns a position
    } else if (shift < 64) {
        u = (lo >> shift) | (hi << (64 - shift));
    } else {
        u = shift < 128 ? hi >> (shift - 64) : 0;
    }
    return (bits >> 31) ? 0ull - u : u;
}

// Eight 16-bit values as four fp32 pairs, and back.
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& w, f32x2 (&x)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair2(lo_of<BF16>(u[i]), hi_of<BF16>(u[i]));
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const f32x2 (&x)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split2(x[i], lo, hi);
        u[i] = pack2<BF16>(lo, hi);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

constexpr int STEPS = 2;                                // of 32 / LPR rows each, worked on side by side
constexpr int MIN_CTAS = 2;
constexpr int WARPS = 8;

template <bool BF16, int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * WARPS, MIN_CTAS)
pa_rope_append_kernel(const RopeArgs a) {
    constexpr int RPS = 32 / LPR;                       // rows per step
    constexpr int U = STEPS;
    constexpr int PAIRS = 8 * LPR;                      // at most, in a row
    __shared__ __align__(16) uint64_t sfreq[PAIRS];
    __shared__ float sscale[PAIRS];                     // of a pair's cosine and sine
    __shared__ __align__(16) float sweight[2][2 * PAIRS];  // of queries and of keys
    __shared__ __align__(16) float2 sturn[WARPS][PAIRS];   // (cos, sin) of the warp's token
    for (int i = threadIdx.x; i < a.rot / 2; i += 32 * WARPS) {
        const float f = __ldg(a.inv_freq + i);
        sfreq[i] = turns_per_position(f);
        sscale[i] = isfinite(f) ? a.scale : __int_as_float(0x7fc00000);
    }
    for (int i = threadIdx.x; i < a.D; i += 32 * WARPS) {
        auto f = [](uint16_t w) -> float { return lo_of<BF16>(w); };
        sweight[0][i] = a.q_weight ? f(__ldg(a.q_weight + i)) : 1.f;
        sweight[1][i] = a.k_weight ? f(__ldg(a.k_weight + i)) : 1.f;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % LPR, sub = lane / LPR;
    const bool active = 16 * c < a.D;
    const bool turns = 16 * c < a.rot;
    // the lane's two vectors of a row: both halves of its pairs
    const bool halves = turns && !INTERLEAVED;
    const int oa = halves ? 8 * c : 16 * c, ob = halves ? a.rot / 2 + 8 * c : 16 * c + 8;
    const float inv_d = 1.f / (float)a.D;
    const bool norm = a.q_weight || a.k_weight;
    // A token's rows, queries first, then keys, then values, in groups of ROWS
    constexpr int ROWS = U * RPS;
    const int end_q = a.Hq, end_k = a.Hq + a.Hkv, end_v = a.Hq + 2 * a.Hkv;
    const int groups = (end_v + ROWS - 1) / ROWS;
    const int per = (groups + a.splits - 1) / a.splits; // groups of one warp
    const long long units = (long long)a.T * a.splits;
    const long long nwarps = (long long)gridDim.x * WARPS;
    auto vec = [](const uint16_t* p) -> const uint4* { return reinterpret_cast<const uint4*>(p); };
    // unit -> token and first group (several warps share a token only when there are few)
    auto token_of = [&](long long un, int& s0) -> int {
        if (a.splits == 1) {
            s0 = 0;
            return (int)un;
        }
        const int t = (int)((uint32_t)un / (uint32_t)a.splits);
        s0 = ((int)un - t * a.splits) * per;
        return t;
    };
    auto fetch = [&](int t, int s, uint4 (&va)[U], uint4 (&vb)[U]) {
        const uint16_t* bq = a.q + t * a.q_stride;
        const uint16_t* bk = a.k + t * a.k_stride - (long long)end_q * a.D;
        const uint16_t* bv = a.v + t * a.v_stride - (long long)end_k * a.D;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = s * ROWS + i * RPS + sub;
            va[i] = vb[i] = make_uint4(0u, 0u, 0u, 0u);
            if (active && r < end_v) {
                const uint16_t* src = (r < end_q ? bq : r < end_k ? bk : bv) + r * a.D;
                va[i] = *vec(src + oa);
                vb[i] = *vec(src + ob);
            }
        }
    };
    long long un = (long long)blockIdx.x * WARPS + warp;
    if (un >= units) return;
    int s, t = token_of(un, s);
    int s1 = min(groups, s + per);
    int pos = __ldg(a.positions + t);
    long long slot = __ldg(a.slots + t);
    uint4 va[U], vb[U];
    fetch(t, s, va, vb);
    bool fresh = true;                                  // the token's angles are still to be computed
    // The lane's cosines and sines.  Halves, pairs (x, y) two by two: x' = x cc - y sa, y' = y cc + x sa.
    // Interleaved, x and y two runs of four pairs: x' = x cc + swapped(x) sa with cc = (c, c),
    // sa = (-s, s); y' the same with cb, sb.
    f32x2 cc[4], sa[4], cb[4], sb[4];
    bool cached = false;                                // the token has a slot,
    uint16_t *kdst = a.k_pool, *vdst = a.v_pool;        // here in the pools, at KV head 0
    while (true) {
        // the next group's rows are on their way while this one is worked on
        long long un2 = un;
        int t2 = t, s2 = s + 1, s1_2 = s1, pos2 = pos;
        long long slot2 = slot;
        if (s2 >= s1) {
            un2 = un + nwarps;
            if (un2 < units) {
                t2 = token_of(un2, s2);
                s1_2 = min(groups, s2 + per);
                pos2 = __ldg(a.positions + t2);
                slot2 = __ldg(a.slots + t2);
            }
        }
        uint4 na[U], nb[U];
        if (un2 < units) fetch(t2, s2, na, nb);
        if (fresh) {
            cached = slot >= 0 && slot < a.num_slots;
            if (slot >= a.num_slots && s == 0 && lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_SLOT);
            if (cached) {
                const uint32_t blk = (uint32_t)slot / (uint32_t)a.BS, off = (uint32_t)slot - blk * (uint32_t)a.BS;
                const long long at = ((long long)blk * a.Hkv * a.BS + off) * a.D;
                kdst = a.k_pool + at;
                vdst = a.v_pool + at;
            }
            __syncwarp();
            for (int j = lane; j < a.rot / 2; j += 32) {
                // signed fraction of a turn, in half turns: [-1, 1)
                const uint64_t turn = (uint64_t)(int64_t)pos * sfreq[j];
                const float h = (float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f;
                float2 w;
                sincospif(h, &w.y, &w.x);
                w.x *= sscale[j];
                w.y *= sscale[j];
                sturn[warp][j] = w;
            }
            __syncwarp();
            if (turns) {
                const float4* cs = reinterpret_cast<const float4*>(sturn[warp] + 8 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = cs[e];             // two pairs' (cos, sin)
                    if (INTERLEAVED) {
                        f32x2* C = e < 2 ? cc : cb;
                        f32x2* S = e < 2 ? sa : sb;
                        C[2 * (e & 1)] = pair2(w.x, w.x);
                        S[2 * (e & 1)] = pair2(-w.y, w.y);
                        C[2 * (e & 1) + 1] = pair2(w.z, w.z);
                        S[2 * (e & 1) + 1] = pair2(-w.w, w.w);
                    } else {
                        cc[e] = pair2(w.x, w.z);
                        sa[e] = pair2(w.y, w.w);
                        sb[e] = pair2(-w.y, -w.w);
                    }
                }
            }
        }
        const int r0 = s * ROWS + sub;                  // the lane's rows: r0 + i * RPS
        if (s * ROWS < end_k) {                         // not values alone
            f32x2 x[U][4], y[U][4];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                widen8<BF16>(va[i], x[i]);
                widen8<BF16>(vb[i], y[i]);
            }
            if (norm) {
                float ss[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    f32x2 p = mul2(x[i][0], x[i][0]), q = mul2(y[i][0], y[i][0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) {
                        p = fma2(x[i][e], x[i][e], p);
                        q = fma2(y[i][e], y[i][e], q);
                    }
                    float p0, p1, q0, q1;
                    split2(p, p0, p1);
                    split2(q, q0, q1);
                    ss[i] = (p0 + p1) + (q0 + q1);
                }
                // the row's lanes add up its squares
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
                    for (int i = 0; i < U; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
                f32x2 inv[U];
                const float4 *wx[U], *wy[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const bool key = r0 + i * RPS >= end_q;
                    float f = rsqrtf(ss[i] * inv_d + a.eps);
                    if (!(key ? a.k_weight : a.q_weight)) f = 1.f;
                    inv[i] = pair2(f, f);
                    wx[i] = reinterpret_cast<const float4*>(sweight[key] + oa);
                    wy[i] = reinterpret_cast<const float4*>(sweight[key] + ob);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const float4 fx = wx[i][e], fy = wy[i][e];
                        x[i][2 * e] = mul2(mul2(x[i][2 * e], inv[i]), pair2(fx.x, fx.y));
                        x[i][2 * e + 1] = mul2(mul2(x[i][2 * e + 1], inv[i]), pair2(fx.z, fx.w));
                        y[i][2 * e] = mul2(mul2(y[i][2 * e], inv[i]), pair2(fy.x, fy.y));
                        y[i][2 * e + 1] = mul2(mul2(y[i][2 * e + 1], inv[i]), pair2(fy.z, fy.w));
                    }
            }
            if (turns) {
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x2 p = x[i][e], q = y[i][e];
                        if (INTERLEAVED) {
                            x[i][e] = fma2(swap2(p), sa[e], mul2(p, cc[e]));
                            y[i][e] = fma2(swap2(q), sb[e], mul2(q, cb[e]));
                        } else {
                            x[i][e] = fma2(q, sb[e], mul2(p, cc[e]));
                            y[i][e] = fma2(p, sa[e], mul2(q, cc[e]));
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (r0 + i * RPS < end_k) {
                    va[i] = narrow8<BF16>(x[i]);
                    vb[i] = narrow8<BF16>(y[i]);
                }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = r0 + i * RPS;
            uint16_t* dst = r < end_q ? a.q_out + ((long long)t * a.Hq + r) * a.D
                                      : (r < end_k ? kdst : vdst) + (long long)(r - (r < end_k ? end_q : end_k)) * a.BS * a.D;
            if (active && r < end_v && (r < end_q || cached)) {
                *reinterpret_cast<uint4*>(dst + oa) = va[i];
                *reinterpret_cast<uint4*>(dst + ob) = vb[i];
            }
        }
        if (un2 >= units) break;
        fresh = un2 != un;
        un = un2;
        t = t2;
        s = s2;
        s1 = s1_2;
        pos = pos2;
        slot = slot2;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            va[i] = na[i];
            vb[i] = nb[i];
        }
    }
}

template <bool BF16, int LPR>
cudaError_t rope_append_run(const RopeArgs& a, unsigned blocks, cudaStream_t stream) {
    return launch(a.interleaved ? pa_rope_append_kernel<BF16, LPR, true> : pa_rope_append_kernel<BF16, LPR, false>,
                  blocks, 32 * WARPS, 0, stream, a);
}

cudaError_t rope_append_launch(RopeArgs a, bool bf16, cudaStream_t stream, int sms) {
    int lpr = 1;
    while (16 * lpr < a.D) lpr *= 2;
    const int rows = STEPS * 32 / lpr;
    const int steps = (a.Hq + 2 * a.Hkv + rows - 1) / rows;
    // enough warps to fill the device (32 per SM) while there are rows to share
    const long long want = ((long long)sms * 32 + a.T - 1) / a.T;
    a.splits = (int)(want < steps ? want : steps);
    long long blocks = ((long long)a.T * a.splits + WARPS - 1) / WARPS;
    const long long cap = (long long)sms * MIN_CTAS;
    if (blocks > cap) blocks = cap;
    const unsigned n = (unsigned)blocks;
    switch (lpr) {
        case 1: return bf16 ? rope_append_run<true, 1>(a, n, stream) : rope_append_run<false, 1>(a, n, stream);
        case 2: return bf16 ? rope_append_run<true, 2>(a, n, stream) : rope_append_run<false, 2>(a, n, stream);
        case 4: return bf16 ? rope_append_run<true, 4>(a, n, stream) : rope_append_run<false, 4>(a, n, stream);
        case 8: return bf16 ? rope_append_run<true, 8>(a, n, stream) : rope_append_run<false, 8>(a, n, stream);
        default: return bf16 ? rope_append_run<true, 16>(a, n, stream) : rope_append_run<false, 16>(a, n, stream);
    }
}

}  // namespace pa
