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
// fraction of a turn exactly (whole turns fall off the top; a negative p works
// alike), with an error below p * 2^-64 turns.  Its top 32 bits go to
// sincospif.  u_j comes from the fp32 frequency's mantissa times 1 / 2 pi in
// integer arithmetic: no fp64 (2 operations per clock and SM here).
//
// What bounds it: HBM (every value is read once and written once).  A row of D
// values is held by D / 16 lanes, 16 values each in two 16-byte vectors that
// hold both halves of the lane's eight pairs, so the rotation needs no shuffle
// and a lane's eight (cos, sin) serve every head of its token.  A warp takes a
// token's rows (queries, keys, values) 32 / LPR at a time, two such steps in
// flight; few tokens are split over several warps each.
#include "rope_ops.cuh"

#include <cuda_fp16.h>

#include "decode_common.cuh"
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

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = lo_of<BF16>(u[i]);
        x[2 * i + 1] = hi_of<BF16>(u[i]);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
    return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                      pack2<BF16>(x[6], x[7]));
}

template <bool BF16, int LPR>
__global__ void __launch_bounds__(256)
pa_rope_append_kernel(const RopeArgs a) {
    constexpr int RPS = 32 / LPR;                       // rows per step
    constexpr int U = 2;                                // steps in flight
    const int lane = threadIdx.x & 31;
    const int c = lane % LPR, sub = lane / LPR;
    const bool active = 16 * c < a.D;
    const bool turns = 16 * c < a.rot;
    // the lane's two vectors of a row: both halves of its pairs
    const bool halves = turns && !a.interleaved;
    const int oa = halves ? 8 * c : 16 * c, ob = halves ? a.rot / 2 + 8 * c : 16 * c + 8;
    uint64_t freq[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) freq[e] = turns ? turns_per_position(__ldg(a.inv_freq + 8 * c + e)) : 0;
    const bool norm = a.q_weight || a.k_weight;
    uint4 wq[2], wk[2];
    auto vec = [](const uint16_t* p) -> const uint4* { return reinterpret_cast<const uint4*>(p); };
    if (a.q_weight && active) {
        wq[0] = __ldg(vec(a.q_weight + oa));
        wq[1] = __ldg(vec(a.q_weight + ob));
    }
    if (a.k_weight && active) {
        wk[0] = __ldg(vec(a.k_weight + oa));
        wk[1] = __ldg(vec(a.k_weight + ob));
    }
    const int R = a.Hq + 2 * a.Hkv;
    const int steps = (R + RPS - 1) / RPS;
    const int per = (steps + a.splits - 1) / a.splits;  // steps of one warp
    const long long units = (long long)a.T * a.splits;
    const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
    for (long long un = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; un < units; un += nwarps) {
        const long long t = un / a.splits;
        const int sp = (int)(un - t * a.splits);
        const int s0 = sp * per, s1 = min(steps, s0 + per);
        const uint64_t pos = (uint64_t)(int64_t)__ldg(a.positions + t);
        const long long slot = __ldg(a.slots + t);
        const bool cached = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && sp == 0 && lane == 0 && a.err) atomicOr(a.err, PA_DEVERR_SLOT);
        const uint32_t blk = cached ? (uint32_t)slot / (uint32_t)a.BS : 0u;
        const uint32_t off = cached ? (uint32_t)slot - blk * (uint32_t)a.BS : 0u;
        float cs[8], sn[8];
        if (turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // signed fraction of a turn, in half turns: [-1, 1)
                const float h = (float)(int32_t)(uint32_t)((pos * freq[e]) >> 32) * 0x1p-31f;
                sincospif(h, &sn[e], &cs[e]);
                sn[e] *= a.scale;
                cs[e] *= a.scale;
            }
        }
        for (int s = s0; s < s1; s += U) {
            uint4 va[U], vb[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = (s + i) * RPS + sub;
                va[i] = vb[i] = make_uint4(0u, 0u, 0u, 0u);
                if (active && s + i < s1 && r < R) {
                    const uint16_t* src = r < a.Hq            ? a.q + t * a.q_stride + (long long)r * a.D
                                          : r < a.Hq + a.Hkv ? a.k + t * a.k_stride + (long long)(r - a.Hq) * a.D
                                                             : a.v + t * a.v_stride + (long long)(r - a.Hq - a.Hkv) * a.D;
                    va[i] = *vec(src + oa);
                    vb[i] = *vec(src + ob);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = (s + i) * RPS + sub;
                const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
                float x[8], y[8];
                widen8<BF16>(va[i], x);
                widen8<BF16>(vb[i], y);
                if (norm) {                              // the row's lanes add up its squares (all lanes take part)
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (!is_v && (is_q ? a.q_weight : a.k_weight)) {
                        const float inv = rsqrtf(ss / (float)a.D + a.eps);
                        float w[8], z[8];
                        widen8<BF16>(is_q ? wq[0] : wk[0], w);
                        widen8<BF16>(is_q ? wq[1] : wk[1], z);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] = x[e] * inv * w[e];
                            y[e] = y[e] * inv * z[e];
                        }
                    }
                }
                if (!active || s + i >= s1 || r >= R) continue;
                if (!is_v) {
                    if (turns) {
                        if (a.interleaved) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
                                x[2 * e] = x0 * cs[e] - x1 * sn[e];
                                x[2 * e + 1] = x1 * cs[e] + x0 * sn[e];
                                y[2 * e] = y0 * cs[4 + e] - y1 * sn[4 + e];
                                y[2 * e + 1] = y1 * cs[4 + e] + y0 * sn[4 + e];
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float x0 = x[e], y0 = y[e];
                                x[e] = x0 * cs[e] - y0 * sn[e];
                                y[e] = y0 * cs[e] + x0 * sn[e];
                            }
                        }
                    }
                    va[i] = narrow8<BF16>(x);
                    vb[i] = narrow8<BF16>(y);
                }
                uint16_t* dst;
                if (is_q) {
                    dst = a.q_out + (t * a.Hq + r) * a.D;
                } else {
                    if (!cached) continue;
                    const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
                    dst = (is_v ? a.v_pool : a.k_pool) + (((long long)blk * a.Hkv + h) * a.BS + off) * a.D;
                }
                *reinterpret_cast<uint4*>(dst + oa) = va[i];
                *reinterpret_cast<uint4*>(dst + ob) = vb[i];
            }
        }
    }
}

cudaError_t rope_append_launch(RopeArgs a, bool bf16, cudaStream_t stream, int sms) {
    int lpr = 1;
    while (16 * lpr < a.D) lpr *= 2;
    const int rps = 32 / lpr;
    const int steps = (a.Hq + 2 * a.Hkv + rps - 1) / rps;
    // enough warps to fill the device (32 per SM) while there are rows to share
    const long long want = ((long long)sms * 32 + a.T - 1) / a.T;
    a.splits = (int)(want < steps ? want : steps);
    long long blocks = ((long long)a.T * a.splits + 7) / 8;
    const long long cap = (long long)sms * 8;
    if (blocks > cap) blocks = cap;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, 256, 0, stream>>>(a);
        return cudaGetLastError();
    };
    switch (lpr) {
        case 1: return bf16 ? go(pa_rope_append_kernel<true, 1>) : go(pa_rope_append_kernel<false, 1>);
        case 2: return bf16 ? go(pa_rope_append_kernel<true, 2>) : go(pa_rope_append_kernel<false, 2>);
        case 4: return bf16 ? go(pa_rope_append_kernel<true, 4>) : go(pa_rope_append_kernel<false, 4>);
        case 8: return bf16 ? go(pa_rope_append_kernel<true, 8>) : go(pa_rope_append_kernel<false, 8>);
        default: return bf16 ? go(pa_rope_append_kernel<true, 16>) : go(pa_rope_append_kernel<false, 16>);
    }
}

}  // namespace pa
