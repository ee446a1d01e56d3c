// Writes of the 8-bit cache with a scale for each block and KV head: appending new
// tokens, and whole blocks from and to a 16-bit cache.
//
// Mathematics, per (block, KV head) and for keys and values apart, with F the format's
// largest value (448 or 57344): the scale that values x need is 2^e, e >= -126 the
// smallest with max |x| <= F 2^e over the finite x.  New tokens raise the block's scale s
// to s' = max(s, 2^e) (s = 0 when they start the block); if it rose, older codes c become
// round(c * (s / s')), and new codes are round(x / s') (to nearest, ties to even; an
// infinity becomes the largest code, NaN stays).  A power of two keeps every quotient
// exact, so a code is one rounding of its value and older codes change by shifts of the
// exponent alone (they lose bits only below the format's normal range), and a float code
// is as precise under any of them.
//
// One warp per (block, KV head, keys or values): it holds the block's new rows in
// registers as they came (16 bits), so they are read once, their largest value is
// known before any is rounded, and no other warp touches the rows.  The pool's bytes
// that no new token falls in are read only when the scale rises.
//
// Bound by HBM where there is enough to do.  Measured on GB300, heads of 128 in blocks of 16: packing 4096
// blocks of 8 heads 58 us (6.9 TB/s); 16 prompts of up to 2047 tokens 21.5 to 23.1 us a call (4.4 to 4.7 TB/s: launch,
// one wave of loads, and half the warps without a block because lengths differ); one token of 256
// sequences 7 us, four loads that wait on one another.  777 blocks of 32 tokens and 8 heads of 64 are
// unpacked in 12 us.  Registers are held to four blocks of threads per SM: the prompts took 32 us at two,
// with nothing spilled.
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "bs8.cuh"
#include "bs8_ops.cuh"
#include "decode_common.cuh"
#include "launch.cuh"
#include "packed.cuh"

namespace pa {

namespace {

constexpr int WARPS = 8;

template <int D, int BS, bool BF16, bool E5M2>
struct Rows {
    static constexpr int LPR = D / 8;            // lanes of a row, 8 values each
    static constexpr int RPI = 32 / LPR;         // rows a warp loads at once
    static constexpr int NL = BS / RPI;          // loads of a whole block
    static constexpr int TOP = E5M2 ? 15 : 8;    // F = 1.75 * 2^TOP
    // blocks of threads that an SM holds at least: as many rows in flight as the registers allow
    static constexpr int OCC = NL <= 4 ? 6 : NL <= 8 ? 4 : 2;

    // The exponent of the scale that values up to `top` need.
    static __device__ __forceinline__ int need(float top) {
        const uint32_t b = __float_as_uint(top);
        const int e = (int)(b >> 23) - 127 - TOP + ((b & 0x7fffffu) > 0x600000u);
        return max(e, -126);
    }
    static __device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

    // The largest finite absolute value of the rows that a warp holds.
    static __device__ __forceinline__ float top(const uint4 (&x)[NL]) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
        }
        if (__any_sync(0xffffffffu, pair_not_finite<BF16>(m) != 0)) {   // rare: once more, without them
            m = 0;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = w[j] & 0x7fff7fffu, bad = pair_not_finite<BF16>(a);
                    m = __vmaxu2(m, a & ((bad & 0x8000u ? 0u : 0xffffu) | (bad & 0x80000000u ? 0u : 0xffff0000u)));
                }
            }
        }
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        return widen16<BF16>(m);
    }

    // Eight 16-bit values times a power of two, as codes.
    static __device__ __forceinline__ uint2 codes(const uint4& x, float inv) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const f32x2 by = pair2(inv, inv);
        uint16_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            split2(mul2(pair2(lo_of<BF16>(w[j]), hi_of<BF16>(w[j])), by), a, b);
            c[j] = f32x2_to_fp8x2<E5M2>(a, b);
        }
        uint2 r;
        asm("mov.b32 %0, {%1, %2};" : "=r"(r.x) : "h"(c[0]), "h"(c[1]));
        asm("mov.b32 %0, {%1, %2};" : "=r"(r.y) : "h"(c[2]), "h"(c[3]));
        return r;
    }

    // The same by a division, for scales that are no power of two.
    static __device__ __forceinline__ uint2 quotients(const uint4& x, float s) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = f32x2_to_fp8x2<E5M2>(__fdiv_rn(lo_of<BF16>(w[j]), s), __fdiv_rn(hi_of<BF16>(w[j]), s));
        return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }

    // Codes [lo half, hi half] -> codes of the values times `ratio`.
    static __device__ __forceinline__ uint32_t scaled(uint32_t c, float ratio) {
        const uint32_t a = fp8x2_to_f16x2<E5M2>((uint16_t)(c & 0xffffu)), b = fp8x2_to_f16x2<E5M2>((uint16_t)(c >> 16));
        return (uint32_t)f32x2_to_fp8x2<E5M2>(lo_of<false>(a) * ratio, hi_of<false>(a) * ratio) |
               ((uint32_t)f32x2_to_fp8x2<E5M2>(lo_of<false>(b) * ratio, hi_of<false>(b) * ratio) << 16);
    }

    // Where 8 codes from dimension 8 * sub of row r stand in the piece.
    static __device__ __forceinline__ int place(int op, int r, int sub) {
        // bs8_value and bs8_key in one form: which bits of r permute the parts is all that differs
        const int sh = op ? 2 : 0, mask = D == 128 ? (op ? 6 : 7) : (op ? 2 : 0);
        const int row = D == 64 && BS == 32 ? r ^ (op ? (r >> 4) & 1 : 0) : r;
        return BS8_HEAD + (op ? BS * D : 0) + row * D + (((sub >> 1) ^ ((r >> sh) & mask)) << 4) + 8 * (sub & 1);
    }
};

template <int D, int BS, bool BF16, bool E5M2>
__global__ void __launch_bounds__(32 * WARPS, Rows<D, BS, BF16, E5M2>::OCC) pa_append_bs8_kernel(const AppendBs8Args a) {
    using R = Rows<D, BS, BF16, E5M2>;
    const int lane = threadIdx.x & 31, sub = lane % R::LPR, rr = lane / R::LPR;
    // warps: (sequence, block of its span, KV head, keys or values), the last fastest, so
    // that neighbours read one token's heads
    const uint32_t w = blockIdx.x * WARPS + (threadIdx.x >> 5), per = 2 * a.Hkv, unit = w / per;
    const int s = (int)(unit / a.span), j = (int)(unit % a.span), h = (int)(w % per) >> 1, op = (int)(w & 1);
    if (s >= a.N) return;
    const int q0 = __ldg(a.q_start + s), q1 = __ldg(a.q_start + s + 1), ctx = __ldg(a.context_lens + s);
    const long long n = (long long)q1 - q0;
    if (q0 < 0 || q1 > a.T || n < 0 || n > a.max_new || ctx < 0 || n > ctx || ctx > a.MB * BS) {
        if (j == 0 && h == 0 && op == 0 && lane == 0) set_err(a.err, PA_DEVERR_CONTEXT);
        return;
    }
    const int from = ctx - (int)n;                       // first new position
    const int b = from / BS + j;                         // logical block
    if (n == 0 || b > (ctx - 1) / BS) return;
    const int lo = max(0, from - b * BS), hi = min(BS, ctx - b * BS);   // the block's new rows
    const int id = __ldg(a.block_tables + (size_t)s * a.MB + b);
    const int64_t stride = op ? a.v_stride : a.k_stride;
    const uint16_t* src = (op ? a.v : a.k) + (int64_t)(q0 + b * BS + lo - from) * stride + h * D + 8 * sub;
    uint4 x[R::NL];
#pragma unroll
    for (int i = 0; i < R::NL; ++i) {
        const int r = i * R::RPI + rr;                   // of the new rows
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < hi - lo) x[i] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * stride));
    }
    if ((unsigned)id >= (unsigned)a.NB) {
        if (lane == 0) set_err(a.err, PA_DEVERR_BLOCK_ID);
        return;
    }
    uint8_t* piece = a.pool + ((size_t)id * a.Hkv + h) * bs8_piece_bytes(BS, D);
    float* scale_at = reinterpret_cast<float*>(piece) + op;
    const float old = lo > 0 ? *scale_at : 0.f;
    if (!bs8_is_scale(old)) {
        if (lane == 0) set_err(a.err, PA_DEVERR_SCALE);
        return;
    }
    const int e = R::need(R::top(x));
    const float need = R::pow2(e);
    const bool rises = need > old;
    const float now = rises ? need : old;
    if (rises) {
        const float ratio = __fdiv_rn(old, need);
        for (int r0 = rr; r0 < lo; r0 += 4 * R::RPI) {   // older rows, four loads in flight
            uint2 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r0 + k * R::RPI < lo) c[k] = *reinterpret_cast<const uint2*>(piece + R::place(op, r0 + k * R::RPI, sub));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r0 + k * R::RPI < lo)
                    *reinterpret_cast<uint2*>(piece + R::place(op, r0 + k * R::RPI, sub)) =
                        make_uint2(R::scaled(c[k].x, ratio), R::scaled(c[k].y, ratio));
        }
        if (lane == 0) *scale_at = now;
    }
    // a power of two from 2^-126 (what `need` is at least) to 2^126: its reciprocal is a normal number
    const uint32_t bits = __float_as_uint(now);
    const bool exact = (bits & 0x7fffffu) == 0 && bits < 0x7f000000u;
    const float inv = __uint_as_float(0x7f000000u - bits);
    auto put = [&](int i, uint2 c) {
        const int r = i * R::RPI + rr;
        if (r < hi - lo) *reinterpret_cast<uint2*>(piece + R::place(op, lo + r, sub)) = c;
    };
    if (exact) {
#pragma unroll
        for (int i = 0; i < R::NL; ++i) put(i, R::codes(x[i], inv));
    } else {
#pragma unroll
        for (int i = 0; i < R::NL; ++i) put(i, R::quotients(x[i], now));
    }
}

// One warp per (pair, KV head, keys or values), as the append of a whole block.
template <int D, int BS, bool BF16, bool E5M2>
__global__ void __launch_bounds__(32 * WARPS, Rows<D, BS, BF16, E5M2>::OCC) pa_pack_bs8_kernel(const ConvertBs8Args a) {
    using R = Rows<D, BS, BF16, E5M2>;
    const int lane = threadIdx.x & 31, sub = lane % R::LPR, rr = lane / R::LPR;
    const uint32_t w = blockIdx.x * WARPS + (threadIdx.x >> 5), per = 2 * a.Hkv, i0 = w / per;
    if (i0 >= (uint32_t)a.n) return;
    const int op = (int)(w % per) / a.Hkv, h = (int)(w % per) % a.Hkv;
    const int from = __ldg(a.pairs + 2 * (size_t)i0), to = __ldg(a.pairs + 2 * (size_t)i0 + 1);
    if ((unsigned)from >= (unsigned)a.NB16 || (unsigned)to >= (unsigned)a.NB8) {
        if (lane == 0) set_err(a.err, PA_DEVERR_COPY_PAIR);
        return;
    }
    const uint16_t* src = (op ? a.v : a.k) + ((size_t)from * a.Hkv + h) * BS * D + rr * D + 8 * sub;
    uint4 x[R::NL];
#pragma unroll
    for (int i = 0; i < R::NL; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src + i * R::RPI * D));
    uint8_t* piece = a.pool + ((size_t)to * a.Hkv + h) * bs8_piece_bytes(BS, D);
    const int e = R::need(R::top(x));
    if (lane == 0) reinterpret_cast<float*>(piece)[op] = R::pow2(e);
    const float inv = R::pow2(-e);
#pragma unroll
    for (int i = 0; i < R::NL; ++i)
        *reinterpret_cast<uint2*>(piece + R::place(op, i * R::RPI + rr, sub)) = R::codes(x[i], inv);
}

template <int D, int BS, bool BF16, bool E5M2>
__global__ void __launch_bounds__(32 * WARPS) pa_unpack_bs8_kernel(const ConvertBs8Args a) {
    using R = Rows<D, BS, BF16, E5M2>;
    const int lane = threadIdx.x & 31, sub = lane % R::LPR, rr = lane / R::LPR;
    const uint32_t w = blockIdx.x * WARPS + (threadIdx.x >> 5), per = 2 * a.Hkv, i0 = w / per;
    if (i0 >= (uint32_t)a.n) return;
    const int op = (int)(w % per) / a.Hkv, h = (int)(w % per) % a.Hkv;
    const int from = __ldg(a.pairs + 2 * (size_t)i0), to = __ldg(a.pairs + 2 * (size_t)i0 + 1);
    if ((unsigned)from >= (unsigned)a.NB8 || (unsigned)to >= (unsigned)a.NB16) {
        if (lane == 0) set_err(a.err, PA_DEVERR_COPY_PAIR);
        return;
    }
    const uint8_t* piece = a.pool + ((size_t)from * a.Hkv + h) * bs8_piece_bytes(BS, D);
    const float s = __ldg(reinterpret_cast<const float*>(piece) + op);
    uint2 c[R::NL];
#pragma unroll
    for (int i = 0; i < R::NL; ++i)
        c[i] = __ldg(reinterpret_cast<const uint2*>(piece + R::place(op, i * R::RPI + rr, sub)));
    if (!bs8_is_scale(s) && lane == 0) set_err(a.err, PA_DEVERR_SCALE);   // and the values are NaN
    const float f = bs8_is_scale(s) ? s : __int_as_float(0x7fc00000);
    uint16_t* dst = (op ? a.v : a.k) + ((size_t)to * a.Hkv + h) * BS * D + rr * D + 8 * sub;
#pragma unroll
    for (int i = 0; i < R::NL; ++i) {
        const uint32_t w4[4] = {c[i].x & 0xffffu, c[i].x >> 16, c[i].y & 0xffffu, c[i].y >> 16};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = fp8x2_to_f16x2<E5M2>((uint16_t)w4[j]);
            y[j] = pack2<BF16>(lo_of<false>(v) * f, hi_of<false>(v) * f);
        }
        *reinterpret_cast<uint4*>(dst + i * R::RPI * D) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

// f(D, BS, BF16, E5M2 as types) for the kind's values.
template <class F>
cudaError_t by_kind(Bs8Kind k, F f) {
    auto fmt = [&](auto d, auto bs, auto bf) {
        return k.e5m2 ? f(d, bs, bf, std::true_type{}) : f(d, bs, bf, std::false_type{});
    };
    auto type = [&](auto d, auto bs) { return k.bf16 ? fmt(d, bs, std::true_type{}) : fmt(d, bs, std::false_type{}); };
    auto block = [&](auto d) {
        return k.bs32 ? type(d, std::integral_constant<int, 32>{}) : type(d, std::integral_constant<int, 16>{});
    };
    return k.d128 ? block(std::integral_constant<int, 128>{}) : block(std::integral_constant<int, 64>{});
}

}  // namespace

cudaError_t append_bs8_launch(const AppendBs8Args& a, Bs8Kind kind, cudaStream_t stream) {
    const long long warps = (long long)a.N * a.span * 2 * a.Hkv;
    return by_kind(kind, [&](auto d, auto bs, auto bf, auto e5) {
        return launch(pa_append_bs8_kernel<d(), bs(), bf(), e5()>, (unsigned)((warps + WARPS - 1) / WARPS), 32 * WARPS, 0,
                      stream, a);
    });
}

cudaError_t pack_bs8_launch(const ConvertBs8Args& a, Bs8Kind kind, cudaStream_t stream) {
    const long long warps = (long long)a.n * 2 * a.Hkv;
    return by_kind(kind, [&](auto d, auto bs, auto bf, auto e5) {
        return launch(pa_pack_bs8_kernel<d(), bs(), bf(), e5()>, (unsigned)((warps + WARPS - 1) / WARPS), 32 * WARPS, 0,
                      stream, a);
    });
}

cudaError_t unpack_bs8_launch(const ConvertBs8Args& a, Bs8Kind kind, cudaStream_t stream) {
    const long long warps = (long long)a.n * 2 * a.Hkv;
    return by_kind(kind, [&](auto d, auto bs, auto bf, auto e5) {
        return launch(pa_unpack_bs8_kernel<d(), bs(), bf(), e5()>, (unsigned)((warps + WARPS - 1) / WARPS), 32 * WARPS, 0,
                      stream, a);
    });
}

}  // namespace pa
