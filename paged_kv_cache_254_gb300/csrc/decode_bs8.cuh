// The per-stage update of the 8-bit cache with a scale for each block and KV head
// (layout: bs8.cuh), with the stage's tokens as the MMA rows as in decode_tok.cuh.
//
// Mathematics.  With codes kc, vc and the block's scales a (keys) and b (values),
//     s_t = scale a <q, kc_t>,   out = sum_t e^(s_t) b vc_t / sum_t e^(s_t).
// b is taken into the exponent: in log2 units x_t = s_t + lb with lb = log2 b, weights
// w_t = 2^(x_t - m) with m the running maximum of x_t, so sums are
//     O = sum_t w_t vc_t,   l = sum_t w_t 2^-lb,   out = O / l,
// at the cost of two multiply-adds per score in place of a multiplication and an
// addition.  Weights are at most 1, and precise where they count: in the terms that
// make up the output.  (Weights e^(s_t - max s) times b would lose their last bits in
// fp16 wherever b is far below the row's largest.)
// Blocks whose values are all but zero would leave their tokens no weight, though the
// softmax counts them in l: lb is therefore held above R - 100 (R the largest lb of the
// stream so far) and above -100, and what is cut off, f = 2^(log2 b - lb), multiplies
// the weights that enter O (1 but for such blocks).  In 32 bits that is far enough: m is at most the
// row's largest score plus R, so a token that has 2^-24 or more of the softmax keeps w_t of 2^-124 or more,
// and l, no more than 2^100 a token, stays above 2^-R.  (A smaller range, 24, took a row's own values
// to zero in fp16 wherever a block that the row all but ignores had a scale 2^40 times theirs.)
// When R rises behind blocks that were held at -100, l is multiplied by 2^(m - m') of 2^-126 at least
// as long as R is no more than 26.
//
// Queries enter as fp16.  A bf16 query row is multiplied by the power of two that brings
// its largest value between 2^14 and 2^15, which no finite row overflows and which
// keeps every value down to 2^-29 of the largest exact; the factor's inverse goes into
// the scores.
//
// Bound by HBM: 361 us for 256 sequences of 1024 to 8192 tokens, 64 query and 8 KV heads of 128 (6.7
// TB/s; issue 34 %), 277 us for 4 of 24576 to 32768 with 64 KV heads (6.8 TB/s).
#pragma once

#include "bs8.cuh"
#include "decode_common.cuh"
#include "decode_tok.cuh"

namespace pa {

// A ring stage: UB consecutive pieces of one (sequence, KV head) pair, 32 tokens.
template <int D_, int BS_>
struct GeomB8 {
    static constexpr int D = D_;
    static constexpr int BS = BS_;
    static constexpr int PIECE_BYTES = bs8_piece_bytes(BS, D);   // 32 modulo 128
    static constexpr int UB = 32 / BS;
    // with two pieces per stage the second starts 64 bytes off a 128-byte line, so that
    // the value rows of both that one load reads fall in different banks
    static constexpr int PIECE_PAD = UB == 2 ? PIECE_BYTES + 32 : PIECE_BYTES;
    static constexpr int STAGE_BYTES = (UB * PIECE_PAD + 127) / 128 * 128;
    static constexpr int COPY_BYTES = UB * PIECE_BYTES;
    static constexpr int KD = D / 16;
    static constexpr int TOK = 32;
    __host__ __device__ static constexpr int poff(int u) { return u * PIECE_PAD; }
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(BS == 16 || BS == 32, "block_size");
    static_assert(UB == 1 || PIECE_PAD % 128 == 64, "bank spread of the second piece");
};

constexpr float BS8_LB_RANGE = 100.f, BS8_LB_FLOOR = -100.f;   // of lb, see above

// Running state of one warp: as WarpAccT (m and l as above), and R.  Row e >> 1 of
// m-tile mt is dimension D / 8 g + 2 mt + (e >> 1): a lane holds D / 8 consecutive ones.
template <int D, int NH>
struct WarpAccB8 {
    float m[NH][2], l[NH][2], R;
    float o[D / 16][NH][4];

    __device__ __forceinline__ void reset() {
        R = -INFINITY;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[nh][c] = -INFINITY;
                l[nh][c] = 0.f;
            }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nh][e] = 0.f;
    }
};

// The power of two that multiplies a bf16 row whose largest absolute value has the
// exponent field `eb`, and (second) its inverse.  Rows that are not finite are left alone.
__device__ __forceinline__ float2 row_factor(int eb) {
    if (eb == 255) return make_float2(1.f, 1.f);
    const int up = min(254, 268 - eb);                       // field of 2^(14 - (eb - 127)), at most 2^127
    return make_float2(__uint_as_float((uint32_t)up << 23),
                       up == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - up) << 23));
}

// Q fragments (load_q_frags8) to fp16; qf[nh][c]: what turns the MMA's sums for the lane's
// head 8 nh + 2 t4 + c into scores in log2 units, before the block's scale.
template <bool BF16, int KD, int NH>
__device__ __forceinline__ void normalise_q(uint32_t (&qa)[KD][4], float (&qf)[NH][2], float scale_log2, int lane) {
    if constexpr (!BF16) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) qf[nh][0] = qf[nh][1] = scale_log2;
    } else {
        const int t4 = lane & 3;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            uint32_t top = 0;
#pragma unroll
            for (int kk = 0; kk < KD; ++kk)
                top = __vmaxu2(top, __vmaxu2(qa[kk][nh] & 0x7fff7fffu, qa[kk][2 + nh] & 0x7fff7fffu));
            top = max(top & 0xffffu, top >> 16);             // dims of head 8 nh + g; four lanes hold them all
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float2 f = row_factor((int)(top >> 7));
#pragma unroll
            for (int kk = 0; kk < KD; ++kk)
#pragma unroll
                for (int i = nh; i < 4; i += 2)
                    qa[kk][i] = pack2<false>(lo_of<true>(qa[kk][i]) * f.x, hi_of<true>(qa[kk][i]) * f.x);
            const float back = f.y * scale_log2;
#pragma unroll
            for (int c = 0; c < 2; ++c) qf[nh][c] = __shfl_sync(0xffffffffu, back, (2 * t4 + c) * 4);
        }
    }
}

// Folds one 32-token stage in (piece u at poff(u); pieces from valid / BS on were not
// copied).  Masked tokens may hold any byte: their scores are -inf and their value
// operands zero (MASK: a partial stage).  False if a scale is none.
template <class Gm, int NH, bool E5M2, bool MASK>
__device__ __forceinline__ bool consume_stage_b8_impl(uint32_t kb, int valid, const uint32_t (&qa)[Gm::KD][4],
                                                      const float (&qf)[NH][2], WarpAccB8<Gm::D, NH>& acc, int lane) {
    constexpr int BS = Gm::BS, D = Gm::D;
    const int g = lane >> 2;
    const int t4 = lane & 3;
    // this lane's score rows are stage tokens tb + 4 mt + 2 h, all in one piece
    const int tb = 8 * (g >> 1) + (g & 1);
    float ka, lb;                                            // the lane's piece: key scale, log2 of the value scale
    bool fine;
    {
        uint32_t a0, b0;
        lds64(kb, a0, b0);
        fine = a0 < 0x7f800000u && b0 < 0x7f800000u;
        const float l0 = fmaxf(__log2f(__uint_as_float(b0)), -126.f);
        ka = __uint_as_float(a0);
        lb = l0;
        acc.R = fmaxf(acc.R, l0);
        if (Gm::UB == 2 && (!MASK || valid > BS)) {
            uint32_t a1, b1;
            lds64(kb + Gm::poff(1), a1, b1);
            fine = fine && a1 < 0x7f800000u && b1 < 0x7f800000u;
            const float l1 = fmaxf(__log2f(__uint_as_float(b1)), -126.f);
            acc.R = fmaxf(acc.R, l1);
            if (g >= 4) {
                ka = __uint_as_float(a1);
                lb = l1;
            }
        }
    }
    const float held = fmaxf(lb, fmaxf(acc.R - BS8_LB_RANGE, BS8_LB_FLOOR));
    const float f = ex2(lb - held), back = ex2(-held);

    float sc[2][NH][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nh][e] = 0.f;
        const int r0 = tb + 4 * mt, r1 = r0 + 2;             // rows of the same piece
        const uint32_t b = kb + Gm::poff(r0 / BS);
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {                // 16-byte parts D / 64 t4 + hf of rows g and g + 8
            uint32_t w0[4], w1[4];
            lds128(b + bs8_key<D>(r0 % BS, D / 64 * t4 + hf), w0);
            lds128(b + bs8_key<D>(r1 % BS, D / 64 * t4 + hf), w1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int kk = 4 * hf + k;
                const uint32_t a0 = fp8x2_to_f16x2<E5M2>((uint16_t)(w0[k] & 0xffffu));
                const uint32_t a2 = fp8x2_to_f16x2<E5M2>((uint16_t)(w0[k] >> 16));
                const uint32_t a1 = fp8x2_to_f16x2<E5M2>((uint16_t)(w1[k] & 0xffffu));
                const uint32_t a3 = fp8x2_to_f16x2<E5M2>((uint16_t)(w1[k] >> 16));
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma16816<false>(sc[mt][nh], a0, a1, a2, a3, qa[kk][nh], qa[kk][2 + nh]);
            }
        }
    }
    // x_t; the running maximum over the stage
    float alpha[NH][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float by = ka * qf[nh][c];
            float mx = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float& x = sc[mt][nh][2 * h + c];
                    x = fmaf(x, by, held);
                    if (MASK && tb + 4 * mt + 2 * h >= valid) x = -INFINITY;
                    mx = fmaxf(mx, x);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(acc.m[nh][c], mx);
            alpha[nh][c] = ex2(acc.m[nh][c] - m_new);
            acc.m[nh][c] = m_new;
            acc.l[nh][c] *= alpha[nh][c];
        }
    uint32_t pb[2][NH][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float pe = ex2(sc[mt][nh][e] - acc.m[nh][e & 1]);
                acc.l[nh][e & 1] = fmaf(pe, back, acc.l[nh][e & 1]);
                w[e] = pe * f;
            }
            pb[mt][nh][0] = movm_trans(pack2<false>(w[0], w[1]));
            pb[mt][nh][1] = movm_trans(pack2<false>(w[2], w[3]));
        }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        if (__any_sync(0xffffffffu, alpha[nh][0] != 1.f || alpha[nh][1] != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < Gm::KD; ++mt) {
                acc.o[mt][nh][0] *= alpha[nh][0];
                acc.o[mt][nh][1] *= alpha[nh][1];
                acc.o[mt][nh][2] *= alpha[nh][0];
                acc.o[mt][nh][3] *= alpha[nh][1];
            }
        }
    }
    // Values: lane (g, t4) reads dims D / 8 g .. of the stage tokens 8 t4 .. 8 t4 + 7 (rows
    // of tokens) and pairs neighbouring tokens' bytes: bytes i of tokens j and j + 1 are the
    // operand of dimension i.
    const int t0 = (8 * t4) % BS;
    const uint32_t vb = kb + Gm::poff((8 * t4) / BS);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
        constexpr int W = D / 32;                            // words of a lane's dims
        uint32_t v[4][W];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = t0 + 4 * kt + j;
            if constexpr (D == 128) {
                lds128(vb + bs8_value<BS, D>(r, g), v[j]);
            } else {
                lds64(vb + bs8_value<BS, D>(r, g >> 1) + 8 * (g & 1), v[j][0], v[j][1]);
            }
        }
        const int t = 8 * t4 + 4 * kt;
#pragma unroll
        for (int mt = 0; mt < Gm::KD; ++mt) {
            const uint32_t sel = mt & 1 ? 0x7362u : 0x5140u; // bytes 2, 3 or 0, 1 of a word
            const uint32_t x = __byte_perm(v[0][mt / 2], v[1][mt / 2], sel), y = __byte_perm(v[2][mt / 2], v[3][mt / 2], sel);
            uint32_t a0 = fp8x2_to_f16x2<E5M2>((uint16_t)(x & 0xffffu)), a1 = fp8x2_to_f16x2<E5M2>((uint16_t)(x >> 16));
            uint32_t a2 = fp8x2_to_f16x2<E5M2>((uint16_t)(y & 0xffffu)), a3 = fp8x2_to_f16x2<E5M2>((uint16_t)(y >> 16));
            if (MASK) {
                a0 = keep_pair(a0, t, valid);
                a1 = keep_pair(a1, t, valid);
                a2 = keep_pair(a2, t + 2, valid);
                a3 = keep_pair(a3, t + 2, valid);
            }
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma16816<false>(acc.o[mt][nh], a0, a1, a2, a3, pb[kt][nh][0], pb[kt][nh][1]);
        }
    }
    return fine;
}

template <class Gm, int NH, bool E5M2>
__device__ __forceinline__ bool consume_stage_b8(uint32_t kb, int valid, const uint32_t (&qa)[Gm::KD][4],
                                                 const float (&qf)[NH][2], WarpAccB8<Gm::D, NH>& acc, int lane) {
    return valid < 32 ? consume_stage_b8_impl<Gm, NH, E5M2, true>(kb, valid, qa, qf, acc, lane)
                      : consume_stage_b8_impl<Gm, NH, E5M2, false>(kb, valid, qa, qf, acc, lane);
}

// A finished segment: the output rows at orow, or the partial state at prow (rows of D + 4
// floats: o, m, l); acc.l is summed over the lanes.
template <int D, int NH, bool BF16>
__device__ __forceinline__ void store_b8(const WarpAccB8<D, NH>& acc, bool complete, bool poisoned, int G,
                                         uint16_t* orow, float* prow, int lane) {
    const int g = lane >> 2, t4 = lane & 3;
    const float qnan = __int_as_float(0x7fc00000);
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int head = 8 * nh + 2 * t4 + c;
            if (head >= G) continue;
            const float by = poisoned ? qnan : complete ? 1.f / acc.l[nh][c] : 1.f;
            float x[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) x[i] = acc.o[i / 2][nh][2 * (i & 1) + c] * by;
            if (complete) {
                uint4* at = reinterpret_cast<uint4*>(orow + head * D + D / 8 * g);
#pragma unroll
                for (int i = 0; i < D / 8; i += 8)
                    at[i / 8] = make_uint4(pack2<BF16>(x[i], x[i + 1]), pack2<BF16>(x[i + 2], x[i + 3]),
                                           pack2<BF16>(x[i + 4], x[i + 5]), pack2<BF16>(x[i + 6], x[i + 7]));
            } else {
                float* at = prow + head * (D + 4);
#pragma unroll
                for (int i = 0; i < D / 8; i += 4)
                    *reinterpret_cast<float4*>(at + D / 8 * g + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                if (g == 0) {
                    at[D] = acc.m[nh][c];
                    at[D + 1] = acc.l[nh][c];
                }
            }
        }
}

}  // namespace pa
