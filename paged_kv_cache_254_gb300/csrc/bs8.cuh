// Layout of the 8-bit cache with a scale for each block and KV head, shared by
// the kernels that write, copy and read it.
//
// A (block, KV head) piece is one run of 32 + 2 * BS * D bytes: the keys' scale and the
// values' scale (fp32), 24 spare bytes, BS key rows of D codes, BS value rows of D
// codes.  The scales travel with the codes, so one bulk copy fetches both (the first
// half of a piece, keys and scales, another) and a block copy moves both; the spare
// bytes keep pieces on 32-byte sectors.
//
// The 16-byte parts of a row are permuted so that a plain copy of the piece is read
// from shared memory without bank conflicts by the decode's fragment loads:
//  * keys: lanes read parts of rows r and r + 1 (r a multiple of 4) at once.  Rows of
//    128 bytes: part c of row r at c ^ (r & 7).  Rows of 64 bytes need nothing, two
//    of them are one 128-byte line.
//  * values (rows of tokens too, so that an append writes whole rows; the decode
//    transposes them in registers): lanes read the same parts of rows r, r + 8, r + 16,
//    r + 24 at once.  128 bytes: part c at c ^ 2 (r / 8 & 3); 64 bytes: c ^ 2 (r / 8 & 1),
//    and rows from 16 on change places in pairs.
#pragma once

#include <cstdint>

#include "../../include/pa.h"
#include "ptx.cuh"

namespace pa {

constexpr int BS8_HEAD = 32;                     // scales and spare bytes of a piece

__host__ __device__ constexpr int bs8_piece_bytes(int BS, int D) { return BS8_HEAD + 2 * BS * D; }

// Byte offsets inside a piece of the 16-byte part `c` of key row r and value row r.
template <int D>
__host__ __device__ constexpr int bs8_key(int r, int c) {
    return BS8_HEAD + r * D + 16 * (D == 128 ? c ^ (r & 7) : c);
}
template <int BS, int D>
__host__ __device__ constexpr int bs8_value(int r, int c) {
    return BS8_HEAD + BS * D + (D == 128 ? r * D + 16 * (c ^ (2 * ((r >> 3) & 3)))
                                         : (r ^ ((r >> 4) & 1)) * D + 16 * (c ^ (2 * ((r >> 3) & 1))));
}

// Is x a scale: finite and not negative?
__device__ __forceinline__ bool bs8_is_scale(float x) { return __float_as_uint(x) < 0x7f800000u; }

// Does a packed 16-bit pair of absolute values hold one that is not finite?
template <bool BF16>
__device__ __forceinline__ uint32_t pair_not_finite(uint32_t abs2) {
    return (abs2 + (BF16 ? 0x00800080u : 0x04000400u)) & 0x80008000u;   // the exponent's carry
}

template <bool BF16>
__device__ __forceinline__ float widen16(uint32_t bits) {
    if constexpr (BF16) return __uint_as_float(bits << 16);
    return lo_of<false>(bits);
}

}  // namespace pa
