// Launch interface of the fused norm + rotary + append kernel (rope_ops.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace pa {

struct RopeArgs {
    const uint16_t* q;         // token t, head h at q + t * q_stride + h * D (k, v likewise)
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;   // elements between tokens
    const int32_t* positions;  // [T]
    const int64_t* slots;      // [T]
    const float* inv_freq;     // [rot / 2]
    const uint16_t* q_weight;  // [D] or null: queries are not normed
    const uint16_t* k_weight;  // [D] or null: keys are not normed
    uint16_t* q_out;           // [T][Hq][D]
    uint16_t* k_pool;          // [NB][Hkv][BS][D]
    uint16_t* v_pool;
    uint32_t* err;
    long long num_slots;       // NB * BS
    int32_t T, Hq, Hkv, D, BS;
    int32_t rot;               // first rot values of a head are rotated (multiple of 16, 0: none)
    int32_t interleaved;       // pairs (2j, 2j + 1) instead of (j, j + rot / 2)
    int32_t splits;            // warps sharing one token's rows
    float scale;               // multiplies cos and sin
    float eps;
};

cudaError_t rope_append_launch(RopeArgs a, bool bf16, cudaStream_t stream, int sms);

}  // namespace pa
