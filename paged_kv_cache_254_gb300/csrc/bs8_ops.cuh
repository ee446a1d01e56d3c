// Launch interface of the block-scaled 8-bit cache's writes and conversions (bs8_ops.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace pa {

struct AppendBs8Args {
    const uint16_t *k, *v;          // [T] rows of [Hkv][D], k_stride / v_stride elements apart
    int64_t k_stride, v_stride;
    const int32_t* q_start;         // [N + 1]
    const int32_t* block_tables;    // [N][MB]
    const int32_t* context_lens;    // [N], the new tokens included
    uint8_t* pool;
    uint32_t* err;
    int32_t N, T, max_new, span;    // span: blocks that max_new tokens can lie in
    int32_t Hkv, NB, MB;
};

struct ConvertBs8Args {
    const int32_t* pairs;           // [n][2] (source block, destination block)
    uint16_t *k, *v;                // the 16-bit pools
    uint8_t* pool;
    uint32_t* err;
    int32_t n, Hkv, NB8, NB16;         // blocks of the 8-bit pool, of the 16-bit pools
};

// Kernels by type: the values' 16-bit type, the codes' format, block size and head_dim.
struct Bs8Kind {
    bool bf16, e5m2, bs32, d128;
};

cudaError_t append_bs8_launch(const AppendBs8Args& a, Bs8Kind kind, cudaStream_t stream);
cudaError_t pack_bs8_launch(const ConvertBs8Args& a, Bs8Kind kind, cudaStream_t stream);
cudaError_t unpack_bs8_launch(const ConvertBs8Args& a, Bs8Kind kind, cudaStream_t stream);

}  // namespace pa
