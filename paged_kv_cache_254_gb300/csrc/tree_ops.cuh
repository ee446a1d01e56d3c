// Launch interface of the tree bookkeeping kernels (tree_ops.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace pa {

struct VerifyArgs {
    const int32_t* q_start;       // [N + 1]
    const uint64_t* masks;        // [T]
    const int64_t* draft;         // [T]
    const int64_t* target;        // [T]
    const int32_t* context_lens;  // [N]
    int32_t* path;                // [N][P]
    int32_t* accepted;            // [N]
    int64_t* next;                // [N]
    int32_t* new_lens;            // [N]
    uint32_t* err;
    int32_t N, P, total_q;
};

struct KeepArgs {
    const int32_t* path;          // [N][P]
    const int32_t* q_start;       // [N + 1]
    const int32_t* context_lens;  // [N]
    const int32_t* block_tables;  // [N][MB]
    uint4* k_pool;
    uint4* v_pool;
    uint32_t* err;
    int32_t N, P, Hkv, BS, NB, MB;
    int32_t vec_per_row;          // head_dim * 2 / 16
};

cudaError_t tree_verify_launch(const VerifyArgs& a, cudaStream_t stream);
cudaError_t keep_launch(const KeepArgs& a, cudaStream_t stream);

}  // namespace pa
