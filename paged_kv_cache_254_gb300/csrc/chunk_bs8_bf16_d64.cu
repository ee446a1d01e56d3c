// Instantiations of the chunk kernel over the 8-bit cache with a scale per block and head, bf16 queries, head_dim 64.
#include "chunk_bs8_kernel.cuh"

namespace pa {

void chunk_bs8_table_bf16_d64(MultiKernelInfo (&t)[2][2][2]) {
    t[0][0][0] = chunk_bs8_info<ChunkTraits<64, 16, true, false, true>>();
    t[0][0][1] = chunk_bs8_info<ChunkTraits<64, 16, true, false, false>>();
    t[0][1][0] = chunk_bs8_info<ChunkTraits<64, 32, true, false, true>>();
    t[0][1][1] = chunk_bs8_info<ChunkTraits<64, 32, true, false, false>>();
    t[1][0][0] = chunk_bs8_info<ChunkTraits<64, 16, true, true, true>>();
    t[1][0][1] = chunk_bs8_info<ChunkTraits<64, 16, true, true, false>>();
    t[1][1][0] = chunk_bs8_info<ChunkTraits<64, 32, true, true, true>>();
    t[1][1][1] = chunk_bs8_info<ChunkTraits<64, 32, true, true, false>>();
}

}  // namespace pa
