// Instantiations of the paged decode kernel over the 8-bit cache with a scale per block and head, bf16 queries, head_dim 128.
#include "decode_kernel.cuh"

namespace pa {

void decode_bs8_table_bf16_d128(DecodeKernelInfo (&t)[2][2][2]) {
    t[0][0][0] = decode_info<DecodeTraits<128, 16, 8, true, 4>>();
    t[0][0][1] = decode_info<DecodeTraits<128, 16, 16, true, 4>>();
    t[0][1][0] = decode_info<DecodeTraits<128, 32, 8, true, 4>>();
    t[0][1][1] = decode_info<DecodeTraits<128, 32, 16, true, 4>>();
    t[1][0][0] = decode_info<DecodeTraits<128, 16, 8, true, 5>>();
    t[1][0][1] = decode_info<DecodeTraits<128, 16, 16, true, 5>>();
    t[1][1][0] = decode_info<DecodeTraits<128, 32, 8, true, 5>>();
    t[1][1][1] = decode_info<DecodeTraits<128, 32, 16, true, 5>>();
}

}  // namespace pa
