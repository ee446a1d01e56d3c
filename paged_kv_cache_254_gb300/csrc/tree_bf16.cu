// Instantiations of the tree attention kernels: bf16.
#include "multi_kernel.cuh"

namespace pa {

void tree_table_bf16(MultiKernelInfo (&t)[2][2]) {
    t[0][0] = multi_info<MultiTraits<64, 16, 1, true, true>>();
    t[0][1] = multi_info<MultiTraits<64, 32, 1, true, true>>();
    t[1][0] = multi_info<MultiTraits<128, 16, 1, true, true>>();
    t[1][1] = multi_info<MultiTraits<128, 32, 1, true, true>>();
}

}  // namespace pa
