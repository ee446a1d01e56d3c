// Instantiations of the tensor-core tree attention kernel: fp16.
#include "tree_tc_kernel.cuh"

namespace pa {

void tree_tc_table_fp16(MultiKernelInfo (&t)[2][2]) {
    t[0][0] = tree_tc_info<TreeTcTraits<64, 16, false>>();
    t[0][1] = tree_tc_info<TreeTcTraits<64, 32, false>>();
    t[1][0] = tree_tc_info<TreeTcTraits<128, 16, false>>();
    t[1][1] = tree_tc_info<TreeTcTraits<128, 32, false>>();
}

}  // namespace pa
