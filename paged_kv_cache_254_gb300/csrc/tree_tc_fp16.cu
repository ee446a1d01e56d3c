// Instantiations of the tensor-core tree attention kernel: fp16.
#include "multi_tc_kernel.cuh"

namespace pa {

void tree_tc_table_fp16(MultiKernelInfo (&t)[2][2]) {
    t[0][0] = multi_tc_info<TcTraits<64, 16, false, true>>();
    t[0][1] = multi_tc_info<TcTraits<64, 32, false, true>>();
    t[1][0] = multi_tc_info<TcTraits<128, 16, false, true>>();
    t[1][1] = multi_tc_info<TcTraits<128, 32, false, true>>();
}

}  // namespace pa
