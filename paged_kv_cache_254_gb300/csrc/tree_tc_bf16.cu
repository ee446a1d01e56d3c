// Instantiations of the tensor-core tree attention kernel: bf16.
#include "multi_tc_kernel.cuh"

namespace pa {

void tree_tc_table_bf16(MultiKernelInfo (&t)[2][2]) {
    t[0][0] = multi_tc_info<TcTraits<64, 16, true, true>>();
    t[0][1] = multi_tc_info<TcTraits<64, 32, true, true>>();
    t[1][0] = multi_tc_info<TcTraits<128, 16, true, true>>();
    t[1][1] = multi_tc_info<TcTraits<128, 32, true, true>>();
}

}  // namespace pa
