// Instantiations of the two-tile tree attention kernel: bf16.
#include "tree_wide_kernel.cuh"

namespace pa {

void tree_wide_table_bf16(MultiKernelInfo (&t)[2][2]) {
    t[0][0] = tree_wide_info<WideTraits<64, 16, true>>();
    t[0][1] = tree_wide_info<WideTraits<64, 32, true>>();
    t[1][0] = tree_wide_info<WideTraits<128, 16, true>>();
    t[1][1] = tree_wide_info<WideTraits<128, 32, true>>();
}

}  // namespace pa
