// Block-scaled products of an e4m3 operand A and an e4m3 operand B.
#include "tg_fp8.hpp"

namespace tg {

const Fp8Kernel* fp8_kernels_e4m3_e4m3() { return fp8_kernel_table<FMT_E4M3, FMT_E4M3>(); }

}  // namespace tg
