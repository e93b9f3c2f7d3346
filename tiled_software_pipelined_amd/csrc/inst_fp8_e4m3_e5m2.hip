// Block-scaled products of an e4m3 operand A and an e5m2 operand B.
#include "tg_fp8.hpp"

namespace tg {

const Fp8Kernel* fp8_kernels_e4m3_e5m2() { return fp8_kernel_table<FMT_E4M3, FMT_E5M2>(); }

}  // namespace tg
