// Block-scaled products of an e5m2 operand A and an e5m2 operand B.
#include "tg_fp8.hpp"

namespace tg {

const Fp8Kernel* fp8_kernels_e5m2_e5m2() { return fp8_kernel_table<FMT_E5M2, FMT_E5M2>(); }

}  // namespace tg
