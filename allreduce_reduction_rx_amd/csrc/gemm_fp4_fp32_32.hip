// gemm_fp4_fp32_32.hip -- products of FP32 rows with 4-bit weights in groups of 32.
#include "gemm_fp4.hpp"

namespace rx {

hipError_t launch_fp4_fp32_32(const GemmFp4Args& a, hipStream_t s) { return launch_fp4<0, 32>(a, s); }

}  // namespace rx
