// gemm_fp4_bf16_32.hip -- products of BF16 rows with 4-bit weights in groups of 32.
#include "gemm_fp4.hpp"

namespace rx {

hipError_t launch_fp4_bf16_32(const GemmFp4Args& a, hipStream_t s) { return launch_fp4<1, 32>(a, s); }

}  // namespace rx
