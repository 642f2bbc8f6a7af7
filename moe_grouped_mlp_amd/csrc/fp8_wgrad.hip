// Launch of the block-scaled FP8 weight gradient (fp8_gemm_kernel.h).
#include "fp8_gemm_kernel.h"

namespace moe {

hipError_t launch_fp8_wgrad(const Fp8Args& g, bool f32, int grid, hipStream_t s) {
  if (f32) fp8_gemm_kernel<2, true, true><<<grid, kFp8Threads, 0, s>>>(g);
  else fp8_gemm_kernel<4, true, false><<<grid, kFp8Threads, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace moe
