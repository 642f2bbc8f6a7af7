// Launch of the tiled block-scaled FP8 product (fp8_gemm_kernel.h).
#include "fp8_gemm_kernel.h"

namespace moe {

hipError_t launch_fp8_gemm(const Fp8Args& g, bool f32, int grid, hipStream_t s) {
  if (f32) fp8_gemm_kernel<2, false, true><<<grid, kFp8Threads, 0, s>>>(g);
  else fp8_gemm_kernel<4, false, false><<<grid, kFp8Threads, 0, s>>>(g);
  if (hipError_t e = hipGetLastError()) return e;
  if (g.part) {
    if (f32) fp8_join_kernel<2, true><<<grid, kFp8Threads, 0, s>>>(g, grid);
    else fp8_join_kernel<4, false><<<grid, kFp8Threads, 0, s>>>(g, grid);
  }
  return hipGetLastError();
}

}  // namespace moe
