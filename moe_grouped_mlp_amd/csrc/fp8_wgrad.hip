// Launch of the block-scaled FP8 weight gradient (fp8_gemm_kernel.h).
#include "fp8_gemm_kernel.h"

namespace moe {

hipError_t launch_fp8_wgrad(const Fp8Args& g, bool f32, bool wide, int groups, hipStream_t s) {
  auto go = [&](auto kernel) { kernel<<<g.grid, kFp8Threads, 0, s>>>(g); };
  if (f32) groups == 1 ? go(fp8_gemm_kernel<1, true, true, true>) : go(fp8_gemm_kernel<2, true, true, true>);
  else if (wide) groups == 1 ? go(fp8_gemm_kernel<1, true, false, true>) : go(fp8_gemm_kernel<2, true, false, true>);
  else if (groups == 1) go(fp8_gemm_kernel<1, true, false, false>);
  else groups == 2 ? go(fp8_gemm_kernel<2, true, false, false>) : go(fp8_gemm_kernel<4, true, false, false>);
  return hipGetLastError();
}

}  // namespace moe
